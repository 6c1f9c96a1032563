"""Long chunks over 8-bit pages: their results are as exact as those of shorter ones."""
import pytest
import torch

from fibonacci_spaced_sparse_gb300 import api
from _fp8 import Cache8
from _fp8_exact import forward64, fp32_bounds, halves_bound, split_bound, workspace
from _paged import within

pytestmark = pytest.mark.gpu

KW = dict(alpha=0.87, rungs=api.FIBONACCI_BASE)


@pytest.mark.parametrize("lens,page,block,W", [([(7001, 0)], 64, 16, 12), ([(3803, 70), (0, 9), (3302, 0), (1, 1200), (133, 986)], 16, 8, 12),
                                               ([(230, 40 * s) for s in range(32)], 256, 64, 5), ([(1024, 0)] * 7, 64, 16, 28),
                                               ([(7100, 4000)], 32, 32, 0)])
def test_probabilities_are_not_rounded_to_bf16(lens, page, block, W):
    """Copied rows are exact where scales are powers of two, and a probability keeps 16
    bits, so that rounding the output once is nearly all of its error.  (The 32 chunks of
    230 are not copied: what they reach is more than three times their own rows.)"""
    cache = Cache8(lens, page, "bf16", block, seed=len(lens) + W)
    o, lse = api.sfa_paged_forward_fp8(cache.q.cuda(), *cache.pages8(), *cache.meta(), W=W, **KW)
    ref = forward64(cache, W=W, **KW)
    bo, bl = fp32_bounds(ref, "bf16")
    used = ref[0].shape[0]
    copied = workspace(cache, W, **KW) > 0
    assert copied == (len(lens) < 32)
    within(o[:used], ref[0], bo + (split_bound if copied else halves_bound)(ref), "o")
    within(lse[:used], ref[1], bl, "lse")
    # the norm of the error: that of rounding to bf16 alone, uniform in a half step, is 1.66e-3
    off = (o[:used].double().cpu() - ref[0]).norm() / ref[0].norm()
    assert float(off) < 1.75e-3


@pytest.mark.parametrize("lens,page,W", [([(3803, 70), (0, 9), (3302, 0), (1, 1200), (133, 986)], 8, 12), ([(7001, 37), (160, 0)], 32, 29),
                                         ([(40, 30)] * 180, 64, 12), ([(6992, 0)], 64, 12)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_calls_that_copy_nothing(lens, page, W, dtype):
    """Pages of 8 rows, wide windows, chunks too short for what they reach and one token row too
    few: each kernel against its own bound."""
    cache = Cache8(lens, page, dtype, 8, seed=page + W)
    assert dtype == "f32" or workspace(cache, W, **KW) == 0
    o, lse = api.sfa_paged_forward_fp8(cache.q.cuda(), *cache.pages8(), *cache.meta(), W=W, **KW)
    ref = forward64(cache, W=W, **KW)
    bo, bl = fp32_bounds(ref, dtype)
    used = ref[0].shape[0]
    within(o[:used], ref[0], bo + (halves_bound(ref) if dtype == "bf16" and W <= 28 else 0), "o")
    within(lse[:used], ref[1], bl, "lse")
