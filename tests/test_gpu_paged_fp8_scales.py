"""The 8-bit attention with value scales that differ by any factor within a query's rows:
the size of a block's scale says nothing about the rows that it holds."""
import pytest
import torch

from fibonacci_spaced_sparse_gb300 import api
from _fp8 import FP8, Cache8
from _fp8_exact import forward64, fp32_bounds, halves_bound
from _paged import D, HQ, HKV, within

pytestmark = pytest.mark.gpu

KW = dict(alpha=0.87, W=12, rungs=api.FIBONACCI_BASE)


def _cache(lens, power, code, dtype="bf16", every=5):
    """Every `every`-th block of rows has a value scale 2^power of what it would be, and
    codes that are all `code`."""
    cache = Cache8(lens, 16, dtype, 8, seed=7 + power)
    for s in range(len(lens)):
        big = (torch.arange(cache.v[s].shape[0]) // 8) % every == 2
        if not len(big):
            continue
        cache.scales[1][s][big] *= 2.0 ** power
        cache.codes[1][s][big] = torch.full((int(big.sum()), HKV, D), code).to(FP8)
        cache.v[s] = cache.codes[1][s].float() * cache.scales[1][s][..., None]
    return cache


def _check(cache, **kw):
    kw = {**KW, **kw}
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = api.sfa_paged_forward_fp8(cache.q.cuda(), *cache.pages8(), *cache.meta(), status=status, **kw)
    assert api.sfa_read_status(status) == 0
    ref = forward64(cache, **kw)
    bo, bl = fp32_bounds(ref, cache.dtype)
    used = ref[0].shape[0]
    within(o[:used], ref[0], bo + (halves_bound(ref) if cache.dtype == "bf16" else 0), "o")
    within(lse[:used], ref[1], bl, "lse")


@pytest.mark.parametrize("code", [0.0, 2.0 ** -9, -0.5, 448.0])
@pytest.mark.parametrize("power", [8, 16, 20, 23, 26, 40, 90])
def test_a_block_with_a_large_scale(power, code):
    """Short chunks in both forms of the tensor-core kernel (640 and 4000 tokens)."""
    for lens in ([(640, 300)], [(3, 40)] * 30 + [(400, 0), (600, 1000)], [(2000, 100), (2000, 0)]):
        _check(_cache(lens, power, code))


@pytest.mark.parametrize("power", [-20, -60, -90])
def test_a_block_with_a_small_scale(power):
    _check(_cache([(640, 300), (50, 3)], power, 448.0))
    _check(_cache([(640, 300), (50, 3)], power, 448.0, every=3), scale=0.5)


def test_a_sharp_softmax_on_rows_of_zeros():
    """The row that takes nearly all of the softmax holds zeros, so the output is what
    the others make of the rest of it."""
    cache = _cache([(700, 40)], 0, 0.0)
    cache.q = (4.0 * cache.q.float()).bfloat16()
    _check(cache, scale=0.5)


@pytest.mark.parametrize("n", [1, 40, 640, 7100])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_same_in_every_kernel(n, dtype):
    if dtype == "f32" and n > 5000:
        pytest.skip("no kernel of its own")
    _check(_cache([(n, 400)], 26, 0.0, dtype))


def test_values_that_are_all_zero():
    """No value at all: zeros, and the sums of the softmax as ever."""
    cache = Cache8([(640, 300), (3, 5)], 16, "bf16", 16, seed=3)
    for s in range(2):
        cache.codes[1][s] = torch.zeros_like(cache.codes[1][s].float()).to(FP8)
        cache.scales[1][s][:] = 2.0 ** -100
        cache.v[s] = torch.zeros_like(cache.v[s])
    _check(cache)
