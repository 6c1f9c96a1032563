"""Scores far below zero: the softmax of rows that all score about -1e32 is as
ordinary as any other, in every kernel of the call."""
import math

import pytest
import torch

from fibonacci_spaced_sparse_gb300 import api
from _paged import Cache, D, DT, HALF_STEP, HKV, HQ, rung_list

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("exponent", [49, 51, 56])
@pytest.mark.parametrize("lens", [[(1, 40), (2, 0)], [(1, 40)] * 640, [(700, 30), (1, 5)], [(4200, 30), (1, 5)]])
def test_equal_scores_far_below_zero(lens, exponent, dtype):
    """Queries 2^e, keys -2^e: every score is -64 2^(2e) / 8, a power of two that
    fp32 holds, so every entry of a token has the same weight: o is the mean of
    the value rows, lse the score plus the logarithm of their number.

    Bounds.  Rungs at whole distances, so a score is exact but for the scale (two
    roundings); all entries of a head go through the same operations.  o: the
    sum's and the quotient's roundings (40 u), the approximate exponential and
    reciprocal (2^-20), on the tensor cores the probability's rounding to bf16
    (2^-8 of it), and one rounding of the result.  lse: 2^-20 of its size."""
    cache = Cache(lens, 16, dtype, seed=exponent)
    cache.q.fill_(2.0 ** exponent)
    for x in cache.k:
        x.fill_(-2.0 ** exponent)
    score = -8.0 * 2.0 ** (2 * exponent)
    kp, vp = cache.pages()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    W, rungs = 12, (20.0, 33.0)
    o, lse = api.sfa_paged_forward(cache.q.cuda(), kp, vp, *cache.meta(), alpha=1.0, W=W, rungs=rungs, status=status)
    assert api.sfa_read_status(status) == 0
    o, lse = o.double().cpu(), lse.double().cpu()
    probability = 2.0 ** -8 if dtype == "bf16" else 0.0
    for t, s, i in cache.tokens():
        rows = [i - d for d in range(min(W, i) + 1)] + [i - n for n, _, c in rung_list(1.0, W, rungs) if i >= c]
        v = cache.v[s][rows].double().repeat_interleave(HQ // HKV, 1)
        want, size = v.mean(0), v.abs().mean(0)
        assert bool(((o[t] - want).abs() <= (probability + 2.0 ** -18) * size + HALF_STEP[dtype] * want.abs() + 1e-30).all()), (t, i)
        target = score + math.log(len(rows))
        assert bool(((lse[t] - target).abs() <= 2.0 ** -20 * abs(target)).all()), (t, i, lse[t], target)
