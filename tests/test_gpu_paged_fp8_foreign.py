"""The 8-bit attention over caches whose scales are no powers of two, as a cache that
was made elsewhere has them: as exact for long chunks as for short ones."""
import pytest
import torch

from fibonacci_spaced_sparse_gb300 import api
from _fp8 import Cache8, NAN_CODE
from _fp8_exact import forward64, fp32_bounds, halves_bound, split_bound, workspace
from _paged import D, HKV, rung_list, within

pytestmark = pytest.mark.gpu

FIB = api.FIBONACCI_BASE
MANY_RUNGS = tuple(13.0 + 3.7 * k for k in range(30))


def _check(cache, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = api.sfa_paged_forward_fp8(cache.q.cuda(), *cache.pages8(), *cache.meta(), status=status, **kw)
    assert api.sfa_read_status(status) == 0
    ref = forward64(cache, **kw)
    bo, bl = fp32_bounds(ref, "bf16")
    used = ref[0].shape[0]
    copied = workspace(cache, kw["W"], kw["alpha"], kw["rungs"]) > 0
    within(o[:used], ref[0], bo + (split_bound if copied else halves_bound)(ref), "o")
    within(lse[:used], ref[1], bl, "lse")
    return o


@pytest.mark.parametrize("lens,page,block,W,rungs", [([(7200, 30)], 16, 8, 12, FIB), ([(1024, 0)] * 16, 64, 16, 12, FIB),
                                                     ([(300, 40 * s) for s in range(64)], 64, 64, 5, FIB),
                                                     ([(4000, 900), (1, 7), (0, 3), (3333, 0)], 256, 32, 28, MANY_RUNGS),
                                                     ([(20000, 50)], 128, 16, 0, (400.5,))])
def test_scales_that_are_no_powers_of_two(lens, page, block, W, rungs):
    _check(Cache8(lens, page, "bf16", block, seed=len(lens), powers=False), alpha=0.93, W=W, rungs=rungs)


@pytest.mark.parametrize("every", [2, 7, 100])
def test_a_few_such_blocks(every):
    """A few blocks with such a scale among others: what reads none of them keeps every bit."""
    lens = [(5000, 300), (2500, 0), (40, 100)]
    kw = dict(alpha=0.93, W=12, rungs=FIB)
    cache = Cache8(lens, 64, "bf16", 16, seed=11)
    before = _check(cache, **kw)
    s = 1
    hit = (torch.arange(cache.v[s].shape[0]) // 16) % every == every - 1
    for i, x in enumerate((cache.k, cache.v)):
        cache.scales[i][s][hit] *= 1.37
        x[s] = cache.codes[i][s].float() * cache.scales[i][s][..., None]
    after = _check(cache, **kw)
    for rows in (slice(0, 5000), slice(7500, 7540)):      # of the other sequences
        assert torch.equal(before[rows], after[rows])


def test_bad_values_and_pages_beside_such_scales():
    """A NaN element and a page out of range: queries that read neither keep every bit, alone
    or not, and the others get what the formula gives."""
    cache = Cache8([(7200, 300), (60, 0)], 32, "bf16", 16, seed=13, powers=False)
    kw = dict(alpha=0.93, W=5, rungs=FIB)
    pages, (table, cu, seq) = cache.pages8(), cache.meta()
    q = cache.q.cuda()
    clean = api.sfa_paged_forward_fp8(q, *pages, table, cu, seq, **kw)
    row, page = 4000, 5000 // 32
    pages[1].view(torch.uint8).view(-1, HKV, D)[cache.slots(0)[row], :, 17] = NAN_CODE
    table[0, page] = cache.num_pages
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = api.sfa_paged_forward_fp8(q, *pages, table, cu, seq, status=status, **kw)
    assert api.sfa_read_status(status) == 0x2
    reach = set(range(kw["W"] + 1)) | {n + e for n, t, _ in rung_list(kw["alpha"], kw["W"], kw["rungs"]) for e in ((0, 1) if t else (0,))}
    reads = lambda rows: torch.tensor([any(i - d in rows for d in reach) for i in range(300, 7500)])  # noqa: E731
    nan, hole = reads({row}), reads(set(range(32 * page, 32 * page + 32)))
    o, lse = got[0][:7260].cpu(), got[1][:7260].cpu()
    other = torch.cat((~nan & ~hole, torch.ones(60, dtype=torch.bool)))
    assert torch.equal(o[other], clean[0][:7260].cpu()[other]) and torch.equal(lse[other], clean[1][:7260].cpu()[other])
    bad = torch.isnan(o[:7200, :, 17]).all(1)
    assert torch.equal(bad, nan) and not bool(torch.isnan(o[:7200, :, :17]).any())
