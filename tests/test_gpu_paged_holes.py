"""Bad pages and bad values in long chunks, in pages of every size that the
kernels tell apart: parts of a window and of a rung's rows that lie in a bad page
are left out, alone and together with NaN rows, where blocks go through their
slots a grid apart and where they ask for them."""
import numpy as np
import pytest
import torch

from fibonacci_spaced_sparse_gb300 import api
from _paged import Cache, D, DT, HQ, attention64, within

pytestmark = pytest.mark.gpu

FIB = api.FIBONACCI_BASE


def _forward(cache, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((cache.N, HQ, D), 7.0, dtype=DT[cache.dtype], device="cuda")
    lse = torch.full((cache.N, HQ), 7.0, device="cuda")
    kp, vp = cache.pages()
    api.sfa_paged_forward(cache.q.cuda(), kp, vp, *cache.meta(), out=out, lse=lse, status=status, **kw)
    return out.cpu(), lse.cpu(), api.sfa_read_status(status)


def _spoil(cache, s, pages):
    """Table entries `pages` of sequence s point nowhere; returns its positions there."""
    length = cache.lens[s][0] + cache.lens[s][1]
    for i, j in enumerate(pages):
        cache.table[s, j] = (cache.num_pages, -7, 2 ** 31 - 1, -2 ** 31)[i % 4]
    return [(s, i) for i in range(length) if i // cache.page in pages]


def _compare(got, ref, rows, what):
    """Rows of `got` against those of `ref` (whose NaN are the definition's own)."""
    o, lse = got[0][rows].double(), got[1][rows].double()
    want, want_l = torch.from_numpy(ref[0]), torch.from_numpy(ref[1])
    finite = torch.isfinite(want)
    assert torch.equal(torch.isfinite(o), finite), what
    within(torch.where(finite, o, 0), torch.where(finite, want, 0), torch.from_numpy(ref[2]).nan_to_num(0, 0, 0) + 1e-30, what)
    there = torch.isfinite(want_l)
    assert torch.equal(torch.isneginf(lse), torch.isneginf(want_l)), what
    within(lse[there], want_l[there], torch.from_numpy(ref[3])[there], what + " lse")


def _one(cache, s):
    """Sequence s alone, for the definition."""
    a, b = int(cache.cu[s]), int(cache.cu[s + 1])
    one = Cache([cache.lens[s]], cache.page, cache.dtype, behind=0)
    one.k, one.v, one.q = [cache.k[s]], [cache.v[s]], cache.q[a:b]
    return one, slice(a, b)


@pytest.mark.parametrize("nan", [False, True])
@pytest.mark.parametrize("W", [4, 12, 28])
@pytest.mark.parametrize("page", [8, 16, 64, 512])
def test_holes_in_a_long_chunk(page, W, nan):
    """4200 new tokens over 60 rows: a bad page at the start, two neighbours in the
    middle, one two pages later, and the last one."""
    cache = Cache([(4200, 60), (3, 5)], page, "bf16", seed=page + W)
    mid, last = 2100 // page, (4260 - 1) // page
    bad = _spoil(cache, 0, sorted({0, mid, mid + 1, mid + 3, last}))
    kw = dict(alpha=0.87, W=W, rungs=FIB)
    clean = _forward(cache, **kw) if nan else None
    if nan:
        for at, x in ((1500, cache.k), (1700, cache.v), (2100 - page, cache.v)):   # the last one beside the holes
            x[0][at, :, 5] = float("nan")
    got = _forward(cache, **kw)
    assert got[2] == 0x2
    ref = attention64(cache, bad_rows=bad, tensor_cores=True, **kw)
    used = int(cache.cu[-1])
    _compare(got, [x[:used] for x in ref], slice(0, used), f"page {page}")
    assert bool((got[0][used:] == 7).all()) and bool((got[1][used:] == 7).all())
    if nan:   # queries that read no NaN: the same bits as without
        whole = torch.from_numpy(np.isfinite(ref[0][:used])).flatten(1).all(1)
        assert 0 < int(whole.sum()) < used and torch.equal(got[0][:used][whole], clean[0][:used][whole])


@pytest.mark.parametrize("nan", [False, True])
@pytest.mark.parametrize("page", [16, 64])
def test_holes_in_many_short_chunks(page, nan):
    """Ragged chunks of 300 to 800 tokens, whose blocks ask for their slots: bad
    pages in the first, a middle and the last sequence."""
    rng = np.random.default_rng(page)
    lens = [(int(rng.integers(300, 800)), int(rng.integers(0, 900))) for _ in range(60)]
    cache = Cache(lens, page, "bf16", seed=page)
    bad = {}
    for s in (0, 31, 59):
        n, c = lens[s]
        first, last = c // page, (n + c - 1) // page
        bad[s] = _spoil(cache, s, sorted({first, (first + last) // 2, (first + last) // 2 + 1, last}))
        if nan:
            cache.v[s][c + n // 4, :, 40] = float("nan")
            cache.k[s][c + n // 3, :, 2] = float("nan")
    kw = dict(alpha=0.87, W=12, rungs=FIB)
    got = _forward(cache, **kw)
    assert got[2] == 0x2
    for s in (0, 1, 31, 59):
        one, rows = _one(cache, s)
        ref = attention64(one, bad_rows=[(0, i) for _, i in bad.get(s, ())], tensor_cores=True, **kw)
        _compare(got, ref, rows, f"sequence {s}")
