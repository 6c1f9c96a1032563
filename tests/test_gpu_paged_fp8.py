"""The paged cache in 8 bits: appending a step's keys and values
(sfa_paged_append_fp8) and the attention of its tokens over the pages
(sfa_paged_forward_fp8), against definitions in 64 bits with derived bounds.
Every place of a cache that a call must not use holds NaN or a page number out
of range."""
import numpy as np
import pytest
import torch

from fibonacci_spaced_sparse_gb300 import api
from _fp8 import FP8, NAN_CODE, Cache8, block_scale, codes, expanded, half_bound
from _paged import D, DT, HALF_STEP, HKV, HQ, U, attention64, head64, rung_list, within

pytestmark = pytest.mark.gpu

FIB = api.FIBONACCI_BASE
ONE = [(1, 0)]
SINGLES = [(1, c) for c in (0, 1, 7, 8, 12, 13, 15, 16, 20, 21, 89, 144, 986, 987, 1300)]
RAGGED = [(5, 0), (0, 33), (1, 21), (37, 95), (0, 0), (2, 1000), (130, 3), (1, 0)]
CHUNK = [(503, 0)]
LONG = [(1803, 70), (0, 9), (2402, 0), (1, 1200), (33, 986)]
# enough tokens for bf16 copies of the rows (7000, and 32 a sequence)
LONGER = [(3803, 70), (0, 9), (3302, 0), (1, 1200), (133, 986)]
MANY = [(0, 5)] * 3 + [(1, 40 + s) for s in range(40)] + [(3, 0)] * 5 + [(0, 0)] * 2


def _forward(cache, pages=None, **kw):
    kp, vp, sc = pages or cache.pages8()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((cache.N, HQ, D), 7.0, dtype=DT[cache.dtype], device="cuda")
    lse = torch.full((cache.N, HQ), 7.0, device="cuda")
    o, l = api.sfa_paged_forward_fp8(cache.q.cuda(), kp, vp, sc, *cache.meta(), out=out, lse=lse, status=status, **kw)
    assert o.data_ptr() == out.data_ptr() and l.data_ptr() == lse.data_ptr()
    return o, l, api.sfa_read_status(status)


def _reference(cache, bad_rows=(), **kw):
    """attention64 and its bounds: those of fp32 arithmetic, and for bf16 what the
    halves of the tensor-core kernel add (a probability's 2^-11 of the size of the
    output's sum, which attention64 gives for bf16's 2^-8, and half_bound), or bf16
    probabilities over copied rows, which are exact with scales that are powers of two."""
    o, lse, bo, bl = attention64(cache, bad_rows=bad_rows, tensor_cores=expanded(cache), **kw)
    if cache.dtype == "bf16" and not expanded(cache):
        wide = attention64(cache, bad_rows=bad_rows, tensor_cores=True, **kw)[2]
        plan = rung_list(kw["alpha"], kw["W"], kw["rungs"], kw.get("round_offsets", False))
        bo = bo + (wide - bo) * 2.0 ** -3 + half_bound(cache, kw["W"], plan)
    return o, lse, bo, bl


def _check(cache, got, ref, what=""):
    o, l = got[:2]
    used = int(cache.cu[-1])
    within(o[:used], ref[0][:used], ref[2][:used], f"{what} o")
    want = torch.from_numpy(ref[1][:used])
    none = torch.isinf(want)
    assert torch.equal(torch.isinf(l[:used].cpu()), none)
    within(l[:used].cpu()[~none], want[~none], torch.from_numpy(ref[3][:used])[~none], f"{what} lse")
    assert bool((o[used:] == 7).all()) and bool((l[used:] == 7).all()), what


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,page,block", [(ONE, 16, 16), (SINGLES, 16, 16), (SINGLES, 8, 8), (RAGGED, 64, 16), (CHUNK, 32, 8),
                                             (MANY, 16, 16), (MANY, 256, 64), (LONG, 16, 16), (LONG, 64, 32), (LONG, 8, 8),
                                             (LONG, 2048, 2048), (LONGER, 16, 8), (LONGER, 64, 16), (LONGER, 8, 8),
                                             (LONGER, 1024, 128)])
def test_forward_against_definition(lens, page, block, dtype):
    cache = Cache8(lens, page, dtype, block, seed=len(lens) + page)
    kw = dict(alpha=0.87, W=12, rungs=FIB)
    got = _forward(cache, **kw)
    assert got[2] == 0
    _check(cache, got, _reference(cache, **kw))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [0, 1, 3, 11, 12, 13, 19, 27, 28, 29, 45, 300])
def test_windows(W, dtype):
    for lens in ([(45, 11), (1, 400), (7, 0)], [(345, 11), (1, 400), (7, 0)]):
        cache = Cache8(lens, 16, dtype, 16, seed=W)
        kw = dict(alpha=1.21, W=W, rungs=FIB)
        got = _forward(cache, **kw)
        assert got[2] == 0
        _check(cache, got, _reference(cache, **kw))


@pytest.mark.parametrize("W", [0, 1, 7, 12, 13, 28, 29])
def test_windows_of_long_chunks(W):
    for lens in ([(4001, 37), (160, 0)], [(7001, 2037), (160, 0)]):
        cache = Cache8(lens, 32, "bf16", 16, seed=W)
        kw = dict(alpha=0.71, W=W, rungs=FIB)
        got = _forward(cache, **kw)
        assert got[2] == 0
        _check(cache, got, _reference(cache, **kw))


@pytest.mark.parametrize("alpha,rungs,rounded", [(1.0, FIB, False), (1.5, api.pow2_base(2048), False), (0.77, FIB, True),
                                                 (1.0, (), False), (1.3, (40.5,), False), (1.0, (30.0, 30.0, 14.25), False),
                                                 (1.1, tuple(13.0 + 0.4 * k for k in range(32)), False)])
@pytest.mark.parametrize("lens", [[(70, 60), (1, 1500), (9, 1490)], [(470, 600), (31, 1490)], [(4100, 500)], [(7100, 4000)]])
def test_rung_lists(lens, alpha, rungs, rounded):
    for dtype in ("bf16", "f32") if lens[0][0] < 4000 else ("bf16",):
        cache = Cache8(lens, 32, dtype, 16, seed=3)
        kw = dict(alpha=alpha, W=12, rungs=rungs, round_offsets=rounded)
        got = _forward(cache, **kw)
        assert got[2] == 0
        _check(cache, got, _reference(cache, **kw), dtype)


@pytest.mark.parametrize("n", [1, 2, 100, 153, 200, 310, 500, 640])
def test_every_number_of_warps_a_token(n):
    for dtype in ("bf16", "f32"):
        cache = Cache8([(1, (37 * s) % 400) for s in range(n)], 16, dtype, 16, seed=n, behind=3)
        kw = dict(alpha=0.87, W=12, rungs=FIB)
        _check(cache, _forward(cache, **kw), _reference(cache, **kw))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[(30, 70), (1, 90)], [(640, 300)], [(4200, 30)]])
def test_scales_that_differ_widely(lens, dtype):
    """Scales that are no powers of two, blocks whose sizes differ by factors of
    hundreds, a sharp softmax scale, and queries of very different sizes."""
    cache = Cache8(lens, 16, dtype, 8, seed=5, powers=False, spread=2.0)
    cache.q = (cache.q.float() * torch.exp2(torch.randint(-40, 3, (cache.N, HQ, 1)).float())).to(DT[dtype])
    kw = dict(alpha=0.93, W=12, rungs=FIB, scale=0.2)
    got = _forward(cache, **kw)
    assert got[2] == 0
    _check(cache, got, _reference(cache, **kw))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("power", [-100, -60, 60, 90])
def test_scales_far_from_one(power, dtype):
    """Values' scales at the ends of what a float holds: the output scales with
    them exactly (powers of two), lse stays."""
    for lens in ([(20, 70), (1, 90)], [(700, 30)], [(4100, 30)], [(7100, 30)]):
        cache = Cache8(lens, 16, dtype, 16, seed=6)
        kp, vp, sc = cache.pages8()
        kw = dict(alpha=0.9, W=12, rungs=FIB)
        want = _forward(cache, (kp, vp, sc), **kw)
        far = sc.clone()
        far[:, :, 1] *= 2.0 ** power
        got = _forward(cache, (kp, vp, far), **kw)
        used = int(cache.cu[-1])
        # the first pass's own bound: the running maximum sits elsewhere, so halves round elsewhere
        ref = _reference(cache, **kw)
        back = got[0][:used].double().cpu() * 2.0 ** -power
        within(back, ref[0][:used], ref[2][:used])
        within(got[1][:used], ref[1][:used], ref[3][:used])
        assert torch.allclose(back, want[0][:used].double().cpu(), rtol=0.05, atol=1e-2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[(400, 200)], [(1, 300 + 7 * s) for s in range(20)], [(900, 0), (1, 500)], [(4200, 150)],
                                  [(7200, 3150), (33, 8)]])
def test_bad_values_reach_only_the_queries_that_read_them(lens, dtype):
    """A NaN key element, a NaN value element and a block whose values' scale is NaN:
    the queries that read them get what the formula gives, the others what they
    got before, bit for bit."""
    cache = Cache8(lens, 16, dtype, 8, seed=12)
    kw = dict(alpha=0.87, W=5, rungs=FIB)
    pages = cache.pages8()
    clean = _forward(cache, pages, **kw)
    length = lens[0][0] + lens[0][1]
    slots = cache.slots(0)
    kpos, vpos, spos = length // 2, length // 2 + 40, (length // 2 + 80) // 8 * 8
    pages[0].view(torch.uint8).view(-1, HKV, D)[slots[kpos], :, 3] = NAN_CODE
    pages[1].view(torch.uint8).view(-1, HKV, D)[slots[vpos], :, 17] = NAN_CODE
    pages[2].view(-1, 2, HKV)[slots[spos] // 8, 1] = float("nan")
    cache.k[0][kpos, :, 3] = float("nan")
    cache.v[0][vpos, :, 17] = float("nan")
    cache.v[0][spos:spos + 8] = float("nan")
    got = _forward(cache, pages, **kw)
    ref = attention64(cache, **kw)
    used = int(cache.cu[-1])
    finite = torch.isfinite(torch.from_numpy(ref[0][:used]))
    o, c = got[0][:used].cpu(), clean[0][:used].cpu()
    assert torch.equal(torch.isfinite(o.float()), finite)
    whole = finite.flatten(1).all(1) & torch.from_numpy(np.isfinite(ref[1][:used])).all(1)
    assert torch.equal(o[whole], c[whole])
    assert not bool(whole.all()) or lens[0][0] == 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,page", [([(30, 70), (1, 90)], 8), ([(1, 99), (1, 40)], 8), ([(640, 60), (3, 5)], 8),
                                       ([(4200, 60), (3, 5)], 8), ([(7200, 60), (3, 5)], 16), ([(7200, 5060), (30, 5)], 128)])
def test_bad_pages_are_left_out_and_reported(lens, page, dtype):
    if dtype == "f32" and lens[0][0] > 5000:
        pytest.skip("the copied rows are bf16's")
    cache = Cache8(lens, page, dtype, 8, seed=15)
    length = lens[0][0] + lens[0][1]
    mid, last = length // (2 * page), (length - 1) // page
    if lens[0][1] > 5000:
        mid = (lens[0][1] + 3000) // page
    cache.table[0, mid], cache.table[0, last] = cache.num_pages, -7
    bad = [(0, i) for i in range(length) if i // page in (mid, last)]
    kw = dict(alpha=0.87, W=4, rungs=FIB)
    got = _forward(cache, **kw)
    assert got[2] == 0x2
    _check(cache, got, _reference(cache, bad_rows=bad, **kw))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("more", [0, 700, 4200, 7200])
def test_bad_positions_give_zeros(dtype, more):
    if dtype == "f32" and more > 5000:
        pytest.skip("the copied rows are bf16's")
    cache = Cache8([(4, 0), (20 + more, 10), (3, 60)], 16, dtype, 16, seed=18)
    cap = cache.max_pages * 16
    seq = torch.tensor([2, 30 + more, cap + 2], dtype=torch.int32).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(alpha=0.9, W=12, rungs=())
    o, lse = api.sfa_paged_forward_fp8(cache.q.cuda(), *cache.pages8(), *cache.meta()[:2], seq, status=status, **kw)
    assert api.sfa_read_status(status) & 0x2
    end = 24 + more
    for rows in (slice(0, 2), slice(end + 1, end + 3)):
        assert bool((o[rows] == 0).all()) and bool((lse[rows] == 0).all())
    ref = _reference(cache, **kw)
    within(o[4:end], ref[0][4:end], ref[2][4:end])
    within(lse[4:end], ref[1][4:end], ref[3][4:end])


def test_copied_rows_of_sequences_far_into_a_wide_table():
    """Chunks that start far behind the first position, in a table so wide that the
    copies' own is narrower, beside a sequence whose length passes its capacity: two
    tokens at the last positions, which have no pages, and one behind them."""
    page = 16
    cache = Cache8([(7000, 20000), (500, 11000), (3, 0)], page, "bf16", 16, seed=8)
    wide = torch.full((3, 2100), -1, dtype=torch.int32)
    wide[:, :cache.max_pages] = cache.table
    cap = 2100 * page
    seq = cache.seq.clone()
    seq[2] = cap + 1
    kw = dict(alpha=0.9, W=12, rungs=FIB)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = api.sfa_paged_forward_fp8(cache.q.cuda(), *cache.pages8(), wide.cuda(), cache.meta()[1], seq.cuda(), status=status, **kw)
    assert api.sfa_read_status(status) == 0x2
    ref = _reference(cache, **kw)
    within(o[:7500], ref[0][:7500], ref[2][:7500])
    within(lse[:7500], ref[1][:7500], ref[3][:7500])
    assert bool((o[7500:7503] == 0).all()) and bool(torch.isneginf(lse[7500:7502]).all()) and bool((lse[7502] == 0).all())


def test_copied_rows_with_other_scales():
    """Scales that are no powers of two: a copied element is off by 2^-8 of itself, so a
    score by 2^-8 scale |q| |k| and 2^-8 of the output's sum more."""
    cache = Cache8([(7200, 30)], 16, "bf16", 8, seed=5, powers=False)
    kw = dict(alpha=0.93, W=12, rungs=FIB)
    got = _forward(cache, **kw)
    ref = _reference(cache, **kw)
    used = int(cache.cu[-1])
    q = cache.q[:used].double().norm(dim=-1)
    k = cache.k[0].double().norm(dim=-1).amax(0).repeat_interleave(HQ // HKV)
    delta = 2.0 ** -8 * 0.125 * q * k                                         # [tokens, heads]
    size = (torch.from_numpy(ref[2][:used]) - 2.0 ** -8 * torch.from_numpy(ref[0][:used]).abs()) * 2.0 ** 8   # sum p |v| at least
    within(got[0][:used], ref[0][:used], torch.from_numpy(ref[2][:used]) + (2 * delta[..., None] + 2.0 ** -8) * size)
    within(got[1][:used], ref[1][:used], torch.from_numpy(ref[3][:used]) + delta)


@pytest.mark.parametrize("n,before", [(1, 1300), (300, 200), (1800, 900), (4001, 1000)])
def test_pages_of_two_sequences(n, before):
    """Two sequences that read the same pages (a prefix that they share), against the
    same calls with a copy of the pages each; and both calls at once, on two streams."""
    cache = Cache8([(n, before)], 16, "bf16", 16, seed=n)
    pages, table = cache.pages8(), cache.table.cuda()
    q = torch.randn((2 * n, HQ, D), generator=torch.Generator().manual_seed(n)).to(torch.bfloat16).cuda()
    cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    seq = torch.full((2,), n + before, dtype=torch.int32, device="cuda")
    kw = dict(alpha=0.87, W=12, rungs=FIB)
    twice = [torch.cat((x.view(torch.uint8), x.view(torch.uint8))).view(x.dtype) for x in pages]
    calls = [(*twice, torch.cat((table, table + cache.num_pages))), (*pages, torch.cat((table, table)))]
    want = [api.sfa_paged_forward_fp8(q, *c, cu, seq, **kw) for c in calls]
    assert all(torch.equal(x, y) for x, y in zip(*want))
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in calls]
    got = [api.sfa_paged_forward_fp8(q, *c, cu, seq, stream=s, **kw) for _ in range(4) for c, s in zip(calls, sides)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for g in got for x, y in zip(g, want[0]))


@pytest.mark.parametrize("lens", [SINGLES, RAGGED, LONG, LONGER])
def test_packed_queries_other_stream_and_no_lse(lens):
    cache = Cache8(lens, 16, "bf16", 16, seed=41)
    wide = torch.randn((cache.N, 12 * D)).to(torch.bfloat16).cuda()
    wide[:, :HQ * D] = cache.q.cuda().flatten(1)
    pages, meta = cache.pages8(), cache.meta()
    kw = dict(alpha=0.87, W=12, rungs=FIB)
    want, _ = api.sfa_paged_forward_fp8(cache.q.cuda(), *pages, *meta, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, none = api.sfa_paged_forward_fp8(wide[:, :HQ * D].unflatten(-1, (HQ, D)), *pages, *meta, need_lse=False, stream=side,
                                          **kw)
    side.synchronize()
    used = int(cache.cu[-1])
    assert none is None and torch.equal(got[:used], want[:used])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cache_rows_past_32_bits(dtype):
    """Pages whose bytes lie past 2^32."""
    rows = (1 << 25) + (1 << 20)          # 128 bytes a row
    for n in (600,) if dtype == "f32" else (4100, 7100):
        cache = Cache8([(70, 30), (1, 500), (n, 0)], 64, dtype, 16, seed=5, num_pages=rows // 64)
        assert int(cache.table[0, 0]) * 64 * HKV * D > 1 << 32
        kw = dict(alpha=0.87, W=12, rungs=FIB)
        got = _forward(cache, **kw)
        assert got[2] == 0
        _check(cache, got, _reference(cache, **kw))


# -------------------------------------------------------------------- append


def _inputs(N, dtype, packed, seed=77, size=1.0):
    g = torch.Generator().manual_seed(seed)
    grow = size * torch.exp(0.8 * torch.randn((N, 1, 1), generator=g))
    if packed:
        x = (torch.randn((N, 12, D), generator=g) * grow).to(DT[dtype]).cuda()
        return x.split((HQ, HKV, HKV), 1)
    return tuple((torch.randn((N, h, D), generator=g) * grow).to(DT[dtype]).cuda() for h in (HQ, HKV, HKV))


def _check_append(cache, before, after, k64, v64, kbound, start=None):
    """The pages after an append of the keys k64 and values v64 (64 bits, in token
    order; kbound: error of the kernel's keys before their rounding) to the pages
    before it; `start`: first new position of each sequence."""
    block = cache.block
    flat = lambda x: x.view(torch.uint8).view(-1, HKV, D).cpu()  # noqa: E731
    touched = torch.zeros(cache.num_pages * cache.page, dtype=torch.bool)
    blocks = torch.zeros(touched.numel() // block, dtype=torch.bool)
    old_sc, new_sc = before[2].view(-1, 2, HKV).cpu(), after[2].view(-1, 2, HKV).cpu()
    old_c, new_c = [flat(x) for x in before[:2]], [flat(x) for x in after[:2]]
    grown = 0
    for s, (n, c) in enumerate(cache.lens):
        if not n:
            continue
        at = int(cache.cu[s])
        slots = cache.slots(s)
        for b in range(c // block, (c + n - 1) // block + 1):
            lo, hi = max(c, b * block), min(c + n, (b + 1) * block)
            blk = int(slots[lo]) // block
            blocks[blk] = True
            rows, older = slots[lo:hi], slots[b * block:lo]
            touched[rows] = touched[older] = True
            for i, (x, err) in enumerate(((k64, kbound), (v64, torch.zeros_like(v64)))):
                x, err = x[at + lo - c:at + hi - c], err[at + lo - c:at + hi - c]
                for h in range(HKV):
                    xx = x[:, h]
                    fine = torch.isfinite(xx)
                    amax = float(torch.where(fine, xx.abs(), 0.0).max())
                    slack = float(err[:, h].max())
                    allowed = {block_scale(max(0.0, amax - slack)), block_scale(amax + slack)}  # next to a border either will do
                    if len(older):
                        allowed = {max(a, float(old_sc[blk, i, h])) for a in allowed}
                    got = float(new_sc[blk, i, h])
                    assert got in allowed, (s, b, i, h, got, allowed)
                    stored = new_c[i][rows, h].view(FP8).double()
                    assert torch.equal(torch.isnan(stored), ~fine)
                    off = (stored * got - xx).abs()[fine]
                    bound = (2.0 ** -4 * xx.abs() + 2.0 ** -10 * got + 1.1 * err[:, h])[fine]
                    assert bool((off <= bound).all()), (s, b, i, h, float((off / bound).max()))
                    if i == 1:   # values are rounded once, from what came in
                        assert torch.equal(new_c[i][rows, h], codes(xx / got).view(torch.uint8))
                    if len(older):
                        was = old_c[i][older, h].view(FP8).float()
                        ratio = float(old_sc[blk, i, h]) / got
                        grown += ratio < 1
                        want = codes(was * ratio).view(torch.uint8)
                        assert torch.equal(new_c[i][older, h], want if ratio != 1 else old_c[i][older, h])
    for a, b in zip(new_c, old_c):   # nothing else changed
        assert torch.equal(a[~touched], b[~touched])
    assert torch.equal(new_sc[~blocks].nan_to_num(3.0), old_sc[~blocks].nan_to_num(3.0))
    return grown


def _append(cache, pages, q, k, v, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = api.sfa_paged_append_fp8(k, v, *pages, *cache.meta(), q=q, status=status, **kw)
    return r, api.sfa_read_status(status)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,page,block", [(ONE, 16, 16), (SINGLES, 16, 16), (SINGLES, 8, 8), (SINGLES, 64, 32), (RAGGED, 16, 8),
                                             (CHUNK, 64, 16), (MANY, 16, 16), (MANY, 128, 128), (LONG, 64, 16), (LONG, 64, 64),
                                             ([(2, c) for c in range(40)], 32, 32)])
@pytest.mark.parametrize("with_q,norm,packed,theta", [(True, True, True, 1e4), (False, True, True, 0.0), (False, False, False, 1e4)])
def test_append_against_definition(lens, page, block, dtype, with_q, norm, packed, theta):
    cache = Cache8(lens, page, dtype, block, seed=2 * len(lens) + page)
    q, k, v = _inputs(cache.N, dtype, packed)
    g = torch.Generator().manual_seed(1)
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=g)).cuda() if norm else None for _ in range(2))
    pages = cache.pages8(rows_before=True)
    before = [x.clone() for x in pages]
    q_out = torch.full((cache.N, HQ, D), 7.0, dtype=DT[dtype], device="cuda") if with_q else None
    qo, status = _append(cache, pages, q if with_q else None, k, v, wq=wq if with_q else None, wk=wk, rope_theta=theta, q_out=q_out)
    assert status == 0 and (qo is None) == (not with_q)
    used = int(cache.cu[-1])
    pos = torch.cat([torch.arange(c, c + n) for n, c in lens])
    k64, kb = head64(k[:used].double().cpu(), wk.double().cpu() if norm else None, 1e-6, pos, theta)
    grown = _check_append(cache, before, pages, k64, v[:used].double().cpu(), kb)
    assert grown or lens in (ONE, CHUNK) or len(lens) < 10
    if with_q:
        want, bound = head64(q[:used].double().cpu(), wq.double().cpu() if norm else None, 1e-6, pos, theta)
        within(qo[:used], want, bound + HALF_STEP[dtype] * want.abs() + 1e-30, "q")
        assert bool((qo[used:] == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("step", [1, 3])
def test_growing_block_token_by_token(dtype, step):
    """Tokens of rising and falling sizes, one or three a call: the scale of a block
    is that of all of its tokens so far, its older rows keep their values but for
    what sinks below the smallest normal one, and a new block starts anew."""
    block, T = 16, 60
    cache = Cache8([(T, 0)], 16, dtype, block, seed=1, behind=0)
    g = torch.Generator().manual_seed(5)
    size = torch.exp2(torch.randint(-6, 7, (T, 1, 1), generator=g).float())
    k, v = ((torch.randn((T, HKV, D), generator=g) * size).to(DT[dtype]) for _ in range(2))
    pages = cache.pages8(rows_before=True)
    for t in range(0, T, step):
        cache.lens, cache.cu, cache.seq = [(step, t)], torch.tensor([0, step], dtype=torch.int32), torch.tensor([t + step], dtype=torch.int32)
        cache.N = step
        before = [x.clone() for x in pages]
        _, status = _append(cache, pages, None, k[t:t + step].cuda(), v[t:t + step].cuda(), rope_theta=0.0)
        assert status == 0
        _check_append(cache, before, pages, k[t:t + step].double(), v[t:t + step].double(), torch.zeros((step, HKV, D), dtype=torch.float64))
    cache.lens = [(T, 0)]
    rows = cache.slots(0)
    for i, x in enumerate((k, v)):
        got = pages[i].view(-1, HKV, D).cpu().double()[rows]
        sc = pages[2].view(-1, 2, HKV).cpu()[rows // block, i].double()
        final = torch.tensor([[block_scale(float(x[b * block:(b + 1) * block, h].abs().max())) for h in range(HKV)]
                              for b in range(-(-T // block))]).double()
        assert torch.equal(sc, final.repeat_interleave(block, 0)[:T])
        # one rounding to 2^-4, and for small values one to a subnormal step each time the scale grew
        off = (got * sc[..., None] - x.double()).abs()
        assert bool((off <= 2.0 ** -4 * x.double().abs() + 4 * 2.0 ** -10 * sc[..., None]).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_values_that_are_not_finite(dtype):
    """Infinity and NaN become NaN, do not count towards the scale, and leave the
    other rows of their block alone; zeros get the smallest scale."""
    cache = Cache8([(20, 3), (16, 0), (1, 31)], 16, dtype, 16, seed=3, behind=0)
    _, k, v = _inputs(cache.N, dtype, False)
    k[4, 0, 5], k[5, 1, 6], v[6, 0, 7], v[30, 1, 1] = float("inf"), float("nan"), -float("inf"), float("nan")
    k[20:36, 1] = 0
    v[20:36, 0] = float("nan")
    pages = cache.pages8(rows_before=True)
    before = [x.clone() for x in pages]
    _, status = _append(cache, pages, None, k, v, rope_theta=0.0)
    assert status == 0
    _check_append(cache, before, pages, k.double().cpu(), v.double().cpu(), torch.zeros_like(k).double().cpu())
    b = int(cache.slots(1)[0]) // 16
    sc = pages[2].view(-1, 2, HKV)[b].cpu()
    assert float(sc[0, 1]) == 2.0 ** -100 and float(sc[1, 0]) == 2.0 ** -100


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("amax", [448.0, 449.0, 3.5, 3.515625, 2.0 ** -100 * 448, 2.0 ** -110, 1.5 * 2.0 ** 126])
def test_append_scale_borders(dtype, amax):
    cache = Cache8([(16, 0)], 16, dtype, 16, behind=0)
    k = (torch.zeros((16, HKV, D)) + amax / 8).to(DT[dtype]).cuda()
    k[3, 0, 9] = amax
    v = -k
    pages = cache.pages8(rows_before=True)
    before = [x.clone() for x in pages]
    _append(cache, pages, None, k, v, rope_theta=0.0)
    _check_append(cache, before, pages, k.double().cpu(), v.double().cpu(), torch.zeros_like(k).double().cpu())


def test_append_bad_metadata():
    """Bad pages are not stored to, bad positions neither; both are reported, their
    queries get zeros, and the other tokens are stored."""
    for lens in ([(20, 3), (4, 0), (6, 10)], [(1, 3), (1, 0), (1, 10), (1, 30)]):
        single = lens[0][0] == 1
        cache = Cache8(lens, 8, "bf16", 8, seed=9)
        cache.table[0, 0 if single else 1] = cache.num_pages + 5
        seq = list(cache.seq.tolist())
        seq[1] = 0 if single else 2                          # positions -1, or -2, -1, 0, 1
        if single:
            seq[3] = cache.max_pages * 8 + 1                  # past the capacity
        q, k, v = _inputs(cache.N, "bf16", False)
        pages = cache.pages8(rows_before=True)
        before = [x.clone() for x in pages]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        table, cu, _ = cache.meta()
        qo = api.sfa_paged_append_fp8(k, v, *pages, table, cu, torch.tensor(seq, dtype=torch.int32).cuda(), q=q, status=status)
        assert api.sfa_read_status(status) == 0x2
        flat, old = pages[1].view(torch.uint8).view(-1, HKV, D), before[1].view(torch.uint8).view(-1, HKV, D)
        touched = torch.zeros(flat.shape[0], dtype=torch.bool, device="cuda")
        for s, (n, _) in enumerate(lens):
            first = int(cu[s])
            for j in range(n):
                pos = seq[s] - n + j
                good = 0 <= pos < cache.max_pages * 8
                assert bool((qo[first + j] == 0).all()) == (not good)
                page = int(table[s, pos // 8]) if good else -1
                if 0 <= page < cache.num_pages:
                    row = page * 8 + pos % 8
                    touched[page * 8:row + 1] = True         # older rows of its block may move
                    sc = pages[2].view(-1, 2, HKV)[page, 1]
                    off = (flat[row].view(FP8).float() * sc[:, None] - v[first + j].float()).abs()
                    assert bool((off <= 2.0 ** -4 * v[first + j].float().abs() + 2.0 ** -10 * sc[:, None]).all())
        assert torch.equal(flat[~touched], old[~touched])


@pytest.mark.parametrize("offsets,lens", [([0, 5, 2, 9], [5, 9, 9]), ([3, 7, 7, 9], [8, 0, 4]), ([-4, 2, 6, 6], [6, 6, 1]),
                                          ([0, 40, 41, 41], [44, 10, 3]), ([0, 3, 6, 9], [-7, -(1 << 31), (1 << 31) - 1])])
def test_append_offsets_that_make_no_sense(offsets, lens):
    """Offsets that decrease, start past 0 or below it, or end past the rows, and
    lengths far out of range: nothing outside the sequences' own pages changes."""
    cache = Cache8([(3, 5)] * 3, 16, "bf16", 16, seed=2, behind=0)
    q, k, v = _inputs(cache.N, "bf16", False)
    pages = cache.pages8()
    before = [x.clone() for x in pages]
    table = cache.meta()[0]
    cu, seq = (torch.tensor(x, dtype=torch.int64).int().cuda() for x in (offsets, lens))
    api.sfa_paged_append_fp8(k, v, *pages, table, cu, seq, q=q)
    torch.cuda.synchronize()
    own = torch.zeros(cache.num_pages, dtype=torch.bool)
    own[cache.table[:, 0].long()] = True
    for a, b in zip(pages, before):
        a, b = (x.view(torch.uint8).view(cache.num_pages, -1).cpu() for x in (a, b))
        assert torch.equal(a[~own], b[~own])


def test_append_rows_past_32_bits():
    rows = (1 << 25) + (1 << 20)
    cache = Cache8([(70, 30), (1, 500), (40, 0)], 64, "bf16", 16, seed=5, num_pages=rows // 64)
    assert int(cache.table[0, 0]) * 64 * HKV * D > 1 << 32
    q, k, v = _inputs(cache.N, "bf16", True)
    pages = cache.pages8(rows_before=True)
    total = [int(x.view(torch.uint8).view(-1).sum(dtype=torch.int64)) for x in pages[:2]]
    _, status = _append(cache, pages, None, k, v, rope_theta=0.0)
    assert status == 0
    for i, (x, t) in enumerate(zip((k, v), total)):
        at = 0
        for s, (n, c) in enumerate(cache.lens):
            slots = cache.slots(s)[c:].cuda()
            sc = pages[2].view(-1, 2, HKV)[slots // 16, i][..., None]
            got = pages[i].view(-1, HKV, D)[slots].float() * sc
            assert bool(((got - x[at:at + n].float()).abs() <= 2.0 ** -4 * x[at:at + n].float().abs() + 2.0 ** -10 * sc).all())
            at += n


@pytest.mark.parametrize("lens", [SINGLES, LONG])
def test_append_on_another_stream(lens):
    cache = Cache8(lens, 16, "bf16", 16, seed=4)
    q, k, v = _inputs(cache.N, "bf16", True)
    a, b = cache.pages8(rows_before=True), cache.pages8(rows_before=True)
    want = api.sfa_paged_append_fp8(k, v, *a, *cache.meta(), q=q)
    meta = cache.meta()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = api.sfa_paged_append_fp8(k, v, *b, *meta, q=q, stream=side)
    side.synchronize()
    used = int(cache.cu[-1])
    assert torch.equal(got[:used], want[:used])
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_append_twice_changes_nothing():
    """The same step again: older rows have moved to the scale already."""
    for lens in (SINGLES, RAGGED):
        cache = Cache8(lens, 16, "bf16", 16, seed=4)
        q, k, v = _inputs(cache.N, "bf16", True)
        pages = cache.pages8(rows_before=True)
        api.sfa_paged_append_fp8(k, v, *pages, *cache.meta())
        once = [x.clone() for x in pages]
        api.sfa_paged_append_fp8(k, v, *pages, *cache.meta())
        for x, y in zip(pages, once):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("pad_to", [64, 900, 4200, 8000])
def test_captured_step_replayed_with_other_lengths(pad_to):
    """One captured step (append, then attention) of a fixed number of token rows,
    replayed with other lengths, tables and inputs, equals the calls alone."""
    S, page, block = 12, 16, 16
    g = torch.Generator().manual_seed(pad_to)
    max_pages = 4 + pad_to // page
    bufs = {n: torch.zeros((pad_to, h, D), dtype=torch.bfloat16, device="cuda") for n, h in (("q", HQ), ("k", HKV), ("v", HKV))}
    table = torch.full((S, max_pages), -1, dtype=torch.int32, device="cuda")
    cu, seq = torch.zeros(S + 1, dtype=torch.int32, device="cuda"), torch.zeros(S, dtype=torch.int32, device="cuda")
    num_pages = S * max_pages
    def fresh():
        return [torch.full((num_pages, page, HKV, D), NAN_CODE, dtype=torch.uint8, device="cuda").view(FP8) for _ in range(2)] + \
            [torch.full((num_pages, page // block, 2, HKV), float("nan"), device="cuda")]
    pages = fresh()
    rope = api.rope_table(max_pages * page, "cuda")
    qo, o = (torch.zeros((pad_to, HQ, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lse = torch.zeros((pad_to, HQ), device="cuda")
    def step():
        api.sfa_paged_append_fp8(bufs["k"], bufs["v"], *pages, table, cu, seq, q=bufs["q"], rope=rope, q_out=qo)
        api.sfa_paged_forward_fp8(qo, *pages, table, cu, seq, alpha=0.87, W=12, out=o, lse=lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for turn in range(4):
        lens = [(int(torch.randint(0, 1 + 2 * pad_to // (3 * S), (1,), generator=g)), 0) for _ in range(S)] if turn % 2 else \
            [(1, 0)] * S
        ctx = [int(torch.randint(0, 30, (1,), generator=g)) for _ in range(S)]
        order = torch.randperm(num_pages, generator=g).view(S, max_pages).int()
        table.copy_(order)
        cu.copy_(torch.tensor([0] + list(np.cumsum([n for n, _ in lens])), dtype=torch.int32))
        seq.copy_(torch.tensor([n + c for (n, _), c in zip(lens, ctx)], dtype=torch.int32))
        for x in bufs.values():
            x.copy_(torch.randn(x.shape, generator=g).to(torch.bfloat16))
        start = fresh()
        for x in start[:2]:
            x.view(torch.uint8).copy_(torch.randint(0, 0x70, x.shape, generator=g, dtype=torch.uint8))
        start[2].fill_(2.0 ** -7)
        results = []
        for replay in (False, True):
            for a, b in zip(pages, start):
                a.view(torch.uint8).copy_(b.view(torch.uint8))
            o.fill_(7), lse.fill_(7), qo.fill_(7)
            torch.cuda.synchronize()
            graph.replay() if replay else step()
            torch.cuda.synchronize()
            results.append([o.clone(), lse.clone(), qo.clone()] + [x.view(torch.uint8).clone() for x in pages])
        for a, b in zip(*results):
            assert torch.equal(a, b)
        used = int(cu[-1])
        assert bool((results[0][0][used:] == 7).all()) and not bool((results[0][0][:used] == 7).all())
