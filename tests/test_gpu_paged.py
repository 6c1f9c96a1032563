"""The paged cache: appending a step's keys and values (sfa_paged_append) and
the attention of its tokens over the pages (sfa_paged_forward), against
definitions in 64 bits with derived bounds (tests/_paged.py).  Every place of
a cache that a call must not use holds NaN or a page number out of range."""
import numpy as np
import pytest
import torch

from fibonacci_spaced_sparse_gb300 import api
from oracle import oracle
from _paged import Cache, D, DT, HALF_STEP, HKV, HQ, attention64, head64, within

pytestmark = pytest.mark.gpu

FIB = api.FIBONACCI_BASE
# (new tokens, rows before) of the sequences of a step
ONE = [(1, 0)]
SINGLES = [(1, c) for c in (0, 1, 7, 8, 12, 13, 20, 21, 89, 144, 986, 987, 1300)]
RAGGED = [(5, 0), (0, 33), (1, 21), (37, 95), (0, 0), (2, 1000), (130, 3), (1, 0)]
CHUNK = [(203, 0)]
# enough tokens for the kernel of long chunks (more than 3648, and 32 a sequence)
LONG = [(1803, 70), (0, 9), (2402, 0), (1, 1200), (33, 986)]
MANY = [(0, 5)] * 3 + [(1, 40 + s) for s in range(40)] + [(3, 0)] * 5 + [(0, 0)] * 2


def _forward(cache, **kw):
    kp, vp = cache.pages()
    table, cu, seq = cache.meta()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((cache.N, HQ, D), 7.0, dtype=DT[cache.dtype], device="cuda")
    lse = torch.full((cache.N, HQ), 7.0, device="cuda")
    o, l = api.sfa_paged_forward(cache.q.cuda(), kp, vp, table, cu, seq, out=out, lse=lse, status=status, **kw)
    assert o.data_ptr() == out.data_ptr() and l.data_ptr() == lse.data_ptr()
    return o, l, api.sfa_read_status(status)


def _check(cache, got, ref, what=""):
    o, l = got[:2]
    used = int(cache.cu[-1])
    within(o[:used], ref[0][:used], ref[2][:used], f"{what} o")
    want = torch.from_numpy(ref[1][:used])
    none = torch.isinf(want)
    assert torch.equal(torch.isinf(l[:used].cpu()), none)
    within(l[:used].cpu()[~none], want[~none], torch.from_numpy(ref[3][:used])[~none], f"{what} lse")
    # rows behind the last sequence stay as they were
    assert bool((o[used:] == 7).all()) and bool((l[used:] == 7).all()), what


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,page", [(ONE, 16), (SINGLES, 16), (SINGLES, 1), (RAGGED, 8), (RAGGED, 64), (CHUNK, 32),
                                       (MANY, 16), (MANY, 256), (LONG, 16), (LONG, 64), (LONG, 8), (LONG, 2048)])
def test_forward_against_definition(lens, page, dtype):
    cache = Cache(lens, page, dtype, seed=len(lens) + page)
    kw = dict(alpha=0.87, W=12, rungs=FIB)
    got = _forward(cache, **kw)
    assert got[2] == 0
    _check(cache, got, attention64(cache, tensor_cores=dtype == "bf16", **kw))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [0, 1, 3, 8, 11, 12, 13, 19, 27, 28, 29, 45, 300])
def test_windows(W, dtype):
    cache = Cache([(45, 11), (1, 400), (7, 0)], 16, dtype, seed=W)
    kw = dict(alpha=1.21, W=W, rungs=FIB)
    got = _forward(cache, **kw)
    assert got[2] == 0
    _check(cache, got, attention64(cache, tensor_cores=dtype == "bf16", **kw))


@pytest.mark.parametrize("W", [0, 1, 7, 12, 13, 28, 29])
def test_windows_of_long_chunks(W):
    cache = Cache([(4001, 37), (160, 0)], 32, "bf16", seed=W)
    kw = dict(alpha=0.71, W=W, rungs=FIB)
    got = _forward(cache, **kw)
    assert got[2] == 0
    _check(cache, got, attention64(cache, tensor_cores=True, **kw))


@pytest.mark.parametrize("alpha,rungs,rounded", [(1.0, FIB, False), (0.77, FIB, True), (1.0, (), False),
                                                 (1.1, tuple(13.0 + 0.4 * k for k in range(32)), False),
                                                 (1.0, (30.0, 30.0, 14.25, 100.5, 31.5), False)])
def test_rung_lists_of_long_chunks(alpha, rungs, rounded):
    cache = Cache([(4100, 500)], 16, "bf16", seed=6)
    kw = dict(alpha=alpha, W=12, rungs=rungs, round_offsets=rounded)
    got = _forward(cache, **kw)
    assert got[2] == 0
    _check(cache, got, attention64(cache, tensor_cores=True, **kw))


@pytest.mark.parametrize("n", [1, 2, 100, 153, 200, 310, 500, 640])
def test_every_number_of_warps_a_token(n):
    """Single tokens on 8, 4, 2 and 1 warps each."""
    for dtype in ("bf16", "f32"):
        cache = Cache([(1, (37 * s) % 400) for s in range(n)], 16, dtype, seed=n, behind=3)
        kw = dict(alpha=0.87, W=12, rungs=FIB)
        _check(cache, _forward(cache, **kw), attention64(cache, **kw))


@pytest.mark.parametrize("alpha,rungs,rounded", [(1.0, FIB, False), (0.5, FIB, False), (1.5, api.pow2_base(2048), False),
                                                 (0.77, FIB, True), (1.0, (), False), (1.3, (40.5,), False),
                                                 (1.0, (30.0, 30.0, 14.25), False), (0.02, FIB, False),
                                                 (1.1, tuple(13.0 + 0.4 * k for k in range(32)), False)])
def test_rung_lists(alpha, rungs, rounded):
    """Integer and rounded offsets, none, one, the same one twice, 32 of them,
    and some just past the window (d in (W, W + 1))."""
    for dtype in ("bf16", "f32"):
        cache = Cache([(70, 60), (1, 1500), (9, 1490)], 32, dtype, seed=3)
        kw = dict(alpha=alpha, W=12, rungs=rungs, round_offsets=rounded)
        got = _forward(cache, **kw)
        assert got[2] == 0
        _check(cache, got, attention64(cache, tensor_cores=dtype == "bf16", **kw), f"{dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_chunk_and_scale(dtype):
    """More tokens than one launch wave of small calls, a sharp scale, scores
    that grow along the key list."""
    cache = Cache([(1500, 700), (601, 0)], 64, dtype, seed=8, gen_scale=2.0, behind=66)
    kw = dict(alpha=0.93, W=12, rungs=FIB, scale=0.3)
    _check(cache, _forward(cache, **kw), attention64(cache, tensor_cores=dtype == "bf16", **kw))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [SINGLES, RAGGED, [(700, 300)]])
def test_against_the_oracle(lens, dtype):
    """The same rows from the contiguous attention's own oracle."""
    cache = Cache(lens, 16, dtype, seed=31)
    o, lse, _ = _forward(cache, alpha=1.37, W=8, rungs=FIB)
    at = 0
    for s, (n, c) in enumerate(lens):
        if n:
            q = np.zeros((1, n + c, HQ, D))
            q[0, c:] = cache.q[at:at + n].double().numpy()
            rows = np.array([[0, c + j] for j in range(n)], dtype=np.int32)
            o_ref, lse_ref = oracle.forward_rows(q, cache.k[s][None].double().numpy(), cache.v[s][None].double().numpy(),
                                                 rows, W=8, rungs=FIB, alpha=1.37, rope_theta=0.0)
            tol = {"bf16": 2e-2, "f32": 1e-4}[dtype]
            assert np.abs(o[at:at + n].double().cpu().numpy() - o_ref).max() <= tol
            assert np.abs(lse[at:at + n].double().cpu().numpy() - lse_ref).max() <= 1e-4
        at += n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[(400, 200)], [(1, 300 + 7 * s) for s in range(20)], [(900, 0), (1, 500)], [(4200, 150)]])
def test_bad_values_reach_only_the_queries_that_read_them(lens, dtype):
    """NaN and infinity in one key row and one value row of a sequence: the
    queries whose key lists hold the row get what the formula gives, and every
    other query what it got before, bit for bit."""
    cache = Cache(lens, 16, dtype, seed=12)
    kw = dict(alpha=0.87, W=5, rungs=FIB)
    clean = _forward(cache, **kw)
    length = lens[0][0] + lens[0][1]
    kpos, vpos, ipos = length // 2, length // 2 + 40, length // 2 + 41
    cache.k[0][kpos, :, 3] = float("nan")
    cache.v[0][vpos, :, 17] = float("nan")
    cache.v[0][ipos, :, 60] = float("inf")
    got = _forward(cache, **kw)
    ref = attention64(cache, tensor_cores=dtype == "bf16", **kw)
    used = int(cache.cu[-1])
    want = torch.from_numpy(ref[0][:used])
    o, c = got[0][:used].cpu(), clean[0][:used].cpu()
    finite = torch.isfinite(want)
    assert bool((~finite).any()) or lens[0][0] == 1
    assert torch.equal(torch.isfinite(o.float()), finite)
    whole = finite.flatten(1).all(1) & torch.from_numpy(np.isfinite(ref[1][:used])).all(1)
    assert torch.equal(o[whole], c[whole])
    within(torch.where(finite, o.double(), 0), torch.where(finite, want, 0), torch.from_numpy(ref[2][:used]).nan_to_num(0, 0, 0) + 1e-30)


def test_more_bad_values_than_a_block_lists():
    """Every fourth value row NaN and keys lists of one row: a query's output is
    its own value row, NaN or not, in a chunk so long that a block meets more
    queries beside a NaN row than it can list."""
    n, page = 61000, 64
    g = torch.Generator("cuda").manual_seed(3)
    kp, vp = (torch.randn((n // page + 1, page, HKV, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    vp.view(-1, HKV, D)[::4, :, 11] = float("nan")
    q = torch.randn((n, HQ, D), generator=g, device="cuda").to(torch.bfloat16)
    table = torch.arange(n // page + 1, dtype=torch.int32, device="cuda")[None]
    cu, seq = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [n]))
    o, lse = api.sfa_paged_forward(q, kp, vp, table, cu, seq, alpha=1.0, W=0, rungs=())
    own = vp.view(-1, HKV, D)[:n].repeat_interleave(HQ // HKV, 1)
    assert torch.equal(o.isnan(), own.isnan()) and torch.equal(o.nan_to_num(9.0), own.nan_to_num(9.0))
    assert bool(lse.isfinite().all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[(30, 70), (1, 90)], [(1, 99), (1, 40)], [(640, 60), (3, 5)], [(4200, 60), (3, 5)]])
def test_bad_pages_are_left_out_and_reported(lens, dtype):
    """A page number out of range in the middle and one at the end of a
    sequence's table: entries with a row there leave the softmax, a query
    whose own page is bad keeps the others, and the status bit is set."""
    cache = Cache(lens, 8, dtype, seed=15)
    length = lens[0][0] + lens[0][1]
    mid, last = length // 16, (length - 1) // 8
    cache.table[0, mid], cache.table[0, last] = cache.num_pages, -7
    bad = [(0, i) for i in range(length) if i // 8 in (mid, last)]
    kw = dict(alpha=0.87, W=4, rungs=FIB)
    got = _forward(cache, **kw)
    assert got[2] == 0x2
    _check(cache, got, attention64(cache, bad_rows=bad, tensor_cores=dtype == "bf16", **kw))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_entry_left_gives_zeros(dtype):
    for more in (600, 4200):
        _no_entry(dtype, more)


def _no_entry(dtype, long):
    cache = Cache([(3, 0), (long, 0)], 16, dtype, seed=16)
    cache.table[0, 0] = -1
    kw = dict(alpha=1.0, W=6, rungs=FIB)
    got = _forward(cache, **kw)
    assert got[2] == 0x2
    assert bool((got[0][:3] == 0).all()) and bool(torch.isneginf(got[1][:3]).all())
    _check(cache, got, attention64(cache, bad_rows=[(0, i) for i in range(3)], tensor_cores=dtype == "bf16", **kw))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("more", [0, 700, 4200])
def test_bad_positions_give_zeros(dtype, more):
    """More new tokens than rows (negative positions), a length past the
    table's capacity, and a good sequence between them."""
    cache = Cache([(4, 0), (20 + more, 10), (3, 60)], 16, dtype, seed=18)
    cap = cache.max_pages * 16
    table, cu, _ = cache.meta()
    seq = torch.tensor([2, 30 + more, cap + 2], dtype=torch.int32).cuda()
    kp, vp = cache.pages()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(alpha=0.9, W=12, rungs=())
    o, lse = api.sfa_paged_forward(cache.q.cuda(), kp, vp, table, cu, seq, status=status, **kw)
    assert api.sfa_read_status(status) & 0x2
    end = 24 + more
    for rows in (slice(0, 2), slice(end + 1, end + 3)):
        assert bool((o[rows] == 0).all()) and bool((lse[rows] == 0).all())
    ref = attention64(cache, tensor_cores=dtype == "bf16", **kw)
    within(o[4:end], ref[0][4:end], ref[2][4:end])
    within(lse[4:end], ref[1][4:end], ref[3][4:end])


@pytest.mark.parametrize("lens", [SINGLES, RAGGED, LONG])
def test_packed_queries_other_stream_and_no_lse(lens):
    cache = Cache(lens, 16, "bf16", seed=41)
    wide = torch.randn((cache.N, 12 * D)).to(torch.bfloat16).cuda()
    wide[:, :HQ * D] = cache.q.cuda().flatten(1)
    kp, vp = cache.pages()
    kw = dict(alpha=0.87, W=12, rungs=FIB)
    want, _ = api.sfa_paged_forward(cache.q.cuda(), kp, vp, *cache.meta(), **kw)
    meta = cache.meta()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, none = api.sfa_paged_forward(wide[:, :HQ * D].unflatten(-1, (HQ, D)), kp, vp, *meta, need_lse=False, stream=side,
                                      **kw)
    side.synchronize()
    used = int(cache.cu[-1])
    assert none is None and torch.equal(got[:used], want[:used])


@pytest.mark.parametrize("lens", [SINGLES, [(700, 20)], LONG])
def test_pages_16_bytes_off(lens):
    """Pages that start 16 bytes past a 32-byte boundary (any fp32-arithmetic
    path: the tensor-core kernels load 32 bytes at a time), packed queries and
    outputs that start 16 bytes off too."""
    cache = Cache(lens, 16, "bf16", seed=44)
    kp, vp = cache.pages()

    def off(t):
        room = torch.zeros(t.numel() + 8, dtype=t.dtype, device="cuda")
        room[8:] = t.flatten()
        return room[8:].view(t.shape)

    kw = dict(alpha=0.87, W=12, rungs=FIB)
    o, lse = api.sfa_paged_forward(off(cache.q.cuda()), off(kp), off(vp), *cache.meta(), out=off(torch.full_like(cache.q, 7).cuda()),
                                   lse=torch.full((cache.N, HQ), 7.0, device="cuda"), **kw)
    _check(cache, (o, lse), attention64(cache, **kw))
    new = [torch.randn((cache.N, HKV, D), device="cuda").to(torch.bfloat16) for _ in range(2)]
    both = [(kp.clone(), vp.clone()), (off(kp), off(vp))]
    for k_pages, v_pages in both:
        api.sfa_paged_append(*(off(x) for x in new), k_pages, v_pages, *cache.meta())
    for a, b in zip(*both):
        assert torch.equal(a.nan_to_num(5.0), b.nan_to_num(5.0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cache_rows_past_32_bits(dtype):
    """Pages whose elements lie past 2^31 (and bytes past 2^32)."""
    es = 2 if dtype == "bf16" else 4
    rows = (1 << 24) + (1 << 20)          # 128 elements a row: past 2^31 elements
    cache = Cache([(70, 30), (1, 500), (600 if dtype == "f32" else 4100, 0)], 64, dtype, seed=5, num_pages=rows // 64)
    assert int(cache.table[0, 0]) * 64 * HKV * D > 1 << 31 and rows * HKV * D * es > 1 << 32
    kw = dict(alpha=0.87, W=12, rungs=FIB)
    got = _forward(cache, **kw)
    assert got[2] == 0
    _check(cache, got, attention64(cache, tensor_cores=dtype == "bf16", **kw))


# -------------------------------------------------------------------- append


def _append(cache, dtype, *, with_q, norm, packed, theta, k_in=None):
    """Appends cache's new rows to the state before the step; returns the pages,
    q_out and what went in."""
    g = torch.Generator().manual_seed(77)
    if packed:
        x = torch.randn((cache.N, 12 * D), generator=g).to(DT[dtype]).cuda()
        q, k, v = (t.unflatten(-1, (-1, D)) for t in x.split((HQ * D, HKV * D, HKV * D), -1))
    else:
        q, k, v = (torch.randn((cache.N, h, D), generator=g).to(DT[dtype]).cuda() for h in (HQ, HKV, HKV))
    wq = (1 + 0.3 * torch.randn(D, generator=g)).cuda() if norm and with_q else None
    wk = (1 + 0.3 * torch.randn(D, generator=g)).cuda() if norm else None
    kp, vp = cache.pages(rows_before=True)
    before = kp.clone(), vp.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.full((cache.N, HQ, D), 7.0, dtype=DT[dtype], device="cuda") if with_q else None
    r = api.sfa_paged_append(k, v, kp, vp, *cache.meta(), q=q if with_q else None, wq=wq, wk=wk, rope_theta=theta,
                             q_out=q_out, status=status)
    assert (r is None) == (not with_q)
    return (kp, vp, r), before, (q, k, v, wq, wk), api.sfa_read_status(status)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,page", [(ONE, 16), (SINGLES, 16), (SINGLES, 1), (RAGGED, 8), (CHUNK, 64), (MANY, 16),
                                       (LONG, 16), (LONG + [(3900, 11), (0, 0), (5000, 0)], 64)])
@pytest.mark.parametrize("with_q,norm,packed,theta", [(True, True, True, 1e4), (True, False, False, 1e4),
                                                      (False, True, True, 0.0), (False, False, False, 0.0)])
def test_append_against_definition(lens, page, dtype, with_q, norm, packed, theta):
    cache = Cache(lens, page, dtype, seed=2 * len(lens) + page)
    (kp, vp, qo), before, (q, k, v, wq, wk), status = _append(cache, dtype, with_q=with_q, norm=norm, packed=packed,
                                                              theta=theta)
    assert status == 0
    flat = [x.view(-1, HKV, D) for x in (kp, vp, *before)]
    touched = torch.zeros(flat[0].shape[0], dtype=torch.bool, device="cuda")
    at = 0
    for s, (n, c) in enumerate(lens):
        if n:
            rows = cache.slots(s).cuda()[c:]
            touched[rows] = True
            pos = torch.arange(c, c + n)
            want, bound = head64(k[at:at + n].double().cpu(), wk.double().cpu() if norm else None, 1e-6, pos, theta)
            within(flat[0][rows], want, bound + HALF_STEP[dtype] * want.abs() + 1e-30, f"k {s}")
            if not norm and theta == 0:
                assert torch.equal(flat[0][rows], k[at:at + n])
            assert torch.equal(flat[1][rows], v[at:at + n])
            if with_q:
                want, bound = head64(q[at:at + n].double().cpu(), wq.double().cpu() if norm else None, 1e-6, pos, theta)
                within(qo[at:at + n], want, bound + HALF_STEP[dtype] * want.abs() + 1e-30, f"q {s}")
        at += n
    for new, old in zip(flat[:2], flat[2:]):   # nothing else changed, NaN places included
        assert torch.equal(new[~touched].nan_to_num(123.0), old[~touched].nan_to_num(123.0))
    if with_q:
        assert bool((qo[at:] == 7).all())


def test_append_bad_metadata():
    """Bad pages are not stored to, bad positions give zero queries; both are
    reported, and the other tokens are stored."""
    cache = Cache([(20, 3), (4, 0), (6, 10)], 8, "bf16", seed=9)
    cache.table[0, 1] = cache.num_pages + 5
    good = cache.seq.clone()
    cache.seq = torch.tensor([23, 2, 16], dtype=torch.int32)     # sequence 1: positions -2, -1, 0, 1
    (kp, vp, qo), before, (q, k, v, _, _), status = _append(cache, "bf16", with_q=True, norm=False, packed=False, theta=1e4)
    assert status == 0x2
    assert bool((qo[20:22] == 0).all()) and not bool((qo[22:24] == 0).all())
    flat_v, old_v = vp.view(-1, HKV, D), before[1].view(-1, HKV, D)
    touched = torch.zeros(flat_v.shape[0], dtype=torch.bool, device="cuda")
    for s, first, start, n in ((0, 0, 3, 20), (1, 22, 0, 2), (2, 24, 10, 6)):
        for j in range(n):
            pos = start + j
            page = int(cache.table[s, pos // 8])
            if 0 <= page < cache.num_pages:
                row = page * 8 + pos % 8
                touched[row] = True
                assert torch.equal(flat_v[row], v[first + j])
    assert torch.equal(flat_v[~touched].nan_to_num(9.0), old_v[~touched].nan_to_num(9.0))
    assert int(good.sum()) != int(cache.seq.sum())


# ------------------------------------------------------------------ together


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_serving_steps_equal_one_contiguous_pass(dtype):
    """A prompt in two chunks, then single tokens, append and attention each
    step: every token's output against the oracle's attention at the rows that
    the contiguous norm wrote."""
    T, W, alpha = 300, 12, 0.87
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn((2, T, h, D), generator=g).to(DT[dtype]).cuda() for h in (HQ, HKV, HKV))
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g)).cuda() for _ in range(2))
    qh, kh = api.sfa_qk_norm_rope(q, k, wq, wk)
    o_ref, lse_ref = oracle.forward(qh.double().cpu().numpy(), kh.double().cpu().numpy(), v.double().cpu().numpy(), W=W,
                                    rungs=FIB, alpha=alpha, rope_theta=0.0)
    page = 16
    kp, vp = (torch.full((2 * 20, page, HKV, D), float("nan"), dtype=DT[dtype], device="cuda") for _ in range(2))
    table = torch.randperm(40, generator=g).view(2, 20).int().cuda()
    done = [0, 0]
    steps = [(150, 1), (130, 200), (1, 1)] + [(1, 0), (0, 1)] + [(1, 1)] * 17 + [(0, 80)]
    for step in steps:
        cu = torch.tensor([0, step[0], step[0] + step[1]], dtype=torch.int32).cuda()
        seq = torch.tensor([done[0] + step[0], done[1] + step[1]], dtype=torch.int32).cuda()
        rows = [torch.cat([x[s, done[s]:done[s] + step[s]] for s in range(2)]) for x in (q, k, v)]
        qo = api.sfa_paged_append(rows[1], rows[2], kp, vp, table, cu, seq, q=rows[0], wq=wq, wk=wk)
        want_q = torch.cat([qh[s, done[s]:done[s] + step[s]] for s in range(2)])
        assert torch.equal(qo, want_q)
        o, lse = api.sfa_paged_forward(qo, kp, vp, table, cu, seq, alpha=alpha, W=W)
        at = 0
        for s in range(2):
            n = step[s]
            tol = {"bf16": 2e-2, "f32": 1e-4}[dtype]
            assert np.abs(o[at:at + n].double().cpu().numpy() - o_ref[s, done[s]:done[s] + n]).max(initial=0) <= tol
            assert np.abs(lse[at:at + n].double().cpu().numpy() - lse_ref[s, done[s]:done[s] + n]).max(initial=0) <= 1e-4
            done[s] += n
            at += n


@pytest.mark.parametrize("pad_to", [64, 900, 4200])
def test_captured_step_replayed_with_other_lengths(pad_to):
    """One captured step (append, then attention) of a fixed number of token
    rows, replayed with other lengths, tables and inputs; two captured graphs
    replayed at the same time on two streams."""
    S, page, cap = 6, 16, 96
    g = torch.Generator().manual_seed(14)
    rope = api.rope_table(cap * page, "cuda")

    class Step:
        def __init__(self):
            self.q, self.k, self.v = (torch.zeros((pad_to, h, D), dtype=torch.bfloat16, device="cuda") for h in (HQ, HKV, HKV))
            self.kp, self.vp = (torch.full((S * cap, page, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda")
                                for _ in range(2))
            self.table = torch.zeros((S, cap), dtype=torch.int32, device="cuda")
            self.cu, self.seq = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (S + 1, S))
            self.o = torch.zeros((pad_to, HQ, D), dtype=torch.bfloat16, device="cuda")
            self.lse = torch.zeros((pad_to, HQ), device="cuda")
            self.qo = torch.zeros_like(self.q)
            self.graph = torch.cuda.CUDAGraph()
            self.call()
            torch.cuda.synchronize()
            with torch.cuda.graph(self.graph):
                self.call()

        def call(self):
            api.sfa_paged_append(self.k, self.v, self.kp, self.vp, self.table, self.cu, self.seq, q=self.q, q_out=self.qo,
                                 rope=rope)
            api.sfa_paged_forward(self.qo, self.kp, self.vp, self.table, self.cu, self.seq, alpha=1.1, W=12, out=self.o,
                                  lse=self.lse)

    def fill(step, lens, seed):
        cache = Cache(lens, page, "bf16", seed=seed, behind=pad_to - sum(n for n, _ in lens), num_pages=S * cap)
        kp, vp = cache.pages(rows_before=True)
        step.kp.copy_(kp)
        step.vp.copy_(vp)
        step.table.fill_(-1)
        step.table[:, :cache.max_pages] = cache.table.cuda()
        step.cu.copy_(cache.cu)
        step.seq.copy_(cache.seq)
        at = 0
        for s, (n, c) in enumerate(lens):
            step.k[at:at + n] = cache.k[s][c:].cuda()
            step.v[at:at + n] = cache.v[s][c:].cuda()
            at += n
        step.q.copy_(cache.q)
        step.o.fill_(7)
        step.lse.fill_(7)
        return cache

    def check(step, cache):
        # the attention of the rows that the append left in the pages
        used = int(cache.cu[-1])
        for s in range(S):
            rows = cache.slots(s).cuda()
            cache.k[s] = step.kp.view(-1, HKV, D)[rows].cpu()
            cache.v[s] = step.vp.view(-1, HKV, D)[rows].cpu()
        cache.q = step.qo.cpu()
        ref = attention64(cache, alpha=1.1, W=12, rungs=FIB, tensor_cores=True)
        _check(cache, (step.o, step.lse), ref)
        assert used < pad_to

    a, b = Step(), Step()
    sets = [[(1, 40 + 3 * s) for s in range(S)], [(0, 0), (17, 33), (1, 9), (0, 100), (30, 500), (2, 0)]]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(2):
        caches = [fill(step, sets[(turn + i) % 2], 50 + 2 * turn + i) for i, step in enumerate((a, b))]
        torch.cuda.synchronize()
        for step, stream in zip((a, b), streams):
            with torch.cuda.stream(stream):
                step.graph.replay()
        torch.cuda.synchronize()
        for step, cache in zip((a, b), caches):
            check(step, cache)


def test_shared_pages_of_a_common_prefix():
    """Two sequences whose tables share the pages of a common prefix."""
    cache = Cache([(3, 64), (3, 64)], 16, "bf16", seed=21)
    cache.k[1][:64], cache.v[1][:64] = cache.k[0][:64], cache.v[0][:64]
    cache.table[1, :4] = cache.table[0, :4]
    kw = dict(alpha=0.87, W=12, rungs=FIB)
    _check(cache, _forward(cache, **kw), attention64(cache, tensor_cores=True, **kw))


@pytest.mark.parametrize("W", [-1, -2 ** 31, 8 - 2 ** 32])
def test_negative_windows_are_refused(W):
    cache = Cache(SINGLES, 16, "bf16")
    kp, vp = cache.pages()
    with pytest.raises(RuntimeError):
        api.sfa_paged_forward(cache.q.cuda(), kp, vp, *cache.meta(), alpha=0.87, W=W)


@pytest.mark.parametrize("W", [2 ** 31 - 1, 2 ** 31 + 8, 2 ** 40])
def test_windows_wider_than_any_sequence(W):
    """Every row of the sequence, as with a window that just holds it."""
    cache = Cache(RAGGED, 16, "bf16")
    a, b = (_forward(cache, alpha=0.87, W=w, rungs=FIB) for w in (W, 2000))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and a[2] == 0


@pytest.mark.parametrize("lens", [MANY, [(120, 9), (500, 0)], LONG, [(300 + s, 40) for s in range(60)]])
def test_two_calls_at_once(lens):
    """The same entry points on two streams at the same time, each on its own
    cache: the results of one call after the other, bit for bit."""
    caches = [Cache(lens, 16, "bf16", seed=s) for s in (31, 32)]
    wk = torch.linspace(0.5, 1.5, D, device="cuda")
    given = []
    for c in caches:
        new = [torch.cat([x[s][n0:] for s, (_, n0) in enumerate(c.lens)] + [torch.zeros((7, HKV, D), dtype=DT["bf16"])])
               .cuda() for x in (c.k, c.v)]
        given.append((c.q.cuda(), *new, *c.pages(rows_before=True), *c.meta()))
    rope = api.rope_table(4096, "cuda")

    def step(q, k, v, kp, vp, *meta):
        kp, vp = kp.clone(), vp.clone()
        for _ in range(4):
            qo = torch.zeros_like(q)
            api.sfa_paged_append(k, v, kp, vp, *meta, q=q, wq=wk, wk=wk, q_out=qo, rope=rope)
            o, lse = api.sfa_paged_forward(qo, kp, vp, *meta, alpha=0.87, W=12, out=torch.zeros_like(q),
                                           lse=torch.zeros(q.shape[:2], device="cuda"))
        return qo, o, lse

    want = [step(*g) for g in given]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s, g in zip(streams, given):
        with torch.cuda.stream(s):
            got.append(step(*g))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))


def test_lookups_written_by_the_launch_before():
    """Each call reads what the launch right before it wrote: queries, pages and
    metadata, in a captured chain with no other work between them."""
    sets = [Cache([(1, 40 + 7 * s + t) for s in range(6)], 16, "bf16", seed=60 + t, behind=0, num_pages=128) for t in range(2)]
    width = min(c.max_pages for c in sets)
    kw = dict(alpha=0.87, W=12, rungs=FIB)
    want = []
    for c in sets:
        kp, vp = c.pages()
        want.append(api.sfa_paged_forward(c.q.cuda(), kp, vp, *c.meta(), **kw)[0])
    src = [(c.q.cuda(), c.table[:, :width].contiguous().cuda(), c.cu.cuda(), c.seq.cuda()) for c in sets]
    pages = [c.pages() for c in sets]
    q, table, cu, seq = (torch.empty_like(x) for x in src[0])
    outs = [[torch.empty_like(q), torch.empty_like(q)] for _ in range(8)]

    def chain():
        for o in outs:
            for t in range(2):
                for dst, x in zip((table, cu, q, seq), (src[t][1], src[t][2], src[t][0], src[t][3])):
                    dst.copy_(x)
                api.sfa_paged_forward(q, *pages[t], table, cu, seq, out=o[t], need_lse=False, **kw)

    chain()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for _ in range(5):
        for o in outs:
            o[0].fill_(7), o[1].fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o[t], want[t]) for o in outs for t in range(2))


@pytest.mark.parametrize("lens,behind", [([(304, 5)], 0), ([(304, 5)], 1), ([(2, 30 + 5 * s) for s in range(152)], 0),
                                         ([(2, 30 + 5 * s) for s in range(153)], 0),
                                         ([(1, 0)] * 20 + [(290, 100)] + [(1, 5)] * 9, 2), ([(500, 9)], 0),
                                         ([(2428, 40)], 0), ([(2432, 40)], 0), ([(3644, 9)], 0), ([(3648, 9)], 0)])
def test_where_the_kernels_change(lens, behind):
    """Token rows on both sides of where the kernels take over from one another."""
    cache = Cache(lens, 16, "bf16", seed=70 + len(lens) + behind, behind=behind)
    kw = dict(alpha=0.87, W=12, rungs=FIB)
    _check(cache, _forward(cache, **kw), attention64(cache, tensor_cores=True, **kw))


def test_more_bad_values_than_a_block_lists_in_short_chunks():
    """The same in many short chunks, whose blocks ask for their slots."""
    S, n, page = 75, 600, 64
    each = -(-n // page)
    g = torch.Generator("cuda").manual_seed(5)
    kp, vp = (torch.randn((S * each, page, HKV, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    vp.view(-1, HKV, D)[::4, :, 11] = float("nan")
    q = torch.randn((S * n, HQ, D), generator=g, device="cuda").to(torch.bfloat16)
    table = torch.arange(S * each, dtype=torch.int32, device="cuda").view(S, each)
    cu = torch.arange(0, S * n + 1, n, dtype=torch.int32, device="cuda")
    seq = torch.full((S,), n, dtype=torch.int32, device="cuda")
    o, lse = api.sfa_paged_forward(q, kp, vp, table, cu, seq, alpha=1.0, W=0, rungs=())
    own = vp.view(S, each * page, HKV, D)[:, :n].reshape(S * n, HKV, D).repeat_interleave(HQ // HKV, 1)
    assert torch.equal(o.isnan(), own.isnan()) and torch.equal(o.nan_to_num(9.0), own.nan_to_num(9.0))
    assert bool(lse.isfinite().all())


def test_short_chunks_of_one_call():
    """Ragged chunks over several rounds of blocks, three of them against the
    definition."""
    rng = np.random.default_rng(9)
    lens = [(int(rng.integers(1, 900)), int(rng.integers(0, 900))) for _ in range(60)]
    cache = Cache(lens, 64, "bf16", seed=90)
    kw = dict(alpha=0.87, W=12, rungs=FIB)
    o, lse, status = _forward(cache, **kw)
    assert status == 0
    for s in (0, 17, 59):
        a, b = int(cache.cu[s]), int(cache.cu[s + 1])
        one = Cache([lens[s]], 64, "bf16", behind=0)
        one.k, one.v, one.q = [cache.k[s]], [cache.v[s]], cache.q[a:b]
        ref = attention64(one, tensor_cores=True, **kw)
        within(o[a:b], ref[0], ref[2], f"o of sequence {s}")
        within(lse[a:b], ref[1], ref[3], f"lse of sequence {s}")


@pytest.mark.parametrize("lens", [MANY, [(120, 9), (500, 0)], [(4, 30)] * 500, LONG, [(300 + s, 40) for s in range(60)]])
def test_launches_in_a_row_wait_for_one_another(lens):
    """Append and attention in turn on one buffer of queries, nothing between them:
    an append that ran into the attention before it would change what that reads."""
    cache = Cache(lens, 16, "bf16", seed=95)
    kp, vp = cache.pages()
    meta = cache.meta()
    new = [torch.cat([x[s][c:] for s, (_, c) in enumerate(lens)] + [torch.zeros((7, HKV, D), dtype=DT["bf16"])]).cuda()
           for x in (cache.k, cache.v)]
    qs = [cache.q.cuda(), cache.q.flip(0).contiguous().cuda()]
    rope = api.rope_table(4096, "cuda")
    qo = torch.zeros_like(qs[0])
    outs = [torch.zeros_like(qo) for _ in range(12)]
    kw = dict(alpha=0.87, W=12, rungs=FIB, need_lse=False)

    def step(q, o):
        api.sfa_paged_append(*new, kp, vp, *meta, q=q, q_out=qo, rope=rope)
        api.sfa_paged_forward(qo, kp, vp, *meta, out=o, **kw)

    want = []
    for q in qs:
        o = torch.zeros_like(qo)
        step(q, o)
        torch.cuda.synchronize()
        want.append(o)
    assert not torch.equal(*want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i, o in enumerate(outs):
            step(qs[i % 2], o)
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want[i % 2]) for i, o in enumerate(outs))
