"""The residual's addition and the RMS norm of rows (sfa_add_rms_norm), to the
rows' type and to 8 bits, its backward pass, and rows to 8 bits as they are,
against 64 bits with derived bounds."""
import pytest
import torch

from fibonacci_spaced_sparse_gb300 import api
from _fp8 import FP8, TOP, codes, row_scales
from _paged import DT, HALF_STEP, U, within

pytestmark = pytest.mark.gpu

EPS = 1e-6
# every split of a row over lanes and warps, whole and ragged
DIMS = [8, 64, 72, 256, 264, 320, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384]


def _rows(N, dim, dtype, seed=0, size=1.0):
    g = torch.Generator().manual_seed(seed + N + dim)
    return (size * torch.randn((N, dim), generator=g)).to(DT[dtype])


def _weight(dim, seed=0):
    return 1 + 0.3 * torch.randn(dim, generator=torch.Generator().manual_seed(seed + dim))


def norm64(h, w, eps=EPS):
    h = h.double()
    return h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps) * w.double()


# The mean of squares: a lane sums at most 32 of them, five shuffles and 16 warps
# follow, with the product by 1 / dim (rounded) and eps below 60 u; the root
# halves that and adds two units in the last place, two products two more.
Y_ERROR = 40 * U


def _check_y(y, h, w, dtype, eps=EPS):
    want = norm64(h, w, eps)
    within(y, want, (Y_ERROR + HALF_STEP[dtype]) * want.abs() + 1e-38)


def _check_fp8(y8, scale, want, rel):
    """8-bit rows of the 64-bit values `want`, which the kernel has to `rel`."""
    y8, scale = y8.cpu(), scale.double().cpu()
    s = row_scales(want)
    assert bool(((scale - s).abs() <= (rel + 3 * U) * s).all())
    got = y8.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), ~fine)
    off = (got * scale[..., None] - want).abs()
    bound = (2.0 ** -4 + rel + 4 * U) * want.abs() + 2.0 ** -10 * scale[..., None]
    assert bool((off <= bound)[fine].all())
    most = torch.where(fine, got.abs(), 0.0).amax(-1)
    assert bool(((most == TOP) | (s <= 2.0 ** -126)).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("N", [1, 7, 8, 133])
def test_forward_against_definition(N, dim, dtype):
    x, r, w = _rows(N, dim, dtype), _rows(N, dim, dtype, 1, 3.0), _weight(dim)
    h, y = api.sfa_add_rms_norm(x.cuda(), r.cuda(), w.cuda())
    want_h = (x.float() + r.float()).to(DT[dtype])
    assert torch.equal(h.cpu(), want_h)
    _check_y(y, want_h, w, dtype)
    h8, y8, scale = api.sfa_add_rms_norm(x.cuda(), r.cuda(), w.cuda(), fp8=True)
    assert torch.equal(h8, h) and y8.dtype == FP8 and y8.shape == x.shape and scale.shape == (N,)
    _check_fp8(y8, scale, norm64(want_h, w), Y_ERROR)
    same, y = api.sfa_add_rms_norm(x.cuda(), None, w.cuda(), eps=1e-3)
    assert torch.equal(same.cpu(), x)
    _check_y(y, x, w, dtype, 1e-3)
    x8, s8 = api.sfa_quantize_rows_fp8(x.cuda())
    _check_fp8(x8, s8, x.double(), 0.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows(dtype):
    for N, dim in ((20011, 512), (3001, 2048), (70001, 64)):
        x, r, w = _rows(N, dim, dtype), _rows(N, dim, dtype, 1), _weight(dim)
        h, y = api.sfa_add_rms_norm(x.cuda(), r.cuda(), w.cuda())
        assert torch.equal(h.cpu(), (x.float() + r.float()).to(DT[dtype]))
        _check_y(y, h.cpu(), w, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_shapes_and_outputs(dtype):
    dim, w = 320, _weight(320)
    wide = _rows(6 * 5, 3 * dim, dtype).cuda().view(6, 5, 3 * dim)
    x, r = wide[..., :dim], wide[..., dim:2 * dim]
    want = api.sfa_add_rms_norm(x.contiguous(), r.contiguous(), w.cuda())
    got = api.sfa_add_rms_norm(x, r, w.cuda())
    assert got[0].shape == x.shape and all(torch.equal(a, b) for a, b in zip(got, want))
    part = api.sfa_add_rms_norm(x[:, 2], r[:, 2], w.cuda(), fp8=True)
    assert part[2].shape == (6,) and torch.equal(part[0], want[0][:, 2])
    one = api.sfa_add_rms_norm(x[1, 1], r[1, 1], w.cuda())
    assert one[1].shape == (dim,) and torch.equal(one[1], want[1][1, 1])
    # the sum over x or the residual itself, and given outputs between guards
    for over in (0, 1):
        a = [x.contiguous().clone(), r.contiguous().clone()]
        room = torch.full((32, dim), 7.0, dtype=DT[dtype], device="cuda")
        y = room[1:31].view(6, 5, dim)
        h, got_y = api.sfa_add_rms_norm(*a, w.cuda(), out=(a[over], y))
        assert h.data_ptr() == a[over].data_ptr() and got_y.data_ptr() == y.data_ptr()
        assert torch.equal(h, want[0]) and torch.equal(y, want[1])
        assert bool((room[0] == 7).all()) and bool((room[31] == 7).all())
        assert torch.equal(a[1 - over], (x, r)[1 - over])


@pytest.mark.parametrize("dim", [320, 1024, 4096])
def test_rows_that_are_not_ordinary(dim):
    """Zeros, values near the ends of the range, infinity and NaN: each row by
    itself, none of it reaching another."""
    w = _weight(dim)
    x = _rows(40, dim, "f32")
    clean = api.sfa_add_rms_norm(x.cuda(), None, w.cuda(), fp8=True)
    plain = api.sfa_quantize_rows_fp8(x.cuda())
    odd = x.clone()
    odd[3] = 0
    odd[5] *= 1e-30
    odd[7, 11] = float("inf")
    odd[9, 8] = float("nan")
    odd[11] *= 1e30
    odd[13] = 0
    odd[13, 4] = 1e-40
    same = [i for i in range(40) if i not in (3, 5, 7, 9, 11, 13)]
    got = api.sfa_add_rms_norm(odd.cuda(), None, w.cuda(), fp8=True)
    as_is = api.sfa_quantize_rows_fp8(odd.cuda())
    for a, b in ((got[1:], clean[1:]), (as_is, plain)):
        assert torch.equal(a[0].view(torch.uint8)[same], b[0].view(torch.uint8)[same]) and torch.equal(a[1][same], b[1][same])
    _check_fp8(as_is[0], as_is[1], odd.double(), 0.0)
    y = norm64(odd, w)
    rows = [3, 5, 13]
    _check_fp8(got[1][rows], got[2][rows], y[rows], Y_ERROR)
    assert bool(torch.isnan(got[1][9].float()).all())                    # a NaN makes the mean NaN
    inf = got[1][7].float().cpu()                                        # x / infinity = 0, infinity / infinity
    assert bool(torch.isnan(inf[11])) and bool((inf[torch.arange(dim) != 11] == 0).all())
    _, same_type = api.sfa_add_rms_norm(odd.cuda(), None, w.cuda(), eps=0.0)
    assert bool(torch.isnan(same_type[3]).all())                         # 0 / 0
    within(same_type[same], norm64(odd[same], w, 0.0), (Y_ERROR + U) * norm64(odd[same], w, 0.0).abs())


def test_no_rows():
    w = torch.ones(64, device="cuda")
    before = api.launch_count()
    for dt in (torch.bfloat16, torch.float32):
        x = torch.empty((0, 64), dtype=dt, device="cuda")
        h, y8, s = api.sfa_add_rms_norm(x, x, w, fp8=True)
        assert h.shape == (0, 64) and y8.shape == (0, 64) and s.shape == (0,)
        assert api.sfa_quantize_rows_fp8(x)[1].shape == (0,)
        dx, dw = api.sfa_add_rms_norm_backward(x, w, x, x, out=(torch.empty_like(x), torch.full((64,), 7.0, device="cuda")))
        assert dx.shape == (0, 64) and bool((dw == 0).all())
    assert api.launch_count() == before


# ------------------------------------------------------------------ backward


def backward64(h, w, dy, dh=None, eps=EPS):
    """(dx, dw, bound of dx, bound of dw) from the formula.  The bounds: r is known
    to 40 u (above); the mean of g n is a sum like that of squares, to 60 u of the
    mean of |g n|, with its three products and r's square below 160 u in all; the
    rest is a few roundings.  dw: each term to 45 u and a sum of at most (rows of a
    warp) + 8 + 16 + 8 additions in a row."""
    h, w, dy = h.double(), w.double(), dy.double()
    r = 1 / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
    n, g = h * r, dy * w
    dx = r * (g - n * (g * n).mean(-1, keepdim=True))
    size = r * (g.abs() + n.abs() * (g * n).abs().mean(-1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double()
        size = size + dh.double().abs()
    rows = -(-h.shape[0] // 152) + 40  # (wide rows: one a block at a time, a block a SM)
    return dx, (dy * n).sum(0), 200 * U * size, (45 + rows) * U * (dy * n).abs().sum(0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("N,with_dh", [(1, True), (8, False), (67, True), (1003, False)])
def test_backward_against_formula(N, with_dh, dim, dtype):
    if N * dim > 9 << 20:
        N = 301
    h, dy, dh = _rows(N, dim, dtype, 0, 2.0), _rows(N, dim, dtype, 1), _rows(N, dim, dtype, 2) if with_dh else None
    w = _weight(dim)
    dx, dw = api.sfa_add_rms_norm_backward(h.cuda(), w.cuda(), dy.cuda(), dh.cuda() if with_dh else None)
    want, want_w, bx, bw = backward64(h, w, dy, dh)
    within(dx, want, bx + HALF_STEP[dtype] * want.abs() + 1e-38, "dx")
    within(dw, want_w, bw + 1e-38, "dw")
    again = api.sfa_add_rms_norm_backward(h.cuda(), w.cuda(), dy.cuda(), dh.cuda() if with_dh else None)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("N,dim", [(9, 24), (70, 264), (5, 1032)])
def test_backward_against_differences(N, dim):
    """The formula's gradient and the kernel's against central differences of a
    scalar loss through the forward's definition in 64 bits."""
    h, dy, dh, w = _rows(N, dim, "f32"), _rows(N, dim, "f32", 1), _rows(N, dim, "f32", 2), _weight(dim)
    dx, dw = api.sfa_add_rms_norm_backward(h.cuda(), w.cuda(), dy.cuda(), dh.cuda())

    def loss(hh, ww):
        return float((norm64(hh, ww) * dy.double()).sum() + (hh.double() * dh.double()).sum())

    g = torch.Generator().manual_seed(3)
    for _ in range(12):
        i, j, e = int(torch.randint(N, (1,), generator=g)), int(torch.randint(dim, (1,), generator=g)), 1e-4
        up, down = h.double().clone(), h.double().clone()
        up[i, j] += e
        down[i, j] -= e
        slope = (loss(up, w) - loss(down, w)) / (2 * e)
        assert abs(slope - float(dx[i, j])) <= 1e-5 * (1 + abs(slope))      # e^2 of the third derivative, 2^-52 / e of the loss
        up, down = w.double().clone(), w.double().clone()
        up[j] += e
        down[j] -= e
        slope = (loss(h, up) - loss(h, down)) / (2 * e)
        assert abs(slope - float(dw[j])) <= 1e-5 * (1 + abs(slope))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_many_rows_in_place_and_given_buffers(dtype):
    for N, dim in ((20011, 512), (70001, 64), (2503, 4096), (2441, 520), (1301, 2056), (307, 8192), (309, 12000)):
        h, dy, dh, w = _rows(N, dim, dtype), _rows(N, dim, dtype, 1), _rows(N, dim, dtype, 2), _weight(dim)
        want, want_w, bx, bw = backward64(h, w, dy, dh)
        own = dh.cuda()
        need = 4 * dim * 760
        room = torch.full((dim + 8,), 7.0, device="cuda")
        ws = torch.full((need + 256,), 0xff, dtype=torch.uint8, device="cuda")
        dx, dw = api.sfa_add_rms_norm_backward(h.cuda(), w.cuda(), dy.cuda(), own, out=(own, room[4:4 + dim]), workspace=ws[:need])
        assert dx.data_ptr() == own.data_ptr()
        within(dx, want, bx + HALF_STEP[dtype] * want.abs(), "dx")
        within(dw, want_w, bw, "dw")
        assert bool((room[:4] == 7).all()) and bool((room[4 + dim:] == 7).all()) and bool((ws[need:] == 0xff).all())


@pytest.mark.parametrize("residual", [True, False])
def test_autograd(residual):
    N, dim = 37, 320
    w = _weight(dim).cuda().requires_grad_()
    x = _rows(N, dim, "f32").cuda().requires_grad_()
    r = _rows(N, dim, "f32", 1).cuda().requires_grad_() if residual else None
    a, b = _rows(N, dim, "f32", 2).cuda(), _rows(N, dim, "f32", 3).cuda()
    for use_h, use_y in ((True, True), (False, True), (True, False)) if residual else ((False, True),):
        for t in (x, r, w):
            if t is not None:
                t.grad = None
        out = api.AddRMSNorm.apply(x, r, w)
        h, y = out if residual else (None, out)
        loss = sum(([(h * a).sum()] if use_h else []) + ([(y * b).sum()] if use_y else []))
        loss.backward()
        hh = (x + r if residual else x).detach()
        want, want_w, bx, bw = backward64(hh.cpu(), w.detach().cpu(), (b if use_y else torch.zeros_like(b)).cpu(),
                                          a.cpu() if use_h else None)
        within(x.grad, want, bx + 2 * U * want.abs() + 1e-30)
        if residual:
            assert torch.equal(x.grad, r.grad)
        if use_y:
            within(w.grad, want_w, bw + 1e-30)


@pytest.mark.parametrize("N,dim,dtype", [(5, 512, "bf16"), (700, 512, "bf16"), (3000, 4096, "bf16"), (700, 320, "f32")])
def test_captured_steps_in_a_row(N, dim, dtype):
    """Forward and backward launched one after another on the same buffers, captured
    and replayed with other inputs, on a stream of their own."""
    w = _weight(dim).cuda()
    given = [[_rows(N, dim, dtype, 10 * i + j).cuda() for j in range(3)] for i in range(2)]
    bufs = [torch.zeros((N, dim), dtype=DT[dtype], device="cuda") for _ in range(5)]
    x, r, dh, h, y = bufs
    y8, s = torch.zeros((N, dim), dtype=torch.uint8, device="cuda").view(FP8), torch.zeros(N, device="cuda")
    dx, dw = torch.zeros((N, dim), dtype=DT[dtype], device="cuda"), torch.zeros(dim, device="cuda")
    ws = torch.zeros(4 * dim * 760, dtype=torch.uint8, device="cuda")

    def step():
        api.sfa_add_rms_norm(x, r, w, out=(h, y))
        api.sfa_add_rms_norm_backward(h, w, y, dh, out=(dx, dw), workspace=ws)
        api.sfa_add_rms_norm(dx, h, w, out=(h, y8, s), fp8=True)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
        step()
    want = []
    for i in range(2):
        for a, b in zip((x, r, dh), given[i]):
            a.copy_(b)
        step()
        step()
        torch.cuda.synchronize()
        want.append([t.view(torch.uint8).clone() for t in (h, y, y8, s, dx, dw)])
    for i in (0, 1, 0):
        for a, b in zip((x, r, dh), given[i]):
            a.copy_(b)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b) for a, b in zip((h, y, y8, s, dx, dw), want[i]))


def test_one_tensor_as_both_addends():
    """x beside itself: h = 2 x (exact), and the leaf gets the gradient twice."""
    x, w = _rows(37, 320, "f32").cuda().requires_grad_(), _weight(320).cuda()
    a, b = _rows(37, 320, "f32", 2).cuda(), _rows(37, 320, "f32", 3).cuda()
    h, y = api.AddRMSNorm.apply(x, x, w)
    assert torch.equal(h, 2 * x)
    ((h * a).sum() + (y * b).sum()).backward()
    dx, _ = api.sfa_add_rms_norm_backward(h.detach(), w, b, a)
    assert torch.equal(x.grad, 2 * dx)


def test_calls_at_once():
    """Backward passes on two streams, each with a scratch of its own."""
    w = _weight(512).cuda()
    args = [(_rows(30000, 512, "bf16", i).cuda(), w, _rows(30000, 512, "bf16", 5 + i).cuda()) for i in range(2)]
    want = [api.sfa_add_rms_norm_backward(*a) for a in args]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in args]
    got = [[] for _ in args]
    for _ in range(5):
        for i, a in enumerate(args):
            got[i].append(api.sfa_add_rms_norm_backward(*a, stream=sides[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, y) for g in got[i] for x, y in zip(g, want[i]))


def test_other_stream():
    x, r, w = _rows(3000, 512, "bf16").cuda(), _rows(3000, 512, "bf16", 1).cuda(), _weight(512).cuda()
    want = api.sfa_add_rms_norm(x, r, w, fp8=True)
    back = api.sfa_add_rms_norm_backward(want[0], w, x, r)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = api.sfa_add_rms_norm(x, r, w, fp8=True, stream=side)
    got_back = api.sfa_add_rms_norm_backward(want[0], w, x, r, stream=side)
    rows = api.sfa_quantize_rows_fp8(x, stream=side)
    side.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip((*got, *got_back), (*want, *back)))
    assert torch.equal(codes(x.cpu().double() / rows[1].cpu().double()[:, None]).float().abs().amax(-1), torch.full((3000,), TOP))


def test_rows_past_32_bits():
    """Rows whose elements lie past 2^31."""
    dim, N = 512, (1 << 22) + 100
    x = torch.zeros((N, dim), dtype=torch.bfloat16, device="cuda")
    tail = _rows(90, dim, "bf16")
    x[-90:] = tail.cuda()
    w = _weight(dim)
    h, y = api.sfa_add_rms_norm(x, x, w.cuda())
    assert torch.equal(h[-90:].cpu(), tail + tail)
    _check_y(y[-90:], h[-90:].cpu(), w, "bf16")
    assert not bool(y[:-90].any())
    dx, dw = api.sfa_add_rms_norm_backward(h, w.cuda(), x)
    want, want_w, bx, bw = backward64(h[-90:].cpu(), w, tail)
    within(dx[-90:], want, bx + HALF_STEP["bf16"] * want.abs())
    within(dw, want_w, bw)
