"""RMS norm of queries and keys with the rotation (sfa_qk_norm_rope) and its
backward pass against the formulas in 64 bits, element by element, with bounds
derived from the kernels' fp32 arithmetic (tests/_paged.py)."""
import pytest
import torch

from fibonacci_spaced_sparse_gb300 import api
from oracle import oracle
from _paged import DT, HALF_STEP, HKV, HQ, D, U, head64, norm64, pair_size, rotate64, within

pytestmark = pytest.mark.gpu


def _draw(B, T, dtype, packed, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    if packed:
        x = (scale * torch.randn((B, T, 12 * D), generator=g)).to(DT[dtype]).cuda()
        q, k = x[..., :HQ * D].unflatten(-1, (HQ, D)), x[..., HQ * D:10 * D].unflatten(-1, (HKV, D))
    else:
        q, k = ((scale * torch.randn((B, T, h, D), generator=g)).to(DT[dtype]).cuda() for h in (HQ, HKV))
    wq, wk = (1 + 0.3 * torch.randn(D, generator=g)).cuda(), (0.5 + 0.3 * torch.randn(D, generator=g)).cuda()
    return q, k, wq, wk, g


def _flat(x):
    return x.double().cpu().reshape(-1, x.shape[-2], D)


def _check_fwd(out, x, w, eps, pos, theta, dtype, what):
    want, bound = head64(_flat(x), w.double().cpu(), eps, pos, theta)
    within(out.reshape(-1, *out.shape[-2:]), want, bound + HALF_STEP[dtype] * want.abs() + 1e-30, what)


def _check_bwd(got, x, w, up, eps, pos, theta, dtype, what):
    dx, dw = got
    x, w, up = _flat(x), w.double().cpu(), _flat(up)
    _, n, r = norm64(x, w, eps)
    g = rotate64(up, pos, theta, back=True) if theta > 0 else up
    wg = w * g
    m = (wg * n).mean(-1, keepdim=True)
    want = r * (wg - n * m)
    # n carries 40 u, g 4 u of its pair; the mean sums 64 products of them
    gs = pair_size(up) if theta > 0 else up.abs()
    size = r * (w.abs() * gs + 2 * n.abs() * (w.abs() * gs * n.abs()).mean(-1, keepdim=True))
    within(dx.reshape(want.shape), want, 120 * U * size + HALF_STEP[dtype] * want.abs() + 1e-30, what + " dx")
    # a sum of len products: a thread's, a block's and the blocks' chains, each at most this long
    tokens = x.shape[0]
    chain = 2 * (tokens // (16 * 608) + 1) + 64 + 19 + 32 + 48
    want_w = (g * n).sum((0, 1))
    within(dw, want_w, chain * U * (gs * n.abs()).sum((0, 1)) + 1e-30, what + " dw")


CASES = [(1, 1, "bf16", False), (1, 1, "f32", True), (2, 3, "f32", False), (3, 17, "bf16", True), (1, 255, "bf16", False),
         (5, 64, "f32", True), (2, 1021, "bf16", True), (257, 1, "bf16", True), (1, 16, "bf16", False),
         (1, 64, "f32", False), (8, 8, "bf16", True), (5, 13, "bf16", False), (65, 1, "f32", True)]


@pytest.mark.parametrize("theta", [1e4, 0.0])
@pytest.mark.parametrize("B,T,dtype,packed", CASES)
def test_forward_against_formula(B, T, dtype, packed, theta):
    q, k, wq, wk, _ = _draw(B, T, dtype, packed, seed=B + T)
    qh, kh = api.sfa_qk_norm_rope(q, k, wq, wk, rope_theta=theta)
    pos = torch.arange(T).repeat(B)
    _check_fwd(qh, q, wq, 1e-6, pos, theta, dtype, "q")
    _check_fwd(kh, k, wk, 1e-6, pos, theta, dtype, "k")
    assert qh.is_contiguous() and kh.is_contiguous()


@pytest.mark.parametrize("theta", [1e4, 0.0])
@pytest.mark.parametrize("B,T,dtype,packed", CASES)
def test_backward_against_formula(B, T, dtype, packed, theta):
    q, k, wq, wk, g = _draw(B, T, dtype, packed, seed=3 * B + T)
    up = [torch.randn((B, T, h, D), generator=g).to(DT[dtype]).cuda() for h in (HQ, HKV)]
    dq, dk, dwq, dwk = api.sfa_qk_norm_rope_backward(q, k, wq, wk, *up, rope_theta=theta)
    pos = torch.arange(T).repeat(B)
    _check_bwd((dq, dwq), q, wq, up[0], 1e-6, pos, theta, dtype, "q")
    _check_bwd((dk, dwk), k, wk, up[1], 1e-6, pos, theta, dtype, "k")


def test_many_tokens_more_than_the_blocks_of_one_pass():
    """More than 608 x 16 tokens: blocks take several groups of tokens."""
    q, k, wq, wk, g = _draw(3, 3571, "bf16", True, seed=5)
    up = [torch.randn((3, 3571, h, D), generator=g).to(torch.bfloat16).cuda() for h in (HQ, HKV)]
    first = api.sfa_qk_norm_rope_backward(q, k, wq, wk, *up)
    again = api.sfa_qk_norm_rope_backward(q, k, wq, wk, *up)
    assert all(torch.equal(a, b) for a, b in zip(first, again))  # sums in a fixed order
    pos = torch.arange(3571).repeat(3)
    _check_bwd((first[0], first[2]), q, wq, up[0], 1e-6, pos, 1e4, "bf16", "q")
    _check_bwd((first[1], first[3]), k, wk, up[1], 1e-6, pos, 1e4, "bf16", "k")


@pytest.mark.parametrize("eps,scale", [(1e-5, 1e-3), (1e-6, 300.0), (0.0, 1.0)])
def test_eps_and_scales(eps, scale):
    q, k, wq, wk, g = _draw(2, 33, "f32", False, seed=9, scale=scale)
    up = [torch.randn((2, 33, h, D), generator=g).cuda() for h in (HQ, HKV)]
    qh, kh = api.sfa_qk_norm_rope(q, k, wq, wk, eps=eps)
    eps = float(torch.tensor(eps, dtype=torch.float32))
    pos = torch.arange(33).repeat(2)
    _check_fwd(qh, q, wq, eps, pos, 1e4, "f32", "q")
    _check_fwd(kh, k, wk, eps, pos, 1e4, "f32", "k")
    got = api.sfa_qk_norm_rope_backward(q, k, wq, wk, *up, eps=eps)
    _check_bwd((got[0], got[2]), q, wq, up[0], eps, pos, 1e4, "f32", "q")
    _check_bwd((got[1], got[3]), k, wk, up[1], eps, pos, 1e4, "f32", "k")


def test_zero_rows_and_bad_values_stay_in_their_row():
    q, k, wq, wk, g = _draw(1, 40, "bf16", False, seed=11)
    clean = api.sfa_qk_norm_rope(q, k, wq, wk)
    q[0, 7, 3] = 0
    q[0, 9, 0, 5] = float("nan")
    k[0, 12, 1, 63] = float("inf")
    qh, kh = api.sfa_qk_norm_rope(q, k, wq, wk)
    assert bool((qh[0, 7, 3] == 0).all())
    assert bool(qh[0, 9, 0].isnan().all()) and bool(kh[0, 12, 1].isnan().any())
    mask_q, mask_k = torch.ones_like(qh, dtype=torch.bool), torch.ones_like(kh, dtype=torch.bool)
    mask_q[0, 7, 3] = mask_q[0, 9, 0] = False
    mask_k[0, 12, 1] = False
    assert torch.equal(qh[mask_q], clean[0][mask_q]) and torch.equal(kh[mask_k], clean[1][mask_k])


def test_positions_of_single_tokens_and_bad_ones():
    """Positions given per token; one outside the table reads nothing, gives
    zeros, no gradient and the status bit."""
    B = 37
    q, k, wq, wk, g = _draw(B, 1, "f32", True, seed=13)
    rope = api.rope_table(5000, "cuda")
    rows = rope.shape[0]
    pos = torch.randint(0, rows, (B, 1), generator=g)
    pos[3], pos[5] = 0, rows - 1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = dict(positions=pos.int().cuda(), rope=rope, status=status)
    qh, kh = api.sfa_qk_norm_rope(q, k, wq, wk, **call)
    assert api.sfa_read_status(status) == 0
    _check_fwd(qh, q, wq, 1e-6, pos.view(-1), 1e4, "f32", "q")
    _check_fwd(kh, k, wk, 1e-6, pos.view(-1), 1e4, "f32", "k")
    bad = pos.clone()
    bad[0], bad[9], bad[20] = -1, rows, 1 << 30
    call["positions"] = bad.int().cuda()
    qb, kb = api.sfa_qk_norm_rope(q, k, wq, wk, **call)
    assert api.sfa_read_status(status) == 0x2
    keep = torch.ones(B, dtype=torch.bool)
    keep[[0, 9, 20]] = False
    assert torch.equal(qb[keep], qh[keep]) and torch.equal(kb[keep], kh[keep])
    assert bool((qb[~keep] == 0).all()) and bool((kb[~keep] == 0).all())
    up = [torch.randn((B, 1, h, D), generator=g).cuda() for h in (HQ, HKV)]
    status.zero_()
    got = api.sfa_qk_norm_rope_backward(q, k, wq, wk, *up, **call)
    assert api.sfa_read_status(status) == 0x2
    assert bool((got[0][~keep] == 0).all()) and bool((got[1][~keep] == 0).all())
    kp = pos.view(-1)[keep]
    _check_bwd((got[0][keep], got[2]), q[keep], wq, up[0][keep], 1e-6, kp, 1e4, "f32", "q")
    _check_bwd((got[1][keep], got[3]), k[keep], wk, up[1][keep], 1e-6, kp, 1e4, "f32", "k")


def test_empty_calls():
    q, k, wq, wk, _ = _draw(2, 4, "bf16", False)
    qh, kh = api.sfa_qk_norm_rope(q[:0], k[:0], wq, wk)
    assert qh.shape == (0, 4, HQ, D) and kh.shape == (0, 4, HKV, D)
    got = api.sfa_qk_norm_rope_backward(q[:0], k[:0], wq, wk, q[:0], k[:0])
    assert got[0].shape == (0, 4, HQ, D) and bool((got[2] == 0).all()) and bool((got[3] == 0).all())


def test_gradient_against_differences():
    """dx along random directions and dw against central differences of the
    64-bit forward (step 1e-5: truncation 1e-10, cancellation 1e-11)."""
    B, T = 2, 9
    q, k, wq, wk, g = _draw(B, T, "f32", False, seed=17)
    up = [torch.randn((B, T, h, D), generator=g) for h in (HQ, HKV)]
    got = api.sfa_qk_norm_rope_backward(q, k, wq, wk, up[0].cuda(), up[1].cuda())
    pos = torch.arange(T).repeat(B)
    for x, w, u, dx, dw in ((q, wq, up[0], got[0], got[2]), (k, wk, up[1], got[1], got[3])):
        x, w, u = _flat(x), w.double().cpu(), _flat(u)
        loss = lambda x, w: float((head64(x, w, 1e-6, pos, 1e4)[0] * u).sum())  # noqa: E731
        for _ in range(4):
            a, b = torch.randn(x.shape, generator=g).double(), torch.randn(D, generator=g).double()
            h = 1e-5
            num = (loss(x + h * a, w + h * b) - loss(x - h * a, w - h * b)) / (2 * h)
            ana = float((_flat(dx) * a).sum() + (dw.double().cpu() * b).sum())
            size = float((_flat(dx) * a).abs().sum() + (dw.double().cpu() * b).abs().sum())
            assert abs(num - ana) <= 1e-6 * size, (num, ana)


def test_other_stream_and_graph_replay():
    """Outputs allocated and written on a given stream; forward and backward
    captured once and replayed on new inputs."""
    q, k, wq, wk, g = _draw(4, 130, "bf16", False, seed=19)
    up = [torch.randn((4, 130, h, D), generator=g).to(torch.bfloat16).cuda() for h in (HQ, HKV)]
    want = (*api.sfa_qk_norm_rope(q, k, wq, wk), *api.sfa_qk_norm_rope_backward(q, k, wq, wk, *up))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (*api.sfa_qk_norm_rope(q, k, wq, wk, stream=side), *api.sfa_qk_norm_rope_backward(q, k, wq, wk, *up, stream=side))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    q2, k2 = torch.zeros_like(q), torch.zeros_like(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = (*api.sfa_qk_norm_rope(q2, k2, wq, wk), *api.sfa_qk_norm_rope_backward(q2, k2, wq, wk, *up))
    q2.copy_(q)
    k2.copy_(k)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_training_chain_against_the_oracle():
    """QKNormRope and SparseAttention together in fp32: outputs and every
    gradient (inputs, norm weights, theta) against the oracle's attention at
    rotated rows and the norm's formulas in 64 bits.  The bounds are the fp32
    path's (1e-4 of max(1, size)); the weights' gradients sum 2 x 90 tokens."""
    B, T, W = 2, 90, 8
    q, k, wq, wk, g = _draw(B, T, "f32", True, seed=23)
    q, k = q.detach().requires_grad_(), k.detach().requires_grad_()
    wq.requires_grad_()
    wk.requires_grad_()
    v = torch.randn((B, T, HKV, D), generator=g).cuda().requires_grad_()
    theta = torch.tensor(0.21, device="cuda", requires_grad=True)
    dO = torch.randn((B, T, HQ, D), generator=g)
    qh, kh = api.QKNormRope.apply(q, k, wq, wk)
    o = api.SparseAttention.apply(qh, kh, v, theta, W, api.FIBONACCI_BASE, 0.0)
    o.backward(dO.cuda())
    pos = torch.arange(T).repeat(B)
    leaf = {n: t.detach().double().cpu().requires_grad_() for n, t in (("q", q), ("k", k), ("wq", wq), ("wk", wk))}
    hat = {n: rotate64(norm64(leaf[n].reshape(B * T, -1, D), leaf["w" + n], 1e-6)[0], pos).view(B, T, -1, D) for n in "qk"}
    alpha = api.alpha_from_theta(0.21)
    args = [hat["q"].detach().numpy(), hat["k"].detach().numpy(), v.detach().double().cpu().numpy()]
    o_ref, _ = oracle.forward(*args, W=W, rungs=api.FIBONACCI_BASE, alpha=alpha, rope_theta=0.0)
    gq, gk, gv, _, gth, _ = oracle.backward(*args, dO.double().numpy(), W=W, rungs=api.FIBONACCI_BASE, alpha=alpha,
                                            rope_theta=0.0)
    (hat["q"] * torch.from_numpy(gq)).sum().backward()
    (hat["k"] * torch.from_numpy(gk)).sum().backward()
    for name, got, want in (("o", o, torch.from_numpy(o_ref)), ("dv", v.grad, torch.from_numpy(gv)),
                            ("dq", q.grad, leaf["q"].grad), ("dk", k.grad, leaf["k"].grad),
                            ("dwq", wq.grad, leaf["wq"].grad), ("dwk", wk.grad, leaf["wk"].grad)):
        within(got, want, torch.full_like(want, 1e-4 * max(1.0, float(want.abs().max()))), name)
    assert abs(theta.grad.item() - gth) <= 1e-3 * abs(gth) + 1e-4


def test_autograd_takes_broadcast_gradients():
    """A summed loss hands expanded (stride 0) gradients to the backward."""
    q, k, wq, wk, _ = _draw(2, 20, "f32", False, seed=29)
    q, k = q.requires_grad_(), k.requires_grad_()
    qh, kh = api.QKNormRope.apply(q, k, wq.requires_grad_(), wk)
    qh.sum().backward()   # khat unused: its gradient is zero
    one = torch.ones_like(qh)
    want = api.sfa_qk_norm_rope_backward(q.detach(), k.detach(), wq.detach(), wk, one, torch.zeros_like(kh))
    assert torch.equal(q.grad, want[0]) and torch.equal(wq.grad, want[2]) and bool((k.grad == 0).all())


def test_captured_call_outlives_a_grown_table():
    """A graph captured with the shared RoPE table, replayed after the table has
    grown and the memory it might have left has been written over."""
    theta = 12345.0  # a table of its own
    q, k, wq, wk, _ = _draw(2, 40, "bf16", False, seed=31)
    want = api.sfa_qk_norm_rope(q, k, wq, wk, rope_theta=theta)
    rows = api.rope_table(1, "cuda", rope_theta=theta).shape[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = api.sfa_qk_norm_rope(q, k, wq, wk, rope_theta=theta)
    grown = api.rope_table(rows + 1, "cuda", rope_theta=theta)
    assert grown.shape[0] > rows
    junk = [torch.full((rows, 32, 2), float("nan"), device="cuda") for _ in range(8)]
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want)) and len(junk) == 8


def test_two_backward_calls_at_once():
    """Two streams at the same time, workspaces from the allocator: the results
    of one call after the other, bit for bit."""
    given = []
    for seed in (41, 42):
        q, k, wq, wk, g = _draw(3, 2000, "bf16", True, seed=seed)
        up = [torch.randn((3, 2000, h, D), generator=g).to(torch.bfloat16).cuda() for h in (HQ, HKV)]
        given.append((q, k, wq, wk, *up))
    want = [api.sfa_qk_norm_rope_backward(*x) for x in given]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [None, None]
    for i in (0, 1) * 4:
        got[i] = api.sfa_qk_norm_rope_backward(*given[i], stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))


def test_captured_training_step():
    """Forward and backward of QKNormRope and SparseAttention captured together,
    replayed on new inputs, against the eager gradients: those that no atomic
    sum enters bit for bit, dV to one step of bf16 (its fp32 sums run in a free
    order, which may move the value before the rounding by 2^-12 of the largest)."""
    q, k, wq, wk, g = _draw(2, 150, "bf16", False, seed=43)
    v = torch.randn((2, 150, HKV, D), generator=g).to(torch.bfloat16).cuda()
    theta = torch.tensor(0.2)  # on the host: read there when the call is made

    def step(*leaves):
        o = api.SparseAttention.apply(*api.QKNormRope.apply(*leaves[:4]), leaves[4], theta, 12, api.FIBONACCI_BASE, 0.0)
        return torch.autograd.grad(o.float().square().sum(), leaves)

    leaves = [x.detach().clone().requires_grad_() for x in (q, k, wq, wk, v)]
    want = step(*leaves)
    static = [x.detach().clone().requires_grad_() for x in leaves]
    with torch.no_grad():
        for x in static[:2]:
            x.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*static)
    with torch.no_grad():
        for x, y in zip(static[:2], leaves[:2]):
            x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    b = want[4].double().cpu()
    within(got[4], b, 2.0 ** -7 * b.abs() + 2.0 ** -12 * b.abs().max(), "dv")


@pytest.mark.parametrize("T", [1, 64, 65])
def test_few_tokens_captured(T):
    """The backward pass of few tokens (one launch) and of one more (two), captured
    with the launch that writes its input and replayed: the eager results."""
    q, k, wq, wk, g = _draw(1, T, "bf16", True, seed=47)
    up = [torch.randn((1, T, h, D), generator=g).to(torch.bfloat16).cuda() for h in (HQ, HKV)]
    want = api.sfa_qk_norm_rope_backward(q, k, wq, wk, *up)
    given = [torch.zeros_like(x) for x in up]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(4):
            for x, y in zip(given, up):
                x.copy_(y)
            got = api.sfa_qk_norm_rope_backward(q, k, wq, wk, *given)
            for x in given:
                x.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
