"""Norm with rotation of many tokens: the forward kernel that copies its rows
ahead (bf16, 10240 tokens and more) and the backward pass where a block goes
through several steps, in both types, against the formulas in 64 bits."""
import pytest
import torch

from fibonacci_spaced_sparse_gb300 import api
from _paged import DT, HALF_STEP, HKV, HQ, D, U, head64, norm64, pair_size, rotate64, within

pytestmark = pytest.mark.gpu

H10 = HQ + HKV


def _draw(B, T, dtype, packed, seed):
    g = torch.Generator().manual_seed(seed)
    if packed:
        x = torch.randn((B, T, 12 * D), generator=g).to(DT[dtype]).cuda()
        q, k = x[..., :HQ * D].unflatten(-1, (HQ, D)), x[..., HQ * D:H10 * D].unflatten(-1, (HKV, D))
    else:
        q, k = (torch.randn((B, T, h, D), generator=g).to(DT[dtype]).cuda() for h in (HQ, HKV))
    wq, wk = (1 + 0.3 * torch.randn(D, generator=g)).cuda(), (0.5 + 0.3 * torch.randn(D, generator=g)).cuda()
    return q, k, wq, wk, g


def _flat(x):
    return x.double().cpu().reshape(-1, x.shape[-2], D)


def _check_fwd(out, x, w, pos, theta, dtype, what):
    want, bound = head64(_flat(x), w.double().cpu(), 1e-6, pos, theta)
    within(out.reshape(-1, *out.shape[-2:]), want, bound + HALF_STEP[dtype] * want.abs() + 1e-30, what)


@pytest.mark.parametrize("theta", [1e4, 0.0])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("B,T", [(1, 10239), (1, 10240), (1, 10241), (3, 3571), (11, 1024), (10247, 1)])
def test_forward_of_many_tokens(B, T, packed, theta):
    q, k, wq, wk, _ = _draw(B, T, "bf16", packed, seed=B + T)
    qh, kh = api.sfa_qk_norm_rope(q, k, wq, wk, rope_theta=theta)
    pos = torch.arange(T).repeat(B)
    _check_fwd(qh, q, wq, pos, theta, "bf16", "q")
    _check_fwd(kh, k, wk, pos, theta, "bf16", "k")


@pytest.mark.parametrize("packed", [False, True])
def test_given_positions_of_many_tokens(packed):
    """Positions given a token, some outside the table: zeros and the status bit."""
    B, T = 5, 2303
    q, k, wq, wk, g = _draw(B, T, "bf16", packed, seed=71)
    rope = api.rope_table(6000, "cuda")
    rows = rope.shape[0]
    pos = torch.randint(0, rows, (B, T), generator=g)
    bad = torch.zeros((B, T), dtype=torch.bool)
    for i, (b, t) in enumerate(((0, 0), (0, 1), (1, 77), (2, 2302), (3, 1000), (4, 2302))):
        pos[b, t] = (-1, rows, 2 ** 31 - 1, -2 ** 31, rows + 5, -7)[i]
        bad[b, t] = True
    q[1, 78, 2, 9] = float("nan")              # stays in its row
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qh, kh = api.sfa_qk_norm_rope(q, k, wq, wk, positions=pos.int().cuda(), rope=rope, status=status)
    assert api.sfa_read_status(status) == 0x2
    assert bool((qh[bad] == 0).all()) and bool((kh[bad] == 0).all())
    assert bool(qh[1, 78, 2].isnan().all()) and int(qh.isnan().sum()) == D and not bool(kh.isnan().any())
    good = ~bad
    good[1, 78] = False
    _check_fwd(qh[good], q[good], wq, pos[good], 1e4, "bf16", "q")
    _check_fwd(kh[good], k[good], wk, pos[good], 1e4, "bf16", "k")


@pytest.mark.parametrize("packed", [False, True])
def test_forward_captured_with_its_input(packed):
    """A captured chain: the launch before writes the input, the call reads it, the
    next launch overwrites it."""
    given = [_draw(4, 3001, "bf16", packed, seed=s)[:4] for s in (81, 82)]
    want = [api.sfa_qk_norm_rope(*x) for x in given]
    q, k = (torch.empty_like(x) for x in given[0][:2])       # keeps the strides
    weights = given[0][2:]
    want[1] = api.sfa_qk_norm_rope(*given[1][:2], *weights)
    api.sfa_qk_norm_rope(q, k, *weights)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = []
        for i in range(8):
            q.copy_(given[i % 2][0])
            k.copy_(given[i % 2][1])
            got.append(api.sfa_qk_norm_rope(q, k, *weights))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(got):
        assert torch.equal(a, want[i % 2][0]) and torch.equal(b, want[i % 2][1]), i


def _check_bwd(got, x, w, up, pos, theta, dtype, blocks, heads, what):
    """dx element by element.  dw is a sum of `heads` products a token: two a step
    and thread, over the steps of one block of `blocks`; over a block's 8 tokens
    (and 4 pairs of query heads); over the blocks (8 a thread, two shuffles, 16
    rows).  A product carries the 40 u of n, the 4 u of g and its own rounding."""
    dx, dw = got
    x, w, up = _flat(x), w.double().cpu(), _flat(up)
    _, n, r = norm64(x, w, 1e-6)
    g = rotate64(up, pos, theta, back=True) if theta > 0 else up
    wg = w * g
    want = r * (wg - n * (wg * n).mean(-1, keepdim=True))
    gs = pair_size(up) if theta > 0 else up.abs()
    size = r * (w.abs() * gs + 2 * n.abs() * (w.abs() * gs * n.abs()).mean(-1, keepdim=True))
    within(dx.reshape(want.shape), want, 120 * U * size + HALF_STEP[dtype] * want.abs() + 1e-30, what + " dx")
    steps = -(-x.shape[0] // (8 * blocks))
    chain = 2 * steps + 8 * max(1, heads // 2) + 8 + 2 + 16 + 45
    within(dw, (g * n).sum((0, 1)), chain * U * (gs * n.abs()).sum((0, 1)) + 1e-30, what + " dw")


@pytest.mark.parametrize("theta", [1e4, 0.0])
@pytest.mark.parametrize("B,T,dtype,packed", [(1, 2432, "f32", True), (1, 2433, "f32", False), (3, 1361, "f32", True),
                                              (2, 4000, "f32", False), (1, 3648, "bf16", True), (1, 3649, "bf16", False),
                                              (3, 3571, "bf16", False)])
def test_backward_of_several_steps_a_block(B, T, dtype, packed, theta):
    q, k, wq, wk, g = _draw(B, T, dtype, packed, seed=B + T)
    up = [torch.randn((B, T, h, D), generator=g).to(DT[dtype]).cuda() for h in (HQ, HKV)]
    got = api.sfa_qk_norm_rope_backward(q, k, wq, wk, *up, rope_theta=theta)
    again = api.sfa_qk_norm_rope_backward(q, k, wq, wk, *up, rope_theta=theta)
    assert all(torch.equal(a, b) for a, b in zip(got, again))     # sums in a fixed order
    pos, blocks = torch.arange(T).repeat(B), {"f32": 304, "bf16": 456}[dtype]
    _check_bwd((got[0], got[2]), q, wq, up[0], pos, theta, dtype, blocks, HQ, "q")
    _check_bwd((got[1], got[3]), k, wk, up[1], pos, theta, dtype, blocks, HKV, "k")


def test_backward_of_many_given_positions():
    """fp32, several steps a block, bad positions among them: no gradient, and none
    of it in dw."""
    B, T = 3, 1361
    q, k, wq, wk, g = _draw(B, T, "f32", True, seed=91)
    up = [torch.randn((B, T, h, D), generator=g).cuda() for h in (HQ, HKV)]
    rope = api.rope_table(6000, "cuda")
    pos = torch.randint(0, rope.shape[0], (B, T), generator=g)
    bad = torch.zeros((B, T), dtype=torch.bool)
    for b, t, p in ((0, 0, -1), (1, 1360, rope.shape[0]), (2, 1360, 2 ** 31 - 1), (2, 5, -2 ** 31)):
        pos[b, t], bad[b, t] = p, True
        for x in (*up, q, k):
            x[b, t] = float("nan")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = api.sfa_qk_norm_rope_backward(q, k, wq, wk, *up, positions=pos.int().cuda(), rope=rope, status=status)
    assert api.sfa_read_status(status) == 0x2
    assert bool((got[0][bad] == 0).all()) and bool((got[1][bad] == 0).all())
    good = ~bad
    _check_bwd((got[0][good], got[2]), q[good], wq, up[0][good], pos[good], 1e4, "f32", 304, HQ, "q")
    _check_bwd((got[1][good], got[3]), k[good], wk, up[1][good], pos[good], 1e4, "f32", 304, HKV, "k")
