"""The projection of 8-bit rows (sfa_qkv_rope_fp8) against 64 bits, and the whole
8-bit layer: norm, projection, append, attention."""
import numpy as np
import pytest
import torch

from fibonacci_spaced_sparse_gb300 import api
from _fp8 import FP8, NAN_CODE
from _paged import D, HALF_STEP, HKV, HQ, U, pair_size, rotate64, within

pytestmark = pytest.mark.gpu

ROWS = (HQ + 2 * HKV) * D


def _draw(B, T, dm, seed=0):
    g = torch.Generator().manual_seed(seed + B * T + dm)
    x = (torch.randn((B, T, dm), generator=g) * torch.exp(torch.randn((B, T, 1), generator=g))).to(torch.bfloat16)
    w = (torch.randn((ROWS, dm), generator=g) * dm ** -0.5).to(torch.bfloat16)
    x8, sx = api.sfa_quantize_rows_fp8(x.cuda())
    w8, sw = api.sfa_quantize_rows_fp8(w.cuda())
    return x8, sx, w8, sw


def _check(out, x8, sx, w8, sw, theta, pos=None, rows=slice(None)):
    """Products of e4m3 values are exact; the sum of dm of them goes through dm / 32
    steps of the tensor core, each off by at most a unit in the last place (2^-23) of
    what is summed so far, so by (dm / 32 + 33) 2^-23 of the sum of sizes.  Two scales
    and the rotation add 8 u of the pair's size, the result is rounded once."""
    B, T, dm = x8.shape
    x = x8.cpu().double() * sx.cpu().double()[..., None]
    w = w8.cpu().double() * sw.cpu().double()[:, None]
    x = x.view(B * T, dm)[rows]
    pos = torch.arange(T).repeat(B)[rows]
    y, size = (x @ w.t()).view(-1, 12, D), (x.abs() @ w.abs().t()).view(-1, 12, D)
    bound = (dm / 32 + 33) * 2.0 ** -23 * size + 2 * U * y.abs()
    y = torch.cat((rotate64(y[:, :10], pos, theta) if theta > 0 else y[:, :10], y[:, 10:]), 1)
    bound = torch.cat((pair_size(bound[:, :10]) + 8 * U * pair_size(y[:, :10]) if theta > 0 else bound[:, :10], bound[:, 10:]), 1)
    bound = bound + HALF_STEP["bf16"] * y.abs()
    got = torch.cat([t.reshape(B * T, -1, D) for t in out], 1)[rows]
    within(got, y, bound)


@pytest.mark.parametrize("B,T,dm", [(1, 1, 64), (1, 5, 64), (2, 300, 512), (3, 97, 192), (256, 1, 512), (1, 256, 1024),
                                    (2, 150, 320), (1, 40, 16384), (5, 1361, 512), (1, 3001, 576), (2, 1700, 2048),
                                    (1, 1537, 128)])
@pytest.mark.parametrize("theta", [1e4, 0.0])
def test_against_definition(B, T, dm, theta):
    a = _draw(B, T, dm)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = api.sfa_qkv_rope_fp8(*a, rope_theta=theta, status=status)
    assert api.sfa_read_status(status) == 0
    assert out[0].shape == (B, T, 8, 64) and out[2].shape == (B, T, 2, 64)
    _check(out, *a, theta)


def test_model_shape_sampled():
    """32 x 1024 tokens at d_model 512: rows at every place of a tile, given outputs
    between guards, on a stream of its own."""
    B, T, dm = 32, 1024, 512
    a = _draw(B, T, dm)
    rows = sorted({0, 127, 128, B * T - 1} | set(np.random.default_rng(0).integers(0, B * T, 500).tolist()))
    rooms = [torch.full((B * T + 2, h * D), 7.0, dtype=torch.bfloat16, device="cuda") for h in (HQ, HKV, HKV)]
    given = [r[1:-1].view(B, T, -1, D) for r in rooms]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = api.sfa_qkv_rope_fp8(*a, out=given, stream=side)
    side.synchronize()
    _check(out, *a, 1e4, rows=rows)
    for r in rooms:
        assert bool((r[0] == 7).all()) and bool((r[-1] == 7).all())
    again = api.sfa_qkv_rope_fp8(*a)
    assert all(torch.equal(x, y) for x, y in zip(again, out))


@pytest.mark.parametrize("B,T,dm", [(1, 5000, 1472), (4, 5000, 4096), (1, 5000, 640), (3, 2731, 2048), (1, 8157, 4096)])
@pytest.mark.parametrize("theta", [1e4, 0.0])
def test_weights_through_the_ring_sampled(B, T, dm, theta):
    """Wide rows, whose weights do not stay in shared memory: tiles of 128 and of 256
    tokens, one and several of them a block, the last one ragged."""
    a = _draw(B, T, dm)
    rows = sorted({0, 127, 128, 255, 256, T - 1, B * T - 1} | set(np.random.default_rng(1).integers(0, B * T, 150).tolist()))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = api.sfa_qkv_rope_fp8(*a, rope_theta=theta, status=status)
    assert api.sfa_read_status(status) == 0
    _check(out, *a, theta, rows=rows)
    again = api.sfa_qkv_rope_fp8(*a, rope_theta=theta)
    assert all(torch.equal(x, y) for x, y in zip(again, out))


@pytest.mark.parametrize("M", [3, 2000])
def test_values_that_are_not_finite_stay_in_their_row(M):
    a = _draw(1, M, 512)
    clean = api.sfa_qkv_rope_fp8(*a)
    a[0].view(torch.uint8)[0, 1, 77] = NAN_CODE
    a[1][0, 2] = float("inf")
    out = api.sfa_qkv_rope_fp8(*a)
    for x, y in zip(out, clean):
        assert bool(torch.isnan(x[0, 1]).all()) and not bool(torch.isfinite(x[0, 2]).any())
        keep = [i for i in range(M) if i not in (1, 2)]
        assert torch.equal(x[0, keep], y[0, keep])


def test_nothing_to_do():
    _, _, w8, sw = _draw(1, 1, 128)
    e = torch.empty((2, 0, 128), dtype=torch.uint8, device="cuda").view(FP8)
    before = api.launch_count()
    q, k, v = api.sfa_qkv_rope_fp8(e, torch.empty((2, 0), device="cuda"), w8, sw)
    assert q.shape == (2, 0, 8, 64) and k.shape == (2, 0, 2, 64) and api.launch_count() == before


# ------------------------------------------------------------------ together


class Layer:
    """An attention layer served in 8 bits: its weights and its cache."""

    def __init__(self, S, dm, max_len, seed, page=16, block=16):
        g = torch.Generator().manual_seed(seed)
        self.w = (1 + 0.2 * torch.randn(dm, generator=g)).cuda()
        self.w8, self.sw = api.sfa_quantize_rows_fp8((torch.randn((ROWS, dm), generator=g) * dm ** -0.5).cuda())
        self.wq, self.wk = ((1 + 0.2 * torch.randn(D, generator=g)).cuda() for _ in range(2))
        per = -(-max_len // page)
        self.pages = [torch.full((S * per, page, HKV, D), NAN_CODE, dtype=torch.uint8, device="cuda").view(FP8) for _ in range(2)]
        self.scales = torch.full((S * per, page // block, 2, HKV), float("nan"), device="cuda")
        self.table = torch.randperm(S * per, generator=g).view(S, per).int().cuda()
        self.block = block

    def cache(self):
        return (*self.pages, self.scales, self.table)

    def step(self, x, res, cu, seq):
        """One step's tokens x [N, dm] beside the residual stream: (h, queries, o, lse)."""
        h, y8, s = api.sfa_add_rms_norm(x, res, self.w, fp8=True)
        q, k, v = api.sfa_qkv_rope_fp8(y8[None], s[None], self.w8, self.sw, rope_theta=0.0)
        q = api.sfa_paged_append_fp8(k[0], v[0], *self.cache(), cu, seq, q=q[0], wq=self.wq, wk=self.wk)
        o, lse = api.sfa_paged_forward_fp8(q, *self.cache(), cu, seq, alpha=0.87, W=12)
        return h, q, o, lse

    def values(self, s, length):
        """Keys and values (64 bits) that the cache holds of sequence s."""
        pos = torch.arange(length)
        page = self.pages[0].shape[1]
        rows = self.table[s].cpu().long()[pos // page] * page + pos % page
        return [self.pages[i].view(-1, HKV, D).cpu().double()[rows]
                * self.scales.view(-1, 2, HKV).cpu()[rows // self.block, i].double()[..., None] for i in range(2)]


def _attention(q, k, v, i, alpha=0.87, W=12):
    """Query i (q [8, 64], 64 bits) over k, v [positions, 2, 64]."""
    rows = [(k[i - d], v[i - d]) for d in range(min(W, i) + 1)]
    for f in api.FIBONACCI_BASE:
        d = float(np.float32(alpha) * np.float32(f))
        n, t = int(d), d - int(d)
        if d > W and i >= n + (t > 0):
            rows.append(tuple((1 - t) * x[i - n] + (t * x[i - n - 1] if t else 0) for x in (k, v)))
    kk, vv = (torch.stack([r[j] for r in rows], 1).repeat_interleave(HQ // HKV, 0) for j in range(2))   # [8, E, 64]
    p = torch.softmax((kk * q[:, None]).sum(-1) / 8, -1)
    return (p[..., None] * vv).sum(1)


def test_serving_steps():
    """Prompts in chunks and single tokens of several sequences through norm,
    projection, append and attention.  Each step's output is the attention over
    what the cache holds (bound of one rounding, and of halves in chunks), and what
    it holds is the layer's keys and values in full precision to what 8 bits
    allow: rows, weights and the cache round by 2^-4 of a value at most, 2^-4 / sqrt(3)
    in the mean over a binade, and three of them in a row stay below 0.1 of the norm."""
    S, dm, T = 3, 320, 500
    layer = Layer(S, dm, T, seed=1)
    g = torch.Generator().manual_seed(2)
    x, res = (torch.randn((S, T, dm), generator=g).to(torch.bfloat16) for _ in range(2))
    done = [0] * S
    for step in [(130, 1, 0), (200, 2, 400), (1, 1, 1), (0, 1, 1), (1, 0, 1)] + [(1, 1, 1)] * 20 + [(100, 40, 1)]:
        cu = torch.tensor([0, *np.cumsum(step)], dtype=torch.int32).cuda()
        seq = torch.tensor([d + n for d, n in zip(done, step)], dtype=torch.int32).cuda()
        rows = [torch.cat([t[s, done[s]:done[s] + step[s]] for s in range(S)]).cuda() for t in (x, res)]
        h, q, o, _ = layer.step(*rows, cu, seq)
        assert torch.equal(h, (rows[0].float() + rows[1].float()).to(torch.bfloat16))
        at = 0
        for s in range(S):
            length = done[s] + step[s]
            if step[s]:
                k, v = layer.values(s, length)
                for j in {0, step[s] // 2, step[s] - 1}:
                    want = _attention(q[at + j].double().cpu(), k, v, done[s] + j)
                    # the rounding of o; halves: 2^-11 of the values' size, and 43 rows times 2^-17 of
                    # 448 scales, which are at most twice the largest value
                    within(o[at + j], want, 2.0 ** -8 * want.abs() + 2.0 ** -9 * v.abs().max())
            at += step[s]
            done[s] = length
    w = layer.w8.cpu().double() * layer.sw.cpu().double()[:, None]
    for s in range(S):
        hh = (x[s].float() + res[s].float()).to(torch.bfloat16).double()[:done[s]]
        y = hh / torch.sqrt(hh.square().mean(-1, keepdim=True) + 1e-6) * layer.w.cpu().double()
        full = (y @ w.t()).view(-1, 12, D)
        kk = full[:, 8:10]
        kk = kk / torch.sqrt(kk.square().mean(-1, keepdim=True) + 1e-6) * layer.wk.cpu().double()
        want = (rotate64(kk, torch.arange(done[s])), full[:, 10:])
        for got, ref in zip(layer.values(s, done[s]), want):
            assert float((got - ref).norm() / ref.norm()) <= 0.1


@pytest.mark.parametrize("S", [4, 300])
def test_captured_decode_steps(S):
    """Decode steps of S sequences captured once and replayed, against the same
    calls made one by one: bit for bit, cache included."""
    dm, T = 512, 64
    layers = [Layer(S, dm, T, seed=3) for _ in range(2)]
    g = torch.Generator().manual_seed(4)
    x = torch.randn((T, S, dm), generator=g).to(torch.bfloat16).cuda()
    cu = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    api.rope_table(T, "cuda")
    buf, res, seq = torch.zeros_like(x[0]), torch.zeros_like(x[0]), torch.zeros(S, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layers[0].step(buf, res, cu, seq)
    for layer in layers:       # the capture ran nothing; both start alike
        for p in layer.pages:
            p.view(torch.uint8).fill_(NAN_CODE)
        layer.scales.fill_(float("nan"))
    stream_res = torch.zeros_like(res)
    for t in range(40):
        buf.copy_(x[t])
        seq.fill_(t + 1)
        graph.replay()
        want = layers[1].step(x[t], stream_res, cu, torch.full((S,), t + 1, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), t
        res.copy_(out[0])
        stream_res = want[0].clone()
    for a, b in zip(layers[0].cache(), layers[1].cache()):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
