"""The operators of an attention layer served in 8 bits, and the norm before it, case by case.

Six calls, in the order in which a layer makes them:

  norm_fwd   sfa_add_rms_norm: the residual's addition and the RMS norm of every
             row, to the rows' own type or to 8 bits with a scale a row;
  norm_bwd   its backward pass: the gradient of the sum and of the norm's weight;
  qkv        sfa_qkv_rope_fp8: the query, key and value projection of 8-bit rows
             and 8-bit weights, scales and position rotation in its epilogue;
  append     sfa_paged_append_fp8: keys (normed, rotated) and values into a paged
             cache of 8-bit rows with a scale for each block of rows, key or value,
             and head; queries normed and rotated beside them;
  paged      sfa_paged_forward_fp8: attention of each sequence's new tokens, one or
             many, over such pages (window 0..W and one interpolated row per rung).

The 8-bit type is e4m3.  Shapes: 8 query heads, 2 key/value heads of dimension
64; model widths, lengths, windows and offset bases of this repository's
workloads and tests.  ``run`` computes the plain form in elementary torch
operations, in 32 bits and rounded once at the end, or, where ``own`` is true,
calls the library.  ``exact`` is the definition in 64 bits; of an 8-bit output it
gives the value before its rounding.
"""
import math
import random

import numpy as np
import torch

own = False

HQ, HKV, D = 8, 2, 64
HALF = D // 2
QKV = (HQ + 2 * HKV) * D
THETA = 1e4
EPS = 1e-6
TOP = 448.0                # largest e4m3 value
LEAST_ROW = 2.0 ** -126    # smallest scale of a row
LEAST_EXP = -100           # of the smallest scale of a block, as a power of two
FIBONACCI = (1, 2, 3, 5, 8, 13, 21, 34, 55, 89, 144, 233, 377, 610, 987)
POW2 = tuple(1 << k for k in range(12))
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
FP8 = torch.float8_e4m3fn


# ---------------------------------------------------------------------- cases


def listed():
    return [
        # the norm in front of a layer's projection, a training batch at the training length
        {"name": "norm_fwd_train", "op": "norm_fwd", "dtype": "bf16", "N": 32768, "dim": 512, "res": True, "fp8": False},
        # one token of each of 256 running sequences, its output for an 8-bit projection
        {"name": "norm_fwd_decode_fp8", "op": "norm_fwd", "dtype": "bf16", "N": 256, "dim": 512, "res": True, "fp8": True},
        # prompts entering a wider model, an odd number of tokens, 8 bits
        {"name": "norm_fwd_wide_fp8", "op": "norm_fwd", "dtype": "bf16", "N": 5443, "dim": 4096, "res": True, "fp8": True},
        # the training batch's backward pass, with the gradient that comes along the residual
        {"name": "norm_bwd_train", "op": "norm_bwd", "dtype": "bf16", "N": 32768, "dim": 512, "res": True},
        # gradients in 32 bits, odd numbers of tokens and a narrow model
        {"name": "norm_bwd_f32_odd", "op": "norm_bwd", "dtype": "f32", "N": 4083, "dim": 320, "res": True},
        # a decode step's projection: one token of 256 sequences
        {"name": "qkv_decode", "op": "qkv", "B": 256, "T": 1, "dm": 512, "rope": False},
        # whole prompts of the training length
        {"name": "qkv_prefill", "op": "qkv", "B": 32, "T": 1024, "dm": 512, "rope": True},
        # a wider model, ragged prompts packed into one row of tokens
        {"name": "qkv_wide", "op": "qkv", "B": 1, "T": 8157, "dm": 4096, "rope": False},
        # a decode step's new keys and values, norm and rotation on the way
        {"name": "append_decode", "op": "append", "dtype": "bf16", "S": 256, "most_q": 1, "chunks": 256, "most_ctx": 511,
         "lens": 31, "page": 16, "rows": 16, "pad": 0, "norm": True, "packed": True, "q": True},
        # ragged prompts entering the cache, rotation only
        {"name": "append_prefill", "op": "append", "dtype": "bf16", "S": 16, "most_q": 2048, "chunks": 16, "most_ctx": 300,
         "lens": 32, "page": 64, "rows": 16, "pad": 0, "norm": False, "packed": False, "q": True},
        # a decode step of 256 sequences over caches of up to 4096 rows
        {"name": "paged_decode", "op": "paged", "dtype": "bf16", "S": 256, "most_q": 1, "chunks": 256, "most_ctx": 4095,
         "lens": 41, "page": 16, "rows": 16, "pad": 0, "W": 12, "alpha": 0.9, "base": "fibonacci"},
        # whole prompts of the training length, caches empty before
        {"name": "paged_prefill", "op": "paged", "dtype": "bf16", "S": 32, "most_q": -1024, "chunks": 32, "most_ctx": 0,
         "lens": 45, "page": 64, "rows": 16, "pad": 0, "W": 12, "alpha": 0.8333333, "base": "fibonacci"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm_fwd", "norm_bwd", "qkv", "append", "paged", "paged"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if op.startswith("norm"):
        dim = 8 * _log(rng, 8, 1024)
        case = {"op": op, "dtype": dtype, "N": _log(rng, 1, min(32768, 8000000 // dim)), "dim": dim, "res": rng.random() < 0.8}
        if op == "norm_fwd":
            case["fp8"] = rng.random() < 0.5
        return case
    if op == "qkv":
        dm = 64 * _log(rng, 1, 64)
        B = _log(rng, 1, 256)
        return {"op": op, "B": B, "T": _log(rng, 1, max(1, min(8192, 16000000 // dm // B))), "dm": dm,
                "rope": rng.random() < 0.5}
    S = _log(rng, 1, 256)
    kind = rng.choice(("single", "mixed", "chunks"))
    chunks = {"single": S, "mixed": rng.randint(0, S), "chunks": S}[kind]
    most_q = 1 if kind == "single" else _log(rng, 2, max(2, min(4096, 12000 // max(1, chunks))))
    page = rng.choice((8, 16, 16, 32, 64, 128, 256))
    case = {"op": op, "dtype": dtype, "S": S, "most_q": most_q, "chunks": chunks,
            "most_ctx": _log(rng, 1, max(2, min(8192, 400000 // S) if op == "paged" else min(2048, 60000 // S))),
            "lens": rng.randrange(1 << 30), "page": page, "rows": min(page, rng.choice((8, 16, 16, 16, 32, 64))),
            "pad": rng.choice((0, 0, rng.randint(1, 64)))}
    if op == "append":
        case.update(norm=rng.random() < 0.5, packed=rng.random() < 0.5, q=rng.random() < 0.8)
    else:
        case.update(W=rng.choice((0, 5, 6, 8, 10, 12, 12, 12, 16, 24)), alpha=round(rng.uniform(0.5, 1.5), 4),
                    base=rng.choice(("fibonacci", "fibonacci", "pow2")))
    return case


def _lens(case):
    """(new tokens, rows before them) of every sequence of a cache's case: the
    first ``chunks`` sequences bring up to most_q tokens, the others one; a
    negative bound is the length itself."""
    rng = random.Random(case["lens"])
    def of(most, least):
        return -most if most < 0 else rng.randint(least, max(least, most))
    out = [(of(case["most_q"], 1) if s < case["chunks"] else 1, of(case["most_ctx"], 0)) for s in range(case["S"])]
    rng.shuffle(out)
    return out


def _plan(case):
    """The kept rungs as (floor d, fraction, ceil d): d = fl32(alpha) * fl32(f), d > W."""
    base = FIBONACCI if case["base"] == "fibonacci" else POW2
    plan = []
    for f in base:
        d = float(np.float32(case["alpha"]) * np.float32(f))
        if d > case["W"]:
            plan.append((math.floor(d), d - math.floor(d), math.ceil(d)))
    return plan


# --------------------------------------------------------------------- inputs


def _rope_table(rows):
    """(cos, sin) of position * THETA^(-2m/D), angles in 64 bits: [rows, D/2, 2]."""
    w = THETA ** (-2.0 * torch.arange(HALF, dtype=torch.float64, device="cuda") / D)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * w
    return torch.stack((a.cos(), a.sin()), -1).float().contiguous()


def _row_codes(x):
    """A row's scale and its values in 8 bits, as an 8-bit checkpoint holds them."""
    s = (x.abs().amax(-1, keepdim=True) / TOP).clamp_min(LEAST_ROW)
    return (x / s).clamp(-TOP, TOP).to(FP8), s.squeeze(-1)


def _power(amax):
    """The smallest power of two s >= 2^LEAST_EXP with amax <= TOP s."""
    m, e = torch.frexp(amax)                      # amax = m 2^e, m in [1/2, 1); TOP = 0.875 * 2^9
    e = (e - 9 + (m > 0.875).int()).clamp_min(LEAST_EXP)
    return ((e + 127) << 23).view(torch.float32)


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    s = {"case": case, "op": case["op"]}
    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")
    if case["op"].startswith("norm"):
        N, dim, dtype = case["N"], case["dim"], TYPES[case["dtype"]]
        s["w"] = 1.0 + 0.2 * randn(dim)
        if case["op"] == "norm_fwd":
            s["x"] = randn(N, dim).to(dtype)
            s["res"] = (2.0 * randn(N, dim)).to(dtype) if case["res"] else None
        else:
            s["h"] = (2.0 * randn(N, dim)).to(dtype)
            s["dy"] = randn(N, dim).to(dtype)
            s["dh"] = randn(N, dim).to(dtype) if case["res"] else None
        return s
    if case["op"] == "qkv":
        B, T, dm = case["B"], case["T"], case["dm"]
        s["x"], s["sx"] = _row_codes(randn(B, T, dm) * torch.exp(0.3 * randn(B, T, 1)))
        s["w"], s["sw"] = _row_codes(randn(QKV, dm) * dm ** -0.5)
        s["rope"] = _rope_table(T) if case["rope"] else None
        return s
    dtype = TYPES[case["dtype"]]
    s["dtype"] = dtype
    lens, page, rows = _lens(case), case["page"], case["rows"]
    N = sum(n for n, _ in lens) + case["pad"]
    need = [-(-(n + c) // page) for n, c in lens]
    num_pages = sum(need) + 3
    shuffled = torch.randperm(num_pages, generator=gen, device="cuda").int()
    # a sequence's entries behind its last page are never looked at: -1
    table = torch.full((case["S"], max(need)), -1, dtype=torch.int32)
    owned = torch.zeros((case["S"], max(need)), dtype=torch.bool)
    for i, n in enumerate(need):
        owned[i, :n] = True
    s["block_table"] = table.cuda().masked_scatter_(owned.cuda(), shuffled)
    s["cu_q"] = torch.tensor([0] + list(np.cumsum([n for n, _ in lens])), dtype=torch.int32).cuda()
    s["seq_lens"] = torch.tensor([n + c for n, c in lens], dtype=torch.int32).cuda()
    # cached rows whose size differs from block to block
    scales = []
    for name in ("k_pages", "v_pages"):
        x = randn(num_pages, page // rows, rows, HKV, D) * torch.exp(0.5 * randn(num_pages, page // rows, 1, HKV, 1))
        sc = _power(x.abs().amax((2, 4)))
        s[name] = (x / sc[:, :, None, :, None]).to(FP8).view(num_pages, page, HKV, D)
        scales.append(sc)
    s["scales"] = torch.stack(scales, 2).contiguous()  # [num_pages, page / rows, key or value, head]
    if case["op"] == "append":
        size = torch.exp(0.5 * randn(N, 1, 1))
        if case["packed"]:
            x = (randn(N, HQ + 2 * HKV, D) * size).to(dtype)
            s["q"], s["k"], s["v"] = x.split((HQ, HKV, HKV), 1)
        else:
            s["q"], s["k"], s["v"] = ((randn(N, h, D) * size).to(dtype) for h in (HQ, HKV, HKV))
        s["wq"], s["wk"] = (1.0 + 0.2 * randn(D), 1.0 + 0.2 * randn(D)) if case["norm"] else (None, None)
        if not case["q"]:
            s["q"] = s["wq"] = None
        else:
            s["q_out"] = torch.zeros((N, HQ, D), dtype=dtype, device="cuda")
        s["table"] = _rope_table(max(n + c for n, c in lens))
        return s
    s["q"] = randn(N, HQ, D).to(dtype)
    # rows behind the last sequence stay as they are
    s["o"] = torch.zeros((N, HQ, D), dtype=dtype, device="cuda")
    s["lse"] = torch.zeros((N, HQ), dtype=torch.float32, device="cuda")
    return s


# ----------------------------------------------------------------- plain form


def _plain_norm_fwd(s):
    x = s["x"]
    h = x if s["res"] is None else (x.float() + s["res"].float()).to(x.dtype)
    f = h.float()
    y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * s["w"]
    if not s["case"]["fp8"]:
        return {"h": h, "y": y.to(x.dtype)}
    scale = (y.abs().amax(-1, keepdim=True) / TOP).clamp_min(LEAST_ROW)
    return {"h": h, "y8": (y / scale).clamp(-TOP, TOP).to(FP8), "scale": scale.squeeze(-1)}


def _plain_norm_bwd(s):
    h, dy = s["h"].float(), s["dy"].float()
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    n = h * r
    g = dy * s["w"]
    dx = r * (g - n * (g * n).mean(-1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["h"].dtype), "dw": (dy * n).sum(0)}


def _rotate(x, cs):
    """x [..., heads, 64] rotated by the table rows cs [..., 32, 2] of its tokens."""
    c, s = cs[..., 0].unsqueeze(-2), cs[..., 1].unsqueeze(-2)
    a, b = x[..., :HALF], x[..., HALF:]
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def _plain_qkv(s):
    B, T = s["case"]["B"], s["case"]["T"]
    y = torch.matmul(s["x"].float().view(B * T, -1), s["w"].float().t())
    y = (y * s["sx"].view(-1, 1) * s["sw"]).view(B, T, -1, D)
    q, k, v = y.split((HQ, HKV, HKV), 2)
    if s["rope"] is not None:
        q, k = _rotate(q, s["rope"]), _rotate(k, s["rope"])
    return {"q": q.to(torch.bfloat16), "k": k.to(torch.bfloat16), "v": v.to(torch.bfloat16)}


def _tokens(s, N):
    """(sequence, position, whether it belongs to one) of every token row."""
    t = torch.arange(N, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["cu_q"][1:], t, right=True)
    valid = seq < s["seq_lens"].numel()
    seq = seq.clamp(max=s["seq_lens"].numel() - 1)
    pos = s["seq_lens"][seq] - s["cu_q"][seq + 1] + t
    return seq, torch.where(valid, pos, 0), valid


def _slots(s, seq, pos):
    """Rows of the flattened cache that hold the positions pos of the sequences seq."""
    page = s["k_pages"].shape[1]
    return s["block_table"][seq, pos // page].long() * page + pos % page


def _norm(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _plain_append(s):
    N, rows = s["k"].shape[0], s["case"]["rows"]
    seq, pos, valid = _tokens(s, N)
    slot = _slots(s, seq, pos)
    cs = s["table"][pos.long()]
    k, v = s["k"].float(), s["v"].float()
    if s["wk"] is not None:
        k = _norm(k, s["wk"])
    new = torch.stack((_rotate(k, cs), v), 1)                              # [N, key or value, head, 64]
    # rows of no sequence repeat the first token's write
    slot = torch.where(valid, slot, slot[0])
    live = valid[:, None, None]
    new = torch.where(live[..., None], new, new[0])
    block = slot // rows
    old = s["scales"].view(-1, 2, HKV)
    amax = torch.zeros_like(old).index_reduce_(0, block, new.abs().amax(-1), "amax")
    first = torch.full((old.shape[0],), rows, device="cuda").index_reduce_(0, block, slot % rows, "amin")
    begun, touched = ((first > 0) & (first < rows))[:, None, None], (first < rows)[:, None, None]
    scale = _power(amax)
    scale = torch.where(touched, torch.where(begun, torch.maximum(scale, old), scale), old)
    # older rows of a block whose scale has grown
    ratio = (old / scale).permute(1, 0, 2)                                 # [key or value, block, head]
    older = torch.arange(rows, device="cuda") < first[:, None]
    older = (older & begun[:, 0])[..., None, None]
    for i, name in enumerate(("k_pages", "v_pages")):
        flat = s[name].view(-1, rows, HKV, D)
        x = flat.float()
        x = torch.where(older, x * ratio[i][:, None, :, None], x).view(-1, HKV, D)
        x[slot] = new[:, i] / scale[block, i][..., None]
        flat.copy_(x.view(flat.shape).to(FP8))
    old.copy_(scale)
    out = {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "scales": s["scales"]}
    if s["q"] is not None:
        q = s["q"].float()
        if s["wq"] is not None:
            q = _norm(q, s["wq"])
        out["q"] = torch.where(live, _rotate(q, cs).to(s["dtype"]), s["q_out"])
    return out


def _plain_paged(s):
    case, q = s["case"], s["q"].float()
    N, W = q.shape[0], case["W"]
    seq, pos, valid = _tokens(s, N)
    plan = _plan(case)
    near = torch.tensor(list(range(W + 1)) + [n for n, _, _ in plan], device="cuda", dtype=torch.int32)
    t = torch.tensor([f for _, f, _ in plan], device="cuda", dtype=torch.float32)
    least = torch.tensor(list(range(W + 1)) + [c for _, _, c in plan], device="cuda", dtype=torch.int32)
    a = pos[:, None] - near
    used = (pos[:, None] >= least) & valid[:, None]
    row_a = _slots(s, seq[:, None], torch.where(used, a, 0))
    row_b = _slots(s, seq[:, None], torch.where(used & (a > 0), a - 1, 0)[:, W + 1:])
    scales = s["scales"].view(-1, 2, HKV)
    def rows_of(pages, i, row):
        return pages.view(-1, HKV, D)[row].float() * scales[row // case["rows"], i][..., None]
    def entries(pages, i):
        x = rows_of(pages, i, row_a)
        x[:, W + 1:] = x[:, W + 1:] * (1 - t)[:, None, None] + rows_of(pages, i, row_b) * t[:, None, None]
        return torch.where(used[..., None, None], x, 0.0)  # [N, E, 2, 64]
    qg = q.view(N, HKV, HQ // HKV, D)
    k = entries(s["k_pages"], 0)
    score = torch.matmul(qg, k.permute(0, 2, 3, 1)) / math.sqrt(D)  # [N, 2, 4, E]
    del k
    score = torch.where(used[:, None, None], score, -math.inf)
    top = torch.where(valid[:, None, None, None], score.amax(-1, keepdim=True), 0.0)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p / total, entries(s["v_pages"], 1).permute(0, 2, 1, 3)).view(N, HQ, D)
    lse = (top + total.log()).view(N, HQ)
    return {"o": torch.where(valid[:, None, None], o.to(s["dtype"]), s["o"]), "lse": torch.where(valid[:, None], lse, s["lse"])}


# ------------------------------------------------------------ the library's calls


def _own(s):
    from fibonacci_spaced_sparse_gb300 import api
    op, case = s["op"], s["case"]
    if op == "norm_fwd":
        out = api.sfa_add_rms_norm(s["x"], s["res"], s["w"], eps=EPS, fp8=case["fp8"])
        return dict(zip(("h", "y8", "scale") if case["fp8"] else ("h", "y"), out))
    if op == "norm_bwd":
        dx, dw = api.sfa_add_rms_norm_backward(s["h"], s["w"], s["dy"], s["dh"], eps=EPS)
        return {"dx": dx, "dw": dw}
    if op == "qkv":
        q, k, v = api.sfa_qkv_rope_fp8(s["x"], s["sx"], s["w"], s["sw"], rope_theta=THETA if case["rope"] else 0.0,
                                       rope=s["rope"])
        return {"q": q, "k": k, "v": v}
    pages = (s["k_pages"], s["v_pages"], s["scales"], s["block_table"], s["cu_q"], s["seq_lens"])
    if op == "append":
        q = api.sfa_paged_append_fp8(s["k"], s["v"], *pages, q=s["q"], wq=s["wq"], wk=s["wk"], eps=EPS, rope_theta=THETA,
                                     rope=s["table"], q_out=s.get("q_out"))
        out = {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "scales": s["scales"]}
        if q is not None:
            out["q"] = q
        return out
    o, lse = api.sfa_paged_forward_fp8(s["q"], *pages, alpha=case["alpha"], W=case["W"],
                                       rungs=FIBONACCI if case["base"] == "fibonacci" else POW2, out=s["o"], lse=s["lse"])
    return {"o": o, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "qkv": _plain_qkv, "append": _plain_append,
            "paged": _plain_paged}[state["op"]](state)


# ------------------------------------------------------------------------ work


def _union(ranges):
    """How many integers >= 0 the closed ranges hold together."""
    total, end = 0, -1
    for lo, hi in sorted(ranges):
        lo = max(lo, end + 1, 0)
        if hi >= lo:
            total += hi - lo + 1
            end = hi
    return total


def work(case):
    if case["op"] == "qkv":
        M = case["B"] * case["T"]
        table = case["T"] * 256 if case["rope"] else 0
        return {"bytes": M * case["dm"] + 4 * M + QKV * (case["dm"] + 4) + M * QKV * 2 + table, "flops": 2 * M * QKV * case["dm"]}
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("norm"):
        N, dim = case["N"], case["dim"]
        if case["op"] == "norm_bwd":
            return {"bytes": (4 if case["res"] else 3) * N * dim * es + 8 * dim, "flops": 10 * N * dim}
        out = N * dim + 4 * N if case["fp8"] else N * dim * es
        return {"bytes": (3 if case["res"] else 1) * N * dim * es + out + 4 * dim, "flops": 6 * N * dim}
    lens = _lens(case)
    N, meta = sum(n for n, _ in lens), 4 * (2 * case["S"] + 1)
    if case["op"] == "append":
        q = HQ * D if case["q"] else 0
        rows = _union([(c, c + n - 1) for n, c in lens])
        pages = sum(-(-(n + c) // case["page"]) - c // case["page"] for n, c in lens)
        blocks = sum(-(-(n + c) // case["rows"]) - c // case["rows"] for n, c in lens)
        return {"bytes": N * (q * 2 * es + 2 * HKV * D * (es + 1)) + rows * 256 + 4 * pages + 32 * blocks + meta,
                "flops": N * (q + 2 * HKV * D) * (8 if case["norm"] else 4)}
    W, plan = case["W"], _plan(case)
    cached = pairs = 0
    for n, c in lens:
        first, last = c, c + n - 1
        ranges = [(max(0, first - W), last)]
        for fl, t, ce in plan:
            if last >= ce:
                ranges.append((max(first, ce) - fl - (1 if t else 0), last - fl))
                pairs += last - max(first, ce) + 1
        cached += _union(ranges)
        # window entries of the queries first..last: min(W, i) + 1 of query i
        short = max(0, min(last, W) - first + 1)
        pairs += sum(i + 1 for i in range(first, first + short)) + (n - short) * (W + 1)
    return {"bytes": N * HQ * (2 * D * es + 4) + cached * 2 * HKV * D + 16 * (cached // case["rows"]) + meta
            + 4 * (cached // case["page"] + case["S"]), "flops": pairs * HQ * D * 4}


# ------------------------------------------------------------- 64-bit definition


def _exact_norm(s):
    case = s["case"]
    if case["op"] == "norm_fwd":
        h = s["x"].double() + (s["res"].double() if s["res"] is not None else 0.0)
        z = h.to(s["x"].dtype).double()                      # the norm reads the sum as it is kept
        y = z / torch.sqrt(z.square().sum(-1, keepdim=True) / case["dim"] + EPS) * s["w"].double()
        if not case["fp8"]:
            return {"h": h, "y": y}
        scale = torch.clamp(y.abs().max(-1, keepdim=True).values / TOP, min=LEAST_ROW)
        return {"h": h, "y8": y / scale, "scale": scale[:, 0]}
    h = s["h"].double().requires_grad_()
    w = s["w"].double().requires_grad_()
    y = h / torch.sqrt(h.square().sum(-1, keepdim=True) / case["dim"] + EPS) * w
    loss = (y * s["dy"].double()).sum()
    if s["dh"] is not None:
        loss = loss + (h * s["dh"].double()).sum()
    loss.backward()
    return {"dx": h.grad, "dw": w.grad}


def _exact_turn(x, pos):
    """x [tokens, heads, 64] rotated at the positions pos, as complex numbers."""
    m = torch.arange(HALF, device=x.device, dtype=torch.float64)
    angle = pos.double()[:, None] * torch.exp(-(2.0 * m / D) * math.log(THETA))
    z = torch.complex(x[..., :HALF], x[..., HALF:]) * torch.polar(torch.ones_like(angle), angle)[:, None]
    return torch.cat((z.real, z.imag), -1)


def _exact_qkv(s):
    case = s["case"]
    B, T = case["B"], case["T"]
    x = s["x"].double().view(B * T, -1) * s["sx"].double().view(-1, 1)
    w = s["w"].double() * s["sw"].double()[:, None]
    y = (x @ w.t()).view(B * T, -1, D)
    if case["rope"]:
        turned = _exact_turn(y[:, :HQ + HKV], torch.arange(T, device="cuda").repeat(B))
        y = torch.cat((turned, y[:, HQ + HKV:]), 1)
    return {"q": y[:, :HQ].reshape(B, T, HQ, D), "k": y[:, HQ:HQ + HKV].reshape(B, T, HKV, D),
            "v": y[:, HQ + HKV:].reshape(B, T, HKV, D)}


def _exact_head(x, w, pos):
    x = x.double()
    if w is not None:
        x = x / ((x ** 2).sum(-1, keepdim=True) / D + EPS).sqrt() * w.double()
    return _exact_turn(x, pos)


def _exact_rows(s, i, length):
    """Flattened cache rows of the positions 0..length-1 of sequence i."""
    page = s["k_pages"].shape[1]
    pages = s["block_table"][i, : -(-length // page)].long()
    return (pages[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:length]


def _exact_append(s):
    """One sequence at a time: the values that its touched blocks hold, then their scales."""
    rows = s["case"]["rows"]
    codes = [s[n].double().view(-1, HKV, D) for n in ("k_pages", "v_pages")]
    scales = s["scales"].double().view(-1, 2, HKV)
    q_all = s["q_out"].double() if s["q"] is not None else None
    powers = torch.tensor([2.0 ** e for e in range(LEAST_EXP, 128)], dtype=torch.float64, device="cuda")
    at = 0
    for i, (n, c) in enumerate(_lens(s["case"])):
        pos = torch.arange(c, c + n, device="cuda")
        begin = c // rows * rows                                   # of the first block that gets a row
        where = _exact_rows(s, i, c + n)[begin:]
        block = torch.unique_consecutive(where // rows)
        got = (_exact_head(s["k"][at:at + n], s["wk"], pos), s["v"][at:at + n].double())
        for j in range(2):
            old = scales[block[0], j].clone()
            values = torch.cat((codes[j][where[:c - begin]] * old[:, None], got[j]))
            fresh = torch.zeros((len(block) * rows, HKV), dtype=torch.float64, device="cuda")
            fresh[c - begin:c - begin + n] = got[j].abs().amax(-1)
            scale = powers[torch.searchsorted(TOP * powers, fresh.view(-1, rows, HKV).amax(1))]
            if c > begin:
                scale[0] = torch.maximum(scale[0], old)
            scales[block, j] = scale
            each = scale.repeat_interleave(rows, 0)[:len(where)]
            codes[j][where] = values / each[..., None]
        if q_all is not None:
            q_all[at:at + n] = _exact_head(s["q"][at:at + n], s["wq"], pos)
        at += n
    out = {"k_pages": codes[0].view(s["k_pages"].shape), "v_pages": codes[1].view(s["v_pages"].shape),
           "scales": scales.view(s["scales"].shape)}
    if q_all is not None:
        out["q"] = q_all
    return out


def _exact_paged(s):
    case = s["case"]
    o, lse = s["o"].double(), s["lse"].double()
    # (least position, [(distance, weight), ...]) of every entry of the key list
    keys = [(d, [(d, 1.0)]) for d in range(case["W"] + 1)]
    keys += [(c, [(n, 1.0 - t), (n + 1, t)] if t else [(n, 1.0)]) for n, t, c in _plan(case)]
    scales = s["scales"].double().view(-1, 2, HKV)
    at = 0
    for i, (n, c) in enumerate(_lens(case)):
        rows = _exact_rows(s, i, c + n)
        k, v = ((s[name].view(-1, HKV, D)[rows].double() * scales[rows // case["rows"], j][..., None])
                .repeat_interleave(HQ // HKV, 1) for j, name in enumerate(("k_pages", "v_pages")))
        q = s["q"][at:at + n].double()
        pos = torch.arange(c, c + n, device="cuda")
        mine = [(least, parts) for least, parts in keys if c + n - 1 >= least]
        scores = torch.full((len(mine), n, HQ), -math.inf, dtype=torch.float64, device="cuda")
        for e, (least, parts) in enumerate(mine):
            f = max(0, least - c)  # the first query that has this entry
            x = sum(w * k[pos[f:] - d] for d, w in parts)
            scores[e, f:] = (q[f:] * x).sum(-1) / 8.0
        l = torch.logsumexp(scores, 0)
        p = torch.exp(scores - l)
        acc = torch.zeros((n, HQ, D), dtype=torch.float64, device="cuda")
        for e, (least, parts) in enumerate(mine):
            f = max(0, least - c)
            acc[f:] += p[e, f:, :, None] * sum(w * v[pos[f:] - d] for d, w in parts)
        o[at:at + n], lse[at:at + n] = acc, l
        at += n
    return {"o": o, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(s)
    return {"qkv": _exact_qkv, "append": _exact_append, "paged": _exact_paged}[case["op"]](s)
