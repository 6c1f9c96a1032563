"""The serving and training operators around the sparse attention, case by case.

Four calls that a program makes between its projections and its attention:

  norm_fwd   sfa_qk_norm_rope: RMS norm of every query and key head, then the
             position rotation, [B, T] tokens (or single tokens at given positions);
  norm_bwd   its backward pass: dQ, dK and the gradients of the two norm weights;
  append     sfa_paged_append: keys rotated (and normed) into a paged cache with
             their values, queries rotated (and normed) beside them;
  paged      sfa_paged_forward: attention of each sequence's new tokens, one or
             many, over its pages (window 0..W and one interpolated row per rung).

Shapes: 8 query heads, 2 key/value heads of dimension 64; lengths, windows and
offset bases of this repository's workloads.  ``run`` computes the plain form
in elementary torch operations, in 32 bits and rounded once at the end, or,
where ``own`` is true, calls the library.  ``exact`` is the definition in 64
bits, one sequence and one entry of the key list at a time.
"""
import math
import random

import numpy as np
import torch

own = False

HQ, HKV, D = 8, 2, 64
HALF = D // 2
THETA = 1e4
EPS = 1e-6
FIBONACCI = (1, 2, 3, 5, 8, 13, 21, 34, 55, 89, 144, 233, 377, 610, 987)
POW2 = tuple(1 << k for k in range(12))
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------- cases


def listed():
    return [
        # one token of each of 256 running sequences, before a step over their caches
        {"name": "norm_fwd_single", "op": "norm_fwd", "dtype": "bf16", "B": 256, "T": 1, "far": 4096, "packed": True},
        # a layer of a training batch at the training length
        {"name": "norm_fwd_train", "op": "norm_fwd", "dtype": "bf16", "B": 32, "T": 1024, "far": 0, "packed": False},
        # the same layer's backward pass
        {"name": "norm_bwd_train", "op": "norm_bwd", "dtype": "bf16", "B": 32, "T": 1024, "far": 0, "packed": False},
        # gradients in 32 bits at an odd length, from a packed projection
        {"name": "norm_bwd_f32_odd", "op": "norm_bwd", "dtype": "f32", "B": 3, "T": 1361, "far": 0, "packed": True},
        # a decode step's new keys and values, queries with them, norm and rotation on the way
        {"name": "append_decode", "op": "append", "dtype": "bf16", "S": 256, "most_q": 1, "chunks": 256, "most_ctx": 511,
         "lens": 11, "page": 16, "pad": 0, "norm": True, "packed": True, "q": True},
        # ragged prompts entering the cache, rotation only
        {"name": "append_prefill", "op": "append", "dtype": "bf16", "S": 16, "most_q": 2048, "chunks": 16, "most_ctx": 300,
         "lens": 12, "page": 64, "pad": 0, "norm": False, "packed": False, "q": True},
        # a decode step of 256 sequences over caches of up to 4096 rows
        {"name": "paged_decode", "op": "paged", "dtype": "bf16", "S": 256, "most_q": 1, "chunks": 256, "most_ctx": 4095,
         "lens": 21, "page": 16, "pad": 0, "W": 12, "alpha": 0.9, "base": "fibonacci"},
        # a few users, one token each: latency alone
        {"name": "paged_decode_few", "op": "paged", "dtype": "bf16", "S": 3, "most_q": 1, "chunks": 3, "most_ctx": 2047,
         "lens": 22, "page": 64, "pad": 0, "W": 12, "alpha": 1.3, "base": "fibonacci"},
        # 32-bit serving of short ragged chunks
        {"name": "paged_f32_ragged", "op": "paged", "dtype": "f32", "S": 7, "most_q": 200, "chunks": 7, "most_ctx": 1200,
         "lens": 23, "page": 16, "pad": 5, "W": 8, "alpha": 1.0, "base": "fibonacci"},
        # a mixed step: most sequences decode, some enter with a chunk; the batch padded to its graph's size
        {"name": "paged_mixed", "op": "paged", "dtype": "bf16", "S": 64, "most_q": 512, "chunks": 6, "most_ctx": 3000,
         "lens": 24, "page": 16, "pad": 37, "W": 12, "alpha": 0.7, "base": "fibonacci"},
        # whole prompts of the training length, caches empty before
        {"name": "paged_prefill", "op": "paged", "dtype": "bf16", "S": 32, "most_q": -1024, "chunks": 32, "most_ctx": 0,
         "lens": 25, "page": 64, "pad": 0, "W": 12, "alpha": 0.8333333, "base": "fibonacci"},
        # the second half of two long prompts, chunks of 8192 over caches of 8192 rows, power-of-two offsets
        {"name": "paged_long", "op": "paged", "dtype": "bf16", "S": 2, "most_q": -8192, "chunks": 2, "most_ctx": -8192,
         "lens": 26, "page": 128, "pad": 0, "W": 10, "alpha": 1.21, "base": "pow2"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm_fwd", "norm_bwd", "append", "paged", "paged", "paged"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if op.startswith("norm"):
        single = op == "norm_fwd" and rng.random() < 0.3
        T = 1 if single else _log(rng, 1, 8192)
        B = _log(rng, 1, max(1, min(512, 24000 // T)))
        return {"op": op, "dtype": dtype, "B": B, "T": T, "far": _log(rng, 2, 16384) if single else 0,
                "packed": rng.random() < 0.5}
    S = _log(rng, 1, 256)
    kind = rng.choice(("single", "mixed", "chunks"))
    chunks = {"single": S, "mixed": rng.randint(0, S), "chunks": S}[kind]
    most_q = 1 if kind == "single" else _log(rng, 2, max(2, min(4096, 12000 // max(1, chunks))))
    case = {"op": op, "dtype": dtype, "S": S, "most_q": most_q, "chunks": chunks,
            "most_ctx": _log(rng, 1, max(2, min(8192, 400000 // S) if op == "paged" else min(2048, 60000 // S))),
            "lens": rng.randrange(1 << 30), "page": rng.choice((8, 16, 16, 32, 64, 128, 256)),
            "pad": rng.choice((0, 0, rng.randint(1, 64)))}
    if op == "append":
        case.update(norm=rng.random() < 0.5, packed=rng.random() < 0.5, q=rng.random() < 0.8)
    else:
        case.update(W=rng.choice((0, 5, 6, 8, 10, 12, 12, 12, 16, 24)), alpha=round(rng.uniform(0.5, 1.5), 4),
                    base=rng.choice(("fibonacci", "fibonacci", "pow2")))
    return case


def _lens(case):
    """(new tokens, rows before them) of every sequence of a paged case: the
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


def _rope_table(rows, dev):
    """(cos, sin) of position * THETA^(-2m/D), angles in 64 bits: [rows, D/2, 2]."""
    w = THETA ** (-2.0 * torch.arange(HALF, dtype=torch.float64, device=dev) / D)
    a = torch.arange(rows, dtype=torch.float64, device=dev)[:, None] * w
    return torch.stack((a.cos(), a.sin()), -1).float().contiguous()


def _heads(gen, lead, dtype, packed, names):
    """q, k, v of the named ones, [*lead, heads, 64]: separate, or views of one packed projection."""
    heads = {"q": HQ, "k": HKV, "v": HKV}
    if packed:
        x = torch.randn((*lead, (HQ + 2 * HKV) * D), generator=gen, device="cuda").to(dtype)
        q, k, v = x.split((HQ * D, HKV * D, HKV * D), -1)
        full = {"q": q.unflatten(-1, (HQ, D)), "k": k.unflatten(-1, (HKV, D)), "v": v.unflatten(-1, (HKV, D))}
        return [full[n] for n in names]
    return [torch.randn((*lead, heads[n], D), generator=gen, device="cuda").to(dtype) for n in names]


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    dtype = TYPES[case["dtype"]]
    s = {"case": case, "op": case["op"], "dtype": dtype}
    def weight():
        return (1.0 + 0.2 * torch.randn(D, generator=gen, device="cuda")).contiguous()
    if case["op"].startswith("norm"):
        B, T = case["B"], case["T"]
        s["q"], s["k"] = _heads(gen, (B, T), dtype, case["packed"], "qk")
        s["wq"], s["wk"] = weight(), weight()
        s["positions"] = (torch.randint(0, case["far"], (B, T), generator=gen, device="cuda").int() if case["far"] else None)
        s["rope"] = _rope_table(max(T, case["far"]), "cuda")
        if case["op"] == "norm_bwd":
            s["dqhat"], s["dkhat"] = _heads(gen, (B, T), dtype, False, "qk")
        return s
    lens, page = _lens(case), case["page"]
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
    for name in ("k_pages", "v_pages"):
        s[name] = torch.randn((num_pages, page, HKV, D), generator=gen, device="cuda", dtype=dtype)
    if case["op"] == "append":
        s["q"], s["k"], s["v"] = _heads(gen, (N,), dtype, case["packed"], "qkv")
        s["wq"], s["wk"] = (weight(), weight()) if case["norm"] else (None, None)
        if not case["q"]:
            s["q"] = s["wq"] = None
        else:
            s["q_out"] = torch.zeros((N, HQ, D), dtype=dtype, device="cuda")
        s["rope"] = _rope_table(max(n + c for n, c in lens), "cuda")
        return s
    s["q"] = torch.randn((N, HQ, D), generator=gen, device="cuda").to(dtype)
    # rows behind the last sequence stay as they are
    s["o"] = torch.zeros((N, HQ, D), dtype=dtype, device="cuda")
    s["lse"] = torch.zeros((N, HQ), dtype=torch.float32, device="cuda")
    return s


# ----------------------------------------------------------------- plain form


def _norm(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _rotate(x, cs):
    """x [..., heads, 64] rotated by the table rows cs [..., 32, 2] of its tokens."""
    c, s = cs[..., 0].unsqueeze(-2), cs[..., 1].unsqueeze(-2)
    a, b = x[..., :HALF], x[..., HALF:]
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def _table_rows(s):
    T = s["case"]["T"]
    return s["rope"][s["positions"].long()] if s["positions"] is not None else s["rope"][:T].unsqueeze(0)


def _plain_norm_fwd(s):
    cs = _table_rows(s)
    out = [_rotate(_norm(s[n].float(), s["w" + n]), cs).to(s["dtype"]) for n in "qk"]
    return {"qhat": out[0], "khat": out[1]}


def _plain_norm_bwd(s):
    cs = _table_rows(s)
    cs = torch.stack((cs[..., 0], -cs[..., 1]), -1)  # the rotation's transpose
    out = {}
    for n in "qk":
        x, w, dz = s[n].float(), s["w" + n], s["d" + n + "hat"].float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        y, dy = x * r, _rotate(dz, cs)
        dn = dy * w
        out["d" + n] = (r * (dn - y * (dn * y).mean(-1, keepdim=True))).to(s["dtype"])
        out["dw" + n] = (dy * y).sum((0, 1, 2))
    return out


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


def _plain_append(s):
    N = s["k"].shape[0]
    seq, pos, valid = _tokens(s, N)
    slot = _slots(s, seq, pos)
    cs = s["rope"][pos.long()]
    k = s["k"].float()
    if s["wk"] is not None:
        k = _norm(k, s["wk"])
    k, v = _rotate(k, cs).to(s["dtype"]), s["v"]
    # rows of no sequence repeat the first token's write
    slot = torch.where(valid, slot, slot[0])
    live = valid[:, None, None]
    s["k_pages"].view(-1, HKV, D)[slot] = torch.where(live, k, k[0])
    s["v_pages"].view(-1, HKV, D)[slot] = torch.where(live, v, v[0])
    out = {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
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
    def entries(pages):
        flat = pages.view(-1, HKV, D)
        x = flat[row_a].float()
        far = x[:, W + 1:]
        x[:, W + 1:] = far * (1 - t)[:, None, None] + flat[row_b].float() * t[:, None, None]
        return torch.where(used[..., None, None], x, 0.0)  # [N, E, 2, 64]
    qg = q.view(N, HKV, HQ // HKV, D)
    k = entries(s["k_pages"])
    score = torch.matmul(qg, k.permute(0, 2, 3, 1)) / math.sqrt(D)  # [N, 2, 4, E]
    del k
    score = torch.where(used[:, None, None], score, -math.inf)
    top = torch.where(valid[:, None, None, None], score.amax(-1, keepdim=True), 0.0)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p / total, entries(s["v_pages"]).permute(0, 2, 1, 3)).view(N, HQ, D)
    lse = (top + total.log()).view(N, HQ)
    return {"o": torch.where(valid[:, None, None], o.to(s["dtype"]), s["o"]), "lse": torch.where(valid[:, None], lse, s["lse"])}


# ------------------------------------------------------------ the library's calls


def _own(s):
    from fibonacci_spaced_sparse_gb300 import api
    op = s["op"]
    if op == "norm_fwd":
        qhat, khat = api.sfa_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], eps=EPS, rope_theta=THETA,
                                          positions=s["positions"], rope=s["rope"])
        return {"qhat": qhat, "khat": khat}
    if op == "norm_bwd":
        dq, dk, dwq, dwk = api.sfa_qk_norm_rope_backward(s["q"], s["k"], s["wq"], s["wk"], s["dqhat"], s["dkhat"], eps=EPS,
                                                         rope_theta=THETA, positions=s["positions"], rope=s["rope"])
        return {"dq": dq, "dwq": dwq, "dk": dk, "dwk": dwk}
    if op == "append":
        q = api.sfa_paged_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["block_table"], s["cu_q"], s["seq_lens"],
                                 q=s["q"], wq=s["wq"], wk=s["wk"], eps=EPS, rope_theta=THETA, rope=s["rope"],
                                 q_out=s.get("q_out"))
        out = {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        if q is not None:
            out["q"] = q
        return out
    case = s["case"]
    o, lse = api.sfa_paged_forward(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["cu_q"], s["seq_lens"],
                                   alpha=case["alpha"], W=case["W"], rungs=FIBONACCI if case["base"] == "fibonacci" else POW2,
                                   out=s["o"], lse=s["lse"])
    return {"o": o, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "append": _plain_append,
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
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("norm"):
        N = case["B"] * case["T"]
        rows = min(N, case["far"]) if case["far"] else case["T"]
        row = (HQ + HKV) * D
        if case["op"] == "norm_fwd":
            return {"bytes": 2 * N * row * es + rows * 256 + (N * 4 if case["far"] else 0) + 512, "flops": N * row * 8}
        return {"bytes": 3 * N * row * es + rows * 256 + 1024, "flops": N * row * 16}
    lens = _lens(case)
    N, meta = sum(n for n, _ in lens), 4 * (2 * case["S"] + 1)
    if case["op"] == "append":
        row = ((HQ if case["q"] else 0) + 2 * HKV) * D
        rows = _union([(c, c + n - 1) for n, c in lens])
        pages = sum(-(-(n + c) // case["page"]) - c // case["page"] for n, c in lens)
        return {"bytes": 2 * N * row * es + rows * 256 + 4 * pages + meta, "flops": N * row * (8 if case["norm"] else 4)}
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
    return {"bytes": N * HQ * (2 * D * es + 4) + cached * 2 * HKV * D * es + meta + 4 * (cached // case["page"] + case["S"]),
            "flops": pairs * HQ * D * 4}


# ------------------------------------------------------------- 64-bit definition


def _exact_head(x, w, pos):
    """Norm (where w is given) and rotation of x [tokens, heads, 64] at the positions pos, as complex numbers."""
    x = x.double()
    if w is not None:
        x = x / ((x ** 2).sum(-1, keepdim=True) / D + EPS).sqrt() * w.double()
    m = torch.arange(HALF, device=x.device, dtype=torch.float64)
    angle = pos.double()[:, None] * torch.exp(-(2.0 * m / D) * math.log(THETA))
    z = torch.complex(x[..., :HALF], x[..., HALF:]) * torch.polar(torch.ones_like(angle), angle)[:, None]
    return torch.cat((z.real, z.imag), -1)


def _exact_norm(s):
    B, T = s["case"]["B"], s["case"]["T"]
    pos = s["positions"].reshape(-1) if s["positions"] is not None else torch.arange(T, device="cuda").repeat(B)
    leaves = {n: s[n].reshape(B * T, -1, D).double().requires_grad_() for n in "qk"}
    weights = {n: s["w" + n].double().requires_grad_() for n in "qk"}
    hat = {n: _exact_head(leaves[n], weights[n], pos) for n in "qk"}
    if s["op"] == "norm_fwd":
        return {n + "hat": hat[n].detach().view(s[n].shape) for n in "qk"}
    loss = sum((hat[n] * s["d" + n + "hat"].reshape(B * T, -1, D).double()).sum() for n in "qk")
    loss.backward()
    out = {}
    for n in "qk":
        out["d" + n] = leaves[n].grad.view(s[n].shape)
        out["dw" + n] = weights[n].grad
    return out


def _exact_rows(s, i, length):
    """Flattened cache rows of the positions 0..length-1 of sequence i."""
    page = s["k_pages"].shape[1]
    pages = s["block_table"][i, : -(-length // page)].long()
    return (pages[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:length]


def _exact_append(s):
    k_all, v_all = (s[n].double().view(-1, HKV, D) for n in ("k_pages", "v_pages"))
    q_all = s["q_out"].double() if s["q"] is not None else None
    at = 0
    for i, (n, c) in enumerate(_lens(s["case"])):
        pos = torch.arange(c, c + n, device="cuda")
        rows = _exact_rows(s, i, c + n)[c:]
        k_all[rows] = _exact_head(s["k"][at:at + n], s["wk"], pos)
        v_all[rows] = s["v"][at:at + n].double()
        if q_all is not None:
            q_all[at:at + n] = _exact_head(s["q"][at:at + n], s["wq"], pos)
        at += n
    out = {"k_pages": k_all.view(s["k_pages"].shape), "v_pages": v_all.view(s["v_pages"].shape)}
    if q_all is not None:
        out["q"] = q_all
    return out


def _exact_paged(s):
    case = s["case"]
    o, lse = s["o"].double(), s["lse"].double()
    # (least position, [(distance, weight), ...]) of every entry of the key list
    keys = [(d, [(d, 1.0)]) for d in range(case["W"] + 1)]
    keys += [(c, [(n, 1.0 - t), (n + 1, t)] if t else [(n, 1.0)]) for n, t, c in _plan(case)]
    k_flat, v_flat = s["k_pages"].view(-1, HKV, D), s["v_pages"].view(-1, HKV, D)
    at = 0
    for i, (n, c) in enumerate(_lens(case)):
        rows = _exact_rows(s, i, c + n)
        k = k_flat[rows].double().repeat_interleave(HQ // HKV, 1)
        v = v_flat[rows].double().repeat_interleave(HQ // HKV, 1)
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
    return _exact_append(s) if case["op"] == "append" else _exact_paged(s)
