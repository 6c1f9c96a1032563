"""Attention over a paged cache of 8-bit rows in 64 bits, all tokens of a sequence
at once, and the bounds of the kernels' roundings, for chunks too long to go through
token by token."""
from __future__ import annotations

import ctypes
import math

import torch

from fibonacci_spaced_sparse_gb300 import _lib, api
from _paged import HALF_STEP, HKV, HQ, U, rung_list


def forward64(cache, *, alpha, W, rungs, scale=0.125, round_offsets=False):
    """o, lse of every token row that belongs to a sequence, sum p |v| (as o) and delta,
    the bound of a score's error in fp32 arithmetic (as lse): 80 u scale |q| |k| of the
    largest row read, as attention64 in _paged.py derives it."""
    plan = rung_list(alpha, W, rungs, round_offsets)
    keys = [(d, [(d, 1.0)]) for d in range(W + 1)]
    keys += [(c, [(n, 1.0 - t), (n + 1, t)] if t else [(n, 1.0)]) for n, t, c in plan]
    used = int(cache.cu[-1])
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    o = torch.zeros((used, HQ, 64), dtype=torch.float64, device=dev)
    size, lse, delta = torch.zeros_like(o), torch.zeros_like(o[..., 0]), torch.zeros_like(o[..., 0])
    at = 0
    for s, (n, c) in enumerate(cache.lens):
        if n == 0:
            continue
        k, v = (x[s].to(dev).double() for x in (cache.k, cache.v))
        q = cache.q[at:at + n].to(dev).double()
        pos = torch.arange(c, c + n, device=dev)
        wide = lambda x: x.repeat_interleave(HQ // HKV, 1)  # noqa: E731
        mine = [(least, parts) for least, parts in keys if c + n - 1 >= least]
        score = torch.full((len(mine), n, HQ), -math.inf, dtype=torch.float64, device=dev)
        largest = torch.zeros((n, HQ), dtype=torch.float64, device=dev)
        rows = lambda x, f, parts: sum(w * x[pos[f:] - d] for d, w in parts)  # noqa: E731
        for e, (least, parts) in enumerate(mine):
            f = max(0, least - c)
            score[e, f:] = (q[f:] * wide(rows(k, f, parts))).sum(-1) * scale
            for d, _ in parts:
                largest[f:] = torch.maximum(largest[f:], wide(k[pos[f:] - d].norm(dim=-1)))
        lse[at:at + n] = torch.logsumexp(score, 0)
        p = torch.exp(score - lse[at:at + n])
        for e, (least, parts) in enumerate(mine):
            f = max(0, least - c)
            o[at + f:at + n] += p[e, f:, :, None] * wide(rows(v, f, parts))
            size[at + f:at + n] += p[e, f:, :, None] * wide(rows(v.abs(), f, parts))
        delta[at:at + n] = 80 * U * scale * q.norm(dim=-1) * largest
        at += n
    return o.cpu(), lse.cpu(), size.cpu(), delta.cpu()


def fp32_bounds(ref, dtype):
    """Bounds of o and lse in fp32 arithmetic, rounded once: a probability moves by
    2 delta + 2^-20 of itself, lse by delta and its own few operations."""
    o, lse, size, delta = ref
    return (2 * delta[..., None] + 2.0 ** -20) * size + HALF_STEP[dtype] * o.abs() + 1e-30, delta + 2.0 ** -20 * (1 + lse.abs())


def halves_bound(ref):
    """What the halves of the tensor-core kernel on 8-bit rows add to the bound of o: 2^-11
    of each probability, and what is lost of the small ones, which is at most 2^-13 of the
    largest element of the head's output (the kernel redoes a query where it could be more)."""
    o, _, size, _ = ref
    return 2.0 ** -11 * 1.01 * size + 2.0 ** -13 * (o.abs() + 2.0 ** -10 * size).amax(-1, keepdim=True)


def split_bound(ref):
    """What the tensor cores add over bf16 copies: a probability is the sum of two bf16
    parts, the second rounded by 2^-8 of at most 2^-8 of it."""
    return 2.0 ** -16 * 1.01 * ref[2]


def workspace(cache, W, alpha, rungs):
    """The library's workspace for a bf16 call on this cache; 0: no rows are copied."""
    p = api.Params(len(cache.lens), cache.max_pages * cache.page, W=W, alpha=alpha, rungs=rungs, rope_theta=0.0)
    at = 0x100000                       # never read
    c = _lib.SfaPagedFp8(_lib.SfaPaged(k_pages=at, v_pages=at, num_pages=cache.num_pages, page_size=cache.page, block_table=at,
                                       max_pages=cache.max_pages, cu_q=at, seq_lens=at, N=cache.N), at, cache.block)
    return _lib.load().sfa_paged_forward_fp8_workspace_size(p.ref(), ctypes.byref(c))
