"""Helpers of the norm and paged-cache tests: definitions in 64 bits, written
from the formulas, caches whose unused places hold NaN, and error bounds
derived from the arithmetic of the kernels."""
from __future__ import annotations

import math

import numpy as np
import torch

HQ, HKV, D, HALF = 8, 2, 64, 32
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24                                # half a step of fp32, relative
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def rotate64(x, pos, theta=1e4, back=False):
    """x [n, heads, 64] rotated at the positions pos [n]."""
    m = torch.arange(HALF, dtype=torch.float64)
    ang = pos.double()[:, None] * theta ** (-2.0 * m / D)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    if back:
        s = -s
    a, b = x[..., :HALF], x[..., HALF:]
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def pair_size(x):
    """|x_m| + |x_{m + 32}| at both members of every pair: what bounds a
    rotated element and the error of one."""
    s = x[..., :HALF].abs() + x[..., HALF:].abs()
    return torch.cat((s, s), -1)


def norm64(x, w, eps):
    """(y, n, r): w n, n = x r and r = 1 / sqrt(mean x^2 + eps)."""
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return x * r * w, x * r, r


def head64(x, w, eps, pos, theta):
    """Norm (with w) and rotation (theta > 0) of x [n, heads, 64], and the
    bound of its fp32 evaluation: the mean of squares takes 64 products and
    sums (relative error at most 66 u, halved by the root), the root, the
    division, two products and the rotation's three roundings and the table's
    one follow: below 48 u of the pair's size."""
    y = norm64(x, w, eps)[0] if w is not None else x
    z = rotate64(y, pos, theta) if theta > 0 else y
    return z, 48 * U * pair_size(y)


def within(got, want, bound, what=""):
    got = got.detach().double().cpu()
    want, bound = torch.as_tensor(want).double(), torch.as_tensor(bound).double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = (got - want).abs()
    assert bool((off <= bound).all()), (what, float((off / bound.clamp_min(1e-300)).max()),
                                        int((off > bound).sum()), off.numel())


class Cache:
    """A paged cache holding contiguous keys and values of several sequences.
    lens: (new tokens, rows before them) a sequence.  Rows that hold no
    position are NaN, pages are shuffled, and the table's entries behind a
    sequence's pages are garbage."""

    def __init__(self, lens, page, dtype, seed=0, spare=3, behind=7, gen_scale=1.0, num_pages=None):
        g = torch.Generator().manual_seed(1000 + seed)
        self.lens, self.page, self.dtype = lens, page, dtype
        dt = DT[dtype]
        self.k = [(gen_scale * torch.randn((n + c, HKV, D), generator=g)).to(dt) for n, c in lens]
        self.v = [torch.randn((n + c, HKV, D), generator=g).to(dt) for n, c in lens]
        self.N = sum(n for n, _ in lens) + behind
        self.q = (gen_scale * torch.randn((self.N, HQ, D), generator=g)).to(dt)
        need = [-(-(n + c) // page) for n, c in lens]
        used = sum(need)
        self.num_pages = num_pages or used + spare
        order = torch.randperm(self.num_pages, generator=g)[:used] if self.num_pages < 1 << 16 else \
            torch.randperm(used, generator=g) + self.num_pages - used
        self.max_pages = max(max(need, default=0), 1) + 2
        self.table = torch.full((len(lens), self.max_pages), -1, dtype=torch.int32)
        self.table[:, 1::2] = 1 << 30
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n].int()
            at += n
        self.cu = torch.tensor([0] + list(np.cumsum([n for n, _ in lens], dtype=np.int64)), dtype=torch.int32)
        self.seq = torch.tensor([n + c for n, c in lens], dtype=torch.int32)

    def slots(self, s, length=None):
        """Flattened page rows of the positions 0 .. of sequence s."""
        n = self.lens[s][0] + self.lens[s][1] if length is None else length
        pos = torch.arange(n)
        return self.table[s].long()[pos // self.page] * self.page + pos % self.page

    def pages(self, device="cuda", rows_before=None):
        """k_pages, v_pages on the device; rows_before: only the rows there
        before the step (the state an append starts from)."""
        out = []
        for x in (self.k, self.v):
            p = torch.full((self.num_pages * self.page, HKV, D), float("nan"), dtype=DT[self.dtype], device=device)
            for s, (n, c) in enumerate(self.lens):
                upto = c if rows_before else n + c
                slots = self.slots(s, upto)
                there = (slots >= 0) & (slots < self.num_pages * self.page)   # rows of bad pages are nowhere
                p[slots[there].to(device)] = x[s][:upto][there].to(device)
            out.append(p.view(self.num_pages, self.page, HKV, D))
        return out

    def meta(self):
        return self.table.cuda(), self.cu.cuda(), self.seq.cuda()

    def tokens(self):
        """(row, sequence, position) of every token that belongs to a sequence."""
        at = 0
        for s, (n, c) in enumerate(self.lens):
            for j in range(n):
                yield at + j, s, c + j
            at += n


def rung_list(alpha, W, rungs, round_offsets=False):
    out = []
    for f in rungs:
        d = float(np.float32(alpha) * np.float32(f))
        if round_offsets:
            d = math.floor(d + 0.5)
        if d > W:
            out.append((math.floor(d), d - math.floor(d), math.ceil(d)))
    return out


def attention64(cache, *, alpha, W, rungs, scale=0.125, round_offsets=False, bad_rows=(), tensor_cores=False):
    """(o, lse, bound of o, bound of lse) of every token row in 64 bits; rows of
    no sequence are NaN.  bad_rows: (sequence, position) that lie in bad pages.

    Bounds.  A score is 64 products summed in fp32, a scale and a lerp: its
    error is below 80 u scale |q| |k|max =: delta (Cauchy-Schwarz; k runs over
    the rows read).  lse moves by at most delta plus the rounding of its own
    few operations (2^-20 of 1 + |lse|; the exponential's error is 2^-22).
    A probability moves by a relative 2 delta + 2^-20, so o by that times
    sum p |v|, and it is rounded once.  On the tensor cores every probability
    is also rounded to bf16 before the value product: 2^-8 sum p |v|."""
    plan = rung_list(alpha, W, rungs, round_offsets)
    bad = set(bad_rows)
    N = cache.N
    o = np.full((N, HQ, D), np.nan)
    lse = np.full((N, HQ), np.nan)
    bo, bl = np.zeros((N, HQ, D)), np.zeros((N, HQ))
    k64 = [x.double().numpy() for x in cache.k]
    v64 = [x.double().numpy() for x in cache.v]
    q64 = cache.q.double().numpy()
    for t, s, i in cache.tokens():
        rows, weights = [], []
        for d in range(min(W, i) + 1):
            if (s, i - d) not in bad:
                rows.append((i - d, i - d))
                weights.append((1.0, 0.0))
        for n, frac, c in plan:
            if i >= c:
                need = [i - n] + ([i - n - 1] if frac else [])
                if not any((s, r) in bad for r in need):
                    rows.append((i - n, need[-1]))
                    weights.append((1.0 - frac, frac))
        if not rows:
            o[t], lse[t] = 0.0, -np.inf
            continue
        rows, weights = np.array(rows), np.array(weights)
        with np.errstate(invalid="ignore"):
            kk, vv = (np.where(weights[:, :1, None] == 0, 0, weights[:, :1, None] * x[s][rows[:, 0]])
                      + np.where(weights[:, 1:, None] == 0, 0, weights[:, 1:, None] * x[s][rows[:, 1]])
                      for x in (k64, v64))                              # [E, 2, 64]
            va = (np.where(weights[:, :1, None] == 0, 0, weights[:, :1, None] * np.abs(v64[s][rows[:, 0]]))
                  + np.where(weights[:, 1:, None] == 0, 0, weights[:, 1:, None] * np.abs(v64[s][rows[:, 1]])))
        kmax = np.sqrt((k64[s][rows.reshape(-1)] ** 2).sum(-1)).max()
        for h in range(HQ):
            g = h // (HQ // HKV)
            sc = kk[:, g] @ q64[t, h] * scale
            m = sc.max()
            p = np.exp(sc - m)
            tot = p.sum()
            p /= tot
            o[t, h] = p @ vv[:, g]
            lse[t, h] = m + math.log(tot)
            delta = 80 * U * scale * math.sqrt((q64[t, h] ** 2).sum()) * kmax
            size = p @ va[:, g]
            bo[t, h] = (2 * delta + 2.0 ** -20 + (2.0 ** -8 if tensor_cores else 0)) * size \
                + HALF_STEP[cache.dtype] * np.abs(o[t, h]) + 1e-30
            bl[t, h] = delta + 2.0 ** -20 * (1 + abs(lse[t, h]))
    return o, lse, bo, bl
