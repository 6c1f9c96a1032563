"""Helpers of the 8-bit tests: e4m3 on the CPU, the scales' rules in exact
arithmetic, and a paged cache of 8-bit rows whose unused places hold NaN."""
from __future__ import annotations

import math

import torch

from _paged import Cache, D, DT, HKV, HQ

FP8 = torch.float8_e4m3fn
TOP = 448.0
NAN_CODE = 0x7f


def codes(x):
    """x (fp32 or fp64, any values) rounded to e4m3: to nearest even, past 448 to
    448, what is not finite to NaN."""
    x = torch.where(torch.isfinite(x), x.clamp(-TOP, TOP), float("nan"))
    return x.float().to(FP8)


def block_scale(amax: float) -> float:
    """The smallest power of two s >= 2^-100 with amax <= 448 s."""
    s = 2.0 ** -100
    while amax > TOP * s:
        s *= 2.0
    return s


def row_scales(x):
    """max |x| / 448 of the finite values of each row, at least 2^-126."""
    size = torch.where(torch.isfinite(x), x.abs(), 0.0)
    return (size.amax(-1) / TOP).clamp_min(2.0 ** -126)


class Cache8(Cache):
    """Cache with 8-bit rows in blocks of ``block`` positions: codes [s][position]
    and scales [s][position] (keys, values; a head each); k and v are the values
    that they stand for."""

    def __init__(self, lens, page, dtype, block, seed=0, powers=True, spread=0.7, **kw):
        super().__init__(lens, page, dtype, seed=seed, **kw)
        self.block = block
        g = torch.Generator().manual_seed(9000 + seed)
        self.codes, self.scales, values = [], [], []
        for raw in (self.k, self.v):
            cs, ss, vs = [], [], []
            for x in raw:
                n = x.shape[0]
                nb = -(-n // block)
                x = x.float() * torch.exp(spread * torch.randn((nb, HKV), generator=g)).repeat_interleave(block, 0)[:n, :, None]
                room = torch.zeros((nb * block, HKV))
                room[:n] = x.abs().amax(-1)
                amax = room.view(nb, block, HKV).amax(1)
                s = torch.tensor([[block_scale(float(a)) for a in row] for row in amax.tolist()]).view(nb, HKV)
                if not powers:
                    s = s * (1.0 + torch.rand((nb, HKV), generator=g))
                s = s.float().repeat_interleave(block, 0)[:n]
                c = codes(x / s[..., None])
                cs.append(c)
                ss.append(s)
                vs.append(c.float() * s[..., None])
            self.codes.append(cs)
            self.scales.append(ss)
            values.append(vs)
        self.k, self.v = values

    def pages8(self, rows_before=False, device="cuda"):
        """k_pages, v_pages, page_scales on the device."""
        out = [torch.full((self.num_pages * self.page, HKV, D), NAN_CODE, dtype=torch.uint8, device=device) for _ in range(2)]
        sc = torch.full((self.num_pages * self.page // self.block, 2, HKV), float("nan"), device=device)
        for i in range(2):
            for s, (n, c) in enumerate(self.lens):
                upto = c if rows_before else n + c
                slots = self.slots(s, upto)
                there = (slots >= 0) & (slots < self.num_pages * self.page)
                out[i][slots[there].to(device)] = self.codes[i][s][:upto].view(torch.uint8)[there].to(device)
                sc[(slots[there] // self.block).to(device), i] = self.scales[i][s][:upto][there].to(device)
        pages = [x.view(FP8).view(self.num_pages, self.page, HKV, D) for x in out]
        return pages + [sc.view(self.num_pages, self.page // self.block, 2, HKV)]


def expanded(cache):
    """Whether a bf16 call on this cache runs on bf16 copies of its rows."""
    return cache.dtype == "bf16" and cache.N >= 7000


def half_bound(cache, W, plan):
    """What the tensor-core kernel's halves add to the bound of o, for each token
    row and query head: a probability times its value row's scale is rounded to a
    half, by 2^-11 of it or 2^-25 in units in which the largest of a query's is at
    least 2^-8 (the margin of the running maximum), so by 2^-17 of that largest
    at most.  With the largest p s <= max s and codes up to 448 an entry adds
    2^-17 max(s) 448; the 2^-11 is the caller's."""
    out = torch.zeros((cache.N, HQ, 1), dtype=torch.float64)
    for t, s, i in cache.tokens():
        rows = [i - d for d in range(min(W, i) + 1)]
        for n, frac, c in plan:
            if i >= c:
                rows += [i - n] + ([i - n - 1] if frac else [])
        most = cache.scales[1][s][rows].double().amax(0)
        out[t, :, 0] = (2.0 ** -17 * len(rows) * TOP * most).repeat_interleave(HQ // HKV)
    return out.numpy()
