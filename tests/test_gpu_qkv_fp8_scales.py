"""The 8-bit projection with scales at the ends of what a float holds: the product of a
row's scale and a weight's may be too small for one, the result is not."""
import pytest
import torch

from fibonacci_spaced_sparse_gb300 import api
from _fp8 import FP8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,dm,theta", [(1, 5, 512, 0.0), (3, 700, 512, 1e4), (1, 2500, 1024, 0.0), (1, 8200, 4096, 0.0)])
@pytest.mark.parametrize("x_power,w_power", [(-126, -18), (-126, -30), (-110, -20), (100, -20), (80, 20)])
def test_scales_at_the_ends(B, T, dm, theta, x_power, w_power):
    g = torch.Generator("cuda").manual_seed(dm + x_power)
    x, w = (torch.randn((n, dm), generator=g, device="cuda").mul(60).clamp(-448, 448).to(FP8) for n in (B * T, 768))
    sx, sw = ((1.0 + torch.rand(n, generator=g, device="cuda")) * 2.0 ** p for n, p in ((B * T, x_power), (768, w_power)))
    got = api.sfa_qkv_rope_fp8(x.view(B, T, dm), sx.view(B, T), w, sw, rope_theta=theta)
    rows = torch.arange(0, B * T, max(1, B * T // 500), device="cuda")
    want = (x[rows].double() @ w.double().t()) * sx[rows].double()[:, None] * sw.double()
    size = (x[rows].double().abs() @ w.double().abs().t()) * sx[rows].double()[:, None] * sw.double()
    want, size = want.view(-1, 12, 64), size.view(-1, 12, 64)
    if theta > 0:
        cs = api.rope_table(T, "cuda", rope_theta=theta).view(-1, 32, 2).double()[rows % T][:, None]
        a, b, c, s = want[:, :10, :32], want[:, :10, 32:], cs[..., 0], cs[..., 1]
        turned = torch.cat((a * c - b * s, b * c + a * s), -1)
        pair = size[:, :10, :32] + size[:, :10, 32:]
        want, size = torch.cat((turned, want[:, 10:]), 1), torch.cat((torch.cat((pair, pair), -1), size[:, 10:]), 1)
    got = torch.cat([t.reshape(B * T, -1, 64)[rows] for t in got], 1).double()
    # fp32 sums of dm products (dm 2^-24 of their sizes; as little for the scales and the rotation)
    # and one rounding to bf16, which below 2^-126 has steps of 2^-133
    bound = (dm + 16) * 2.0 ** -24 * size + 2.0 ** -8 * want.abs() + 2.0 ** -134 + 2.0 ** -148
    assert bool(((got - want).abs() <= bound).all()), float(((got - want).abs() / bound).max())
