"""The norm's results in the contiguous decode (sfa_decode with rope_theta = 0),
launched one after another: every decode reads what the norm right before it
wrote, into the same buffers, in a captured chain."""
import pytest
import torch

from fibonacci_spaced_sparse_gb300 import api
from _paged import DT, HKV, HQ, D

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S,W", [(3, 12), (256, 12), (64, 40)])
def test_decode_reads_the_norm_before_it(S, W, dtype):
    g = torch.Generator().manual_seed(S + W)
    cap = 1200
    kc, vc = (torch.randn((S, cap, HKV, D), generator=g).to(DT[dtype]).cuda() for _ in range(2))
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g)).cuda() for _ in range(2))
    new = [[torch.randn((S, 1, h, D), generator=g).to(DT[dtype]).cuda() for h in (HQ, HKV)] for _ in range(2)]
    pos = [torch.randint(0, cap, (S, 1), generator=g).int().cuda() for _ in range(2)]
    rope = api.rope_table(cap, "cuda")
    kw = dict(alpha=0.87, W=W, rope_theta=0.0, need_lse=False)
    want = []
    for (q, k), p in zip(new, pos):
        qh, _ = api.sfa_qk_norm_rope(q, k, wq, wk, positions=p, rope=rope)
        torch.cuda.synchronize()
        want.append(api.sfa_decode(qh.view(S, HQ, D), kc, vc, p.view(S), **kw)[0])
    qh, kh = (torch.zeros((S, 1, h, D), dtype=DT[dtype], device="cuda") for h in (HQ, HKV))
    outs = [torch.zeros((S, HQ, D), dtype=DT[dtype], device="cuda") for _ in range(12)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i, o in enumerate(outs):
            api.sfa_qk_norm_rope(*new[i % 2], wq, wk, positions=pos[i % 2], rope=rope, out=(qh, kh))
            api.sfa_decode(qh.view(S, HQ, D), kc, vc, pos[i % 2].view(S), out=o, **kw)
    for _ in range(10):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want[i % 2]) for i, o in enumerate(outs))
