"""Training steps launched one after another on the same buffers: norm, attention,
its backward pass and the norm's, each reading what the launch right before it
wrote, in a captured chain with other inputs every step."""
import pytest
import torch

from fibonacci_spaced_sparse_gb300 import api
from _paged import DT, HKV, HQ, D

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,dtype,W", [(1, 50, "bf16", 12), (2, 1100, "bf16", 12), (12, 1024, "bf16", 12), (2, 300, "f32", 12),
                                         (2, 300, "bf16", 40)])
def test_steps_in_a_row(B, T, dtype, W):
    g = torch.Generator().manual_seed(B + T)
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g)).cuda() for _ in range(2))

    def tensors():
        return [torch.randn((B, T, h, D), generator=g).to(DT[dtype]).cuda() for h in (HQ, HKV, HKV, HQ)]

    given = [tensors() for _ in range(2)]                                  # q, k, v, dO
    kw = dict(alpha=0.87, W=W, rope_theta=0.0)
    need = api.sfa_backward_workspace_size(B, T, alpha=0.87, W=W, dtype=DT[dtype])
    buf = {n: torch.zeros((B, T, h, D), dtype=DT[dtype], device="cuda")
           for n, h in (("qh", HQ), ("kh", HKV), ("dqh", HQ), ("dkh", HKV), ("dv", HKV), ("dk", HKV))}
    buf["lse"] = torch.zeros((B, T, HQ), device="cuda")
    buf["da"], buf["dth"] = (torch.zeros(1, device="cuda") for _ in range(2))
    buf["dwk"] = torch.zeros(D, device="cuda")
    ws = torch.zeros(max(need, 1), dtype=torch.uint8, device="cuda")

    def step(q, k, v, dO, o, dq, dwq):
        api.sfa_qk_norm_rope(q, k, wq, wk, out=(buf["qh"], buf["kh"]))
        api.sfa_forward(buf["qh"], buf["kh"], v, out=o, lse=buf["lse"], **kw)
        api.sfa_backward(buf["qh"], buf["kh"], v, o, dO, buf["lse"], workspace=ws,
                         out=(buf["dqh"], buf["dkh"], buf["dv"], buf["da"], buf["dth"]), **kw)
        api.sfa_qk_norm_rope_backward(q, k, wq, wk, buf["dqh"], buf["dkh"], out=(dq, buf["dk"], dwq, buf["dwk"]))

    def outs():
        return [torch.zeros((B, T, HQ, D), dtype=DT[dtype], device="cuda") for _ in range(2)] + [torch.zeros(D, device="cuda")]

    want = []
    for x in given:
        want.append(outs())
        step(*x, *want[-1])
        torch.cuda.synchronize()
    got = [outs() for _ in range(6)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i, o in enumerate(got):
            step(*given[i % 2], *o)
    for _ in range(4):
        for o in got:
            for x in o:
                x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for i, o in enumerate(got):      # o, dq and dwq: no sum of theirs runs in a free order
            assert all(torch.equal(a, b) for a, b in zip(o, want[i % 2])), i
