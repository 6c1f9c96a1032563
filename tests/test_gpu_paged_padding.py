"""Token rows behind the last sequence may hold anything: NaN there changes no
bit of what the step's tokens get, in every kernel of the attention and in the
append."""
import pytest
import torch

from fibonacci_spaced_sparse_gb300 import api
from _paged import Cache, D, DT, HKV, HQ

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("behind", [1, 3, 64])
@pytest.mark.parametrize("lens", [[(1, 30), (0, 4), (1, 700)], [(701, 30), (2, 5), (0, 0)], [(4203, 30), (0, 9)],
                                  [(301 + s, 40) for s in range(40)] + [(0, 3)]])
def test_what_padding_rows_hold_does_not_matter(lens, behind, dtype):
    cache = Cache(lens, 16, dtype, seed=len(lens), behind=behind)
    used = int(cache.cu[-1])
    meta = cache.meta()
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn((cache.N, h, D), generator=g).to(DT[dtype]).cuda() for h in (HQ, HKV, HKV))
    w = torch.linspace(0.5, 1.5, D, device="cuda")
    got = []
    for filled in (0.25, float("nan"), float("inf")):
        for x in (q, k, v):
            x[used:] = filled
        kp, vp = cache.pages(rows_before=True)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        q_out, o = (torch.full((cache.N, HQ, D), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2))
        lse = torch.full((cache.N, HQ), 7.0, device="cuda")
        api.sfa_paged_append(k, v, kp, vp, *meta, q=q, wq=w, wk=w, q_out=q_out, status=status)
        assert bool((q_out[used:] == 7).all())
        q_out[used:] = filled
        api.sfa_paged_forward(q_out, kp, vp, *meta, alpha=0.87, W=12, out=o, lse=lse, status=status)
        assert api.sfa_read_status(status) == 0
        assert bool((o[used:] == 7).all()) and bool((lse[used:] == 7).all())
        got.append((q_out[:used], o[:used], lse[:used], kp.nan_to_num(9.0), vp.nan_to_num(9.0)))
    assert all(bool(x.isfinite().all()) for x in got[0])
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))
