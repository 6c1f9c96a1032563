"""Flags without a truth value are refused with torch's own error, and the next
call is as good as any."""
import pytest
import torch

from fibonacci_spaced_sparse_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("flag", ["need_lse", "round_offsets"])
def test_flags_without_a_truth_value(flag):
    q = torch.randn((1, 8, 64), device="cuda").to(torch.bfloat16)
    kp, vp = (torch.randn((2, 16, 2, 64), device="cuda").to(torch.bfloat16) for _ in range(2))
    meta = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([[0, 1]], [0, 1], [20])]
    want = api.sfa_paged_forward(q, kp, vp, *meta, alpha=1.0, W=4)
    with pytest.raises(RuntimeError, match="ambiguous"):
        api.sfa_paged_forward(q, kp, vp, *meta, alpha=1.0, W=4, **{flag: torch.zeros(2)})
    got = api.sfa_paged_forward(q, kp, vp, *meta, alpha=1.0, W=4)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
