"""The gradients of the norm's weights are tensors of their own."""
import pytest
import torch

from fibonacci_spaced_sparse_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [5, 200])
def test_weight_gradients_share_no_storage(T):
    q, k = (torch.randn((1, T, h, 64), device="cuda") for h in (8, 2))
    w = torch.ones(64, device="cuda")
    outs = api.sfa_qk_norm_rope_backward(q, k, w, w, q, k)
    assert len({x.untyped_storage().data_ptr() for x in outs}) == 4
    for x in outs[2:]:
        assert x.untyped_storage().nbytes() == 64 * 4 and x.storage_offset() == 0
