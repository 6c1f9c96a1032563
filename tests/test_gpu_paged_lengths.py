"""Lengths that no sequence can have, at both ends of int32: every token of such
a sequence is at a position out of range (zeros, the status bit, no access), in
every kernel of the attention and in the append."""
import pytest
import torch

from fibonacci_spaced_sparse_gb300 import api
from _paged import Cache, D, DT, HKV, HQ, attention64, within

pytestmark = pytest.mark.gpu

LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 4, 30, 700, 4200])
@pytest.mark.parametrize("length", [LOW, LOW + 1, LOW + 3, LOW + 4, LOW + 27, LOW + 28, LOW + 399, -1, HIGH - 1, HIGH])
def test_lengths_no_sequence_has(length, n, dtype):
    """The sequence of that length between two good ones."""
    cache = Cache([(3, 20), (n, 0), (2, 50)], 16, dtype, seed=7)
    table, cu, seq = cache.meta()
    seq[1] = length
    kp, vp = cache.pages()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((cache.N, HQ, D), 7.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((cache.N, HQ), 7.0, device="cuda")
    kw = dict(alpha=0.9, W=12, rungs=(20.0, 31.5))
    api.sfa_paged_forward(cache.q.cuda(), kp, vp, table, cu, seq, out=out, lse=lse, status=status, **kw)
    assert api.sfa_read_status(status) == 0x2
    bad, used = slice(3, 3 + n), n + 5
    assert bool((out[bad] == 0).all()) and bool((lse[bad] == 0).all())
    assert bool((out[used:] == 7).all()) and bool((lse[used:] == 7).all())
    ref = attention64(cache, tensor_cores=dtype == "bf16", **kw)
    for rows in (slice(0, 3), slice(n + 3, used)):
        within(out[rows], ref[0][rows], ref[2][rows])
        within(lse[rows], ref[1][rows], ref[3][rows])

    new = [torch.ones((cache.N, h, D), dtype=DT[dtype], device="cuda") for h in (HKV, HKV, HQ)]
    before = [x.clone() for x in (kp, vp)]
    status.zero_()
    q_out = api.sfa_paged_append(*new[:2], kp, vp, table, cu, seq, q=new[2], rope_theta=0.0, status=status)
    assert api.sfa_read_status(status) == 0x2
    assert bool((q_out[bad] == 0).all()) and bool((q_out[:3] == 1).all())
    rows = torch.cat((cache.slots(0)[20:], cache.slots(2)[50:])).cuda()
    for x, old in zip((kp, vp), before):
        old.view(-1, HKV, D)[rows] = 1
        assert torch.equal(x.nan_to_num(9.0), old.nan_to_num(9.0))
