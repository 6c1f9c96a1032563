"""The 8-bit attention's workspace: what it holds before a call reaches no result, not
even with offsets that make no sense."""
import pytest
import torch

from fibonacci_spaced_sparse_gb300 import api
from _fp8 import Cache8
from _paged import D, HQ

pytestmark = pytest.mark.gpu

KW = dict(alpha=0.9, W=12, rungs=api.FIBONACCI_BASE)
LENS = [(3700, 204), (3500, 70), (33, 1200)]


def _runs(cache, cu, seq):
    """The call with four different contents of its workspace."""
    q, pages, table = cache.q.cuda(), cache.pages8(), cache.table.cuda()
    cu, seq = (torch.tensor(x, dtype=torch.int64).int().cuda() for x in (cu, seq))
    out = []
    for poison in (0x00, 0x01, 0x7f, 0xff):
        ws = torch.full((24 << 20,), poison, dtype=torch.uint8, device="cuda")
        if poison == 0x01:
            ws.view(torch.int32).fill_(1)     # page numbers and lengths that could be some
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o = torch.full((cache.N, HQ, D), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((cache.N, HQ), 7.0, device="cuda")
        api.sfa_paged_forward_fp8(q, *pages, table, cu, seq, out=o, lse=lse, status=status, workspace=ws, **KW)
        out.append((o.cpu(), lse.cpu(), api.sfa_read_status(status)))
    return out


@pytest.mark.parametrize("cu,seq", [([-4, 3700, 7200, 7233], None), ([-100000, 3700, 7200, 7233], None),
                                    ([0, 4000, 3500, 7230], [4100, 100, 4000]), ([7230, 40, 100, 7000], [900, 3904, 3904]),
                                    ([0, 3700, 7200, 9000], None), ([-(1 << 31), (1 << 31) - 1, 3000, 7230], [4000, -5, 4000]),
                                    ([0, 7233, 3600, 7200], [-(1 << 31), (1 << 31) - 1, 3700])])
def test_offsets_that_make_no_sense(cu, seq):
    cache = Cache8(LENS, 16, "bf16", 16, seed=4)
    got = _runs(cache, cu, seq or cache.seq.tolist())
    for other in got[1:]:
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got[0][:2], other[:2])) and got[0][2] == other[2]
