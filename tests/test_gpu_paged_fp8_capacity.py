"""The 8-bit attention through the C ABI with capacities of every remainder: what a
token gets goes by its position, not by how near the capacity is."""
import ctypes

import pytest
import torch

from fibonacci_spaced_sparse_gb300 import _lib, api
from _fp8 import Cache8
from _fp8_exact import forward64, fp32_bounds, halves_bound
from _paged import D, HQ, within

pytestmark = pytest.mark.gpu


def _forward(cache, pages, T, W, alpha, poison):
    """sfa_paged_forward_fp8 with the capacity T; the workspace holds `poison` on entry."""
    lib = _lib.load()
    kp, vp, sc = pages
    table, cu, seq = cache.meta()
    q = cache.q.cuda()
    p = api.Params(len(cache.lens), T, W=W, alpha=alpha, rope_theta=0.0)
    c = _lib.SfaPagedFp8(_lib.SfaPaged(k_pages=kp.data_ptr(), v_pages=vp.data_ptr(), num_pages=kp.shape[0], page_size=cache.page,
                                       block_table=table.data_ptr(), max_pages=table.shape[1], cu_q=cu.data_ptr(),
                                       seq_lens=seq.data_ptr(), N=cache.N), sc.data_ptr(), cache.block)
    need = lib.sfa_paged_forward_fp8_workspace_size(p.ref(), ctypes.byref(c))
    ws = torch.full((max(need, 1),), poison, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.full((cache.N, HQ, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((cache.N, HQ), 7.0, device="cuda")
    st = lib.sfa_paged_forward_fp8(p.ref(), ctypes.byref(c), q.data_ptr(), HQ * D, o.data_ptr(), lse.data_ptr(),
                                   ws.data_ptr() if need else None, need, status.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == _lib.SFA_OK
    return o, lse, api.sfa_read_status(status), need


@pytest.mark.parametrize("lens,page,W,alpha", [([(7039, 1051)], 64, 12, 1.0), ([(7035, 1144)], 32, 12, 1.0),
                                               ([(7051, 1081)], 16, 12, 1.0), ([(7032, 1883)], 128, 12, 1.0),
                                               ([(6999, 2047), (64, 1)], 64, 5, 0.9)])
def test_capacities_of_every_remainder(lens, page, W, alpha):
    cache = Cache8(lens, page, "bf16", 16, seed=page, behind=0)
    pages = cache.pages8()
    ref = forward64(cache, alpha=alpha, W=W, rungs=api.FIBONACCI_BASE)
    bo, bl = fp32_bounds(ref, "bf16")
    used, length = ref[0].shape[0], max(n + c for n, c in lens)
    room = cache.max_pages * page
    for T in [*range(length, room, 5), room - 1, room, room + 5]:
        o, lse, status, need = _forward(cache, pages, T, W, alpha, poison=0xff)
        assert need > 0 and status == 0, T
        within(o[:used], ref[0], bo + halves_bound(ref), f"o, T = {T}")
        within(lse[:used], ref[1], bl, f"lse, T = {T}")


@pytest.mark.parametrize("T", [8090, 8101, 8128, 8129, 8150, 8192])
def test_tokens_past_the_capacity(T):
    """A sequence longer than the capacity beside one inside it: the tokens behind the
    capacity get zeros and are reported, the others their results."""
    lens = [(7039, 1051), (200, 8050)]
    cache = Cache8(lens, 64, "bf16", 16, seed=T, behind=0)
    ref = forward64(cache, alpha=1.0, W=12, rungs=api.FIBONACCI_BASE)
    o, lse, status, _ = _forward(cache, cache.pages8(), T, 12, 1.0, poison=0x11)
    assert status == 0x2
    pos = torch.cat([torch.arange(c, c + n) for n, c in lens])
    there = pos < T
    bo, bl = fp32_bounds(ref, "bf16")
    used = ref[0].shape[0]
    within(o[:used].cpu()[there], ref[0][there], (bo + halves_bound(ref))[there], "o")
    within(lse[:used].cpu()[there], ref[1][there], bl[there], "lse")
    assert bool((o[:used].cpu()[~there] == 0).all()) and bool((lse[:used].cpu()[~there] == 0).all())
