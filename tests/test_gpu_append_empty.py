"""Appending to a cache whose sequences mostly bring no token: long runs of them
between two tokens, in front, and behind the last one with padding rows after it."""
import pytest
import torch

from fibonacci_spaced_sparse_gb300 import api
from _paged import Cache, D, DT, HKV, HQ

pytestmark = pytest.mark.gpu


def _lens(*parts):
    return [x for n, lens in parts for x in [lens] * n]


@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("behind", [0, 1, 70])
@pytest.mark.parametrize("lens", [_lens((1, (1, 3)), (300, (0, 2)), (1, (1, 7))), _lens((100, (1, 9)), (156, (0, 4))),
                                  _lens((40, (0, 0)), (3, (1, 0)), (40, (0, 5)), (1, (2, 1)), (1, (1, 1)), (1100, (0, 0)), (2, (1, 2))),
                                  _lens((70, (0, 1)), (1, (1, 0)), (70, (0, 1)), (1, (1, 0)), (70, (0, 1)), (1, (1, 0)), (70, (0, 1)),
                                        (1, (9, 1)), (70, (0, 1)))])
def test_runs_of_empty_sequences(lens, behind, with_q):
    cache = Cache(lens, 8, "bf16", seed=len(lens), behind=behind)
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn((cache.N, h, D), generator=g).to(DT["bf16"]).cuda() for h in (HQ, HKV, HKV))
    kp, vp = cache.pages(rows_before=True)
    want_k, want_v = kp.clone().view(-1, HKV, D), vp.clone().view(-1, HKV, D)
    for t, s, i in cache.tokens():
        row = int(cache.slots(s, i + 1)[-1])
        want_k[row], want_v[row] = k[t], v[t]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.full_like(q, 7.0) if with_q else None
    api.sfa_paged_append(k, v, kp, vp, *cache.meta(), q=q if with_q else None, q_out=q_out, rope_theta=0.0, status=status)
    assert api.sfa_read_status(status) == 0
    assert torch.equal(kp.view(-1, HKV, D).nan_to_num(9.0), want_k.nan_to_num(9.0))
    assert torch.equal(vp.view(-1, HKV, D).nan_to_num(9.0), want_v.nan_to_num(9.0))
    if with_q:
        used = int(cache.cu[-1])
        assert torch.equal(q_out[:used], q[:used]) and bool((q_out[used:] == 7).all())


@pytest.mark.parametrize("last", [True, False])
def test_a_run_of_empty_sequences_is_not_walked(last):
    """2^18 sequences without a token between two tokens, or behind one with padding
    after it.  One look-up after another would take 2^18 of them, above 100 ms; a
    search takes a few microseconds.  5 ms stands far from both."""
    S = 1 << 18
    cu = torch.ones(S + 1, dtype=torch.int32)
    cu[0] = 0
    if last:
        cu[-1] = 2
    cu = cu.cuda()
    seq = torch.ones(S, dtype=torch.int32, device="cuda")
    table = torch.arange(S, dtype=torch.int32, device="cuda")[:, None].contiguous()
    kp, vp = (torch.zeros((S, 1, HKV, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = (torch.randn((2, HKV, D), device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn((2, HQ, D), device="cuda").to(torch.bfloat16)
    times = []
    for _ in range(3):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        q_out = api.sfa_paged_append(k, v, kp, vp, table, cu, seq, q=q, q_out=torch.zeros_like(q), rope_theta=0.0)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    assert min(times) < 5.0, times
    assert torch.equal(kp[0, 0], k[0]) and torch.equal(q_out[0], q[0])
    assert torch.equal(kp[-1, 0], k[1] if last else torch.zeros_like(k[1]))
    assert torch.equal(q_out[1], q[1] if last else torch.zeros_like(q[1]))
