"""What the residual norm and the 8-bit calls refuse, without a GPU: the argument
checks of the C ABI (every call here fails them, or has nothing to launch, or
meets the injected fault) and of the Python binding."""
import ctypes
import json
import os
import subprocess
import sys

import pytest
import torch

from fibonacci_spaced_sparse_gb300 import _lib, api
from _fp8 import FP8, block_scale, codes

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, NULL = 0x100000, None           # 256-byte aligned, never dereferenced
OK, BAD, UNSUP = _lib.SFA_OK, _lib.SFA_ERR_INVALID_ARG, _lib.SFA_ERR_UNSUPPORTED
BF16, F32 = _lib.SFA_BF16, _lib.SFA_F32


@pytest.fixture(scope="module")
def lib():
    from fibonacci_spaced_sparse_gb300 import build
    build.build()
    return _lib.load()


def _p(B=2, T=64, **kw):
    return api.Params(B, T, **{"W": 12, "alpha": 1.0, **kw})


def _norm(lib, dt=BF16, N=5, dim=512, x=FAKE, xs=None, r=FAKE, rs=None, w=FAKE, eps=1e-6, h=FAKE, y=FAKE, y8=NULL, s=NULL):
    return lib.sfa_add_rms_norm(dt, N, dim, x, dim if xs is None else xs, r, dim if rs is None else rs, w, eps, h, y, y8, s, NULL)


def _quantize(lib, dt=BF16, N=5, dim=512, x=FAKE, xs=None, y8=FAKE, s=FAKE):
    return lib.sfa_quantize_rows_fp8(dt, N, dim, x, dim if xs is None else xs, y8, s, NULL)


def _bwd(lib, dt=BF16, N=500, dim=512, h=FAKE, w=FAKE, eps=1e-6, dy=FAKE, dh=NULL, dx=FAKE, dw=FAKE, ws=FAKE, nbytes=None):
    need = lib.sfa_add_rms_norm_backward_workspace_size(dt, N, dim)
    return lib.sfa_add_rms_norm_backward(dt, N, dim, h, w, eps, dy, dh, dx, dw, ws, need if nbytes is None else nbytes, NULL)


def _qkv(lib, p=None, dm=512, x=FAKE, sx=FAKE, w=FAKE, sw=FAKE, tab=FAKE, q=FAKE, k=FAKE, v=FAKE, status=NULL):
    return lib.sfa_qkv_rope_fp8((p or _p()).ref(), dm, x, sx, w, sw, tab, q, k, v, status, NULL)


def _cache(scales=FAKE, block=16, **kw):
    d = dict(k_pages=FAKE, v_pages=FAKE, num_pages=8, page_size=16, block_table=FAKE, max_pages=4, cu_q=FAKE, seq_lens=FAKE,
             N=5)
    d.update(kw)
    return _lib.SfaPagedFp8(_lib.SfaPaged(**d), scales, block)


def _append(lib, c, p=None, q=FAKE, qs=512, k=FAKE, ks=128, v=FAKE, vs=128, wq=FAKE, wk=FAKE, eps=1e-6, tab=FAKE, qh=FAKE):
    return lib.sfa_paged_append_fp8((p or _p()).ref(), ctypes.byref(c) if c is not None else None, q, qs, k, ks, v, vs, wq, wk,
                                    eps, tab, qh, NULL, NULL)


def _fwd(lib, c, p=None, q=FAKE, qs=512, o=FAKE, lse=NULL, ws=NULL, nbytes=0, status=NULL):
    return lib.sfa_paged_forward_fp8((p or _p(rope_theta=0.0)).ref(), ctypes.byref(c) if c is not None else None, q, qs, o, lse,
                                     ws, nbytes, status, NULL)


@pytest.mark.parametrize("call", [_norm, _quantize, _bwd])
def test_row_shapes(lib, call):
    for bad in (dict(dt=2), dict(dt=-1), dict(N=-1), dict(dim=0), dict(dim=-8)):
        assert call(lib, **bad) == BAD, bad
    for bad in (dict(dim=4), dict(dim=500), dict(dim=16392), dict(dim=1 << 20), dict(N=(1 << 28) + 1), dict(N=(1 << 31) - 1, dim=8)):
        assert call(lib, **bad) == UNSUP, bad
    if call is not _bwd:
        assert call(lib, N=0, x=NULL) == OK
        assert call(lib, x=NULL) == BAD and call(lib, x=FAKE + 8) == BAD
        assert call(lib, xs=504) == BAD and call(lib, xs=513) == BAD      # inside a row; not a multiple of 16 bytes
        assert call(lib, dt=F32, xs=514) == BAD


def test_norm_refusals(lib):
    assert _norm(lib, r=FAKE + 4) == BAD and _norm(lib, rs=511) == BAD and _norm(lib, rs=516) == BAD
    assert _norm(lib, w=NULL) == BAD and _norm(lib, w=FAKE + 4) == BAD
    for eps in (-1e-6, float("nan"), float("inf")):
        assert _norm(lib, eps=eps) == BAD
    assert _norm(lib, h=FAKE + 2) == BAD and _norm(lib, r=NULL) == BAD           # a sum without a residual
    assert _norm(lib, y=NULL) == BAD and _norm(lib, y8=FAKE, s=FAKE) == BAD      # neither and both
    assert _norm(lib, y=FAKE + 8) == BAD and _norm(lib, s=FAKE) == BAD
    assert _norm(lib, y=NULL, y8=FAKE) == BAD and _norm(lib, y=NULL, y8=FAKE + 4, s=FAKE) == BAD
    assert _norm(lib, y=NULL, y8=FAKE, s=FAKE + 2) == BAD
    assert _quantize(lib, y8=NULL) == BAD and _quantize(lib, y8=FAKE + 4) == BAD and _quantize(lib, s=NULL) == BAD


def test_norm_backward_refusals(lib):
    size = lib.sfa_add_rms_norm_backward_workspace_size
    need = size(BF16, 500, 512)
    assert need > 0 and size(BF16, 0, 512) == 0 and size(BF16, 8, 512) == 0 and size(BF16, 500, 500) == 0 and size(7, 500, 512) == 0
    assert size(F32, 1 << 20, 16384) <= 304 * 16384 * 4
    for bad in (dict(h=NULL), dict(dy=FAKE + 8), dict(dh=FAKE + 2), dict(dx=NULL), dict(w=NULL), dict(dw=NULL), dict(dw=FAKE + 4),
                dict(ws=NULL), dict(ws=FAKE + 16), dict(nbytes=need - 1), dict(eps=-1.0), dict(N=0, dw=NULL)):
        assert _bwd(lib, **bad) == BAD, bad


def test_projection_refusals(lib):
    assert _qkv(lib, p=_p(Hq=4)) == UNSUP and _qkv(lib, p=_p(dtype=torch.float32)) == UNSUP
    assert _qkv(lib, p=_p(B=17, T=1 << 24)) == UNSUP
    for dm in (0, 32, 100, 16448, -64):
        assert _qkv(lib, dm=dm) == BAD
    for name in ("x", "w", "q", "k", "v"):
        assert _qkv(lib, **{name: NULL}) == BAD and _qkv(lib, **{name: FAKE + 8}) == BAD, name
    for name in ("sx", "sw"):
        assert _qkv(lib, **{name: NULL}) == BAD and _qkv(lib, **{name: FAKE + 2}) == BAD, name
    assert _qkv(lib, tab=NULL) == BAD and _qkv(lib, status=FAKE + 1) == BAD
    assert _qkv(lib, p=_p(B=0), x=NULL) == OK


@pytest.mark.parametrize("call", [_append, _fwd])
def test_paged_refusals(lib, call):
    assert call(lib, None) == BAD
    for bad in (dict(num_pages=0), dict(max_pages=0), dict(page_size=0), dict(page_size=24), dict(k_pages=NULL),
                dict(v_pages=FAKE + 8), dict(block_table=NULL), dict(cu_q=FAKE + 2), dict(seq_lens=NULL), dict(N=-1),
                dict(scales=NULL), dict(scales=FAKE + 8), dict(block=0), dict(block=-16), dict(block=12), dict(block=32)):
        assert call(lib, _cache(**bad)) == BAD, bad
    assert call(lib, _cache(num_pages=1 << 27)) == UNSUP
    assert call(lib, _cache(N=(1 << 28) + 1)) == UNSUP
    assert call(lib, _cache(block=4)) == UNSUP and call(lib, _cache(page_size=4, block=4)) == UNSUP
    theta = 0.0 if call is _fwd else 1e4
    assert call(lib, _cache(), p=_p(Hkv=1, rope_theta=theta)) == UNSUP
    assert call(lib, _cache(), p=_p(T=0, rope_theta=theta)) == BAD
    assert call(lib, _cache(), q=FAKE + 8) == BAD
    assert call(lib, _cache(), qs=504) == BAD and call(lib, _cache(), qs=513) == BAD
    assert call(lib, _cache(N=0), q=NULL) == OK
    assert call(lib, _cache(), p=_p(B=0, rope_theta=theta)) == OK


def test_append_and_forward_refusals(lib):
    c = _cache()
    assert _append(lib, c, k=NULL) == BAD and _append(lib, c, v=FAKE + 8) == BAD
    assert _append(lib, c, ks=64) == BAD and _append(lib, c, vs=132) == BAD
    assert _append(lib, c, q=NULL) == BAD and _append(lib, c, qh=NULL) == BAD
    assert _append(lib, c, wk=FAKE + 8) == BAD and _append(lib, c, eps=-1.0) == BAD and _append(lib, c, tab=NULL) == BAD
    assert _fwd(lib, c, p=_p()) == BAD                                # unrotated queries
    assert _fwd(lib, c, o=NULL) == BAD and _fwd(lib, c, o=FAKE + 4) == BAD
    assert _fwd(lib, c, lse=FAKE + 4) == BAD and _fwd(lib, c, status=FAKE + 1) == BAD
    assert _fwd(lib, c, p=_p(rope_theta=0.0, W=-1)) == BAD and _fwd(lib, c, p=_p(rope_theta=0.0, alpha=0.0)) == BAD


def test_forward_workspace(lib):
    def size(c, **kw):
        return lib.sfa_paged_forward_fp8_workspace_size(_p(**{"T": 4096, "rope_theta": 0.0, **kw}).ref(), ctypes.byref(c))
    long = _cache(N=8000, num_pages=1024, max_pages=256)
    need = size(long)
    # bf16 keys and values of the tokens and of what lies before two chunks, in pages of 16 rows
    assert 2 * 8000 * 256 < need < 2 * (8000 + 2 * 1100) * 256 + (1 << 16)
    assert size(_cache(N=6999, num_pages=1024, max_pages=256)) == 0
    assert size(long, dtype=torch.float32) == 0 and size(long, W=29) == 0 and size(long, B=251) == 0 and size(long, B=0) == 0
    assert size(long, rungs=(4000.0,), B=4) == 0                      # rows far back that few queries read
    assert size(_cache(N=8000, num_pages=1024, max_pages=256, page_size=8, block=8)) == 0
    assert size(_cache(N=8000, num_pages=0)) == 0 and lib.sfa_paged_forward_fp8_workspace_size(_p().ref(), None) == 0
    p = _p(T=4096, rope_theta=0.0)
    assert _fwd(lib, long, p=p) == BAD and _fwd(lib, long, p=p, ws=FAKE, nbytes=need - 1) == BAD
    assert _fwd(lib, long, p=p, ws=FAKE + 128, nbytes=need) == BAD


CHILD = r"""
import json, sys
sys.path.insert(0, "tests")
import test_fp8_refusals as t
from fibonacci_spaced_sparse_gb300 import _lib
lib = _lib.load()
print(json.dumps([t._norm(lib), t._norm(lib, r=None, h=None), t._norm(lib, h=None), t._norm(lib, dt=t.F32, y=None, y8=t.FAKE, s=t.FAKE),
                  t._quantize(lib), t._quantize(lib, xs=520), t._bwd(lib), t._bwd(lib, N=8, ws=None), t._bwd(lib, N=0, h=None),
                  t._bwd(lib, dh=t.FAKE), t._qkv(lib), t._qkv(lib, p=t._p(rope_theta=0.0), tab=None), t._qkv(lib, dm=16384),
                  t._append(lib, t._cache()), t._append(lib, t._cache(block=8), q=None, qh=None, wq=None, wk=None),
                  t._fwd(lib, t._cache()), t._fwd(lib, t._cache(page_size=256, block=256)),
                  t._fwd(lib, t._cache(N=8000, num_pages=1024, max_pages=256), ws=t.FAKE, nbytes=1 << 30)]))
print(json.dumps([t._norm(lib, x=None), t._append(lib, t._cache(scales=None)), t._fwd(lib, t._cache(N=0))]))
"""


def test_accepted_calls_reach_the_launch(lib):
    env = dict(os.environ, SFA_TEST_FAULT="launch", PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", CHILD], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    got = [json.loads(x) for x in r.stdout.strip().splitlines()[-2:]]
    assert got[0] == [_lib.SFA_ERR_CUDA] * 18 and got[1] == [BAD, BAD, OK]


def test_binding_refuses_before_the_library(lib):
    """Shapes, types and devices that the binding turns away (CPU tensors)."""
    x, w = torch.zeros(4, 64), torch.ones(64)
    with pytest.raises(ValueError, match="CUDA"):
        api.sfa_add_rms_norm(x, x, w)
    with pytest.raises(ValueError, match="CUDA"):
        api.sfa_quantize_rows_fp8(x)
    with pytest.raises(ValueError, match="CUDA"):
        api.sfa_add_rms_norm_backward(x, w, x)
    with pytest.raises(TypeError, match="dtype"):
        api.sfa_add_rms_norm(x.half(), None, w)
    with pytest.raises(TypeError, match="tensor"):
        api.sfa_add_rms_norm(None, None, w)
    x8, w8 = x[None].to(FP8), torch.zeros(768, 64).to(FP8)
    with pytest.raises(ValueError, match="CUDA"):
        api.sfa_qkv_rope_fp8(x8, torch.ones(1, 4), w8, torch.ones(768))
    with pytest.raises(ValueError, match="x8"):
        api.sfa_qkv_rope_fp8(x[None], torch.ones(1, 4), w8, torch.ones(768))
    q, k = torch.zeros(4, 8, 64), torch.zeros(4, 2, 64)
    pages, scales, none = torch.zeros(4, 16, 2, 64), torch.ones(4, 1, 2, 2), torch.zeros(1, 2, dtype=torch.int32)
    for bad in (pages, pages.bfloat16(), pages.to(torch.uint8)):      # 8-bit pages only
        with pytest.raises(TypeError, match="float8_e4m3fn"):
            api.sfa_paged_forward_fp8(q, bad, bad, scales, none, None, None, alpha=1.0, W=12)
        with pytest.raises(TypeError, match="float8_e4m3fn"):
            api.sfa_paged_append_fp8(k, k, bad, bad, scales, none, None, None)
    with pytest.raises(TypeError, match="dtype"):                     # and the other calls take none
        api.sfa_paged_forward(q, pages.to(FP8), pages.to(FP8), none, None, None, alpha=1.0, W=12)
    with pytest.raises(ValueError, match="CUDA"):
        api.sfa_paged_forward_fp8(q, pages.to(FP8), pages.to(FP8), scales, none, None, None, alpha=1.0, W=12)
    with pytest.raises(TypeError, match="arguments"):
        api._native().add_rms_norm(x, x)


def test_scale_rule():
    """The test helper's own scale and codes at their borders."""
    assert block_scale(0.0) == 2.0 ** -100 and block_scale(448.0) == 1.0 and block_scale(448.5) == 2.0
    assert block_scale(3.5) == 2.0 ** -7 and block_scale(3.6) == 2.0 ** -6
    got = codes(torch.tensor([1.0625, 1.1875, 500.0, -1e9, float("inf"), float("nan"), 2.0 ** -10, 2.0 ** -9 * 1.5])).float()
    assert got[:4].tolist() == [1.0, 1.25, 448.0, -448.0] and bool(got[4:6].isnan().all()) and got[6:].tolist() == [0.0, 2.0 ** -8]
