"""What the norm and paged-cache calls refuse, without a GPU: the argument
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

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, NULL = 0x100000, None           # 256-byte aligned, never dereferenced
OK, BAD, UNSUP = _lib.SFA_OK, _lib.SFA_ERR_INVALID_ARG, _lib.SFA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    from fibonacci_spaced_sparse_gb300 import build
    build.build()
    return _lib.load()


def _p(B=2, T=64, **kw):
    kw = {"W": 12, "alpha": 1.0, **kw}
    return api.Params(B, T, **kw)


def _norm(lib, p=None, q=FAKE, qs=512, k=FAKE, ks=128, wq=FAKE, wk=FAKE, eps=1e-6, pos=NULL, tab=FAKE, rows=64, qh=FAKE,
          kh=FAKE, status=NULL):
    return lib.sfa_qk_norm_rope((p or _p()).ref(), q, qs, k, ks, wq, wk, eps, pos, tab, rows, qh, kh, status, NULL)


def _norm_bwd(lib, p=None, q=FAKE, qs=512, ks=128, up=FAKE, dq=FAKE, dwq=FAKE, ws=FAKE, nbytes=None, rows=64, pos=NULL):
    p = p or _p()
    need = lib.sfa_qk_norm_rope_backward_workspace_size(p.ref())
    return lib.sfa_qk_norm_rope_backward(p.ref(), q, qs, FAKE, ks, FAKE, FAKE, 1e-6, pos, FAKE, rows, up, FAKE, dq, FAKE, dwq,
                                         FAKE, ws, need if nbytes is None else nbytes, NULL, NULL)


def _cache(**kw):
    d = dict(k_pages=FAKE, v_pages=FAKE, num_pages=8, page_size=16, block_table=FAKE, max_pages=4, cu_q=FAKE, seq_lens=FAKE,
             N=5)
    d.update(kw)
    return _lib.SfaPaged(**d)


def _append(lib, c, p=None, q=FAKE, qs=512, k=FAKE, ks=128, v=FAKE, vs=128, wq=FAKE, wk=FAKE, eps=1e-6, tab=FAKE, qh=FAKE):
    return lib.sfa_paged_append((p or _p()).ref(), ctypes.byref(c) if c is not None else None, q, qs, k, ks, v, vs, wq, wk,
                                eps, tab, qh, NULL, NULL)


def _fwd(lib, c, p=None, q=FAKE, qs=512, o=FAKE, lse=NULL, status=NULL):
    return lib.sfa_paged_forward((p or _p(rope_theta=0.0)).ref(), ctypes.byref(c) if c is not None else None, q, qs, o, lse,
                                 status, NULL)


@pytest.mark.parametrize("call", [_norm, _norm_bwd])
def test_norm_refusals(lib, call):
    assert call(lib, p=_p(Hq=4)) == UNSUP
    assert call(lib, p=_p(D=128)) == UNSUP
    assert call(lib, p=_p(B=17, T=1 << 24)) == UNSUP
    assert call(lib, q=NULL) == BAD
    assert call(lib, q=FAKE + 8) == BAD
    assert call(lib, qs=511) == BAD and call(lib, qs=516) == BAD      # inside a row; not a multiple of 16 bytes
    assert call(lib, ks=64) == BAD
    assert call(lib, rows=63) == BAD                                  # a table shorter than the sequence
    assert call(lib, rows=-1, pos=FAKE) == BAD and call(lib, rows=0, pos=FAKE) == BAD
    assert call(lib, pos=FAKE + 2) == BAD


def test_norm_forward_refusals(lib):
    assert _norm(lib, wq=NULL) == BAD and _norm(lib, wk=FAKE + 4) == BAD
    for eps in (-1e-6, float("nan"), float("inf")):
        assert _norm(lib, eps=eps) == BAD
    assert _norm(lib, tab=NULL) == BAD
    assert _norm(lib, qh=NULL) == BAD and _norm(lib, kh=FAKE + 4) == BAD
    assert _norm(lib, status=FAKE + 1) == BAD
    assert _norm(lib, p=_p(B=0), q=NULL, k=NULL, qh=NULL, kh=NULL) == OK
    assert lib.sfa_qk_norm_rope(None, FAKE, 512, FAKE, 128, FAKE, FAKE, 1e-6, NULL, FAKE, 64, FAKE, FAKE, NULL, NULL) == BAD


def test_norm_backward_refusals(lib):
    p = _p()
    need = lib.sfa_qk_norm_rope_backward_workspace_size(p.ref())
    assert need > 0 and lib.sfa_qk_norm_rope_backward_workspace_size(_p(B=0).ref()) == 0
    few, more = (lib.sfa_qk_norm_rope_backward_workspace_size(_p(B=1, T=n).ref()) for n in (64, 65))
    assert few == 0 and more == need
    assert _norm_bwd(lib, nbytes=need - 1) == BAD
    assert _norm_bwd(lib, ws=NULL) == BAD and _norm_bwd(lib, ws=FAKE + 16) == BAD
    assert _norm_bwd(lib, up=NULL) == BAD and _norm_bwd(lib, dq=FAKE + 2) == BAD
    assert _norm_bwd(lib, dwq=NULL) == BAD and _norm_bwd(lib, p=_p(B=0), dwq=NULL) == BAD


@pytest.mark.parametrize("call", [_append, _fwd])
def test_paged_refusals(lib, call):
    assert call(lib, None) == BAD
    for bad in (dict(num_pages=0), dict(max_pages=0), dict(page_size=0), dict(page_size=24), dict(page_size=-16),
                dict(k_pages=NULL), dict(v_pages=FAKE + 8), dict(block_table=NULL), dict(cu_q=FAKE + 2), dict(seq_lens=NULL),
                dict(N=-1)):
        assert call(lib, _cache(**bad)) == BAD, bad
    assert call(lib, _cache(num_pages=1 << 27)) == UNSUP              # 2^31 rows
    assert call(lib, _cache(N=(1 << 28) + 1)) == UNSUP
    theta = 0.0 if call is _fwd else 1e4
    assert call(lib, _cache(), p=_p(Hkv=1, rope_theta=theta)) == UNSUP
    assert call(lib, _cache(), p=_p(T=0, rope_theta=theta)) == BAD
    assert call(lib, _cache(), p=_p(T=1 << 25, rope_theta=theta)) == UNSUP
    assert call(lib, _cache(), q=FAKE + 8) == BAD
    assert call(lib, _cache(), qs=504) == BAD and call(lib, _cache(), qs=513) == BAD
    # nothing to do
    assert call(lib, _cache(N=0), q=NULL) == OK
    assert call(lib, _cache(), p=_p(B=0, rope_theta=theta)) == OK


def test_append_refusals(lib):
    c = _cache()
    assert _append(lib, c, k=NULL) == BAD and _append(lib, c, v=FAKE + 8) == BAD
    assert _append(lib, c, ks=64) == BAD and _append(lib, c, vs=132) == BAD
    assert _append(lib, c, q=NULL) == BAD and _append(lib, c, qh=NULL) == BAD   # one without the other
    assert _append(lib, c, wk=FAKE + 8) == BAD and _append(lib, c, eps=-1.0) == BAD
    assert _append(lib, c, tab=NULL) == BAD


def test_forward_refusals(lib):
    c = _cache()
    assert _fwd(lib, c, p=_p()) == BAD                                # unrotated queries
    assert _fwd(lib, c, o=NULL) == BAD and _fwd(lib, c, o=FAKE + 4) == BAD
    assert _fwd(lib, c, lse=FAKE + 2) == BAD and _fwd(lib, c, lse=FAKE + 4) == BAD and _fwd(lib, c, status=FAKE + 1) == BAD
    assert _fwd(lib, c, p=_p(rope_theta=0.0, W=-1)) == BAD
    assert _fwd(lib, c, p=_p(rope_theta=0.0, alpha=0.0)) == BAD


CHILD = r"""
import json, sys
sys.path.insert(0, "tests")
import test_paged_refusals as t
from fibonacci_spaced_sparse_gb300 import _lib
lib = _lib.load()
empty = t._p(B=0)
print(json.dumps([t._norm(lib), t._norm_bwd(lib), t._norm_bwd(lib, p=empty), t._append(lib, t._cache()),
                  t._append(lib, t._cache(), q=None, qh=None, wq=None, wk=None), t._fwd(lib, t._cache()),
                  t._fwd(lib, t._cache(), p=t._p(B=1 << 20, T=1 << 24, rope_theta=0.0)),
                  t._norm(lib, rows=1, pos=t.FAKE), t._norm(lib, p=t._p(rope_theta=0.0), tab=None, rows=0), t._norm_bwd(lib, p=t._p(B=1), ws=None)]))
print(json.dumps([t._norm(lib, q=None), t._append(lib, t._cache(k_pages=None)), t._fwd(lib, t._cache(N=0))]))
"""


def test_accepted_calls_reach_the_launch(lib):
    """Calls that pass every check meet the injected launch fault; those that
    fail one, or have nothing to launch, do not."""
    env = dict(os.environ, SFA_TEST_FAULT="launch", PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", CHILD], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    got = [json.loads(x) for x in r.stdout.strip().splitlines()[-2:]]
    assert got[0] == [_lib.SFA_ERR_CUDA] * 10 and got[1] == [BAD, BAD, OK]


def test_binding_refuses_before_the_library(lib):
    """Shapes, types and devices that the binding turns away (CPU tensors)."""
    q, k = torch.zeros(1, 4, 8, 64), torch.zeros(1, 4, 2, 64)
    w = torch.ones(64)
    with pytest.raises(ValueError, match="CUDA"):
        api.sfa_qk_norm_rope(q, k, w, w)
    with pytest.raises(ValueError, match="must be"):
        api.sfa_qk_norm_rope(q[0], k, w, w)
    with pytest.raises(TypeError, match="dtype"):
        api.sfa_qk_norm_rope(q.half(), k.half(), w, w)
    with pytest.raises(TypeError, match="tensor"):
        api._native().norm_rope(None, k, w, w, 1e-6, 0.0, None, None, None, None, None)
    with pytest.raises(TypeError, match="arguments"):
        api._native().norm_rope(q, k)
    pages = torch.zeros(4, 16, 2, 64)
    with pytest.raises(ValueError, match="k_pages"):
        api.sfa_paged_append(k[0], k[0], pages, pages, torch.zeros(1, 2, dtype=torch.int32), None, None)
    with pytest.raises(ValueError, match="k_pages"):
        api.sfa_paged_forward(q[0], pages, pages, None, None, None, alpha=1.0, W=12)
    with pytest.raises(ValueError, match="must be"):
        api.sfa_paged_forward(q, pages, pages, None, None, None, alpha=1.0, W=12)


def test_token_strides_of_the_binding(lib):
    stride = api._native().stride_of
    x = torch.zeros(3, 5, 768)
    q, k = x[..., :512].unflatten(-1, (8, 64)), x[..., 512:640].unflatten(-1, (2, 64))
    assert stride(q, 8) == 768 and stride(k, 2) == 768
    assert stride(q[:, :1], 8) == 5 * 768             # single tokens of a longer batch
    assert stride(q[0], 8) == 768
    assert stride(q[:1, :1], 8) == 512                # one token: any stride
    assert stride(q[:0], 8) == 512
    bad = (q[:, :3],                                  # sequences further apart than their tokens
           q.transpose(0, 1), q.transpose(2, 3).contiguous().transpose(2, 3),
           torch.zeros(1, 1, 8, 64).expand(3, 5, 8, 64),
           torch.zeros(3, 5, 516, dtype=torch.bfloat16)[..., :512].unflatten(-1, (8, 64)),  # 1032 bytes apart
           q[..., :32], x[..., :384].unflatten(-1, (8, 48)))
    for t in bad:
        with pytest.raises(ValueError):
            stride(t, 8)


def test_missing_binding_fails_loudly(lib, monkeypatch, tmp_path):
    monkeypatch.setattr(_lib, "_bind", None)
    monkeypatch.setattr(_lib, "BIND_PATH", str(tmp_path / "nope.so"))
    with pytest.raises(RuntimeError, match="not built"):
        _lib.bind()
