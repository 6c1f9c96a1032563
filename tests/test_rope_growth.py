"""The binding's shared RoPE table: how it grows, without a GPU (tables on the
meta device, a library that records its calls)."""
import contextlib

import pytest
import torch

from fibonacci_spaced_sparse_gb300 import api

LIMIT = 1 << 24     # rows of the longest table that sfa_rope_table makes


class _Library:
    def __init__(self):
        self.rows, self.devices, self.current = [], [], None

    def sfa_rope_table_floats(self, T, D):
        return T * D

    def sfa_rope_table(self, table, T, D, theta, stream):
        self.rows.append(T)
        self.devices.append(self.current)
        return 0 if T <= LIMIT else 1


class _Stream:
    cuda_stream = 0

    def synchronize(self):
        pass


@pytest.fixture
def lib(monkeypatch):
    lib = _Library()

    @contextlib.contextmanager
    def device(d):
        before, lib.current = lib.current, torch.device(d)
        yield
        lib.current = before

    monkeypatch.setattr(api._lib, "load", lambda: lib)
    monkeypatch.setattr(api, "_rope_cache", {})
    monkeypatch.setattr(api, "_rope_outgrown", [])
    monkeypatch.setattr(torch.cuda, "device", device)
    return lib


def _table(T, index=0, **kw):
    return api.rope_table(T, torch.device("meta", index), stream=_Stream(), **kw)


def test_growth_stops_at_the_longest_table(lib):
    for T in (1, 1024, 1025, 3_000_000, 9_000_000, 10_000_000, LIMIT):
        assert _table(T).shape[0] >= T
    assert lib.rows == [1024, 2048, 3_000_000, 9_000_000, LIMIT]
    with pytest.raises(RuntimeError):
        _table(LIMIT + 1)
    assert _table(LIMIT).shape[0] == LIMIT


def test_tables_are_made_on_their_own_device(lib):
    """The launch goes to the table's device, whichever one is current."""
    for index in (0, 1, 1, 0):
        _table(10, index, rope_theta=500.0)
    assert lib.devices == [torch.device("meta", 0), torch.device("meta", 1)] and lib.current is None
