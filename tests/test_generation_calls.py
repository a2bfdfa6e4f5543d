"""What the binding of the generation operators hands to the library, on the
CPU: a stand-in for the library records the call's arguments, as the C side
would receive them, and writes nothing."""
import ctypes

import pytest
import torch

from state_passing_amd import linrec


class Recorder:
    """Stands in for the loaded library: sizes are 0, calls succeed and are kept."""

    def __init__(self):
        self.calls = {}

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_bytes"):
                return 0
            self.calls[name] = args
            return 0
        return call


@pytest.fixture
def recorder(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(linrec, "_lib", lambda: r)
    monkeypatch.setattr(linrec, "context", lambda device=None: None)
    monkeypatch.setattr(linrec, "_same_device", lambda first, *others: 0)
    monkeypatch.setattr(linrec, "_raw_stream", lambda index: None)
    return r


def small_cache(B=2, H=2, page=16, D=64, max_pages=3):
    return linrec.kv_cache(5, H, page, D, torch.zeros(B, max_pages, dtype=torch.int32))


# ----------------------------------------------------------------- windows

ATTN_WINDOW = 9   # its place among linrec_kv_attn's arguments


@pytest.mark.parametrize("window", [0, -1, -(1 << 31), -(1 << 40), 1 << 31, (1 << 32) + 100, 1 << 40, linrec.MAX_T,
                                    linrec.MAX_T + 1, -(1 << 32) + 7])
def test_windows_without_a_lower_bound(recorder, window):
    """Any window <= 0 or >= MAX_T means none, also where it does not fit 32 bits."""
    q = torch.zeros(2, 4, 3, 64).bfloat16()
    linrec.kv_attn(small_cache(), q, torch.zeros(2, dtype=torch.int32), window=window)
    got = ctypes.c_int32(recorder.calls["linrec_kv_attn"][ATTN_WINDOW]).value
    assert got <= 0 or got >= linrec.MAX_T


@pytest.mark.parametrize("window", [1, 100, linrec.MAX_T - 1])
def test_windows_with_a_lower_bound(recorder, window):
    q = torch.zeros(2, 4, 3, 64).bfloat16()
    linrec.kv_attn(small_cache(), q, torch.zeros(2, dtype=torch.int32), window=window)
    assert ctypes.c_int32(recorder.calls["linrec_kv_attn"][ATTN_WINDOW]).value == window


# ----------------------------------------------------------------- new outputs

@pytest.fixture
def dirty_memory(monkeypatch):
    """Memory that is not asked to be cleared comes full of NaN."""
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: empty(*a, **kw).fill_(float("nan")))


@pytest.mark.parametrize("n_new", [None, [2, 3]])
def test_rows_that_are_not_there_are_zeros_in_new_outputs(recorder, dirty_memory, n_new):
    """The calls write no row of a sequence with a negative past, n_new or not."""
    q, k = torch.zeros(2, 4, 3, 64).bfloat16(), torch.zeros(2, 2, 3, 64).bfloat16()
    past = torch.full((2,), -1, dtype=torch.int32)
    n = None if n_new is None else torch.tensor(n_new, dtype=torch.int32)
    assert (linrec.kv_attn(small_cache(), q, past, n_new=n) == 0).all()
    assert (linrec.kv_append(small_cache(), k, k, past, n_new=n, q=q) == 0).all()
