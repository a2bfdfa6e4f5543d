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


# ----------------------------------------------------------------- sizes

def hollow(*shape, dtype=torch.bfloat16):
    """A tensor of any size that holds no memory."""
    return torch.empty(*shape, dtype=dtype, device="meta")


def hollow_cache(pages=5, H=2, page=16, D=64, B=2, max_pages=3):
    return linrec.KvCache(hollow(pages, H, page, D, dtype=torch.float8_e4m3fn), hollow(pages, H, D, page, dtype=torch.float8_e4m3fn),
                          hollow(pages, H, dtype=torch.float32), hollow(pages, H, dtype=torch.float32),
                          hollow(B, max_pages, dtype=torch.int32))


BIG = (1 << 32) + 16     # 16 in the low 32 bits


def test_sizes_past_32_bits_are_refused():
    """A size that the C structures would cut to its low bits is refused by name, before
    anything else looks at the call."""
    i32 = lambda *s: hollow(*s, dtype=torch.int32)  # noqa: E731
    f32 = lambda *s: hollow(*s, dtype=torch.float32)  # noqa: E731
    for B, T, C in ((BIG, 3, 8), (2, BIG, 8), (2, 3, BIG)):
        g = hollow(B, T, C)
        with pytest.raises(ValueError, match="32 bits"):
            linrec.diag_fwd(g, g)
        with pytest.raises(ValueError, match="32 bits"):
            linrec.diag_bwd(g, g, f32(1 << 40), g)
    for B, H, T in ((BIG, 2, 1), (2, BIG, 1), (2, 2, BIG)):
        q = hollow(B, H, T, 64)
        with pytest.raises(ValueError, match="32 bits"):
            linrec.step(q, q, q, None, f32(max(B, 4), H, 64, 64))
    q = hollow(2, 2, 1, 64)
    with pytest.raises(ValueError, match="32 bits"):
        linrec.step(q, q, q, None, f32(BIG, 2, 64, 64), slots=i32(2))
    for cache, B, H, T in ((hollow_cache(pages=BIG), 2, 2, 1), (hollow_cache(H=BIG), 2, BIG, 1), (hollow_cache(page=BIG), 2, 2, 1),
                           (hollow_cache(max_pages=BIG), 2, 2, 1), (hollow_cache(B=BIG), BIG, 2, 1), (hollow_cache(), 2, 2, BIG)):
        k = hollow(B, H, T, 64)
        with pytest.raises(ValueError, match="32 bits"):
            linrec.kv_append(cache, k, k, i32(B))
        with pytest.raises(ValueError, match="32 bits"):
            linrec.kv_attn(cache, k, i32(B))
    k, q = hollow(2, 2, 1, 64), hollow(2, BIG, 1, 64)
    with pytest.raises(ValueError, match="32 bits"):
        linrec.kv_append(hollow_cache(), k, k, i32(2), q=q)
    with pytest.raises(ValueError, match="32 bits"):
        linrec.kv_attn(hollow_cache(), q, i32(2))
    with pytest.raises(ValueError, match="32 bits"):
        linrec.kv_append(hollow_cache(), k, k, i32(2), inv_freq=hollow(BIG, dtype=torch.float64))


def test_sizes_within_32_bits_are_left_to_the_library():
    with pytest.raises(ValueError, match="on a GPU"):
        linrec.kv_attn(hollow_cache(max_pages=1 << 20), hollow(2, 4, 3, 64), hollow(2, dtype=torch.int32))
