"""What the elementwise recurrence, the token step and the paged cache's calls
refuse, on the CPU: the C entries by status (with fake addresses that a refused
call must not touch; every valid-looking call stops at the NULL context, which
is checked last), the binding by exception (CPU tensors stand in for device
memory and are themselves refused last)."""
import ctypes

import pytest
import torch

from state_passing_amd import linrec

FAKE = 0x10000000
E = {v: k for k, v in linrec.STATUS.items()}
BF, F32 = linrec.BF16, linrec.F32
NONE = linrec.Tensor(None, 0, 0, 0)


def status(rc, name):
    assert rc == E[name], (linrec.STATUS.get(rc), name)


# ----------------------------------------------------------------- elementwise recurrence

def dd(B=2, T=300, C=64, form=0, dtype=BF, out=BF):
    return linrec.DiagDesc(B, T, C, form, dtype, out)


def rows(ptr=FAKE, sb=300 * 64, st=64):
    return linrec.Tensor(ptr, sb, 0, st)


def diag_fwd(d=None, g=None, x=None, h_in=None, h=None, h_out=FAKE, states=FAKE, work=FAKE):
    return linrec._lib().linrec_diag_fwd(None, ctypes.byref(d or dd()), g or rows(), x or rows(), h_in, h or rows(), h_out,
                                         states, work, None)


def diag_bwd(d=None, states=FAKE, dh=None, dh_out=None, dg=None, dx=None, dh_in=FAKE, work=FAKE):
    return linrec._lib().linrec_diag_bwd(None, ctypes.byref(d or dd()), rows(), rows(), states, dh or rows(), dh_out,
                                         dg or rows(), dx or rows(), dh_in, work, None)


def test_diag_sizes():
    assert linrec.diag_states_bytes(dd()) == 2 * 2 * 64 * 4
    assert linrec.diag_states_bytes(dd(T=256)) == 2 * 64 * 4
    assert linrec.diag_states_bytes(dd(T=0)) == 0
    assert linrec.diag_workspace_bytes(dd(T=256)) == 0
    w = linrec.diag_workspace_bytes(dd(T=257))
    assert w >= 12 * 2 * 2 * 64 and w % 16 == 0
    for bad in (dd(B=0), dd(T=-1), dd(C=0), dd(C=(1 << 20) + 1), dd(B=32768), dd(form=2), dd(dtype=3), dd(dtype=F32),
                dd(B=1000, T=linrec.MAX_T)):
        assert linrec.diag_states_bytes(bad) == 0 and linrec.diag_workspace_bytes(bad) == 0


@pytest.mark.parametrize("kw,name", [
    (dict(), "LINREC_E_NULL"), (dict(d=dd(form=7)), "LINREC_E_LAYOUT"), (dict(d=dd(dtype=F32, out=BF)), "LINREC_E_DTYPE"),
    (dict(d=dd(C=0)), "LINREC_E_SHAPE"), (dict(d=dd(T=-5)), "LINREC_E_SHAPE"),
    (dict(g=rows(None)), "LINREC_E_NULL"), (dict(g=rows(FAKE + 8)), "LINREC_E_ALIGN"),
    (dict(x=rows(st=60)), "LINREC_E_LAYOUT"), (dict(x=rows(st=68)), "LINREC_E_ALIGN"), (dict(x=rows(sb=-64)), "LINREC_E_LAYOUT"),
    (dict(h=rows(sb=0)), "LINREC_E_LAYOUT"), (dict(h=rows(sb=64, st=64)), "LINREC_E_LAYOUT"),
    (dict(x=rows(sb=0)), "LINREC_E_NULL"),                       # an input may be broadcast
    (dict(h_out=None), "LINREC_E_NULL"), (dict(h_in=FAKE + 2), "LINREC_E_ALIGN"),
    (dict(states=None), "LINREC_E_WORKSPACE"), (dict(work=None), "LINREC_E_WORKSPACE"), (dict(work=FAKE + 8), "LINREC_E_WORKSPACE"),
    (dict(d=dd(T=200), work=None), "LINREC_E_NULL"),             # short pieces need no workspace
    (dict(d=dd(T=0), g=NONE, x=NONE, h=NONE, states=None, work=None), "LINREC_E_NULL"),
])
def test_diag_fwd_statuses(kw, name):
    status(diag_fwd(**kw), name)
    if name != "LINREC_E_NULL":
        assert name != "LINREC_OK"


@pytest.mark.parametrize("kw,name", [
    (dict(), "LINREC_E_NULL"), (dict(dh=rows(FAKE + 2)), "LINREC_E_ALIGN"), (dict(dg=rows(st=32)), "LINREC_E_LAYOUT"),
    (dict(dx=rows(sb=0)), "LINREC_E_LAYOUT"), (dict(dh_in=None), "LINREC_E_NULL"), (dict(dh_out=FAKE + 1), "LINREC_E_ALIGN"),
    (dict(states=FAKE + 4), "LINREC_E_WORKSPACE"), (dict(work=None), "LINREC_E_WORKSPACE"),
])
def test_diag_bwd_statuses(kw, name):
    status(diag_bwd(**kw), name)


def test_diag_binding():
    g = torch.zeros(2, 5, 16)
    f = linrec.diag_fwd
    for exc, kw, match in [
        (ValueError, dict(g=g[0], x=g), "B,T,C"), (ValueError, dict(g=g, x=g[:, :4]), "x: shape"),
        (TypeError, dict(g=g, x=g.bfloat16()), "x: dtype"), (TypeError, dict(g=g.half(), x=g.half()), "unsupported"),
        (ValueError, dict(g=g, x=g, form="sqrt"), "form"), (TypeError, dict(g=g, x=g, out_dtype=torch.float16), "output"),
        (ValueError, dict(g=g, x=g, h_in=torch.zeros(2, 15)), "h_in: shape"),
        (TypeError, dict(g=g, x=g, h_in=torch.zeros(2, 16).double()), "h_in"),
        (ValueError, dict(g=g, x=g, h=torch.zeros(2, 5, 8)), "h: shape"),
        (ValueError, dict(g=g.transpose(1, 2).contiguous().transpose(1, 2), x=g), "contiguous"),
        (ValueError, dict(g=g, x=g, states=torch.zeros(4)), "states: .* bytes"), (ValueError, dict(g=g, x=g), "on a GPU"),
    ]:
        with pytest.raises(exc, match=match):
            f(**kw)
    st = torch.zeros(2, 16)
    b = linrec.diag_bwd
    for exc, args, kw, match in [
        (ValueError, (g, g, st[:1], g), {}, "states: .* bytes"), (TypeError, (g, g, None, g), {}, "states"),
        (ValueError, (g, g, st, g[:, :2]), {}, "dh: shape"), (ValueError, (g, g, st, g, torch.zeros(2)), {}, "dh_out: shape"),
        (TypeError, (g, g, st, g), dict(dg=g.bfloat16(), dx=g), "share one dtype"), (ValueError, (g, g, st, g), {}, "on a GPU"),
    ]:
        with pytest.raises(exc, match=match):
            b(*args, **kw)


# ----------------------------------------------------------------- token step

def act(ptr=FAKE, sb=4 * 128, sh=128, st=128):
    return linrec.Tensor(ptr, sb, sh, st)


def step(d=None, q=None, o=None, beta=None, decay=None, S=FAKE, slots=None, n=2):
    d = d or linrec.desc(2, 4, 1, 128, 128, BF, linrec.DECAY_HEAD)
    return linrec._lib().linrec_step(None, ctypes.byref(d), q or act(), act(), act(), beta or NONE,
                                     decay or linrec.Tensor(FAKE, 0, 1, 0), S, slots, n, o or act(), None)


@pytest.mark.parametrize("kw,name", [
    (dict(), "LINREC_E_NULL"), (dict(S=None), "LINREC_E_NULL"), (dict(S=FAKE + 8), "LINREC_E_ALIGN"),
    (dict(n=1), "LINREC_E_SHAPE"), (dict(n=0, slots=FAKE), "LINREC_E_SHAPE"), (dict(n=1, slots=FAKE), "LINREC_E_NULL"),
    (dict(slots=FAKE + 1), "LINREC_E_ALIGN"), (dict(q=act(FAKE + 4)), "LINREC_E_ALIGN"), (dict(q=act(sh=-128)), "LINREC_E_LAYOUT"),
    (dict(o=act(sh=0)), "LINREC_E_LAYOUT"), (dict(o=act(sb=128)), "LINREC_E_LAYOUT"), (dict(q=act(st=0)), "LINREC_E_NULL"),
    (dict(beta=linrec.Tensor(FAKE + 2, 4, 1, 1)), "LINREC_E_ALIGN"), (dict(beta=linrec.Tensor(FAKE, -4, 1, 1)), "LINREC_E_LAYOUT"),
    (dict(decay=linrec.Tensor(None, 0, 0, 0)), "LINREC_E_NULL"),
    (dict(d=linrec.desc(2, 4, 1, 96, 128, BF, 0)), "LINREC_E_SHAPE"), (dict(d=linrec.desc(2, 4, 1, 128, 128, F32, 0)), "LINREC_E_DTYPE"),
    (dict(d=linrec.desc(2, 4, 0, 128, 128, BF, 0), S=None, n=0), "LINREC_E_NULL"),
])
def test_step_statuses(kw, name):
    status(step(**kw), name)


def test_step_binding():
    q, S = torch.zeros(2, 3, 1, 64).bfloat16(), torch.zeros(4, 3, 64, 64)
    ok = dict(q=q, k=q, v=q, decay=None, S=S)
    for exc, kw, match in [
        (ValueError, dict(q=q[0]), "q: must be"), (ValueError, dict(k=q[:, :2]), "k: shape"), (TypeError, dict(v=q.float()), "v: dtype"),
        (TypeError, dict(S=S.double()), "S: must be float32"), (ValueError, dict(S=S[:, :2]), "S: shape"),
        (ValueError, dict(S=S[:1]), "1 states for 2"), (ValueError, dict(S=S.transpose(2, 3)), "S: must be contiguous"),
        (TypeError, dict(slots=torch.zeros(2).long()), "slots"), (ValueError, dict(slots=torch.zeros(3).int()), "slots: shape"),
        (ValueError, dict(beta=torch.zeros(2, 3)), "beta"), (ValueError, dict(decay=torch.zeros(2)), "decay must be"),
        (ValueError, dict(o=q[..., :32]), "o: shape"), (TypeError, dict(out_dtype=torch.float16), "output"), (ValueError, {}, "on a GPU"),
    ]:
        with pytest.raises(exc, match=match):
            linrec.step(**{**ok, **kw})


# ----------------------------------------------------------------- paged cache

def cache(**kw):
    base = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, table=FAKE, table_stride=4, pages=8, page=64, max_pages=4, H=2, D=128)
    base.update(kw)
    return linrec.KvCacheDesc(*base.values())


def kact(H=2, T=3, D=128, **kw):
    base = dict(ptr=FAKE, sb=H * T * D, sh=T * D, st=D)
    base.update(kw)
    return linrec.Tensor(*base.values())


def append(c=None, B=2, T=3, k=None, v=None, past=FAKE, n=None, freq=FAKE, rot=128, Hq=4, q=None, q_out=None, work=None):
    return linrec._lib().linrec_kv_append(None, ctypes.byref(c or cache()), B, T, k or kact(), v or kact(), past, n, freq, rot, 0, Hq,
                                          q or kact(4), q_out or kact(4), work, None)


def attn(c=None, B=2, T=3, Hq=4, q=None, past=FAKE, n=None, scale=0.1, window=0, o=None, lse=None, work=FAKE):
    return linrec._lib().linrec_kv_attn(None, ctypes.byref(c or cache()), B, T, Hq, q or kact(4), past, n, scale, window,
                                        o or kact(4), lse, work, None)


CACHE = [
    (dict(c=cache(page=48)), "LINREC_E_SHAPE"), (dict(c=cache(page=8)), "LINREC_E_SHAPE"), (dict(c=cache(D=96)), "LINREC_E_SHAPE"),
    (dict(c=cache(H=0)), "LINREC_E_SHAPE"), (dict(c=cache(pages=0)), "LINREC_E_SHAPE"), (dict(c=cache(max_pages=0)), "LINREC_E_SHAPE"),
    (dict(c=cache(max_pages=1 << 26)), "LINREC_E_SHAPE"), (dict(B=0), "LINREC_E_SHAPE"), (dict(T=-1), "LINREC_E_SHAPE"),
    (dict(c=cache(k=None)), "LINREC_E_NULL"), (dict(c=cache(v_scale=None)), "LINREC_E_NULL"), (dict(c=cache(table=None)), "LINREC_E_NULL"),
    (dict(past=None), "LINREC_E_NULL"), (dict(c=cache(v=FAKE + 8)), "LINREC_E_ALIGN"), (dict(past=FAKE + 2), "LINREC_E_ALIGN"),
    (dict(n=FAKE + 1), "LINREC_E_ALIGN"), (dict(c=cache(table_stride=-4)), "LINREC_E_LAYOUT"), (dict(), "LINREC_E_NULL"),
]


@pytest.mark.parametrize("kw,name", CACHE + [
    (dict(rot=24), "LINREC_E_SHAPE"), (dict(rot=144), "LINREC_E_SHAPE"), (dict(rot=-16), "LINREC_E_SHAPE"),
    (dict(freq=None), "LINREC_E_NULL"), (dict(freq=FAKE + 4), "LINREC_E_ALIGN"), (dict(Hq=0), "LINREC_E_SHAPE"),
    (dict(k=kact(ptr=None)), "LINREC_E_NULL"), (dict(v=kact(st=64)), "LINREC_E_LAYOUT"), (dict(q_out=kact(4, sh=0)), "LINREC_E_LAYOUT"),
    (dict(q_out=kact(4, ptr=None)), "LINREC_E_NULL"), (dict(k=kact(ptr=FAKE + 2)), "LINREC_E_ALIGN"), (dict(T=1 << 24), "LINREC_E_SHAPE"),
    (dict(B=1024, T=1), "LINREC_E_WORKSPACE"), (dict(B=1024, T=1, work=FAKE + 8), "LINREC_E_WORKSPACE"),
])
def test_append_statuses(kw, name):
    status(append(**kw), name)


@pytest.mark.parametrize("kw,name", CACHE + [
    (dict(Hq=3), "LINREC_E_SHAPE"), (dict(Hq=0), "LINREC_E_SHAPE"), (dict(scale=float("inf")), "LINREC_E_SHAPE"),
    (dict(scale=float("nan")), "LINREC_E_SHAPE"), (dict(q=kact(4, ptr=None)), "LINREC_E_NULL"), (dict(o=kact(4, sb=0)), "LINREC_E_LAYOUT"),
    (dict(lse=FAKE + 2), "LINREC_E_ALIGN"), (dict(B=30000, T=30000), "LINREC_E_SHAPE"),
    (dict(c=cache(max_pages=400), B=1, T=1, work=None), "LINREC_E_WORKSPACE"),      # split over the keys
])
def test_attn_statuses(kw, name):
    status(attn(**kw), name)


def test_append_workspace_sizes():
    size = lambda c, B, T: linrec._lib().linrec_kv_append_workspace_bytes(ctypes.byref(c), B, T)  # noqa: E731
    for B in (1, 64, 1023):
        assert size(cache(), B, 1) == 0
    assert size(cache(), 1024, 1) == 8 * cache().pages      # an owner of every page
    # (the binding does not ask below 1024 tokens)
    assert not any(size(cache(page=p), B, T) for p in (16, 128) for B, T in ((1, 1023), (511, 2), (341, 3), (2, 511)))
    assert size(cache(page=16), 1, 32768) == 8 * cache().pages and size(cache(page=128), 1, 32768) == 0
    assert size(cache(), 2048, 0) == 0 and size(cache(D=32), 2048, 1) == 0 and size(cache(page=100), 2048, 1) == 0


def test_attn_workspace_sizes():
    size = lambda c, B, T, Hq: linrec._lib().linrec_kv_attn_workspace_bytes(ctypes.byref(c), B, T, Hq)  # noqa: E731
    assert size(cache(), 2, 3, 4) == 0                      # 256 keys: one split
    w = size(cache(max_pages=400), 1, 1, 4)
    assert w > 0 and w % (4 * 130 * 4) == 0                 # splits x rows x (D + 2) floats
    assert size(cache(max_pages=400), 32767, 1, 4) == 0     # the batch fills the GPU
    for bad in (cache(D=32), cache(page=100)):
        assert size(bad, 1, 1, 4) == 0
    assert size(cache(), 1, 1, 3) == 0 and size(cache(), 1, 0, 4) == 0


def test_cache_binding():
    table = torch.zeros(2, 3, dtype=torch.int32)
    c = linrec.kv_cache(5, 2, 16, 64, table)
    k = torch.zeros(2, 2, 4, 64).bfloat16()
    q = torch.zeros(2, 4, 4, 64).bfloat16()
    past = torch.zeros(2, dtype=torch.int32)
    freq = torch.zeros(16, dtype=torch.float64)

    def app(c=c, k=k, v=k, past=past, **kw):
        linrec.kv_append(c, k, v, past, **kw)

    def att(c=c, q=q, past=past, **kw):
        linrec.kv_attn(c, q, past, **kw)

    for f in (app, att):
        for exc, kw, match in [
            (TypeError, dict(c=c._replace(k=c.k.float())), "cache.k: must be float8"),
            (ValueError, dict(c=c._replace(k=c.k[:, :, :, :32])), "contiguous"),
            (ValueError, dict(c=c._replace(v=c.k)), "cache.v: shape"),
            (ValueError, dict(c=c._replace(k_scale=c.k_scale[:4])), "k_scale: shape"),
            (ValueError, dict(c=c._replace(v_scale=None)), "scales are needed"),
            (TypeError, dict(c=c._replace(table=table.long())), "cache.table"),
            (ValueError, dict(c=c._replace(table=table[:1])), "1 rows for 2"),
            (ValueError, dict(c=c._replace(table=torch.zeros(3, 2, dtype=torch.int32).t())), "rows must be contiguous"),
            (TypeError, dict(past=None), "past"), (TypeError, dict(past=past.long()), "past"), (ValueError, dict(past=past[:1]), "past: shape"),
            (TypeError, dict(n_new=past.float()), "n_new"), (ValueError, {}, "on a GPU"),
        ]:
            with pytest.raises(exc, match=match):
                f(**kw)
    for exc, kw, match in [
        (TypeError, dict(v=k.float()), "v: dtype"), (ValueError, dict(v=k[:, :, :3]), "v: shape"), (ValueError, dict(k=k[:, :1]), "k: shape"),
        (TypeError, dict(inv_freq=freq.float()), "inv_freq"), (ValueError, dict(inv_freq=freq[None]), "inv_freq"),
        (ValueError, dict(q=q[..., :32]), "q: shape"), (ValueError, dict(q=q, q_out=q[:, :3]), "q_out: shape"),
        (ValueError, dict(q_out=q), "there is no q"),
    ]:
        with pytest.raises(exc, match=match):
            app(**kw)
    for exc, kw, match in [
        (TypeError, dict(q=q.float()), "q: dtype"), (ValueError, dict(q=q[:, :3]), "multiple"), (ValueError, dict(o=q[:, :, :2]), "o: shape"),
        (TypeError, dict(lse=torch.zeros(2, 4, 4).double()), "lse"), (ValueError, dict(lse=torch.zeros(2, 4)), "lse: shape"),
    ]:
        with pytest.raises(exc, match=match):
            att(**kw)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,H,group,T", [(1, 1, 1, 1), (1, 1, 1, 3), (3, 1, 5, 1), (1, 3, 1, 129), (1, 1, 2, 1)])
def test_attn_workspace_holds_aligned_splits(D, B, H, group, T):
    """Two splits of an odd number of rows: each has whole 16-byte vectors, so that the
    second one's are aligned as the first one's are."""
    c = cache(max_pages=16 if T > 64 else 8, H=H, D=D)      # 8 tiles of keys (16 for a piece): two splits
    w = linrec._lib().linrec_kv_attn_workspace_bytes(ctypes.byref(c), B, T, H * group)
    rows = B * H * group * T
    assert w % 32 == 0 and 0 <= w - 2 * rows * (D + 2) * 4 < 32
