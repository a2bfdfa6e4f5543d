"""What the causal convolution's and the state-space scan's calls refuse, on the
CPU: the C entries by status (with fake addresses that a refused call must not
touch; every valid-looking call stops at the NULL context, which is checked
last), the binding by exception (CPU tensors stand in for device memory and are
themselves refused last)."""
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


def rows(ptr=FAKE, sb=300 * 64, st=64):
    return linrec.Tensor(ptr, sb, 0, st)


# ----------------------------------------------------------------- convolution

def cd(B=2, T=300, C=64, K=4, act=1, dtype=BF, out=BF):
    return linrec.ConvDesc(B, T, C, K, act, dtype, out)


def conv_fwd(d=None, x=None, w=FAKE, bias=None, s_in=None, n=None, y=None, s_out=FAKE):
    return linrec._lib().linrec_conv_fwd(None, ctypes.byref(d or cd()), x or rows(), w, bias, s_in, n, y or rows(), s_out, None)


def conv_bwd(d=None, x=None, w=FAKE, bias=None, s_in=None, n=None, dy=None, ds_out=None, dx=None, dw=FAKE, db=None, ds_in=FAKE,
             work=FAKE):
    return linrec._lib().linrec_conv_bwd(None, ctypes.byref(d or cd()), x or rows(), w, bias, s_in, n, dy or rows(), ds_out,
                                         dx or rows(), dw, db, ds_in, work, None)


def conv_step(d=None, x=None, w=FAKE, S=FAKE, slots=None, n=2, y=None):
    return linrec._lib().linrec_conv_step(None, ctypes.byref(d or cd()), x or rows(), w, None, S, slots, n, y or rows(), None)


DESCS = [
    (dict(d=cd(B=0)), "LINREC_E_SHAPE"), (dict(d=cd(B=32768)), "LINREC_E_SHAPE"), (dict(d=cd(T=-1)), "LINREC_E_SHAPE"),
    (dict(d=cd(C=0)), "LINREC_E_SHAPE"), (dict(d=cd(C=(1 << 20) + 1)), "LINREC_E_SHAPE"), (dict(d=cd(K=1)), "LINREC_E_SHAPE"),
    (dict(d=cd(K=5)), "LINREC_E_SHAPE"), (dict(d=cd(act=2)), "LINREC_E_LAYOUT"), (dict(d=cd(dtype=2)), "LINREC_E_DTYPE"),
    (dict(d=cd(dtype=F32)), "LINREC_E_DTYPE"), (dict(d=cd(T=linrec.MAX_T, C=1 << 20)), "LINREC_E_SHAPE"),
    (dict(x=rows(None)), "LINREC_E_NULL"), (dict(x=rows(FAKE + 8)), "LINREC_E_ALIGN"), (dict(x=rows(st=60)), "LINREC_E_LAYOUT"),
    (dict(x=rows(st=68)), "LINREC_E_ALIGN"), (dict(x=rows(sb=-64)), "LINREC_E_LAYOUT"), (dict(x=rows(sb=0)), "LINREC_E_NULL"),
    (dict(w=None), "LINREC_E_NULL"), (dict(w=FAKE + 2), "LINREC_E_ALIGN"), (dict(), "LINREC_E_NULL"),
]


@pytest.mark.parametrize("kw,name", DESCS + [
    (dict(bias=FAKE + 1), "LINREC_E_ALIGN"), (dict(y=rows(sb=0)), "LINREC_E_LAYOUT"), (dict(y=rows(sb=64)), "LINREC_E_LAYOUT"),
    (dict(s_out=None), "LINREC_E_NULL"), (dict(s_in=FAKE + 2), "LINREC_E_ALIGN"), (dict(n=FAKE + 2), "LINREC_E_ALIGN"),
    (dict(d=cd(T=0), x=NONE, w=None, y=NONE), "LINREC_E_NULL"),
])
def test_conv_fwd_statuses(kw, name):
    status(conv_fwd(**kw), name)


@pytest.mark.parametrize("kw,name", DESCS + [
    (dict(dy=rows(FAKE + 2)), "LINREC_E_ALIGN"), (dict(dx=rows(st=32)), "LINREC_E_LAYOUT"), (dict(dx=rows(sb=0)), "LINREC_E_LAYOUT"),
    (dict(dw=None), "LINREC_E_NULL"), (dict(db=FAKE + 2), "LINREC_E_ALIGN"), (dict(ds_in=None), "LINREC_E_NULL"),
    (dict(ds_out=FAKE + 1), "LINREC_E_ALIGN"), (dict(work=None), "LINREC_E_WORKSPACE"), (dict(work=FAKE + 4), "LINREC_E_WORKSPACE"),
    (dict(d=cd(T=0), x=NONE, w=None, dy=NONE, dx=NONE, work=None), "LINREC_E_NULL"),
])
def test_conv_bwd_statuses(kw, name):
    status(conv_bwd(**kw), name)


@pytest.mark.parametrize("kw,name", DESCS + [
    (dict(S=None), "LINREC_E_NULL"), (dict(S=FAKE + 2), "LINREC_E_ALIGN"), (dict(n=1), "LINREC_E_SHAPE"),
    (dict(n=0, slots=FAKE), "LINREC_E_SHAPE"), (dict(n=1, slots=FAKE), "LINREC_E_NULL"), (dict(slots=FAKE + 2), "LINREC_E_ALIGN"),
    (dict(y=rows(sb=0)), "LINREC_E_LAYOUT"), (dict(d=cd(T=0), S=None, n=0), "LINREC_E_NULL"),
])
def test_conv_step_statuses(kw, name):
    status(conv_step(**kw), name)


def test_conv_launches_fit():
    """Every direction's own grid: the fp32 forward has 128 tokens and 256 channels a workgroup, 256 threads
    each (4096 times 4095 workgroups are the most below 2^32 threads), the others 256 tokens."""
    wide = 1 << 20

    def fwd(T, dtype):
        at = rows(sb=T * wide, st=wide)
        return conv_fwd(d=cd(B=1, T=T, C=wide, dtype=dtype, out=F32), x=at, y=at)

    def bwd(T, dtype):
        at = rows(sb=T * wide, st=wide)
        return conv_bwd(d=cd(B=1, T=T, C=wide, dtype=dtype, out=F32), x=at, dy=at, dx=at)

    for call, dtype, most in ((fwd, F32, 4095 * 128), (fwd, BF, 4095 * 256), (bwd, F32, 4095 * 256), (bwd, BF, 4095 * 256)):
        status(call(most, dtype), "LINREC_E_NULL")      # the context
        status(call(most + 1, dtype), "LINREC_E_SHAPE")


def test_conv_sizes():
    size = lambda d: linrec._lib().linrec_conv_bwd_workspace_bytes(ctypes.byref(d))  # noqa: E731
    assert size(cd(T=0)) == 0 and size(cd(K=7)) == 0 and size(cd(C=0)) == 0
    assert size(cd()) % 16 == 0 and size(cd()) >= 2 * 3 * 64 * 4 + 5 * 64 * 4
    assert size(cd(T=600)) > size(cd())


def test_conv_binding():
    x, w, b, S = torch.zeros(2, 5, 16), torch.zeros(16, 4), torch.zeros(16), torch.zeros(2, 3, 16)
    n = torch.zeros(2, dtype=torch.int32)
    ok = dict(x=x, w=w)
    for exc, kw, match in [
        (ValueError, dict(x=x[0]), "B,T,C"), (TypeError, dict(x=x.half()), "unsupported"), (ValueError, dict(w=b), "w: must be"),
        (ValueError, dict(w=w.t()), "w: shape"), (ValueError, dict(w=torch.zeros(4, 16).t()), "w: must be contiguous"),
        (TypeError, dict(w=w.bfloat16()), "w: must be float32"), (ValueError, dict(bias=b[:8]), "bias: shape"),
        (ValueError, dict(act="gelu"), "act"), (ValueError, dict(state_in=S[:, :2]), "state_in: shape"),
        (TypeError, dict(n_new=n.long()), "n_new"), (ValueError, dict(n_new=n[:1]), "n_new: shape"),
        (ValueError, dict(y=x[:, :4]), "y: shape"), (TypeError, dict(out_dtype=torch.float16), "output"),
        (ValueError, dict(x=x.transpose(1, 2).contiguous().transpose(1, 2)), "contiguous"), (ValueError, {}, "on a GPU"),
    ]:
        with pytest.raises(exc, match=match):
            linrec.conv_fwd(**{**ok, **kw})
    for exc, kw, match in [
        (ValueError, dict(dy=x[:, :2]), "dy: shape"), (TypeError, dict(dy=x.bfloat16()), "dy: dtype"),
        (ValueError, dict(dstate_out=S[:1]), "dstate_out: shape"), (ValueError, dict(dw=w.t()), "dw: shape"),
        (ValueError, dict(dstate_in=S[:1]), "dstate_in: shape"), (ValueError, dict(workspace=torch.zeros(4)), "workspace: .* bytes"),
        (ValueError, {}, "on a GPU"),
    ]:
        with pytest.raises(exc, match=match):
            linrec.conv_bwd(**{**dict(x=x, w=w, bias=b, state_in=S, dy=x), **kw})
    for exc, kw, match in [
        (ValueError, dict(S=S[:, :2]), "S: shape"), (ValueError, dict(S=S[:1]), "1 states for 2"), (ValueError, dict(S=S[0]), "S: must be"),
        (TypeError, dict(S=S.double()), "S: must be float32"), (TypeError, dict(slots=n.long()), "slots"), (ValueError, {}, "on a GPU"),
    ]:
        with pytest.raises(exc, match=match):
            linrec.conv_step(**{**dict(x=x, w=w, bias=b, S=S), **kw})


# ----------------------------------------------------------------- scan

def sd(B=2, T=300, C=64, N=16, G=1, sp=1, dtype=BF, out=BF):
    return linrec.ScanDesc(B, T, C, N, G, sp, dtype, out)


def proj(ptr=FAKE, sb=2 * 300 * 16, sh=300 * 16, st=16):
    return linrec.Tensor(ptr, sb, sh, st)


def inputs(**kw):
    base = dict(x=rows(), dt=rows(), b=proj(), c=proj(), z=NONE, A=FAKE, D=None, dt_bias=None)
    base.update(kw)
    return linrec.ScanInputs(*base.values())


def grads(**kw):
    base = dict(dx=rows(), ddt=rows(), db=proj(), dc=proj(), dz=NONE, dA=FAKE, dD=None, ddt_bias=None, dh_in=FAKE)
    base.update(kw)
    return linrec.ScanGradsDesc(*base.values())


def ref(s):
    return None if s is None else ctypes.byref(s)


def scan_fwd(d=None, i=0, h_in=None, n=None, y=None, h_out=FAKE, saved=None, work=FAKE):
    return linrec._lib().linrec_scan_fwd(None, ref(d or sd()), ref(inputs() if i == 0 else i), h_in, n, y or rows(), h_out, saved,
                                         work, None)


def scan_bwd(d=None, i=0, saved=FAKE, n=None, dy=None, dh_out=None, o=0, work=FAKE):
    return linrec._lib().linrec_scan_bwd(None, ref(d or sd()), ref(inputs() if i == 0 else i), saved, n, dy or rows(), dh_out,
                                         ref(grads() if o == 0 else o), work, None)


def scan_step(d=None, i=0, S=FAKE, slots=None, n=2, y=None):
    return linrec._lib().linrec_scan_step(None, ref(d or sd()), ref(inputs() if i == 0 else i), S, slots, n, y or rows(), None)


SCAN = [
    (dict(d=sd(B=0)), "LINREC_E_SHAPE"), (dict(d=sd(B=32768)), "LINREC_E_SHAPE"), (dict(d=sd(T=-1)), "LINREC_E_SHAPE"),
    (dict(d=sd(C=0)), "LINREC_E_SHAPE"), (dict(d=sd(C=(1 << 20) + 8)), "LINREC_E_SHAPE"), (dict(d=sd(N=12)), "LINREC_E_SHAPE"),
    (dict(d=sd(N=128)), "LINREC_E_SHAPE"), (dict(d=sd(G=3)), "LINREC_E_SHAPE"), (dict(d=sd(G=0)), "LINREC_E_SHAPE"),
    (dict(d=sd(G=16)), "LINREC_E_SHAPE"), (dict(d=sd(G=2)), "LINREC_E_NULL"), (dict(d=sd(sp=2)), "LINREC_E_LAYOUT"),
    (dict(d=sd(dtype=F32)), "LINREC_E_DTYPE"), (dict(d=sd(out=5)), "LINREC_E_DTYPE"), (dict(i=None), "LINREC_E_NULL"),
    (dict(i=inputs(x=rows(None))), "LINREC_E_NULL"), (dict(i=inputs(dt=rows(st=32))), "LINREC_E_LAYOUT"),
    (dict(i=inputs(b=proj(FAKE + 8))), "LINREC_E_ALIGN"), (dict(i=inputs(c=proj(st=20))), "LINREC_E_ALIGN"),
    (dict(i=inputs(c=proj(st=8))), "LINREC_E_LAYOUT"), (dict(i=inputs(z=rows(FAKE + 2))), "LINREC_E_ALIGN"),
    (dict(i=inputs(A=None)), "LINREC_E_NULL"), (dict(i=inputs(A=FAKE + 1)), "LINREC_E_ALIGN"), (dict(i=inputs(D=FAKE + 2)), "LINREC_E_ALIGN"),
    (dict(i=inputs(dt_bias=FAKE + 2)), "LINREC_E_ALIGN"), (dict(), "LINREC_E_NULL"),
]


@pytest.mark.parametrize("kw,name", SCAN + [
    (dict(h_out=None), "LINREC_E_NULL"), (dict(h_in=FAKE + 2), "LINREC_E_ALIGN"), (dict(n=FAKE + 1), "LINREC_E_ALIGN"),
    (dict(y=rows(sb=0)), "LINREC_E_LAYOUT"), (dict(saved=FAKE + 8), "LINREC_E_WORKSPACE"), (dict(work=None), "LINREC_E_WORKSPACE"),
    (dict(d=sd(T=64), work=None), "LINREC_E_NULL"),      # not split: no workspace
    (dict(d=sd(T=0), i=None, y=NONE, work=None), "LINREC_E_NULL"),
])
def test_scan_fwd_statuses(kw, name):
    status(scan_fwd(**kw), name)


@pytest.mark.parametrize("kw,name", SCAN + [
    (dict(saved=None), "LINREC_E_WORKSPACE"), (dict(work=None), "LINREC_E_WORKSPACE"), (dict(work=FAKE + 8), "LINREC_E_WORKSPACE"),
    (dict(dy=rows(None)), "LINREC_E_NULL"), (dict(dh_out=FAKE + 2), "LINREC_E_ALIGN"), (dict(o=None), "LINREC_E_NULL"),
    (dict(o=grads(dA=None)), "LINREC_E_NULL"), (dict(o=grads(dh_in=None)), "LINREC_E_NULL"), (dict(o=grads(dD=FAKE + 2)), "LINREC_E_ALIGN"),
    (dict(o=grads(dx=rows(sb=0))), "LINREC_E_LAYOUT"), (dict(o=grads(db=proj(sb=0))), "LINREC_E_LAYOUT"),
    (dict(o=grads(dc=proj(None))), "LINREC_E_NULL"), (dict(i=inputs(z=rows())), "LINREC_E_NULL"),   # a z, and no dz
    (dict(d=sd(T=0), i=None, saved=None, work=None), "LINREC_E_NULL"),
])
def test_scan_bwd_statuses(kw, name):
    status(scan_bwd(**kw), name)


@pytest.mark.parametrize("kw,name", SCAN + [
    (dict(S=None), "LINREC_E_NULL"), (dict(S=FAKE + 4), "LINREC_E_ALIGN"), (dict(n=1), "LINREC_E_SHAPE"),
    (dict(n=0, slots=FAKE), "LINREC_E_SHAPE"), (dict(n=1, slots=FAKE), "LINREC_E_NULL"), (dict(slots=FAKE + 3), "LINREC_E_ALIGN"),
    (dict(d=sd(T=0), i=None, S=None, n=0), "LINREC_E_NULL"),
])
def test_scan_step_statuses(kw, name):
    status(scan_step(**kw), name)


def test_scan_sizes():
    lib = linrec._lib()
    for f in (lib.linrec_scan_saved_bytes, lib.linrec_scan_fwd_workspace_bytes, lib.linrec_scan_bwd_workspace_bytes):
        for bad in (sd(T=0), sd(N=10), sd(C=0), sd(G=7), sd(dtype=9)):
            assert f(ctypes.byref(bad)) == 0
        assert f(ctypes.byref(sd())) % 16 == 0
    assert lib.linrec_scan_fwd_workspace_bytes(ctypes.byref(sd(T=64))) == 0
    # a state a block of tokens, and the whole of long pieces in 64 bits
    one = lib.linrec_scan_saved_bytes(ctypes.byref(sd(T=1)))
    assert one == 2 * 64 * 16 * 4
    assert lib.linrec_scan_saved_bytes(ctypes.byref(sd(T=1 << 30))) >= one * (1 << 26)


def test_scan_binding():
    x, A, D = torch.zeros(2, 5, 16), torch.zeros(16, 8), torch.zeros(16)
    B, h = torch.zeros(2, 1, 5, 8), torch.zeros(2, 16, 8)
    n = torch.zeros(2, dtype=torch.int32)
    ok = dict(x=x, dt=x, A=A, B=B, C=B)
    for exc, kw, match in [
        (ValueError, dict(x=x[0]), "B,T,C"), (TypeError, dict(x=x.half()), "unsupported"), (ValueError, dict(dt=x[:, :2]), "dt: shape"),
        (TypeError, dict(dt=x.bfloat16()), "dt: dtype"), (ValueError, dict(B=x), "B: must be"), (ValueError, dict(C=B[:, :, :4]), "C: shape"),
        (ValueError, dict(C=torch.zeros(2, 2, 5, 8)), "C: shape"), (ValueError, dict(A=A[:, :4]), "A: shape"), (TypeError, dict(A=None), "A"),
        (TypeError, dict(A=A.double()), "A: must be float32"), (ValueError, dict(A=torch.zeros(8, 16).t()), "A: must be contiguous"),
        (ValueError, dict(D=D[:3]), "D: shape"), (ValueError, dict(dt_bias=D[:3]), "dt_bias: shape"), (ValueError, dict(z=x[:1]), "z: shape"),
        (ValueError, dict(h_in=h[:1]), "h_in: shape"), (ValueError, dict(n_new=n[:1]), "n_new: shape"), (ValueError, dict(y=x[:1]), "y: shape"),
        (ValueError, dict(saved=torch.zeros(8)), "saved: .* bytes"), (TypeError, dict(out_dtype=torch.int8), "output"),
        (ValueError, {}, "on a GPU"),
    ]:
        with pytest.raises(exc, match=match):
            linrec.scan_fwd(**{**ok, **kw})
    saved = torch.zeros(2, 16, 8)
    for exc, kw, match in [
        (ValueError, dict(saved=saved[:1]), "saved: .* bytes"), (TypeError, dict(saved=None), "saved"), (ValueError, dict(dy=x[:1]), "dy: shape"),
        (ValueError, dict(dz=x), "there is no z"), (ValueError, dict(dB=x), "dB: must be"), (ValueError, dict(dA=A[:2]), "dA: shape"),
        (TypeError, dict(dx=x, ddt=x.bfloat16()), "share one dtype"), (ValueError, dict(dh_out=h[:1]), "dh_out: shape"),
        (ValueError, dict(workspace=torch.zeros(2)), "workspace: .* bytes"), (ValueError, {}, "on a GPU"),
    ]:
        with pytest.raises(exc, match=match):
            linrec.scan_bwd(**{**ok, **dict(saved=saved, dy=x), **kw})
    for exc, kw, match in [
        (ValueError, dict(S=h[:1]), "1 states for 2"), (ValueError, dict(S=h[:, :, :4]), "S: shape"), (ValueError, dict(S=A), "S: must be"),
        (TypeError, dict(slots=n.long()), "slots"), (ValueError, {}, "on a GPU"),
    ]:
        with pytest.raises(exc, match=match):
            linrec.scan_step(**{**ok, **dict(S=h), **kw})


def test_sizes_past_32_bits_are_refused():
    big = torch.zeros(1, 1, 8).expand(1, 1 << 32, 8)
    with pytest.raises(ValueError, match="32 bits"):
        linrec.conv_fwd(big, torch.zeros(8, 4))
    with pytest.raises(ValueError, match="32 bits"):
        linrec.scan_fwd(big, big, torch.zeros(8, 8), torch.zeros(1, 1, 1, 8).expand(1, 1, 1 << 32, 8), torch.zeros(1, 1, 1, 8))


def test_packed_descriptions_are_the_structures():
    """What the binding packs has the layout of the structures."""
    v = list(range(1, 9))
    assert linrec._CONV(*v[:7]) == bytes(linrec.ConvDesc(*v[:7])) and linrec._SCAN(*v) == bytes(linrec.ScanDesc(*v))
    t = [linrec.Tensor(4 * i + 1, 4 * i + 2, 4 * i + 3, 4 * i + 4) for i in range(5)]
    assert linrec._SCAN_INPUTS(*range(1, 24)) == bytes(linrec.ScanInputs(*t, 21, 22, 23))
    assert linrec._SCAN_GRADS(*range(1, 25)) == bytes(linrec.ScanGradsDesc(*t, 21, 22, 23, 24))
