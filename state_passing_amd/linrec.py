"""ctypes binding of liblinrec.so (include/linrec.h).

Argument marshalling only: every step of the layer runs in the HIP kernels
of the library.  PyTorch provides device memory and the current stream.
Importing this module never loads the library; the first call does, and
raises if it has not been built -- there is no fallback path.

Layer (per batch b, head h): S_0 = S_in, S_t = a_t S_{t-1} + k_t^T v_t,
o_t = q_t S_t, S_out = S_T; the backward returns dq, dk, dv and dS_in for the
loss <dO, o> + <dS_out, S_out>.  Sub-sequences chain through S_out -> S_in
forward and dS_in -> dS_out backward (StateFlow, Abstract; Sequence
Accumulation and Beyond, "Approach").
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import NamedTuple, Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblinrec.so")

CHUNK = 64
BF16, F32 = 0, 1
DECAY_NONE, DECAY_HEAD, DECAY_TOKEN = 0, 1, 2

STATUS = {
    0: "LINREC_OK", 1: "LINREC_E_NULL", 2: "LINREC_E_SHAPE", 3: "LINREC_E_DTYPE",
    4: "LINREC_E_LAYOUT", 5: "LINREC_E_ALIGN", 6: "LINREC_E_WORKSPACE",
    7: "LINREC_E_DEVICE", 8: "LINREC_E_LAUNCH", 9: "LINREC_E_SCRATCH",
}

# Fixed device scratch of linrec_bwd_noalloc (LINREC_NOALLOC_SCRATCH_BYTES).
NOALLOC_SCRATCH_BYTES = 32 << 20
# Largest T of a call (LINREC_MAX_T).
MAX_T = 2147479552

# Every function include/linrec.h declares.
EXPORTS = (
    "linrec_ctx_create", "linrec_ctx_destroy", "linrec_states_bytes", "linrec_seq_states_bytes",
    "linrec_bwd_workspace_bytes", "linrec_fwd", "linrec_bwd", "linrec_fwd_seq",
    "linrec_bwd_seq_workspace_bytes", "linrec_bwd_seq", "linrec_status_str",
    "linrec_last_hip_error", "linrec_version", "linrec_ctx_set_timing",
    "linrec_ctx_kernel_times", "linrec_bwd_recompute_workspace_bytes", "linrec_bwd_recompute",
    "linrec_bwd_da_workspace_bytes", "linrec_bwd_da", "linrec_bwd_noalloc",
    "linrec_delta_workspace_bytes", "linrec_delta_fwd", "linrec_delta_saved_bytes",
    "linrec_delta_bwd_workspace_bytes", "linrec_delta_bwd", "linrec_delta_seq_saved_bytes",
    "linrec_delta_fwd_seq_workspace_bytes", "linrec_delta_bwd_seq_workspace_bytes",
    "linrec_delta_fwd_seq", "linrec_delta_bwd_seq",
    "linrec_diag_states_bytes", "linrec_diag_workspace_bytes", "linrec_diag_fwd", "linrec_diag_bwd",
    "linrec_step", "linrec_kv_append_workspace_bytes", "linrec_kv_append",
    "linrec_kv_attn_workspace_bytes", "linrec_kv_attn",
    "linrec_conv_fwd", "linrec_conv_bwd_workspace_bytes", "linrec_conv_bwd", "linrec_conv_step",
    "linrec_scan_saved_bytes", "linrec_scan_fwd_workspace_bytes", "linrec_scan_bwd_workspace_bytes",
    "linrec_scan_fwd", "linrec_scan_bwd", "linrec_scan_step",
)

KERNEL_KINDS = {0: "fwd_sum", 1: "fwd_fold", 2: "fwd_seg", 3: "bwd_sum", 4: "bwd_fold",
                5: "bwd_seg", 6: "da_finish", 7: "delta_fwd", 8: "delta_bwd", 9: "diag_fwd",
                10: "diag_bwd", 11: "step", 12: "kv_append", 13: "kv_attn", 14: "conv_fwd",
                15: "conv_bwd", 16: "conv_step", 17: "scan_fwd", 18: "scan_bwd", 19: "scan_step"}

# Forms of the elementwise recurrence (linrec_diag_form).
DIAG_FORMS = {"plain": 0, "mix": 1}
# Activations of the causal convolution (linrec_act).
ACTS = {None: 0, "silu": 1}


class LinrecError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} "
                         f"({_lib().linrec_status_str(status).decode()}; "
                         f"hip error {_lib().linrec_last_hip_error()})")


class Tensor(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("sb", ctypes.c_int64),
                ("sh", ctypes.c_int64), ("st", ctypes.c_int64)]


class Desc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("T", ctypes.c_int32),
                ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("chunk", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("decay", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32)]


class DiagDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("C", ctypes.c_int32),
                ("form", ctypes.c_int32), ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


class ConvDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("C", ctypes.c_int32), ("K", ctypes.c_int32),
                ("act", ctypes.c_int32), ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


class ScanDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("C", ctypes.c_int32), ("N", ctypes.c_int32),
                ("G", ctypes.c_int32), ("softplus", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32)]


class ScanInputs(ctypes.Structure):
    _fields_ = [("x", Tensor), ("dt", Tensor), ("b", Tensor), ("c", Tensor), ("z", Tensor),
                ("A", ctypes.c_void_p), ("D", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p)]


class ScanGradsDesc(ctypes.Structure):
    _fields_ = [("dx", Tensor), ("ddt", Tensor), ("db", Tensor), ("dc", Tensor), ("dz", Tensor),
                ("dA", ctypes.c_void_p), ("dD", ctypes.c_void_p), ("ddt_bias", ctypes.c_void_p),
                ("dh_in", ctypes.c_void_p)]


class KvCacheDesc(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("pages", ctypes.c_int32), ("page", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("H", ctypes.c_int32), ("D", ctypes.c_int32)]


_LIB = None


def _lib():
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it first "
                           "(python -m state_passing_amd.build)")
    lib = ctypes.CDLL(LIB_PATH)
    P, T, D = ctypes.c_void_p, Tensor, ctypes.POINTER(Desc)
    I32, DD, KC = ctypes.c_int32, ctypes.POINTER(DiagDesc), ctypes.POINTER(KvCacheDesc)
    CD = SD = SI = P   # packed, or structures by reference
    sig = {
        "linrec_ctx_create": ([ctypes.POINTER(P), ctypes.c_int], ctypes.c_int),
        "linrec_ctx_destroy": ([P], ctypes.c_int),
        "linrec_states_bytes": ([D], ctypes.c_size_t),
        "linrec_bwd_workspace_bytes": ([D], ctypes.c_size_t),
        "linrec_bwd_seq_workspace_bytes": ([D, I32, P], ctypes.c_size_t),
        "linrec_seq_states_bytes": ([D, I32, P], ctypes.c_size_t),
        "linrec_fwd": ([P, D, T, T, T, T, P, T, P, P, P], ctypes.c_int),
        "linrec_bwd": ([P, D, T, T, T, T, P, T, P, T, T, T, P, P, P], ctypes.c_int),
        "linrec_bwd_recompute_workspace_bytes": ([D], ctypes.c_size_t),
        "linrec_bwd_recompute": ([P, D, T, T, T, T, P, T, P, T, T, T, P, P, P], ctypes.c_int),
        "linrec_bwd_da_workspace_bytes": ([D], ctypes.c_size_t),
        "linrec_bwd_noalloc": ([P, D, T, T, T, T, P, T, P, T, T, T, P, P], ctypes.c_int),
        "linrec_delta_workspace_bytes": ([D], ctypes.c_size_t),
        "linrec_delta_fwd": ([P, D, T, T, T, T, T, P, T, P, P, P, P], ctypes.c_int),
        "linrec_delta_saved_bytes": ([D], ctypes.c_size_t),
        "linrec_delta_bwd_workspace_bytes": ([D], ctypes.c_size_t),
        "linrec_delta_bwd": ([P, D, T, T, T, T, T, P, T, P, T, T, T, T, P, P, P], ctypes.c_int),
        "linrec_delta_seq_saved_bytes": ([D, I32, P], ctypes.c_size_t),
        "linrec_delta_fwd_seq_workspace_bytes": ([D, I32, P], ctypes.c_size_t),
        "linrec_delta_bwd_seq_workspace_bytes": ([D, I32, P], ctypes.c_size_t),
        "linrec_delta_fwd_seq": ([P, D, I32, P, T, T, T, T, T, P, T, P, P, P, P], ctypes.c_int),
        "linrec_delta_bwd_seq": ([P, D, I32, P, T, T, T, T, T, P, T, P, T, T, T, T, P, P, P],
                                 ctypes.c_int),
        "linrec_bwd_da": ([P, D, T, T, T, T, P, T, P, T, T, T, P, T, P, P, P, P], ctypes.c_int),
        "linrec_fwd_seq": ([P, D, I32, P, T, T, T, T, P, T, P, P, P], ctypes.c_int),
        "linrec_bwd_seq": ([P, D, I32, P, T, T, T, T, P, T, P, T, T, T, P, P, P], ctypes.c_int),
        "linrec_diag_states_bytes": ([DD], ctypes.c_size_t),
        "linrec_diag_workspace_bytes": ([DD], ctypes.c_size_t),
        "linrec_diag_fwd": ([P, DD, T, T, P, T, P, P, P, P], ctypes.c_int),
        "linrec_diag_bwd": ([P, DD, T, T, P, T, P, T, T, P, P, P], ctypes.c_int),
        "linrec_step": ([P, D, T, T, T, T, T, P, P, I32, T, P], ctypes.c_int),
        "linrec_kv_append_workspace_bytes": ([KC, I32, I32], ctypes.c_size_t),
        "linrec_kv_append": ([P, KC, I32, I32, T, T, P, P, P, I32, I32, I32, T, T, P, P], ctypes.c_int),
        "linrec_kv_attn_workspace_bytes": ([KC, I32, I32, I32], ctypes.c_size_t),
        "linrec_kv_attn": ([P, KC, I32, I32, I32, T, P, P, ctypes.c_float, I32, T, P, P, P],
                           ctypes.c_int),
        "linrec_conv_fwd": ([P, CD, T, P, P, P, P, T, P, P], ctypes.c_int),
        "linrec_conv_bwd_workspace_bytes": ([CD], ctypes.c_size_t),
        "linrec_conv_bwd": ([P, CD, T, P, P, P, P, T, P, T, P, P, P, P, P], ctypes.c_int),
        "linrec_conv_step": ([P, CD, T, P, P, P, P, I32, T, P], ctypes.c_int),
        "linrec_scan_saved_bytes": ([SD], ctypes.c_size_t),
        "linrec_scan_fwd_workspace_bytes": ([SD], ctypes.c_size_t),
        "linrec_scan_bwd_workspace_bytes": ([SD], ctypes.c_size_t),
        "linrec_scan_fwd": ([P, SD, SI, P, P, T, P, P, P, P], ctypes.c_int),
        "linrec_scan_bwd": ([P, SD, SI, P, P, T, P, P, P, P], ctypes.c_int),
        "linrec_scan_step": ([P, SD, SI, P, P, I32, T, P], ctypes.c_int),
        "linrec_status_str": ([ctypes.c_int], ctypes.c_char_p),
        "linrec_last_hip_error": ([], ctypes.c_int),
        "linrec_version": ([], ctypes.c_int),
        "linrec_ctx_set_timing": ([P, ctypes.c_int], ctypes.c_int),
        "linrec_ctx_kernel_times": ([P, ctypes.c_int, ctypes.POINTER(ctypes.c_int64),
                                     ctypes.POINTER(ctypes.c_double)], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _LIB = lib
    return lib


def exported_symbols():
    """Names from EXPORTS that the loaded library resolves."""
    lib = _lib()
    return [n for n in EXPORTS if hasattr(lib, n)]


# ----------------------------------------------------------------- context

_CTX = {}


def context(device: Optional[int] = None) -> int:
    """The (cached) linrec_ctx of a device, as an opaque pointer value."""
    if device is None:
        device = torch.cuda.current_device()
    if device not in _CTX:
        p = ctypes.c_void_p()
        rc = _lib().linrec_ctx_create(ctypes.byref(p), int(device))
        if rc != 0:
            raise LinrecError(rc, "linrec_ctx_create")
        _CTX[device] = p.value
    return _CTX[device]


def set_kernel_timing(enable: bool, device: Optional[int] = None) -> None:
    """Turn the context's per-kernel event timing on or off (resets totals)."""
    _check(_lib().linrec_ctx_set_timing(context(device), 1 if enable else 0),
           "linrec_ctx_set_timing")


def kernel_times(device: Optional[int] = None) -> dict:
    """{kernel name: (launches, total ms)} since timing was enabled."""
    out = {}
    for kind, name in KERNEL_KINDS.items():
        n, ms = ctypes.c_int64(), ctypes.c_double()
        _check(_lib().linrec_ctx_kernel_times(context(device), kind, ctypes.byref(n),
                                              ctypes.byref(ms)), "linrec_ctx_kernel_times")
        out[name] = (int(n.value), float(ms.value))
    return out


# ----------------------------------------------------------------- marshalling

def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported activation dtype {t.dtype}")


def _act(t: Optional[torch.Tensor]) -> Tensor:
    if t is None:
        return Tensor(None, 0, 0, 0)
    if t.dim() != 4:
        raise ValueError(f"activation must be [B,H,T,d], got {tuple(t.shape)}")
    s = t.stride()
    return Tensor(t.data_ptr(), s[0], s[1], s[2])


def _decay(a: Optional[torch.Tensor]):
    if a is None:
        return DECAY_NONE, Tensor(None, 0, 0, 0)
    if a.dtype != torch.float32:
        raise TypeError("decay must be float32")
    if a.dim() == 1:
        return DECAY_HEAD, Tensor(a.data_ptr(), 0, a.stride(0), 0)
    if a.dim() == 3:
        s = a.stride()
        return DECAY_TOKEN, Tensor(a.data_ptr(), s[0], s[1], s[2])
    raise ValueError("decay must be [H] or [B,H,T]")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def desc(B, H, T, dk, dv, dtype_code, decay_kind, out_code=None) -> Desc:
    return Desc(B, H, T, dk, dv, CHUNK, dtype_code, decay_kind,
                dtype_code if out_code is None else out_code)


def _desc_of(q, v, decay_kind, out_dtype=None) -> Desc:
    B, H, T, dk = q.shape
    code = _dtype_code(q)
    out = code if out_dtype is None else _dtype_code(torch.empty(0, dtype=out_dtype))
    return desc(B, H, T, dk, v.shape[3], code, decay_kind, out)


def states_bytes(d: Desc) -> int:
    return int(_lib().linrec_states_bytes(ctypes.byref(d)))


def bwd_workspace_bytes(d: Desc) -> int:
    return int(_lib().linrec_bwd_workspace_bytes(ctypes.byref(d)))


def seq_states_bytes(d: Desc, lengths: Sequence[int]) -> int:
    arr = (ctypes.c_int32 * len(lengths))(*lengths)
    return int(_lib().linrec_seq_states_bytes(ctypes.byref(d), len(lengths), arr))


def bwd_seq_workspace_bytes(d: Desc, lengths: Sequence[int]) -> int:
    arr = (ctypes.c_int32 * len(lengths))(*lengths)
    return int(_lib().linrec_bwd_seq_workspace_bytes(ctypes.byref(d), len(lengths), arr))


def _state_out(like: torch.Tensor, B, H, dk, dv, given):
    if given is not None:
        return given
    return torch.empty(B, H, dk, dv, dtype=torch.float32, device=like.device)


def _check(rc, where):
    if rc != 0:
        raise LinrecError(rc, where)



# ----------------------------------------------------------------- validation
#
# The C ABI checks what it can see (shapes in the descriptor, alignment,
# strides, NULL pointers).  It cannot see tensor shapes, dtypes, devices or
# buffer sizes, so a mismatch there would become an out-of-bounds access on
# the GPU.  These checks run before any library call; the device check comes
# last so that every structural mistake is reported as such.

def _fail(msg: str, exc=ValueError):
    raise exc(msg)


def _check_act(name, t, shape, dtype=None):
    # conditions first, messages only on failure (this runs on every call)
    if not isinstance(t, torch.Tensor):
        _fail(f"{name}: expected a tensor", TypeError)
    if t.dim() != 4:
        _fail(f"{name}: must be [B,H,T,d], got {tuple(t.shape)}")
    if t.shape != shape:
        _fail(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        _fail(f"{name}: dtype {t.dtype} != {dtype}", TypeError)
    if t.stride(-1) != 1:
        _fail(f"{name}: the feature dimension must be contiguous (stride 1)")


def _check_state(name, t, shape):
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        _fail(f"{name}: expected a tensor", TypeError)
    if t.dtype != torch.float32:
        _fail(f"{name}: must be float32, got {t.dtype}", TypeError)
    if t.shape != shape:
        _fail(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if not t.is_contiguous():
        _fail(f"{name}: must be contiguous")


def _check_decay(decay, B, H, T):
    if decay is None:
        return
    if not isinstance(decay, torch.Tensor):
        _fail("decay: expected a tensor", TypeError)
    if decay.dtype != torch.float32:
        _fail("decay must be float32", TypeError)
    if decay.shape != (H,) and decay.shape != (B, H, T):
        _fail(f"decay must be [H] or [B,H,T], got {tuple(decay.shape)} for B={B} H={H} T={T}")


def _check_buffer(name, t, nbytes):
    if not isinstance(t, torch.Tensor):
        _fail(f"{name}: expected a tensor", TypeError)
    if not t.is_contiguous():
        _fail(f"{name}: must be contiguous")
    have = t.numel() * t.element_size()
    if have < nbytes:
        _fail(f"{name}: {have} bytes, the call needs {nbytes}")


def _check_device(q, *others):
    if not q.is_cuda:
        _fail(f"tensors must be on a GPU, got {q.device}")
    dev = q.device
    for name, t in others:
        if t is not None and t.device != dev:
            _fail(f"{name}: on {t.device}, q on {dev}")


def _validate(q, k, v, decay, *, dO=None, outs=(), states_in=(), states_out=(), extra=()):
    """Check every tensor of a call against q's [B,H,T,d_k] and v's d_v.

    outs: (name, tensor or None, out dtype, d) activation outputs;
    states_in / states_out: (name, tensor or None) fp32 [B,H,d_k,d_v];
    extra: (name, tensor or None) other tensors that only need the device check.
    Returns the (name, tensor) pairs for _check_device, which the caller runs
    after its buffer-size checks, so that structural errors are reported first."""
    if not isinstance(q, torch.Tensor):
        _fail("q: expected a tensor", TypeError)
    if q.dim() != 4:
        _fail(f"q: must be [B,H,T,d_k], got {tuple(q.shape)}")
    B, H, T, DK = q.shape
    if q.dtype not in (torch.bfloat16, torch.float32):
        _fail(f"unsupported activation dtype {q.dtype}", TypeError)
    qs = q.shape
    _check_act("q", q, qs, q.dtype)
    _check_act("k", k, qs, q.dtype)
    if not isinstance(v, torch.Tensor) or v.dim() != 4:
        _fail("v: must be [B,H,T,d_v]")
    DV = v.shape[3]
    vs = torch.Size((B, H, T, DV))
    _check_act("v", v, vs, q.dtype)
    if dO is not None:
        _check_act("dO", dO, vs, q.dtype)
    _check_decay(decay, B, H, T)
    odts = set()
    for name, t, odt, d in outs:
        if t is not None:
            _check_act(name, t, torch.Size((B, H, T, d)))
            odts.add(t.dtype)
        else:
            odts.add(odt)
    if len(odts) > 1:
        _fail(f"outputs must share one dtype, got {sorted(map(str, odts))}", TypeError)
    ss = torch.Size((B, H, DK, DV))
    for name, t in states_in:
        _check_state(name, t, ss)
    for name, t in states_out:
        _check_state(name, t, ss)
    return (("k", k), ("v", v), ("dO", dO), ("decay", decay),
            *((n, t) for n, t, _, _ in outs), *states_in, *states_out, *extra)

# ----------------------------------------------------------------- calls

def _out_dtype(q, out_dtype, given):
    if given is not None:
        return given.dtype
    return q.dtype if out_dtype is None else out_dtype


def _piece_lengths(lengths, T):
    lengths = [int(x) for x in lengths]
    if not lengths:
        _fail("lengths: need at least one piece")
    if sum(lengths) != T:
        _fail(f"lengths sum to {sum(lengths)}, the sequence has {T} tokens")
    return lengths


def _outs(q, v, odt, **given):
    """(name, tensor or None, dtype, width) for the activation outputs."""
    DK, DV = q.shape[3], v.shape[3]
    width = {"o": DV, "dq": DK, "dk": DK, "dv": DV}
    return tuple((n, t, odt, width[n]) for n, t in given.items())


def _new_act(q, d, odt, t):
    B, H, T = q.shape[:3]
    return torch.empty(B, H, T, d, dtype=odt, device=q.device) if t is None else t


def fwd(q, k, v, decay=None, S_in=None, *, o=None, S_out=None, states=None, out_dtype=None):
    """Forward over one piece.  Returns (o, S_out, states)."""
    odt = _out_dtype(q, out_dtype, o)
    devs = _validate(q, k, v, decay, outs=_outs(q, v, odt, o=o), states_in=(("S_in", S_in),),
              states_out=(("S_out", S_out),), extra=(("states", states),))
    kind, dec = _decay(decay)
    d = _desc_of(q, v, kind, odt)
    B, H, T, dk = q.shape
    dv = v.shape[3]
    if states is not None:
        _check_buffer("states", states, states_bytes(d))
    _check_device(q, *devs)
    o = _new_act(q, dv, odt, o)
    S_out = _state_out(q, B, H, dk, dv, S_out)
    if states is None:
        states = torch.empty(max(states_bytes(d), 16), dtype=torch.uint8, device=q.device)
    rc = _lib().linrec_fwd(context(q.device.index), ctypes.byref(d), _act(q), _act(k), _act(v),
                           dec, _ptr(S_in), _act(o), _ptr(S_out), _ptr(states),
                           _stream(q.device))
    _check(rc, "linrec_fwd")
    return o, S_out, states


def bwd(q, k, v, decay, states, dO, dS_out=None, *, dq=None, dk=None, dv=None,
        dS_in=None, workspace=None, out_dtype=None):
    """Backward over one piece.  Returns (dq, dk, dv, dS_in)."""
    odt = _out_dtype(q, out_dtype, dq)
    devs = _validate(q, k, v, decay, dO=dO, outs=_outs(q, v, odt, dq=dq, dk=dk, dv=dv),
              states_in=(("dS_out", dS_out),), states_out=(("dS_in", dS_in),),
              extra=(("states", states), ("workspace", workspace)))
    kind, dec = _decay(decay)
    d = _desc_of(q, v, kind, odt)
    B, H, T, DK = q.shape
    DV = v.shape[3]
    _check_buffer("states", states, states_bytes(d))
    if workspace is not None:
        _check_buffer("workspace", workspace, bwd_workspace_bytes(d))
    _check_device(q, *devs)
    dq, dk, dv = _new_act(q, DK, odt, dq), _new_act(q, DK, odt, dk), _new_act(q, DV, odt, dv)
    dS_in = _state_out(q, B, H, DK, DV, dS_in)
    if workspace is None:
        workspace = torch.empty(max(bwd_workspace_bytes(d), 16), dtype=torch.uint8, device=q.device)
    rc = _lib().linrec_bwd(context(q.device.index), ctypes.byref(d), _act(q), _act(k), _act(v),
                           dec, _ptr(states), _act(dO), _ptr(dS_out), _act(dq), _act(dk),
                           _act(dv), _ptr(dS_in), _ptr(workspace), _stream(q.device))
    _check(rc, "linrec_bwd")
    return dq, dk, dv, dS_in


def bwd_noalloc(q, k, v, decay, states, dO, dS_out=None, *, dq=None, dk=None, dv=None,
                dS_in=None, out_dtype=None):
    """linrec_bwd_noalloc: the backward of one piece in the library's fixed
    device scratch (no workspace).  The library call allocates nothing; pass
    dq, dk, dv and dS_in to keep this wrapper from allocating them.  Returns
    (dq, dk, dv, dS_in)."""
    odt = _out_dtype(q, out_dtype, dq)
    devs = _validate(q, k, v, decay, dO=dO, outs=_outs(q, v, odt, dq=dq, dk=dk, dv=dv),
                     states_in=(("dS_out", dS_out),), states_out=(("dS_in", dS_in),),
                     extra=(("states", states),))
    kind, dec = _decay(decay)
    d = _desc_of(q, v, kind, odt)
    B, H, T, DK = q.shape
    DV = v.shape[3]
    _check_buffer("states", states, states_bytes(d))
    _check_device(q, *devs)
    dq, dk, dv = _new_act(q, DK, odt, dq), _new_act(q, DK, odt, dk), _new_act(q, DV, odt, dv)
    dS_in = _state_out(q, B, H, DK, DV, dS_in)
    rc = _lib().linrec_bwd_noalloc(context(q.device.index), ctypes.byref(d), _act(q), _act(k),
                                   _act(v), dec, _ptr(states), _act(dO), _ptr(dS_out), _act(dq),
                                   _act(dk), _act(dv), _ptr(dS_in), _stream(q.device))
    _check(rc, "linrec_bwd_noalloc")
    return dq, dk, dv, dS_in


def bwd_recompute_workspace_bytes(d: Desc) -> int:
    return int(_lib().linrec_bwd_recompute_workspace_bytes(ctypes.byref(d)))


def bwd_recompute(q, k, v, decay, S_in, dO, dS_out=None, *, dq=None, dk=None, dv=None,
                  dS_in=None, workspace=None, out_dtype=None):
    """Backward over one piece from its boundary state S_in alone (the
    per-segment states are rebuilt).  Returns (dq, dk, dv, dS_in)."""
    odt = _out_dtype(q, out_dtype, dq)
    devs = _validate(q, k, v, decay, dO=dO, outs=_outs(q, v, odt, dq=dq, dk=dk, dv=dv),
              states_in=(("S_in", S_in), ("dS_out", dS_out)), states_out=(("dS_in", dS_in),),
              extra=(("workspace", workspace),))
    kind, dec = _decay(decay)
    d = _desc_of(q, v, kind, odt)
    B, H, T, DK = q.shape
    DV = v.shape[3]
    if workspace is not None:
        _check_buffer("workspace", workspace, bwd_recompute_workspace_bytes(d))
    _check_device(q, *devs)
    dq, dk, dv = _new_act(q, DK, odt, dq), _new_act(q, DK, odt, dk), _new_act(q, DV, odt, dv)
    dS_in = _state_out(q, B, H, DK, DV, dS_in)
    if workspace is None:
        workspace = torch.empty(max(bwd_recompute_workspace_bytes(d), 16), dtype=torch.uint8,
                                device=q.device)
    rc = _lib().linrec_bwd_recompute(context(q.device.index), ctypes.byref(d), _act(q), _act(k),
                                     _act(v), dec, _ptr(S_in), _act(dO), _ptr(dS_out), _act(dq),
                                     _act(dk), _act(dv), _ptr(dS_in), _ptr(workspace),
                                     _stream(q.device))
    _check(rc, "linrec_bwd_recompute")
    return dq, dk, dv, dS_in


def bwd_da_workspace_bytes(d: Desc) -> int:
    return int(_lib().linrec_bwd_da_workspace_bytes(ctypes.byref(d)))


def bwd_da(q, k, v, decay, states, dO, dS_out=None, da_carry=None, *, dq=None, dk=None,
           dv=None, dS_in=None, da=None, da_carry_out=None, workspace=None, out_dtype=None):
    """Backward over one piece plus the decay gradient.

    da_carry: fp32 [B,H], the gradient carried from later pieces (<dS_out,
    S_out>; None = 0).  Returns (dq, dk, dv, dS_in, da, da_carry_out) with
    da fp32 [B,H,T] and da_carry_out the carry for the previous piece."""
    odt = _out_dtype(q, out_dtype, dq)
    devs = _validate(q, k, v, decay, dO=dO, outs=_outs(q, v, odt, dq=dq, dk=dk, dv=dv),
              states_in=(("dS_out", dS_out),), states_out=(("dS_in", dS_in),),
              extra=(("states", states), ("workspace", workspace), ("da", da),
                     ("da_carry", da_carry), ("da_carry_out", da_carry_out)))
    if decay is None:
        _fail("bwd_da: needs a decay tensor")
    B, H, T, DK = q.shape
    DV = v.shape[3]
    if da is not None and (da.dtype != torch.float32 or da.shape != (B, H, T)):
        _fail(f"da: must be float32 [B,H,T] = {(B, H, T)}, got {da.dtype} {tuple(da.shape)}")
    for name, t in (("da_carry", da_carry), ("da_carry_out", da_carry_out)):
        if t is not None and (t.dtype != torch.float32 or t.shape != (B, H) or
                              not t.is_contiguous()):
            _fail(f"{name}: must be contiguous float32 [B,H] = {(B, H)}")
    kind, dec = _decay(decay)
    d = _desc_of(q, v, kind, odt)
    _check_buffer("states", states, states_bytes(d))
    if workspace is not None:
        _check_buffer("workspace", workspace, bwd_da_workspace_bytes(d))
    _check_device(q, *devs)
    dq, dk, dv = _new_act(q, DK, odt, dq), _new_act(q, DK, odt, dk), _new_act(q, DV, odt, dv)
    dS_in = _state_out(q, B, H, DK, DV, dS_in)
    da = torch.empty(B, H, T, dtype=torch.float32, device=q.device) if da is None else da
    if da_carry_out is None:
        da_carry_out = torch.empty(B, H, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(max(bwd_da_workspace_bytes(d), 16), dtype=torch.uint8,
                                device=q.device)
    rc = _lib().linrec_bwd_da(context(q.device.index), ctypes.byref(d), _act(q), _act(k), _act(v),
                              dec, _ptr(states), _act(dO), _ptr(dS_out), _act(dq), _act(dk),
                              _act(dv), _ptr(dS_in), Tensor(da.data_ptr(), da.stride(0),
                                                            da.stride(1), da.stride(2)),
                              _ptr(da_carry), _ptr(da_carry_out), _ptr(workspace),
                              _stream(q.device))
    _check(rc, "linrec_bwd_da")
    return dq, dk, dv, dS_in, da, da_carry_out


def fwd_seq(q, k, v, decay, lengths: Sequence[int], S_in=None, *, o=None, S_out=None,
            states=None, out_dtype=None):
    """Sequence accumulation forward over consecutive pieces (native driver).

    Returns (o, S_out, states) with states covering the whole sequence."""
    odt = _out_dtype(q, out_dtype, o)
    devs = _validate(q, k, v, decay, outs=_outs(q, v, odt, o=o), states_in=(("S_in", S_in),),
              states_out=(("S_out", S_out),), extra=(("states", states),))
    lengths = _piece_lengths(lengths, q.shape[2])
    kind, dec = _decay(decay)
    d = _desc_of(q, v, kind, odt)
    B, H, T, dk = q.shape
    dv = v.shape[3]
    if states is not None:
        _check_buffer("states", states, seq_states_bytes(d, lengths))
    _check_device(q, *devs)
    o = _new_act(q, dv, odt, o)
    S_out = _state_out(q, B, H, dk, dv, S_out)
    if states is None:
        states = torch.empty(max(seq_states_bytes(d, lengths), 16), dtype=torch.uint8,
                             device=q.device)
    arr = (ctypes.c_int32 * len(lengths))(*lengths)
    rc = _lib().linrec_fwd_seq(context(q.device.index), ctypes.byref(d), len(lengths), arr,
                               _act(q), _act(k), _act(v), dec, _ptr(S_in), _act(o),
                               _ptr(S_out), _ptr(states), _stream(q.device))
    _check(rc, "linrec_fwd_seq")
    return o, S_out, states


def bwd_seq(q, k, v, decay, lengths: Sequence[int], states, dO, dS_out=None, *, dq=None,
            dk=None, dv=None, dS_in=None, workspace=None, out_dtype=None):
    """Sequence accumulation backward (pieces in reverse, dS carried back)."""
    odt = _out_dtype(q, out_dtype, dq)
    devs = _validate(q, k, v, decay, dO=dO, outs=_outs(q, v, odt, dq=dq, dk=dk, dv=dv),
              states_in=(("dS_out", dS_out),), states_out=(("dS_in", dS_in),),
              extra=(("states", states), ("workspace", workspace)))
    lengths = _piece_lengths(lengths, q.shape[2])
    kind, dec = _decay(decay)
    d = _desc_of(q, v, kind, odt)
    B, H, T, DK = q.shape
    DV = v.shape[3]
    _check_buffer("states", states, seq_states_bytes(d, lengths))
    if workspace is not None:
        _check_buffer("workspace", workspace, bwd_seq_workspace_bytes(d, lengths))
    _check_device(q, *devs)
    dq, dk, dv = _new_act(q, DK, odt, dq), _new_act(q, DK, odt, dk), _new_act(q, DV, odt, dv)
    dS_in = _state_out(q, B, H, DK, DV, dS_in)
    if workspace is None:
        workspace = torch.empty(max(bwd_seq_workspace_bytes(d, lengths), 16), dtype=torch.uint8,
                                device=q.device)
    arr = (ctypes.c_int32 * len(lengths))(*lengths)
    rc = _lib().linrec_bwd_seq(context(q.device.index), ctypes.byref(d), len(lengths), arr,
                               _act(q), _act(k), _act(v), dec, _ptr(states), _act(dO),
                               _ptr(dS_out), _act(dq), _act(dk), _act(dv), _ptr(dS_in),
                               _ptr(workspace), _stream(q.device))
    _check(rc, "linrec_bwd_seq")
    return dq, dk, dv, dS_in


# ----------------------------------------------------------------- delta rule

def delta_workspace_bytes(d: Desc) -> int:
    return int(_lib().linrec_delta_workspace_bytes(ctypes.byref(d)))


def delta_saved_bytes(d: Desc) -> int:
    return int(_lib().linrec_delta_saved_bytes(ctypes.byref(d)))


def delta_bwd_workspace_bytes(d: Desc) -> int:
    return int(_lib().linrec_delta_bwd_workspace_bytes(ctypes.byref(d)))


def _beta_arg(name, x, B, H, T):
    if not isinstance(x, torch.Tensor) or x.dtype != torch.float32 or x.shape != (B, H, T):
        _fail(f"{name}: must be float32 [B,H,T] = {(B, H, T)}")
    st = x.stride()
    return Tensor(x.data_ptr(), st[0], st[1], st[2])


def delta_fwd(q, k, v, beta, decay=None, S_in=None, *, o=None, S_out=None, saved=None,
              save=False, workspace=None, out_dtype=None):
    """Gated delta rule, forward over one piece (linrec_delta_fwd):
    S_t = a_t (I - beta_t k_t^T k_t) S_{t-1} + beta_t k_t^T v_t, o_t = q_t S_t.
    beta: fp32 [B,H,T].  With save=True (or a `saved` buffer) the states and
    values the backward needs are kept.  Returns (o, S_out, saved or None)."""
    odt = _out_dtype(q, out_dtype, o)
    devs = _validate(q, k, v, decay, outs=_outs(q, v, odt, o=o), states_in=(("S_in", S_in),),
                     states_out=(("S_out", S_out),),
                     extra=(("beta", beta), ("workspace", workspace), ("saved", saved)))
    B, H, T, DK = q.shape
    DV = v.shape[3]
    barg = _beta_arg("beta", beta, B, H, T)
    kind, dec = _decay(decay)
    d = _desc_of(q, v, kind, odt)
    if workspace is not None:
        _check_buffer("workspace", workspace, delta_workspace_bytes(d))
    if saved is not None:
        _check_buffer("saved", saved, delta_saved_bytes(d))
    _check_device(q, *devs)
    o = _new_act(q, DV, odt, o)
    S_out = _state_out(q, B, H, DK, DV, S_out)
    if workspace is None:
        workspace = torch.empty(max(delta_workspace_bytes(d), 16), dtype=torch.uint8, device=q.device)
    if saved is None and save:
        saved = torch.empty(max(delta_saved_bytes(d), 16), dtype=torch.uint8, device=q.device)
    rc = _lib().linrec_delta_fwd(context(q.device.index), ctypes.byref(d), _act(q), _act(k), _act(v),
                                 barg, dec, _ptr(S_in), _act(o), _ptr(S_out), _ptr(saved),
                                 _ptr(workspace), _stream(q.device))
    _check(rc, "linrec_delta_fwd")
    return o, S_out, saved


def delta_bwd(q, k, v, beta, decay, saved, dO, dS_out=None, *, dq=None, dk=None, dv=None,
              dbeta=None, dS_in=None, workspace=None, out_dtype=None):
    """Gated delta rule, backward over one piece (linrec_delta_bwd) from the
    forward's `saved` buffer.  Returns (dq, dk, dv, dbeta, dS_in)."""
    odt = _out_dtype(q, out_dtype, dq)
    devs = _validate(q, k, v, decay, dO=dO, outs=_outs(q, v, odt, dq=dq, dk=dk, dv=dv),
                     states_in=(("dS_out", dS_out),), states_out=(("dS_in", dS_in),),
                     extra=(("beta", beta), ("saved", saved), ("workspace", workspace),
                            ("dbeta", dbeta)))
    B, H, T, DK = q.shape
    DV = v.shape[3]
    barg = _beta_arg("beta", beta, B, H, T)
    kind, dec = _decay(decay)
    d = _desc_of(q, v, kind, odt)
    _check_buffer("saved", saved, delta_saved_bytes(d))
    if workspace is not None:
        _check_buffer("workspace", workspace, delta_bwd_workspace_bytes(d))
    if dbeta is not None:
        _beta_arg("dbeta", dbeta, B, H, T)
    _check_device(q, *devs)
    dq, dk, dv = _new_act(q, DK, odt, dq), _new_act(q, DK, odt, dk), _new_act(q, DV, odt, dv)
    dS_in = _state_out(q, B, H, DK, DV, dS_in)
    if dbeta is None:
        dbeta = torch.empty(B, H, T, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(max(delta_bwd_workspace_bytes(d), 16), dtype=torch.uint8,
                                device=q.device)
    rc = _lib().linrec_delta_bwd(context(q.device.index), ctypes.byref(d), _act(q), _act(k), _act(v),
                                 barg, dec, _ptr(saved), _act(dO), _ptr(dS_out), _act(dq), _act(dk),
                                 _act(dv), _beta_arg("dbeta", dbeta, B, H, T), _ptr(dS_in),
                                 _ptr(workspace), _stream(q.device))
    _check(rc, "linrec_delta_bwd")
    return dq, dk, dv, dbeta, dS_in


def _lengths_arg(lengths):
    return (ctypes.c_int32 * len(lengths))(*lengths)


def delta_seq_saved_bytes(d: Desc, lengths: Sequence[int]) -> int:
    return int(_lib().linrec_delta_seq_saved_bytes(ctypes.byref(d), len(lengths),
                                                   _lengths_arg(lengths)))


def delta_fwd_seq_workspace_bytes(d: Desc, lengths: Sequence[int]) -> int:
    return int(_lib().linrec_delta_fwd_seq_workspace_bytes(ctypes.byref(d), len(lengths),
                                                           _lengths_arg(lengths)))


def delta_bwd_seq_workspace_bytes(d: Desc, lengths: Sequence[int]) -> int:
    return int(_lib().linrec_delta_bwd_seq_workspace_bytes(ctypes.byref(d), len(lengths),
                                                           _lengths_arg(lengths)))


def delta_fwd_seq(q, k, v, beta, decay, lengths: Sequence[int], S_in=None, *, o=None,
                  S_out=None, saved=None, save=False, workspace=None, out_dtype=None):
    """Gated delta rule forward over consecutive pieces, S carried (native
    driver, linrec_delta_fwd_seq).  Returns (o, S_out, saved or None)."""
    odt = _out_dtype(q, out_dtype, o)
    devs = _validate(q, k, v, decay, outs=_outs(q, v, odt, o=o), states_in=(("S_in", S_in),),
                     states_out=(("S_out", S_out),),
                     extra=(("beta", beta), ("workspace", workspace), ("saved", saved)))
    lengths = _piece_lengths(lengths, q.shape[2])
    B, H, T, DK = q.shape
    DV = v.shape[3]
    barg = _beta_arg("beta", beta, B, H, T)
    kind, dec = _decay(decay)
    d = _desc_of(q, v, kind, odt)
    if workspace is not None:
        _check_buffer("workspace", workspace, delta_fwd_seq_workspace_bytes(d, lengths))
    if saved is not None:
        _check_buffer("saved", saved, delta_seq_saved_bytes(d, lengths))
    _check_device(q, *devs)
    o = _new_act(q, DV, odt, o)
    S_out = _state_out(q, B, H, DK, DV, S_out)
    if workspace is None:
        workspace = torch.empty(max(delta_fwd_seq_workspace_bytes(d, lengths), 16),
                                dtype=torch.uint8, device=q.device)
    if saved is None and save:
        saved = torch.empty(max(delta_seq_saved_bytes(d, lengths), 16), dtype=torch.uint8,
                            device=q.device)
    rc = _lib().linrec_delta_fwd_seq(context(q.device.index), ctypes.byref(d), len(lengths),
                                     _lengths_arg(lengths), _act(q), _act(k), _act(v), barg, dec,
                                     _ptr(S_in), _act(o), _ptr(S_out), _ptr(saved),
                                     _ptr(workspace), _stream(q.device))
    _check(rc, "linrec_delta_fwd_seq")
    return o, S_out, saved


def delta_bwd_seq(q, k, v, beta, decay, lengths: Sequence[int], saved, dO, dS_out=None, *,
                  dq=None, dk=None, dv=None, dbeta=None, dS_in=None, workspace=None,
                  out_dtype=None):
    """Gated delta rule backward over consecutive pieces in reverse, dS
    carried (linrec_delta_bwd_seq), from delta_fwd_seq's `saved`.  Returns
    (dq, dk, dv, dbeta, dS_in)."""
    odt = _out_dtype(q, out_dtype, dq)
    devs = _validate(q, k, v, decay, dO=dO, outs=_outs(q, v, odt, dq=dq, dk=dk, dv=dv),
                     states_in=(("dS_out", dS_out),), states_out=(("dS_in", dS_in),),
                     extra=(("beta", beta), ("saved", saved), ("workspace", workspace),
                            ("dbeta", dbeta)))
    lengths = _piece_lengths(lengths, q.shape[2])
    B, H, T, DK = q.shape
    DV = v.shape[3]
    barg = _beta_arg("beta", beta, B, H, T)
    kind, dec = _decay(decay)
    d = _desc_of(q, v, kind, odt)
    _check_buffer("saved", saved, delta_seq_saved_bytes(d, lengths))
    if workspace is not None:
        _check_buffer("workspace", workspace, delta_bwd_seq_workspace_bytes(d, lengths))
    if dbeta is not None:
        _beta_arg("dbeta", dbeta, B, H, T)
    _check_device(q, *devs)
    dq, dk, dv = _new_act(q, DK, odt, dq), _new_act(q, DK, odt, dk), _new_act(q, DV, odt, dv)
    dS_in = _state_out(q, B, H, DK, DV, dS_in)
    if dbeta is None:
        dbeta = torch.empty(B, H, T, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(max(delta_bwd_seq_workspace_bytes(d, lengths), 16),
                                dtype=torch.uint8, device=q.device)
    rc = _lib().linrec_delta_bwd_seq(context(q.device.index), ctypes.byref(d), len(lengths),
                                     _lengths_arg(lengths), _act(q), _act(k), _act(v), barg, dec,
                                     _ptr(saved), _act(dO), _ptr(dS_out), _act(dq), _act(dk),
                                     _act(dv), _beta_arg("dbeta", dbeta, B, H, T), _ptr(dS_in),
                                     _ptr(workspace), _stream(q.device))
    _check(rc, "linrec_delta_bwd_seq")
    return dq, dk, dv, dbeta, dS_in


# ----------------------------------------------------------------- elementwise recurrence
#
# The calls from here on are also made for single tokens, where the time of
# their checks counts: each argument is checked and described in one go, and
# the functions that word the errors run only when a check fails.

_CODE = {torch.bfloat16: BF16, torch.float32: F32}
_NONE = Tensor(None, 0, 0, 0)


def _too_large(*sizes):
    """Sizes become 32-bit integers, which ctypes would cut to their low bits.
    (Callers ask `(a | b | ...) >> 31`: a call of this would cost every token 0.3 us.)"""
    _fail(f"sizes {sizes}: not all fit 32 bits")


def _arg4(name, t, shape, dtype) -> Tensor:
    """The description of a [B,H,T,d] activation of this shape and type."""
    if not isinstance(t, torch.Tensor):
        _fail(f"{name}: expected a tensor", TypeError)
    if t.shape == shape and t.dtype is dtype:
        b, h, r, one = t.stride()
        if one == 1:
            return Tensor(t.data_ptr(), b, h, r)
    _check_act(name, t, torch.Size(shape), dtype)
    return _act(t)


def _arg3(name, t, shape, dtype) -> Tensor:
    """The description of a [B,T,C] activation of this shape and type."""
    if not isinstance(t, torch.Tensor):
        _fail(f"{name}: expected a tensor", TypeError)
    if t.shape != shape:
        _fail(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if t.dtype is not dtype:
        _fail(f"{name}: dtype {t.dtype} != {dtype}", TypeError)
    s = t.stride()
    if s[2] != 1 and shape[2] > 1:
        _fail(f"{name}: the channel dimension must be contiguous (stride 1)")
    return Tensor(t.data_ptr(), s[0], 0, s[1])


def _state_ptr(name, t, shape):
    """The address of a contiguous fp32 tensor of this shape, or None."""
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.float32 and t.shape == shape and t.is_contiguous()):
        _check_state(name, t, torch.Size(shape))
    return t.data_ptr()


def _int_ptr(name, t, shape, dtype=torch.int32):
    """The address of a contiguous tensor of this shape and type, or None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        _fail(f"{name}: expected a tensor", TypeError)
    if t.dtype is not dtype:
        _fail(f"{name}: must be {dtype}, got {t.dtype}", TypeError)
    if t.shape != shape:
        _fail(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if not t.is_contiguous():
        _fail(f"{name}: must be contiguous")
    return t.data_ptr()


def _same_device(first, *others) -> int:
    """The GPU that holds `first` and every tensor of the (name, tensor) pairs."""
    index = first.get_device()
    if index >= 0:
        for _, t in others:
            if t is not None and t.get_device() != index:
                break
        else:
            return index
    _check_device(first, *others)
    return index


def _raw_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# the same handle without building a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


def _bytes(n, like):
    return torch.empty(n, dtype=torch.uint8, device=like.device)


def diag_desc(B, T, C, form, dtype_code, out_code=None) -> DiagDesc:
    return DiagDesc(B, T, C, form, dtype_code, dtype_code if out_code is None else out_code)


def diag_states_bytes(d: DiagDesc) -> int:
    return int(_lib().linrec_diag_states_bytes(ctypes.byref(d)))


def diag_workspace_bytes(d: DiagDesc) -> int:
    return int(_lib().linrec_diag_workspace_bytes(ctypes.byref(d)))


def _new_rows(like, dtype):
    """A new [B,T,C] output whose rows are 16-byte aligned (a view of padded rows where C is odd)."""
    n = 8 if dtype is torch.bfloat16 else 4
    C = like.shape[2]
    if C % n == 0:
        return torch.empty_like(like, dtype=dtype)
    return torch.empty(*like.shape[:2], -(-C // n) * n, dtype=dtype, device=like.device)[..., :C]


def _diag_setup(g, form, out_dtype, *outs):
    """The shape, description and output type of a diag call."""
    if not isinstance(g, torch.Tensor) or g.dim() != 3:
        _fail("g: must be a [B,T,C] tensor")
    code = _CODE.get(g.dtype)
    if code is None:
        _fail(f"unsupported activation dtype {g.dtype}", TypeError)
    kind = DIAG_FORMS.get(form)
    if kind is None:
        _fail(f"form: {form!r} is none of {sorted(DIAG_FORMS)}")
    odt = g.dtype if out_dtype is None else out_dtype
    given = [t.dtype for t in outs if isinstance(t, torch.Tensor)]
    if given:
        odt = given[0]
        if len(set(given)) > 1:
            _fail(f"outputs must share one dtype, got {sorted(map(str, set(given)))}", TypeError)
    out = _CODE.get(odt)
    if out is None:
        _fail(f"unsupported output dtype {odt}", TypeError)
    B, T, C = shape = g.shape
    if (B | T | C) >> 31:
        _too_large(B, T, C)
    return shape, DiagDesc(B, T, C, kind, code, out), odt


def diag_fwd(g, x, h_in=None, *, form="plain", h=None, h_out=None, states=None, workspace=None,
             out_dtype=None):
    """Elementwise gated recurrence over one piece (linrec_diag_fwd):
    h_t = exp(g_t) h_{t-1} + b_t per channel, b = x ("plain") or
    (1 - exp(g)) x ("mix"); g, x: [B,T,C], h_in, h_out: fp32 [B,C].
    Returns (h, h_out, states); states is what diag_bwd needs."""
    shape, d, odt = _diag_setup(g, form, out_dtype, h)
    carry = (shape[0], shape[2])
    ga, xa = _arg3("g", g, shape, g.dtype), _arg3("x", x, shape, g.dtype)
    ha = None if h is None else _arg3("h", h, shape, odt)
    in_ptr, out_ptr = _state_ptr("h_in", h_in, carry), _state_ptr("h_out", h_out, carry)
    need, work = diag_states_bytes(d), diag_workspace_bytes(d) if shape[1] > 256 else 0
    if states is not None:
        _check_buffer("states", states, need)
    if workspace is not None:
        _check_buffer("workspace", workspace, work)
    dev = _same_device(g, ("x", x), ("h_in", h_in), ("h", h), ("h_out", h_out), ("states", states),
                       ("workspace", workspace))
    if h is None:
        h = _new_rows(g, odt)
        ha = _arg3("h", h, shape, odt)
    if h_out is None:
        h_out = torch.empty(carry, dtype=torch.float32, device=g.device)
        out_ptr = h_out.data_ptr()
    if states is None:
        states = _bytes(max(need, 16), g)
    if workspace is None and work:
        workspace = _bytes(work, g)
    rc = _lib().linrec_diag_fwd(context(dev), ctypes.byref(d), ga, xa, in_ptr, ha, out_ptr,
                                states.data_ptr(), _ptr(workspace), _raw_stream(dev))
    _check(rc, "linrec_diag_fwd")
    return h, h_out, states


def diag_bwd(g, x, states, dh, dh_out=None, *, form="plain", dg=None, dx=None, dh_in=None,
             workspace=None, out_dtype=None):
    """Backward of diag_fwd over one piece (linrec_diag_bwd), from its states,
    for the loss <dh, h> + <dh_out, h_out>.  Returns (dg, dx, dh_in)."""
    shape, d, odt = _diag_setup(g, form, out_dtype, dg, dx)
    carry = (shape[0], shape[2])
    ga, xa = _arg3("g", g, shape, g.dtype), _arg3("x", x, shape, g.dtype)
    da = _arg3("dh", dh, shape, g.dtype)
    dga = None if dg is None else _arg3("dg", dg, shape, odt)
    dxa = None if dx is None else _arg3("dx", dx, shape, odt)
    out_ptr, in_ptr = _state_ptr("dh_out", dh_out, carry), _state_ptr("dh_in", dh_in, carry)
    work = diag_workspace_bytes(d) if shape[1] > 256 else 0
    _check_buffer("states", states, diag_states_bytes(d))
    if workspace is not None:
        _check_buffer("workspace", workspace, work)
    dev = _same_device(g, ("x", x), ("states", states), ("dh", dh), ("dh_out", dh_out), ("dg", dg),
                       ("dx", dx), ("dh_in", dh_in), ("workspace", workspace))
    if dg is None:
        dg = _new_rows(g, odt)
        dga = _arg3("dg", dg, shape, odt)
    if dx is None:
        dx = _new_rows(g, odt)
        dxa = _arg3("dx", dx, shape, odt)
    if dh_in is None:
        dh_in = torch.empty(carry, dtype=torch.float32, device=g.device)
        in_ptr = dh_in.data_ptr()
    if workspace is None and work:
        workspace = _bytes(work, g)
    rc = _lib().linrec_diag_bwd(context(dev), ctypes.byref(d), ga, xa, states.data_ptr(), da, out_ptr,
                                dga, dxa, in_ptr, _ptr(workspace), _raw_stream(dev))
    _check(rc, "linrec_diag_bwd")
    return dg, dx, dh_in


# ----------------------------------------------------------------- state-space layer
#
# Descriptions go to the library as packed bytes (the layouts of ConvDesc,
# ScanDesc, ScanInputs and ScanGradsDesc): building the structures takes a token call several
# times as long.

_CONV = struct.Struct("7i").pack
_SCAN = struct.Struct("8i").pack
_SCAN_INPUTS = struct.Struct("23q").pack
_SCAN_GRADS = struct.Struct("24q").pack
# The tensors of a call beside x, in the order their devices are compared.
_CONV_FWD_NAMES = ("w", "bias", "state_in", "n_new", "y", "state_out")
_CONV_BWD_NAMES = ("w", "bias", "state_in", "n_new", "dy", "dstate_out", "dx", "dw", "dbias", "dstate_in", "workspace")
_CONV_STEP_NAMES = ("w", "bias", "S", "slots", "y")
_SCAN_NAMES = ("dt", "A", "B", "C", "D", "z", "dt_bias")
_SCAN_FWD_NAMES = (*_SCAN_NAMES, "h_in", "n_new", "y", "h_out", "saved", "workspace")
_SCAN_BWD_NAMES = (*_SCAN_NAMES, "saved", "n_new", "dy", "dh_out", "dx", "ddt", "dB", "dC", "dz", "workspace", "dA", "dD",
                   "ddt_bias", "dh_in")
_SCAN_STEP_NAMES = (*_SCAN_NAMES, "S", "slots", "y")

def _out_code(dt, out_dtype, *outs):
    """The output type of a call and its code: of the given outputs, else out_dtype, else dt."""
    odt = dt if out_dtype is None else out_dtype
    for t in outs:
        if t is not None:
            given = {t.dtype for t in outs if isinstance(t, torch.Tensor)}
            if len(given) > 1:
                _fail(f"outputs must share one dtype, got {sorted(map(str, given))}", TypeError)
            odt = given.pop() if given else odt
            break
    code = _CODE.get(odt)
    if code is None:
        _fail(f"unsupported output dtype {odt}", TypeError)
    return odt, code


def _new_rows_of(like, dtype, ragged):
    """A new [B,T,C] output as _new_rows; zeros where rows may not be written."""
    t = torch.empty_like(like) if dtype is like.dtype and not like.shape[2] & 7 else _new_rows(like, dtype)
    return t.zero_() if ragged else t


def _device_of(first, names, *tensors) -> int:
    """_same_device with the names apart, paired with the tensors only if it fails."""
    index = first.get_device()
    if index >= 0:
        for t in tensors:
            if t is not None and t.get_device() != index:
                break
        else:
            return index
    return _same_device(first, *zip(names, tensors))


def _view3(name, t, shape, dtype):
    """(address, sb, sh, st) of a [B,T,C] activation of this shape and type."""
    if isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype:
        sb, st, one = t.stride()
        if one == 1:
            return t.data_ptr(), sb, 0, st
    a = _arg3(name, t, shape, dtype)   # words the error
    return a.ptr, a.sb, 0, a.st


def _view4(name, t, shape, dtype):
    """(address, sb, sh, st) of a [B,G,T,N] activation of this shape and type."""
    if isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype:
        sb, sh, st, one = t.stride()
        if one == 1:
            return t.data_ptr(), sb, sh, st
    a = _arg4(name, t, shape, dtype)
    return a.ptr, a.sb, a.sh, a.st


def _conv_setup(x, w, bias, act, out_dtype, *outs):
    """The shape, description and output type of a convolution, with its parameters' addresses."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        _fail("x: must be a [B,T,C] tensor")
    code = _CODE.get(x.dtype)
    if code is None:
        _fail(f"unsupported activation dtype {x.dtype}", TypeError)
    kind = ACTS.get(act)
    if kind is None:
        _fail(f"act: {act!r} is none of {list(ACTS)}")
    odt, out = _out_code(x.dtype, out_dtype, *outs)
    B, T, C = shape = x.shape
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        _fail("w: must be a float32 [C,K] tensor")
    K = w.shape[1]
    if (B | T | C | K) >> 31:
        _too_large(B, T, C, K)
    return (shape, K, _CONV(B, T, C, K, kind, code, out), odt, _state_ptr("w", w, (C, K)),
            _state_ptr("bias", bias, (C,)))


def conv_fwd(x, w, bias=None, state_in=None, *, act="silu", n_new=None, y=None, state_out=None,
             out_dtype=None):
    """Short causal convolution over one piece (linrec_conv_fwd):
    y_t = act(bias + sum_k w[:,k] x_{t-K+1+k}) per channel; x: [B,T,C]; w: fp32
    [C,K], K = 2, 3 or 4; bias: fp32 [C] or None; act: "silu" or None; state_in,
    state_out: fp32 [B,K-1,C], the K-1 inputs before the piece and its last ones.
    n_new: int32 [B] on the device, the first n_new[b] tokens are there (rows
    behind them are left as they were, zeros in a new y).  Returns (y, state_out)."""
    shape, K, d, odt, w_ptr, b_ptr = _conv_setup(x, w, bias, act, out_dtype, y)
    carry = (shape[0], K - 1, shape[2])
    xa = _arg3("x", x, shape, x.dtype)
    ya = None if y is None else _arg3("y", y, shape, odt)
    in_ptr, out_ptr = _state_ptr("state_in", state_in, carry), _state_ptr("state_out", state_out, carry)
    n_ptr = _int_ptr("n_new", n_new, (shape[0],))
    dev = _device_of(x, _CONV_FWD_NAMES, w, bias, state_in, n_new, y, state_out)
    if y is None:
        y = _new_rows_of(x, odt, n_new is not None)
        ya = _arg3("y", y, shape, odt)
    if state_out is None:
        state_out = torch.empty(carry, dtype=torch.float32, device=x.device)
        out_ptr = state_out.data_ptr()
    rc = _lib().linrec_conv_fwd(context(dev), d, xa, w_ptr, b_ptr, in_ptr, n_ptr, ya, out_ptr,
                                _raw_stream(dev))
    _check(rc, "linrec_conv_fwd")
    return y, state_out


def conv_bwd(x, w, bias, state_in, dy, dstate_out=None, *, act="silu", n_new=None, dx=None, dw=None,
             dbias=None, dstate_in=None, workspace=None, out_dtype=None):
    """Backward of conv_fwd over one piece (linrec_conv_bwd), for the loss
    <dy, y> + <dstate_out, state_out>.  Returns (dx, dw, dbias, dstate_in);
    dbias is None without a bias.  dw and dbias are this piece's alone."""
    shape, K, d, odt, w_ptr, b_ptr = _conv_setup(x, w, bias, act, out_dtype, dx)
    C = shape[2]
    carry = (shape[0], K - 1, C)
    xa, da = _arg3("x", x, shape, x.dtype), _arg3("dy", dy, shape, x.dtype)
    dxa = None if dx is None else _arg3("dx", dx, shape, odt)
    in_ptr, dout_ptr = _state_ptr("state_in", state_in, carry), _state_ptr("dstate_out", dstate_out, carry)
    din_ptr = _state_ptr("dstate_in", dstate_in, carry)
    dw_ptr, db_ptr = _state_ptr("dw", dw, (C, K)), _state_ptr("dbias", dbias, (C,))
    n_ptr = _int_ptr("n_new", n_new, (shape[0],))
    need = int(_lib().linrec_conv_bwd_workspace_bytes(d))
    if workspace is not None:
        _check_buffer("workspace", workspace, need)
    dev = _device_of(x, _CONV_BWD_NAMES, w, bias, state_in, n_new, dy, dstate_out, dx, dw, dbias, dstate_in, workspace)
    if dx is None:
        dx = _new_rows_of(x, odt, n_new is not None)
        dxa = _arg3("dx", dx, shape, odt)
    if dw is None:
        dw = torch.empty_like(w)
        dw_ptr = dw.data_ptr()
    if dbias is None and bias is not None:
        dbias = torch.empty_like(bias)
        db_ptr = dbias.data_ptr()
    if dstate_in is None:
        dstate_in = torch.empty(carry, dtype=torch.float32, device=x.device)
        din_ptr = dstate_in.data_ptr()
    if workspace is None and need:
        workspace = _bytes(need, x)
    rc = _lib().linrec_conv_bwd(context(dev), d, xa, w_ptr, b_ptr, in_ptr, n_ptr, da, dout_ptr, dxa,
                                dw_ptr, db_ptr, din_ptr, _ptr(workspace), _raw_stream(dev))
    _check(rc, "linrec_conv_bwd")
    return dx, dw, dbias, dstate_in


def _pool(name, S, rest, B, slots):
    """The address and size of a pool of fp32 states [n, *rest]."""
    if not isinstance(S, torch.Tensor) or S.dim() != 1 + len(rest):
        _fail(f"{name}: must be a float32 [n,{','.join(map(str, rest))}] tensor")
    n = S.shape[0]
    if n >> 31:
        _too_large(n)
    ptr = _state_ptr(name, S, (n, *rest))
    if slots is None and n < B:
        _fail(f"{name}: {n} states for {B} entries")
    return ptr, n


def conv_step(x, w, bias, S, *, act="silu", slots=None, y=None, out_dtype=None):
    """One or a few tokens of conv_fwd (linrec_conv_step), the states updated in
    place.  x: [B,T,C]; S: fp32 [n,K-1,C], entry b at slots[b] (int32 [B] on the
    device) or at b.  An entry whose slot is outside the pool, or taken by an
    earlier entry, is skipped (y = 0).  Returns y."""
    shape, K, d, odt, w_ptr, b_ptr = _conv_setup(x, w, bias, act, out_dtype, y)
    B, T, C = shape
    xa = _arg3("x", x, shape, x.dtype)
    ya = None if y is None else _arg3("y", y, shape, odt)
    S_ptr, n = _pool("S", S, (K - 1, C), B, slots)
    slot_ptr = _int_ptr("slots", slots, (B,))
    dev = _device_of(x, _CONV_STEP_NAMES, w, bias, S, slots, y)
    if y is None:
        y = _new_rows(x, odt)
        sb, st, _ = y.stride()
        ya = Tensor(y.data_ptr(), sb, 0, st)
    rc = _lib().linrec_conv_step(context(dev), d, xa, w_ptr, b_ptr, S_ptr, slot_ptr, n, ya,
                                 _raw_stream(dev))
    _check(rc, "linrec_conv_step")
    return y


def _scan_setup(x, dt, A, B, C, D, z, dt_bias, softplus, out_dtype, *outs):
    """The shapes, description, inputs and output type of a scan."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        _fail("x: must be a [B,T,C] tensor")
    t = x.dtype
    code = _CODE.get(t)
    if code is None:
        _fail(f"unsupported activation dtype {t}", TypeError)
    odt, out = _out_code(t, out_dtype, *outs)
    n, T, ch = shape = x.shape
    if not isinstance(B, torch.Tensor) or B.dim() != 4:
        _fail("B: must be a [B,G,T,N] tensor")
    G, N = B.shape[1], B.shape[3]
    proj = (n, G, T, N)
    if (n | T | ch | N | G) >> 31:
        _too_large(n, T, ch, N, G)
    if A is None:
        _fail("A: expected a tensor", TypeError)
    inputs = _SCAN_INPUTS(*_view3("x", x, shape, t), *_view3("dt", dt, shape, t), *_view4("B", B, proj, t),
                          *_view4("C", C, proj, t), *((0, 0, 0, 0) if z is None else _view3("z", z, shape, t)),
                          _state_ptr("A", A, (ch, N)), _state_ptr("D", D, (ch,)) or 0,
                          _state_ptr("dt_bias", dt_bias, (ch,)) or 0)
    return shape, proj, _SCAN(n, T, ch, N, G, 1 if softplus else 0, code, out), inputs, odt


def scan_saved_bytes(d) -> int:
    """Bytes of `saved` for a ScanDesc (as a structure by reference, or packed)."""
    return int(_lib().linrec_scan_saved_bytes(d))


def scan_fwd(x, dt, A, B, C, h_in=None, *, D=None, z=None, dt_bias=None, softplus=True, n_new=None,
             y=None, h_out=None, saved=None, save=False, workspace=None, out_dtype=None):
    """Selective state-space scan over one piece (linrec_scan_fwd): with
    d = softplus(dt + dt_bias) (softplus=False: dt + dt_bias),
    h_t = exp(d_t A) h_{t-1} + d_t x_t B_t,  y_t = (C_t . h_t + D x_t) silu(z_t).
    x, dt, z: [B,T,C]; A: fp32 [C,N]; B, C: [B,G,T,N], G groups of channels; D,
    dt_bias: fp32 [C] or None; z: None means no gate; h_in, h_out: fp32 [B,C,N].
    n_new: int32 [B] on the device, the first n_new[b] tokens are there (rows
    behind them are left as they were, zeros in a new y).  With save=True (or a
    `saved` buffer) the states that scan_bwd needs are kept.
    Returns (y, h_out, saved or None)."""
    shape, proj, d, inputs, odt = _scan_setup(x, dt, A, B, C, D, z, dt_bias, softplus, out_dtype, y)
    carry = (shape[0], shape[2], proj[3])
    ya = None if y is None else _arg3("y", y, shape, odt)
    in_ptr, out_ptr = _state_ptr("h_in", h_in, carry), _state_ptr("h_out", h_out, carry)
    n_ptr = _int_ptr("n_new", n_new, (shape[0],))
    need = int(_lib().linrec_scan_fwd_workspace_bytes(d))
    if workspace is not None:
        _check_buffer("workspace", workspace, need)
    if saved is not None:
        _check_buffer("saved", saved, scan_saved_bytes(d))
    dev = _device_of(x, _SCAN_FWD_NAMES, dt, A, B, C, D, z, dt_bias, h_in, n_new, y, h_out, saved, workspace)
    if y is None:
        y = _new_rows_of(x, odt, n_new is not None)
        ya = _arg3("y", y, shape, odt)
    if h_out is None:
        h_out = torch.empty(carry, dtype=torch.float32, device=x.device)
        out_ptr = h_out.data_ptr()
    if saved is None and save:
        saved = _bytes(max(scan_saved_bytes(d), 16), x)
    if workspace is None and need:
        workspace = _bytes(need, x)
    rc = _lib().linrec_scan_fwd(context(dev), d, inputs, in_ptr, n_ptr, ya, out_ptr,
                                _ptr(saved), _ptr(workspace), _raw_stream(dev))
    _check(rc, "linrec_scan_fwd")
    return y, h_out, saved


class ScanGrads(NamedTuple):
    """What scan_bwd returns; dD, dz and ddt_bias are None without D, z and dt_bias."""
    dx: torch.Tensor
    ddt: torch.Tensor
    dA: torch.Tensor
    dB: torch.Tensor
    dC: torch.Tensor
    dh_in: torch.Tensor
    dD: Optional[torch.Tensor]
    dz: Optional[torch.Tensor]
    ddt_bias: Optional[torch.Tensor]


def scan_bwd(x, dt, A, B, C, saved, dy, dh_out=None, *, D=None, z=None, dt_bias=None, softplus=True,
             n_new=None, dx=None, ddt=None, dA=None, dB=None, dC=None, dh_in=None, dD=None, dz=None,
             ddt_bias=None, workspace=None, out_dtype=None) -> ScanGrads:
    """Backward of scan_fwd over one piece (linrec_scan_bwd), from its `saved`
    buffer, for the loss <dy, y> + <dh_out, h_out>.  Gradients of parameters and
    of B and C are sums over what shares them, of this piece alone."""
    shape, proj, d, inputs, odt = _scan_setup(x, dt, A, B, C, D, z, dt_bias, softplus, out_dtype, dx, ddt, dB, dC, dz)
    ch = shape[2]
    carry = (shape[0], ch, proj[3])
    da = _arg3("dy", dy, shape, x.dtype)
    dout_ptr = _state_ptr("dh_out", dh_out, carry)
    if dz is not None and z is None:
        _fail("dz: there is no z")
    n_ptr = _int_ptr("n_new", n_new, (shape[0],))
    need = int(_lib().linrec_scan_bwd_workspace_bytes(d))
    _check_buffer("saved", saved, scan_saved_bytes(d))
    if workspace is not None:
        _check_buffer("workspace", workspace, need)
    # outputs that are not given are made before the devices are compared: all are described in one go
    ragged, f32 = n_new is not None, torch.float32
    if dx is None:
        dx = _new_rows_of(x, odt, ragged)
    if ddt is None:
        ddt = _new_rows_of(x, odt, ragged)
    if z is not None and dz is None:
        dz = _new_rows_of(x, odt, ragged)
    new = torch.zeros if ragged else torch.empty
    if dB is None:
        dB = new(proj, dtype=odt, device=x.device)
    if dC is None:
        dC = new(proj, dtype=odt, device=x.device)
    if dA is None:
        dA = torch.empty_like(A)
    if dD is None and D is not None:
        dD = torch.empty_like(D)
    if ddt_bias is None and dt_bias is not None:
        ddt_bias = torch.empty_like(dt_bias)
    if dh_in is None:
        dh_in = torch.empty(carry, dtype=f32, device=x.device)
    out = _SCAN_GRADS(*_view3("dx", dx, shape, odt), *_view3("ddt", ddt, shape, odt), *_view4("dB", dB, proj, odt),
                      *_view4("dC", dC, proj, odt), *((0, 0, 0, 0) if dz is None else _view3("dz", dz, shape, odt)),
                      _state_ptr("dA", dA, (ch, proj[3])), _state_ptr("dD", dD, (ch,)) or 0,
                      _state_ptr("ddt_bias", ddt_bias, (ch,)) or 0, _state_ptr("dh_in", dh_in, carry))
    dev = _device_of(x, _SCAN_BWD_NAMES, dt, A, B, C, D, z, dt_bias, saved, n_new, dy, dh_out, dx, ddt, dB, dC, dz, workspace,
                     dA, dD, ddt_bias, dh_in)
    if workspace is None and need:
        workspace = _bytes(need, x)
    rc = _lib().linrec_scan_bwd(context(dev), d, inputs, _ptr(saved), n_ptr, da, dout_ptr, out, _ptr(workspace), _raw_stream(dev))
    _check(rc, "linrec_scan_bwd")
    return ScanGrads(dx, ddt, dA, dB, dC, dh_in, dD, dz, ddt_bias)


def scan_step(x, dt, A, B, C, S, *, D=None, z=None, dt_bias=None, softplus=True, slots=None, y=None,
              out_dtype=None):
    """One or a few tokens of scan_fwd (linrec_scan_step), the states updated in
    place.  S: fp32 [n,C,N], entry b at slots[b] (int32 [B] on the device) or at
    b; slots as conv_step.  Returns y."""
    shape, proj, d, inputs, odt = _scan_setup(x, dt, A, B, C, D, z, dt_bias, softplus, out_dtype, y)
    ya = None if y is None else _arg3("y", y, shape, odt)
    S_ptr, n = _pool("S", S, (shape[2], proj[3]), shape[0], slots)
    slot_ptr = _int_ptr("slots", slots, (shape[0],))
    dev = _device_of(x, _SCAN_STEP_NAMES, dt, A, B, C, D, z, dt_bias, S, slots, y)
    if y is None:
        y = _new_rows(x, odt)
        sb, st, _ = y.stride()
        ya = Tensor(y.data_ptr(), sb, 0, st)
    rc = _lib().linrec_scan_step(context(dev), d, inputs, S_ptr, slot_ptr, n, ya,
                                 _raw_stream(dev))
    _check(rc, "linrec_scan_step")
    return y


# ----------------------------------------------------------------- generation

def step(q, k, v, decay, S, *, beta=None, slots=None, o=None, out_dtype=None):
    """One or a few tokens of the layer (beta None) or of the gated delta rule
    (linrec_step), S updated in place.  q, k: [B,H,T,d_k]; v: [B,H,T,d_v];
    decay as fwd; beta: fp32 [B,H,T]; S: fp32 [n,H,d_k,d_v], entry b at slots[b]
    (int32 [B] on the device) or at b.  An entry whose slot is outside the
    pool, or taken by an earlier entry, is skipped (o = 0).  Returns o."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        _fail("q: must be a [B,H,T,d_k] tensor")
    if not isinstance(v, torch.Tensor) or v.dim() != 4:
        _fail("v: must be a [B,H,T,d_v] tensor")
    dt = q.dtype
    code = _CODE.get(dt)
    if code is None:
        _fail(f"unsupported activation dtype {dt}", TypeError)
    B, H, T, DK = q.shape
    DV = v.shape[3]
    qa, ka = _arg4("q", q, q.shape, dt), _arg4("k", k, q.shape, dt)
    va = _arg4("v", v, (B, H, T, DV), dt)
    odt = o.dtype if isinstance(o, torch.Tensor) else dt if out_dtype is None else out_dtype
    out = _CODE.get(odt)
    if out is None:
        _fail(f"unsupported output dtype {odt}", TypeError)
    oa = None if o is None else _arg4("o", o, (B, H, T, DV), odt)
    kind, dec = DECAY_NONE, _NONE
    if decay is not None:
        _check_decay(decay, B, H, T)
        kind, dec = _decay(decay)
    if not isinstance(S, torch.Tensor) or S.dim() != 4:
        _fail("S: must be a float32 [n,H,d_k,d_v] tensor")
    n = S.shape[0]
    if (B | H | T | DK | DV | n) >> 31:
        _too_large(B, H, T, DK, DV, n)
    S_ptr = _state_ptr("S", S, (n, H, DK, DV))
    slot_ptr = _int_ptr("slots", slots, (B,))
    if slots is None and n < B:
        _fail(f"S: {n} states for {B} entries")
    barg = _NONE if beta is None else _beta_arg("beta", beta, B, H, T)
    dev = _same_device(q, ("k", k), ("v", v), ("decay", decay), ("S", S), ("beta", beta),
                       ("slots", slots), ("o", o))
    if o is None:
        o = torch.empty_like(v, dtype=odt)
        oa = _arg4("o", o, o.shape, odt)
    rc = _lib().linrec_step(context(dev), ctypes.byref(Desc(B, H, T, DK, DV, CHUNK, code, kind, out)), qa, ka,
                            va, barg, dec, S_ptr, slot_ptr, n, oa, _raw_stream(dev))
    _check(rc, "linrec_step")
    return o


class KvCache(NamedTuple):
    """A paged 8-bit key/value cache (layouts in include/linrec.h): codes as
    float8_e4m3fn tensors k [pages,H,page,D] and v [pages,H,D,page], scales
    fp32 [pages,H], table int32 [B,max_pages]."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    table: torch.Tensor


def kv_cache(pages, heads, page, width, table, device=None) -> KvCache:
    """An empty cache of `pages` pages for the block table `table`."""
    dev = table.device if device is None else device
    codes = lambda *shape: torch.zeros(*shape, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)  # noqa: E731
    scale = lambda: torch.zeros(pages, heads, dtype=torch.float32, device=dev)  # noqa: E731
    return KvCache(codes(pages, heads, page, width), codes(pages, heads, width, page), scale(), scale(),
                   table)


def _codes_ptr(name, t, shape):
    if not isinstance(t, torch.Tensor) or t.dim() != 4:
        _fail(f"{name}: must be a 4-dimensional tensor")
    if t.dtype is not torch.float8_e4m3fn:
        _fail(f"{name}: must be float8_e4m3fn, got {t.dtype}", TypeError)
    if shape is not None and t.shape != shape:
        _fail(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if not t.is_contiguous():
        _fail(f"{name}: must be contiguous")
    return t.data_ptr()


def _kv_desc(cache: KvCache, B: int) -> KvCacheDesc:
    """Checks of a cache's tensors; returns the C description."""
    k, v, ks, vs, table = cache
    k_ptr = _codes_ptr("cache.k", k, None)
    pages, H, page, D = k.shape
    v_ptr = _codes_ptr("cache.v", v, (pages, H, D, page))
    if ks is None or vs is None:
        _fail("cache: the scales are needed")
    ks_ptr = _state_ptr("cache.k_scale", ks, (pages, H))
    vs_ptr = _state_ptr("cache.v_scale", vs, (pages, H))
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        _fail("cache.table: must be an int32 [B,max_pages] tensor")
    if table.dtype is not torch.int32:
        _fail(f"cache.table: must be torch.int32, got {table.dtype}", TypeError)
    rows, width = table.shape
    if rows != B:
        _fail(f"cache.table: {rows} rows for {B} sequences")
    stride, one = table.stride()
    if width > 1 and one != 1:
        _fail("cache.table: rows must be contiguous")
    if (B | pages | H | page | D | width) >> 31:
        _too_large(B, pages, H, page, D, width)
    return KvCacheDesc(k_ptr, v_ptr, ks_ptr, vs_ptr, table.data_ptr(), stride, pages, page, width, H, D)


def kv_append(cache: KvCache, k, v, past, *, n_new=None, inv_freq=None, interleaved=False, q=None,
              q_out=None, workspace=None):
    """Append k, v [B,H,T,D] (bf16) behind past[b] (int32 [B]) tokens of every
    sequence's cache, the first n_new[b] of the T, with the rotation of
    inv_freq (fp64 [rot/2]) applied to the keys and to q [B,Hq,T,D]
    (linrec_kv_append).  Returns the rotated queries (None without q); rows
    that are not there (behind n_new, of a sequence with a negative past) are
    left as they were (zeros in a new q_out)."""
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        _fail("k: must be a [B,H,T,D] tensor")
    B, _, T, _ = k.shape
    c = _kv_desc(cache, B)
    shape, bf = (B, c.H, T, c.D), torch.bfloat16
    ka, va = _arg4("k", k, shape, bf), _arg4("v", v, shape, bf)
    if past is None:
        _fail("past: expected a tensor", TypeError)
    past_ptr, n_ptr = _int_ptr("past", past, (B,)), _int_ptr("n_new", n_new, (B,))
    rot, freq_ptr = 0, None
    if inv_freq is not None:
        if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
            _fail("inv_freq: must be a float64 vector")
        freq_ptr, rot = _int_ptr("inv_freq", inv_freq, inv_freq.shape, torch.float64), 2 * inv_freq.numel()
    Hq, qa, oa = 0, _NONE, _NONE
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != 4:
            _fail("q: must be a [B,Hq,T,D] tensor")
        Hq = q.shape[1]
        qa = _arg4("q", q, (B, Hq, T, c.D), bf)
        if q_out is not None:
            oa = _arg4("q_out", q_out, (B, Hq, T, c.D), bf)
    elif q_out is not None:
        _fail("q_out: there is no q")
    if (T | Hq | rot) >> 31:
        _too_large(T, Hq, rot)
    # a call of fewer than 1024 tokens, so of fewer pages, needs none
    need = _lib().linrec_kv_append_workspace_bytes(ctypes.byref(c), B, T) if B * T >= 1024 else 0
    if workspace is not None:
        _check_buffer("workspace", workspace, need)
    dev = _same_device(k, ("v", v), ("past", past), ("n_new", n_new), ("inv_freq", inv_freq), ("q", q),
                       ("q_out", q_out), ("workspace", workspace), *zip(KvCache._fields, cache))
    if q is not None and q_out is None:
        q_out = torch.zeros((B, Hq, T, c.D), dtype=bf, device=q.device)   # rows that are not there stay zeros
        oa = _arg4("q_out", q_out, q_out.shape, bf)
    if workspace is None and need:
        workspace = _bytes(need, k)
    rc = _lib().linrec_kv_append(context(dev), ctypes.byref(c), B, T, ka, va, past_ptr, n_ptr, freq_ptr, rot,
                                 1 if interleaved else 0, Hq, qa, oa, _ptr(workspace), _raw_stream(dev))
    _check(rc, "linrec_kv_append")
    return q_out


def kv_attn(cache: KvCache, q, past, *, n_new=None, scale=None, window=0, o=None, lse=None,
            workspace=None):
    """Attention of q [B,Hq,T,D] (bf16) over the cache, which already holds
    these T tokens behind past[b] earlier ones (linrec_kv_attn).  scale:
    1/sqrt(D) by default; window: the last `window` tokens only (<= 0 or >=
    MAX_T: all).  lse: fp32 [B,Hq,T] to be filled, or None.  Returns o; rows
    that are not there (behind n_new, of a sequence with a negative past) are
    left as they were (zeros in a new o)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        _fail("q: must be a [B,Hq,T,D] tensor")
    B, Hq, T, _ = q.shape
    c = _kv_desc(cache, B)
    shape, bf = (B, Hq, T, c.D), torch.bfloat16
    qa = _arg4("q", q, shape, bf)
    oa = None if o is None else _arg4("o", o, shape, bf)
    if past is None:
        _fail("past: expected a tensor", TypeError)
    past_ptr, n_ptr = _int_ptr("past", past, (B,)), _int_ptr("n_new", n_new, (B,))
    lse_ptr = _state_ptr("lse", lse, (B, Hq, T))
    if (T | Hq) >> 31:
        _too_large(T, Hq)
    if c.H < 1 or Hq % c.H:
        _fail(f"q: {Hq} heads are no multiple of the cache's {c.H}")
    window = int(window)
    if not 0 < window < MAX_T:
        window = 0   # no lower bound; the C argument has 32 bits
    need = _lib().linrec_kv_attn_workspace_bytes(ctypes.byref(c), B, T, Hq)
    if workspace is not None:
        _check_buffer("workspace", workspace, need)
    dev = _same_device(q, ("past", past), ("n_new", n_new), ("o", o), ("lse", lse), ("workspace", workspace),
                       *zip(KvCache._fields, cache))
    if o is None:
        o = torch.zeros(shape, dtype=bf, device=q.device)   # rows that are not there stay zeros
        oa = _arg4("o", o, shape, bf)
    if workspace is None and need:
        workspace = _bytes(need, q)
    rc = _lib().linrec_kv_attn(context(dev), ctypes.byref(c), B, T, Hq, qa, past_ptr, n_ptr,
                               c.D ** -0.5 if scale is None else float(scale), window, oa, lse_ptr,
                               _ptr(workspace), _raw_stream(dev))
    _check(rc, "linrec_kv_attn")
    return o


def piece_loop(q, k, v, decay, lengths: Sequence[int], S_in=None, dO=None, dS_out=None,
               out_dtype=None):
    """Sequence accumulation through the per-piece calls, one call per piece
    (S carried forward, dS carried back).  Returns (o, S_out, dq, dk, dv, dS_in)
    -- the gradients are None when dO is None."""
    B, H, T, DK = q.shape
    DV = v.shape[3]
    odt = q.dtype if out_dtype is None else out_dtype
    o = torch.empty(B, H, T, DV, dtype=odt, device=q.device)
    S = S_in
    bounds = [0]
    for L in lengths:
        bounds.append(bounds[-1] + L)

    def dsl(i):
        if decay is None or decay.dim() == 1:
            return decay
        return decay[:, :, bounds[i]:bounds[i + 1]]

    saved = []
    for i in range(len(lengths)):
        sl = slice(bounds[i], bounds[i + 1])
        _, S, st = fwd(q[:, :, sl], k[:, :, sl], v[:, :, sl], dsl(i), S, o=o[:, :, sl])
        saved.append(st)
    if dO is None:
        return o, S, None, None, None, None
    dq, dk, dv = (torch.empty(x.shape, dtype=odt, device=q.device) for x in (q, k, v))
    dS = dS_out
    for i in reversed(range(len(lengths))):
        sl = slice(bounds[i], bounds[i + 1])
        _, _, _, dS = bwd(q[:, :, sl], k[:, :, sl], v[:, :, sl], dsl(i), saved[i],
                          dO[:, :, sl], dS, dq=dq[:, :, sl], dk=dk[:, :, sl], dv=dv[:, :, sl])
    return o, S, dq, dk, dv, dS
