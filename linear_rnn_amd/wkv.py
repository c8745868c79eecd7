"""Thin ctypes binding of librwkv7_wkv.so (argument marshalling only).

Function names match the C ABI in include/rwkv7_wkv.h. Each takes torch tensors
(device memory owned by the caller) or None, passes their addresses, sizes and
dtype to the library, launches on the current torch stream unless a stream is
given, and raises RuntimeError with the library's message on a non-zero status.
The functions without the rwkv7_ prefix allocate their outputs as well, as tensors of the
stream they launch on (torch.Tensor.record_stream says so where another one uses them).
Before the call it checks every tensor against the sizes the call takes (shape,
one input dtype, contiguity, 16-byte alignment, one HIP device) and raises
ValueError on a mismatch: the C ABI receives bare pointers and cannot.
Every step of the computation runs in the HIP kernels; there is no fallback:
if the library is missing, loading it raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "librwkv7_wkv.so")

RWKV7_OK = 0
RWKV7_DTYPE_F32 = 0
RWKV7_DTYPE_BF16 = 1
RWKV7_STATE_F32 = 0
RWKV7_STATE_BF16 = 1
RWKV7_STATE_F16 = 2
RWKV7_ALGO_AUTO = 0
RWKV7_ALGO_SEQUENTIAL = 1
RWKV7_ALGO_CHUNKED = 2
RWKV7_ALGO_CHUNKED_SPLIT = 3
RWKV7_ERR_SCRATCH = -9
RWKV7_ERR_DECAY = -10
RWKV7_DECAY_HEAD = 0
RWKV7_DECAY_TOKEN = 1
RWKV7_NOALLOC_SCRATCH_BYTES = 64 << 20
_PER_THREAD = 2  # the handle hipStreamPerThread

EXPORTED = ("rwkv7_wkv_prefill", "rwkv7_wkv_step", "rwkv7_wkv_step_q", "rwkv7_wkv_prefill_ex",
            "rwkv7_tmix_prefill", "rwkv7_tmix_prefill_ex", "rwkv7_tmix_step", "rwkv7_wkv_backward",
            "rwkv7_wkv_backward_ex",
            "rwkv7_stack_forward", "rwkv7_wkv_prefill_algo", "rwkv7_wkv_prefill_noalloc",
            "rwkv7_linattn_prefill", "rwkv7_linattn_step", "rwkv7_linattn_backward",
            "rwkv7_layernorm_forward", "rwkv7_layernorm_backward",
            "rwkv7_wkv_strerror")

_lib = None
_lock = threading.Lock()


class Rwkv7Error(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__("rwkv7 status %d: %s" % (status, msg))
        self.status = status


def lib() -> ctypes.CDLL:
    """Load the HIP library (raises OSError if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise OSError("HIP library %s is missing: run `python -m linear_rnn_amd.build`" % LIB_PATH)
            L = ctypes.CDLL(LIB_PATH)
            vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
            sig = [vp] * 9 + [i64] * 4 + [ci]
            for name in ("rwkv7_wkv_prefill", "rwkv7_wkv_step", "rwkv7_wkv_prefill_noalloc"):
                f = getattr(L, name)
                f.restype = ci
                f.argtypes = sig + [vp]
            L.rwkv7_wkv_step_q.restype = ci
            L.rwkv7_wkv_step_q.argtypes = sig + [ci, vp]
            L.rwkv7_wkv_prefill_ex.restype = ci
            L.rwkv7_wkv_prefill_ex.argtypes = sig + [ci, vp]
            for name in ("rwkv7_tmix_prefill", "rwkv7_tmix_step"):
                f = getattr(L, name)
                f.restype = ci
                f.argtypes = [vp] * 11 + [i64] * 4 + [ci, vp]
            L.rwkv7_tmix_prefill_ex.restype = ci
            L.rwkv7_tmix_prefill_ex.argtypes = [vp] * 11 + [i64] * 4 + [ci, ci, vp]
            L.rwkv7_wkv_backward.restype = ci
            L.rwkv7_wkv_backward.argtypes = [vp] * 16 + [i64] * 4 + [ci, vp]
            L.rwkv7_wkv_backward_ex.restype = ci
            L.rwkv7_wkv_backward_ex.argtypes = [vp] * 16 + [i64] * 4 + [ci, ci, vp]
            L.rwkv7_stack_forward.restype = ci
            L.rwkv7_stack_forward.argtypes = [vp] * 5 + [i64] * 5 + [ci, vp]
            L.rwkv7_linattn_prefill.restype = ci
            L.rwkv7_linattn_prefill.argtypes = [vp] * 8 + [i64] * 4 + [ci, ci, vp]
            L.rwkv7_linattn_step.restype = ci
            L.rwkv7_linattn_step.argtypes = [vp] * 7 + [i64] * 4 + [ci, ci, vp]
            L.rwkv7_linattn_backward.restype = ci
            L.rwkv7_linattn_backward.argtypes = [vp] * 13 + [i64] * 4 + [ci, ci, vp]
            cf = ctypes.c_float
            L.rwkv7_layernorm_forward.restype = ci
            L.rwkv7_layernorm_forward.argtypes = [vp] * 6 + [i64] * 3 + [cf, ci, ci, vp]
            L.rwkv7_layernorm_backward.restype = ci
            L.rwkv7_layernorm_backward.argtypes = [vp] * 8 + [i64] * 3 + [ci, ci, vp]
            L.rwkv7_wkv_prefill_algo.restype = ci
            L.rwkv7_wkv_prefill_algo.argtypes = [i64] * 4 + [ci]
            L.rwkv7_wkv_strerror.restype = ctypes.c_char_p
            L.rwkv7_wkv_strerror.argtypes = [ci]
            _lib = L
    return _lib


def rwkv7_wkv_prefill_algo(B: int, T: int, H: int, N: int = 64, dtype: int = RWKV7_DTYPE_BF16) -> int:
    """The RWKV7_ALGO_* value that rwkv7_wkv_prefill runs for this shape and dtype (raises on invalid sizes)."""
    st = lib().rwkv7_wkv_prefill_algo(int(B), int(T), int(H), int(N), int(dtype))
    _check(min(st, 0))
    return st


def rwkv7_wkv_strerror(status: int) -> str:
    return lib().rwkv7_wkv_strerror(int(status)).decode()


def _ptr(t):
    return None if t is None else (t.data_ptr() or None)


# torch is imported at the first use (the library's own functions need none), and what every call asks of it is
# kept here: a single-token step takes a few microseconds, and so would a handful of imports and lookups.
class _Torch:
    module = None

    def __getattr__(self, name):
        import torch
        self.module = torch
        self.Tensor = torch.Tensor
        self.empty_like = torch.empty_like
        self.f32 = (torch.float32,)
        self.inputs = (torch.bfloat16, torch.float32)
        self.i32 = (torch.int32,)
        self.codes = {torch.bfloat16: RWKV7_DTYPE_BF16, torch.float32: RWKV7_DTYPE_F32}
        self.current_device = torch.cuda.current_device
        # the current stream's handle of a device, without the stream object around it
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda device: torch.cuda.current_stream(device).cuda_stream)
        return self.__dict__[name]


_T = _Torch()


def _dtype_code(t) -> int:
    return _T.codes.get(t.dtype, -1)


def _stream(stream):
    if stream is None:
        return _T.raw_stream(_T.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _on_stream_of(stream, like, make):
    """make(), which allocates, with `stream` current: torch's allocator gives out memory that the current stream has
    left, so memory for a kernel on another stream has to be of that stream, or work still under way uses it too."""
    if stream is None or like.device.type != "cuda":
        return make()
    import torch
    if isinstance(stream, int):
        if stream == _PER_THREAD:
            raise ValueError("hipStreamPerThread is another stream in every thread, which torch's allocator does not "
                             "know: allocate the outputs and call the rwkv7_ function")
        stream = torch.cuda.ExternalStream(stream, device=like.device)
    with torch.cuda.stream(stream):
        return make()


# ---- argument checks. The C ABI sees raw pointers and cannot check a buffer's size,
# layout or device, so every tensor is checked here against the sizes the call takes
# from r (or the state / residual stream) before the library is called. Shapes,
# dtypes, contiguity and alignment are checked first and the device last, so each
# mistake is named even for host tensors.

def _expect(t, name, shape, dtypes, like, optional=False):
    """Raise unless t is a contiguous, 16-byte aligned tensor of this shape and dtype on like's device."""
    if t is None:
        if optional:
            return
        raise ValueError("%s is required" % name)
    if isinstance(t, _T.Tensor) and t.shape == shape and t.dtype in dtypes and t.is_contiguous() and \
            not t.data_ptr() & 15 and t.device == like.device:
        return
    # something is wrong (or an empty tensor's address is odd, which does not matter): say what
    if not isinstance(t, _T.Tensor):
        raise TypeError("%s must be a torch.Tensor, not %s" % (name, type(t).__name__))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.dtype not in dtypes:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, " or ".join(str(d) for d in dtypes)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous (row-major), got strides %s" % (name, tuple(t.stride())))
    if t.numel() and t.data_ptr() % 16:
        raise ValueError("%s must be 16-byte aligned" % name)
    if t.device != like.device:
        raise ValueError("%s is on %s, the other tensors on %s" % (name, t.device, like.device))


def _at(t, name, shape, dtypes, like, optional=False):
    """The address of a tensor that is as _expect() wants it (None for an empty or a left out one)."""
    if t.__class__ is _T.Tensor and t.shape == shape and t.dtype in dtypes and t.is_contiguous() and \
            t.get_device() == like.get_device():
        p = t.data_ptr()
        if not p & 15:
            return p or None
    _expect(t, name, shape, dtypes, like, optional)
    return _ptr(t)


def _on_gpu(like, stream):
    """The tensors must be device memory of the device the kernels launch on."""
    if like.device.type != "cuda":
        raise ValueError("tensors must be on a HIP device (torch 'cuda'), got %s" % like.device)
    if stream is None and like.device.index != _T.current_device():
        raise ValueError("tensors are on %s but the current device is cuda:%d; pass a stream of that device or "
                         "select it" % (like.device, _T.current_device()))
    where = getattr(stream, "device", None)  # a bare handle does not say
    if where is not None and where != like.device:
        raise ValueError("the stream is on %s, the tensors on %s" % (where, like.device))


def _launch(name, args, like, stream):
    """Call the library with `like`'s device current (a stream given by the caller may be another device's)."""
    index = like.get_device()
    if index < 0 or stream is not None or index != _T.current_device():
        _on_gpu(like, stream)  # says what is wrong
    fn = getattr(lib(), name)
    if index == _T.current_device():
        _check(fn(*args, _T.raw_stream(index) if stream is None else _stream(stream)))
    else:
        with _T.module.cuda.device(index):
            _check(fn(*args, _stream(stream)))


def _input_dtypes():
    return _T.inputs


def _f32():
    return _T.f32


def _args(r, w, k, v, a, b, state_in, y, state_out, stream=None, state_dtypes=None):
    """Checked arguments of the prefill / step entry points (pointers, sizes, input dtype code)."""
    import torch
    if not isinstance(r, torch.Tensor) or r.dim() != 4:
        raise ValueError("r must be a [B, T, H, N] tensor")
    B, T, H, N = r.shape
    _expect(r, "r", r.shape, _input_dtypes(), r)
    for name, t in zip("wkvab", (w, k, v, a, b)):
        _expect(t, name, r.shape, (r.dtype,), r)
    _expect(y, "y", (B, T, H, N), _f32(), r)
    sd = state_dtypes or _f32()
    _expect(state_in, "state_in", (B, H, N, N), sd, r, optional=True)
    _expect(state_out, "state_out", (B, H, N, N), sd, r, optional=True)
    _on_gpu(r, stream)
    return [_ptr(x) for x in (r, w, k, v, a, b, state_in, y, state_out)] + [B, T, H, N, _dtype_code(r)]


def _check(status: int):
    if status != RWKV7_OK:
        raise Rwkv7Error(status, rwkv7_wkv_strerror(status))


def rwkv7_wkv_prefill(r, w, k, v, a, b, state_in, y, state_out, stream=None):
    """Whole-sequence prefill. Tensors as in include/rwkv7_wkv.h ([B,T,H,64] inputs, float32 y and state)."""
    args = _args(r, w, k, v, a, b, state_in, y, state_out, stream)
    _launch("rwkv7_wkv_prefill", args, r, stream)


def rwkv7_wkv_prefill_noalloc(r, w, k, v, a, b, state_in, y, state_out, stream=None):
    """The split chunked prefill with its records in the library's static device array (allocates nothing;
    bfloat16 inputs; calls on one device must not overlap)."""
    args = _args(r, w, k, v, a, b, state_in, y, state_out, stream)
    _launch("rwkv7_wkv_prefill_noalloc", args, r, stream)


def rwkv7_wkv_step(r, w, k, v, a, b, state_in, y, state_out, stream=None):
    """Single-token step (T == 1); state_out may be state_in for an in-place update."""
    args = _args(r, w, k, v, a, b, state_in, y, state_out, stream)
    _launch("rwkv7_wkv_step", args, r, stream)


def _state_code(*states) -> int:
    import torch
    codes = {torch.float32: RWKV7_STATE_F32, torch.bfloat16: RWKV7_STATE_BF16, torch.float16: RWKV7_STATE_F16}
    found = {codes.get(s.dtype, -1) for s in states if s is not None}
    if len(found) > 1:
        raise ValueError("state_in and state_out must share one dtype")
    return found.pop() if found else RWKV7_STATE_F32


def rwkv7_wkv_step_q(r, w, k, v, a, b, state_in, y, state_out, state_dtype=None, stream=None):
    """Single-token step with a float32, bfloat16 or float16 stored state (RWKV7_STATE_*).

    The state format is taken from the state tensors' dtype unless `state_dtype` is given.
    """
    import torch
    sd = _state_code(state_in, state_out) if state_dtype is None else int(state_dtype)
    tdt = {RWKV7_STATE_F32: torch.float32, RWKV7_STATE_BF16: torch.bfloat16, RWKV7_STATE_F16: torch.float16}
    if sd not in tdt:
        raise ValueError("state_dtype must be one of RWKV7_STATE_F32 / _BF16 / _F16")
    args = _args(r, w, k, v, a, b, state_in, y, state_out, stream, state_dtypes=(tdt[sd],))
    _launch("rwkv7_wkv_step_q", args + [sd], r, stream)


def rwkv7_wkv_prefill_ex(r, w, k, v, a, b, state_in, y, state_out, algo=RWKV7_ALGO_AUTO, stream=None):
    """Prefill with an explicit algorithm (RWKV7_ALGO_*)."""
    args = _args(r, w, k, v, a, b, state_in, y, state_out, stream)
    _launch("rwkv7_wkv_prefill_ex", args + [int(algo)], r, stream)


def wkv7(r, w, k, v, a, b, state_in=None, algo=RWKV7_ALGO_AUTO, want_state=True, stream=None):
    """Allocate y ([B,T,H,64] float32) and the final state, run the prefill, return (y, state_out)."""
    B, T, H, N = r.shape
    y, s_out = _on_stream_of(stream, r, lambda: (
        r.new_empty((B, T, H, N), dtype=_T.f32[0]), r.new_empty((B, H, N, N), dtype=_T.f32[0]) if want_state else None))
    rwkv7_wkv_prefill_ex(r, w, k, v, a, b, state_in, y, s_out, algo=algo, stream=stream)
    return y, s_out


def _tmix_args(r, w_raw, k, v, kk, a_lr, ln_w, ln_b, state_in, out, state_out, stream=None):
    import torch
    if not isinstance(r, torch.Tensor) or r.dim() != 4:
        raise ValueError("r must be a [B, T, H, N] tensor")
    B, T, H, N = r.shape
    _expect(r, "r", r.shape, _input_dtypes(), r)
    for name, t in (("k", k), ("v", v), ("kk", kk), ("a_lr", a_lr)):
        _expect(t, name, r.shape, (r.dtype,), r)
    _expect(w_raw, "w_raw", r.shape, _f32(), r)
    _expect(ln_w, "ln_w", (H * N,), _f32(), r, optional=True)
    _expect(ln_b, "ln_b", (H * N,), _f32(), r, optional=True)
    _expect(state_in, "state_in", (B, H, N, N), _f32(), r, optional=True)
    _expect(out, "out", (B, T, H, N), _f32(), r)
    _expect(state_out, "state_out", (B, H, N, N), _f32(), r, optional=True)
    _on_gpu(r, stream)
    return [_ptr(x) for x in (r, w_raw, k, v, kk, a_lr, ln_w, ln_b, state_in, out, state_out)] + \
        [B, T, H, N, _dtype_code(r)]


def rwkv7_tmix_prefill(r, w_raw, k, v, kk, a_lr, ln_w, ln_b, state_in, out, state_out, stream=None):
    """Fused time-mix prefill: prologue (decay, normalised removal key, slots), recurrence, ln_x."""
    args = _tmix_args(r, w_raw, k, v, kk, a_lr, ln_w, ln_b, state_in, out, state_out, stream)
    _launch("rwkv7_tmix_prefill", args, r, stream)


def rwkv7_tmix_prefill_ex(r, w_raw, k, v, kk, a_lr, ln_w, ln_b, state_in, out, state_out, algo=RWKV7_ALGO_AUTO,
                          stream=None):
    """Fused time-mix prefill with an explicit algorithm (RWKV7_ALGO_AUTO / _SEQUENTIAL / _CHUNKED /
    _CHUNKED_SPLIT)."""
    args = _tmix_args(r, w_raw, k, v, kk, a_lr, ln_w, ln_b, state_in, out, state_out, stream)
    _launch("rwkv7_tmix_prefill_ex", args + [int(algo)], r, stream)


def rwkv7_tmix_step(r, w_raw, k, v, kk, a_lr, ln_w, ln_b, state_in, out, state_out, stream=None):
    """Fused time-mix single-token step (T == 1); state_out may be state_in."""
    args = _tmix_args(r, w_raw, k, v, kk, a_lr, ln_w, ln_b, state_in, out, state_out, stream)
    _launch("rwkv7_tmix_step", args, r, stream)


def tmix(r, w_raw, k, v, kk, a_lr, ln_w=None, ln_b=None, state_in=None, want_state=True, algo=RWKV7_ALGO_AUTO,
         stream=None):
    """Allocate out ([B,T,H,64] float32) and the final state, run the fused prefill, return (out, state_out)."""
    B, T, H, N = r.shape
    out, s_out = _on_stream_of(stream, r, lambda: (
        r.new_empty((B, T, H, N), dtype=_T.f32[0]), r.new_empty((B, H, N, N), dtype=_T.f32[0]) if want_state else None))
    rwkv7_tmix_prefill_ex(r, w_raw, k, v, kk, a_lr, ln_w, ln_b, state_in, out, s_out, algo=algo, stream=stream)
    return out, s_out


def rwkv7_wkv_backward(r, w, k, v, a, b, state_in, dy, dstate_out, dr, dw, dk, dv, da, db, dstate_in,
                       stream=None):
    """Gradients of the recurrence: dr..db ([B,T,H,64] float32) and dstate_in ([B,H,64,64] float32 or None)."""
    rwkv7_wkv_backward_ex(r, w, k, v, a, b, state_in, dy, dstate_out, dr, dw, dk, dv, da, db, dstate_in,
                          RWKV7_ALGO_AUTO, stream)


def rwkv7_wkv_backward_ex(r, w, k, v, a, b, state_in, dy, dstate_out, dr, dw, dk, dv, da, db, dstate_in,
                          algo=RWKV7_ALGO_AUTO, stream=None):
    """rwkv7_wkv_backward with an explicit algorithm (RWKV7_ALGO_AUTO / _SEQUENTIAL / _CHUNKED)."""
    import torch
    if not isinstance(r, torch.Tensor) or r.dim() != 4:
        raise ValueError("r must be a [B, T, H, N] tensor")
    B, T, H, N = r.shape
    _expect(r, "r", r.shape, _input_dtypes(), r)
    for name, t in zip("wkvab", (w, k, v, a, b)):
        _expect(t, name, r.shape, (r.dtype,), r)
    _expect(state_in, "state_in", (B, H, N, N), _f32(), r, optional=True)
    _expect(dy, "dy", (B, T, H, N), _f32(), r)
    _expect(dstate_out, "dstate_out", (B, H, N, N), _f32(), r, optional=True)
    for name, t in zip(("dr", "dw", "dk", "dv", "da", "db"), (dr, dw, dk, dv, da, db)):
        _expect(t, name, (B, T, H, N), _f32(), r)
    _expect(dstate_in, "dstate_in", (B, H, N, N), _f32(), r, optional=True)
    _on_gpu(r, stream)
    args = [_ptr(x) for x in (r, w, k, v, a, b, state_in, dy, dstate_out, dr, dw, dk, dv, da, db, dstate_in)]
    _launch("rwkv7_wkv_backward_ex", args + [B, T, H, N, _dtype_code(r), int(algo)], r, stream)


def wkv7_backward(r, w, k, v, a, b, dy, state_in=None, dstate_out=None, want_dstate=True, stream=None,
                  algo=RWKV7_ALGO_AUTO):
    """Allocate the gradients, run the backward, return dict dr, dw, dk, dv, da, db, dstate_in."""
    B, T, H, N = r.shape

    def make():
        out = {n: r.new_empty((B, T, H, N), dtype=_T.f32[0]) for n in ("dr", "dw", "dk", "dv", "da", "db")}
        out["dstate_in"] = r.new_empty((B, H, N, N), dtype=_T.f32[0]) if want_dstate else None
        return out

    out = _on_stream_of(stream, r, make)
    rwkv7_wkv_backward_ex(r, w, k, v, a, b, state_in, dy, dstate_out, *(out[n] for n in
                          ("dr", "dw", "dk", "dv", "da", "db", "dstate_in")), algo=algo, stream=stream)
    return out


def rwkv7_stack_forward(w_in, w_out, vecs, x, states, stream=None):
    """L time-mix layers over the residual stream x ([B,T,D] float32, in place) with per-layer states
    ([L,B,H,64,64] float32, in place). w_in [L,D,5D] and w_out [L,D,D] in float32 or bfloat16."""
    import torch
    if not isinstance(states, torch.Tensor) or states.dim() != 5:
        raise ValueError("states must be an [L, B, H, N, N] tensor")
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a [B, T, D] tensor")
    L, B, H, N = states.shape[0], states.shape[1], states.shape[2], states.shape[3]
    T, D = x.shape[1], H * N
    _expect(states, "states", (L, B, H, N, N), _f32(), states)
    _expect(x, "x", (B, T, D), _f32(), states)
    _expect(w_in, "w_in", (L, D, 5 * D), _input_dtypes(), states)
    _expect(w_out, "w_out", (L, D, D), (w_in.dtype,), states)
    _expect(vecs, "vecs", (L, 5, D), _f32(), states)
    _on_gpu(states, stream)
    args = [_ptr(w_in), _ptr(w_out), _ptr(vecs), _ptr(x), _ptr(states), L, B, T, H, N, _dtype_code(w_in)]
    _launch("rwkv7_stack_forward", args, states, stream)


# ---- linear attention with a decay for each head

def _linattn_inputs(r, log_w, k, v, state_in):
    """The addresses of the inputs that the linear attention's calls share, the sizes and log_w's layout."""
    if not isinstance(r, _T.Tensor) or r.dim() != 4:
        raise ValueError("r must be a [B, T, H, N] tensor")
    shape = r.shape
    B, T, H, N = shape
    at = [_at(r, "r", shape, _T.inputs, r)]
    if not isinstance(log_w, _T.Tensor):
        raise TypeError("log_w must be a torch.Tensor, not %s" % type(log_w).__name__)
    decay = RWKV7_DECAY_HEAD if log_w.dim() == 1 else RWKV7_DECAY_TOKEN
    at.append(_at(log_w, "log_w", (H,) if decay == RWKV7_DECAY_HEAD else (B, T, H), _T.f32, r))
    same = (r.dtype,)
    at.append(_at(k, "k", shape, same, r))
    at.append(_at(v, "v", shape, same, r))
    at.append(None if state_in is None else _at(state_in, "state_in", (B, H, N, N), _T.f32, r))
    return at, shape, same, decay


def rwkv7_linattn_prefill(r, log_w, k, v, state_in, lens, y, state_out, stream=None):
    """Linear attention over a prompt. r, k, v, y [B,T,H,64] in one dtype; log_w float32 [H] or [B,T,H];
    lens int32 [B] or None; states float32 [B,H,64,64] or None."""
    at, shape, same, decay = _linattn_inputs(r, log_w, k, v, state_in)
    B, T, H, N = shape
    at.append(None if lens is None else _at(lens, "lens", (B,), _T.i32, r))
    at.append(_at(y, "y", shape, same, r))
    at.append(None if state_out is None else _at(state_out, "state_out", (B, H, N, N), _T.f32, r))
    at += (B, T, H, N, _dtype_code(r), decay)
    _launch("rwkv7_linattn_prefill", at, r, stream)


def rwkv7_linattn_step(r, log_w, k, v, state_in, y, state_out, stream=None):
    """Single-token step (T == 1) of the linear attention; state_out may be state_in."""
    at, shape, same, decay = _linattn_inputs(r, log_w, k, v, state_in)
    B, T, H, N = shape
    at.append(_at(y, "y", shape, same, r))
    at.append(None if state_out is None else _at(state_out, "state_out", (B, H, N, N), _T.f32, r))
    at += (B, T, H, N, _dtype_code(r), decay)
    _launch("rwkv7_linattn_step", at, r, stream)


def linattn(r, log_w, k, v, state_in=None, lens=None, want_state=True, stream=None):
    """Allocate y ([B,T,H,64] in r's dtype) and the final state, run the prompt, return (y, state_out)."""
    B, T, H, N = r.shape
    y, s_out = _on_stream_of(stream, r, lambda: (
        _T.empty_like(r), r.new_empty((B, H, N, N), dtype=_T.f32[0]) if want_state else None))
    rwkv7_linattn_prefill(r, log_w, k, v, state_in, lens, y, s_out, stream)
    return y, s_out


def linattn_step(r, log_w, k, v, state_in=None, stream=None):
    """Allocate y ([B,1,H,64] in r's dtype) and the new state, run one token, return (y, state_out).
    rwkv7_linattn_step updates a state in place."""
    B, T, H, N = r.shape
    y, s_out = _on_stream_of(stream, r, lambda: (_T.empty_like(r), r.new_empty((B, H, N, N), dtype=_T.f32[0])))
    rwkv7_linattn_step(r, log_w, k, v, state_in, y, s_out, stream)
    return y, s_out


def rwkv7_linattn_backward(r, log_w, k, v, state_in, lens, dy, dstate_out, dr, dlog_w, dk, dv, dstate_in, stream=None):
    """Gradients of the linear attention: dr, dk, dv in r's dtype, dlog_w float32 in log_w's layout, dstate_in
    float32 or None (may be dstate_out)."""
    at, shape, same, decay = _linattn_inputs(r, log_w, k, v, state_in)
    B, T, H, N = shape
    states = (B, H, N, N)
    at.append(None if lens is None else _at(lens, "lens", (B,), _T.i32, r))
    at.append(_at(dy, "dy", shape, same, r))
    at.append(None if dstate_out is None else _at(dstate_out, "dstate_out", states, _T.f32, r))
    at.append(_at(dr, "dr", shape, same, r))
    at.append(_at(dlog_w, "dlog_w", log_w.shape, _T.f32, r))
    at.append(_at(dk, "dk", shape, same, r))
    at.append(_at(dv, "dv", shape, same, r))
    at.append(None if dstate_in is None else _at(dstate_in, "dstate_in", states, _T.f32, r))
    at += (B, T, H, N, _dtype_code(r), decay)
    _launch("rwkv7_linattn_backward", at, r, stream)


def linattn_backward(r, log_w, k, v, dy, state_in=None, lens=None, dstate_out=None, want_dstate=True, stream=None):
    """Allocate the gradients, run the backward, return dict dr, dlog_w, dk, dv, dstate_in."""
    B, T, H, N = r.shape

    def make():
        out = {n: _T.empty_like(r) for n in ("dr", "dk", "dv")}
        out["dlog_w"] = _T.empty_like(log_w)
        out["dstate_in"] = r.new_empty((B, H, N, N), dtype=_T.f32[0]) if want_dstate else None
        return out

    out = _on_stream_of(stream, r, make)
    rwkv7_linattn_backward(r, log_w, k, v, state_in, lens, dy, dstate_out, out["dr"], out["dlog_w"], out["dk"],
                           out["dv"], out["dstate_in"], stream)
    return out


# ---- layer norm over groups of channels

def _rows(x, groups):
    """x's address, rows and channels: the last dimension is normalised, in `groups` groups."""
    if not isinstance(x, _T.Tensor) or x.dim() < 1:
        raise ValueError("x must be a tensor with the channels in its last dimension")
    shape = x.shape
    at = _at(x, "x", shape, _T.inputs, x)
    D, G = shape[-1], int(groups)
    if G < 1 or D % G:
        raise ValueError("groups is %d, expected a divisor of the %d channels" % (G, D))
    M = shape[0] if len(shape) == 2 else shape[:-1].numel()
    return at, shape, M, D, G


def rwkv7_layernorm_forward(x, weight, bias, y, mean, rstd, groups=1, eps=1e-5, stream=None):
    """Layer norm of x's last dimension in `groups` groups. x and y [..., D] in float32 or bfloat16 (each its
    own), weight and bias [D] float32 or None, mean and rstd [..., groups] float32 or None."""
    at_x, shape, M, D, G = _rows(x, groups)
    stats = shape[:-1] + (G,)
    args = [at_x,
            None if weight is None else _at(weight, "weight", (D,), _T.f32, x),
            None if bias is None else _at(bias, "bias", (D,), _T.f32, x),
            _at(y, "y", shape, _T.inputs, x),
            None if mean is None else _at(mean, "mean", stats, _T.f32, x),
            None if rstd is None else _at(rstd, "rstd", stats, _T.f32, x),
            M, D, G, eps, _dtype_code(x), _dtype_code(y)]
    _launch("rwkv7_layernorm_forward", args, x, stream)


def rwkv7_layernorm_backward(x, weight, mean, rstd, dy, dx, dweight, dbias, groups=1, stream=None):
    """Gradients of the layer norm from its x, weight, mean and rstd; dweight and dbias [D] float32 or None."""
    at_x, shape, M, D, G = _rows(x, groups)
    stats = shape[:-1] + (G,)
    args = [at_x,
            None if weight is None else _at(weight, "weight", (D,), _T.f32, x),
            _at(mean, "mean", stats, _T.f32, x),
            _at(rstd, "rstd", stats, _T.f32, x),
            _at(dy, "dy", shape, _T.inputs, x),
            _at(dx, "dx", shape, (x.dtype,), x),
            None if dweight is None else _at(dweight, "dweight", (D,), _T.f32, x),
            None if dbias is None else _at(dbias, "dbias", (D,), _T.f32, x),
            M, D, G, _dtype_code(x), _dtype_code(dy)]
    _launch("rwkv7_layernorm_backward", args, x, stream)


def layernorm(x, weight=None, bias=None, groups=1, eps=1e-5, out_dtype=None, want_stats=True, stream=None):
    """Allocate y (in out_dtype, or x's) and the statistics, run the forward, return (y, mean, rstd)."""
    def make():
        y = _T.empty_like(x, dtype=out_dtype)
        mean = x.new_empty(x.shape[:-1] + (groups,), dtype=_T.f32[0]) if want_stats else None
        return y, mean, _T.empty_like(mean) if want_stats else None

    y, mean, rstd = _on_stream_of(stream, x, make)
    rwkv7_layernorm_forward(x, weight, bias, y, mean, rstd, groups, eps, stream)
    return y, mean, rstd


def layernorm_backward(x, weight, mean, rstd, dy, groups=1, want_dweight=True, stream=None):
    """Allocate the gradients, run the backward, return dict dx, dweight, dbias (the last two None unless
    want_dweight)."""
    def make():
        out = {"dx": _T.empty_like(x), "dweight": None, "dbias": None}
        if want_dweight:
            out["dweight"] = x.new_empty(x.shape[-1:], dtype=_T.f32[0])
            out["dbias"] = _T.empty_like(out["dweight"])
        return out

    out = _on_stream_of(stream, x, make)
    rwkv7_layernorm_backward(x, weight, mean, rstd, dy, out["dx"], out["dweight"], out["dbias"], groups, stream)
    return out
