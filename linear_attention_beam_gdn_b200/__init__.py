"""Python binding of the beam-parallel Gated DeltaNet decode library (C ABI in include/ola.h).

Argument marshalling only: every step of the decode runs in the library's CUDA kernels.
The functions named ``ola_*`` mirror the C entry points one to one and take raw device
pointers (ints); :class:`Decoder` and :func:`prefill` take torch tensors, check their
device, dtype, shape and contiguity, and pass ``data_ptr()`` and the current CUDA stream.

There is no fallback: if the shared object has not been built, importing works but every
call raises :class:`LibraryMissing`.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Optional

__all__ = ["OlaError", "LibraryMissing", "Geometry", "lib", "Decoder", "prefill",
           "OLA_F32", "OLA_BF16", "OLA_PATH_REPLAY", "OLA_PATH_FULLSTATE", "OLA_PATH_REPLAYSSM",
           "OLA_MATH_FP32",
           "OLA_MATH_TENSOR", "LIB_PATH", "HEADER_PATH", "declared_symbols",
           "ConvDesc", "QkDesc", "ScanDesc", "conv", "conv_step", "qk_norm", "scan", "scan_step",
           "layer_status"]

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "_build", "libola.so")
HEADER_PATH = os.path.join(os.path.dirname(PKG_DIR), "include", "ola.h")

OLA_OK, OLA_ERR_INVALID_ARG, OLA_ERR_UNSUPPORTED, OLA_ERR_CAPACITY = 0, 1, 2, 3
OLA_ERR_BAD_PARENT, OLA_ERR_OOM, OLA_ERR_CUDA, OLA_ERR_TIMEOUT = 4, 5, 6, 7
OLA_ERR_SCRATCH_LIMIT = 8
OLA_NOALLOC_SCRATCH_BYTES = 16 << 20
OLA_F32, OLA_BF16 = 0, 1
OLA_PATH_REPLAY, OLA_PATH_FULLSTATE, OLA_PATH_REPLAYSSM = 0, 1, 2
OLA_MATH_FP32, OLA_MATH_TENSOR = 0, 1


class LibraryMissing(RuntimeError):
    pass


class OlaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib().ola_strerror(status).decode()
        super().__init__(f"{where}: {msg} (status {status})")


class Geometry(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int32), ("H", ctypes.c_int32), ("d_k", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("B", ctypes.c_int32), ("T_max", ctypes.c_int32),
                ("in_dtype", ctypes.c_int32), ("path", ctypes.c_int32),
                ("math", ctypes.c_int32)]


class ConvDesc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("R", "P", "C", "W", "in_dtype", "silu")] +
                [(n, ctypes.c_int64) for n in ("x_tok", "x_seq", "y_tok", "y_seq")])


class QkDesc(ctypes.Structure):
    _fields_ = ([("N", ctypes.c_int64)] +
                [(n, ctypes.c_int32) for n in ("Hq", "Hk", "d", "in_dtype", "l2", "rot", "pair")] +
                [("eps", ctypes.c_float)] +
                [(n, ctypes.c_int64) for n in ("q_tok", "k_tok", "qo_tok", "ko_tok")])


class ScanDesc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("R", "P", "H", "G", "d_k", "d_v", "in_dtype",
                                               "softplus")] +
                [(n, ctypes.c_int64) for n in ("v_tok", "v_seq", "k_tok", "k_seq", "q_tok",
                                               "q_seq", "z_tok", "z_seq", "y_tok", "y_seq")])


_LIB: Optional[ctypes.CDLL] = None
_P = ctypes.c_void_p


def _declare(L: ctypes.CDLL) -> None:
    i32, u64p = ctypes.c_int32, ctypes.POINTER(ctypes.c_uint64)
    sig = {
        "ola_version": (i32, []),
        "ola_strerror": (ctypes.c_char_p, [i32]),
        "ola_workspace_bytes": (i32, [ctypes.POINTER(Geometry), u64p]),
        "ola_create": (i32, [ctypes.POINTER(Geometry), _P, _P, ctypes.POINTER(_P)]),
        "ola_step": (i32, [_P, _P, _P, _P, _P, _P, _P, _P, _P]),
        "ola_step_host": (i32, [_P, _P, _P, _P, _P, _P, _P, _P, _P]),
        "ola_step_host_async": (i32, [_P, _P, _P, _P, _P, _P, _P, _P, _P]),
        "ola_host_sync": (i32, [_P]),
        "ola_reset": (i32, [_P]),
        "ola_current_step": (i32, [_P]),
        "ola_get_ancestry": (i32, [_P, _P, _P]),
        "ola_get_error": (i32, [_P]),
        "ola_compact": (i32, [_P, ctypes.POINTER(ctypes.c_int32), _P]),
        "ola_destroy": (i32, [_P]),
        "ola_prefill": (i32, [i32, i32, i32, i32, i32, i32, _P, _P, _P, _P, _P, _P]),
        "ola_layer_status": (i32, [_P]),
        "ola_conv": (i32, [ctypes.POINTER(ConvDesc)] + [_P] * 8),
        "ola_conv_step": (i32, [ctypes.POINTER(ConvDesc), i32] + [_P] * 8),
        "ola_qk_norm": (i32, [ctypes.POINTER(QkDesc)] + [_P] * 9),
        "ola_scan_workspace_bytes": (i32, [ctypes.POINTER(ScanDesc), u64p]),
        "ola_scan": (i32, [ctypes.POINTER(ScanDesc)] + [_P] * 13 + [ctypes.c_uint64, _P]),
        "ola_scan_step": (i32, [ctypes.POINTER(ScanDesc), i32] + [_P] * 13),
        "ola_noalloc_scratch_bytes": (ctypes.c_uint64, [ctypes.POINTER(Geometry)]),
        "ola_decode_noalloc": (i32, [ctypes.POINTER(Geometry), _P, _P, _P, _P, _P, _P, _P, _P,
                                     _P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args


def lib() -> ctypes.CDLL:
    """The loaded shared object (raises LibraryMissing if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise LibraryMissing(
                f"{LIB_PATH} is missing: build it with "
                "`python -m linear_attention_beam_gdn_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        _declare(L)
        _LIB = L
    return _LIB


def declared_symbols(header: str = HEADER_PATH):
    """Names of the functions declared in the C header."""
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(ola_[a-z_]+)\s*\(", text)))


def _check(status: int, where: str) -> None:
    if status != OLA_OK:
        raise OlaError(status, where)


# ------------------------------------------------------------------ raw C entry points

def ola_version() -> int:
    return lib().ola_version()


def ola_strerror(status: int) -> str:
    return lib().ola_strerror(status).decode()


def ola_workspace_bytes(geom: Geometry) -> int:
    out = ctypes.c_uint64(0)
    _check(lib().ola_workspace_bytes(ctypes.byref(geom), ctypes.byref(out)),
           "ola_workspace_bytes")
    return out.value


def ola_create(geom: Geometry, S_ctx_ptr: int, stream: int) -> int:
    h = _P()
    _check(lib().ola_create(ctypes.byref(geom), S_ctx_ptr, stream, ctypes.byref(h)),
           "ola_create")
    return h.value


def ola_step(h, q, k, v, g, beta, parent_idx, out_o, stream) -> int:
    return lib().ola_step(h, q, k, v, g, beta, parent_idx, out_o, stream)


def ola_step_host(h, q, k, v, g, beta, parent_idx, out_o, stream) -> int:
    return lib().ola_step_host(h, q, k, v, g, beta, parent_idx, out_o, stream)


def ola_step_host_async(h, q, k, v, g, beta, parent_idx, out_o, stream) -> int:
    return lib().ola_step_host_async(h, q, k, v, g, beta, parent_idx, out_o, stream)


def ola_host_sync(h) -> int:
    return lib().ola_host_sync(h)


def ola_reset(h) -> int:
    return lib().ola_reset(h)


def ola_current_step(h) -> int:
    return lib().ola_current_step(h)


def ola_get_ancestry(h, out, stream) -> int:
    return lib().ola_get_ancestry(h, out, stream)


def ola_get_error(h) -> int:
    return lib().ola_get_error(h)


def ola_destroy(h) -> int:
    return lib().ola_destroy(h)


def ola_compact(h, stream) -> tuple:
    """(status, number of folded steps)."""
    n = ctypes.c_int32(0)
    st = lib().ola_compact(h, ctypes.byref(n), stream)
    return st, n.value


def ola_prefill(R, H, d_k, d_v, P, in_dtype, k, v, g, beta, S_out, stream) -> int:
    return lib().ola_prefill(R, H, d_k, d_v, P, in_dtype, k, v, g, beta, S_out, stream)


def ola_noalloc_scratch_bytes(geom: Geometry) -> int:
    return lib().ola_noalloc_scratch_bytes(ctypes.byref(geom))


def ola_decode_noalloc(geom: Geometry, S_ctx, q, k, v, g, beta, parent_idx, out_o,
                       stream) -> int:
    return lib().ola_decode_noalloc(ctypes.byref(geom), S_ctx, q, k, v, g, beta, parent_idx,
                                    out_o, stream)


def ola_layer_status(stream) -> int:
    return lib().ola_layer_status(stream)


def ola_conv(desc: ConvDesc, x, w, bias, state_in, lens, y, state_out, stream) -> int:
    return lib().ola_conv(ctypes.byref(desc), x, w, bias, state_in, lens, y, state_out, stream)


def ola_conv_step(desc: ConvDesc, Bp, x, w, bias, state_in, parent_idx, y, state_out,
                  stream) -> int:
    return lib().ola_conv_step(ctypes.byref(desc), Bp, x, w, bias, state_in, parent_idx, y,
                               state_out, stream)


def ola_qk_norm(desc: QkDesc, q, k, wq, wk, positions, inv_freq, q_out, k_out, stream) -> int:
    return lib().ola_qk_norm(ctypes.byref(desc), q, k, wq, wk, positions, inv_freq, q_out, k_out,
                             stream)


def ola_scan_workspace_bytes(desc: ScanDesc) -> int:
    out = ctypes.c_uint64(0)
    _check(lib().ola_scan_workspace_bytes(ctypes.byref(desc), ctypes.byref(out)),
           "ola_scan_workspace_bytes")
    return out.value


def ola_scan(desc: ScanDesc, v, dt, A, k, q, D, dt_bias, z, S_in, lens, y, S_out, ws, ws_bytes,
             stream) -> int:
    return lib().ola_scan(ctypes.byref(desc), v, dt, A, k, q, D, dt_bias, z, S_in, lens, y, S_out,
                          ws, ws_bytes, stream)


def ola_scan_step(desc: ScanDesc, Bp, v, dt, A, k, q, D, dt_bias, z, state_in, parent_idx, y,
                  state_out, stream) -> int:
    return lib().ola_scan_step(ctypes.byref(desc), Bp, v, dt, A, k, q, D, dt_bias, z, state_in,
                               parent_idx, y, state_out, stream)


# ------------------------------------------------------------------ torch-facing wrappers

_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _stream_ptr(stream=None) -> int:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def _dtype_code(dt) -> int:
    torch = _torch()
    if dt == torch.bfloat16:
        return OLA_BF16
    if dt == torch.float32:
        return OLA_F32
    raise TypeError(f"unsupported input dtype {dt}")


def _need(x, shape, dtype, name, device):
    torch = _torch()
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.device != device:
        raise ValueError(f"{name} is on {x.device}, expected {device}")
    if tuple(x.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(x.shape)}, expected {tuple(shape)}")
    if x.dtype != dtype:
        raise TypeError(f"{name} has dtype {x.dtype}, expected {dtype}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return x.data_ptr()


def prefill(k, v, g, beta, stream=None):
    """Shared post-prefill state S [R, H, d_v, d_k] fp32 from prompt tokens
    k [R, P, H, d_k], v [R, P, H, d_v] (bf16 or fp32), g, beta [R, P, H] fp32."""
    torch = _torch()
    R, P, H, d_k = k.shape
    d_v = v.shape[-1]
    dev = k.device
    dt = k.dtype
    S = torch.empty((R, H, d_v, d_k), device=dev, dtype=torch.float32)
    args = [_need(k, (R, P, H, d_k), dt, "k", dev), _need(v, (R, P, H, d_v), dt, "v", dev),
            _need(g, (R, P, H), torch.float32, "g", dev),
            _need(beta, (R, P, H), torch.float32, "beta", dev)]
    _check(ola_prefill(R, H, d_k, d_v, P, _dtype_code(dt), *args, S.data_ptr(),
                       _stream_ptr(stream)), "ola_prefill")
    return S


class Decoder:
    """One GDN layer's beam decoder for R requests (owns an ola handle)."""

    def __init__(self, S_ctx, B: int, T_max: int, in_dtype, path: int = OLA_PATH_REPLAY,
                 math: int = OLA_MATH_TENSOR, stream=None):
        torch = _torch()
        R, H, d_v, d_k = S_ctx.shape
        self.geom = Geometry(R, H, d_k, d_v, B, T_max, _dtype_code(in_dtype), path, math)
        self.device = S_ctx.device
        self.in_dtype = in_dtype
        ptr = _need(S_ctx, (R, H, d_v, d_k), torch.float32, "S_ctx", self.device)
        self.handle = ola_create(self.geom, ptr, _stream_ptr(stream))

    # shapes
    @property
    def R(self): return self.geom.R

    @property
    def H(self): return self.geom.H

    @property
    def B(self): return self.geom.B

    @property
    def d_k(self): return self.geom.d_k

    @property
    def d_v(self): return self.geom.d_v

    @property
    def t(self) -> int:
        return ola_current_step(self.handle)

    def _ptrs(self, q, k, v, g, beta, parent_idx, out):
        torch = _torch()
        R, B, H, dk, dv = self.R, self.B, self.H, self.d_k, self.d_v
        dev, dt = self.device, self.in_dtype
        return [_need(q, (R, B, H, dk), dt, "q", dev), _need(k, (R, B, H, dk), dt, "k", dev),
                _need(v, (R, B, H, dv), dt, "v", dev),
                _need(g, (R, B, H), torch.float32, "g", dev),
                _need(beta, (R, B, H), torch.float32, "beta", dev),
                _need(parent_idx, (R, B), torch.int32, "parent_idx", dev),
                _need(out, (R, B, H, dv), torch.float32, "out_o", dev)]

    def step(self, q, k, v, g, beta, parent_idx, out=None, stream=None):
        """Run one decode step; returns o [R, B, H, d_v] fp32."""
        torch = _torch()
        if out is None:
            out = torch.empty((self.R, self.B, self.H, self.d_v), device=self.device,
                              dtype=torch.float32)
        _check(ola_step(self.handle, *self._ptrs(q, k, v, g, beta, parent_idx, out),
                        _stream_ptr(stream)), "ola_step")
        return out

    def step_host(self, q, k, v, g, beta, parent_idx, out, stream=None):
        """ola_step_host: all tensors on the CPU (pinned for asynchronous copies)."""
        torch = _torch()
        cpu = torch.device("cpu")
        R, B, H, dk, dv = self.R, self.B, self.H, self.d_k, self.d_v
        dt = self.in_dtype
        ptrs = [_need(q, (R, B, H, dk), dt, "q", cpu), _need(k, (R, B, H, dk), dt, "k", cpu),
                _need(v, (R, B, H, dv), dt, "v", cpu),
                _need(g, (R, B, H), torch.float32, "g", cpu),
                _need(beta, (R, B, H), torch.float32, "beta", cpu),
                _need(parent_idx, (R, B), torch.int32, "parent_idx", cpu),
                _need(out, (R, B, H, dv), torch.float32, "out_o", cpu)]
        _check(ola_step_host(self.handle, *ptrs, _stream_ptr(stream)), "ola_step_host")
        return out

    def step_host_async(self, q, k, v, g, beta, parent_idx, out, stream=None):
        """ola_step_host_async: CPU tensors (pinned); `out` is complete after host_sync()."""
        torch = _torch()
        cpu = torch.device("cpu")
        R, B, H, dk, dv = self.R, self.B, self.H, self.d_k, self.d_v
        dt = self.in_dtype
        ptrs = [_need(q, (R, B, H, dk), dt, "q", cpu), _need(k, (R, B, H, dk), dt, "k", cpu),
                _need(v, (R, B, H, dv), dt, "v", cpu),
                _need(g, (R, B, H), torch.float32, "g", cpu),
                _need(beta, (R, B, H), torch.float32, "beta", cpu),
                _need(parent_idx, (R, B), torch.int32, "parent_idx", cpu),
                _need(out, (R, B, H, dv), torch.float32, "out_o", cpu)]
        _check(ola_step_host_async(self.handle, *ptrs, _stream_ptr(stream)),
               "ola_step_host_async")
        return out

    def host_sync(self) -> None:
        _check(ola_host_sync(self.handle), "ola_host_sync")

    def ancestry(self, stream=None):
        """Chains of the current beams: [R, B, t] int32 (device)."""
        torch = _torch()
        t = self.t
        out = torch.empty((self.R, self.B, t), device=self.device, dtype=torch.int32)
        _check(ola_get_ancestry(self.handle, out.data_ptr(), _stream_ptr(stream)),
               "ola_get_ancestry")
        return out

    def error(self) -> int:
        return ola_get_error(self.handle)

    def compact(self, stream=None) -> int:
        """Fold the chain steps every live beam shares into S_ctx and free their slots
        (ola_compact); returns the number of folded steps."""
        st, n = ola_compact(self.handle, _stream_ptr(stream))
        _check(st, "ola_compact")
        return n

    def reset(self) -> None:
        _check(ola_reset(self.handle), "ola_reset")

    def close(self) -> None:
        if getattr(self, "handle", None):
            ola_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


# ------------------------------------------------------------------ operators around the recurrence
#
# Each call runs on the device of its first tensor and on `stream` of it (default: its current
# stream), allocates only the outputs and scratch that it is not given (they belong to that
# stream), and does not wait. Inputs that may be strided are [sequence, token, ...] with contiguous
# channels, so a slice of a wide projection's columns is taken as it is. A decode step of a few
# tokens costs less on the device than its argument checks can on the host, so these are kept to a
# few attribute reads per tensor.

class _Scope:
    """The device of a call and the stream its kernels and allocations belong to."""

    def __init__(self, index, stream):
        torch = _torch()
        self.index, self.stream = index, stream
        self.device = torch.cuda.device(index)
        self.on = torch.cuda.stream(stream) if stream is not None else None

    def __enter__(self):
        self.device.__enter__()
        if self.on is None:
            return _torch()._C._cuda_getCurrentRawStream(self.index)
        self.on.__enter__()
        return self.stream.cuda_stream

    def __exit__(self, *exc):
        if self.on is not None:
            self.on.__exit__(*exc)
        self.device.__exit__(*exc)


class _Here:
    """The same for a call on the current device and stream."""
    __slots__ = ("raw",)

    def __init__(self, raw):
        self.raw = raw

    def __enter__(self):
        return self.raw

    def __exit__(self, *exc):
        pass


def _scope(index, stream):
    c = _torch()._C
    if stream is None:
        if c._cuda_getDevice() == index:
            return _Here(c._cuda_getCurrentRawStream(index))
    elif stream.device_index != index:
        # the kernels would run on that device with another one's pointers
        raise ValueError(f"stream is on cuda:{stream.device_index}, the tensors on cuda:{index}")
    return _Scope(index, stream)


def _first(x, name, ndim):
    """Checks the leading tensor of a call; returns (device index, dtype code)."""
    torch = _torch()
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    index = x.get_device()
    if index < 0 or not x.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if x.dim() != ndim:
        raise ValueError(f"{name} has {x.dim()} dimensions, expected {ndim}")
    return index, _dtype_code(x.dtype)


def _bad(x, name, shape, dtype, index):
    """Raises what is wrong with a tensor argument."""
    torch = _torch()
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.get_device() != index or not x.is_cuda:
        raise ValueError(f"{name} is on {x.device}, expected cuda:{index}")
    if tuple(x.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(x.shape)}, expected {tuple(shape)}")
    if x.dtype != dtype:
        raise TypeError(f"{name} has dtype {x.dtype}, expected {dtype}")
    raise ValueError(f"{name} must be contiguous")


def _ptr(x, name, shape, dtype, index):
    """Pointer of a contiguous tensor argument."""
    try:
        if (x.shape == shape and x.dtype is dtype and x.get_device() == index and
                x.is_contiguous()):
            return x.data_ptr()
    except AttributeError:
        pass
    _bad(x, name, shape, dtype, index)


def _opt(x, name, shape, dtype, index):
    return None if x is None else _ptr(x, name, shape, dtype, index)


def _rows(x, name, shape, dtype, index):
    """(pointer, token stride, sequence stride) of a [sequence, token, ...] argument whose channels
    are contiguous; strides of 0 stand for a contiguous tensor."""
    try:
        fine = x.shape == shape and x.dtype is dtype and x.get_device() == index
    except AttributeError:
        fine = False
    if not fine:
        _bad(x, name, shape, dtype, index)
    if x.is_contiguous():
        return x.data_ptr(), 0, 0
    st, width = x.stride(), 1
    for n, s in zip(reversed(shape[2:]), reversed(st[2:])):
        if n != 1 and s != width:
            raise ValueError(f"{name}: channels must be contiguous")
        width *= n
    R, P = shape[:2]
    tok = st[1] if P > 1 else width
    seq = st[0] if R > 1 else P * tok
    if tok < width or seq < 1:
        raise ValueError(f"{name}: tokens must not overlap")
    return x.data_ptr(), tok, seq


def _opt_rows(x, name, shape, dtype, index):
    return (None, 0, 0) if x is None else _rows(x, name, shape, dtype, index)


def layer_status(device=None, stream=None) -> int:
    """Waits for `stream` and returns the first device-side error that an operator recorded on
    `device` (default: the stream's, or the current one) since the last call (OLA_OK if none), and
    clears it."""
    torch = _torch()
    if stream is not None:
        index = torch.device(device).index if isinstance(device, str) else \
            getattr(device, "index", device)
        if index is not None and index != stream.device_index:
            raise ValueError(f"stream is on cuda:{stream.device_index}, not on {device}")
        device = stream.device_index
    with torch.cuda.device(device):
        st = ola_layer_status(_stream_ptr(stream))
    if st in (OLA_ERR_CUDA, OLA_ERR_UNSUPPORTED):
        raise OlaError(st, "ola_layer_status")
    return st


def _taps(w):
    if not isinstance(w, _torch().Tensor) or w.dim() != 2:
        raise ValueError("w must be a tensor [C, W]")
    return max(w.shape[1], 1)


def conv(x, w, bias=None, *, state=None, lens=None, silu=True, out=None, state_out=None,
         stream=None):
    """Short causal convolution of a prompt (ola_conv): x [R, P, C] (bf16 or fp32, may be a column
    slice), w [C, W] and bias [C] fp32, state [R, W-1, C] (the tokens before, default zeros), lens
    [R] int32 for a padded batch. Returns (y [R, P, C], state_out [R, W-1, C]); rows of `out`
    behind a sequence's end are not written. state_out may be `state`."""
    torch = _torch()
    ix, code = _first(x, "x", 3)
    R, P, C = shape = x.shape
    W, dt, f32 = _taps(w), x.dtype, torch.float32
    with _scope(ix, stream) as st:
        if out is None:
            out = torch.empty(shape, device=x.device, dtype=dt)
        win = (R, W - 1, C)
        if state_out is None:
            state_out = torch.empty(win, device=x.device, dtype=dt)
        xp, x_tok, x_seq = _rows(x, "x", shape, dt, ix)
        yp, y_tok, y_seq = _rows(out, "out", shape, dt, ix)
        d = ConvDesc(R, P, C, W, code, bool(silu), x_tok, x_seq, y_tok, y_seq)
        _check(ola_conv(d, xp, _ptr(w, "w", (C, W), f32, ix), _opt(bias, "bias", (C,), f32, ix),
                        _opt(state, "state", win, dt, ix),
                        _opt(lens, "lens", (R,), torch.int32, ix), yp,
                        _ptr(state_out, "state_out", win, dt, ix), st), "ola_conv")
    return out, state_out


def conv_step(x, w, bias=None, *, state, parent_idx=None, silu=True, out=None, state_out=None,
              stream=None):
    """One token of every beam through the convolution (ola_conv_step): x [R, B, C], state
    [R, Bp, W-1, C], parent_idx [R, B] int32 (default: beam b continues state b, or the only
    one). Returns (y [R, B, C], state_out [R, B, W-1, C]); state_out may be `state` when
    parent_idx is None."""
    torch = _torch()
    ix, code = _first(x, "x", 3)
    R, B, C = shape = x.shape
    W, dt, f32 = _taps(w), x.dtype, torch.float32
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be a tensor [R, Bp, W-1, C]")
    Bp = state.shape[1]
    with _scope(ix, stream) as st:
        if out is None:
            out = torch.empty(shape, device=x.device, dtype=dt)
        if state_out is None:
            state_out = torch.empty((R, B, W - 1, C), device=x.device, dtype=dt)
        xp, x_tok, x_seq = _rows(x, "x", shape, dt, ix)
        yp, y_tok, y_seq = _rows(out, "out", shape, dt, ix)
        d = ConvDesc(R, B, C, W, code, bool(silu), x_tok, x_seq, y_tok, y_seq)
        _check(ola_conv_step(d, Bp, xp, _ptr(w, "w", (C, W), f32, ix),
                             _opt(bias, "bias", (C,), f32, ix),
                             _ptr(state, "state", (R, Bp, W - 1, C), dt, ix),
                             _opt(parent_idx, "parent_idx", (R, B), torch.int32, ix), yp,
                             _ptr(state_out, "state_out", (R, B, W - 1, C), dt, ix), st),
               "ola_conv_step")
    return out, state_out


def _tokens(x, name, shape, dtype, index):
    """(pointer, token stride) of a tensor [R, P, H, d] whose tokens are evenly spaced."""
    ptr, tok, seq = _rows(x, name, shape, dtype, index)
    R, P = shape[:2]
    if P == 1 and R > 1:
        tok = seq
    elif R > 1 and seq != P * tok:
        raise ValueError(f"{name}: sequences must follow one another at the token stride")
    return ptr, tok


def qk_norm(q, k, *, wq=None, wk=None, eps=1e-6, l2=False, positions=None, inv_freq=None,
            pair=False, q_out=None, k_out=None, stream=None):
    """Norm of every query and key head and the position rotation in one pass (ola_qk_norm):
    q [R, P, Hq, d], k [R, P, Hk, d] (may be column slices of one projection), weights [d] fp32,
    l2=True for unit heads instead of unit mean square; with inv_freq [rot/2] fp32 and positions
    [R, P] int32 the first `rot` dims are rotated, pairs (i, i + rot/2) or (pair=True)
    (2i, 2i + 1). Returns (q_out, k_out); q_out may be q and k_out may be k."""
    torch = _torch()
    ix, code = _first(q, "q", 4)
    R, P, Hq, d = qs = q.shape
    dt, f32 = q.dtype, torch.float32
    if not isinstance(k, torch.Tensor) or k.dim() != 4 or k.shape[:2] != qs[:2] or \
            k.shape[3] != d:
        raise ValueError("k must be a tensor [R, P, Hk, d] with q's R, P and d")
    ks = k.shape
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq go together")
    half = inv_freq.numel() if inv_freq is not None else 0
    with _scope(ix, stream) as st:
        if q_out is None:
            q_out = torch.empty(qs, device=q.device, dtype=dt)
        if k_out is None:
            k_out = torch.empty(ks, device=q.device, dtype=dt)
        qp, q_tok = _tokens(q, "q", qs, dt, ix)
        kp, k_tok = _tokens(k, "k", ks, dt, ix)
        qo, qo_tok = _tokens(q_out, "q_out", qs, dt, ix)
        ko, ko_tok = _tokens(k_out, "k_out", ks, dt, ix)
        desc = QkDesc(R * P, Hq, ks[2], d, code, bool(l2), 2 * half, bool(pair), eps, q_tok, k_tok,
                      qo_tok, ko_tok)
        _check(ola_qk_norm(desc, qp, kp, _opt(wq, "wq", (d,), f32, ix),
                           _opt(wk, "wk", (d,), f32, ix),
                           _opt(positions, "positions", (R, P), torch.int32, ix),
                           _opt(inv_freq, "inv_freq", (half,), f32, ix), qo, ko, st),
               "ola_qk_norm")
    return q_out, k_out


def _scan_args(v, dt, A, k, q, D, dt_bias, z, out, softplus, ix, code):
    """Descriptor of a scan call and its pointers v, dt, A, k, q, D, dt_bias, z, y."""
    torch = _torch()
    f32 = torch.float32
    R, P, H, d_v = vs = v.shape
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be a tensor [R, P, G, d_k]")
    G, d_k = k.shape[2:]
    t, ks, hs = v.dtype, (R, P, G, d_k), (H,)
    vp, v_tok, v_seq = _rows(v, "v", vs, t, ix)
    kp, k_tok, k_seq = _rows(k, "k", ks, t, ix)
    qp, q_tok, q_seq = _rows(q, "q", ks, t, ix)
    zp, z_tok, z_seq = _opt_rows(z, "z", vs, t, ix)
    yp, y_tok, y_seq = _rows(out, "out", vs, t, ix)
    desc = ScanDesc(R, P, H, G, d_k, d_v, code, bool(softplus), v_tok, v_seq, k_tok, k_seq, q_tok,
                    q_seq, z_tok, z_seq, y_tok, y_seq)
    return desc, (vp, _ptr(dt, "dt", (R, P, H), f32, ix), _ptr(A, "A", hs, f32, ix), kp, qp,
                  _opt(D, "D", hs, f32, ix), _opt(dt_bias, "dt_bias", hs, f32, ix), zp), yp


_SCAN_WS = {}        # scratch bytes by shape and device (a pure function of them)


def scan(v, dt, A, k, q, *, D=None, dt_bias=None, z=None, S_in=None, lens=None, softplus=True,
         out=None, S_out=None, stream=None):
    """Selective state space scan of a prompt (ola_scan): v [R, P, H, d_v], k, q [R, P, G, d_k]
    (bf16 or fp32, may be column slices), dt [R, P, H] fp32, A [H] fp32 (negative), optional D,
    dt_bias [H] fp32, gate z like v, S_in [R, H, d_v, d_k] fp32, lens [R] int32.
    Returns (y [R, P, H, d_v], S_out [R, H, d_v, d_k]); rows of `out` behind a sequence's end are
    not written. S_out may be S_in. bf16 with 16-byte aligned rows and d_k <= 128 runs in chunks on
    tensor cores: y's token-to-token weights and the copy of the state that meets the queries are
    rounded to bf16 on the way (S_out is not). fp32 tensors keep everything in fp32."""
    torch = _torch()
    ix, code = _first(v, "v", 4)
    R, P, H, d_v = vs = v.shape
    with _scope(ix, stream) as st:
        if out is None:
            out = torch.empty(vs, device=v.device, dtype=v.dtype)
        desc, ptrs, yp = _scan_args(v, dt, A, k, q, D, dt_bias, z, out, softplus, ix, code)
        shape = (R, H, d_v, desc.d_k)
        if S_out is None:
            S_out = torch.empty(shape, device=v.device, dtype=torch.float32)
        key = (R, P, H, desc.d_k, d_v, code, ix)
        n = _SCAN_WS.get(key)
        if n is None:
            if len(_SCAN_WS) >= 4096:
                _SCAN_WS.clear()
            n = _SCAN_WS[key] = ola_scan_workspace_bytes(desc)
        ws = torch.empty((n,), device=v.device, dtype=torch.uint8) if n else None
        _check(ola_scan(desc, *ptrs, _opt(S_in, "S_in", shape, torch.float32, ix),
                        _opt(lens, "lens", (R,), torch.int32, ix), yp,
                        _ptr(S_out, "S_out", shape, torch.float32, ix),
                        ws.data_ptr() if n else None, n, st), "ola_scan")
    return out, S_out


def scan_step(v, dt, A, k, q, *, state, D=None, dt_bias=None, z=None, parent_idx=None,
              softplus=True, out=None, state_out=None, stream=None):
    """One token of every beam through the scan (ola_scan_step): v [R, B, H, d_v], k, q
    [R, B, G, d_k], dt [R, B, H], state [R, Bp, H, d_v, d_k] fp32, parent_idx [R, B] int32
    (default: beam b continues state b, or the only one). Returns (y [R, B, H, d_v], state_out
    [R, B, H, d_v, d_k]); state_out may be `state` when parent_idx is None. Every beam's state is
    materialised: its memory and traffic grow with the beams."""
    torch = _torch()
    ix, code = _first(v, "v", 4)
    R, B, H, d_v = vs = v.shape
    if not isinstance(state, torch.Tensor) or state.dim() != 5:
        raise ValueError("state must be a tensor [R, Bp, H, d_v, d_k]")
    Bp = state.shape[1]
    with _scope(ix, stream) as st:
        if out is None:
            out = torch.empty(vs, device=v.device, dtype=v.dtype)
        desc, ptrs, yp = _scan_args(v, dt, A, k, q, D, dt_bias, z, out, softplus, ix, code)
        if state_out is None:
            state_out = torch.empty((R, B, H, d_v, desc.d_k), device=v.device,
                                    dtype=torch.float32)
        _check(ola_scan_step(desc, Bp, *ptrs,
                             _ptr(state, "state", (R, Bp, H, d_v, desc.d_k), torch.float32, ix),
                             _opt(parent_idx, "parent_idx", (R, B), torch.int32, ix), yp,
                             _ptr(state_out, "state_out", (R, B, H, d_v, desc.d_k),
                                  torch.float32, ix), st), "ola_scan_step")
    return out, state_out
