"""Thin ctypes binding of libssd_b200.so (C ABI in include/ssd.h).

Argument marshalling only: every step of the SSD forward and of the decode
step runs in the library's CUDA kernels.  PyTorch is used for device memory
and streams.  There is no CPU fallback: if the library is missing, or a
tensor is not on a CUDA device, the call raises.

Function names match the C entry points.  Each call enqueues work on the
current torch CUDA stream (or the ``stream`` argument) and returns without
synchronising.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libssd_b200.so")

SSD_OK, SSD_ERR_INVALID_ARG, SSD_ERR_UNSUPPORTED, SSD_ERR_CUDA, SSD_ERR_TIMEOUT = 0, 1, 2, 3, 4
SSD_F32, SSD_BF16 = 0, 1

EXPORTED = ("ssd_status_string", "ssd_last_error_detail", "ssd_chunk_scan_fwd_workspace_size",
            "ssd_chunk_scan_fwd", "ssd_step", "ssd_chunk_state_fwd", "ssd_state_passing_fwd",
            "ssd_chunk_output_fwd", "ssd_chunk_scan_fwd_uses_tensor_cores",
            "ssd_chunk_scan_bwd_uses_tensor_cores",
            "ssd_chunk_scan_fwd_noalloc", "ssd_poll_device_status", "ssd_state_walk_fwd",
            "ssd_debug_expire_wait", "ssd_chunk_scan_bwd_workspace_size", "ssd_chunk_scan_bwd",
            "ssd_chunk_scan_fwd_data_flow", "ssd_seq_logdecay", "ssd_state_exchange_combine",
            "ssd_state_correction_workspace_size", "ssd_state_correction_fwd",
            "ssd_chunk_scan_fwd_flow_workspace_size", "ssd_chunk_scan_fwd_with_flow",
            "ssd_causal_conv_fwd", "ssd_causal_conv_bwd_workspace_size", "ssd_causal_conv_bwd",
            "ssd_causal_conv_step", "ssd_selective_scan_fwd_workspace_size",
            "ssd_selective_scan_fwd", "ssd_selective_scan_bwd_workspace_size",
            "ssd_selective_scan_bwd", "ssd_selective_step", "ssd_bc_norm_rotate_fwd",
            "ssd_bc_norm_rotate_bwd_workspace_size", "ssd_bc_norm_rotate_bwd")

# ssd_chunk_scan_fwd_data_flow results
SSD_FLOW_SIMT, SSD_FLOW_TC_THREE_KERNEL, SSD_FLOW_WALK_OUTPUT, SSD_FLOW_WALK_OUTPUT_FUSED = 0, 1, 2, 3


class SSDError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: {status_name(status)}: {detail}")
        self.status = status


class ssd_dims_t(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("nheads", ctypes.c_int64), ("headdim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64)]


class ssd_stride_t(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("token", ctypes.c_int64)]


class ssd_conv_dims_t(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("channels", ctypes.c_int64), ("width", ctypes.c_int64)]


class ssd_selective_dims_t(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("channels", ctypes.c_int64), ("dstate", ctypes.c_int64),
                ("ngroups", ctypes.c_int64)]


class ssd_selective_strides_t(ctypes.Structure):
    # the C struct's five ssd_stride_t, flat
    _fields_ = [(f"{k}_{s}", ctypes.c_int64) for k in ("x", "dt", "B", "C", "z")
                for s in ("batch", "token")]


class ssd_rotate_dims_t(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("ngroups", ctypes.c_int64), ("dstate", ctypes.c_int64),
                ("rotary", ctypes.c_int64)]


_lib = None
_vp = ctypes.c_void_p


def load(path: str = LIB_PATH):
    """Open the shared library (once).  Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m ssd_chunked_scan_02_b200.build` (no CPU fallback exists)")
    lib = ctypes.CDLL(path)
    dims_p = ctypes.POINTER(ssd_dims_t)
    lib.ssd_status_string.restype = ctypes.c_char_p
    lib.ssd_status_string.argtypes = [ctypes.c_int]
    lib.ssd_last_error_detail.restype = ctypes.c_char_p
    lib.ssd_last_error_detail.argtypes = []
    lib.ssd_chunk_scan_fwd_workspace_size.restype = ctypes.c_int
    lib.ssd_chunk_scan_fwd_workspace_size.argtypes = [dims_p, ctypes.c_int, ctypes.c_int,
                                                      ctypes.POINTER(ctypes.c_size_t)]
    lib.ssd_chunk_scan_fwd_uses_tensor_cores.restype = ctypes.c_int
    lib.ssd_chunk_scan_fwd_uses_tensor_cores.argtypes = [dims_p, ctypes.c_int, ctypes.c_int]
    lib.ssd_chunk_scan_bwd_uses_tensor_cores.restype = ctypes.c_int
    lib.ssd_chunk_scan_bwd_uses_tensor_cores.argtypes = [dims_p, ctypes.c_int]
    lib.ssd_chunk_scan_fwd_data_flow.restype = ctypes.c_int
    lib.ssd_chunk_scan_fwd_data_flow.argtypes = [dims_p, ctypes.c_int, ctypes.c_int]
    lib.ssd_chunk_scan_fwd.restype = ctypes.c_int
    lib.ssd_chunk_scan_fwd.argtypes = [_vp] * 6 + [ctypes.c_int, _vp, _vp, _vp, dims_p,
                                                   ctypes.c_int, _vp, ctypes.c_size_t, _vp]
    lib.ssd_chunk_scan_fwd_flow_workspace_size.restype = ctypes.c_int
    lib.ssd_chunk_scan_fwd_flow_workspace_size.argtypes = [dims_p, ctypes.c_int, ctypes.c_int,
                                                           ctypes.c_int,
                                                           ctypes.POINTER(ctypes.c_size_t)]
    lib.ssd_chunk_scan_fwd_with_flow.restype = ctypes.c_int
    lib.ssd_chunk_scan_fwd_with_flow.argtypes = lib.ssd_chunk_scan_fwd.argtypes + [ctypes.c_int]
    lib.ssd_chunk_scan_fwd_noalloc.restype = ctypes.c_int
    lib.ssd_chunk_scan_fwd_noalloc.argtypes = [_vp] * 6 + [ctypes.c_int, _vp, _vp, _vp, dims_p,
                                                           ctypes.c_int, _vp]
    lib.ssd_state_walk_fwd.restype = ctypes.c_int
    lib.ssd_state_walk_fwd.argtypes = [_vp] * 7 + [ctypes.c_int, dims_p, ctypes.c_int, _vp]
    lib.ssd_debug_expire_wait.restype = ctypes.c_int
    lib.ssd_debug_expire_wait.argtypes = [ctypes.c_uint, _vp]
    lib.ssd_poll_device_status.restype = ctypes.c_int
    lib.ssd_poll_device_status.argtypes = [_vp]
    lib.ssd_step.restype = ctypes.c_int
    lib.ssd_step.argtypes = [_vp] * 8 + [dims_p, ctypes.c_int, _vp]
    lib.ssd_chunk_state_fwd.restype = ctypes.c_int
    lib.ssd_chunk_state_fwd.argtypes = [_vp] * 4 + [ctypes.c_int, _vp, _vp, dims_p,
                                                    ctypes.c_int, _vp]
    lib.ssd_state_passing_fwd.restype = ctypes.c_int
    lib.ssd_state_passing_fwd.argtypes = [_vp] * 5 + [ctypes.c_int, dims_p, ctypes.c_int, _vp]
    lib.ssd_chunk_output_fwd.restype = ctypes.c_int
    lib.ssd_chunk_output_fwd.argtypes = [_vp] * 7 + [ctypes.c_int, _vp, dims_p, ctypes.c_int, _vp]
    lib.ssd_chunk_scan_bwd_workspace_size.restype = ctypes.c_int
    lib.ssd_chunk_scan_bwd_workspace_size.argtypes = [dims_p, ctypes.c_int,
                                                      ctypes.POINTER(ctypes.c_size_t)]
    lib.ssd_chunk_scan_bwd.restype = ctypes.c_int
    lib.ssd_chunk_scan_bwd.argtypes = [_vp] * 16 + [dims_p, ctypes.c_int, _vp, ctypes.c_size_t,
                                                    _vp]
    lib.ssd_seq_logdecay.restype = ctypes.c_int
    lib.ssd_seq_logdecay.argtypes = [_vp] * 3 + [dims_p, _vp]
    lib.ssd_state_exchange_combine.restype = ctypes.c_int
    lib.ssd_state_exchange_combine.argtypes = [_vp] * 3 + [ctypes.c_int, ctypes.c_int, _vp, dims_p,
                                                           _vp]
    lib.ssd_state_correction_workspace_size.restype = ctypes.c_int
    lib.ssd_state_correction_workspace_size.argtypes = [dims_p, ctypes.c_int,
                                                        ctypes.POINTER(ctypes.c_size_t)]
    lib.ssd_state_correction_fwd.restype = ctypes.c_int
    lib.ssd_state_correction_fwd.argtypes = [_vp] * 6 + [dims_p, ctypes.c_int, _vp,
                                                         ctypes.c_size_t, _vp]
    stride_p, conv_p = ctypes.POINTER(ssd_stride_t), ctypes.POINTER(ssd_conv_dims_t)
    size_p, ci, cs = ctypes.POINTER(ctypes.c_size_t), ctypes.c_int, ctypes.c_size_t
    _declare(lib, "ssd_causal_conv_fwd", _vp, stride_p, *[_vp] * 4, ci, _vp, _vp, conv_p, ci, _vp)
    _declare(lib, "ssd_causal_conv_bwd_workspace_size", conv_p, ci, size_p)
    _declare(lib, "ssd_causal_conv_bwd", _vp, stride_p, *[_vp] * 4, ci, _vp, ci, *[_vp] * 5, conv_p,
             ci, _vp, cs, _vp)
    _declare(lib, "ssd_causal_conv_step", _vp, _vp, stride_p, _vp, _vp, ci, _vp, conv_p, ci, _vp)
    sel_p, sst_p = ctypes.POINTER(ssd_selective_dims_t), ctypes.POINTER(ssd_selective_strides_t)
    for which in ("fwd", "bwd"):
        _declare(lib, f"ssd_selective_scan_{which}_workspace_size", sel_p, ci, size_p)
    _declare(lib, "ssd_selective_scan_fwd", *[_vp] * 8, ci, *[_vp] * 4, sst_p, sel_p, ci, _vp, cs,
             _vp)
    _declare(lib, "ssd_selective_scan_bwd", *[_vp] * 8, ci, *[_vp] * 13, sst_p, sel_p, ci, _vp, cs,
             _vp)
    _declare(lib, "ssd_selective_step", *[_vp] * 9, ci, _vp, sst_p, sel_p, ci, _vp)
    rot_p, rot = ctypes.POINTER(ssd_rotate_dims_t), [_vp, stride_p] * 2 + [_vp, _vp, ci, _vp, _vp,
                                                                           ctypes.c_float, ci]
    _declare(lib, "ssd_bc_norm_rotate_fwd", *rot, _vp, _vp, rot_p, ci, _vp)
    _declare(lib, "ssd_bc_norm_rotate_bwd_workspace_size", rot_p, ci, size_p)
    _declare(lib, "ssd_bc_norm_rotate_bwd", *rot, _vp, _vp, ci, *[_vp] * 4, rot_p, ci, _vp, cs, _vp)
    _lib = lib
    return lib


def _declare(lib, name, *argtypes):
    """One entry point that returns a status."""
    f = getattr(lib, name)
    f.restype = ctypes.c_int
    f.argtypes = list(argtypes)


def status_name(status: int) -> str:
    return load().ssd_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != SSD_OK:
        raise SSDError(status, where, load().ssd_last_error_detail().decode())


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return SSD_F32
    if t == torch.bfloat16:
        return SSD_BF16
    raise TypeError(f"unsupported element dtype {t} (float32 or bfloat16)")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device (there is no CPU path)")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream, device=None):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _device_of(t):
    """The CUDA device the call runs on: the main input's.  Calls are made
    with that device current (the library looks up its per-device state for
    the current device and rejects tensors of another one)."""
    if not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device (there is no CPU path)")
    return t.device


def _expect(name, t, shape, dtype, device):
    """Shape, dtype and device of one argument, checked before the C call (a
    wrong shape would otherwise become an out-of-bounds access)."""
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device} (the device of x)")


def _check_fwd_args(x, dt, A, B, C, D, init, y, final):
    """Shapes, dtypes and devices of the forward's arguments (against x and
    B), then that they are on a CUDA device.  Returns that device."""
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be (b, L, H, P) and B (b, L, G, N)")
    dev = x.device
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    f32 = torch.float32
    _expect("dt", dt, (b, L, H), f32, dev)
    _expect("A", A, (H,), f32, dev)
    _expect("D", D, (H,), f32, dev)
    _expect("B", B, (b, L, G, N), x.dtype, dev)
    _expect("C", C, (b, L, G, N), x.dtype, dev)
    _expect("init_states", init, (b, H, P, N), f32, dev)
    _expect("y", y, (b, L, H, P), x.dtype, dev)
    _expect("final_states", final, (b, H, P, N), f32, dev)
    return _device_of(x)


def make_dims(batch, seqlen, nheads, headdim, dstate, ngroups) -> ssd_dims_t:
    return ssd_dims_t(int(batch), int(seqlen), int(nheads), int(headdim), int(dstate),
                      int(ngroups))


def _fwd_dims(x, B) -> ssd_dims_t:
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    return make_dims(b, L, H, P, N, G)


def ssd_chunk_scan_fwd_workspace_size(dims: ssd_dims_t, chunk_size: int, dtype: torch.dtype,
                                      flow=None) -> int:
    n = ctypes.c_size_t(0)
    fl = -1 if flow is None else int(flow)
    _check(load().ssd_chunk_scan_fwd_flow_workspace_size(ctypes.byref(dims), int(chunk_size),
                                                         _dtype_code(dtype), fl, ctypes.byref(n)),
           "ssd_chunk_scan_fwd_workspace_size")
    return int(n.value)


def ssd_chunk_scan_fwd_uses_tensor_cores(dims: ssd_dims_t, chunk_size: int,
                                         dtype: torch.dtype) -> int:
    return int(load().ssd_chunk_scan_fwd_uses_tensor_cores(ctypes.byref(dims), int(chunk_size),
                                                           _dtype_code(dtype)))


def ssd_chunk_scan_fwd_data_flow(dims: ssd_dims_t, chunk_size: int, dtype: torch.dtype) -> int:
    """SSD_FLOW_WALK_OUTPUT_FUSED, SSD_FLOW_WALK_OUTPUT, SSD_FLOW_TC_THREE_KERNEL,
    SSD_FLOW_SIMT or -1 (rejected)."""
    return int(load().ssd_chunk_scan_fwd_data_flow(ctypes.byref(dims), int(chunk_size),
                                                   _dtype_code(dtype)))


def ssd_chunk_scan_fwd(x, dt, A, B, C, D, chunk_size: int, init_states=None,
                       return_final_states: bool = False, y=None, final_states=None,
                       workspace=None, stream=None, flow=None):
    """y (b,L,H,P) [, final_states (b,H,P,N) fp32] for the whole sequences.
    ``flow``: an SSD_FLOW_* value to force that data flow (None: the
    library's choice)."""
    dev = _check_fwd_args(x, dt, A, B, C, D, init_states, y, final_states)
    dims = _fwd_dims(x, B)
    if y is None:
        y = torch.empty_like(x)
    if return_final_states and final_states is None:
        final_states = torch.empty((x.shape[0], x.shape[2], x.shape[3], B.shape[3]),
                                   device=x.device, dtype=torch.float32)
    fl = -1 if flow is None else int(flow)
    need = ssd_chunk_scan_fwd_workspace_size(dims, chunk_size, x.dtype, flow=flow)
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=x.device, dtype=torch.uint8)
    with torch.cuda.device(dev):
        st = load().ssd_chunk_scan_fwd_with_flow(
            _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), int(chunk_size),
            _ptr(init_states), _ptr(y), _ptr(final_states), ctypes.byref(dims),
            _dtype_code(x.dtype), _ptr(workspace), workspace.numel(), _stream(stream, dev), fl)
    _check(st, "ssd_chunk_scan_fwd")
    return (y, final_states) if (return_final_states or final_states is not None) else y


def ssd_chunk_scan_fwd_noalloc(x, dt, A, B, C, D, chunk_size: int, init_states=None,
                               return_final_states: bool = False, y=None, final_states=None,
                               stream=None):
    """ssd_chunk_scan_fwd without a caller workspace: the library's built-in
    scratch array (SSD_NOALLOC_SCRATCH_BYTES) is used instead.  For callers
    that cannot allocate device memory; calls that overlap on the GPU race on
    that array."""
    dev = _check_fwd_args(x, dt, A, B, C, D, init_states, y, final_states)
    dims = _fwd_dims(x, B)
    if y is None:
        y = torch.empty_like(x)
    if return_final_states and final_states is None:
        final_states = torch.empty((x.shape[0], x.shape[2], x.shape[3], B.shape[3]),
                                   device=x.device, dtype=torch.float32)
    with torch.cuda.device(dev):
        st = load().ssd_chunk_scan_fwd_noalloc(_ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C),
                                               _ptr(D), int(chunk_size), _ptr(init_states),
                                               _ptr(y), _ptr(final_states), ctypes.byref(dims),
                                               _dtype_code(x.dtype), _stream(stream, dev))
    _check(st, "ssd_chunk_scan_fwd_noalloc")
    return (y, final_states) if (return_final_states or final_states is not None) else y


NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


def ssd_step(state, x, dt, A, B, C, D, y=None, stream=None):
    """One decode step; ``state`` (b,H,P,N) fp32 is updated in place.  Returns y (b,H,P)."""
    b, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    dev = x.device
    f32 = torch.float32
    _expect("state", state, (b, H, P, N), f32, dev)
    _expect("dt", dt, (b, H), f32, dev)
    _expect("A", A, (H,), f32, dev)
    _expect("D", D, (H,), f32, dev)
    _expect("B", B, (b, G, N), x.dtype, dev)
    _expect("C", C, (b, G, N), x.dtype, dev)
    _expect("y", y, (b, H, P), x.dtype, dev)
    dev = _device_of(x)
    dims = make_dims(b, 1, H, P, N, G)
    if y is None:
        y = torch.empty_like(x)
    with torch.cuda.device(dev):
        st = load().ssd_step(_ptr(state), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                             _ptr(y), ctypes.byref(dims), _dtype_code(x.dtype),
                             _stream(stream, dev))
    _check(st, "ssd_step")
    return y


def ssd_poll_device_status(stream=None):
    """Raise SSDError(SSD_ERR_TIMEOUT) if a bounded device-side wait gave up
    since the last poll (synchronises the stream)."""
    _check(load().ssd_poll_device_status(_stream(stream)), "ssd_poll_device_status")


def ssd_debug_expire_wait(polls: int = 4096, stream=None):
    """Launch the bounded-wait failure probe (see include/ssd.h)."""
    _check(load().ssd_debug_expire_wait(int(polls), _stream(stream)), "ssd_debug_expire_wait")


def n_chunks(seqlen: int, chunk_size: int) -> int:
    return (int(seqlen) + int(chunk_size) - 1) // int(chunk_size)


def ssd_chunk_state_fwd(x, dt, A, B, chunk_size: int, stream=None):
    """Step (2): per-chunk zero-start states (b,T,H,P,N) fp32 and log-decays (b,T,H)."""
    dims = _fwd_dims(x, B)
    b, L, H, P = x.shape
    T = n_chunks(L, chunk_size)
    dev = _check_fwd_args(x, dt, A, B, None, None, None, None, None)
    states = torch.empty((b, T, H, P, B.shape[3]), device=x.device, dtype=torch.float32)
    logdecay = torch.empty((b, T, H), device=x.device, dtype=torch.float32)
    with torch.cuda.device(dev):
        st = load().ssd_chunk_state_fwd(_ptr(x), _ptr(dt), _ptr(A), _ptr(B), int(chunk_size),
                                        _ptr(states), _ptr(logdecay), ctypes.byref(dims),
                                        _dtype_code(x.dtype), _stream(stream, dev))
    _check(st, "ssd_chunk_state_fwd")
    return states, logdecay


def ssd_state_passing_fwd(chunk_states, chunk_logdecay, chunk_size: int, seqlen: int,
                          dtype: torch.dtype, init_states=None, want_final: bool = True,
                          stream=None):
    """Step (3): states entering each chunk (b,T,H,P,N) in ``dtype`` and the final state."""
    b, T, H, P, N = chunk_states.shape
    dims = make_dims(b, seqlen, H, P, N, 1)
    dev = _device_of(chunk_states)
    _expect("chunk_states", chunk_states, (b, T, H, P, N), torch.float32, dev)
    _expect("chunk_logdecay", chunk_logdecay, (b, T, H), torch.float32, dev)
    _expect("init_states", init_states, (b, H, P, N), torch.float32, dev)
    if n_chunks(seqlen, chunk_size) != T:
        raise ValueError(f"chunk_states has {T} chunks; seqlen {seqlen} / chunk {chunk_size} "
                         f"gives {n_chunks(seqlen, chunk_size)}")
    prev = torch.empty((b, T, H, P, N), device=chunk_states.device, dtype=dtype)
    final = (torch.empty((b, H, P, N), device=chunk_states.device, dtype=torch.float32)
             if want_final else None)
    with torch.cuda.device(dev):
        st = load().ssd_state_passing_fwd(_ptr(chunk_states), _ptr(chunk_logdecay),
                                          _ptr(init_states), _ptr(prev), _ptr(final),
                                          int(chunk_size), ctypes.byref(dims),
                                          _dtype_code(dtype), _stream(stream, dev))
    _check(st, "ssd_state_passing_fwd")
    return prev, final


def ssd_state_walk_fwd(x, dt, A, B, chunk_size: int, init_states=None, want_final: bool = True,
                       stream=None):
    """Steps (2) + (3) fused (the on-chip state walk): entering states
    (b,T,H,P,N) bf16 and the final state (b,H,P,N) fp32."""
    dims = _fwd_dims(x, B)
    b, L, H, P = x.shape
    N = B.shape[3]
    T = n_chunks(L, chunk_size)
    dev = _check_fwd_args(x, dt, A, B, None, None, init_states, None, None)
    prev = torch.empty((b, T, H, P, N), device=x.device, dtype=torch.bfloat16)
    final = torch.empty((b, H, P, N), device=x.device, dtype=torch.float32) if want_final else None
    with torch.cuda.device(dev):
        st = load().ssd_state_walk_fwd(_ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(init_states),
                                       _ptr(prev), _ptr(final), int(chunk_size),
                                       ctypes.byref(dims), _dtype_code(x.dtype),
                                       _stream(stream, dev))
    _check(st, "ssd_state_walk_fwd")
    return prev, final


def ssd_chunk_output_fwd(x, dt, A, B, C, D, prev_states, chunk_size: int, y=None, stream=None):
    """Steps (1) and (4): y from the inputs and the states entering each chunk."""
    dev = _check_fwd_args(x, dt, A, B, C, D, None, y, None)
    b, L, H, P = x.shape
    _expect("prev_states", prev_states, (b, n_chunks(L, chunk_size), H, P, B.shape[3]), x.dtype,
            dev)
    dims = _fwd_dims(x, B)
    if y is None:
        y = torch.empty_like(x)
    with torch.cuda.device(dev):
        st = load().ssd_chunk_output_fwd(_ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                         _ptr(prev_states), int(chunk_size), _ptr(y),
                                         ctypes.byref(dims), _dtype_code(x.dtype),
                                         _stream(stream, dev))
    _check(st, "ssd_chunk_output_fwd")
    return y


def ssd_chunk_scan_bwd_uses_tensor_cores(dims: ssd_dims_t, dtype: torch.dtype) -> int:
    """1: the backward runs on the tcgen05 tensor cores; 0: exact fp32 on the
    CUDA cores; -1: these sizes are rejected."""
    return int(load().ssd_chunk_scan_bwd_uses_tensor_cores(ctypes.byref(dims), _dtype_code(dtype)))


def ssd_chunk_scan_bwd_workspace_size(dims: ssd_dims_t, dtype: torch.dtype) -> int:
    n = ctypes.c_size_t(0)
    _check(load().ssd_chunk_scan_bwd_workspace_size(ctypes.byref(dims), _dtype_code(dtype),
                                                    ctypes.byref(n)),
           "ssd_chunk_scan_bwd_workspace_size")
    return int(n.value)


def ssd_chunk_scan_bwd(x, dt, A, B, C, D, dy, init_states=None, dfinal_states=None,
                       want_dinit: bool = True, workspace=None, stream=None):
    """Gradients of ssd_chunk_scan_fwd for dL/dy = dy (b,L,H,P, x's dtype) and
    dL/dfinal_states = dfinal_states ((b,H,P,N) fp32 or None).  Returns a dict
    of fp32 tensors: dx, ddt, dA, dB, dC, dD and (if want_dinit) dinit."""
    dev = _check_fwd_args(x, dt, A, B, C, D, init_states, None, dfinal_states)
    _expect("dy", dy, tuple(x.shape), x.dtype, dev)
    dims = _fwd_dims(x, B)
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    f32 = dict(device=x.device, dtype=torch.float32)
    out = {"dx": torch.empty((b, L, H, P), **f32), "ddt": torch.empty((b, L, H), **f32),
           "dA": torch.empty((H,), **f32), "dB": torch.empty((b, L, G, N), **f32),
           "dC": torch.empty((b, L, G, N), **f32), "dD": torch.empty((H,), **f32),
           "dinit": torch.empty((b, H, P, N), **f32) if want_dinit else None}
    need = ssd_chunk_scan_bwd_workspace_size(dims, x.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=x.device, dtype=torch.uint8)
    with torch.cuda.device(dev):
        st = load().ssd_chunk_scan_bwd(_ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                       _ptr(init_states), _ptr(dy), _ptr(dfinal_states),
                                       _ptr(out["dx"]), _ptr(out["ddt"]), _ptr(out["dA"]),
                                       _ptr(out["dB"]), _ptr(out["dC"]), _ptr(out["dD"]),
                                       _ptr(out["dinit"]), ctypes.byref(dims),
                                       _dtype_code(x.dtype), _ptr(workspace), workspace.numel(),
                                       _stream(stream, dev))
    _check(st, "ssd_chunk_scan_bwd")
    return out


# ---------------------------------------------------------------- sequence parallelism
def ssd_seq_logdecay(dt, A, stream=None):
    """sum_t dt[b,t,h] * A[h] over the (shard's) sequence: (b, H) fp32."""
    b, L, H = dt.shape
    _expect("dt", dt, (b, L, H), torch.float32, dt.device)
    _expect("A", A, (H,), torch.float32, dt.device)
    dev = _device_of(dt)
    out = torch.empty((b, H), device=dt.device, dtype=torch.float32)
    dims = make_dims(b, L, H, 1, 1, 1)
    with torch.cuda.device(dev):
        st = load().ssd_seq_logdecay(_ptr(dt), _ptr(A), _ptr(out), ctypes.byref(dims),
                                     _stream(stream, dev))
    _check(st, "ssd_seq_logdecay")
    return out


def ssd_state_exchange_combine(local_final, logdecay, rank: int, init_states=None, out=None,
                               stream=None):
    """The state entering rank ``rank``'s shard from the gathered local final
    states (R,b,H,P,N) and log-decays (R,b,H) of all ranks (rank order) and
    the state entering the whole sequence (None = zero).  rank = R gives the
    state after the whole sequence."""
    R, b, H, P, N = local_final.shape
    dev = local_final.device
    _expect("logdecay", logdecay, (R, b, H), torch.float32, dev)
    _expect("local_final", local_final, (R, b, H, P, N), torch.float32, dev)
    _expect("init_states", init_states, (b, H, P, N), torch.float32, dev)
    _expect("out", out, (b, H, P, N), torch.float32, dev)
    dev = _device_of(local_final)
    if out is None:
        out = torch.empty((b, H, P, N), device=local_final.device, dtype=torch.float32)
    dims = make_dims(b, 0, H, P, N, 1)
    with torch.cuda.device(dev):
        st = load().ssd_state_exchange_combine(_ptr(local_final), _ptr(logdecay), _ptr(init_states),
                                               int(rank), int(R), _ptr(out), ctypes.byref(dims),
                                               _stream(stream, dev))
    _check(st, "ssd_state_exchange_combine")
    return out


def ssd_state_correction_workspace_size(dims: ssd_dims_t, dtype: torch.dtype) -> int:
    n = ctypes.c_size_t(0)
    _check(load().ssd_state_correction_workspace_size(ctypes.byref(dims), _dtype_code(dtype),
                                                      ctypes.byref(n)),
           "ssd_state_correction_workspace_size")
    return int(n.value)


def ssd_state_correction_fwd(h_in, dt, A, C, y, final_states=None, workspace=None, stream=None):
    """In place: y_t += exp(cs_t) h_in C_t over the shard and, if given,
    final_states += exp(cs_last) h_in.  h_in (b,H,P,N) fp32."""
    b, L, H, P = y.shape
    G, N = C.shape[2], C.shape[3]
    dev = y.device
    _expect("h_in", h_in, (b, H, P, N), torch.float32, dev)
    _expect("dt", dt, (b, L, H), torch.float32, dev)
    _expect("A", A, (H,), torch.float32, dev)
    _expect("C", C, (b, L, G, N), y.dtype, dev)
    _expect("final_states", final_states, (b, H, P, N), torch.float32, dev)
    dev = _device_of(y)
    dims = make_dims(b, L, H, P, N, G)
    need = ssd_state_correction_workspace_size(dims, y.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=y.device, dtype=torch.uint8)
    with torch.cuda.device(dev):
        st = load().ssd_state_correction_fwd(_ptr(h_in), _ptr(dt), _ptr(A), _ptr(C), _ptr(y),
                                             _ptr(final_states), ctypes.byref(dims),
                                             _dtype_code(y.dtype), _ptr(workspace),
                                             workspace.numel(), _stream(stream, dev))
    _check(st, "ssd_state_correction_fwd")
    return y


# ---------------------------------------------------------------- operators around the layer
class _scope:
    """Makes the call's device, and the stream it is asked to run on, current,
    so that what the call allocates belongs to the stream that uses it.  Nothing
    is entered where they are current already (the raw handle is asked for
    directly: a single-token call takes less time than a stream object)."""
    __slots__ = ("index", "entered")

    def __init__(self, device, stream):
        self.index, self.entered = device.index, ()
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                stream = (torch.cuda.ExternalStream(int(stream), device=device) if int(stream)
                          else torch.cuda.default_stream(device))
            if stream.device != device:
                raise ValueError(f"stream: on {stream.device}, expected {device} (the device of x)")
            self.entered = (torch.cuda.stream(stream),)
        elif device.index != torch._C._cuda_getDevice():
            self.entered = (torch.cuda.device(device),)

    def __enter__(self):
        for c in self.entered:
            c.__enter__()
        return torch._C._cuda_getCurrentRawStream(self.index)

    def __exit__(self, *exc):
        for c in self.entered:
            c.__exit__(*exc)


def _dense(name, t, shape, dtype, device):
    """A dense argument (or None): checked, then its address."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype or t.device != device:
        _expect(name, t, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _view(name, t, shape, dtype, device, lead=2):
    """An argument that may be a view of a wider tensor: checked, then its
    address and its strides (batch, token; with lead 1 the batch's alone, and 0).
    The dimensions behind those have to be contiguous."""
    if t is None:
        return None, 0, 0
    if t.shape != shape or t.dtype != dtype or t.device != device:
        _expect(name, t, shape, dtype, device)
    strides = t.stride()
    if not t.is_contiguous():
        run = 1
        for i in range(len(shape) - 1, lead - 1, -1):
            if shape[i] != 1 and strides[i] != run:
                raise ValueError(f"{name}: its last {len(shape) - lead} dimension(s) must be "
                                 "contiguous")
            run *= shape[i]
    return t.data_ptr(), strides[0], strides[1] if lead == 2 else 0


def _out_like(t):
    """A dense output of t's shape (the cheapest way to ask for one)."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _workspace(workspace, need, like):
    """The caller's workspace, or one of ``need`` bytes on the device of ``like``."""
    device = like.device
    if workspace is None:
        workspace = like.new_empty(max(need, 16), dtype=torch.uint8)
    elif not workspace.is_contiguous() or workspace.device != device:
        raise ValueError(f"workspace: must be contiguous and on {device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _conv_dims(x, weight):
    if x.dim() != 3 or weight.dim() != 2:
        raise ValueError("x must be (b, L, D) and weight (D, W)")
    b, L, D = x.shape
    return b, L, D, weight.shape[1], ssd_conv_dims_t(b, L, D, weight.shape[1])


def ssd_causal_conv_fwd(x, weight, bias=None, init_state=None, seq_lens=None, silu: bool = True,
                        return_final_state: bool = False, y=None, final_state=None, stream=None):
    """Causal depthwise convolution of x (b,L,D; may be a view with strided
    tokens) by weight (D,W) and bias (D), then (``silu``) the SiLU activation.
    init_state (b,W-1,D): the inputs before token 0, oldest first (None: zero).
    seq_lens (b,) int32: the sequences' own lengths in a padded batch; rows of y
    behind them are zero.  Returns y [, final_state (b,W-1,D): the last inputs]."""
    b, L, D, W, dims = _conv_dims(x, weight)
    dev, T, f32 = x.device, x.dtype, torch.float32
    code = _dtype_code(T)
    px, *sx = _view("x", x, (b, L, D), T, dev)
    sx = ssd_stride_t(*sx)
    pw = _dense("weight", weight, (D, W), f32, dev)
    pb = _dense("bias", bias, (D,), f32, dev)
    pi = _dense("init_state", init_state, (b, W - 1, D), T, dev)
    pl = _dense("seq_lens", seq_lens, (b,), torch.int32, dev)
    py = _dense("y", y, (b, L, D), T, dev)
    pf = _dense("final_state", final_state, (b, W - 1, D), T, dev)
    with _scope(_device_of(x), stream) as st:
        if y is None:
            y = _out_like(x)
            py = y.data_ptr()
        if return_final_state and final_state is None:
            final_state = x.new_empty((b, W - 1, D))
            pf = final_state.data_ptr()
        _check(load().ssd_causal_conv_fwd(px, sx, pw, pb, pi, pl, int(silu), py, pf, dims, code, st),
               "ssd_causal_conv_fwd")
    return (y, final_state) if final_state is not None else y


def ssd_causal_conv_bwd_workspace_size(dims: ssd_conv_dims_t, dtype: torch.dtype) -> int:
    n = ctypes.c_size_t(0)
    _check(load().ssd_causal_conv_bwd_workspace_size(dims, _dtype_code(dtype), n),
           "ssd_causal_conv_bwd_workspace_size")
    return int(n.value)


def ssd_causal_conv_bwd(x, weight, bias, dy, init_state=None, dfinal_state=None, seq_lens=None,
                        silu: bool = True, want_dinit: bool = True, workspace=None, stream=None):
    """Gradients of ssd_causal_conv_fwd for dL/dy = dy ((b,L,D), x's dtype or
    fp32) and dL/dfinal_state (None: zero).  Returns a dict: dx and (if
    want_dinit) dinit in x's dtype, dweight and dbias fp32."""
    b, L, D, W, dims = _conv_dims(x, weight)
    dev, T, f32 = x.device, x.dtype, torch.float32
    code = _dtype_code(T)
    px, *sx = _view("x", x, (b, L, D), T, dev)
    sx = ssd_stride_t(*sx)
    pw = _dense("weight", weight, (D, W), f32, dev)
    pb = _dense("bias", bias, (D,), f32, dev)
    pi = _dense("init_state", init_state, (b, W - 1, D), T, dev)
    pl = _dense("seq_lens", seq_lens, (b,), torch.int32, dev)
    pdy = _dense("dy", dy, (b, L, D), f32 if dy.dtype == f32 else T, dev)
    pdf = _dense("dfinal_state", dfinal_state, (b, W - 1, D), T, dev)
    with _scope(_device_of(x), stream) as st:
        out = {"dx": _out_like(x), "dweight": weight.new_empty((D, W)),
               "dbias": weight.new_empty((D,)),
               "dinit": x.new_empty((b, W - 1, D)) if want_dinit else None}
        workspace, pws, nws = _workspace(workspace, ssd_causal_conv_bwd_workspace_size(dims, T), x)
        _check(load().ssd_causal_conv_bwd(
            px, sx, pw, pb, pi, pl, int(silu), pdy, int(dy.dtype == f32), pdf,
            out["dx"].data_ptr(), out["dweight"].data_ptr(), out["dbias"].data_ptr(),
            out["dinit"].data_ptr() if want_dinit else None, dims, code, pws, nws, st),
            "ssd_causal_conv_bwd")
    return out


def ssd_causal_conv_step(state, x, weight, bias=None, silu: bool = True, y=None, stream=None):
    """One token: ``state`` (b,W-1,D), the last inputs, is updated in place;
    x (b,D).  Returns y (b,D)."""
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x must be (b, D) and weight (D, W)")
    b, D = x.shape
    W = weight.shape[1]
    dev, T, f32 = x.device, x.dtype, torch.float32
    code = _dtype_code(T)
    px, *sx = _view("x", x, (b, D), T, dev, 1)
    sx = ssd_stride_t(*sx)
    ps = _dense("state", state, (b, W - 1, D), T, dev)
    pw = _dense("weight", weight, (D, W), f32, dev)
    pb = _dense("bias", bias, (D,), f32, dev)
    py = _dense("y", y, (b, D), T, dev)
    with _scope(_device_of(x), stream) as st:
        if y is None:
            y = _out_like(x)
            py = y.data_ptr()
        _check(load().ssd_causal_conv_step(ps, px, sx, pw, pb, int(silu), py,
                                           ssd_conv_dims_t(b, 1, D, W), code, st),
               "ssd_causal_conv_step")
    return y


def _selective_args(x, dt, A, B, C, D, z, dt_bias, softplus, tokens=True):
    """Checks the inputs that the selective scan's calls share; returns their C
    arguments, strides, dims, device and dtype code."""
    lead = 2 if tokens else 1
    if x.dim() != lead + 1 or B.dim() != lead + 2 or A.dim() != 2:
        raise ValueError("x must be (b, L, D), B (b, L, G, N) and A (D, N)" if tokens else
                         "x must be (b, D), B (b, G, N) and A (D, N)")
    shape, bc = tuple(x.shape), tuple(B.shape)
    b, ch, G, N = shape[0], shape[-1], bc[-2], bc[-1]
    L = shape[1] if tokens else 1
    dev, T, f32 = x.device, x.dtype, torch.float32
    code = _dtype_code(T)
    bc = shape[:lead] + (G, N)
    px, x0, x1 = _view("x", x, shape, T, dev, lead)
    pdt, t0, t1 = _view("dt", dt, shape, T, dev, lead)
    pB, B0, B1 = _view("B", B, bc, T, dev, lead)
    pC, C0, C1 = _view("C", C, bc, T, dev, lead)
    pz, z0, z1 = _view("z", z, shape, T, dev, lead)
    args = (px, pdt, _dense("A", A, (ch, N), f32, dev), pB, pC, _dense("D", D, (ch,), f32, dev), pz,
            _dense("dt_bias", dt_bias, (ch,), f32, dev), int(softplus))
    return (args, ssd_selective_strides_t(x0, x1, t0, t1, B0, B1, C0, C1, z0, z1),
            ssd_selective_dims_t(b, L, ch, N, G), dev, code)


def ssd_selective_scan_fwd_workspace_size(dims: ssd_selective_dims_t, dtype: torch.dtype) -> int:
    n = ctypes.c_size_t(0)
    _check(load().ssd_selective_scan_fwd_workspace_size(dims, _dtype_code(dtype), n),
           "ssd_selective_scan_fwd_workspace_size")
    return int(n.value)


def ssd_selective_scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus: bool = True,
                           init_states=None, seq_lens=None, return_final_states: bool = False,
                           y=None, final_states=None, workspace=None, stream=None):
    """Selective scan with a decay per (channel, state): x, dt and the gate z
    (b,L,D), B, C (b,L,G,N), all of one dtype and each possibly a view with
    strided tokens; A (D,N), D and dt_bias (D) fp32.  dt is
    softplus(dt + dt_bias), or dt + dt_bias without ``softplus``.  seq_lens (b,)
    int32: the sequences' own lengths in a padded batch; rows of y behind them
    are zero.  Returns y (b,L,D) [, final_states (b,D,N) fp32]."""
    args, strides, dims, dev, code = _selective_args(x, dt, A, B, C, D, z, dt_bias, softplus)
    b, L, ch = x.shape
    N, T, f32 = A.shape[1], x.dtype, torch.float32
    pi = _dense("init_states", init_states, (b, ch, N), f32, dev)
    pl = _dense("seq_lens", seq_lens, (b,), torch.int32, dev)
    py = _dense("y", y, (b, L, ch), T, dev)
    pf = _dense("final_states", final_states, (b, ch, N), f32, dev)
    with _scope(_device_of(x), stream) as st:
        if y is None:
            y = _out_like(x)
            py = y.data_ptr()
        if return_final_states and final_states is None:
            final_states = A.new_empty((b, ch, N))
            pf = final_states.data_ptr()
        need = ssd_selective_scan_fwd_workspace_size(dims, T)
        pws, nws = None, 0
        if need or workspace is not None:
            workspace, pws, nws = _workspace(workspace, need, x)
        _check(load().ssd_selective_scan_fwd(*args, pi, pl, py, pf, strides, dims, code, pws, nws,
                                             st), "ssd_selective_scan_fwd")
    return (y, final_states) if final_states is not None else y


def ssd_selective_scan_bwd_workspace_size(dims: ssd_selective_dims_t, dtype: torch.dtype) -> int:
    n = ctypes.c_size_t(0)
    _check(load().ssd_selective_scan_bwd_workspace_size(dims, _dtype_code(dtype), n),
           "ssd_selective_scan_bwd_workspace_size")
    return int(n.value)


def ssd_selective_scan_bwd(x, dt, A, B, C, D, dy, z=None, dt_bias=None, softplus: bool = True,
                           init_states=None, dfinal_states=None, seq_lens=None,
                           want_dinit: bool = True, workspace=None, stream=None):
    """Gradients of ssd_selective_scan_fwd for dL/dy = dy (b,L,D; x's dtype) and
    dL/dfinal_states ((b,D,N) fp32 or None).  Returns a dict: dx, ddt, dB, dC and
    dz in x's dtype, dA, dD, ddt_bias and dinit fp32; None for an input that
    was None (and for dinit without want_dinit)."""
    args, strides, dims, dev, code = _selective_args(x, dt, A, B, C, D, z, dt_bias, softplus)
    b, L, ch = x.shape
    N, T, f32 = A.shape[1], x.dtype, torch.float32
    pi = _dense("init_states", init_states, (b, ch, N), f32, dev)
    pl = _dense("seq_lens", seq_lens, (b,), torch.int32, dev)
    pdy = _dense("dy", dy, (b, L, ch), T, dev)
    pdf = _dense("dfinal_states", dfinal_states, (b, ch, N), f32, dev)
    with _scope(_device_of(x), stream) as st:
        new, par = x.new_empty, A.new_empty
        out = {"dx": new(x.shape), "ddt": new(x.shape), "dA": par(A.shape), "dB": new(B.shape),
               "dC": new(C.shape), "dD": par((ch,)) if D is not None else None,
               "dz": new(x.shape) if z is not None else None,
               "ddt_bias": par((ch,)) if dt_bias is not None else None,
               "dinit": par((b, ch, N)) if want_dinit else None}
        workspace, pws, nws = _workspace(workspace,
                                         ssd_selective_scan_bwd_workspace_size(dims, T), x)
        _check(load().ssd_selective_scan_bwd(*args, pi, pl, pdy, pdf,
                                             *(None if v is None else v.data_ptr()
                                               for v in out.values()),
                                             strides, dims, code, pws, nws, st),
               "ssd_selective_scan_bwd")
    return out


def ssd_selective_step(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus: bool = True,
                       y=None, stream=None):
    """One token: ``state`` (b,D,N) fp32 is updated in place; x, dt, z (b,D), B, C
    (b,G,N).  Returns y (b,D)."""
    args, strides, dims, dev, code = _selective_args(x, dt, A, B, C, D, z, dt_bias, softplus,
                                                     tokens=False)
    b, ch = x.shape
    ps = _dense("state", state, (b, ch, A.shape[1]), torch.float32, dev)
    py = _dense("y", y, (b, ch), x.dtype, dev)
    with _scope(_device_of(x), stream) as st:
        if y is None:
            y = _out_like(x)
            py = y.data_ptr()
        _check(load().ssd_selective_step(ps, *args, py, strides, dims, code, st),
               "ssd_selective_step")
    return y


def _rotate_args(B, C, B_weight, C_weight, positions, freq, eps, interleaved):
    """Checks the inputs that ssd_bc_norm_rotate_fwd and _bwd share; returns
    their C arguments, the dims, the device and the weights' shape."""
    if B.dim() != 4 or freq.dim() != 1:
        raise ValueError("B and C must be (b, L, G, N) and freq (R / 2)")
    b, L, G, N = B.shape
    dev, T, f32 = B.device, B.dtype, torch.float32
    code = _dtype_code(T)
    pB, *sB = _view("B", B, (b, L, G, N), T, dev)
    pC, *sC = _view("C", C, (b, L, G, N), T, dev)
    per_group = B_weight.dim() == 2
    shape = (G, N) if per_group else (N,)
    args = (pB, ssd_stride_t(*sB), pC, ssd_stride_t(*sC), _dense("B_weight", B_weight, shape, f32, dev),
            _dense("C_weight", C_weight, shape, f32, dev), int(per_group),
            _dense("positions", positions, (b, L), torch.int64, dev),
            _dense("freq", freq, (freq.shape[0],), f32, dev), float(eps), int(interleaved))
    return args, ssd_rotate_dims_t(b, L, G, N, 2 * freq.shape[0]), dev, code, shape


def ssd_bc_norm_rotate_fwd(B, C, B_weight, C_weight, positions, freq, eps: float = 1e-5,
                           interleaved: bool = False, B_out=None, C_out=None, stream=None):
    """Each row (one group of one token) of B and of C (b,L,G,N; may be views with
    strided tokens) divided by its root mean square, multiplied by the weight ((N)
    or (G,N)), and its first 2 * len(freq) elements turned in pairs by
    positions (b,L, int64) * freq.  Returns dense B, C for ssd_chunk_scan_fwd or
    (at L = 1) ssd_step."""
    args, dims, dev, code, _ = _rotate_args(B, C, B_weight, C_weight, positions, freq, eps,
                                            interleaved)
    oB = _dense("B_out", B_out, tuple(B.shape), B.dtype, dev)
    oC = _dense("C_out", C_out, tuple(B.shape), B.dtype, dev)
    with _scope(_device_of(B), stream) as st:
        if B_out is None:
            B_out = _out_like(B)
            oB = B_out.data_ptr()
        if C_out is None:
            C_out = _out_like(B)
            oC = C_out.data_ptr()
        _check(load().ssd_bc_norm_rotate_fwd(*args, oB, oC, dims, code, st),
               "ssd_bc_norm_rotate_fwd")
    return B_out, C_out


def ssd_bc_norm_rotate_bwd_workspace_size(dims: ssd_rotate_dims_t, dtype: torch.dtype) -> int:
    n = ctypes.c_size_t(0)
    _check(load().ssd_bc_norm_rotate_bwd_workspace_size(dims, _dtype_code(dtype), n),
           "ssd_bc_norm_rotate_bwd_workspace_size")
    return int(n.value)


def ssd_bc_norm_rotate_bwd(B, C, B_weight, C_weight, positions, freq, dB_out, dC_out,
                           eps: float = 1e-5, interleaved: bool = False, workspace=None,
                           stream=None):
    """Gradients of ssd_bc_norm_rotate_fwd for dL/d its outputs (b,L,G,N), in B's
    dtype or fp32.  Returns a dict: dB, dC in B's dtype, dwB, dwC fp32 (of the
    weights' shape)."""
    args, dims, dev, code, shape = _rotate_args(B, C, B_weight, C_weight, positions, freq, eps,
                                                interleaved)
    f32 = torch.float32
    gt = f32 if dB_out.dtype == f32 else B.dtype
    gB = _dense("dB_out", dB_out, tuple(B.shape), gt, dev)
    gC = _dense("dC_out", dC_out, tuple(B.shape), gt, dev)
    with _scope(_device_of(B), stream) as st:
        out = {"dB": _out_like(B), "dC": _out_like(B),
               "dwB": B_weight.new_empty(shape), "dwC": B_weight.new_empty(shape)}
        workspace, pws, nws = _workspace(workspace,
                                         ssd_bc_norm_rotate_bwd_workspace_size(dims, B.dtype), B)
        _check(load().ssd_bc_norm_rotate_bwd(*args, gB, gC, int(gt == f32),
                                             *(v.data_ptr() for v in out.values()), dims, code,
                                             pws, nws, st), "ssd_bc_norm_rotate_bwd")
    return out
