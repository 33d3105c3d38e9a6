"""MI355X (gfx950) selective-scan forward (S6): a thin Python binding over libselscan.so.

Every step of the computation runs in the HIP kernels of ``csrc/``; this module only
marshals torch tensors (device memory) and the current HIP stream into the C ABI declared
in ``include/selscan.h``, and raises on a non-zero status.  There is no fallback: if the
library is not built, importing the binding's functions raises.

    y, last = selective_scan_fwd(u, delta, A, B, C, Dskip, z, return_last_state=True)

Shapes (torch tensors on the current GPU):
    u, z           [batch, L, D]        float32 or bfloat16 (same dtype for u, delta, B, C, z)
    delta          [batch, L, D]        (selective) or [D] (time-invariant)
    A              [D, N] float32
    B, C           [batch, L, N]        (selective) or [D, N] (time-invariant)
    Dskip          [D] float32 or None
Options: ``discretization="euler"`` (Bbar = delta * B instead of the ZOH coefficient),
``delta_softplus=True`` and ``delta_bias`` ([D] float32): the step size is
softplus(delta + delta_bias) (the bias alone is added without softplus).
The innermost axis of every tensor must be unit-stride; other strides are passed through
(zero strides, i.e. expanded views, are allowed).

Linear attention with a decay for each head, and the output stage of such a layer:

    o, last = linear_attention_fwd(q, k, v, log_decay, scale=K ** -0.5, return_last_state=True)
    y = group_norm_fwd(o.flatten(2), weight, bias, z, groups=H)
    d = group_norm_bwd(o.flatten(2), weight, bias, z, dy=dy, groups=H)
    d = linear_attention_bwd(q, k, v, log_decay, do=d["dx"].view_as(o), scale=K ** -0.5)
    o = linear_attention_step(q1, k1, v1, log_decay1, state=last)

    q, k           [batch, L, Hk, K]    (H heads share Hk of them, in runs of H / Hk; K, V at most 256)
    v, o           [batch, L, H, V]     the I/O type of q and k
    log_decay      [H] or [batch, L, H] float32; -inf starts the state anew
    state          [batch, H, K, V]     float32
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libselscan.so")

SELSCAN_ABI_VERSION = 2
SELSCAN_F32, SELSCAN_BF16 = 0, 1
SELSCAN_OK = 0
SELSCAN_ERR_NULL, SELSCAN_ERR_DIMS, SELSCAN_ERR_UNSUPPORTED = -1, -2, -3
SELSCAN_ERR_ALIGN, SELSCAN_ERR_HIP, SELSCAN_ERR_WORKSPACE, SELSCAN_ERR_ABI = -4, -5, -6, -7
SELSCAN_ERR_SCRATCH_LIMIT = -8
NOALLOC_SCRATCH_BYTES = 64 << 20          # SELSCAN_NOALLOC_SCRATCH_BYTES
PATHS = {"auto": 0, "single": 1, "chunked": 2, "conv": 3}   # conv: fixed coefficients only
FLAG_SCALAR_IO = 0x100   # tests only: force the general per-element kernel
DISCRETIZATIONS = {"zoh": 0, "euler": 1}


class SelscanDims(ctypes.Structure):
    """Mirror of ``selscan_dims`` in include/selscan.h (same field order and types)."""
    _fields_ = [
        ("abi_version", ctypes.c_int32), ("io_dtype", ctypes.c_int32),
        ("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("dim", ctypes.c_int64), ("dstate", ctypes.c_int64),
        ("u_sb", ctypes.c_int64), ("u_sl", ctypes.c_int64),
        ("delta_sb", ctypes.c_int64), ("delta_sl", ctypes.c_int64),
        ("z_sb", ctypes.c_int64), ("z_sl", ctypes.c_int64),
        ("y_sb", ctypes.c_int64), ("y_sl", ctypes.c_int64),
        ("B_sb", ctypes.c_int64), ("B_sl", ctypes.c_int64), ("B_sd", ctypes.c_int64),
        ("C_sb", ctypes.c_int64), ("C_sl", ctypes.c_int64), ("C_sd", ctypes.c_int64),
        ("path", ctypes.c_int32), ("chunk_len", ctypes.c_int32),
        ("discretization", ctypes.c_int32), ("delta_softplus", ctypes.c_int32),
    ]


class SelscanError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = "%s failed: %s (status %d)" % (where, strerror(status), status)
        if status == SELSCAN_ERR_HIP:
            msg += ", hipError %d" % last_hip_error()
        super().__init__(msg)


_lib = None

# (name, restype, argtypes) of every exported entry point
_VP = ctypes.c_void_p
_SIGNATURES = [
    ("selscan_dims_init", None, [ctypes.POINTER(SelscanDims), ctypes.c_int, ctypes.c_int64, ctypes.c_int64,
                                 ctypes.c_int64, ctypes.c_int64, ctypes.c_int]),
    ("selective_scan_fwd", ctypes.c_int, [_VP] * 9 + [ctypes.POINTER(SelscanDims), _VP]),
    ("selective_scan_workspace_size", ctypes.c_size_t, [ctypes.POINTER(SelscanDims)]),
    ("selective_scan_plan_path", ctypes.c_int, [ctypes.POINTER(SelscanDims)]),
    ("selective_scan_fwd_ws", ctypes.c_int, [_VP] * 9 + [ctypes.POINTER(SelscanDims), _VP, ctypes.c_size_t, _VP]),
    ("selective_scan_fwd_ex", ctypes.c_int, [_VP] * 11 + [ctypes.POINTER(SelscanDims), _VP, ctypes.c_size_t, _VP]),
    ("selective_scan_fwd_noalloc", ctypes.c_int, [_VP] * 11 + [ctypes.POINTER(SelscanDims), _VP]),
    ("selective_scan_step", ctypes.c_int, [_VP] * 10 + [ctypes.POINTER(SelscanDims), _VP]),
    ("selective_scan_bwd", ctypes.c_int, [_VP] * 20 + [ctypes.POINTER(SelscanDims), _VP, ctypes.c_size_t, _VP]),
    ("selective_scan_bwd_workspace_size", ctypes.c_size_t, [ctypes.POINTER(SelscanDims)]),
    ("selective_scan_ssd_fwd", ctypes.c_int, [_VP] * 10 + [ctypes.c_void_p, _VP, ctypes.c_size_t, _VP]),
    ("selective_scan_ssd_workspace_size", ctypes.c_size_t, [ctypes.c_void_p]),
    ("gated_scan_dims_init", None, [_VP, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64]),
    ("gated_scan_fwd", ctypes.c_int, [_VP] * 9 + [_VP, _VP, ctypes.c_size_t, _VP]),
    ("gated_scan_workspace_size", ctypes.c_size_t, [_VP]),
    ("gated_scan_bwd", ctypes.c_int, [_VP] * 14 + [_VP, _VP, ctypes.c_size_t, _VP]),
    ("gated_scan_bwd_workspace_size", ctypes.c_size_t, [_VP, ctypes.c_int]),
    ("gated_scan_step", ctypes.c_int, [_VP] * 6 + [_VP, _VP]),
    ("state_cache_write", ctypes.c_int, [_VP, _VP, ctypes.c_int64, _VP, _VP, _VP, _VP, _VP]),
    ("state_cache_read", ctypes.c_int, [_VP, _VP, _VP, ctypes.c_int64, _VP, ctypes.c_int, _VP, _VP]),
    ("selective_scan_step_cached", ctypes.c_int, [_VP] * 17),
    ("selective_scan_ssd_step_cached", ctypes.c_int, [_VP] * 16),
    ("linear_attention_dims_init", None, [_VP, ctypes.c_int] + [ctypes.c_int64] * 6),
    ("linear_attention_fwd", ctypes.c_int, [_VP] * 7 + [_VP, _VP, ctypes.c_size_t, _VP]),
    ("linear_attention_workspace_size", ctypes.c_size_t, [_VP]),
    ("linear_attention_bwd", ctypes.c_int, [_VP] * 12 + [_VP, _VP, ctypes.c_size_t, _VP]),
    ("linear_attention_bwd_workspace_size", ctypes.c_size_t, [_VP, ctypes.c_int]),
    ("linear_attention_step", ctypes.c_int, [_VP] * 6 + [ctypes.c_int64, _VP, _VP, _VP, _VP]),
    ("group_norm_dims_init", None, [_VP, ctypes.c_int] + [ctypes.c_int64] * 4),
    ("group_norm_fwd", ctypes.c_int, [_VP] * 7),
    ("group_norm_bwd", ctypes.c_int, [_VP] * 9 + [_VP, _VP, ctypes.c_size_t, _VP]),
    ("group_norm_bwd_workspace_size", ctypes.c_size_t, [_VP]),
    ("selective_scan_strerror", ctypes.c_char_p, [ctypes.c_int]),
    ("selective_scan_last_hip_error", ctypes.c_int, []),
    ("selective_scan_abi_version", ctypes.c_int, []),
]


def lib():
    """The loaded libselscan.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libselscan.so is not built (expected at %s); run "
                               "`python -m selective_state_space_s6_amd.build`" % LIB_PATH)
        # PyTorch's wheel carries its own HIP runtime; it is loaded first so that this library
        # binds to the runtime that owns PyTorch's streams and memory (loaded the other way
        # round, HIP calls from here fail with hipErrorNoDevice)
        try:
            import torch  # noqa: F401
        except ImportError:
            pass
        handle = ctypes.CDLL(LIB_PATH)
        for name, res, args in _SIGNATURES:
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        if handle.selective_scan_abi_version() != SELSCAN_ABI_VERSION:
            raise RuntimeError("libselscan.so ABI version mismatch")
        _lib = handle
    return _lib


def strerror(status: int) -> str:
    return lib().selective_scan_strerror(int(status)).decode()


def last_hip_error() -> int:
    return int(lib().selective_scan_last_hip_error())


def abi_version() -> int:
    return int(lib().selective_scan_abi_version())


def dims_init(io_dtype: int, batch: int, seqlen: int, dim: int, dstate: int, time_invariant: bool = False) -> SelscanDims:
    d = SelscanDims()
    lib().selscan_dims_init(ctypes.byref(d), int(io_dtype), int(batch), int(seqlen), int(dim), int(dstate),
                            1 if time_invariant else 0)
    return d


def workspace_size(dims: SelscanDims) -> int:
    return int(lib().selective_scan_workspace_size(ctypes.byref(dims)))


def plan_path(dims: SelscanDims) -> str:
    """The path a forward call with these dims takes ("single", "chunked" or "conv")."""
    code = int(lib().selective_scan_plan_path(ctypes.byref(dims)))
    if code < 0:
        raise SelscanError(code, "selective_scan_plan_path")
    return {v: k for k, v in PATHS.items()}[code]


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _io_code(dtype):
    import torch
    if dtype == torch.float32:
        return SELSCAN_F32
    if dtype == torch.bfloat16:
        return SELSCAN_BF16
    raise TypeError("u/delta/B/C/z/y must be float32 or bfloat16, got %s" % dtype)


def _strides_bld(t, name, batch, L, D):
    """(sb, sl) element strides of a [batch, L, D] tensor whose last axis is unit-stride."""
    if t.dim() != 3 or tuple(t.shape) != (batch, L, D):
        raise ValueError("%s must have shape %s, got %s" % (name, (batch, L, D), tuple(t.shape)))
    if D > 1 and t.stride(2) != 1:
        raise ValueError("%s: the channel axis must be unit-stride" % name)
    return t.stride(0), t.stride(1)


def make_dims(u, delta, A, B, C, z=None, y=None, *, path: str = "auto", chunk_len: int = 0,
              scalar_io: bool = False, discretization: str = "zoh", delta_softplus: bool = False) -> SelscanDims:
    """Build selscan_dims from tensor shapes and strides (see the module docstring)."""
    if u.dim() != 3:
        raise ValueError("u must be [batch, L, D]")
    batch, L, D = (int(x) for x in u.shape)
    if A.dim() != 2 or int(A.shape[0]) != D:
        raise ValueError("A must be [D, N]")
    N = int(A.shape[1])
    d = SelscanDims()
    d.abi_version = SELSCAN_ABI_VERSION
    d.io_dtype = _io_code(u.dtype)
    d.batch, d.seqlen, d.dim, d.dstate = batch, L, D, N
    d.u_sb, d.u_sl = _strides_bld(u, "u", batch, L, D)
    if delta.dim() == 1:
        if int(delta.shape[0]) != D or (D > 1 and delta.stride(0) != 1):
            raise ValueError("per-channel delta must be a contiguous [D] tensor")
        d.delta_sb = d.delta_sl = 0
    else:
        d.delta_sb, d.delta_sl = _strides_bld(delta, "delta", batch, L, D)
    for name, t in (("B", B), ("C", C)):
        if t.dim() == 2:
            if tuple(t.shape) != (D, N) or (N > 1 and t.stride(1) != 1):
                raise ValueError("per-channel %s must be [D, N] with a unit-stride state axis" % name)
            sb, sl, sd = 0, 0, t.stride(0)
        elif t.dim() == 3:
            if tuple(t.shape) != (batch, L, N) or (N > 1 and t.stride(2) != 1):
                raise ValueError("per-token %s must be [batch, L, N] with a unit-stride state axis" % name)
            sb, sl, sd = t.stride(0), t.stride(1), 0
        else:
            raise ValueError("%s must be [batch, L, N] or [D, N]" % name)
        setattr(d, name + "_sb", sb)
        setattr(d, name + "_sl", sl)
        setattr(d, name + "_sd", sd)
    if z is not None:
        d.z_sb, d.z_sl = _strides_bld(z, "z", batch, L, D)
    if y is not None:
        d.y_sb, d.y_sl = _strides_bld(y, "y", batch, L, D)
    d.path = PATHS[path] | (FLAG_SCALAR_IO if scalar_io else 0)
    d.chunk_len = int(chunk_len)
    d.discretization = DISCRETIZATIONS[discretization]
    d.delta_softplus = 1 if delta_softplus else 0
    return d


def _check_dskip(Dskip, D):
    """Dskip is read as Dskip[d] for every channel d < D: anything but a contiguous float32
    [D] GPU tensor is rejected before any launch."""
    import torch
    if Dskip is not None and (Dskip.dtype != torch.float32 or tuple(Dskip.shape) != (D,)
                              or not Dskip.is_contiguous() or not Dskip.is_cuda):
        raise ValueError("Dskip must be a contiguous float32 [D] GPU tensor (D = %d), got %s %s"
                         % (D, tuple(Dskip.shape), Dskip.dtype))


def _check_bias(delta_bias, D):
    import torch
    if delta_bias is not None and (delta_bias.dtype != torch.float32 or tuple(delta_bias.shape) != (D,)
                                   or not delta_bias.is_contiguous() or not delta_bias.is_cuda):
        raise ValueError("delta_bias must be a contiguous float32 [D] GPU tensor")


def selective_scan_fwd(u, delta, A, B, C, Dskip=None, z=None, y=None, last_state=None, *,
                       initial_state=None, delta_bias=None, delta_softplus: bool = False,
                       discretization: str = "zoh", return_last_state: bool = False, path: str = "auto",
                       chunk_len: int = 0, scalar_io: bool = False, workspace=None,
                       stream=None) -> Tuple["object", Optional["object"]]:
    """Selective-scan forward on the GPU.  Returns (y, last_state or None).

    ``y`` / ``last_state`` may be given (outputs are written in place) or are allocated.
    ``initial_state`` ([batch, D, N] float32, selective coefficients only) is the state the
    sequence continues from; it may be the ``last_state`` tensor itself (continue in place).

    ``workspace`` (a uint8 CUDA tensor of at least ``workspace_size`` bytes) selects the
    non-allocating entry point; when it is omitted and the call needs one, it is taken from
    torch's caching allocator.  ``stream`` defaults to torch's current stream."""
    import torch
    io = u.dtype
    for name, t in (("delta", delta), ("B", B), ("C", C), ("z", z), ("y", y)):
        if t is not None and t.dtype != io:
            raise TypeError("%s has dtype %s, expected %s like u" % (name, t.dtype, io))
    if A.dtype != torch.float32 or not A.is_contiguous():
        raise TypeError("A must be a contiguous float32 [D, N] tensor")
    if u.dim() != 3:
        raise ValueError("u must be [batch, L, D]")
    _check_dskip(Dskip, int(u.shape[2]))
    for name, t in (("u", u), ("delta", delta), ("A", A), ("B", B), ("C", C), ("Dskip", Dskip), ("z", z), ("y", y),
                    ("last_state", last_state)):
        if t is not None and not t.is_cuda:
            raise ValueError("%s must be a GPU tensor" % name)
    if y is None:
        y = torch.empty(u.shape, dtype=io, device=u.device)
    batch, L, D = (int(x) for x in u.shape)
    N = int(A.shape[1])
    if last_state is None and return_last_state:
        last_state = torch.empty((batch, D, N), dtype=torch.float32, device=u.device)
    for name, t in (("last_state", last_state), ("initial_state", initial_state)):
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous() or tuple(t.shape) != (batch, D, N)
                              or not t.is_cuda):
            raise ValueError("%s must be a contiguous float32 [batch, D, N] GPU tensor" % name)
    _check_bias(delta_bias, D)
    dims = make_dims(u, delta, A, B, C, z, y, path=path, chunk_len=chunk_len, scalar_io=scalar_io,
                     discretization=discretization, delta_softplus=delta_softplus)
    torch_stream = stream if (stream is None or hasattr(stream, "cuda_stream")) else None
    if stream is None:
        stream = torch.cuda.current_stream(u.device).cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    if workspace is None and (torch_stream is not None or stream == torch.cuda.current_stream(u.device).cuda_stream):
        # Scratch of the chunked path from torch's caching allocator (the C entry point
        # would allocate it stream-ordered on every call); a raw stream handle that is not
        # torch's current stream keeps the library's own allocation.
        need = workspace_size(dims)
        if need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=u.device)
            if torch_stream is not None:
                workspace.record_stream(torch_stream)
    if initial_state is not None or delta_bias is not None:
        ws_args = ((_ptr(workspace), int(workspace.numel() * workspace.element_size())) if workspace is not None
                   else (None, 0))
        st = lib().selective_scan_fwd_ex(_ptr(u), _ptr(delta), _ptr(delta_bias), _ptr(A), _ptr(B), _ptr(C),
                                         _ptr(Dskip), _ptr(z), _ptr(y), _ptr(initial_state), _ptr(last_state),
                                         ctypes.byref(dims), ws_args[0], ws_args[1], ctypes.c_void_p(stream))
        if st != SELSCAN_OK:
            raise SelscanError(st, "selective_scan_fwd_ex")
        return y, last_state
    args = [_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(Dskip), _ptr(z), _ptr(y), _ptr(last_state),
            ctypes.byref(dims)]
    if workspace is not None:
        st = lib().selective_scan_fwd_ws(*args, _ptr(workspace), int(workspace.numel() * workspace.element_size()),
                                         ctypes.c_void_p(stream))
        where = "selective_scan_fwd_ws"
    else:
        st = lib().selective_scan_fwd(*args, ctypes.c_void_p(stream))
        where = "selective_scan_fwd"
    if st != SELSCAN_OK:
        raise SelscanError(st, where)
    return y, last_state


def selective_scan_fwd_noalloc(u, delta, A, B, C, Dskip=None, z=None, *, y, last_state=None, initial_state=None,
                               delta_bias=None, delta_softplus: bool = False, discretization: str = "zoh",
                               path: str = "auto", chunk_len: int = 0, stream=None):
    """The forward pass through selective_scan_fwd_noalloc, which allocates nothing: the
    chunked path's scratch is the library's own per-GPU array (NOALLOC_SCRATCH_BYTES).  The
    outputs ``y`` (and ``last_state`` if wanted) must be given; nothing is allocated here
    either.  Arguments otherwise as selective_scan_fwd.  Calls that overlap on one GPU race
    on the shared scratch.  Returns (y, last_state)."""
    import torch
    io = u.dtype
    if u.dim() != 3:
        raise ValueError("u must be [batch, L, D]")
    batch, L, D = (int(x) for x in u.shape)
    _check_dskip(Dskip, D)
    for name, t in (("delta", delta), ("B", B), ("C", C), ("z", z), ("y", y)):
        if t is not None and (t.dtype != io or not t.is_cuda):
            raise TypeError("%s must be a GPU tensor of dtype %s like u" % (name, io))
    if A.dtype != torch.float32 or not A.is_contiguous() or not A.is_cuda:
        raise TypeError("A must be a contiguous float32 [D, N] GPU tensor")
    N = int(A.shape[1])
    for name, t in (("last_state", last_state), ("initial_state", initial_state)):
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous() or tuple(t.shape) != (batch, D, N)
                              or not t.is_cuda):
            raise ValueError("%s must be a contiguous float32 [batch, D, N] GPU tensor" % name)
    _check_bias(delta_bias, D)
    dims = make_dims(u, delta, A, B, C, z, y, path=path, chunk_len=chunk_len, discretization=discretization,
                     delta_softplus=delta_softplus)
    if stream is None:
        stream = torch.cuda.current_stream(u.device).cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    st = lib().selective_scan_fwd_noalloc(_ptr(u), _ptr(delta), _ptr(delta_bias), _ptr(A), _ptr(B), _ptr(C),
                                          _ptr(Dskip), _ptr(z), _ptr(y), _ptr(initial_state), _ptr(last_state),
                                          ctypes.byref(dims), ctypes.c_void_p(stream))
    if st != SELSCAN_OK:
        raise SelscanError(st, "selective_scan_fwd_noalloc")
    return y, last_state


def selective_scan_step(u, delta, A, B, C, Dskip=None, z=None, y=None, *, state, time_invariant: bool = False,
                        delta_bias=None, delta_softplus: bool = False, discretization: str = "zoh", stream=None):
    """One recurrent decode step (one token per batch row); ``state`` ([batch, D, N] float32,
    contiguous) is read as the running state and overwritten with the new one.

    u, z, y: [batch, D]; A: [D, N]; Dskip: [D].  Selective coefficients: delta [batch, D]
    (or [D] shared by the batch), B, C [batch, N].  time_invariant=True: delta [D], B, C
    [D, N].  delta_bias, delta_softplus, discretization: as selective_scan_fwd.  Returns y."""
    import torch
    if u.dim() != 2:
        raise ValueError("u must be [batch, D] (one token per batch row)")
    batch, D = (int(x) for x in u.shape)
    _check_dskip(Dskip, D)
    if A.dim() != 2 or int(A.shape[0]) != D or A.dtype != torch.float32 or not A.is_contiguous():
        raise ValueError("A must be a contiguous float32 [D, N] tensor")
    N = int(A.shape[1])
    io = u.dtype
    if y is None:
        y = torch.empty((batch, D), dtype=io, device=u.device)
    for name, t in (("delta", delta), ("B", B), ("C", C), ("z", z), ("y", y)):
        if t is not None and (t.dtype != io or not t.is_cuda):
            raise TypeError("%s must be a GPU tensor of dtype %s like u" % (name, io))
    if (state.dtype != torch.float32 or not state.is_contiguous() or tuple(state.shape) != (batch, D, N)
            or not state.is_cuda):
        raise ValueError("state must be a contiguous float32 [batch, D, N] GPU tensor")

    def rows(t, name, width):                  # [batch, width] with a unit-stride last axis
        if t.dim() != 2 or tuple(t.shape) != (batch, width) or (width > 1 and t.stride(1) != 1):
            raise ValueError("%s must be [batch, %d] with a unit-stride last axis" % (name, width))
        return t.stride(0)

    _check_bias(delta_bias, D)
    d = SelscanDims()
    d.abi_version = SELSCAN_ABI_VERSION
    d.io_dtype = _io_code(io)
    d.batch, d.seqlen, d.dim, d.dstate = batch, 1, D, N
    d.discretization = DISCRETIZATIONS[discretization]
    d.delta_softplus = 1 if delta_softplus else 0
    d.u_sb = rows(u, "u", D)
    d.u_sl = D
    d.y_sb = rows(y, "y", D)
    d.y_sl = D                                 # rows of different batch entries must not overlap
    if z is not None:
        d.z_sb = rows(z, "z", D)
        d.z_sl = D
    if delta.dim() == 1:
        if int(delta.shape[0]) != D or (D > 1 and delta.stride(0) != 1):
            raise ValueError("per-channel delta must be a contiguous [D] tensor")
        d.delta_sb = d.delta_sl = 0
    else:
        d.delta_sb = rows(delta, "delta", D)
        d.delta_sl = D
    if time_invariant and delta.dim() != 1:
        raise ValueError("time-invariant coefficients take a per-channel [D] delta")
    for name, t in (("B", B), ("C", C)):
        if time_invariant:
            if t.dim() != 2 or tuple(t.shape) != (D, N) or (N > 1 and t.stride(1) != 1):
                raise ValueError("per-channel %s must be [D, N] with a unit-stride state axis" % name)
            sb, sl, sd = 0, 0, t.stride(0)
        else:
            sb, sl, sd = rows(t, name, N), N, 0
        setattr(d, name + "_sb", sb)
        setattr(d, name + "_sl", sl)
        setattr(d, name + "_sd", sd)
    if stream is None:
        stream = torch.cuda.current_stream(u.device).cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    st = lib().selective_scan_step(_ptr(u), _ptr(delta), _ptr(delta_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(Dskip),
                                   _ptr(z), _ptr(y), _ptr(state), ctypes.byref(d), ctypes.c_void_p(stream))
    if st != SELSCAN_OK:
        raise SelscanError(st, "selective_scan_step")
    return y


def bwd_workspace_size(dims: SelscanDims) -> int:
    return int(lib().selective_scan_bwd_workspace_size(ctypes.byref(dims)))


def selective_scan_bwd(u, delta, A, B, C, Dskip=None, z=None, *, dy, dlast_state=None, initial_state=None,
                       delta_bias=None, delta_softplus: bool = False, discretization: str = "zoh", workspace=None,
                       stream=None) -> dict:
    """Gradients of selective_scan_fwd (same inputs and options) given dy, the gradient of y,
    and optionally dlast_state, the gradient of last_state.

    Returns a dict: du, ddelta, dz (if z) as [batch, L, D] and dB, dC as [batch, L, N], in
    u's dtype; dA [D, N], dDskip [D] (if Dskip), ddelta_bias [D] (if delta_bias) and
    dinitial_state [batch, D, N] (if initial_state), in float32.  With fixed coefficients
    (delta [D], B and C [D, N]) ddelta is [D] and dB, dC are [D, N], in u's dtype.
    ``workspace`` (a uint8 GPU tensor of bwd_workspace_size bytes) is taken from torch's
    caching allocator when omitted."""
    import torch
    io = u.dtype
    if u.dim() != 3:
        raise ValueError("u must be [batch, L, D]")
    batch, L, D = (int(x) for x in u.shape)
    _check_dskip(Dskip, D)
    for name, t in (("delta", delta), ("B", B), ("C", C), ("z", z), ("dy", dy)):
        if t is not None and (t.dtype != io or not t.is_cuda):
            raise TypeError("%s must be a GPU tensor of dtype %s like u" % (name, io))
    if A.dtype != torch.float32 or not A.is_contiguous():
        raise TypeError("A must be a contiguous float32 [D, N] tensor")
    N = int(A.shape[1])
    for name, t in (("dlast_state", dlast_state), ("initial_state", initial_state)):
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous() or tuple(t.shape) != (batch, D, N)
                              or not t.is_cuda):
            raise ValueError("%s must be a contiguous float32 [batch, D, N] GPU tensor" % name)
    _check_bias(delta_bias, D)
    dims = make_dims(u, delta, A, B, C, z, dy, discretization=discretization, delta_softplus=delta_softplus)
    dev = u.device
    ti = delta.dim() == 1 and B.dim() == 2 and C.dim() == 2      # fixed coefficients
    g = {"du": torch.empty((batch, L, D), dtype=io, device=dev),
         "ddelta": torch.empty((D,) if ti else (batch, L, D), dtype=io, device=dev),
         "dA": torch.empty((D, N), dtype=torch.float32, device=dev),
         "dB": torch.empty((D, N) if ti else (batch, L, N), dtype=io, device=dev),
         "dC": torch.empty((D, N) if ti else (batch, L, N), dtype=io, device=dev)}
    if z is not None:
        g["dz"] = torch.empty((batch, L, D), dtype=io, device=dev)
    if Dskip is not None:
        g["dDskip"] = torch.empty((D,), dtype=torch.float32, device=dev)
    if delta_bias is not None:
        g["ddelta_bias"] = torch.empty((D,), dtype=torch.float32, device=dev)
    if initial_state is not None:
        g["dinitial_state"] = torch.empty((batch, D, N), dtype=torch.float32, device=dev)
    torch_stream = stream if (stream is None or hasattr(stream, "cuda_stream")) else None
    if stream is None:
        stream = torch.cuda.current_stream(dev).cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    if workspace is None and (torch_stream is not None or stream == torch.cuda.current_stream(dev).cuda_stream):
        need = bwd_workspace_size(dims)
        if need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
            if torch_stream is not None:
                workspace.record_stream(torch_stream)
    ws = (_ptr(workspace), int(workspace.numel() * workspace.element_size())) if workspace is not None else (None, 0)
    st = lib().selective_scan_bwd(
        _ptr(u), _ptr(delta), _ptr(delta_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(Dskip), _ptr(z), _ptr(initial_state),
        _ptr(dy), _ptr(dlast_state), _ptr(g["du"]), _ptr(g["ddelta"]), _ptr(g.get("ddelta_bias")), _ptr(g["dA"]),
        _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g.get("dDskip")), _ptr(g.get("dz")), _ptr(g.get("dinitial_state")),
        ctypes.byref(dims), ws[0], ws[1], ctypes.c_void_p(stream))
    if st != SELSCAN_OK:
        raise SelscanError(st, "selective_scan_bwd")
    return g


class SsdDims(ctypes.Structure):
    """Mirror of ``selscan_ssd_dims`` in include/selscan.h."""
    _fields_ = [("abi_version", ctypes.c_int32), ("discretization", ctypes.c_int32), ("batch", ctypes.c_int64),
                ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64), ("headdim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("path", ctypes.c_int32), ("segments", ctypes.c_int32)]


SSD_PATHS = {"auto": 0, "fused": 1, "chunked": 2, "segmented": 3}


def ssd_dims(batch, seqlen, nheads, headdim, dstate, discretization="zoh", path="auto", segments=0) -> SsdDims:
    d = SsdDims()
    d.abi_version = SELSCAN_ABI_VERSION
    d.discretization = DISCRETIZATIONS[discretization]
    d.path = SSD_PATHS[path]
    d.segments = int(segments)
    d.batch, d.seqlen, d.nheads, d.headdim, d.dstate = int(batch), int(seqlen), int(nheads), int(headdim), int(dstate)
    return d


def ssd_workspace_size(dims: SsdDims) -> int:
    return int(lib().selective_scan_ssd_workspace_size(ctypes.byref(dims)))


def selective_scan_ssd_fwd(x, delta, A, B, C, Dskip=None, z=None, y=None, *, initial_state=None,
                           return_last_state: bool = False, discretization: str = "zoh", path: str = "auto",
                           segments: int = 0, workspace=None, stream=None):
    """The scalar-decay (Mamba-2) layer on the GPU (bf16 x, delta, B, C, z, y; fp32 A, Dskip,
    states).  x, z: [batch, L, H, 64]; delta: [batch, L, H]; A: [H]; B, C: [batch, L, N] with
    N = 64 or 128; Dskip: [H * 64]; initial_state: [batch, H, 64, N].  All contiguous.
    path: "auto", "fused" (on chip), "chunked" (chunk-parallel) or "segmented" (on chip over
    `segments` sequence segments, 0 = chosen by the library).  Returns (y, last_state or None)."""
    import torch
    if x.dim() != 4:
        raise ValueError("x must be [batch, L, H, headdim]")
    batch, L, H, P = (int(v) for v in x.shape)
    N = int(B.shape[-1])
    for name, t in (("x", x), ("delta", delta), ("B", B), ("C", C), ("z", z), ("y", y)):
        if t is not None and (t.dtype != torch.bfloat16 or not t.is_contiguous() or not t.is_cuda):
            raise TypeError("%s must be a contiguous bfloat16 GPU tensor" % name)
    if tuple(delta.shape) != (batch, L, H) or tuple(B.shape) != (batch, L, N) or tuple(C.shape) != (batch, L, N):
        raise ValueError("delta must be [batch, L, H]; B, C [batch, L, N]")
    for name, t, shape in (("A", A, (H,)), ("Dskip", Dskip, (H * P,)), ("initial_state", initial_state, (batch, H, P, N))):
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous() or tuple(t.shape) != shape or not t.is_cuda):
            raise ValueError("%s must be a contiguous float32 %s GPU tensor" % (name, shape))
    if y is None:
        y = torch.empty_like(x)
    last = torch.empty((batch, H, P, N), dtype=torch.float32, device=x.device) if return_last_state else None
    dims = ssd_dims(batch, L, H, P, N, discretization, path, segments)
    torch_stream = stream if (stream is None or hasattr(stream, "cuda_stream")) else None
    if stream is None:
        stream = torch.cuda.current_stream(x.device).cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    if workspace is None and (torch_stream is not None or stream == torch.cuda.current_stream(x.device).cuda_stream):
        need = ssd_workspace_size(dims)
        if need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
            if torch_stream is not None:
                workspace.record_stream(torch_stream)
    ws = (_ptr(workspace), int(workspace.numel() * workspace.element_size())) if workspace is not None else (None, 0)
    st = lib().selective_scan_ssd_fwd(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(Dskip), _ptr(z), _ptr(y),
                                      _ptr(initial_state), _ptr(last), ctypes.byref(dims), ws[0], ws[1],
                                      ctypes.c_void_p(stream))
    if st != SELSCAN_OK:
        raise SelscanError(st, "selective_scan_ssd_fwd")
    return y, last


class GatedDims(ctypes.Structure):
    """Mirror of ``selscan_gated_dims`` in include/selscan.h."""
    _fields_ = [("abi_version", ctypes.c_int32), ("io_dtype", ctypes.c_int32), ("batch", ctypes.c_int64),
                ("seqlen", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("x_sb", ctypes.c_int64), ("x_sl", ctypes.c_int64), ("r_sb", ctypes.c_int64), ("r_sl", ctypes.c_int64),
                ("g_sb", ctypes.c_int64), ("g_sl", ctypes.c_int64), ("y_sb", ctypes.c_int64), ("y_sl", ctypes.c_int64),
                ("reset_sb", ctypes.c_int64), ("decay_c", ctypes.c_float), ("reserved", ctypes.c_int32)]


class CacheDims(ctypes.Structure):
    """Mirror of ``selscan_cache_dims`` in include/selscan.h."""
    _fields_ = [("abi_version", ctypes.c_int32), ("reserved", ctypes.c_int32), ("slots", ctypes.c_int64),
                ("elems", ctypes.c_int64), ("row_len", ctypes.c_int64)]


GATED_TILE = 64          # SELSCAN_GATED_TILE: tokens between two checkpoints
CACHE_ROW = 64            # row length of a [D] state (the gated recurrence's) in the state cache


_raw_stream = None


def _current_stream(index):
    """The handle of torch's current stream on GPU `index`, without a Stream object where torch has
    that (1 us less a call)."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda i: torch.cuda.current_stream(i).cuda_stream)
    return _raw_stream(index)


class _On:
    """The GPU and the stream of one call: what is allocated inside belongs to that stream."""
    __slots__ = ("device", "index", "handle", "_guards")

    def __init__(self, t, stream):
        import torch
        index = t.get_device()
        if index < 0:
            raise ValueError("the tensors must be GPU tensors")
        self.device, self.index, self._guards = t.device, index, ()
        if stream is None:
            self.handle = _current_stream(index)
        else:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=self.device)
            self.handle = stream.cuda_stream
            self._guards = (torch.cuda.stream(stream),)
        if torch.cuda.current_device() != index:
            self._guards = (torch.cuda.device(index),) + self._guards

    def __enter__(self):
        for g in self._guards:
            g.__enter__()
        return self

    def __exit__(self, *exc):
        for g in reversed(self._guards):
            g.__exit__(*exc)
        return False

    def check(self, name, t, dtype, shape, contiguous=True):
        """t (None passes) must be of this dtype and shape, on this GPU, and contiguous unless said."""
        if t is None or (t.dtype is dtype and t.shape == shape and t.get_device() == self.index
                         and (not contiguous or t.is_contiguous())):
            return
        if t.dtype is not dtype:
            raise TypeError("%s must have dtype %s, got %s" % (name, dtype, t.dtype))
        if t.shape != shape:
            raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
        if t.get_device() != self.index:
            raise ValueError("%s must be on %s, got %s" % (name, self.device, t.device))
        raise ValueError("%s must be contiguous" % name)

    def workspace(self, given, need):
        """(tensor, pointer, bytes) of the workspace: the given one, or one of torch's caching allocator."""
        import torch
        if given is None:
            if need == 0:
                return None, None, 0
            given = torch.empty(need, dtype=torch.uint8, device=self.device)
            return given, given.data_ptr(), need
        if given.get_device() != self.index or not given.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on %s" % self.device)
        return given, given.data_ptr(), given.numel() * given.element_size()


def _p(t):
    return None if t is None else t.data_ptr()


def _gated_dims(on, x, r, g, lam, y, reset, c):
    """selscan_gated_dims of [batch, L, D] tensors; their channel axes are unit-stride."""
    import torch
    batch, L, D = x.shape
    io, shape, strides = x.dtype, x.shape, []
    for name, t in (("x", x), ("r", r), ("g", g), ("y", y)):
        on.check(name, t, io, shape, contiguous=False)
        sb, sl, sd = t.stride()
        if sd != 1 and D > 1:
            raise ValueError("%s: the channel axis must be unit-stride" % name)
        strides += (sb, sl if L > 1 else D)                    # (one token: any stride)
    on.check("lam", lam, torch.float32, (D,))
    d = GatedDims(SELSCAN_ABI_VERSION, _io_code(io), batch, L, D, *strides, 0, c, 0)
    if reset is not None:
        if reset.dtype not in (torch.bool, torch.uint8):
            raise TypeError("reset must be a bool or uint8 [batch, L] tensor")
        on.check("reset", reset, reset.dtype, (batch, L), contiguous=False)
        if L > 1 and reset.stride(1) != 1:
            raise ValueError("reset: the token axis must be unit-stride")
        d.reset_sb = reset.stride(0)
    return d


def gated_checkpoints(x):
    """A tensor for the states that gated_scan_fwd leaves for gated_scan_bwd:
    [batch, ceil(L / GATED_TILE), D] float32 for x [batch, L, D]."""
    import torch
    return torch.empty((x.shape[0], -(-x.shape[1] // GATED_TILE), x.shape[2]), dtype=torch.float32, device=x.device)


def gated_scan_fwd(x, r, g, lam, *, y=None, initial_state=None, last_state=None, return_last_state: bool = False,
                   checkpoints=None, reset=None, c: float = 8.0, workspace=None, stream=None):
    """The gated linear recurrence h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(g_t) x_t with
    a_t = exp(-c softplus(lam) sigmoid(r_t)); y = h.  Returns (y, last_state or None).

    x, r, g, y: [batch, L, D] float32 or bfloat16 (unit-stride channels); lam: [D] float32;
    reset: [batch, L] bool or uint8, true where a packed sequence starts; initial_state,
    last_state: [batch, D] float32; checkpoints (see gated_checkpoints) is filled for the
    backward pass.  ``workspace`` is taken from torch's caching allocator when omitted."""
    import torch
    if x.dim() != 3:
        raise ValueError("x must be [batch, L, D]")
    with _On(x, stream) as on:
        batch, L, D = x.shape
        if y is None:
            y = x.new_empty((batch, L, D))
        if last_state is None and return_last_state:
            last_state = torch.empty((batch, D), dtype=torch.float32, device=x.device)
        dims = _gated_dims(on, x, r, g, lam, y, reset, c)
        on.check("initial_state", initial_state, torch.float32, (batch, D))
        on.check("last_state", last_state, torch.float32, (batch, D))
        on.check("checkpoints", checkpoints, torch.float32, (batch, -(-L // GATED_TILE), D))
        ref = ctypes.byref(dims)
        keep, ws, nbytes = on.workspace(workspace, lib().gated_scan_workspace_size(ref))
        st = lib().gated_scan_fwd(_p(x), _p(r), _p(g), _p(lam), _p(reset), _p(y), _p(initial_state), _p(last_state),
                                  _p(checkpoints), ref, ws, nbytes, on.handle)
        if st != SELSCAN_OK:
            raise SelscanError(st, "gated_scan_fwd")
    return y, last_state


def gated_scan_bwd(x, r, g, lam, *, dy, dlast_state=None, initial_state=None, checkpoints=None, reset=None,
                   c: float = 8.0, workspace=None, stream=None) -> dict:
    """Gradients of gated_scan_fwd (same inputs and options) given dy and optionally
    dlast_state.  Returns a dict: dx, dr, dg as [batch, L, D] in x's dtype; dlam [D] and (with an
    initial_state) dinitial_state [batch, D] in float32.  ``checkpoints``: what the forward call
    filled, or None to form them again."""
    import torch
    if x.dim() != 3:
        raise ValueError("x must be [batch, L, D]")
    with _On(x, stream) as on:
        batch, L, D = x.shape
        dims = _gated_dims(on, x, r, g, lam, dy, reset, c)
        on.check("dlast_state", dlast_state, torch.float32, (batch, D))
        on.check("initial_state", initial_state, torch.float32, (batch, D))
        on.check("checkpoints", checkpoints, torch.float32, (batch, -(-L // GATED_TILE), D))
        out = {k: torch.empty((batch, L, D), dtype=x.dtype, device=x.device) for k in ("dx", "dr", "dg")}
        out["dlam"] = torch.empty((D,), dtype=torch.float32, device=x.device)
        if initial_state is not None:
            out["dinitial_state"] = torch.empty((batch, D), dtype=torch.float32, device=x.device)
        ref = ctypes.byref(dims)
        keep, ws, nbytes = on.workspace(workspace, lib().gated_scan_bwd_workspace_size(ref, checkpoints is not None))
        st = lib().gated_scan_bwd(_p(x), _p(r), _p(g), _p(lam), _p(reset), _p(initial_state), _p(checkpoints), _p(dy),
                                  _p(dlast_state), _p(out["dx"]), _p(out["dr"]), _p(out["dg"]), _p(out["dlam"]),
                                  _p(out.get("dinitial_state")), ref, ws, nbytes, on.handle)
        if st != SELSCAN_OK:
            raise SelscanError(st, "gated_scan_bwd")
    return out


def gated_scan_step(x, r, g, lam, *, state, y=None, c: float = 8.0, stream=None):
    """One token of the gated recurrence per batch row (x, r, g, y: [batch, D]); ``state``
    ([batch, D] float32, contiguous) is overwritten with the new one.  Returns y."""
    import torch
    if x.dim() != 2:
        raise ValueError("x must be [batch, D] (one token per batch row)")
    with _On(x, stream) as on:
        batch, D = x.shape
        if y is None:
            y = x.new_empty((batch, D))
        shape = x.shape
        io, strides = x.dtype, []
        for name, t in (("x", x), ("r", r), ("g", g), ("y", y)):
            on.check(name, t, io, shape, contiguous=False)
            sb, sd = t.stride()
            if sd != 1 and D > 1:
                raise ValueError("%s: the channel axis must be unit-stride" % name)
            strides += (sb, D)
        on.check("lam", lam, torch.float32, (D,))
        dims = GatedDims(SELSCAN_ABI_VERSION, _io_code(io), batch, 1, D, *strides, 0, c, 0)
        on.check("state", state, torch.float32, shape)
        st = lib().gated_scan_step(x.data_ptr(), r.data_ptr(), g.data_ptr(), lam.data_ptr(), y.data_ptr(), state.data_ptr(),
                                   ctypes.byref(dims), on.handle)
        if st != SELSCAN_OK:
            raise SelscanError(st, "gated_scan_step")
    return y


def state_cache(slots: int, *state_shape: int, device="cuda"):
    """An empty 8-bit state cache (q, scale) of `slots` states of this shape: (D, N) for the
    selective scan, (H, 64, N) for the scalar-decay layer (a scale per N values), (D,) for the
    gated recurrence (a scale per 64 channels).  q: [slots, *state_shape] int8; scale:
    [slots, rows] float32.  Every slot holds the zero state."""
    import torch
    rows = -(-state_shape[0] // CACHE_ROW) if len(state_shape) == 1 else 1
    for n in state_shape[:-1]:
        rows *= n
    return (torch.zeros((slots,) + state_shape, dtype=torch.int8, device=device),
            torch.zeros((slots, rows), dtype=torch.float32, device=device))


def _cache_dims(on, q, scale, seed):
    import torch
    shape = q.shape
    if len(shape) < 2:
        raise ValueError("q must be [slots, *state_shape]")
    row_len = CACHE_ROW if len(shape) == 2 else shape[-1]
    elems = 1
    for n in shape[1:]:
        elems *= n
    on.check("q", q, torch.int8, shape)
    on.check("scale", scale, torch.float32, (shape[0], -(-elems // row_len) if row_len else 0))
    on.check("seed", seed, torch.int64, (1,))
    return CacheDims(SELSCAN_ABI_VERSION, 0, shape[0], elems, row_len)


def state_cache_write(state, q, scale, *, slots=None, seed=None, stream=None) -> None:
    """Store states ([count, *state_shape] float32) in the slots that ``slots`` ([count] int32;
    0, 1, 2, ... when omitted) names, as 8-bit codes; ids outside the cache skip their row and
    the others must differ.  ``seed``: a one-element int64 GPU tensor for stochastic rounding
    (nearest when omitted); it is only read, so change it before every call (``seed.add_(1)``,
    which a graph can hold): the same seed rounds the same value the same way each time."""
    import torch
    with _On(q, stream) as on:
        dims = _cache_dims(on, q, scale, seed)
        on.check("state", state, torch.float32, state.shape[:1] + q.shape[1:])
        on.check("slots", slots, torch.int32, (state.shape[0],))
        st = lib().state_cache_write(_p(state), _p(slots), state.shape[0], _p(q), _p(scale), _p(seed),
                                     ctypes.byref(dims), on.handle)
        if st != SELSCAN_OK:
            raise SelscanError(st, "state_cache_write")


def state_cache_read(q, scale, *, slots=None, out=None, dtype=None, stream=None):
    """The states that the slots stand for: [count, *state_shape], zeros for ids outside the cache.
    dtype: float32 (the default) or bfloat16; ``out`` may be given instead."""
    import torch
    with _On(q, stream) as on:
        dims = _cache_dims(on, q, scale, None)
        count, *rest = q.shape
        if slots is not None:
            count = slots.shape[0] if slots.dim() == 1 else -1
            on.check("slots", slots, torch.int32, (count,))
        if out is None:
            out = q.new_empty((count, *rest), dtype=dtype or torch.float32)
        else:
            on.check("out", out, dtype or out.dtype, (count, *rest))
        st = lib().state_cache_read(q.data_ptr(), scale.data_ptr(), _p(slots), count, out.data_ptr(), _io_code(out.dtype),
                                    ctypes.byref(dims), on.handle)
        if st != SELSCAN_OK:
            raise SelscanError(st, "state_cache_read")
    return out


def selective_scan_step_cached(u, delta, A, B, C, Dskip=None, z=None, y=None, *, q, scale, read_slots=None,
                               write_slots=None, seed=None, delta_bias=None, delta_softplus: bool = False,
                               discretization: str = "zoh", stream=None):
    """selective_scan_step with the states in an 8-bit cache (see state_cache): row b starts from
    the state in slot read_slots[b] (the zero state where the id is outside the cache) and stores
    the new one in slot write_slots[b]; rows whose write id is outside the cache are padding and
    keep their y.  Ids: [batch] int32, 0, 1, 2, ... when omitted.  A slot that a row writes may be
    read by that row alone.  ``seed``: as state_cache_write, to be changed before every token (a
    seed that stays rounds every value the same way, and the errors add up).  delta: [batch, D]
    (or [D]); B, C: [batch, N].  Returns y."""
    import torch
    if u.dim() != 2:
        raise ValueError("u must be [batch, D] (one token per batch row)")
    with _On(u, stream) as on:
        batch, D = u.shape
        N = A.shape[-1]
        on.check("A", A, torch.float32, (D, N))
        if y is None:
            y = u.new_empty((batch, D))
        io, per_channel, sb = u.dtype, delta.dim() == 1, []
        row, states = (batch, D), (batch, N)
        for name, t, shape in (("u", u, row), ("delta", delta, (D,) if per_channel else row), ("z", z, row), ("y", y, row),
                               ("B", B, states), ("C", C, states)):
            if t is None:
                sb.append(0)
                continue
            on.check(name, t, io, shape, contiguous=False)
            strides = t.stride()
            if strides[-1] != 1 and shape[-1] > 1:
                raise ValueError("%s must have a unit-stride last axis" % name)
            sb.append(strides[0])
        if per_channel:
            sb[1] = 0
        d = SelscanDims(SELSCAN_ABI_VERSION, _io_code(io), batch, 1, D, N, sb[0], D, sb[1], 0 if per_channel else D, sb[2], D,
                        sb[3], D, sb[4], N, 0, sb[5], N, 0, 0, 0, DISCRETIZATIONS[discretization],
                        1 if delta_softplus else 0)
        on.check("Dskip", Dskip, torch.float32, (D,))
        on.check("delta_bias", delta_bias, torch.float32, (D,))
        cache = _cache_dims(on, q, scale, seed)
        if q.shape[1:] != (D, N):
            raise ValueError("q must be [slots, %d, %d]" % (D, N))
        on.check("read_slots", read_slots, torch.int32, (batch,))
        on.check("write_slots", write_slots, torch.int32, (batch,))
        st = lib().selective_scan_step_cached(_p(u), _p(delta), _p(delta_bias), _p(A), _p(B), _p(C), _p(Dskip), _p(z),
                                              _p(y), _p(q), _p(scale), _p(read_slots), _p(write_slots), _p(seed),
                                              ctypes.byref(d), ctypes.byref(cache), on.handle)
        if st != SELSCAN_OK:
            raise SelscanError(st, "selective_scan_step_cached")
    return y


def selective_scan_ssd_step_cached(x, delta, A, B, C, Dskip=None, z=None, y=None, *, q, scale, read_slots=None,
                                   write_slots=None, seed=None, discretization: str = "zoh", stream=None):
    """One token of the scalar-decay layer with the states in an 8-bit cache (slots, padding and a
    seed to be changed before every token as selective_scan_step_cached; state shape
    (H, 64, N)).  x, z, y: [batch, H, 64]; delta: [batch, H]; B, C: [batch, N], bfloat16 and
    contiguous; A: [H], Dskip: [H * 64] float32.  Returns y."""
    import torch
    if x.dim() != 3:
        raise ValueError("x must be [batch, H, 64] (one token per batch row)")
    with _On(x, stream) as on:
        batch, H, P = x.shape
        N = B.shape[-1]
        if y is None:
            y = x.new_empty((batch, H, P))
        for name, t, shape in (("x", x, (batch, H, P)), ("delta", delta, (batch, H)), ("B", B, (batch, N)),
                               ("C", C, (batch, N)), ("z", z, (batch, H, P)), ("y", y, (batch, H, P))):
            on.check(name, t, torch.bfloat16, shape)
        on.check("A", A, torch.float32, (H,))
        on.check("Dskip", Dskip, torch.float32, (H * P,))
        cache = _cache_dims(on, q, scale, seed)
        if q.shape[1:] != (H, P, N):
            raise ValueError("q must be [slots, %d, %d, %d]" % (H, P, N))
        on.check("read_slots", read_slots, torch.int32, (batch,))
        on.check("write_slots", write_slots, torch.int32, (batch,))
        dims = ssd_dims(batch, 1, H, P, N, discretization)
        st = lib().selective_scan_ssd_step_cached(_p(x), _p(delta), _p(A), _p(B), _p(C), _p(Dskip), _p(z), _p(y),
                                                  _p(q), _p(scale), _p(read_slots), _p(write_slots), _p(seed),
                                                  ctypes.byref(dims), ctypes.byref(cache), on.handle)
        if st != SELSCAN_OK:
            raise SelscanError(st, "selective_scan_ssd_step_cached")
    return y


class LinattnDims(ctypes.Structure):
    """Mirror of ``selscan_linattn_dims`` in include/selscan.h."""
    _fields_ = ([("abi_version", ctypes.c_int32), ("io_dtype", ctypes.c_int32)]
                + [(n, ctypes.c_int64) for n in ("batch", "seqlen", "nheads", "qk_heads", "dk", "dv",
                                                 "q_sb", "q_sl", "q_sh", "k_sb", "k_sl", "k_sh", "v_sb", "v_sl", "v_sh",
                                                 "o_sb", "o_sl", "o_sh", "g_sb", "g_sl", "g_sh")]
                + [("decay_tokens", ctypes.c_int32), ("scale", ctypes.c_float)])


class NormDims(ctypes.Structure):
    """Mirror of ``selscan_norm_dims`` in include/selscan.h."""
    _fields_ = ([("abi_version", ctypes.c_int32), ("io_dtype", ctypes.c_int32)]
                + [(n, ctypes.c_int64) for n in ("batch", "seqlen", "dim", "groups", "x_sb", "x_sl", "z_sb", "z_sl",
                                                 "y_sb", "y_sl")]
                + [("eps", ctypes.c_float), ("activation", ctypes.c_int32)])


ACTIVATIONS = {"none": 0, "silu": 1}


def _linattn_dims(on, q, k, v, log_decay, o, scale, step=False):
    """selscan_linattn_dims of [batch, L, heads, width] tensors (a step: [batch, heads, width])."""
    import torch
    io, lead = q.dtype, q.shape[:-2]
    Hk, K = q.shape[-2:]
    H, V = v.shape[-2:]
    if Hk == 0 or H % Hk:
        raise ValueError("the heads of v (%d) must be a multiple of those of q and k (%d)" % (H, Hk))
    batch, L = (lead[0], 1) if step else lead
    qk, vo, at = q.shape, lead + (H, V), on.index
    sq, sk, sv, so, g = q.stride(), k.stride(), v.stride(), o.stride(), log_decay.stride()
    if not (k.dtype is io and v.dtype is io and o.dtype is io and k.shape == qk and v.shape == vo and o.shape == vo
            and k.get_device() == at and v.get_device() == at and o.get_device() == at):
        for name, t, shape in (("k", k, qk), ("v", v, vo), ("o", o, vo)):
            on.check(name, t, io, shape, contiguous=False)
    if (K > 1 and not sq[-1] == sk[-1] == 1) or (V > 1 and not sv[-1] == so[-1] == 1):
        raise ValueError("q, k, v and o: the last axis must be unit-stride")
    tokens = len(g) > 1
    on.check("log_decay", log_decay, torch.float32, lead + (H,) if tokens else (H,), contiguous=False)
    # (one token: any stride between tokens)
    if step:
        strides = (sq[0], 0, sq[1], sk[0], 0, sk[1], sv[0], 0, sv[1], so[0], 0, so[1])
    elif L > 1:
        strides = sq[:3] + sk[:3] + sv[:3] + so[:3]
    else:
        strides = (sq[0], 0, sq[2], sk[0], 0, sk[2], sv[0], 0, sv[2], so[0], 0, so[2])
    g = (0, 0, g[0]) if not tokens else (g[0], 0, g[1]) if step else g
    return LinattnDims(SELSCAN_ABI_VERSION, _io_code(io), batch, L, H, Hk, K, V, *strides, *g, 1 if tokens else 0, scale)


def linear_attention_fwd(q, k, v, log_decay, *, scale: float = 1.0, o=None, initial_state=None, last_state=None,
                         return_last_state: bool = False, workspace=None, stream=None):
    """Linear attention with a decay for each head: S_t = exp(log_decay_t) S_{t-1} + k_t v_t^T,
    o_t = scale q_t^T S_t.  Returns (o, last_state or None).

    q, k: [batch, L, Hk, K]; v, o: [batch, L, H, V], float32 or bfloat16 with unit-stride last
    axes, K and V up to 256; head h reads query and key head h // (H / Hk).  log_decay: [H] or
    [batch, L, H] float32 (any strides), -inf where the state starts anew (packed documents).
    initial_state, last_state: [batch, H, K, V] float32.  ``workspace`` is taken from torch's
    caching allocator when omitted."""
    import torch
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q and v must be [batch, L, heads, width]")
    with _On(q, stream) as on:
        if o is None:
            o = q.new_empty(v.shape)
        dims = _linattn_dims(on, q, k, v, log_decay, o, scale)
        states = (dims.batch, dims.nheads, dims.dk, dims.dv)
        if last_state is None and return_last_state:
            last_state = q.new_empty(states, dtype=torch.float32)
        on.check("initial_state", initial_state, torch.float32, states)
        on.check("last_state", last_state, torch.float32, states)
        ref = ctypes.byref(dims)
        keep, ws, nbytes = on.workspace(workspace, lib().linear_attention_workspace_size(ref))
        st = lib().linear_attention_fwd(_p(q), _p(k), _p(v), _p(log_decay), _p(o), _p(initial_state), _p(last_state), ref,
                                        ws, nbytes, on.handle)
        if st != SELSCAN_OK:
            raise SelscanError(st, "linear_attention_fwd")
    return o, last_state


def linear_attention_bwd(q, k, v, log_decay, *, do, scale: float = 1.0, initial_state=None, dlast_state=None,
                         decay_grad: bool = True, workspace=None, stream=None) -> dict:
    """Gradients of linear_attention_fwd (same inputs and options) given do ([batch, L, H, V]) and
    optionally dlast_state.  Returns a dict of contiguous tensors: dq, dk, dv in q's dtype; dlog_decay
    (unless decay_grad is False, which leaves the others as they are) in log_decay's shape and, with an
    initial_state, dinitial_state in float32."""
    import torch
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q and v must be [batch, L, heads, width]")
    with _On(q, stream) as on:
        dims = _linattn_dims(on, q, k, v, log_decay, do, scale)
        states = (dims.batch, dims.nheads, dims.dk, dims.dv)
        on.check("initial_state", initial_state, torch.float32, states)
        on.check("dlast_state", dlast_state, torch.float32, states)
        new = lambda shape, dtype: q.new_empty(shape, dtype=dtype)      # noqa: E731
        out = {"dq": new(q.shape, q.dtype), "dk": new(q.shape, q.dtype), "dv": new(v.shape, q.dtype)}
        if decay_grad:
            out["dlog_decay"] = new(log_decay.shape, torch.float32)
        if initial_state is not None:
            out["dinitial_state"] = new(states, torch.float32)
        ref = ctypes.byref(dims)
        keep, ws, nbytes = on.workspace(workspace, lib().linear_attention_bwd_workspace_size(ref, 1 if decay_grad else 0))
        st = lib().linear_attention_bwd(_p(q), _p(k), _p(v), _p(log_decay), _p(initial_state), _p(do), _p(dlast_state),
                                        _p(out["dq"]), _p(out["dk"]), _p(out["dv"]), _p(out.get("dlog_decay")),
                                        _p(out.get("dinitial_state")), ref, ws, nbytes, on.handle)
        if st != SELSCAN_OK:
            raise SelscanError(st, "linear_attention_bwd")
    return out


def linear_attention_step(q, k, v, log_decay, *, state, scale: float = 1.0, o=None, read_slots=None, write_slots=None,
                          stream=None):
    """One token of linear attention per batch row.  q, k: [batch, Hk, K]; v, o: [batch, H, V];
    log_decay: [H] or [batch, H]; state: [slots, H, K, V] float32, contiguous.  Without ids row b's
    state is slot b, updated in place; with them ([batch] int32) row b starts from slot read_slots[b]
    (the zero state where the id is outside) and stores the new state in slot write_slots[b]; rows
    whose write id is outside are padding and keep their o.  A slot that a row writes may be read
    by that row alone.  Returns o."""
    import torch
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q and v must be [batch, heads, width] (one token per batch row)")
    with _On(q, stream) as on:
        if o is None:
            o = q.new_empty(v.shape)
        dims = _linattn_dims(on, q, k, v, log_decay, o, scale, step=True)
        slots = state.shape[0]
        on.check("state", state, torch.float32, (slots, dims.nheads, dims.dk, dims.dv))
        on.check("read_slots", read_slots, torch.int32, (dims.batch,))
        on.check("write_slots", write_slots, torch.int32, (dims.batch,))
        st = lib().linear_attention_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), o.data_ptr(),
                                         state.data_ptr(), slots, _p(read_slots), _p(write_slots), ctypes.byref(dims),
                                         on.handle)
        if st != SELSCAN_OK:
            raise SelscanError(st, "linear_attention_step")
    return o


def _norm_dims(on, x, weight, bias, z, y, groups, eps, activation):
    """selscan_norm_dims of [batch, L, C] or [rows, C] tensors with unit-stride channels."""
    import torch
    if x.dim() not in (2, 3):
        raise ValueError("x must be [batch, L, C] or [rows, C]")
    io, shape = x.dtype, x.shape
    C = shape[-1]
    sx, sz, sy = x.stride(), (0, 0, 1), y.stride()
    if z is not None:
        on.check("z", z, io, shape, contiguous=False)
        sz = z.stride()
    on.check("y", y, io, shape, contiguous=False)
    if C > 1 and not sx[-1] == sz[-1] == sy[-1] == 1:
        raise ValueError("x, z and y: the channel axis must be unit-stride")
    strides = sx[:2] + sz[:2] + sy[:2] if len(shape) == 3 else (0, sx[0], 0, sz[0], 0, sy[0])
    on.check("weight", weight, torch.float32, (C,))
    on.check("bias", bias, torch.float32, (C,))
    batch, L = (1, shape[0]) if len(shape) == 2 else shape[:2]
    return NormDims(SELSCAN_ABI_VERSION, _io_code(io), batch, L, C, groups, *strides, eps, ACTIVATIONS[activation])


def group_norm_fwd(x, weight=None, bias=None, z=None, *, groups: int, eps: float = 1e-5, activation: str = "silu", y=None,
                   stream=None):
    """Group norm with an activation, channels last: each token's groups of C / groups channels are
    normalised for themselves, n = (x - mean) / sqrt(var + eps) * weight + bias; y = act(n), or with a
    gate z  y = n * act(z).  Returns y.

    x, z, y: [batch, L, C] or [rows, C] float32 or bfloat16 (unit-stride channels; y may be x or z);
    weight, bias: [C] float32 or None; activation: "silu" or "none"."""
    with _On(x, stream) as on:
        if y is None:
            y = x.new_empty(x.shape)
        dims = _norm_dims(on, x, weight, bias, z, y, groups, eps, activation)
        st = lib().group_norm_fwd(_p(x), _p(weight), _p(bias), _p(z), _p(y), ctypes.byref(dims), on.handle)
        if st != SELSCAN_OK:
            raise SelscanError(st, "group_norm_fwd")
    return y


def group_norm_bwd(x, weight=None, bias=None, z=None, *, dy, groups: int, eps: float = 1e-5, activation: str = "silu",
                   workspace=None, stream=None) -> dict:
    """Gradients of group_norm_fwd (same inputs and options) given dy.  Returns a dict: dx and (with a
    gate) dz, contiguous in x's dtype; dweight, dbias [C] float32 where weight and bias were given."""
    import torch
    with _On(x, stream) as on:
        dims = _norm_dims(on, x, weight, bias, z, dy, groups, eps, activation)
        C = (x.shape[-1],)
        out = {"dx": x.new_empty(x.shape)}
        if z is not None:
            out["dz"] = x.new_empty(x.shape)
        for name, t in (("dweight", weight), ("dbias", bias)):
            if t is not None:
                out[name] = x.new_empty(C, dtype=torch.float32)
        ref = ctypes.byref(dims)
        need = lib().group_norm_bwd_workspace_size(ref) if weight is not None or bias is not None else 0
        keep, ws, nbytes = on.workspace(workspace, need)
        st = lib().group_norm_bwd(_p(x), _p(weight), _p(bias), _p(z), _p(dy), _p(out["dx"]), _p(out.get("dweight")),
                                  _p(out.get("dbias")), _p(out.get("dz")), ref, ws, nbytes, on.handle)
        if st != SELSCAN_OK:
            raise SelscanError(st, "group_norm_bwd")
    return out


__all__ = ["selective_scan_fwd", "selective_scan_step", "selective_scan_bwd", "bwd_workspace_size",
           "selective_scan_ssd_fwd", "ssd_dims", "ssd_workspace_size", "SsdDims",
           "gated_scan_fwd", "gated_scan_bwd", "gated_scan_step", "gated_checkpoints", "GatedDims", "GATED_TILE",
           "state_cache", "state_cache_write", "state_cache_read", "CacheDims", "CACHE_ROW",
           "linear_attention_fwd", "linear_attention_bwd", "linear_attention_step", "LinattnDims",
           "group_norm_fwd", "group_norm_bwd", "NormDims", "ACTIVATIONS",
           "selective_scan_step_cached", "selective_scan_ssd_step_cached", "make_dims", "dims_init", "workspace_size", "strerror", "last_hip_error",
           "abi_version", "lib", "SelscanDims", "SelscanError", "LIB_PATH"]
