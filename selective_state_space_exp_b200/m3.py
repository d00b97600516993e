"""Thin Python binding of libm3.so (the C ABI in include/m3.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  torch supplies device memory and the current stream.  There is no
fallback: if the library is missing or the tensors are not on a CUDA device,
the calls raise.

The norm, head-loss and 4-bit calls (m3_group_norm_*, m3_linear_xent_*,
m3_linear_w4, m3_w4_quantize) take stream=: the call then runs on that stream,
its outputs and workspace are made in that stream's memory pool (the calls of the
layer make theirs in the current stream's), and every tensor of the call is
recorded on both streams.  The caller orders the streams: the inputs' making
before the call, and the call before its results are used.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# M3_LIBRARY=debug selects the bounds-checked build (lib/libm3_debug.so, see
# _build.build(debug=True)), whose kernels report M3_ERR_BOUNDS.
LIB_PATH = os.path.join(_PKG, "lib", "libm3_debug.so" if os.environ.get("M3_LIBRARY") == "debug"
                        else "libm3.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "m3.h")

M3_F32, M3_BF16 = 0, 1
M3_FLAG_SIMT = 1
M3_FLAG_TEST_TIMEOUT = 2
M3_FLAG_THETA_PER_HEAD = 4
M3_FLAG_DY_F32 = 8
M3_ACT_NONE, M3_ACT_SILU, M3_ACT_GATE = 0, 1, 2
_ACTS = {"none": M3_ACT_NONE, "silu": M3_ACT_SILU, "gate": M3_ACT_GATE}
M3_OK, M3_ERR_INVALID_ARGUMENT, M3_ERR_TIMEOUT = 0, -1, -6


def theta_flag(theta_groups: int, ngroups: int, nheads: int) -> int:
    """M3_FLAG_THETA_PER_HEAD when theta's group dimension is the head count
    (and differs from the B/C group count), 0 when it is the group count."""
    if theta_groups == ngroups:
        return 0
    if theta_groups == nheads:
        return M3_FLAG_THETA_PER_HEAD
    raise ValueError(f"theta has {theta_groups} groups: expected {ngroups} or {nheads}")


STATUS = {0: "M3_OK", -1: "M3_ERR_INVALID_ARGUMENT", -2: "M3_ERR_UNSUPPORTED",
          -3: "M3_ERR_ALIGNMENT", -4: "M3_ERR_WORKSPACE", -5: "M3_ERR_CUDA",
          -6: "M3_ERR_TIMEOUT", -7: "M3_ERR_BOUNDS"}


class M3Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {status} ({STATUS.get(status, 'unknown')})")
        self.status = status


class Shape(ctypes.Structure):
    """m3_shape."""
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("nheads", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("headdim", ctypes.c_int64), ("dstate", ctypes.c_int64),
                ("rank", ctypes.c_int64), ("chunk", ctypes.c_int64),
                ("io_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class NormShape(ctypes.Structure):
    """m3_norm_shape."""
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("channels", ctypes.c_int64), ("groups", ctypes.c_int64),
                ("io_dtype", ctypes.c_int32), ("act", ctypes.c_int32), ("eps", ctypes.c_float)]


_lib = None
_lock = threading.Lock()


def load() -> ctypes.CDLL:
    """Load libm3.so (built by __graft_entry__.build() or _build.py)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"library not built ({LIB_PATH}); run selective_state_space_exp_b200/_build.py")
            L = ctypes.CDLL(LIB_PATH)
            vp, sp = ctypes.c_void_p, ctypes.POINTER(Shape)
            L.m3_version.restype = ctypes.c_char_p
            L.m3_status_string.restype = ctypes.c_char_p
            L.m3_status_string.argtypes = [ctypes.c_int]
            L.m3_check_shape.argtypes = [sp]
            L.m3_check_shape.restype = ctypes.c_int
            L.m3_scan_workspace_size.argtypes = [sp, ctypes.POINTER(ctypes.c_size_t)]
            L.m3_scan_workspace_size.restype = ctypes.c_int
            L.m3_scan_workspace_bytes.argtypes = [sp]
            L.m3_scan_workspace_bytes.restype = ctypes.c_size_t
            L.m3_scan_plan.argtypes = [sp, ctypes.POINTER(ctypes.c_int),
                                       ctypes.POINTER(ctypes.c_int64),
                                       ctypes.POINTER(ctypes.c_int)]
            L.m3_scan_plan.restype = ctypes.c_int
            L.m3_scan_fwd.argtypes = [sp] + [vp] * 13 + [ctypes.c_size_t, vp]
            L.m3_scan_fwd.restype = ctypes.c_int
            L.m3_scan_fwd_noalloc.argtypes = [sp] + [vp] * 13
            L.m3_scan_fwd_noalloc.restype = ctypes.c_int
            L.m3_decode_step.argtypes = [sp] + [vp] * 13
            L.m3_decode_step.restype = ctypes.c_int
            L.m3_stream_status.argtypes = [vp]
            L.m3_stream_status.restype = ctypes.c_int
            L.m3_scan_state_workspace_size.argtypes = [sp, ctypes.POINTER(ctypes.c_size_t)]
            L.m3_scan_state_workspace_size.restype = ctypes.c_int
            L.m3_scan_state.argtypes = [sp] + [vp] * 12 + [ctypes.c_size_t, vp]
            L.m3_scan_state.restype = ctypes.c_int
            L.m3_segment_totals.argtypes = [sp] + [vp] * 6
            L.m3_segment_totals.restype = ctypes.c_int
            L.m3_state_fold.argtypes = [sp, ctypes.c_int64] + [vp] * 6
            L.m3_state_fold.restype = ctypes.c_int
            L.m3_scan_fwd_varlen.argtypes = [sp, vp, ctypes.c_int64] + [vp] * 13 + \
                [ctypes.c_size_t, vp]
            L.m3_scan_fwd_varlen.restype = ctypes.c_int
            L.m3_scan_bwd_workspace_size.argtypes = [sp, ctypes.POINTER(ctypes.c_size_t)]
            L.m3_scan_bwd_workspace_size.restype = ctypes.c_int
            L.m3_scan_bwd.argtypes = [sp] + [vp] * 23 + [ctypes.c_size_t, vp]
            L.m3_scan_bwd.restype = ctypes.c_int
            L.m3_scan_bwd_varlen.argtypes = [sp, vp, ctypes.c_int64] + [vp] * 23 + \
                [ctypes.c_size_t, vp]
            L.m3_scan_bwd_varlen.restype = ctypes.c_int
            L.m3_bc_prep.argtypes = [sp] + [vp] * 6 + [ctypes.c_float, vp, vp, vp]
            L.m3_bc_prep.restype = ctypes.c_int
            L.m3_linear.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64] + [vp] * 4 + \
                [ctypes.c_int32, vp]
            L.m3_linear.restype = ctypes.c_int
            L.m3_mimo_up.argtypes = [sp] + [vp] * 4
            L.m3_mimo_up.restype = ctypes.c_int
            L.m3_mimo_down_gate.argtypes = [sp] + [vp] * 5
            L.m3_mimo_down_gate.restype = ctypes.c_int
            np_ = ctypes.POINTER(NormShape)
            L.m3_group_norm_workspace_size.argtypes = [np_, ctypes.c_int, ctypes.c_int,
                                                       ctypes.POINTER(ctypes.c_size_t)]
            L.m3_group_norm_fwd.argtypes = [np_] + [vp] * 8 + [ctypes.c_size_t, vp]
            L.m3_group_norm_fwd_varlen.argtypes = [np_, vp, ctypes.c_int64] + [vp] * 8 + \
                [ctypes.c_size_t, vp]
            L.m3_group_norm_bwd.argtypes = [np_] + [vp] * 12 + [ctypes.c_size_t, vp]
            L.m3_group_norm_bwd_varlen.argtypes = [np_, vp, ctypes.c_int64] + [vp] * 12 + \
                [ctypes.c_size_t, vp]
            i64 = ctypes.c_int64
            for name in ("m3_linear_xent_fwd_workspace_size", "m3_linear_xent_bwd_workspace_size"):
                getattr(L, name).argtypes = [i64] * 3 + [ctypes.POINTER(ctypes.c_size_t)]
            L.m3_linear_xent_bwd_workspace_size_for.argtypes = [i64] * 3 + [ctypes.c_int] * 2 + \
                [ctypes.POINTER(ctypes.c_size_t)]
            L.m3_linear_xent_fwd.argtypes = [i64] * 3 + [vp] * 3 + [i64] + [vp] * 3 + \
                [ctypes.c_size_t, vp]
            L.m3_linear_xent_bwd.argtypes = [i64] * 3 + [vp] * 3 + [i64] + [vp] * 5 + \
                [ctypes.c_size_t, vp]
            L.m3_linear_w4.argtypes = [i64] * 3 + [ctypes.c_int32] + [vp] * 6 + \
                [ctypes.c_int32, vp]
            L.m3_w4_quantize.argtypes = [i64] * 2 + [ctypes.c_int32] * 2 + [vp] * 5
            for name in ("m3_group_norm_workspace_size", "m3_group_norm_fwd",
                         "m3_group_norm_fwd_varlen", "m3_group_norm_bwd",
                         "m3_group_norm_bwd_varlen", "m3_linear_xent_fwd_workspace_size",
                         "m3_linear_xent_bwd_workspace_size",
                         "m3_linear_xent_bwd_workspace_size_for", "m3_linear_xent_fwd",
                         "m3_linear_xent_bwd", "m3_linear_w4", "m3_w4_quantize"):
                getattr(L, name).restype = ctypes.c_int
            _lib = L
    return _lib


def _check(fn: str, st: int):
    if st != 0:
        raise M3Error(fn, st)


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _io_code(dtype: torch.dtype) -> int:
    if dtype == torch.bfloat16:
        return M3_BF16
    if dtype == torch.float32:
        return M3_F32
    raise ValueError(f"unsupported io dtype {dtype}")


def make_shape(batch, seqlen, nheads, ngroups, headdim, dstate, rank, chunk, io_dtype,
               simt=False) -> Shape:
    return Shape(batch, seqlen, nheads, ngroups, headdim, dstate, rank, chunk,
                 _io_code(io_dtype) if isinstance(io_dtype, torch.dtype) else int(io_dtype),
                 M3_FLAG_SIMT if simt else 0)


def scan_shape(x: torch.Tensor, B: torch.Tensor, chunk: int, simt=False, theta=None) -> Shape:
    """Shape of a scan call; theta (if given) decides grouped or per-head rates."""
    b, L, H, R, P = x.shape
    G, N = B.shape[2], B.shape[4]
    s = make_shape(b, L, H, G, P, N, R, chunk, x.dtype, simt)
    if theta is not None:
        s.flags |= theta_flag(theta.shape[2], G, H)
    return s


def workspace_size(shape: Shape) -> int:
    n = ctypes.c_size_t(0)
    _check("m3_scan_workspace_size", load().m3_scan_workspace_size(ctypes.byref(shape),
                                                                   ctypes.byref(n)))
    return int(n.value)


def scan_plan(shape: Shape) -> dict:
    """How m3_scan_fwd runs `shape`: tensor_core (bool), segments, launches."""
    tc, seg, n = ctypes.c_int(), ctypes.c_int64(), ctypes.c_int()
    _check("m3_scan_plan", load().m3_scan_plan(ctypes.byref(shape), ctypes.byref(tc),
                                               ctypes.byref(seg), ctypes.byref(n)))
    return {"tensor_core": bool(tc.value), "segments": int(seg.value), "launches": int(n.value)}


def m3_scan_fwd(x, dt, A, lam, theta, B, C, chunk: int = 64, h0=None, B_prev=None,
                x_prev=None, *, y=None, final_state=None, want_final=True, workspace=None,
                simt=False, stream=None, extra_flags=0):
    """Chunked prefill scan.  x [b][L][H][R][P] (io dtype), dt/A/lam [b][L][H],
    theta [b][L][G][N/2] fp32, B/C [b][L][G][R][N] (io dtype).  R is x.shape[3].
    extra_flags: further M3_FLAG_* bits (diagnostics).  Returns (y, final_state)."""
    shape = scan_shape(x, B, chunk, simt, theta)
    shape.flags |= extra_flags
    if y is None:
        y = torch.empty_like(x)
    if final_state is None and want_final:
        final_state = torch.empty((x.shape[0], x.shape[2], B.shape[4], x.shape[4]),
                                  dtype=torch.float32, device=x.device)
    need = workspace_size(shape)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    st = load().m3_scan_fwd(ctypes.byref(shape), _ptr(x), _ptr(dt), _ptr(A), _ptr(lam),
                            _ptr(theta), _ptr(B), _ptr(C), _ptr(h0), _ptr(B_prev),
                            _ptr(x_prev), _ptr(y), _ptr(final_state), _ptr(workspace),
                            ctypes.c_size_t(workspace.numel()), _stream(stream))
    _check("m3_scan_fwd", st)
    return y, final_state


def m3_scan_fwd_varlen(cu_seqlens, x, dt, A, lam, theta, B, C, chunk: int = 64, h0=None,
                       B_prev=None, x_prev=None, *, max_seqlen=None, y=None, final_state=None,
                       want_final=True, workspace=None, simt=False, stream=None):
    """Packed batch of S independent sequences: cu_seqlens [S+1] int32 on the
    device (sequence i is token rows cu_seqlens[i]:cu_seqlens[i+1]); x [T][H][R][P],
    dt/A/lam [T][H], theta [T][G][N/2], B/C [T][G][R][N]; h0 [S][H][N][P],
    B_prev [S][G][R][N], x_prev [S][H][R][P].  max_seqlen bounds every
    sequence's length (read from cu_seqlens, with a device sync, when None).
    Returns (y [T][H][R][P], final_state [S][H][N][P])."""
    if cu_seqlens.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")
    S = cu_seqlens.numel() - 1
    T, H, R, P = x.shape
    G, N = B.shape[1], B.shape[3]
    if max_seqlen is None:
        max_seqlen = int((cu_seqlens[1:] - cu_seqlens[:-1]).max().item()) if S > 0 else 0
    shape = make_shape(S, max_seqlen, H, G, P, N, R, chunk, x.dtype, simt)
    shape.flags |= theta_flag(theta.shape[1], G, H)
    if y is None:
        y = torch.empty_like(x)
    if final_state is None and want_final:
        final_state = torch.empty((S, H, N, P), dtype=torch.float32, device=x.device)
    need = workspace_size(shape)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    st = load().m3_scan_fwd_varlen(ctypes.byref(shape), _ptr(cu_seqlens), ctypes.c_int64(T),
                                   _ptr(x), _ptr(dt), _ptr(A), _ptr(lam), _ptr(theta), _ptr(B),
                                   _ptr(C), _ptr(h0), _ptr(B_prev), _ptr(x_prev), _ptr(y),
                                   _ptr(final_state), _ptr(workspace),
                                   ctypes.c_size_t(workspace.numel()), _stream(stream))
    _check("m3_scan_fwd_varlen", st)
    return y, final_state


def m3_bc_prep(B_raw=None, C_raw=None, B_weight=None, B_bias=None, C_weight=None, C_bias=None,
               eps: float = 1e-6, *, B=None, C=None, stream=None):
    """QK-norm + per-channel scale + bias of raw B / C projections, either
    [b][L][G][R][N] (scan layout) or [b][G][R][N] (decode layout), io dtype.
    weight / bias [G][R][N] fp32 or None.  Returns (B, C) (None for a skipped one)."""
    ref = B_raw if B_raw is not None else C_raw
    if ref.dim() == 5:
        b, L, G, R, N = ref.shape
    else:
        (b, G, R, N), L = ref.shape, 1
    if B_raw is not None and B is None:
        B = torch.empty_like(B_raw)
    if C_raw is not None and C is None:
        C = torch.empty_like(C_raw)
    shape = make_shape(b, L, G, G, 16, N, R, 64, ref.dtype)
    st = load().m3_bc_prep(ctypes.byref(shape), _ptr(B_raw), _ptr(C_raw), _ptr(B_weight),
                           _ptr(B_bias), _ptr(C_weight), _ptr(C_bias), ctypes.c_float(eps),
                           _ptr(B), _ptr(C), _stream(stream))
    _check("m3_bc_prep", st)
    return B, C


def dy_flag(dy: torch.Tensor, x: torch.Tensor) -> int:
    """M3_FLAG_DY_F32 when dy is fp32 and the io dtype is not; otherwise dy
    must have x's dtype."""
    if dy.dtype == x.dtype:
        return 0
    if dy.dtype == torch.float32:
        return M3_FLAG_DY_F32
    raise TypeError(f"dy is {dy.dtype}: expected {x.dtype} or torch.float32")


def bwd_workspace_size(shape: Shape) -> int:
    n = ctypes.c_size_t(0)
    _check("m3_scan_bwd_workspace_size",
           load().m3_scan_bwd_workspace_size(ctypes.byref(shape), ctypes.byref(n)))
    return int(n.value)


def m3_scan_bwd(x, dt, A, lam, theta, B, C, dy, chunk: int = 64, h0=None, B_prev=None,
                x_prev=None, d_final=None, *, want_dh0=True, workspace=None, simt=False,
                stream=None):
    """Backward of m3_scan_fwd: gradients of sum(y * dy) + sum(final * d_final)
    with respect to every input.  dy has x's dtype, or fp32 (read unrounded).
    Returns a dict of fp32 tensors: x, dt, A, lam, theta, B, C, and h0 (when
    want_dh0), B_prev and x_prev (when B_prev is given), each in its input's
    layout.  bf16 io at N = 128, P = 64 runs on the tensor cores (bf16
    operands) unless simt is set (CUDA cores, fp32 throughout)."""
    shape = scan_shape(x, B, chunk, simt, theta)
    shape.flags |= dy_flag(dy, x)
    dev, f32 = x.device, torch.float32
    g = {"x": torch.empty(x.shape, dtype=f32, device=dev),
         "dt": torch.empty(dt.shape, dtype=f32, device=dev),
         "A": torch.empty(A.shape, dtype=f32, device=dev),
         "lam": torch.empty(lam.shape, dtype=f32, device=dev),
         "theta": torch.empty(theta.shape, dtype=f32, device=dev),
         "B": torch.empty(B.shape, dtype=f32, device=dev),
         "C": torch.empty(C.shape, dtype=f32, device=dev)}
    if want_dh0:
        g["h0"] = torch.empty((x.shape[0], x.shape[2], B.shape[4], x.shape[4]), dtype=f32,
                              device=dev)
    if B_prev is not None:
        g["B_prev"] = torch.empty(B_prev.shape, dtype=f32, device=dev)
        g["x_prev"] = torch.empty(x_prev.shape, dtype=f32, device=dev)
    need = bwd_workspace_size(shape)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    st = load().m3_scan_bwd(ctypes.byref(shape), _ptr(x), _ptr(dt), _ptr(A), _ptr(lam),
                            _ptr(theta), _ptr(B), _ptr(C), _ptr(h0), _ptr(B_prev), _ptr(x_prev),
                            _ptr(dy), _ptr(d_final), _ptr(g["x"]), _ptr(g["dt"]), _ptr(g["A"]),
                            _ptr(g["lam"]), _ptr(g["theta"]), _ptr(g["B"]), _ptr(g["C"]),
                            _ptr(g.get("h0")), _ptr(g.get("B_prev")), _ptr(g.get("x_prev")),
                            _ptr(workspace), ctypes.c_size_t(workspace.numel()), _stream(stream))
    _check("m3_scan_bwd", st)
    return g


def m3_scan_bwd_varlen(cu_seqlens, x, dt, A, lam, theta, B, C, dy, chunk: int = 64, h0=None,
                       B_prev=None, x_prev=None, d_final=None, *, max_seqlen=None,
                       want_dh0=True, workspace=None, simt=False, stream=None):
    """Backward of m3_scan_fwd_varlen (packed tensors without a batch
    dimension, as there).  Returns the gradient dict of m3_scan_bwd; simt as
    there."""
    if cu_seqlens.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")
    S = cu_seqlens.numel() - 1
    T, H, R, P = x.shape
    G, N = B.shape[1], B.shape[3]
    if max_seqlen is None:
        max_seqlen = int((cu_seqlens[1:] - cu_seqlens[:-1]).max().item()) if S > 0 else 0
    shape = make_shape(S, max_seqlen, H, G, P, N, R, chunk, x.dtype, simt)
    shape.flags |= theta_flag(theta.shape[1], G, H) | dy_flag(dy, x)
    dev, f32 = x.device, torch.float32
    g = {k: torch.empty(v.shape, dtype=f32, device=dev)
         for k, v in (("x", x), ("dt", dt), ("A", A), ("lam", lam), ("theta", theta), ("B", B),
                      ("C", C))}
    if want_dh0:
        g["h0"] = torch.empty((S, H, N, P), dtype=f32, device=dev)
    if B_prev is not None:
        g["B_prev"] = torch.empty(B_prev.shape, dtype=f32, device=dev)
        g["x_prev"] = torch.empty(x_prev.shape, dtype=f32, device=dev)
    need = bwd_workspace_size(shape)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    st = load().m3_scan_bwd_varlen(
        ctypes.byref(shape), _ptr(cu_seqlens), ctypes.c_int64(T), _ptr(x), _ptr(dt), _ptr(A),
        _ptr(lam), _ptr(theta), _ptr(B), _ptr(C), _ptr(h0), _ptr(B_prev), _ptr(x_prev), _ptr(dy),
        _ptr(d_final), _ptr(g["x"]), _ptr(g["dt"]), _ptr(g["A"]), _ptr(g["lam"]),
        _ptr(g["theta"]), _ptr(g["B"]), _ptr(g["C"]), _ptr(g.get("h0")), _ptr(g.get("B_prev")),
        _ptr(g.get("x_prev")), _ptr(workspace), ctypes.c_size_t(workspace.numel()),
        _stream(stream))
    _check("m3_scan_bwd_varlen", st)
    return g


def m3_scan_fwd_noalloc(x, dt, A, lam, theta, B, C, chunk: int = 64, h0=None, B_prev=None,
                        x_prev=None, *, y=None, final_state=None, want_final=True, simt=False,
                        stream=None):
    """m3_scan_fwd without a workspace argument: the library's fixed device
    scratch (M3_NOALLOC_SCRATCH_BYTES) serves instead, for callers that cannot
    allocate device memory.  Returns (y, final_state)."""
    shape = scan_shape(x, B, chunk, simt, theta)
    if y is None:
        y = torch.empty_like(x)
    if final_state is None and want_final:
        final_state = torch.empty((x.shape[0], x.shape[2], B.shape[4], x.shape[4]),
                                  dtype=torch.float32, device=x.device)
    st = load().m3_scan_fwd_noalloc(ctypes.byref(shape), _ptr(x), _ptr(dt), _ptr(A), _ptr(lam),
                                    _ptr(theta), _ptr(B), _ptr(C), _ptr(h0), _ptr(B_prev),
                                    _ptr(x_prev), _ptr(y), _ptr(final_state), _stream(stream))
    _check("m3_scan_fwd_noalloc", st)
    return y, final_state


def m3_scan_state(x, dt, A, lam, theta, B, C, chunk: int = 64, h0=None, B_prev=None,
                  x_prev=None, *, final_state=None, workspace=None, simt=False, stream=None):
    """The state after every sequence's last token, [b][H][N][P] fp32, without y."""
    shape = scan_shape(x, B, chunk, simt, theta)
    if final_state is None:
        final_state = torch.empty((x.shape[0], x.shape[2], B.shape[4], x.shape[4]),
                                  dtype=torch.float32, device=x.device)
    n = ctypes.c_size_t(0)
    _check("m3_scan_state_workspace_size",
           load().m3_scan_state_workspace_size(ctypes.byref(shape), ctypes.byref(n)))
    if workspace is None:
        workspace = torch.empty(max(int(n.value), 1), dtype=torch.uint8, device=x.device)
    st = load().m3_scan_state(ctypes.byref(shape), _ptr(x), _ptr(dt), _ptr(A), _ptr(lam),
                              _ptr(theta), _ptr(B), _ptr(C), _ptr(h0), _ptr(B_prev),
                              _ptr(x_prev), _ptr(final_state), _ptr(workspace),
                              ctypes.c_size_t(workspace.numel()), _stream(stream))
    _check("m3_scan_state", st)
    return final_state


def m3_segment_totals(x, dt, A, theta, B, chunk: int = 64, *, stream=None):
    """(lam_tot [b][H], phi_tot [b][H][N/2]): sum over the tokens of dt*A and
    of dt*theta for every (batch, head)."""
    shape = scan_shape(x, B, chunk, False, theta)
    b, _, H = dt.shape
    K = B.shape[4] // 2
    lam_tot = torch.empty((b, H), dtype=torch.float32, device=dt.device)
    phi_tot = torch.empty((b, H, K), dtype=torch.float32, device=dt.device)
    _check("m3_segment_totals", load().m3_segment_totals(
        ctypes.byref(shape), _ptr(dt), _ptr(A), _ptr(theta), _ptr(lam_tot), _ptr(phi_tot),
        _stream(stream)))
    return lam_tot, phi_tot


def m3_state_fold(h0, T, lam_tot, phi_tot, *, out=None, stream=None):
    """Fold segment summaries: h = h0 (None: zero); for each s:
    h = Rot(phi_tot[s]) exp(lam_tot[s]) h + T[s].  T [nseg][b][H][N][P]."""
    nseg, b, H, N, P = T.shape
    shape = make_shape(b, 1, H, 1, P, N, 1, 64, torch.float32)
    if out is None:
        out = torch.empty((b, H, N, P), dtype=torch.float32, device=T.device)
    _check("m3_state_fold", load().m3_state_fold(
        ctypes.byref(shape), ctypes.c_int64(nseg), _ptr(h0), _ptr(T) if nseg else None,
        _ptr(lam_tot) if nseg else None, _ptr(phi_tot) if nseg else None, _ptr(out),
        _stream(stream)))
    return out


def m3_decode_step(state, x_t, dt, A, lam, theta, B_t, C_t, B_prev=None, x_prev=None, *,
                   state_out=None, y=None, stream=None):
    """One decode step.  state [b][H][N][P] fp32; x_t [b][H][R][P]; dt/A/lam [b][H];
    theta [b][G][N/2] (or [b][H][N/2], per head); B_t/C_t [b][G][R][N].
    state_out defaults to `state` (in place).  Returns (y_t, state_out)."""
    b, H, R, P = x_t.shape
    G, N = B_t.shape[1], B_t.shape[3]
    shape = make_shape(b, 1, H, G, P, N, R, 64, x_t.dtype)
    shape.flags |= theta_flag(theta.shape[1], G, H)
    if state_out is None:
        state_out = state
    if y is None:
        y = torch.empty_like(x_t)
    st = load().m3_decode_step(ctypes.byref(shape), _ptr(state), _ptr(state_out), _ptr(x_t),
                               _ptr(dt), _ptr(A), _ptr(lam), _ptr(theta), _ptr(B_t),
                               _ptr(C_t), _ptr(B_prev), _ptr(x_prev), _ptr(y),
                               _stream(stream))
    _check("m3_decode_step", st)
    return y, state_out


def m3_stream_status(stream=None) -> int:
    """Synchronise the stream and return the first device-side status."""
    return int(load().m3_stream_status(_stream(stream)))


def version() -> str:
    return load().m3_version().decode()


# ---- block projections around the layer ---------------------------------------

def m3_linear(A, W, bias=None, *, out=None, out_dtype=torch.bfloat16, stream=None):
    """out = A W^T (+ bias) on the tensor cores: A [..][K] bf16 (rows are
    tokens), W [N][K] bf16, bias [N] fp32; returns out [..][N] in out_dtype
    (bf16 or fp32)."""
    if A.dtype != torch.bfloat16 or W.dtype != torch.bfloat16:
        raise TypeError("m3_linear takes bf16 A and W")
    K = A.shape[-1]
    M = A.numel() // K if K else 0
    N = W.shape[0]
    if W.shape[1] != K:
        raise ValueError(f"W is {tuple(W.shape)}, expected [N][{K}]")
    if out is None:
        out = torch.empty(A.shape[:-1] + (N,), dtype=out_dtype, device=A.device)
    code = M3_F32 if out.dtype == torch.float32 else M3_BF16
    st = load().m3_linear(ctypes.c_int64(M), ctypes.c_int64(N), ctypes.c_int64(K), _ptr(A),
                          _ptr(W), _ptr(bias), _ptr(out), ctypes.c_int32(code), _stream(stream))
    _check("m3_linear", st)
    return out


def _tokens_shape(T, H, R, P, dtype):
    """m3_shape of a block step over T tokens (one sequence of T tokens; the
    scan-only fields get admissible placeholders)."""
    return make_shape(1, T, H, 1, P, 16, R, 64, dtype, False)


def m3_mimo_up(x, w_up, *, X=None, stream=None):
    """X[..][h][r][p] = x[..][h][p] * w_up[h][r][p]: x [..][H][P] io dtype,
    w_up [H][R][P] fp32; returns X [..][H][R][P]."""
    H, R, P = w_up.shape
    T = x.numel() // (H * P)
    if X is None:
        X = torch.empty(x.shape[:-1] + (R, P), dtype=x.dtype, device=x.device)
    shape = _tokens_shape(T, H, R, P, x.dtype)
    st = load().m3_mimo_up(ctypes.byref(shape), _ptr(x), _ptr(w_up), _ptr(X), _stream(stream))
    _check("m3_mimo_up", st)
    return X


def m3_mimo_down_gate(Y, w_down, z=None, *, out=None, stream=None):
    """out[..][h][p] = (sum_r Y[..][h][r][p] w_down[h][r][p]) * silu(z[..][h][p]):
    Y [..][H][R][P] io dtype, w_down [H][R][P] fp32, z [..][H][P] io dtype or
    None (no gate); returns out [..][H][P]."""
    H, R, P = w_down.shape
    T = Y.numel() // (H * R * P)
    if out is None:
        out = torch.empty(Y.shape[:-2] + (P,), dtype=Y.dtype, device=Y.device)
    shape = _tokens_shape(T, H, R, P, Y.dtype)
    st = load().m3_mimo_down_gate(ctypes.byref(shape), _ptr(Y), _ptr(w_down), _ptr(z), _ptr(out),
                                  _stream(stream))
    _check("m3_mimo_down_gate", st)
    return out


# ---- operators between the layer and a model's tokens ---------------------------
# Their calls can be as short as a few microseconds on the device, so the
# marshalling below keeps to plain integers and looks shapes and workspace sizes
# up once per set of extents.
#
# With stream=, tensors are recorded on that stream and on the current one, so each
# may be let go as soon as its last use is launched.

def _stream_on(stream, device):
    """Handle of `stream`, or of the current stream of `device`."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return stream.cuda_stream


def _elsewhere(stream, device):
    """The context a call has to be made in, or None where the current one will
    do.  Outputs and workspaces are made inside it, so with an explicit stream
    their memory belongs to that stream."""
    if stream is not None:
        return torch.cuda.stream(stream)
    if device.index == torch.cuda.current_device():
        return None
    return torch.cuda.device(device)


def _share(stream, device, *tensors):
    """Of a call on an explicit stream: the memory of its tensors is not given
    out again before what that stream, and the current one, do with them."""
    here = torch.cuda.current_stream(device)
    if here == stream:
        return
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
            t.record_stream(here)


def _device_of(t):
    if not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    return t.device


def _addr(name, t, dtype, shape, device):
    """Address of t after checks of its type, shape, device and layout; None passes."""
    if t is None:
        return None
    if (t.dtype is dtype and t.shape == shape and t.get_device() == device.index and
            t.is_contiguous()):
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name} is {t.dtype}: expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} is {tuple(t.shape)}: expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}: expected {device}")
    raise ValueError(f"{name} must be contiguous")


def _rows(n, width, dtype, device):
    """A new [n][width] (the quickest of torch's ways to make one)."""
    return torch.empty_strided((n, width), (width, 1), dtype=dtype, device=device)


def _scratch(nbytes, workspace, device):
    """(address, bytes, the tensor to keep alive) of a call's workspace."""
    if workspace is None:
        if nbytes == 0:
            return None, 0, None
        workspace = torch.empty_strided((nbytes,), (1,), dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


# ---- the grouped norm on the layer's output ------------------------------------

@functools.lru_cache(maxsize=4096)
def _norm_plan(batch, seqlen, channels, groups, dtype, act, eps, backward, packed):
    """(m3_norm_shape by reference, workspace bytes) of a call."""
    if act not in _ACTS:
        raise ValueError(f"act is {act!r}: expected one of {sorted(_ACTS)}")
    shape = NormShape(batch, seqlen, channels, groups, _io_code(dtype), _ACTS[act], eps)
    n = ctypes.c_size_t(0)
    _check("m3_group_norm_workspace_size", load().m3_group_norm_workspace_size(
        ctypes.byref(shape), int(backward), int(packed), ctypes.byref(n)))
    return ctypes.byref(shape), n.value


def _norm_extent(shape, groups, scope):
    """(samples, positions of each) of x [..][C]."""
    C = shape[-1] if shape else 0
    if groups < 1 or C < 1 or C % groups != 0:
        raise ValueError(f"{tuple(shape)} channels last do not split into {groups} groups")
    if scope == "token":
        return shape.numel() // C, 1
    if scope == "sequence":
        if len(shape) != 3:
            raise ValueError("scope 'sequence' takes x [batch][seqlen][channels]")
        return shape[0], shape[1]
    raise ValueError(f"scope is {scope!r}: expected 'token' or 'sequence'")


def _norm_forward(fn, plan, pre, x, stat, weight, bias, z, act, y, workspace, stream):
    shape, dt, dev = x.shape, x.dtype, _device_of(x)
    if (z is not None) != (act == "gate"):
        raise ValueError("z belongs to act 'gate', and only to it")
    args = (plan[0], *pre, _addr("x", x, dt, shape, dev),
            _addr("weight", weight, torch.float32, shape[-1:], dev),
            _addr("bias", bias, torch.float32, shape[-1:], dev), _addr("z", z, dt, shape, dev))
    st, ctx = _stream_on(stream, dev), _elsewhere(stream, dev)
    if ctx is not None:
        ctx.__enter__()
    try:
        if y is None:
            y = torch.empty_like(x)
            py = y.data_ptr()
        else:
            py = _addr("y", y, dt, shape, dev)
        mean = _rows(*stat, torch.float32, dev)
        rstd = _rows(*stat, torch.float32, dev)
        pws, nws, keep = _scratch(plan[1], workspace, dev)
        status = getattr(load(), fn)(*args, py, mean.data_ptr() or None, rstd.data_ptr() or None,
                                     pws, nws, st)
    finally:
        if ctx is not None:
            ctx.__exit__(None, None, None)
    if stream is not None:
        _share(stream, dev, x, weight, bias, z, y, mean, rstd, keep)
    if status:
        raise M3Error(fn, status)
    return y, mean, rstd


def _norm_backward(fn, plan, pre, x, stat, mean, rstd, dy, weight, bias, z, act, want, workspace,
                   stream):
    shape, dt, dev, f32 = x.shape, x.dtype, _device_of(x), torch.float32
    if (z is not None) != (act == "gate"):
        raise ValueError("z belongs to act 'gate', and only to it")
    args = (plan[0], *pre, _addr("x", x, dt, shape, dev),
            _addr("weight", weight, f32, shape[-1:], dev),
            _addr("bias", bias, f32, shape[-1:], dev), _addr("z", z, dt, shape, dev),
            _addr("mean", mean, f32, stat, dev), _addr("rstd", rstd, f32, stat, dev),
            _addr("dy", dy, dt, shape, dev))
    if dy is None or mean is None or rstd is None:
        raise ValueError("the backward takes mean, rstd and dy")
    st, ctx = _stream_on(stream, dev), _elsewhere(stream, dev)
    if ctx is not None:
        ctx.__enter__()
    try:
        dx = torch.empty_like(x) if want[0] else None
        dw = x.new_empty(shape[-1:], dtype=f32) if want[1] else None
        db = x.new_empty(shape[-1:], dtype=f32) if want[2] else None
        dz = torch.empty_like(x) if z is not None and want[3] else None
        g = {"x": dx, "weight": dw, "bias": db}
        if z is not None:
            g["z"] = dz
        pws, nws, keep = _scratch(plan[1], workspace, dev)
        status = getattr(load(), fn)(*args, dx is not None and dx.data_ptr() or None,
                                     dw is not None and dw.data_ptr() or None,
                                     db is not None and db.data_ptr() or None,
                                     dz is not None and dz.data_ptr() or None, pws, nws, st)
    finally:
        if ctx is not None:
            ctx.__exit__(None, None, None)
    if stream is not None:
        _share(stream, dev, x, weight, bias, z, mean, rstd, dy, *g.values(), keep)
    if status:
        raise M3Error(fn, status)
    return g


def m3_group_norm_fwd(x, groups: int, weight=None, bias=None, z=None, *, act="none",
                      eps: float = 1e-5, scope="token", y=None, workspace=None, stream=None):
    """Grouped norm with an activation, channels last: x [..][C] io dtype,
    statistics over the C / groups channels of every token (scope "token"), or
    over all positions of a sequence too (scope "sequence", x [b][L][C]).
    act "none", "silu", or "gate" (times silu(z), z like x); weight, bias [C]
    fp32 or None.  Returns (y, mean, rstd), the statistics [samples][groups]."""
    batch, seqlen = _norm_extent(x.shape, groups, scope)
    # no sample: to the library, one without positions
    plan = _norm_plan(batch or 1, seqlen if batch else 0, x.shape[-1], groups, x.dtype, act, eps,
                      False, False)
    return _norm_forward("m3_group_norm_fwd", plan, (), x, (batch, groups), weight, bias, z, act,
                         y, workspace, stream)


def m3_group_norm_bwd(x, groups: int, mean, rstd, dy, weight=None, bias=None, z=None, *,
                      act="none", scope="token", want_dx=True, want_dweight=True, want_dbias=True,
                      want_dz=True, workspace=None, stream=None):
    """Backward of m3_group_norm_fwd from its inputs and statistics: a dict of
    x and (act "gate") z in the io dtype, weight and bias fp32 [C] (None for one
    that is not wanted)."""
    batch, seqlen = _norm_extent(x.shape, groups, scope)
    plan = _norm_plan(batch or 1, seqlen if batch else 0, x.shape[-1], groups, x.dtype, act, 0.0,
                      True, False)
    return _norm_backward("m3_group_norm_bwd", plan, (), x, (batch, groups), mean, rstd, dy,
                          weight, bias, z, act, (want_dx, want_dweight, want_dbias, want_dz),
                          workspace, stream)


def _norm_packed(cu_seqlens, x, groups, max_seqlen):
    """(sequences, longest, the call's extra arguments) of a packed batch."""
    if x.dim() != 2:
        raise ValueError("a packed batch is x [tokens][channels]")
    _norm_extent(x.shape, groups, "token")
    S = cu_seqlens.numel() - 1
    if cu_seqlens.dim() != 1 or S < 1:
        raise ValueError("cu_seqlens holds no sequence")
    cu = _addr("cu_seqlens", cu_seqlens, torch.int32, cu_seqlens.shape, _device_of(x))
    if max_seqlen is None:
        max_seqlen = int((cu_seqlens[1:] - cu_seqlens[:-1]).max().item())
    return S, max_seqlen, (cu, x.shape[0])


def m3_group_norm_fwd_varlen(cu_seqlens, x, groups: int, weight=None, bias=None, z=None, *,
                             act="none", eps: float = 1e-5, max_seqlen=None, y=None,
                             workspace=None, stream=None):
    """m3_group_norm_fwd over the sequences of a packed batch: x [T][C],
    cu_seqlens [S+1] int32 on the device; max_seqlen as m3_scan_fwd_varlen.
    Rows of y outside every sequence are left as they are."""
    S, L, pre = _norm_packed(cu_seqlens, x, groups, max_seqlen)
    plan = _norm_plan(S, L, x.shape[1], groups, x.dtype, act, eps, False, True)
    out = _norm_forward("m3_group_norm_fwd_varlen", plan, pre, x, (S, groups), weight, bias, z,
                        act, y, workspace, stream)
    if stream is not None:
        _share(stream, x.device, cu_seqlens)
    return out


def m3_group_norm_bwd_varlen(cu_seqlens, x, groups: int, mean, rstd, dy, weight=None, bias=None,
                             z=None, *, act="none", max_seqlen=None, want_dx=True,
                             want_dweight=True, want_dbias=True, want_dz=True, workspace=None,
                             stream=None):
    """Backward of m3_group_norm_fwd_varlen (the dict of m3_group_norm_bwd);
    rows of dx and dz outside every sequence are undefined."""
    S, L, pre = _norm_packed(cu_seqlens, x, groups, max_seqlen)
    plan = _norm_plan(S, L, x.shape[1], groups, x.dtype, act, 0.0, True, True)
    out = _norm_backward("m3_group_norm_bwd_varlen", plan, pre, x, (S, groups), mean, rstd, dy,
                         weight, bias, z, act, (want_dx, want_dweight, want_dbias, want_dz),
                         workspace, stream)
    if stream is not None:
        _share(stream, x.device, cu_seqlens)
    return out


# ---- the head's cross entropy ---------------------------------------------------

@functools.lru_cache(maxsize=4096)
def _xent_bytes(tokens, vocab, width):
    """Workspace bytes of the forward."""
    n = ctypes.c_size_t(0)
    _check("m3_linear_xent_fwd_workspace_size",
           load().m3_linear_xent_fwd_workspace_size(tokens, vocab, width, ctypes.byref(n)))
    return n.value


@functools.lru_cache(maxsize=4096)
def _xent_bwd_bytes(tokens, vocab, width, want_dh, want_dW):
    """Workspace bytes of the backward for the gradients that are wanted."""
    n = ctypes.c_size_t(0)
    _check("m3_linear_xent_bwd_workspace_size_for",
           load().m3_linear_xent_bwd_workspace_size_for(tokens, vocab, width, int(want_dh),
                                                        int(want_dW), ctypes.byref(n)))
    return n.value


def _xent_args(h, W, targets):
    """(tokens, vocabulary, width, addresses of the three)."""
    if W.dim() != 2 or h.dim() < 1 or h.shape[-1] != W.shape[1]:
        raise ValueError(f"h is {tuple(h.shape)} and W {tuple(W.shape)}: expected [..][K], [V][K]")
    dev = _device_of(h)
    V, K = W.shape
    return (targets.numel(), V, K, _addr("h", h, torch.bfloat16, h.shape, dev),
            _addr("W", W, torch.bfloat16, W.shape, dev),
            _addr("targets", targets, torch.int64, h.shape[:-1], dev))


def m3_linear_xent_fwd(h, W, targets, *, ignore_index: int = -100, workspace=None, stream=None):
    """Softmax cross entropy of logits = h W^T, which are never stored: h [..][K]
    bf16, W [V][K] bf16, targets [..] int64 (ignore_index: not scored).  Returns
    (loss, lse), fp32 and shaped like targets."""
    args = _xent_args(h, W, targets)
    dev = h.device
    need = _xent_bytes(*args[:3])
    st, ctx = _stream_on(stream, dev), _elsewhere(stream, dev)
    if ctx is not None:
        ctx.__enter__()
    try:
        loss = torch.empty_like(targets, dtype=torch.float32)
        lse = torch.empty_like(targets, dtype=torch.float32)
        pws, nws, keep = _scratch(need, workspace, dev)
        status = load().m3_linear_xent_fwd(*args, ignore_index, loss.data_ptr(), lse.data_ptr(),
                                           pws, nws, st)
    finally:
        if ctx is not None:
            ctx.__exit__(None, None, None)
    if stream is not None:
        _share(stream, dev, h, W, targets, loss, lse, keep)
    if status:
        raise M3Error("m3_linear_xent_fwd", status)
    return loss, lse


def m3_linear_xent_bwd(h, W, targets, lse, dloss, *, ignore_index: int = -100, want_dh=True,
                       want_dW=True, workspace=None, stream=None):
    """Backward of m3_linear_xent_fwd: (dh, dW) bf16, the gradients of
    sum(loss * dloss) (None for one that is not wanted).  lse as the forward
    gave it, dloss fp32 shaped like targets."""
    args = _xent_args(h, W, targets)
    dev = h.device
    plse = _addr("lse", lse, torch.float32, targets.shape, dev)
    pdl = _addr("dloss", dloss, torch.float32, targets.shape, dev)
    need = _xent_bwd_bytes(*args[:3], bool(want_dh), bool(want_dW))
    st, ctx = _stream_on(stream, dev), _elsewhere(stream, dev)
    if ctx is not None:
        ctx.__enter__()
    try:
        dh = torch.empty_like(h) if want_dh else None
        dW = torch.empty_like(W) if want_dW else None
        pws, nws, keep = _scratch(need, workspace, dev)
        status = load().m3_linear_xent_bwd(*args, ignore_index, plse, pdl,
                                           dh.data_ptr() if want_dh else None,
                                           dW.data_ptr() if want_dW else None, pws, nws, st)
    finally:
        if ctx is not None:
            ctx.__exit__(None, None, None)
    if stream is not None:
        _share(stream, dev, h, W, targets, lse, dloss, dh, dW, keep)
    if status:
        raise M3Error("m3_linear_xent_bwd", status)
    return dh, dW


# ---- 4-bit weights ---------------------------------------------------------------

def m3_w4_quantize(W, group: int = 128, *, symmetric=False, stream=None):
    """W [N][K] (bf16 or fp32) in four bits with one scale for every `group`
    inputs: (codes [N][K/2] uint8, scales [N][K/group] bf16, zeros [N][K/group]
    uint8, or None when symmetric)."""
    if W.dim() != 2:
        raise ValueError(f"W is {tuple(W.shape)}: expected [N][K]")
    N, K = W.shape
    if group not in (32, 64, 128) or K % group != 0 or K == 0:
        raise ValueError(f"{K} inputs do not split into groups of {group} (32, 64 or 128)")
    dev = _device_of(W)
    code, pW = _io_code(W.dtype), _addr("W", W, W.dtype, W.shape, dev)
    st, ctx = _stream_on(stream, dev), _elsewhere(stream, dev)
    if ctx is not None:
        ctx.__enter__()
    try:
        codes = W.new_empty((N, K // 2), dtype=torch.uint8)
        scales = W.new_empty((N, K // group), dtype=torch.bfloat16)
        zeros = None if symmetric else W.new_empty((N, K // group), dtype=torch.uint8)
        status = load().m3_w4_quantize(N, K, group, code, pW, codes.data_ptr(), scales.data_ptr(),
                                       None if symmetric else zeros.data_ptr(), st)
    finally:
        if ctx is not None:
            ctx.__exit__(None, None, None)
    if stream is not None:
        _share(stream, dev, W, codes, scales, zeros)
    if status:
        raise M3Error("m3_w4_quantize", status)
    return codes, scales, zeros


def m3_linear_w4(A, codes, scales, zeros=None, bias=None, *, out=None, out_dtype=torch.bfloat16,
                 stream=None):
    """out = A W^T (+ bias) with W held in four bits (m3_w4_quantize's layout):
    A [..][K] bf16, codes [N][K/2] uint8, scales [N][K/group] bf16, zeros
    [N][K/group] uint8 or None (8); returns out [..][N] in out_dtype (bf16 or
    fp32)."""
    if codes.dim() != 2 or scales.dim() != 2:
        raise ValueError("codes and scales are [N][..]")
    N, half = codes.shape
    K, ng = 2 * half, scales.shape[1]
    shape = A.shape
    if not shape or shape[-1] != K:
        raise ValueError(f"A is {tuple(shape)}: expected [..][{K}]")
    if ng == 0 or K == 0 or K % ng != 0:
        raise ValueError(f"scales is {tuple(scales.shape)} for {K} inputs")
    dev = _device_of(A)
    if out is not None:
        out_dtype = out.dtype
    groups = (N, ng)
    args = (shape.numel() // K, N, K, K // ng, _addr("A", A, torch.bfloat16, shape, dev),
            _addr("codes", codes, torch.uint8, (N, half), dev),
            _addr("scales", scales, torch.bfloat16, groups, dev),
            _addr("zeros", zeros, torch.uint8, groups, dev),
            _addr("bias", bias, torch.float32, (N,), dev))
    code = _io_code(out_dtype)
    st, ctx = _stream_on(stream, dev), _elsewhere(stream, dev)
    if ctx is not None:
        ctx.__enter__()
    try:
        if out is not None:
            po = _addr("out", out, out_dtype, shape[:-1] + (N,), dev)
        elif len(shape) == 2:
            out = _rows(shape[0], N, out_dtype, dev)
            po = out.data_ptr()
        else:
            out = A.new_empty(shape[:-1] + (N,), dtype=out_dtype)
            po = out.data_ptr()
        status = load().m3_linear_w4(*args, po, code, st)
    finally:
        if ctx is not None:
            ctx.__exit__(None, None, None)
    if stream is not None:
        _share(stream, dev, A, codes, scales, zeros, bias, out)
    if status:
        raise M3Error("m3_linear_w4", status)
    return out
