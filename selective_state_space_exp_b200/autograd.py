"""torch.autograd binding of the scan: the forward is m3_scan_fwd (or
m3_scan_fwd_varlen), the backward m3_scan_bwd (m3_scan_bwd_varlen), both
through the C ABI.  Argument marshalling only; every step runs in the
library's kernels.

    y, final_state = m3_scan(x, dt, A, lam, theta, B, C, chunk=64, h0=None,
                             B_prev=None, x_prev=None)

Layouts as m3_scan_fwd.  Gradients flow to every tensor argument that
requires them.  Precision: the incoming gradient of y is handed to the
backward as it arrives, never rounded here.  torch's engine delivers the
gradient of an output in that output's dtype, so for a bf16 layer dy is
already bf16 when it gets here; callers that hold fp32 output gradients and
want them used unrounded call m3.m3_scan_bwd directly with an fp32 dy (the
C ABI's M3_FLAG_DY_F32).  The final-state gradient is fp32.  The backward
computes every gradient in fp32; each is returned in its input's dtype, as
torch requires (bf16 x, B, C, B_prev, x_prev receive bf16 gradients, rounded
to nearest even once, at the end; dt, A, lam, theta, h0 are fp32).
First derivatives only, here and below: a second one raises.
"""
from __future__ import annotations

import functools

import torch

from . import m3

_NAMES = ("x", "dt", "A", "lam", "theta", "B", "C", "h0", "B_prev", "x_prev")


def _aligned(t):
    """t as the library takes it, contiguous and on a 16-byte boundary.  The engine may hand
    over a part of a larger gradient (torch.cat's), which starts anywhere."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _dy(dy, x):
    """dy as the backward reads it: x's dtype, or fp32 unrounded (anything else
    is converted to fp32 first, which is exact for every narrower float)."""
    if dy.dtype != x.dtype and dy.dtype != torch.float32:
        dy = dy.float()
    return _aligned(dy)


class _NoDerivative(torch.autograd.Function):
    """Identity on a gradient that the library computed; its own derivative raises."""

    @staticmethod
    def forward(ctx, what, g, *roots):
        ctx.what = what
        return g

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError(f"{ctx.what} has first derivatives only: a gradient it gave (create_graph=True) "
                           "cannot be differentiated again")


def _first_derivative(backward):
    """Marks a backward that is no differentiable function itself.  With create_graph its
    gradients hang on the inputs by a node that raises, so a term made from them is never
    left out in silence.  (torch's once_differentiable lets them go without history where
    the incoming gradient has none, as below a plain sum.)"""
    @functools.wraps(backward)
    def run(ctx, *grads):
        if not torch.is_grad_enabled():
            return backward(ctx, *grads)
        with torch.no_grad():
            out = backward(ctx, *grads)
        roots = [t for t in (*ctx.saved_tensors, *grads) if t is not None and t.requires_grad]
        return tuple(None if g is None else _NoDerivative.apply(type(ctx).__name__, g, *roots) for g in out)

    return run


class M3Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, chunk, x, dt, A, lam, theta, B, C, h0, B_prev, x_prev):
        y, fs = m3.m3_scan_fwd(x, dt, A, lam, theta, B, C, chunk, h0, B_prev, x_prev)
        ctx.chunk = chunk
        ctx.save_for_backward(x, dt, A, lam, theta, B, C, h0, B_prev, x_prev)
        return y, fs

    @staticmethod
    @_first_derivative
    def backward(ctx, dy, d_final):
        x, dt, A, lam, theta, B, C, h0, B_prev, x_prev = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros_like(x)
        g = m3.m3_scan_bwd(x, dt, A, lam, theta, B, C, _dy(dy, x), ctx.chunk,
                           h0, B_prev, x_prev,
                           None if d_final is None else _aligned(d_final.float()))
        inputs = dict(zip(_NAMES, (x, dt, A, lam, theta, B, C, h0, B_prev, x_prev)))
        out = [None]  # chunk
        for i, name in enumerate(_NAMES):
            t = inputs[name]
            if t is None or not ctx.needs_input_grad[i + 1] or name not in g:
                out.append(None)
            else:
                out.append(g[name].to(t.dtype))
        return tuple(out)


def m3_scan(x, dt, A, lam, theta, B, C, chunk: int = 64, h0=None, B_prev=None, x_prev=None):
    """Differentiable chunked scan: (y, final_state), gradients by m3_scan_bwd."""
    return M3Scan.apply(chunk, x, dt, A, lam, theta, B, C, h0, B_prev, x_prev)


class M3ScanVarlen(torch.autograd.Function):
    @staticmethod
    def forward(ctx, chunk, max_seqlen, cu_seqlens, x, dt, A, lam, theta, B, C, h0, B_prev,
                x_prev):
        y, fs = m3.m3_scan_fwd_varlen(cu_seqlens, x, dt, A, lam, theta, B, C, chunk, h0, B_prev,
                                      x_prev, max_seqlen=max_seqlen)
        ctx.chunk, ctx.max_seqlen = chunk, max_seqlen
        ctx.save_for_backward(cu_seqlens, x, dt, A, lam, theta, B, C, h0, B_prev, x_prev)
        return y, fs

    @staticmethod
    @_first_derivative
    def backward(ctx, dy, d_final):
        cu, x, dt, A, lam, theta, B, C, h0, B_prev, x_prev = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros_like(x)
        g = m3.m3_scan_bwd_varlen(cu, x, dt, A, lam, theta, B, C, _dy(dy, x),
                                  ctx.chunk, h0, B_prev, x_prev,
                                  None if d_final is None else _aligned(d_final.float()),
                                  max_seqlen=ctx.max_seqlen)
        inputs = dict(zip(_NAMES, (x, dt, A, lam, theta, B, C, h0, B_prev, x_prev)))
        out = [None, None, None]  # chunk, max_seqlen, cu_seqlens
        for i, name in enumerate(_NAMES):
            t = inputs[name]
            if t is None or not ctx.needs_input_grad[i + 3] or name not in g:
                out.append(None)
            else:
                out.append(g[name].to(t.dtype))
        return tuple(out)


def m3_scan_varlen(cu_seqlens, x, dt, A, lam, theta, B, C, chunk: int = 64, h0=None,
                   B_prev=None, x_prev=None, *, max_seqlen=None):
    """Differentiable scan of a packed batch (layouts of m3_scan_fwd_varlen):
    (y, final states), gradients by m3_scan_bwd_varlen."""
    if max_seqlen is None:
        S = cu_seqlens.numel() - 1
        max_seqlen = int((cu_seqlens[1:] - cu_seqlens[:-1]).max().item()) if S > 0 else 0
    return M3ScanVarlen.apply(chunk, max_seqlen, cu_seqlens, x, dt, A, lam, theta, B, C, h0,
                              B_prev, x_prev)


# ---- operators between the layer and a model's tokens ---------------------------

class M3GroupNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, cu_seqlens, max_seqlen, groups, act, eps, scope, x, weight, bias, z):
        kw = dict(weight=weight, bias=bias, z=z, act=act, eps=eps)
        if cu_seqlens is None:
            y, mean, rstd = m3.m3_group_norm_fwd(x, groups, scope=scope, **kw)
        else:
            # rows outside every sequence are not written by the call
            y, mean, rstd = m3.m3_group_norm_fwd_varlen(cu_seqlens, x, groups, y=x.clone(),
                                                        max_seqlen=max_seqlen, **kw)
        ctx.groups, ctx.act, ctx.scope, ctx.max_seqlen = groups, act, scope, max_seqlen
        ctx.save_for_backward(cu_seqlens, x, weight, bias, z, mean, rstd)
        return y

    @staticmethod
    @_first_derivative
    def backward(ctx, dy):
        cu, x, weight, bias, z, mean, rstd = ctx.saved_tensors
        dy = _aligned(dy.to(x.dtype))
        need = ctx.needs_input_grad[6:]
        kw = dict(weight=weight, bias=bias, z=z, act=ctx.act, want_dx=need[0], want_dweight=need[1],
                  want_dbias=need[2], want_dz=need[3])
        if cu is None:
            g = m3.m3_group_norm_bwd(x, ctx.groups, mean, rstd, dy, scope=ctx.scope, **kw)
        else:
            g = m3.m3_group_norm_bwd_varlen(cu, x, ctx.groups, mean, rstd, dy,
                                            max_seqlen=ctx.max_seqlen, **kw)
            # the gradients of rows outside every sequence: y there is x itself
            outside = _outside(cu, x.shape[0])
            if need[0]:
                g["x"] = torch.where(outside, dy, g["x"])
            if need[3]:
                g["z"] = torch.where(outside, torch.zeros_like(z), g["z"])
        return (None,) * 6 + tuple(g.get(name) for name in ("x", "weight", "bias", "z"))


def _outside(cu_seqlens, total):
    """[total][1] bool: rows that belong to no sequence (before the first, behind the last)."""
    row = torch.arange(total, device=cu_seqlens.device)
    return ((row < cu_seqlens[0]) | (row >= cu_seqlens[-1]))[:, None]


def group_norm(x, groups: int, weight=None, bias=None, z=None, *, act="none", eps: float = 1e-5,
               scope="token"):
    """Differentiable m3.m3_group_norm_fwd: y alone, gradients of x, weight, bias
    and z by m3_group_norm_bwd (weight and bias fp32).  First derivatives only: a
    second one raises."""
    return M3GroupNorm.apply(None, None, groups, act, eps, scope, x, weight, bias, z)


def group_norm_varlen(cu_seqlens, x, groups: int, weight=None, bias=None, z=None, *, act="none",
                      eps: float = 1e-5, max_seqlen=None):
    """group_norm over the sequences of a packed batch (x [T][C]); rows outside
    every sequence pass through unchanged.  First derivatives only."""
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens holds no sequence")
    if max_seqlen is None:
        max_seqlen = int((cu_seqlens[1:] - cu_seqlens[:-1]).max().item())
    return M3GroupNorm.apply(cu_seqlens, max_seqlen, groups, act, eps, "sequence", x, weight,
                             bias, z)


class M3LinearXent(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ignore_index, targets, h, W):
        loss, lse = m3.m3_linear_xent_fwd(h, W, targets, ignore_index=ignore_index)
        ctx.ignore_index = ignore_index
        ctx.save_for_backward(targets, h, W, lse)
        return loss

    @staticmethod
    @_first_derivative
    def backward(ctx, dloss):
        targets, h, W, lse = ctx.saved_tensors
        dh, dW = m3.m3_linear_xent_bwd(h, W, targets, lse, dloss.contiguous(),
                                       ignore_index=ctx.ignore_index,
                                       want_dh=ctx.needs_input_grad[2],
                                       want_dW=ctx.needs_input_grad[3])
        return None, None, dh, dW


def linear_cross_entropy(h, W, targets, *, ignore_index: int = -100, reduction="mean"):
    """Softmax cross entropy of the head W [V][K] on hidden states h [..][K]
    (bf16) without the logits, by m3_linear_xent_fwd / _bwd.  reduction "none"
    (shaped like targets), "sum", or "mean" over the scored tokens (0 where there
    is none).  Gradients of h and W, in bf16; first derivatives only: a second one
    raises."""
    if reduction not in ("none", "sum", "mean"):
        raise ValueError(f"reduction is {reduction!r}: expected 'none', 'sum' or 'mean'")
    loss = M3LinearXent.apply(ignore_index, targets, h, W)
    if reduction == "none":
        return loss
    if reduction == "sum":
        return loss.sum()
    return loss.sum() / (targets != ignore_index).sum().clamp(min=1)
