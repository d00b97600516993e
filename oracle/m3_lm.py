"""fp64 oracle of the operators between the layer and a language model's tokens:
the grouped norm with its activation, the head's cross entropy, products with
4-bit weights.

TEST INFRASTRUCTURE ONLY: the library never imports it and it never imports the
library.  Everything is plain numpy in fp64 with explicit loops over samples and
groups; the gradients are written out from the formulas below (not taken by
automatic differentiation) and pinned to finite differences.

  group_norm   over one sample's positions and one group's channels:
               xh = (x - mean) / sqrt(var + eps), u = xh w + b,
               y = u, u sigma(u), or u z sigma(z)
  xent         loss_t = log sum_v exp(h_t . W_v) - h_t . W_{y_t}, 0 for an
               ignored token
  w4           out = A ((q - z) s)^T + bias, codes two a byte, the even input low
"""
from __future__ import annotations

import numpy as np


def f64(a):
    if a is None:
        return None
    if hasattr(a, "detach"):
        a = a.detach().cpu()
        a = a.float().numpy() if a.is_floating_point() else a.numpy()
    return np.asarray(a, dtype=np.float64)


def sigmoid(v):
    return 1.0 / (1.0 + np.exp(-v))


def group_norm(x, groups, w=None, b=None, z=None, act="none", eps=1e-5, spans=None, dy=None):
    """x [T][C] and the samples as (first, end) row pairs (None: every row its
    own).  Returns {"y", "mean", "rstd"} and, given dy, {"x", "w", "b", "z"}.
    Rows of no sample: y, dx and dz are NaN there."""
    x, w, b, z, dy = (f64(v) for v in (x, w, b, z, dy))
    T, C = x.shape
    cg = C // groups
    w = np.ones(C) if w is None else w
    b = np.zeros(C) if b is None else b
    spans = [(t, t + 1) for t in range(T)] if spans is None else spans
    out = {"y": np.full((T, C), np.nan), "mean": np.zeros((len(spans), groups)),
           "rstd": np.zeros((len(spans), groups))}
    if dy is not None:
        out.update(x=np.full((T, C), np.nan), w=np.zeros(C), b=np.zeros(C))
        if z is not None:
            out["z"] = np.full((T, C), np.nan)
    for i, (t0, t1) in enumerate(spans):
        if t1 == t0:
            continue
        for g in range(groups):
            c = slice(g * cg, (g + 1) * cg)
            v = x[t0:t1, c]
            mean = v.mean()
            rstd = 1.0 / np.sqrt(((v - mean) ** 2).mean() + eps)
            out["mean"][i, g], out["rstd"][i, g] = mean, rstd
            xh = (v - mean) * rstd
            u = xh * w[c] + b[c]
            if act == "silu":
                y, du = u * sigmoid(u), sigmoid(u) * (1.0 + u * (1.0 - sigmoid(u)))
            elif act == "gate":
                zz = z[t0:t1, c]
                y, du = u * zz * sigmoid(zz), zz * sigmoid(zz)
            else:
                y, du = u, np.ones_like(u)
            out["y"][t0:t1, c] = y
            if dy is None:
                continue
            d = dy[t0:t1, c]
            gr = d * du
            if act == "gate":
                out["z"][t0:t1, c] = d * u * sigmoid(zz) * (1.0 + zz * (1.0 - sigmoid(zz)))
            out["w"][c] += (gr * xh).sum(0)
            out["b"][c] += gr.sum(0)
            a = gr * w[c]
            out["x"][t0:t1, c] = rstd * (a - a.mean() - xh * (a * xh).mean())
    return out


def xent(h, W, targets, ignore=-100, dloss=None):
    """h [M][K], W [V][K]: {"loss", "lse"} and, given dloss, {"h", "W", "d"}
    (d: the logits' gradients)."""
    h, W, dloss = f64(h), f64(W), f64(dloss)
    t = np.asarray(targets.detach().cpu().numpy() if hasattr(targets, "detach") else targets)
    logits = h @ W.T
    top = logits.max(1, keepdims=True)
    lse = (top + np.log(np.exp(logits - top).sum(1, keepdims=True)))[:, 0]
    on = t != ignore
    loss = np.zeros(len(t))
    loss[on] = lse[on] - logits[on, t[on]]
    out = {"loss": loss, "lse": lse}
    if dloss is not None:
        d = np.exp(logits - lse[:, None])
        d[on, t[on]] -= 1.0
        d *= np.where(on, dloss, 0.0)[:, None]
        out.update(h=d @ W, W=d.T @ h, d=d)
    return out


def w4_weights(codes, scales, zeros=None):
    """Dequantised [N][K] from codes [N][K/2], scales [N][G], zeros [N][G] (8)."""
    c = np.asarray(codes.cpu().numpy() if hasattr(codes, "cpu") else codes)
    N, half = c.shape
    q = np.empty((N, 2 * half))
    q[:, 0::2] = c & 15
    q[:, 1::2] = c >> 4
    s = f64(scales)
    z = np.full(s.shape, 8.0) if zeros is None else f64(zeros)
    per = 2 * half // s.shape[1]
    return (q - np.repeat(z, per, 1)) * np.repeat(s, per, 1)


def w4_linear(A, codes, scales, zeros=None, bias=None):
    out = f64(A) @ w4_weights(codes, scales, zeros).T
    return out if bias is None else out + f64(bias)
