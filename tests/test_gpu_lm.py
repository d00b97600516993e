"""The grouped norm, the head's cross entropy and the 4-bit products on the GPU,
against their fp64 oracle (oracle/m3_lm.py), element by element.

Tolerances, fixed before the first run.  A bf16 output is off by at most half a
step, 2^-8 of its value, from an fp32 result; an fp32 result by its roundings,
2^-24 each of the largest magnitude on the way:
  norm   y, dx, dz: 64 roundings of the largest |x - mean| rstd |w| + |b| (times
         what follows it); dw, db: 256 of the sum of the terms' magnitudes (a
         thread adds at most a few hundred rows in a chain)
  xent   logits: a tensor-core sum of K products is a chain of K / 16 steps, each
         truncated, so (K / 16 + 8) 2^-22 sum_k |h W|; loss and lse besides 16
         roundings of lse.  dh, dW: every logit's gradient is rounded once to bf16
         (2^-8), so 2^-8 of the sum of |d| |W| (|d| |h|) and of the value
  w4     a group's sum is a chain of group / 16 steps, then one rounding a group:
         (group / 16 + K / group + 4) 2^-23 sum_k |A (q - z) s|
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import m3_lm as lm
from selective_state_space_exp_b200 import autograd, m3
from parity_helpers import need_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
IO = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def ok():
    assert m3.m3_stream_status() == 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def near(got, ref, atol, what):
    """|got - ref| <= half a step of got's type + atol, everywhere (NaN in ref: not looked at)."""
    g = got.detach().float().cpu().numpy().astype(np.float64)
    half = torch.finfo(got.dtype).eps / 2
    ref = np.asarray(ref).reshape(g.shape)
    seen = ~np.isnan(ref)
    assert np.isfinite(g[seen]).all(), what
    over = (np.abs(g - ref) - half * np.abs(ref) - atol)[seen]
    assert over.size == 0 or over.max() <= 0, (what, float(over.max()))


# ---- grouped norm ----------------------------------------------------------------

def norm_inputs(T, C, io, act, seed, offset=0.0):
    g = gen(seed)
    dt = IO[io]
    x = (torch.randn((T, C), generator=g) * 1.5 + offset).to(dt)
    z = torch.randn((T, C), generator=g).to(dt) if act == "gate" else None
    dy = torch.randn((T, C), generator=g).to(dt)
    w, b = torch.randn(C, generator=g) * 0.2 + 1.0, torch.randn(C, generator=g) * 0.3
    return x, z, dy, w, b


def check_norm(x, z, dy, w, b, G, act, spans, got_y, mean, rstd, grads, eps=1e-5):
    ref = lm.group_norm(x, G, w, b, z, act, eps, spans, dy)
    xs = lm.f64(x)
    T, C = xs.shape
    wa = np.abs(lm.f64(w)).max() if w is not None else 1.0
    ba = np.abs(lm.f64(b)).max() if b is not None else 0.0
    r = ref["rstd"].max() if ref["rstd"].size else 0.0
    # the mean is rounded relative to |x|, so an offset costs its share
    u = np.abs(xs).max() * r * wa + ba + 1.0 if xs.size else 1.0
    za = np.abs(lm.f64(z)).max() + 1.0 if z is not None else 1.0
    da = np.abs(lm.f64(dy)).max() if dy is not None and dy.numel() else 0.0
    near(got_y, ref["y"], 64 * U * u * za, "y")
    near(mean, ref["mean"], 64 * U * (np.abs(xs).max() if xs.size else 1.0), "mean")
    near(rstd, ref["rstd"], 64 * U * r * u, "rstd")
    if grads is None:
        return
    slope = u * za * da  # of g = dy act'(u), whose slope in u is at most about one
    near(grads["x"], ref["x"], 64 * U * r * (wa + 1) * slope * u, "dx")
    if z is not None:
        near(grads["z"], ref["z"], 64 * U * slope * u, "dz")
    rows = T
    near(grads["weight"], ref["w"], 256 * U * rows * slope * u, "dw")
    near(grads["bias"], ref["b"], 256 * U * rows * slope, "db")


TOKEN = [  # tokens, groups, channels of a group
    (1, 1, 1), (1, 3, 5), (2, 1, 64), (7, 64, 64), (130, 5, 17), (33, 4, 100), (65, 2, 96),
    (40, 3, 256), (9, 1, 600), (19, 2, 1031), (11, 1, 2048), (5, 1, 4096), (3, 2, 5000), (300, 6, 8),
]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "silu", "gate"])
@pytest.mark.parametrize("T,G,cg", TOKEN)
def test_norm_of_tokens(T, G, cg, act, io):
    x, z, dy, w, b = norm_inputs(T, G * cg, io, act, T * 7 + G + cg)
    d = [None if v is None else v.cuda() for v in (x, z, dy, w, b)]
    y, mean, rstd = m3.m3_group_norm_fwd(d[0], G, d[3], d[4], d[1], act=act)
    g = m3.m3_group_norm_bwd(d[0], G, mean, rstd, d[2], d[3], d[4], d[1], act=act)
    ok()
    check_norm(x, z, dy, w, b, G, act, None, y, mean, rstd, g)


SEQ = [  # samples, positions, groups, channels of a group
    (1, 1, 1, 8), (2, 2, 3, 5), (3, 7, 2, 16), (2, 129, 5, 24), (4, 300, 3, 31), (1, 1000, 2, 64),
    (2, 65, 1, 2500), (70, 3, 4, 6), (2, 513, 40, 8), (1, 700, 1, 300),
    # long samples, which several blocks share, and those at the border
    (2, 3000, 2, 24), (1, 9000, 1, 8), (3, 700, 3, 31), (2, 900, 40, 8), (1, 8192, 1, 8), (1, 8193, 1, 8),
]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "silu", "gate"])
@pytest.mark.parametrize("B,L,G,cg", SEQ)
def test_norm_of_sequences(B, L, G, cg, act, io):
    C = G * cg
    x, z, dy, w, b = norm_inputs(B * L, C, io, act, B + L * 3 + G + cg)
    d = [None if v is None else v.cuda().view(B, L, C) for v in (x, z, dy)]
    y, mean, rstd = m3.m3_group_norm_fwd(d[0], G, w.cuda(), b.cuda(), d[1], act=act, scope="sequence")
    g = m3.m3_group_norm_bwd(d[0], G, mean, rstd, d[2], w.cuda(), b.cuda(), d[1], act=act,
                             scope="sequence")
    ok()
    spans = [(i * L, (i + 1) * L) for i in range(B)]
    check_norm(x, z, dy, w, b, G, act, spans, y, mean, rstd, g)


@pytest.mark.parametrize("cu", [[3, 3, 4, 4, 67, 300, 301], [3, 3, 4, 4, 90, 4800, 4801]])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_norm_of_a_packed_batch(io, cu):
    """Lengths 0, 1 and long ones, rows before the first sequence and behind the last:
    these keep what y held."""
    T, G, cg = cu[-1] + 19, 3, 24
    for act in ("silu", "gate"):
        x, z, dy, w, b = norm_inputs(T, G * cg, io, act, 5)
        c = torch.tensor(cu, dtype=torch.int32).cuda()
        d = [None if v is None else v.cuda() for v in (x, z, dy, w, b)]
        y0 = torch.full_like(d[0], 7.0)
        y, mean, rstd = m3.m3_group_norm_fwd_varlen(c, d[0], G, d[3], d[4], d[1], act=act, y=y0)
        g = m3.m3_group_norm_bwd_varlen(c, d[0], G, mean, rstd, d[2], d[3], d[4], d[1], act=act)
        ok()
        spans = list(zip(cu[:-1], cu[1:]))
        assert (y[:3] == 7).all() and (y[cu[-1]:] == 7).all()
        assert (mean[0] == 0).all() and (rstd[0] == 0).all()      # an empty sequence
        check_norm(x, z, dy, w, b, G, act, spans, y, mean, rstd, g)


def test_norm_bad_offsets_are_reported():
    x = torch.randn((10, 8)).cuda()
    for cu in ([0, 12], [4, 2], [-1, 3], [0, 9]):  # past the rows, falling, negative, too long
        c = torch.tensor(cu, dtype=torch.int32).cuda()
        y = torch.zeros_like(x)
        m3.m3_group_norm_fwd_varlen(c, x, 2, max_seqlen=8, y=y)
        assert m3.m3_stream_status() == m3.M3_ERR_INVALID_ARGUMENT, cu
        assert (y == 0).all()
    ok()


@pytest.mark.parametrize("scope,shape", [("token", (6, 96)), ("sequence", (2, 200, 12))])
def test_norm_keeps_its_precision_under_an_offset(scope, shape):
    """fp32 values 4096 +- 1: the statistics are as exact as the values allow."""
    C = shape[-1]
    x, _, _, w, b = norm_inputs(int(np.prod(shape[:-1])), C, "f32", "none", 9, offset=4096.0)
    y, mean, rstd = m3.m3_group_norm_fwd(x.cuda().view(shape), 2, w.cuda(), b.cuda(), scope=scope)
    ok()
    L = shape[1] if scope == "sequence" else 1
    spans = [(i * L, (i + 1) * L) for i in range(x.shape[0] // L)]
    ref = lm.group_norm(x, 2, w, b, spans=spans)
    # x - mean is exact to a rounding of the mean (2^-12 here); rstd to a few roundings
    near(y, ref["y"], 4 * 4096 * U * ref["rstd"].max() * 2, "y")
    near(rstd, ref["rstd"], 64 * U, "rstd")


def test_norm_constant_rows_and_in_place():
    """A slice without spread: xh = 0, so y = b (eps keeps rstd finite)."""
    x = torch.full((5, 32), 3.25).cuda()
    w, b = torch.randn(32).cuda(), torch.randn(32).cuda()
    y, mean, rstd = m3.m3_group_norm_fwd(x, 4, w, b)
    ok()
    assert torch.equal(y, b.expand(5, 32)) and (mean == 3.25).all()
    x = torch.randn((50, 64)).cuda()
    z = torch.randn((50, 64)).cuda()
    for scope in ("token", "sequence"):
        v = x if scope == "token" else x[None]
        zz = z if scope == "token" else z[None]
        want = m3.m3_group_norm_fwd(v, 4, z=zz, act="gate", scope=scope)[0]
        for target in ("x", "z"):
            a, c = v.clone(), zz.clone()
            got = m3.m3_group_norm_fwd(a, 4, z=c, act="gate", scope=scope, y=a if target == "x" else c)[0]
            assert torch.equal(got, want)
    ok()


def test_norm_without_weights_or_wanted_outputs():
    x, _, dy, _, _ = norm_inputs(37, 48, "f32", "none", 11)
    y, mean, rstd = m3.m3_group_norm_fwd(x.cuda(), 4)
    g = m3.m3_group_norm_bwd(x.cuda(), 4, mean, rstd, dy.cuda())
    ok()
    check_norm(x, None, dy, None, None, 4, "none", None, y, mean, rstd, g)
    # C entry: every output of the backward may be left out
    lib, s = m3.load(), m3.NormShape(37, 1, 48, 4, m3.M3_F32, 0, 1e-5)
    import ctypes
    xd, dyd, dx = x.cuda(), dy.cuda(), torch.empty_like(x).cuda()
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    assert lib.m3_group_norm_bwd(ctypes.byref(s), xd.data_ptr(), None, None, None, mean.data_ptr(),
                                 rstd.data_ptr(), dyd.data_ptr(), dx.data_ptr(), None, None, None,
                                 ws.data_ptr(), ws.numel(), st) == 0
    ok()
    assert torch.equal(dx, g["x"])


def test_norm_empty_batches():
    for shape, scope in (((0, 16), "token"), ((0, 5, 16), "sequence"), ((3, 0, 16), "sequence")):
        x = torch.zeros(shape).cuda()
        y, mean, rstd = m3.m3_group_norm_fwd(x, 2, scope=scope)
        g = m3.m3_group_norm_bwd(x, 2, mean, rstd, x, scope=scope)
        assert y.shape == x.shape and (g["weight"] == 0).all() and (g["bias"] == 0).all()
        assert mean.numel() == 0 or (mean == 0).all()
    ok()


def test_norm_values_that_are_not_finite_stay_in_their_group():
    x = torch.randn((4, 64)).cuda()
    x[1, 3], x[2, 40] = float("nan"), float("inf")
    y = m3.m3_group_norm_fwd(x, 4)[0].view(4, 4, 16)
    ok()
    bad = torch.zeros((4, 4), dtype=torch.bool)
    bad[1, 0] = bad[2, 2] = True
    assert torch.equal(~torch.isfinite(y).all(-1).cpu(), bad)


# ---- cross entropy -----------------------------------------------------------------

def xent_inputs(M, V, K, seed, ignored=0.2, scale=2.0):
    g = gen(seed)
    h = torch.randn((M, K), generator=g).bfloat16()
    W = (torch.randn((V, K), generator=g) * scale / K ** 0.5).bfloat16()
    t = torch.randint(0, V, (M,), generator=g)
    t = torch.where(torch.rand(M, generator=g) < ignored, torch.full_like(t, -100), t)
    return h, W, t, torch.rand(M, generator=g) + 0.1


def check_xent(h, W, t, dl, loss, lse, dh, dW, ignore=-100):
    ref = lm.xent(h, W, t, ignore, dl)
    hs, Ws = np.abs(lm.f64(h)), np.abs(lm.f64(W))
    M, K = hs.shape
    logit = (K / 16 + 8) * 2.0 ** -22 * float((hs @ Ws.T).max())
    soft = logit + 16 * U * np.abs(ref["lse"]).max()
    near(lse, ref["lse"], soft, "lse")
    near(loss, ref["loss"], 2 * soft, "loss")
    if dh is None and dW is None:
        return
    d = np.abs(ref["d"]) + np.abs(lm.f64(dl))[:, None] * (2 * soft)  # what a logit's error moves
    steps = 2.0 ** -8 + soft * 4 + 2.0 ** -14
    if dh is not None:
        near(dh, ref["h"], steps * (d @ Ws), "dh")
    if dW is not None:
        near(dW, ref["W"], steps * (d.T @ hs), "dW")


XENT = [(1, 1, 8), (1, 2, 8), (3, 7, 64), (1, 1000, 128), (77, 1003, 256), (128, 256, 64), (129, 257, 72),
        (300, 5, 200), (1000, 130, 40), (513, 4097, 96), (64, 20000, 64), (200, 515, 1032),
        # other cuts of the products: columns of a tile, pairs, splits
        (70, 11000, 136), (40, 9000, 1040), (2000, 120, 1000), (1300, 1900, 200), (246, 2376, 536),
        (260, 9000, 1496)]


@pytest.mark.parametrize("M,V,K", XENT)
def test_xent(M, V, K):
    h, W, t, dl = xent_inputs(M, V, K, M + V + K)
    d = [v.cuda() for v in (h, W, t, dl)]
    loss, lse = m3.m3_linear_xent_fwd(*d[:3])
    dh, dW = m3.m3_linear_xent_bwd(*d[:3], lse, d[3])
    ok()
    check_xent(h, W, t, dl, loss, lse, dh, dW)


def test_xent_in_pieces_of_the_vocabulary():
    """More classes than one piece of the workspace holds: 20000 tokens leave room
    for 6656, so 15000 are three pieces, the last one short."""
    M, V, K = 20000, 15000, 16
    h, W, t, dl = xent_inputs(M, V, K, 1)
    d = [v.cuda() for v in (h, W, t, dl)]
    loss, lse = m3.m3_linear_xent_fwd(*d[:3])
    dh, dW = m3.m3_linear_xent_bwd(*d[:3], lse, d[3])
    ok()
    hd, Wd = d[0].double(), d[1].double()
    z = torch.logsumexp(hd @ Wd.T, 1)
    p = torch.softmax(hd @ Wd.T, 1)
    on = (d[2] >= 0)
    p[on, d[2][on]] -= 1
    p *= (d[3].double() * on)[:, None]
    assert ((lse.double() - z).abs().max() < 1e-5)
    for got, ref, mag in ((dh, p @ Wd, p.abs() @ Wd.abs()), (dW, p.T @ hd, p.abs().T @ hd.abs())):
        over = (got.double() - ref).abs() - 2.0 ** -8 * (ref.abs() + mag) - 1e-4 * mag
        assert over.max() <= 0


def test_xent_targets():
    """All ignored; one target for all; ignore_index that is a class; a target out of range."""
    M, V, K = 40, 300, 64
    h, W, t, dl = xent_inputs(M, V, K, 3, ignored=0.0)
    hd, Wd, dld = h.cuda(), W.cuda(), dl.cuda()
    for tt, ign in ((torch.full((M,), -100), -100), (torch.full((M,), 7), -100), (t, int(t[0]))):
        loss, lse = m3.m3_linear_xent_fwd(hd, Wd, tt.cuda(), ignore_index=ign)
        dh, dW = m3.m3_linear_xent_bwd(hd, Wd, tt.cuda(), lse, dld, ignore_index=ign)
        ok()
        check_xent(h, W, tt, dl, loss, lse, dh, dW, ign)
        if (tt == ign).all():
            assert (loss == 0).all() and (dh == 0).all() and (dW == 0).all()
    for bad in (V, -1, 1 << 40):
        tt = t.clone()
        tt[5] = bad
        loss, lse = m3.m3_linear_xent_fwd(hd, Wd, tt.cuda())
        assert m3.m3_stream_status() == m3.M3_ERR_INVALID_ARGUMENT
        assert torch.isnan(loss[5]) and torch.isfinite(loss[torch.arange(M) != 5]).all()
        dh, dW = m3.m3_linear_xent_bwd(hd, Wd, tt.cuda(), lse, dld)
        assert (dh[5] == 0).all() and torch.isfinite(dW.float()).all()
    ok()


def test_xent_equal_and_uneven_weights_of_the_tokens():
    """dloss: all equal (the mean), all zero, one only, mixed signs and magnitudes, and
    NaN at an ignored token, which is not read."""
    M, V, K = 150, 400, 96
    h, W, t, _ = xent_inputs(M, V, K, 4)
    t[3] = -100
    hd, Wd, td = h.cuda(), W.cuda(), t.cuda()
    loss, lse = m3.m3_linear_xent_fwd(hd, Wd, td)
    one = torch.zeros(M)
    one[10] = 3e-7
    for dl in (torch.full((M,), 1 / 117), torch.zeros(M), one,
               torch.randn(M, generator=gen(1)) * 10.0 ** torch.linspace(-6, 6, M)):
        dl = dl.clone()
        dh, dW = m3.m3_linear_xent_bwd(hd, Wd, td, lse, dl.cuda())
        ok()
        check_xent(h, W, t, dl, loss, lse, dh, dW)
        dl[3] = float("nan")
        again = m3.m3_linear_xent_bwd(hd, Wd, td, lse, dl.cuda())
        ok()
        assert torch.equal(again[0], dh) and torch.equal(again[1], dW)


def test_xent_large_logits_and_one_gradient_only():
    M, V, K = 70, 900, 64
    h, W, t, dl = xent_inputs(M, V, K, 6, scale=60.0)  # logits of some hundreds
    d = [v.cuda() for v in (h, W, t, dl)]
    loss, lse = m3.m3_linear_xent_fwd(*d[:3])
    dh, dW = m3.m3_linear_xent_bwd(*d[:3], lse, d[3])
    only_h = m3.m3_linear_xent_bwd(*d[:3], lse, d[3], want_dW=False)
    only_w = m3.m3_linear_xent_bwd(*d[:3], lse, d[3], want_dh=False)
    ok()
    check_xent(h, W, t, dl, loss, lse, None, None)
    assert torch.isfinite(dh.float()).all() and torch.isfinite(dW.float()).all()
    assert only_h[1] is None and torch.equal(only_h[0], dh)
    assert only_w[0] is None and torch.equal(only_w[1], dW)


@pytest.mark.parametrize("M,V,K", [(70, 300, 64), (600, 9000, 136)])
def test_xent_tokens_not_scored_may_hold_anything(M, V, K):
    """NaN and infinities in the hidden states and dloss of ignored tokens (padding):
    their loss and dh are 0, and dW is the one without them."""
    h, W, t, dl = xent_inputs(M, V, K, 11, ignored=0.4)
    off = (t < 0).nonzero()[:, 0]
    clean = [v.clone() for v in (h, dl)]
    h[off[0::3]], h[off[1::3]], dl[off[::2]] = float("nan"), float("inf"), float("nan")
    clean[0][off], clean[1][off] = 0, 0
    d = [v.cuda() for v in (h, W, t, dl)]
    loss, lse = m3.m3_linear_xent_fwd(*d[:3])
    dh, dW = m3.m3_linear_xent_bwd(*d[:3], lse, d[3])
    ok()
    assert (loss[off.cuda()] == 0).all() and (dh[off.cuda()] == 0).all()
    lse[off.cuda()] = torch.from_numpy(lm.xent(clean[0], W, t)["lse"])[off].float().cuda()
    check_xent(clean[0], W, t, clean[1], loss, lse, dh, dW)


def test_xent_no_token():
    h, W = torch.zeros((0, 64), dtype=torch.bfloat16).cuda(), torch.randn((10, 64)).bfloat16().cuda()
    t = torch.zeros(0, dtype=torch.long).cuda()
    loss, lse = m3.m3_linear_xent_fwd(h, W, t)
    dh, dW = m3.m3_linear_xent_bwd(h, W, t, lse, loss)
    ok()
    assert loss.numel() == 0 and dh.shape == h.shape and (dW == 0).all()


def test_xent_gradient_against_differences():
    """Central differences of the loss the library itself computes, along bf16-exact
    steps of h and of W; their error is of third order, (step)^2 / 6 of the third
    derivative, below 2 % here."""
    M, V, K = 32, 200, 64
    h, W, t, dl = xent_inputs(M, V, K, 8)
    h = (h * 8).round() / 8          # multiples of 1/8 below 8: a step of 1/16 is exact
    W = (W.float() * 64).round() / 64
    W = W.bfloat16()
    d = [v.cuda() for v in (h, W, t, dl)]
    loss, lse = m3.m3_linear_xent_fwd(*d[:3])
    dh, dW = m3.m3_linear_xent_bwd(*d[:3], lse, d[3])
    g = gen(2)
    for which, grad in ((0, dh), (1, dW)):
        base = d[which]
        v = (torch.randint(0, 2, base.shape, generator=g) * 2 - 1).float().cuda()
        step = 1 / 16 if which == 0 else 1 / 128
        side = []
        for sign in (1, -1):
            moved = (base.float() + sign * step * v).bfloat16()
            assert torch.equal(moved.float(), base.float() + sign * step * v)
            args = list(d[:3])
            args[which] = moved
            side.append((m3.m3_linear_xent_fwd(*args)[0].double() * d[3].double()).sum())
        diff = float(side[0] - side[1]) / (2 * step)
        want = float((grad.double() * v.double()).sum())
        size = float(grad.double().norm() * v.double().norm())
        assert abs(diff - want) < 0.02 * size, (which, diff, want, size)
    ok()


# ---- 4-bit products ----------------------------------------------------------------

def w4_inputs(M, N, K, G, zeros, seed, bias=False):
    g = gen(seed)
    A = torch.randn((M, K), generator=g).bfloat16()
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    scales = ((torch.rand((N, K // G), generator=g) + 0.5) * 0.01).bfloat16()
    z = torch.randint(0, 16, (N, K // G), generator=g, dtype=torch.uint8) if zeros else None
    return A, codes, scales, z, torch.randn(N, generator=g) if bias else None


def check_w4(A, codes, scales, z, b, out, G):
    ref = lm.w4_linear(A, codes, scales, z, b)
    K = A.shape[-1]
    mag = np.abs(lm.f64(A)) @ np.abs(lm.w4_weights(codes, scales, z)).T
    if b is not None:
        mag = mag + np.abs(lm.f64(b))
    near(out, ref, (G / 16 + K / G + 4) * 2.0 ** -23 * mag, "out")


W4 = [  # tokens, outputs, inputs, group
    (1, 1, 32, 32), (1, 5, 64, 64), (1, 16, 128, 128), (1, 33, 96, 32), (2, 100, 320, 64), (8, 31, 512, 128),
    (9, 40, 2048, 32), (16, 130, 1152, 128), (16, 7, 4160, 64), (17, 129, 256, 64), (32, 50, 96, 32),
    (33, 300, 2176, 128), (64, 128, 1024, 32), (65, 257, 512, 128), (128, 64, 4096, 64), (130, 70, 320, 32),
    (300, 33, 640, 128), (5, 4100, 384, 128), (1, 20, 20480, 128), (3, 2, 33280, 64),
    (65, 4800, 512, 128), (200, 3300, 384, 64), (129, 3200, 256, 32),
]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K,G", W4)
def test_w4(M, N, K, G, out, zeros):
    A, codes, scales, z, b = w4_inputs(M, N, K, G, zeros, M + N + K + G, bias=(N % 2 == 0))
    d = [None if v is None else v.cuda() for v in (A, codes, scales, z, b)]
    got = m3.m3_linear_w4(*d, out_dtype=IO[out])
    ok()
    check_w4(A, codes, scales, z, b, got, G)


def test_w4_leading_dimensions_and_out():
    A, codes, scales, z, _ = w4_inputs(12, 40, 128, 64, True, 1)
    want = m3.m3_linear_w4(A.cuda(), codes.cuda(), scales.cuda(), z.cuda())
    got = m3.m3_linear_w4(A.cuda().view(3, 4, 128), codes.cuda(), scales.cuda(), z.cuda())
    buf = torch.empty((12, 40), dtype=torch.bfloat16, device="cuda")
    same = m3.m3_linear_w4(A.cuda(), codes.cuda(), scales.cuda(), z.cuda(), out=buf)
    ok()
    assert got.shape == (3, 4, 40) and torch.equal(got.view(12, 40), want)
    assert same is buf and torch.equal(buf, want)
    none = m3.m3_linear_w4(A.cuda()[:0], codes.cuda(), scales.cuda(), z.cuda())
    assert none.shape == (0, 40)


def test_w4_extreme_scales_and_unused_bits():
    """Scales of 0 and of 2^-100 and 2^100; the high half of a zero point is not read."""
    A, codes, scales, z, _ = w4_inputs(20, 64, 256, 64, True, 2)
    scales[0], scales[1], scales[2] = 0.0, 2.0 ** -100, 2.0 ** 100
    for m in (1, 20):
        got = m3.m3_linear_w4(A[:m].cuda(), codes.cuda(), scales.cuda(), z.cuda(), out_dtype=torch.float32)
        same = m3.m3_linear_w4(A[:m].cuda(), codes.cuda(), scales.cuda(), (z | 0xA0).cuda(),
                               out_dtype=torch.float32)
        ok()
        check_w4(A[:m], codes, scales, z, None, got, 64)
        assert (got[:, 0] == 0).all() and torch.equal(same, got)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("symmetric", [False, True])
@pytest.mark.parametrize("G", [32, 64, 128])
def test_w4_quantize(G, symmetric, io):
    """Every weight within half a scale of its value (and of the range's ends, which
    the scale's own rounding to bf16 can move by 2^-8 of them); a group of zeros stays zero."""
    g = gen(G)
    W = (torch.randn((37, 4 * G), generator=g) * torch.rand((37, 1), generator=g) * 3).to(IO[io])
    W[5, :G] = 0
    W[6, G:2 * G] = W[6, G:2 * G].abs()
    codes, scales, zeros = m3.m3_w4_quantize(W.cuda(), G, symmetric=symmetric)
    ok()
    assert (zeros is None) == symmetric
    back = lm.w4_weights(codes, scales, zeros).reshape(37, 4, G)
    w = lm.f64(W).reshape(37, 4, G)
    s = lm.f64(scales)[..., None]
    ends = np.abs(w).max(-1, keepdims=True)
    # half a step; at the ends up to 16 codes times the scale's rounding, and with zero
    # points another half step, since the zero point is rounded too
    assert (np.abs(back - w) <= s * (0.5 if symmetric else 1.0) + 2.0 ** -7 * ends + 1e-12).all()
    assert (back[5, 0] == 0).all()
    A = torch.randn((3, 4 * G), generator=g).bfloat16()
    out = m3.m3_linear_w4(A.cuda(), codes, scales, zeros, out_dtype=torch.float32)
    ok()
    check_w4(A, codes.cpu(), scales.cpu(), None if zeros is None else zeros.cpu(), None, out, G)


# ---- streams, graphs, workspaces, sizes, order ------------------------------------------

def every_call():
    """(name, function of inputs already on the device) over the forms of each operator."""
    x, z, dy, w, b = [v.cuda() for v in norm_inputs(260, 96, "bf16", "gate", 1)]
    h, W, t, dl = [v.cuda() for v in xent_inputs(300, 700, 64, 1)]
    q1 = [v.cuda() for v in w4_inputs(3, 200, 512, 64, True, 1)[:4]]
    q2 = [v.cuda() for v in w4_inputs(100, 200, 1024, 64, True, 2)[:4]]

    def norm(scope, **kw):
        v = (lambda a: a) if scope == "token" else (lambda a: a.view(2, 130, 96))
        y, m, r = m3.m3_group_norm_fwd(v(x), 4, w, b, v(z), act="gate", scope=scope, **kw)
        g = m3.m3_group_norm_bwd(v(x), 4, m, r, v(dy), w, b, v(z), act="gate", scope=scope, **kw)
        return (y, m, r, *g.values())

    def xent(**kw):
        loss, lse = m3.m3_linear_xent_fwd(h, W, t, **kw)
        return (loss, lse, *m3.m3_linear_xent_bwd(h, W, t, lse, dl, **kw))

    return {"norm token": lambda **k: norm("token", **k), "norm sequence": lambda **k: norm("sequence", **k),
            "xent": xent, "w4 few": lambda **k: (m3.m3_linear_w4(*q1, **k),),
            "w4 many": lambda **k: (m3.m3_linear_w4(*q2, **k),)}, x


def test_repeats_streams_and_workspaces_give_the_same_bits():
    calls, _ = every_call()
    side = torch.cuda.Stream()
    bad = torch.full((1 << 24,), float("nan"), device="cuda").view(torch.uint8)
    for name, f in calls.items():
        first = f()
        torch.cuda.synchronize()
        again = f()
        other = f(stream=side)
        side.synchronize()
        outs = [again, other]
        if not name.startswith("w4"):
            outs.append(f(workspace=bad))
        ok()
        for o in outs:
            assert all(torch.equal(a, c) for a, c in zip(first, o)), name


def test_captured_calls_follow_their_inputs():
    """Two graphs of the same calls, replayed in turn on changed inputs, give what
    eager calls give."""
    calls, x = every_call()
    f = calls["norm token"]
    f()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = f()
        graphs.append((g, out))
    for k in range(2):
        x.mul_(-1.25)
        for g, out in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = f()
        for _, out in graphs:
            assert all(torch.equal(a, c) for a, c in zip(out, want)), k
    for name in ("xent", "w4 few", "w4 many", "norm sequence"):
        want = calls[name]()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = calls[name]()
        for o in out:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(out, want)), name
    ok()


def test_two_streams_at_once():
    calls, _ = every_call()
    want = {k: f() for k, f in calls.items()}
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[f(stream=s) for f in calls.values()] for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    ok()
    for outs in got:
        for w, o in zip(want.values(), outs):
            assert all(torch.equal(a, c) for a, c in zip(w, o))


def test_binding_refuses_layouts_and_types():
    x = torch.randn((8, 64)).cuda()
    with pytest.raises(ValueError, match="contiguous"):
        m3.m3_group_norm_fwd(x.t().contiguous().t(), 4)
    with pytest.raises(TypeError, match="weight"):
        m3.m3_group_norm_fwd(x, 4, torch.ones(64, dtype=torch.bfloat16).cuda())
    with pytest.raises(ValueError, match="weight"):
        m3.m3_group_norm_fwd(x, 4, torch.ones(32).cuda())
    with pytest.raises(ValueError, match="weight is on"):
        m3.m3_group_norm_fwd(x, 4, torch.ones(64))
    with pytest.raises(ValueError, match="gate"):
        m3.m3_group_norm_fwd(x, 4, z=x)
    with pytest.raises(ValueError, match="gate"):
        m3.m3_group_norm_fwd(x, 4, act="gate")
    with pytest.raises(ValueError, match="float16"):
        m3.m3_group_norm_fwd(x.half(), 4)
    with pytest.raises(m3.M3Error) as e:  # 8 bytes past a 16-byte boundary
        m3.m3_group_norm_fwd(torch.zeros(66).cuda()[2:].view(1, 64), 4)
    assert e.value.status == -3
    h, W, t, _ = [v.cuda() for v in xent_inputs(4, 9, 64, 1)]
    with pytest.raises(TypeError, match="targets"):
        m3.m3_linear_xent_fwd(h, W, t.int())
    with pytest.raises(TypeError, match="W is"):
        m3.m3_linear_xent_fwd(h, W.float(), t)
    with pytest.raises(ValueError, match="targets"):
        m3.m3_linear_xent_fwd(h, W, t[:3])
    with pytest.raises(m3.M3Error) as e:  # a width that is no multiple of 8
        m3.m3_linear_xent_fwd(h[:, :12].contiguous(), W[:, :12].contiguous(), t)
    assert e.value.status == -2
    with pytest.raises(m3.M3Error) as e:
        m3.m3_linear_xent_fwd(h, W, t, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -4
    A, codes, scales, z, _ = [None if v is None else v.cuda() for v in w4_inputs(2, 8, 128, 64, True, 1)]
    with pytest.raises(TypeError, match="A is"):
        m3.m3_linear_w4(A.float(), codes, scales, z)
    with pytest.raises(ValueError, match="zeros"):
        m3.m3_linear_w4(A, codes, scales, z[:4])
    with pytest.raises(ValueError, match="float16"):
        m3.m3_linear_w4(A, codes, scales, z, out_dtype=torch.float16)
    ok()


def test_offsets_beyond_32_bits():
    """More than 2^31 elements of x, of the head's weights, and bytes of codes: the last
    rows come out right."""
    T, C = 1_060_000, 2048
    x = torch.zeros((T, C), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn((3, C), generator=gen(1)).bfloat16()
    x[-3:] = tail.cuda()
    y, mean, rstd = m3.m3_group_norm_fwd(x, 2)
    ok()
    ref = lm.group_norm(tail, 2)
    near(y[-3:], ref["y"], 64 * U * 8, "y")
    assert (y[:-3] == 0).all()
    del x, y
    V, K, M = 1_060_000, 2048, 3
    W = torch.zeros((V, K), dtype=torch.bfloat16, device="cuda")
    W[-2] = 0.25
    h = torch.ones((M, K), dtype=torch.bfloat16, device="cuda") / 16
    t = torch.tensor([V - 2, V - 1, 0]).cuda()
    loss, lse = m3.m3_linear_xent_fwd(h, W, t)
    ok()
    want = np.log(np.exp(32.0) + V - 1)
    near(lse, np.full(M, want), 1e-5 * want, "lse")
    near(loss, want - np.array([32.0, 0.0, 0.0]), 1e-5 * want, "loss")
    dh, dW = m3.m3_linear_xent_bwd(h, W, t, lse, torch.ones(M).cuda(), want_dh=False)
    ok()
    near(dW[-1], np.full(K, -1 / 16), 2.0 ** -8 / 16, "dW")
    assert torch.isfinite(dW[-2].float()).all()
    del W, dW
    N, K = 300_000, 16384
    codes = torch.full((N, K // 2), 0x88, dtype=torch.uint8, device="cuda")  # all weights 0
    codes[-1] = 0x99                                                      # ... but the last row's, 1
    scales = torch.ones((N, K // 128), dtype=torch.bfloat16, device="cuda")
    for m in (1, 40):
        A = torch.ones((m, K), dtype=torch.bfloat16, device="cuda")
        out = m3.m3_linear_w4(A, codes, scales, out_dtype=torch.float32)
        ok()
        assert (out[:, -1] == K).all() and (out[:, :-1] == 0).all()


def test_every_call_in_bounds():
    """The forms of every operator through the bounds-checked build."""
    from selective_state_space_exp_b200 import _build
    _build.build(debug=True)
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, os.path.join(here, "debug_bounds_lm_child.py")],
                       env=dict(os.environ, M3_LIBRARY="debug"), capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and "ALL OK" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]


# ---- as they are used together -------------------------------------------------------------

def test_training_step_scan_norm_loss():
    """Scan, gated norm, head and loss through autograd: every gradient of the step
    against the same chain in fp64 torch from the scan's output on (the scan's own
    backward has tests of its own)."""
    from selective_state_space_exp_b200 import inputs as I
    w = I.Workload(I.Shape(2, 70, 4, 64, 128, 1, 1, 64, "bf16"), decay="slow")
    inp = {k: v.cuda() for k, v in I.make_scan_inputs(w, seed=77).items()}
    C, V, G = 256, 500, 4
    g = gen(5)
    x = inp["x"].clone().requires_grad_()
    nw = (torch.randn(C, generator=g) * 0.1 + 1).cuda().requires_grad_()
    nb = (torch.randn(C, generator=g) * 0.1).cuda().requires_grad_()
    z = torch.randn((2, 70, C), generator=g).bfloat16().cuda().requires_grad_()
    W = (torch.randn((V, C), generator=g) / 8).bfloat16().cuda().requires_grad_()
    t = torch.randint(0, V, (2, 70), generator=g).cuda()
    t[0, :20] = -100
    y, _ = autograd.m3_scan(x, *(inp[k] for k in ("dt", "A", "lam", "theta", "B", "C")))
    y.retain_grad()
    u = autograd.group_norm(y.view(2, 70, C), G, nw, nb, z, act="gate")
    loss = autograd.linear_cross_entropy(u, W, t)
    loss.backward()
    ok()
    assert torch.isfinite(x.grad.float()).all() and float(x.grad.float().norm()) > 0

    yd = y.detach().double().view(2, 70, G, -1).requires_grad_()
    nwd, nbd, zd, Wd = (v.detach().double().requires_grad_() for v in (nw, nb, z, W))
    xc = yd - yd.mean(-1, keepdim=True)
    xh = (xc / torch.sqrt((xc ** 2).mean(-1, keepdim=True) + 1e-5)).reshape(2, 70, C)
    ud = (xh * nwd + nbd) * torch.nn.functional.silu(zd)
    ud16 = u.detach().double() + (ud - ud.detach())  # the head reads the rounded norm
    ref = torch.nn.functional.cross_entropy((ud16 @ Wd.T).view(-1, V), t.view(-1))
    ref.backward()
    assert abs(float(loss) - float(ref)) < 1e-5
    for name, got, want in (("W", W.grad, Wd.grad), ("w", nw.grad, nwd.grad), ("b", nb.grad, nbd.grad),
                            ("z", z.grad, zd.grad), ("y", y.grad, yd.grad)):
        # three bf16 roundings lie on the way (d, du, the gradient itself): 3 * 2^-8 of the
        # sums' magnitudes, which the random signs keep within twice the norm
        rel = float((got.double().view_as(want) - want).norm() / want.norm())
        assert rel < 3 * 2.0 ** -8, (name, rel)


def test_serving_step_decode_norm_w4():
    """One token: decode step, gated norm, 4-bit projection and 4-bit head, against the
    oracle of each applied to what the one before it gave."""
    from selective_state_space_exp_b200 import inputs as I
    w = I.Workload(I.Shape(3, 1, 4, 64, 128, 1, 1, 64, "bf16"), with_h0=True, with_prev=True)
    d = {k: v.cuda() for k, v in I.make_decode_inputs(w, seed=78, steps=2).items()}
    C, D, V = 256, 192, 700
    g = gen(6)
    Wp = (torch.randn((D, C), generator=g) / 16).cuda()
    Wv = (torch.randn((V, D), generator=g) / 14).bfloat16().cuda()
    proj = m3.m3_w4_quantize(Wp, 64)
    head = m3.m3_w4_quantize(Wv, 32, symmetric=True)
    state = d["state0"].clone()
    for s in range(2):
        Bp, xp = (d["B_prev"], d["x_prev"]) if s == 0 else (d["B"][0], d["x"][0])
        y, state = m3.m3_decode_step(state, *(d[k][s] for k in ("x", "dt", "A", "lam", "theta", "B", "C")), Bp, xp)
        z = torch.randn((3, C), generator=g).bfloat16()
        u, mean, rstd = m3.m3_group_norm_fwd(y.view(3, C), 4, z=z.cuda(), act="gate")
        p = m3.m3_linear_w4(u, *proj)
        logits = m3.m3_linear_w4(p, *head, out_dtype=torch.float32)
        ok()
        check_norm(y.view(3, C).cpu(), z, None, None, None, 4, "gate", None, u, mean, rstd, None)
        c = [None if v is None else v.cpu() for v in (*proj, *head)]
        check_w4(u.cpu(), c[0], c[1], c[2], None, p, 64)
        check_w4(p.cpu(), c[3], c[4], c[5], None, logits, 32)


@pytest.mark.parametrize("scope", ["token", "sequence", "packed"])
def test_autograd_norm_against_differences(scope):
    """fp32, central differences of the library's own forward along random directions:
    rounding of the forward (2^-24 of |y| n over the step) stays below 1 %."""
    g = gen(7)
    T, C, G = 60, 48, 3
    x, z = torch.randn((T, C), generator=g).cuda(), torch.randn((T, C), generator=g).cuda()
    w, b = torch.randn(C, generator=g).cuda(), torch.randn(C, generator=g).cuda()
    dy = torch.randn((T, C), generator=g).cuda()
    cu = torch.tensor([2, 30, 30, 57], dtype=torch.int32).cuda()

    def f(x, w, b, z):
        if scope == "packed":
            return autograd.group_norm_varlen(cu, x, G, w, b, z, act="gate", max_seqlen=28)
        v = (lambda a: a) if scope == "token" else (lambda a: a.view(3, 20, C))
        return autograd.group_norm(v(x), G, w, b, v(z), act="gate", scope=scope).view(T, C)

    args = [v.clone().requires_grad_() for v in (x, w, b, z)]
    (f(*args) * dy).sum().backward()
    for i in range(4):
        v = torch.randn(args[i].shape, generator=g).cuda()
        eps = 2.0 ** -6
        side = []
        for sign in (1, -1):
            moved = [a.detach() for a in args]
            moved[i] = moved[i] + sign * eps * v
            side.append((f(*moved).double() * dy.double()).sum())
        diff = float(side[0] - side[1]) / (2 * eps)
        want = float((args[i].grad.double() * v.double()).sum())
        assert abs(diff - want) < 0.01 * float(args[i].grad.norm() * v.norm()), (i, diff, want)
    ok()


def test_autograd_loss_reductions_and_frozen_head():
    h, W, t, _ = [v.cuda() for v in xent_inputs(50, 90, 64, 12)]
    h.requires_grad_()
    none = autograd.linear_cross_entropy(h, W, t, reduction="none")
    assert torch.equal(autograd.linear_cross_entropy(h, W, t, reduction="sum"), none.sum())
    mean = autograd.linear_cross_entropy(h, W, t)
    assert torch.allclose(mean, none.sum() / (t != -100).sum())
    mean.backward()  # W needs no gradient
    assert W.grad is None and torch.isfinite(h.grad.float()).all()
    empty = autograd.linear_cross_entropy(h, W, torch.full_like(t, -100))
    empty.backward()
    assert float(empty) == 0.0
    ok()


def test_w4_more_tokens_than_a_grid_counts():
    """2^20 + 5 and 5 000 000 tokens (the tiles of a grid's second dimension are 65535 at
    most): the last tokens' outputs, and the ones on both sides of a cut."""
    W = (torch.randn((3, 32), generator=torch.Generator().manual_seed(1))).cuda()
    codes, scales, zeros = m3.m3_w4_quantize(W, 32)
    for M in ((1 << 20) + 5, 5_000_000):
        A = torch.randn((M, 32), device="cuda").bfloat16()
        out = m3.m3_linear_w4(A, codes, scales, zeros, out_dtype=torch.float32)
        ok()
        for a, b in ((0, 40), ((1 << 20) - 20, min((1 << 20) + 20, M)), (M - 40, M)):
            want = m3.m3_linear_w4(A[a:b].clone(), codes, scales, zeros, out_dtype=torch.float32)
            assert torch.equal(out[a:b], want)
