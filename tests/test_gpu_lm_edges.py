"""The grouped norm, the head's cross entropy and the 4-bit products on the GPU, at
inputs and in uses where they could go wrong and that test_gpu_lm.py does not reach,
against the same fp64 oracle (oracle/m3_lm.py)."""
import numpy as np
import pytest
import torch

from oracle import m3_lm as lm
from selective_state_space_exp_b200 import m3
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


def f64(t):
    return t.detach().cpu().double().numpy()


# ---- statistics with an outlier ----------------------------------------------------

# samples, positions, groups, channels of a group.  One block makes both passes; one block
# a tile, but too many rows a thread for both; several blocks a sample; a group wider than a
# block; channels of four bytes
OUTLIER = [(4, 128, 32, 64), (3, 7, 2, 16), (300, 40, 16, 64), (2, 3000, 2, 24), (1, 9000, 1, 8), (3, 61, 1, 4100),
           (3, 1001, 6, 85)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("far", [50.0, 300.0, 1000.0])
@pytest.mark.parametrize("B,L,G,cg", OUTLIER)
def test_statistics_with_an_outlier_first(B, L, G, cg, far, io):
    """The first value of every group, or its whole first position, stands far from the
    others (language models put their largest activations at the first position).

    Sums of squares are of positive terms: 32 in a piece (8 rows x 4 pairs), at most 10
    pieces of a thread, 8 threads of a lane, 5 steps of lanes and 10 of splits, 65 additions
    in a chain, and as much again for what the moves of the reference take off: 130 roundings
    of the variance, 65 of rstd.  The mean's error is as many of the deviation, and one of
    the mean itself."""
    g = gen(B + L + G + cg)
    x = torch.randn((B, L, G, cg), generator=g)
    x[0::2, 0, :, 0] = far
    if B > 1:
        x[1::2, 0] = far
    x = x.to(IO[io]).view(B, L, G * cg)
    y, mean, rstd = m3.m3_group_norm_fwd(x.cuda(), G, scope="sequence")
    ok()
    v = f64(x.float()).reshape(B, L, G, cg).transpose(0, 2, 1, 3).reshape(B, G, -1)
    mu = v.mean(-1)
    inv = 1 / np.sqrt(((v - mu[..., None]) ** 2).mean(-1) + 1e-5)
    assert (np.abs(f64(rstd) / inv - 1)).max() <= 72 * U
    assert (np.abs(f64(mean) - mu) * inv - U * np.abs(mu) * inv).max() <= 72 * U
    want = (v - mu[..., None]) * inv[..., None]
    got = f64(y.float()).reshape(B, L, G, cg).transpose(0, 2, 1, 3).reshape(B, G, -1)
    # xh: 72 roundings from rstd and of the deviation from the mean, a few of its own
    over = np.abs(got - want) - torch.finfo(IO[io]).eps / 2 * np.abs(want) - 80 * U * (np.abs(want) + 1)
    assert over.max() <= 0


def test_packed_statistics_with_outliers_in_a_long_sequence():
    """One long sequence among hundreds of short ones: its rows are one block's."""
    cu = np.concatenate([np.arange(0, 700 * 3, 3), [2100, 2100 + 2000]]).astype(np.int32)
    T, G, cg = int(cu[-1]), 2, 32
    x = torch.randn((T, G * cg), generator=gen(3))
    x[2100] = 1000.0
    x[::7, 5] = 300.0
    c = torch.from_numpy(cu).cuda()
    y, mean, rstd = m3.m3_group_norm_fwd_varlen(c, x.cuda(), G, max_seqlen=2000)
    ok()
    ref = lm.group_norm(x, G, spans=list(zip(cu[:-1], cu[1:])))
    # a thread has 125 rows of the long one: pieces of 8 additions, 31 of them, 8 threads a
    # lane and 5 steps of lanes, twice for the moves: 104 roundings of the variance
    assert (np.abs(f64(rstd) / ref["rstd"] - 1)).max() <= 56 * U
    assert (np.abs(f64(y) - ref["y"]) - 64 * U * (np.abs(ref["y"]) + 1)).max() <= 0


# ---- parameter gradients over many rows ------------------------------------------------

def parameter_bounds(x, z, dy, w, b, G, act, spans):
    """fp64 dw and db, and what roundings may move them by, from the sums of the terms'
    magnitudes.  256 roundings of the sum (a thread, the row slots, the partial rows: far
    shorter chains), and of each term:
      xh  8 (|xh| + 1): x - mean and rstd
      u = xh w + b  |w| of that and 2 (|u| + |b|)
      g   silu' has a slope of at most 1/2: |dy| (du / 2 + 16 (1 + |u|)), the sigmoid's own
          error (2^-22 of ex2 and rcp and the exponent's rounding) among the 16; the gate's
          factor z sigma(z) likewise 16 (1 + |z|)"""
    ref = lm.group_norm(x, G, w, b, z, act, 1e-5, spans, dy)
    xs, dys, ws, bs = (lm.f64(v) for v in (x, dy, w, b))
    C = xs.shape[1]
    xh = np.zeros_like(xs)
    for i, (t0, t1) in enumerate(spans):
        xh[t0:t1] = (xs[t0:t1] - np.repeat(ref["mean"][i], C // G)) * np.repeat(ref["rstd"][i], C // G)
    u = xh * ws + bs
    exh = 8 * U * (np.abs(xh) + 1)
    if act == "silu":
        s = lm.sigmoid(u)
        g = dys * s * (1 + u * (1 - s))
        eg = np.abs(dys) * ((np.abs(ws) * exh + 2 * U * (np.abs(u) + np.abs(bs))) / 2 + 16 * U * (1 + np.abs(u)))
    elif act == "gate":
        zs = lm.f64(z)
        g = dys * zs * lm.sigmoid(zs)
        eg = np.abs(dys) * 16 * U * (1 + np.abs(zs)) * np.abs(zs)
    else:
        g, eg = dys, 0 * dys
    tw = 256 * U * np.abs(g * xh).sum(0) + (eg * np.abs(xh) + np.abs(g) * exh).sum(0)
    tb = 256 * U * np.abs(g).sum(0) + eg.sum(0)
    return ref, tw, tb


# samples, positions, groups, channels of a group: one block each, several splits, groups in
# pieces, and single positions (the unit kernels' partial rows)
MANY = [(2, 3000, 2, 24), (1, 9000, 1, 8), (1, 8193, 1, 8), (2, 900, 40, 8), (4, 300, 3, 31), (3, 700, 3, 31),
        (2, 400, 1, 4100), (700, 40, 2, 24), (5000, 1, 6, 8), (3000, 1, 1, 600), (900, 1, 1, 4104)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "silu", "gate"])
@pytest.mark.parametrize("B,L,G,cg", MANY)
def test_parameter_gradients_over_many_rows(B, L, G, cg, act, io):
    """Every partial sum counts: the bounds are far below the gradients, which is checked."""
    g = gen(B * 3 + L + G + cg)
    C, dt = G * cg, IO[io]
    x, z, dy = (torch.randn((B * L, C), generator=g).to(dt) for _ in range(3))
    x = (x * 1.5).to(dt)
    z = z if act == "gate" else None
    w, b = torch.randn(C, generator=g) * 0.2 + 1, torch.randn(C, generator=g) * 0.3
    d = [None if v is None else v.cuda().view(B, L, C) for v in (x, z, dy)]
    y, mean, rstd = m3.m3_group_norm_fwd(d[0], G, w.cuda(), b.cuda(), d[1], act=act, scope="sequence")
    got = m3.m3_group_norm_bwd(d[0], G, mean, rstd, d[2], w.cuda(), b.cuda(), d[1], act=act, scope="sequence")
    ok()
    ref, tw, tb = parameter_bounds(x, z, dy, w, b, G, act, [(i * L, (i + 1) * L) for i in range(B)])
    for name, tol, want in (("weight", tw, ref["w"]), ("bias", tb, ref["b"])):
        assert tol.max() < 0.01 * np.sqrt((want ** 2).mean()), (name, tol.max())
        assert (np.abs(f64(got[name]) - want) - tol).max() <= 0, name


# ---- pairs of CTAs -----------------------------------------------------------------------

def test_pairs_of_ctas_back_to_back():
    """The loss in pairs of CTAs (at least 55 tiles of 256 x 256), again and again between
    kernels that take the same SMs at once: the last arrivals of a pair reach it, not what
    runs there next, and every repetition gives the same bits."""
    g = gen(21)
    h = torch.randn((600, 136), generator=g).bfloat16().cuda()
    W = (torch.randn((9000, 136), generator=g) / 12).bfloat16().cuda()
    t = torch.randint(0, 9000, (600,), generator=g).cuda()
    dl = torch.rand(600, generator=g).cuda()
    small = torch.randint(0, 1003, (77,), generator=g).cuda()
    codes, scales, zeros = m3.m3_w4_quantize(W[:2048, :128].contiguous(), 64)

    def step():
        loss, lse = m3.m3_linear_xent_fwd(h, W, t)
        out = m3.m3_linear_w4(h[:128, :128].contiguous(), codes, scales, zeros)
        grads = m3.m3_linear_xent_bwd(h, W, t, lse, dl)
        few = m3.m3_linear_xent_fwd(h[:77], W[:1003], small)
        return (loss, lse, out, *grads, *few)

    first = step()
    ok()
    ref = lm.xent(h, W, t)
    assert np.abs(f64(first[1]) - ref["lse"]).max() < 1e-4
    for _ in range(100):
        again = step()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    ok()


# ---- host threads --------------------------------------------------------------------------

def test_w4_from_several_host_threads():
    """Calls whose plans take different amounts of shared memory, from four threads at once
    on streams of their own."""
    import threading
    g = gen(31)
    cases = []
    for K in (64, 512, 4096, 20480):
        A = torch.randn((1, K), generator=g).bfloat16().cuda()
        q = m3.m3_w4_quantize(torch.randn((48, K), generator=g).cuda(), 64)
        cases.append((A, q, m3.m3_linear_w4(A, *q, out_dtype=torch.float32)))
    ok()
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(len(cases))

    def work(A, q, want, stream):
        try:
            start.wait(60)
            outs = [m3.m3_linear_w4(A, *q, out_dtype=torch.float32, stream=stream) for _ in range(400)]
            stream.synchronize()
            assert all(torch.equal(o, want) for o in outs)
        except Exception as e:  # noqa: BLE001  (reported by the test's own thread)
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(*c, torch.cuda.Stream())) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    ok()
    assert not wrong, wrong


# ---- the bounds-checked build ----------------------------------------------------------------

def test_larger_forms_in_bounds():
    """The forms that only larger calls take, through the bounds-checked build."""
    import os
    import subprocess
    import sys
    from selective_state_space_exp_b200 import _build
    _build.build(debug=True)
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, os.path.join(here, "debug_bounds_lm_forms_child.py")],
                       env=dict(os.environ, M3_LIBRARY="debug"), capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and "ALL OK" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]


# ---- gradients that are not wanted, gradients that lie anywhere --------------------------------

@pytest.mark.parametrize("L", [1, 30, 3000])
def test_norm_gradients_that_are_not_wanted(L):
    """Any set of the four gradients has the bits of the whole call (the forms of single
    positions, of both passes in one block, of several splits)."""
    g = gen(41 + L)
    x, z, dy = (torch.randn((2, L, 48), generator=g).cuda() for _ in range(3))
    w, b = torch.randn(48, generator=g).cuda(), torch.randn(48, generator=g).cuda()
    kw = dict(act="gate", scope="sequence")
    y, mean, rstd = m3.m3_group_norm_fwd(x, 2, w, b, z, **kw)
    full = m3.m3_group_norm_bwd(x, 2, mean, rstd, dy, w, b, z, **kw)
    names = ("x", "weight", "bias", "z")
    for bits in range(16):
        on = [bool(bits >> i & 1) for i in range(4)]
        some = m3.m3_group_norm_bwd(x, 2, mean, rstd, dy, w, b, z, want_dx=on[0], want_dweight=on[1],
                                    want_dbias=on[2], want_dz=on[3], **kw)
        for name, want in zip(names, on):
            assert torch.equal(some[name], full[name]) if want else some[name] is None, (bits, name)
    ok()


def test_norm_gradient_of_a_part_of_a_cat():
    """torch.cat along the tokens hands the norm a gradient that starts off a 16-byte
    boundary: 3 channels of 4 bytes."""
    from selective_state_space_exp_b200 import autograd
    x = torch.randn((5, 3), generator=gen(51)).cuda().requires_grad_()
    w = torch.randn((6, 3), generator=gen(52)).cuda()
    head = torch.zeros((1, 3), device="cuda")
    (torch.cat([head, autograd.group_norm(x, 1)]) * w).sum().backward()
    ok()
    ref = lm.group_norm(x, 1, dy=w[1:])
    assert np.abs(f64(x.grad) - ref["x"]).max() < 256 * U * ref["rstd"].max() * 8


# ---- explicit streams -----------------------------------------------------------------------------

def stream_calls():
    """Name: (inputs' maker, call of them on a stream)."""
    g = gen(61)
    x = torch.randn((900, 512), generator=g)
    h = torch.randn((900, 512), generator=g).bfloat16()
    W = (torch.randn((700, 512), generator=g) / 20).bfloat16()
    t = torch.randint(0, 700, (900,), generator=g)
    cu = torch.tensor([0, 400, 900], dtype=torch.int32)
    codes = torch.randint(0, 256, (700, 256), generator=g, dtype=torch.uint8)
    scales = (torch.rand((700, 8), generator=g) / 50).bfloat16()

    def norm(x, stream):
        y, m, r = m3.m3_group_norm_fwd(x, 4, stream=stream)
        return (y, *m3.m3_group_norm_bwd(x, 4, m, r, x, stream=stream).values())

    def packed(c, x, stream):
        y, m, r = m3.m3_group_norm_fwd_varlen(c, x, 4, max_seqlen=500, stream=stream)
        return (y, *m3.m3_group_norm_bwd_varlen(c, x, 4, m, r, x, max_seqlen=500, stream=stream).values())

    def loss(h, W, t, stream):
        out, lse = m3.m3_linear_xent_fwd(h, W, t, stream=stream)
        return (out, *m3.m3_linear_xent_bwd(h, W, t, lse, torch.ones_like(out), stream=stream))

    return {"norm": ((x,), norm), "packed": ((cu, x), packed), "loss": ((h, W, t), loss),
            "w4": ((h, codes, scales), lambda *a, stream: (m3.m3_linear_w4(*a, stream=stream),)),
            "quantize": ((W,), lambda W, stream: m3.m3_w4_quantize(W, 64, stream=stream))}


@pytest.mark.parametrize("name", ["norm", "packed", "loss", "w4", "quantize"])
def test_inputs_may_be_let_go_before_their_stream_has_run(name):
    """The call waits on its stream behind other work; meanwhile its inputs are let go, and
    what the current stream then makes does not land in their memory."""
    host, call = stream_calls()[name]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = call(*[t.cuda() for t in host], stream=None)
    inputs = [t.cuda() for t in host]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # a tenth of a second
    got = call(*inputs, stream=side)
    sizes = [(t.shape, t.dtype) for t in inputs]
    del inputs
    held = [torch.empty(s, dtype=d, device="cuda").view(torch.uint8).fill_(255) for s, d in sizes for _ in range(3)]
    side.synchronize()
    ok()
    assert held and all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("name", ["norm", "packed", "loss", "w4", "quantize"])
def test_outputs_may_be_let_go_before_the_current_stream_has_read_them(name):
    host, call = stream_calls()[name]
    side = torch.cuda.Stream()
    inputs = [t.cuda() for t in host]
    want = call(*inputs, stream=None)
    torch.cuda.synchronize()
    got = call(*inputs, stream=side)
    side.synchronize()
    torch.cuda._sleep(200_000_000)
    copies = [t.clone() for t in got]          # behind the sleep
    sizes = [(t.shape, t.dtype) for t in got]
    del got
    with torch.cuda.stream(side):
        held = [torch.empty(s, dtype=d, device="cuda").view(torch.uint8).fill_(255) for s, d in sizes for _ in range(3)]
    torch.cuda.synchronize()
    ok()
    assert held and all(torch.equal(a, b) for a, b in zip(want, copies))


# ---- workspaces ---------------------------------------------------------------------------------

@pytest.mark.parametrize("M,V,K", [(300, 700, 64), (2000, 120, 1000), (20000, 15000, 16), (40, 9000, 1040)])
def test_loss_workspace_of_the_wanted_gradients(M, V, K):
    """dh or dW alone in a workspace of just its size, what lies behind it left as it was;
    the bits are those of both at once (one piece, a split dW, three pieces, a split dh)."""
    import ctypes
    g = gen(71 + M)
    h = torch.randn((M, K), generator=g).bfloat16().cuda()
    W = (torch.randn((V, K), generator=g) / K ** 0.5).bfloat16().cuda()
    t = torch.randint(0, V, (M,), generator=g).cuda()
    t[::7] = -100
    dl = torch.rand(M, generator=g).cuda()
    loss, lse = m3.m3_linear_xent_fwd(h, W, t)
    dh, dW = m3.m3_linear_xent_bwd(h, W, t, lse, dl)
    n = ctypes.c_size_t()
    for want in ((True, False), (False, True)):
        assert m3.load().m3_linear_xent_bwd_workspace_size_for(M, V, K, *map(int, want), ctypes.byref(n)) == 0
        whole = torch.full((n.value + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
        got = m3.m3_linear_xent_bwd(h, W, t, lse, dl, want_dh=want[0], want_dW=want[1], workspace=whole[:n.value])
        ok()
        assert (whole[n.value:] == 0xAB).all()
        assert all(torch.equal(a, b) if w else a is None for a, b, w in zip(got, (dh, dW), want))


# ---- equal values, values that are not finite, over sequences ------------------------------------

@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,L,G,cg", [(4, 128, 32, 64), (300, 40, 16, 64), (2, 3000, 2, 24), (3, 61, 1, 4100), (3, 1001, 6, 85)])
def test_slices_of_equal_values(B, L, G, cg, io):
    """A slice without spread, far from 0: the mean is its value exactly, and y the bias."""
    v = (torch.randn((B, 1, G, 1), generator=gen(81)) * 3000).to(IO[io]).float()
    x = v.expand(B, L, G, cg).reshape(B, L, G * cg).to(IO[io]).contiguous().cuda()
    b = torch.randn(G * cg, generator=gen(82)).bfloat16().float()
    y, mean, rstd = m3.m3_group_norm_fwd(x, G, bias=b.cuda(), scope="sequence")
    ok()
    assert torch.equal(mean.cpu(), v.view(B, G))
    assert torch.equal(y.float().cpu(), b.expand(B, L, G * cg))


@pytest.mark.parametrize("B,L,G,cg", [(4, 128, 32, 64), (300, 40, 16, 64), (2, 3000, 2, 24), (3, 1001, 6, 85)])
def test_values_that_are_not_finite_stay_in_their_slice(B, L, G, cg):
    x = torch.randn((B, L, G, cg), generator=gen(91))
    x[0, 0, 0, 0], x[1, L - 1, G - 1, 3], x[-1, L // 2, 1, 1] = float("nan"), float("inf"), -float("inf")
    clean = torch.randn((B, L, G, cg), generator=gen(91))
    y, mean, rstd = m3.m3_group_norm_fwd(x.view(B, L, -1).cuda(), G, scope="sequence")
    want = m3.m3_group_norm_fwd(clean.view(B, L, -1).cuda(), G, scope="sequence")
    ok()
    bad = ~torch.isfinite(x).all(3).all(1)                       # [B][G]
    y, ref = y.view(B, L, G, cg).cpu(), want[0].view(B, L, G, cg).cpu()
    for i, g in bad.nonzero().tolist():
        assert not torch.isfinite(y[i, :, g]).any() and not torch.isfinite(rstd[i, g])
    assert torch.equal(torch.where(bad[:, None, :, None], ref, y), ref)
    assert torch.equal(torch.where(bad, want[2].cpu(), rstd.cpu()), want[2].cpu())
