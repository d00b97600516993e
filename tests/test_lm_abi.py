"""Argument checks of the norm, the head's loss and the 4-bit products, at the C
entry points and in the Python binding.  Every case fails on the host: no
kernel is launched and no device address is touched."""
import ctypes

import pytest
import torch

from selective_state_space_exp_b200 import _build, autograd, m3

A16 = 0x7f0000000000
P = [A16 + 0x10000000 * i for i in range(16)]  # fake device addresses, never read
INVALID, UNSUPPORTED, ALIGN, WORKSPACE = -1, -2, -3, -4
BIG = 1 << 24  # below the distance of two addresses


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return m3.load()


def norm_shape(**kw):
    d = dict(batch=4, seqlen=10, channels=24, groups=3, io_dtype=m3.M3_BF16, act=0, eps=1e-5)
    d.update(kw)
    return m3.NormShape(**d)


def norm(lib, s, backward=False, varlen=False, **over):
    d = dict(x=P[0], w=P[1], b=P[2], z=None, y=P[3], mean=P[4], rstd=P[5], ws=P[6], n=BIG, dy=P[7],
             dx=P[8], dw=P[9], db=P[10], dz=None, cu=P[11], T=40)
    d.update(over)
    pre = [d["cu"], d["T"]] if varlen else []
    ref = None if s is None else ctypes.byref(s)
    if backward:
        fn = lib.m3_group_norm_bwd_varlen if varlen else lib.m3_group_norm_bwd
        return fn(ref, *pre, d["x"], d["w"], d["b"], d["z"], d["mean"], d["rstd"], d["dy"], d["dx"],
                  d["dw"], d["db"], d["dz"], d["ws"], d["n"], None)
    fn = lib.m3_group_norm_fwd_varlen if varlen else lib.m3_group_norm_fwd
    return fn(ref, *pre, d["x"], d["w"], d["b"], d["z"], d["y"], d["mean"], d["rstd"], d["ws"],
              d["n"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(batch=0), INVALID), (dict(seqlen=-1), INVALID), (dict(channels=0), INVALID),
    (dict(groups=0), INVALID), (dict(groups=5), INVALID), (dict(io_dtype=7), INVALID),
    (dict(act=3), INVALID), (dict(act=-1), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(batch=1 << 31), UNSUPPORTED), (dict(batch=1 << 30, groups=3), UNSUPPORTED),
    (dict(batch=1 << 20, seqlen=1 << 30), UNSUPPORTED),
])
def test_norm_shape_checks(lib, kw, expect):
    s, n = norm_shape(**kw), ctypes.c_size_t()
    for backward in (0, 1):
        assert lib.m3_group_norm_workspace_size(ctypes.byref(s), backward, 0, ctypes.byref(n)) == expect
        assert norm(lib, s, bool(backward)) == expect


@pytest.mark.parametrize("varlen", [False, True])
def test_norm_refusals(lib, varlen):
    s, gate = norm_shape(batch=1, seqlen=20000, channels=24), norm_shape(act=m3.M3_ACT_GATE)
    for f in (lambda **k: norm(lib, s, False, varlen, **k), lambda **k: norm(lib, s, True, varlen, **k)):
        assert f(x=None) == INVALID
        assert f(x=P[0] + 2) == ALIGN
        assert f(w=P[1] + 2) == ALIGN
        assert f(z=P[12]) == INVALID                 # z without the gate
        assert f(ws=None) == WORKSPACE
        assert f(n=4) == WORKSPACE
        assert f(ws=P[6] + 16) == WORKSPACE
    assert norm(lib, None) == INVALID
    assert norm(lib, s, False, varlen, y=None) == INVALID
    assert norm(lib, s, False, varlen, y=P[0] + 16) == INVALID     # overlaps x
    assert norm(lib, s, False, varlen, mean=P[3]) == INVALID       # two outputs in one place
    assert norm(lib, gate, False, varlen) == INVALID               # the gate without z
    assert norm(lib, s, True, varlen, dy=None) == INVALID
    assert norm(lib, s, True, varlen, mean=None) == INVALID
    assert norm(lib, s, True, varlen, dx=P[7]) == INVALID          # dx over dy
    assert norm(lib, s, True, varlen, dz=P[12]) == INVALID         # dz without the gate
    assert norm(lib, s, True, varlen, dw=P[10]) == INVALID         # dw and db in one place
    if varlen:
        for back in (False, True):
            assert norm(lib, s, back, True, cu=None) == INVALID
            assert norm(lib, s, back, True, cu=P[11] + 2) == INVALID
            assert norm(lib, s, back, True, T=-1) == INVALID


def test_norm_workspace_covers_the_partials(lib):
    n = ctypes.c_size_t()

    def size(s, back, packed):
        assert lib.m3_group_norm_workspace_size(ctypes.byref(s), back, packed, ctypes.byref(n)) == 0
        return n.value

    token = norm_shape(batch=100, seqlen=1, channels=4096, groups=64)
    assert size(token, 0, 0) == 0                       # statistics stay in registers
    assert size(token, 1, 0) >= 2 * 4 * 4096            # a row of partials for dw and db each
    assert size(token, 0, 1) == 0                       # a few rows a block: no partial moments
    assert size(norm_shape(batch=2, seqlen=20000), 0, 0) >= 2 * 3 * 12
    assert size(norm_shape(seqlen=0), 1, 0) == 0
    assert lib.m3_group_norm_workspace_size(None, 0, 0, ctypes.byref(n)) == INVALID
    assert lib.m3_group_norm_workspace_size(ctypes.byref(token), 0, 0, None) == INVALID


def xent(lib, backward=False, M=10, V=100, K=64, **over):
    d = dict(h=P[0], W=P[1], t=P[2], ignore=-100, loss=P[3], lse=P[4], ws=P[5], n=BIG, dl=P[6],
             dh=P[7], dW=P[8])
    d.update(over)
    if backward:
        return lib.m3_linear_xent_bwd(M, V, K, d["h"], d["W"], d["t"], d["ignore"], d["lse"], d["dl"],
                                      d["dh"], d["dW"], d["ws"], d["n"], None)
    return lib.m3_linear_xent_fwd(M, V, K, d["h"], d["W"], d["t"], d["ignore"], d["loss"], d["lse"],
                                  d["ws"], d["n"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(M=-1), INVALID), (dict(V=0), INVALID), (dict(K=0), INVALID), (dict(K=4), INVALID),
    (dict(K=12), UNSUPPORTED), (dict(M=1 << 31), UNSUPPORTED), (dict(V=1 << 31), UNSUPPORTED),
    (dict(M=1 << 30, V=1 << 30), UNSUPPORTED),
    (dict(h=None), INVALID), (dict(W=None), INVALID), (dict(t=None), INVALID),
    (dict(h=P[0] + 8), ALIGN), (dict(W=P[1] + 2), ALIGN), (dict(t=P[2] + 4), ALIGN),
    (dict(lse=P[4] + 2), ALIGN), (dict(ws=None), WORKSPACE), (dict(n=16), WORKSPACE),
    (dict(ws=P[5] + 64), WORKSPACE),
])
def test_xent_refusals(lib, kw, expect):
    for back in (False, True):
        assert xent(lib, back, **kw) == expect
    if set(kw) <= {"M", "V", "K"}:
        n = ctypes.c_size_t()
        d = dict(M=10, V=100, K=64)
        d.update(kw)
        assert lib.m3_linear_xent_fwd_workspace_size(d["M"], d["V"], d["K"], ctypes.byref(n)) == expect
        assert lib.m3_linear_xent_bwd_workspace_size(d["M"], d["V"], d["K"], ctypes.byref(n)) == expect


def test_xent_refusals_of_outputs(lib):
    assert xent(lib, loss=P[4]) == INVALID            # loss and lse in one place
    assert xent(lib, loss=P[0]) == INVALID            # an output over an input
    assert xent(lib, True, lse=None) == INVALID
    assert xent(lib, True, dl=None) == INVALID
    assert xent(lib, True, dh=P[0]) == INVALID
    assert xent(lib, True, dW=P[7]) == INVALID
    assert xent(lib, True, dh=P[7] + 8) == ALIGN
    n = ctypes.c_size_t()
    assert lib.m3_linear_xent_bwd_workspace_size(10, 100, 64, None) == INVALID
    # the workspace does not grow with the vocabulary beyond a piece of it
    assert lib.m3_linear_xent_bwd_workspace_size(16384, 50257, 2048, ctypes.byref(n)) == 0
    small = n.value
    assert lib.m3_linear_xent_bwd_workspace_size(16384, 4 * 50257, 2048, ctypes.byref(n)) == 0
    assert n.value < 1.2 * small < 16384 * 50257 * 2


def w4(lib, M=3, N=40, K=256, G=64, **over):
    d = dict(A=P[0], codes=P[1], scales=P[2], zeros=P[3], bias=P[4], out=P[5], dt=m3.M3_BF16)
    d.update(over)
    return lib.m3_linear_w4(M, N, K, G, d["A"], d["codes"], d["scales"], d["zeros"], d["bias"],
                            d["out"], d["dt"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(K=100), INVALID),
    (dict(G=0), INVALID), (dict(G=16), UNSUPPORTED), (dict(G=256), UNSUPPORTED),
    (dict(N=1 << 30), UNSUPPORTED), (dict(M=1 << 30), UNSUPPORTED), (dict(dt=5), INVALID),
    (dict(A=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(out=None), INVALID), (dict(A=P[0] + 8), ALIGN), (dict(codes=P[1] + 4), ALIGN),
    (dict(scales=P[2] + 2), ALIGN), (dict(zeros=P[3] + 1), ALIGN), (dict(bias=P[4] + 2), ALIGN),
    (dict(out=P[5] + 2), ALIGN), (dict(out=P[0]), INVALID), (dict(out=P[1] + 16), INVALID),
    (dict(out=P[4]), INVALID),
])
def test_w4_refusals(lib, kw, expect):
    assert w4(lib, **kw) == expect


def test_w4_no_token_is_no_work(lib):
    assert w4(lib, M=0, A=None, out=None) == 0


@pytest.mark.parametrize("kw,expect", [
    (dict(N=0), INVALID), (dict(K=100), INVALID), (dict(G=48), UNSUPPORTED), (dict(dt=9), INVALID),
    (dict(W=None), INVALID), (dict(W=P[0] + 2), ALIGN), (dict(codes=P[1] + 8), ALIGN),
    (dict(codes=P[0]), INVALID), (dict(scales=P[1] + 16), INVALID),
])
def test_w4_quantize_refusals(lib, kw, expect):
    d = dict(N=8, K=256, G=64, dt=m3.M3_BF16, W=P[0], codes=P[1], scales=P[2], zeros=P[3])
    d.update(kw)
    assert lib.m3_w4_quantize(d["N"], d["K"], d["G"], d["dt"], d["W"], d["codes"], d["scales"],
                              d["zeros"], None) == expect


def test_binding_refuses_before_the_library():
    """CPU tensors and mismatched arguments never reach a call."""
    x, w = torch.zeros((4, 8)), torch.zeros((8,))
    with pytest.raises(ValueError, match="CUDA device"):
        m3.m3_group_norm_fwd(x, 2, w)
    with pytest.raises(ValueError, match="groups"):
        m3.m3_group_norm_fwd(x, 3)
    with pytest.raises(ValueError, match="groups"):
        m3.m3_group_norm_fwd(x, 0)
    with pytest.raises(ValueError, match="scope"):
        m3.m3_group_norm_fwd(x, 2, scope="row")
    with pytest.raises(ValueError, match="seqlen"):
        m3.m3_group_norm_fwd(x, 2, scope="sequence")
    with pytest.raises(ValueError, match="act"):
        m3.m3_group_norm_fwd(x, 2, act="relu")
    with pytest.raises(ValueError, match="packed"):
        m3.m3_group_norm_fwd_varlen(torch.zeros(2, dtype=torch.int32), x[None], 2)
    h, W, t = torch.zeros((4, 8), dtype=torch.bfloat16), torch.zeros((5, 8)), torch.zeros(4, dtype=torch.long)
    with pytest.raises(ValueError, match="CUDA device"):
        m3.m3_linear_xent_fwd(h, W.bfloat16(), t)
    with pytest.raises(ValueError, match="expected"):
        m3.m3_linear_xent_fwd(h, torch.zeros((5, 16), dtype=torch.bfloat16), t)
    with pytest.raises(ValueError, match="groups of"):
        m3.m3_w4_quantize(torch.zeros((4, 100)), 64)
    with pytest.raises(ValueError, match="groups of"):
        m3.m3_w4_quantize(torch.zeros((4, 128)), 16)
    codes, scales = torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((4, 1), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="expected"):
        m3.m3_linear_w4(torch.zeros((1, 64), dtype=torch.bfloat16), codes, scales)
    with pytest.raises(ValueError, match="inputs"):
        m3.m3_linear_w4(torch.zeros((1, 128), dtype=torch.bfloat16), codes,
                        torch.zeros((4, 3), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="reduction"):
        autograd.linear_cross_entropy(h, W, t, reduction="max")


def test_w4_without_inputs_is_refused():
    with pytest.raises(ValueError, match="0 inputs"):
        m3.m3_linear_w4(torch.zeros((1, 0), dtype=torch.bfloat16), torch.zeros((4, 0), dtype=torch.uint8),
                        torch.zeros((4, 1), dtype=torch.bfloat16))


@pytest.mark.parametrize("dt", [m3.M3_BF16, m3.M3_F32])
def test_norm_of_more_blocks_than_a_grid_has(lib, dt):
    """Groups so wide that a sample takes thousands of blocks: refused by the size query and by
    the calls alike, not at the launch."""
    n = ctypes.c_size_t()
    for kw, packed in ((dict(batch=1 << 20, seqlen=2), False), (dict(batch=1 << 20, seqlen=1), False),
                       (dict(batch=1 << 20, seqlen=2), True)):
        s = norm_shape(channels=(1 << 24) + 8, groups=1, io_dtype=dt, **kw)  # 8193 blocks or more a sample
        for back in (0, 1):
            assert lib.m3_group_norm_workspace_size(ctypes.byref(s), back, int(packed), ctypes.byref(n)) == UNSUPPORTED
        if packed:
            continue
        far = [(i + 1) << 50 for i in range(12)]
        at = dict(x=far[0], w=far[1], b=far[2], mean=far[4], rstd=far[5], ws=far[6], dy=far[7], dw=far[9], db=far[10])
        assert norm(lib, s, False, y=far[3], **at) == UNSUPPORTED
        assert norm(lib, s, True, dx=far[8], **at) == UNSUPPORTED


def test_xent_workspace_is_for_the_wanted_gradients(lib):
    """A frozen head's call holds no copy of the hidden states and no sums of dW."""
    n = ctypes.c_size_t()

    def size(M, V, K, dh, dW):
        assert lib.m3_linear_xent_bwd_workspace_size_for(M, V, K, dh, dW, ctypes.byref(n)) == 0
        return n.value

    for M, V, K in ((10, 100, 64), (2000, 120, 1000), (16384, 50257, 2048), (40, 9000, 1040), (77, 1003, 256)):
        assert lib.m3_linear_xent_bwd_workspace_size(M, V, K, ctypes.byref(n)) == 0
        both = n.value
        assert size(M, V, K, 1, 1) == both
        assert both - size(M, V, K, 1, 0) >= M * K * 2
        assert size(M, V, K, 1, 0) >= M * V * 2 or V > 8000     # d itself
        assert M * K * 2 <= size(M, V, K, 0, 1) <= both
        assert size(M, V, K, 0, 0) == 0
        for want, out in (((1, 0), dict(dW=None)), ((0, 1), dict(dh=None))):
            assert xent(lib, True, M=M, V=V, K=K, n=size(M, V, K, *want) - 1, **dict(far(), **out)) == WORKSPACE
    assert size(0, 100, 64, 1, 1) == 0
    # several pieces of the vocabulary: the running sum of dh is a part
    assert size(16384, 50257, 2048, 1, 1) - size(16384, 50257, 2048, 0, 1) >= 16384 * 2048 * 4
    assert lib.m3_linear_xent_bwd_workspace_size_for(10, 0, 64, 1, 1, ctypes.byref(n)) == INVALID
    assert lib.m3_linear_xent_bwd_workspace_size_for(10, 100, 12, 1, 1, ctypes.byref(n)) == UNSUPPORTED
    assert lib.m3_linear_xent_bwd_workspace_size_for(10, 100, 64, 1, 1, None) == INVALID


def far():
    """Addresses for xent() so far apart that the largest tensors do not overlap."""
    return {k: (i + 1) << 40 for i, k in enumerate(("h", "W", "t", "lse", "ws", "dl", "dh", "dW"))} | {"loss": None}
