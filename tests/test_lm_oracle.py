"""Pins of the fp64 oracle of the norm, the head's loss and the 4-bit products
(oracle/m3_lm.py) to things other than itself: closed forms, invariances, and
central differences for every gradient."""
import numpy as np
import pytest

from oracle import m3_lm as lm


def diff(f, x, i, eps=1e-6):
    a, b = x.copy(), x.copy()
    a.flat[i] += eps
    b.flat[i] -= eps
    return (f(a) - f(b)) / (2 * eps)


@pytest.mark.parametrize("act", ["none", "silu", "gate"])
@pytest.mark.parametrize("spans", [None, [(0, 3), (3, 3), (3, 7)]])
def test_group_norm_gradients_equal_differences(act, spans):
    rng = np.random.default_rng(1)
    T, G, cg = 7, 3, 4
    C = G * cg
    x, dy = rng.standard_normal((T, C)), rng.standard_normal((T, C))
    w, b = rng.standard_normal(C), rng.standard_normal(C)
    z = rng.standard_normal((T, C)) if act == "gate" else None
    kw = dict(groups=G, act=act, spans=spans)
    g = lm.group_norm(x, w=w, b=b, z=z, dy=dy, **kw)

    def total(x=x, w=w, b=b, z=z):
        return float((lm.group_norm(x, w=w, b=b, z=z, **kw)["y"] * dy).sum())

    for name, v, f in (("x", x, lambda v: total(x=v)), ("w", w, lambda v: total(w=v)),
                       ("b", b, lambda v: total(b=v)), ("z", z, lambda v: total(z=v))):
        if v is None:
            continue
        for i in range(0, v.size, 5):
            assert abs(diff(f, v, i) - g[name].flat[i]) < 1e-6, (name, i)


def test_group_norm_closed_forms():
    # two values: xh = (-1, 1) for eps = 0; a shift or a positive scale changes nothing
    y = lm.group_norm(np.array([[3.0, 7.0]]), 1, eps=0.0)
    assert np.allclose(y["y"], [[-1.0, 1.0]]) and y["mean"][0, 0] == 5.0 and y["rstd"][0, 0] == 0.5
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 8))
    a = lm.group_norm(x, 2, eps=0.0)["y"]
    assert np.allclose(a, lm.group_norm(3.0 * x + 11.0, 2, eps=0.0)["y"], atol=1e-12)
    # each group of each sample: mean 0, variance 1
    v = a.reshape(5, 2, 4)
    assert np.allclose(v.mean(-1), 0, atol=1e-12) and np.allclose((v ** 2).mean(-1), 1)
    # one sample over all rows equals normalising the rows' values together
    s = lm.group_norm(x, 1, eps=0.0, spans=[(0, 5)])["y"]
    assert np.allclose(s, (x - x.mean()) / x.std(), atol=1e-12)
    # a gate of 0 closes, a large one passes z through
    assert np.all(lm.group_norm(x, 2, z=np.zeros_like(x), act="gate")["y"] == 0.0)
    big = lm.group_norm(x, 2, z=np.full_like(x, 50.0), act="gate")["y"]
    assert np.allclose(big, 50.0 * lm.group_norm(x, 2)["y"])


def test_xent_closed_forms():
    # equal logits: log V; V = 1: 0; a class far above the others: 0 for it
    h = np.ones((2, 3))
    r = lm.xent(h, np.zeros((7, 3)), np.array([2, 5]))
    assert np.allclose(r["loss"], np.log(7.0)) and np.allclose(r["lse"], np.log(7.0))
    assert np.allclose(lm.xent(h, np.ones((1, 3)), np.array([0, 0]))["loss"], 0.0)
    W = np.zeros((3, 3))
    W[1] = 100.0
    assert abs(lm.xent(h, W, np.array([1, 1]))["loss"][0]) < 1e-12
    # an ignored token: loss 0, no gradient from it
    r = lm.xent(h, np.eye(3), np.array([-100, 1]), dloss=np.array([1.0, 1.0]))
    assert r["loss"][0] == 0.0 and np.all(r["h"][0] == 0.0) and np.any(r["h"][1] != 0.0)
    # the gradient of the logits of a token sums to 0
    assert np.allclose(r["d"].sum(1), 0.0, atol=1e-14)


def test_xent_gradients_equal_differences():
    rng = np.random.default_rng(3)
    M, V, K = 5, 9, 4
    h, W = rng.standard_normal((M, K)), rng.standard_normal((V, K))
    t, dl = np.array([0, 8, -100, 3, 3]), rng.standard_normal(M)
    g = lm.xent(h, W, t, dloss=dl)
    for i in range(h.size):
        assert abs(diff(lambda v: (lm.xent(v, W, t)["loss"] * dl).sum(), h, i) - g["h"].flat[i]) < 1e-6
    for i in range(W.size):
        assert abs(diff(lambda v: (lm.xent(h, v, t)["loss"] * dl).sum(), W, i) - g["W"].flat[i]) < 1e-6


def test_w4_layout_by_hand():
    # codes 1..4 of one row, group of two: (q - z) s
    codes = np.array([[0x21, 0x43]], dtype=np.uint8)
    w = lm.w4_weights(codes, np.array([[2.0, 10.0]]), np.array([[1, 3]]))
    assert w.tolist() == [[0.0, 2.0, 0.0, 10.0]]
    assert lm.w4_weights(codes, np.array([[1.0, 1.0]])).tolist() == [[-7.0, -6.0, -5.0, -4.0]]
    out = lm.w4_linear(np.array([[1.0, 1.0, 1.0, 2.0]]), codes, np.array([[2.0, 10.0]]),
                       np.array([[1, 3]]), bias=np.array([0.5]))
    assert out.tolist() == [[22.5]]
