"""The autograd functions of the norm and the head's loss on the CPU, the library's
calls replaced by the formulas in torch: what the functions make of arguments and
gradients, not the kernels."""
import pytest
import torch

from selective_state_space_exp_b200 import autograd, m3

EPS = 1e-5


def _norm(x, groups, weight, bias, z, act):
    v = x.view(*x.shape[:-1], groups, -1)
    mean = v.mean(-1, keepdim=True)
    rstd = (((v - mean) ** 2).mean(-1, keepdim=True) + EPS).rsqrt()
    u = ((v - mean) * rstd).reshape(x.shape)
    u = u * (1 if weight is None else weight) + (0 if bias is None else bias)
    if act == "silu":
        u = torch.nn.functional.silu(u)
    elif act == "gate":
        u = u * torch.nn.functional.silu(z)
    return u, mean.reshape(-1, groups), rstd.reshape(-1, groups)


@pytest.fixture
def calls(monkeypatch):
    """The library's calls as torch formulas; yields a list of the keyword arguments
    that the backward calls got."""
    seen = []

    def fwd(x, groups, weight=None, bias=None, z=None, *, act="none", y=None, **kw):
        out, mean, rstd = _norm(x, groups, weight, bias, z, act)
        if y is not None:
            out = y.copy_(out)
        return out, mean, rstd

    def bwd(x, groups, mean, rstd, dy, weight=None, bias=None, z=None, *, act="none", **kw):
        seen.append(dict(kw, dy=dy))
        with torch.enable_grad():
            names = [n for n, t in (("x", x), ("weight", weight), ("bias", bias), ("z", z)) if t is not None]
            leaves = [t.detach().clone().requires_grad_() for t in (x, weight, bias, z) if t is not None]
            at = dict(zip(names, leaves))
            y = _norm(at["x"], groups, at.get("weight"), at.get("bias"), at.get("z"), act)[0]
            wants = dict(x="want_dx", weight="want_dweight", bias="want_dbias", z="want_dz")
            return {n: t if kw[wants[n]] else None for n, t in zip(names, torch.autograd.grad(y, leaves, dy))}

    def loss_fwd(h, W, targets, **kw):
        logits = h.float() @ W.float().T
        lse = torch.logsumexp(logits, -1)
        return lse - logits.gather(-1, targets[..., None])[..., 0], lse

    def loss_bwd(h, W, targets, lse, dloss, *, want_dh=True, want_dW=True, **kw):
        seen.append(dict(kw, dloss=dloss, want_dh=want_dh, want_dW=want_dW))
        d = torch.exp(h.float() @ W.float().T - lse[..., None])
        d = (d - torch.nn.functional.one_hot(targets, W.shape[0])) * dloss[..., None]
        return (d @ W.float()).to(h.dtype) if want_dh else None, (d.T @ h.float()).to(W.dtype) if want_dW else None

    monkeypatch.setattr(m3, "m3_group_norm_fwd", fwd)
    monkeypatch.setattr(m3, "m3_group_norm_bwd", bwd)
    monkeypatch.setattr(m3, "m3_group_norm_fwd_varlen", lambda cu, *a, **k: fwd(*a, **k))
    monkeypatch.setattr(m3, "m3_group_norm_bwd_varlen", lambda cu, *a, **k: bwd(*a, **k))
    monkeypatch.setattr(m3, "m3_linear_xent_fwd", loss_fwd)
    monkeypatch.setattr(m3, "m3_linear_xent_bwd", loss_bwd)
    return seen


def randn(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed + sum(shape)))


def norm_calls(T=6, C=8):
    cu = torch.tensor([0, 2, T], dtype=torch.int32)
    return {
        "token": lambda x, w, b, z: autograd.group_norm(x, 2, w, b, z, act="gate"),
        "packed": lambda x, w, b, z: autograd.group_norm_varlen(cu, x, 2, w, b, z, act="gate", max_seqlen=4),
    }


@pytest.mark.parametrize("which", ["token", "packed"])
def test_first_derivatives_pass_and_second_ones_raise(calls, which):
    """A term of the gradient in the loss (a gradient penalty) has no derivative here:
    it must not be left out in silence."""
    f = norm_calls()[which]
    args = [randn(6, 8).requires_grad_(), randn(8).requires_grad_(), randn(8, seed=1).requires_grad_(),
            randn(6, 8, seed=2).requires_grad_()]
    plain = torch.autograd.grad(f(*args).square().sum(), args)
    # below a square the incoming gradient has a history of its own, below a sum it has none
    for top in (lambda y: y.square().sum(), lambda y: y.sum()):
        first = torch.autograd.grad(top(f(*args)), args, create_graph=True)
        assert all(torch.isfinite(g).all() for g in first)
        for g in first:
            assert g.requires_grad
            with pytest.raises(RuntimeError, match="first derivatives only"):
                g.square().sum().backward(retain_graph=True)
    again = torch.autograd.grad(f(*args).square().sum(), args, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(plain, again))


def test_second_derivatives_of_the_loss_raise(calls):
    h, W = randn(5, 8).requires_grad_(), randn(7, 8).requires_grad_()
    t = torch.arange(5)
    for reduction in ("none", "sum", "mean"):
        loss = autograd.linear_cross_entropy(h, W, t, reduction=reduction)
        for g in torch.autograd.grad(loss.sum(), (h, W), create_graph=True):
            with pytest.raises(RuntimeError, match="first derivatives only"):
                g.square().sum().backward(retain_graph=True)


@pytest.mark.parametrize("packed", [False, True])
def test_second_derivatives_of_the_scan_raise(monkeypatch, packed):
    """Stand-ins with the right shapes are enough: the gradients' history is looked at."""
    names = ("x", "dt", "A", "lam", "theta", "B", "C", "h0", "B_prev", "x_prev")
    fwd = lambda *a, **k: (torch.ones(3), torch.ones(2))  # noqa: E731
    bwd = lambda *a, **k: {n: torch.ones(3) for n in names}  # noqa: E731
    for name in ("m3_scan_fwd", "m3_scan_fwd_varlen"):
        monkeypatch.setattr(m3, name, fwd)
    for name in ("m3_scan_bwd", "m3_scan_bwd_varlen"):
        monkeypatch.setattr(m3, name, bwd)
    args = [torch.ones(3).requires_grad_() for _ in range(7)]
    if packed:
        y, state = autograd.m3_scan_varlen(torch.tensor([0, 3], dtype=torch.int32), *args)
    else:
        y, state = autograd.m3_scan(*args)
    for g in torch.autograd.grad(y.sum() + state.sum(), args, create_graph=True):
        with pytest.raises(RuntimeError, match="first derivatives only"):
            g.square().sum().backward(retain_graph=True)


def test_gradients_off_a_16_byte_boundary_are_copied(calls, monkeypatch):
    """The gradient of one part of a torch.cat is a contiguous view that may start anywhere."""
    for f in norm_calls(T=3, C=10).values():
        x, w, b, z = (t.requires_grad_() for t in (randn(3, 10), randn(10), randn(10, seed=1), randn(3, 10, seed=2)))
        torch.cat([torch.zeros((1, 10)), f(x, w, b, z)]).square().sum().backward()
        dy = calls.pop()["dy"]
        assert dy.is_contiguous() and dy.data_ptr() % 16 == 0
    grads = []
    monkeypatch.setattr(m3, "m3_scan_fwd", lambda *a, **k: (torch.ones((3, 2)), torch.ones((3, 2))))
    monkeypatch.setattr(m3, "m3_scan_bwd", lambda *a: grads.append((a[7], a[12])) or {"x": torch.ones((3, 2))})
    x = torch.ones((3, 2)).requires_grad_()
    y, state = autograd.m3_scan(x, *[torch.ones((3, 2))] * 6)
    torch.cat([torch.zeros((1, 2)), y, state]).square().sum().backward()
    for g in grads[0]:
        assert g.is_contiguous() and g.data_ptr() % 16 == 0


@pytest.mark.parametrize("which", ["token", "packed"])
def test_only_wanted_gradients_of_the_norm_are_asked_for(calls, which):
    """A frozen norm, an input without a gradient: the backward leaves them out."""
    f = norm_calls()[which]
    names = ("want_dx", "want_dweight", "want_dbias", "want_dz")
    for wanted in ((1, 0, 0, 0), (0, 1, 1, 0), (0, 0, 0, 1), (1, 1, 0, 1), (0, 0, 1, 0)):
        args = [t.requires_grad_(bool(w)) for t, w in zip(
            (randn(6, 8), randn(8), randn(8, seed=1), randn(6, 8, seed=2)), wanted)]
        f(*args).square().sum().backward()
        asked = calls.pop()
        assert tuple(asked[n] for n in names) == tuple(map(bool, wanted))
        assert all((t.grad is not None) == bool(w) for t, w in zip(args, wanted))


def test_packed_norm_without_sequences_is_refused(calls):
    with pytest.raises(ValueError, match="no sequence"):
        autograd.group_norm_varlen(torch.zeros(1, dtype=torch.int32), randn(3, 4), 2)
