"""CPU tests of the autograd wrappers (block.py): first derivatives with create_graph, and the
refusal of second ones, on stand-ins for the kernels' calls that like them return tensors
without history."""
import pytest
import torch

import structured_mask_linear_gb300 as sml
from lindecay_ref import block as plain_block
from lindecay_ref import lindecay as plain_lindecay
from lindecay_ref import rms
from structured_mask_linear_gb300 import block


def _lindecay_fwd(q, k, v, log_a, lengths=None, state_in=None, state_out=None):
    with torch.no_grad():
        o, s = plain_lindecay(q, k, v, log_a, lengths, state_in)
        state_out.copy_(s)
        return o


def _lindecay_bwd(q, k, v, log_a, dO, lengths=None, state_in=None, dstate_out=None, dstate_in=None):
    with torch.enable_grad():
        x = [t.detach().requires_grad_() for t in (q, k, v)] + ([] if state_in is None else [state_in.detach().requires_grad_()])
        o, s = plain_lindecay(*x[:3], log_a, lengths, x[3] if len(x) > 3 else None)
        loss = (o * dO.detach()).sum() + (0.0 if dstate_out is None else (s * dstate_out.detach()).sum())
    g = torch.autograd.grad(loss, x)
    if dstate_in is not None:
        dstate_in.copy_(g[3])
    return g[:3]


def _norm(y, w_post, x, gate, scale, w_pre, group, act, eps):
    xn = x if y is None else plain_block(y, w_post, x, gate, scale, group, act, eps)
    return xn, None if w_pre is None else rms(xn, xn.shape[-1], eps) * w_pre


def _blocknorm_fwd(y, w_post, x, gate, scale, w_pre, group=None, act="silu", eps=1e-6):
    with torch.no_grad():
        return _norm(y, w_post, x, gate, scale, w_pre, group, act, eps)


def _blocknorm_bwd(dx_new, y, w_post, dh, x_new, gate, scale, w_pre, group=None, act="silu", eps=1e-6, residual=None):
    with torch.enable_grad():
        leaf = lambda t: None if t is None else t.detach().requires_grad_()  # noqa: E731
        v = {n: leaf(t) for n, t in dict(y=y, w_post=w_post, gate=gate, scale=scale, w_pre=w_pre, x=x_new).items()}
        dx = torch.zeros_like(x_new if y is None else y) if dx_new is None else dx_new.detach()
        out = dict.fromkeys(("dx", "dy", "dgate", "dw_post", "dscale", "dw_pre"))
        if dh is not None:
            h = rms(v["x"], v["x"].shape[-1], eps) * v["w_pre"]
            gx, out["dw_pre"] = torch.autograd.grad(h, [v["x"], v["w_pre"]], dh.detach())
            dx = dx + gx
        out["dx"] = dx if residual else None
        names = [n for n in ("y", "w_post", "gate", "scale") if v[n] is not None]
        if y is not None:
            m = plain_block(v["y"], v["w_post"], None, v["gate"], v["scale"], group, act, eps)
            out.update(zip(["d" + n for n in names], torch.autograd.grad(m, [v[n] for n in names], dx)))
    return sml.BlocknormGrads(**out)


@pytest.fixture(autouse=True)
def stand_ins(monkeypatch):
    for f in (_lindecay_fwd, _lindecay_bwd, _blocknorm_fwd, _blocknorm_bwd):
        monkeypatch.setattr(block, f.__name__[1:], f)


def tensors(*shapes, grad=True):
    g = torch.Generator().manual_seed(len(shapes))
    return [torch.randn(s, generator=g, dtype=torch.float64).requires_grad_(grad) for s in shapes]


def attention():
    """Inputs, and o and the state as functions of them: the wrapper's and the plain ones."""
    x = tensors((2, 7, 2, 8), (2, 7, 2, 8), (2, 7, 4, 8), (2, 4, 8, 8))
    log_a = torch.tensor([-0.1, -0.5, -1.0, 0.0], dtype=torch.float64)
    return x, (lambda q, k, v, s: block.lindecay(q, k, v, log_a, None, s)), \
        (lambda q, k, v, s: plain_lindecay(q, k, v, log_a, None, s))


def norms():
    x = tensors((5, 16), (16,), (5, 16), (5, 16), (16,), (16,))
    return x, (lambda *a: block.blocknorm(*a, group=8)), (lambda *a: _norm(*a, 8, "silu", 1e-6))


def first_norm():
    x = tensors((5, 16), (16,))
    return x, (lambda x, w: block.blocknorm(x=x, w_pre=w)), (lambda x, w: _norm(None, None, x, None, None, w, None, "silu", 1e-6))


CASES = [attention, norms, first_norm]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("create_graph", [False, True])
def test_first_derivatives(case, create_graph):
    """In 64 bits but for the states, which the wrapper holds in 32: 2^-24 of values below 16,
    added up over 8 columns."""
    x, f, plain = case()
    loss = lambda out: sum((o * o).sum() for o in out)  # noqa: E731
    got = torch.autograd.grad(loss(f(*x)), x, create_graph=create_graph)
    for g, w in zip(got, torch.autograd.grad(loss(plain(*x)), x)):
        torch.testing.assert_close(g.detach(), w, rtol=0.0, atol=2.0 ** -17)


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("linear", [False, True])
def test_a_second_derivative_is_refused(case, linear):
    """A penalty on the gradients, beside another term that has a gradient of its own.  In a linear
    loss what comes back into the wrapper's backward is a constant, but its gradients still
    depend on the inputs."""
    x, f, _ = case()
    loss = sum(o.sum() if linear else (o * o).sum() for o in f(*x))
    grads = torch.autograd.grad(loss, x, create_graph=True)
    total = sum(t.square().sum() for t in x) + sum(g.square().sum() for g in grads)
    with pytest.raises(RuntimeError, match="second derivative"):
        total.backward()


@pytest.mark.parametrize("case", CASES)
def test_a_second_derivative_by_one_input_is_refused(case):
    x, f, _ = case()
    grads = torch.autograd.grad(sum((o * o).sum() for o in f(*x)), x, create_graph=True)
    for t in x:
        with pytest.raises(RuntimeError, match="second derivative"):
            torch.autograd.grad(grads[0].sum(), t, allow_unused=True, retain_graph=True)


def test_decays_that_ask_for_a_gradient_are_refused():
    """They would get none.  Without a graph, or detached, they are the constants they are."""
    x, _, _ = attention()
    log_a = torch.full((4,), -0.5, dtype=torch.float64, requires_grad=True)
    with pytest.raises(ValueError, match="log_a"):
        block.lindecay(*x[:3], log_a)
    o, _ = block.lindecay(*x[:3], log_a.detach())
    assert o.requires_grad
    with torch.no_grad():
        assert torch.equal(block.lindecay(*x[:3], log_a)[0], o)
