"""GPU tests of the autograd wrappers (block.py) where a graph is asked more than one backward
of first derivatives."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def stack():
    from structured_mask_linear_gb300.block import DecayStack

    torch.manual_seed(4)
    return DecayStack(layers=2, width=64, heads=4, groups=2, d_k=16, d_v=24, dtype=torch.float32, device=DEV)


def draw(T, seed=0):
    return torch.randn((2, T, 64), generator=torch.Generator().manual_seed(seed)).to(DEV)


def test_a_second_derivative_is_refused():
    net, x = stack(), draw(70).requires_grad_()
    params = list(net.parameters())
    loss = net(x)[0].square().sum()
    plain = torch.autograd.grad(loss, [x] + params, retain_graph=True)
    grads = torch.autograd.grad(loss, [x] + params, create_graph=True)
    for a, b in zip(plain, grads):
        torch.testing.assert_close(a, b)
    for g in grads:
        with pytest.raises(RuntimeError, match="second derivative"):
            (loss + g.square().sum()).backward(retain_graph=True)


def modified():
    return pytest.raises(RuntimeError, match="modified by an inplace operation")


def test_a_state_changed_by_a_step_is_noticed():
    """A backward that needs a state as it was before decode steps moved it on."""
    net, x = stack(), draw(30)
    with torch.no_grad():
        _, states = net(x)
    h, _ = net(draw(40, seed=1).requires_grad_(), states=states)
    net.step(x[:, 0].contiguous(), states)
    with modified():
        h.square().sum().backward()


def test_outputs_written_in_place_are_noticed():
    """Every output that a caller gives: one that autograd keeps for a backward is not changed
    without its knowing."""
    import structured_mask_linear_gb300 as sml

    g = torch.Generator(device=DEV).manual_seed(0)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    q, k, v, la, st = rnd(1, 40, 2, 16), rnd(1, 40, 2, 16), rnd(1, 40, 2, 16), -torch.ones(2, device=DEV), rnd(1, 2, 16, 16)
    y, w = rnd(6, 32), rnd(32)
    calls = {
        "fwd o": (v.clone(), lambda t: sml.lindecay_fwd(q, k, v, la, o=t)),
        "fwd state_out": (st.clone(), lambda t: sml.lindecay_fwd(q, k, v, la, state_in=t, state_out=t)),
        "bwd dstate_in": (st.clone(), lambda t: sml.lindecay_bwd(q, k, v, la, v, state_in=st, dstate_in=t)),
        "step states": (st.clone(), lambda t: sml.lindecay_decode_step(q[:, 0].contiguous(), k[:, 0].contiguous(),
                                                                       v[:, 0].contiguous(), la, t)),
        "step o_t": (v[:, 0].clone(), lambda t: sml.lindecay_decode_step(q[:, 0].contiguous(), k[:, 0].contiguous(),
                                                                         v[:, 0].contiguous(), la, st.clone(), o_t=t)),
        "norm x_new": (y.clone(), lambda t: sml.blocknorm_fwd(y, x=t, x_new=t)),
        "norm h": (y.clone(), lambda t: sml.blocknorm_fwd(y, w_pre=w, h=t)),
    }
    for name, (t, call) in calls.items():
        before, leaf = t._version, torch.ones_like(t, requires_grad=True)
        loss = (leaf * t).sum()  # keeps t for leaf's gradient
        call(t)
        assert t._version > before, name
        with modified():
            loss.backward()
        inputs = [x._version for x in (q, k, v, la, st, y, w)]
        call(t.clone())
        assert inputs == [x._version for x in (q, k, v, la, st, y, w)], name


def test_inference_tensors():
    """They have no version to raise, inside inference mode or after it."""
    net, x = stack(), draw(20)
    with torch.inference_mode():
        _, states = net(x)
        first = net.step(x[:, 0].contiguous(), states)
    with torch.no_grad():
        _, again = net(x)
        assert torch.equal(net.step(x[:, 0].contiguous(), again), first)
        net.step(x[:, 1].contiguous(), states)
        net.step(x[:, 1].contiguous(), again)
    assert all(torch.equal(a, b) for a, b in zip(states, again))
