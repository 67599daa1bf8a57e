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
