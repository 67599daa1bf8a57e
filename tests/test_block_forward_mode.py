"""CPU tests of the autograd wrappers (block.py) on inputs that carry a tangent: forward mode has no
derivative here, and says so in grad mode and out of it, on stand-ins for the kernels' calls."""
import pytest
import torch
from torch.autograd import forward_ad

from structured_mask_linear_gb300 import block

MADE = []


@pytest.fixture(autouse=True)
def stand_ins(monkeypatch):
    def out(n, like):
        def f(*a, **k):
            MADE.append(n)
            t = [x for x in (*a, *k.values()) if torch.is_tensor(x)][like]
            return torch.zeros_like(t) if n in ("ffgate", "gatescan", "lindecay") else (torch.zeros_like(t), torch.zeros_like(t))
        return f

    MADE.clear()
    for n, like in (("lindecay", 2), ("gatescan", 0), ("headrope", 0), ("ffgate", 0), ("blocknorm", 0)):
        monkeypatch.setattr(block, n + "_fwd", out(n, like))


def rnd(*s):
    return torch.randn(s, generator=torch.Generator().manual_seed(0))


CALLS = {
    "lindecay": (lambda q, k, v: block.lindecay(q, k, v, torch.zeros(2)), [(1, 3, 2, 8)] * 3),
    "gatescan": (lambda x, r, d: block.gatescan(x, r, d), [(1, 3, 8), (1, 3, 8), (8,)]),
    "headrope": (lambda q, k, a, b: block.headrope(q, k, a, b), [(3, 2, 8), (3, 1, 8), (8,), (8,)]),
    "ffgate": (lambda x, a, b: block.ffgate(x, a, b), [(3, 8), (16, 8), (16, 8)]),
    "blocknorm": (lambda y, w, x, p: block.blocknorm(y, w, x, w_pre=p), [(3, 8), (8,), (3, 8), (8,)]),
}


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("name", CALLS)
def test_a_tangent_is_refused(name, grad):
    call, shapes = CALLS[name]
    for n in range(len(shapes)):
        args = [rnd(*s) for s in shapes]
        with forward_ad.dual_level(), torch.set_grad_enabled(grad):
            args[n] = forward_ad.make_dual(args[n], torch.ones_like(args[n]))
            with pytest.raises(RuntimeError, match="forward"):
                call(*args)


@pytest.mark.parametrize("name", CALLS)
def test_without_one_the_call_is_as_it_was(name):
    call, shapes = CALLS[name]
    args = [rnd(*s).requires_grad_() for s in shapes]
    with torch.no_grad():
        call(*args)
        with forward_ad.dual_level():
            call(*args)
    assert MADE == [name] * 2
