"""GPU tests of a stack's options in blocks of both kinds: what is asked for is what is computed, against the
plain form with the values that were asked for."""
import pytest
import torch

from lindecay_ref import rel
from test_gpu_decoder_block import DEV, OUT, double, draw, plain, stack

pytestmark = pytest.mark.gpu
ASKED = [dict(), dict(mix="lerp"), dict(mix="none"), dict(head_eps=0.5), dict(head_eps=1e-3, mix="lerp")]


@pytest.mark.parametrize("asked", ASKED)
@pytest.mark.parametrize("recurrent", [(0,), (0, 2)])
def test_options_reach_every_block(asked, recurrent):
    net, x = stack(torch.float32, recurrent=recurrent, **asked), draw(2, 60, torch.float32)
    d = double(net)
    for b in d.blocks:
        if hasattr(b, "channels"):
            b.head_eps, b.mixing = asked.get("head_eps", 1e-6), asked.get("mix", "rms")
        else:
            b.head_eps = asked.get("head_eps", 1.0)
    want, _ = plain(d, x.double())
    with torch.no_grad():
        h, _ = net(x.to(DEV))
        assert rel(h, want) <= OUT[torch.float32]
        states = net.states(2)
        for t in range(3):
            p = torch.full((2,), t, dtype=torch.int32, device=DEV)
            assert rel(net.step(x[:, t].to(DEV).contiguous(), states, p), want[:, t]) <= OUT[torch.float32]


def test_an_unknown_mix_is_refused():
    with pytest.raises(ValueError, match="mix"):
        stack(torch.float32, mix="mean")


@pytest.mark.parametrize("qk_norm", ["rms", "l2"])
def test_the_epsilon_of_the_norms_of_q_and_k(qk_norm):
    """Of the size of what it is added to."""
    from decoder_ref import headrope

    net, h = stack(torch.float32, layers=1, recurrent=(), qk_norm=qk_norm, qk_eps=0.75), draw(2, 9, torch.float32)
    b, d = net.blocks[0], double(net).blocks[0]
    p = torch.arange(9, dtype=torch.int32).expand(2, 9).contiguous()
    with torch.no_grad():
        got = b.place(*b.project(h.to(DEV))[:2], p.to(DEV))
    for x, y, w in zip(got, d.project(h.double())[:2], (d.w_q_norm, d.w_k_norm)):
        assert rel(x, headrope(y, w, b.inv_freq.double().cpu(), p, "half", qk_norm, 0.75)) <= OUT[torch.float32]
