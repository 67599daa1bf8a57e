"""GPU test of DecayStack with a model's own epsilons, against the plain 64-bit form (fp32, tolerance
as in test_gpu_block)."""
import copy

import pytest
import torch

from lindecay_ref import ACT, pairs, rel, rms
from test_gpu_block import DEV, OUT, draw, stack

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps,head_eps", [(1e-6, 1.0), (1e-2, 1e-3), (1e-3, 0.3)])
def test_epsilons(eps, head_eps):
    net, x = stack(torch.float32, eps=eps, head_eps=head_eps), draw(2, 60, torch.float32)
    ref, s = copy.deepcopy(net).double().cpu(), x.double()
    h = rms(s, s.shape[-1], eps) * ref.blocks[0].w_pre
    for b, after in zip(ref.blocks, (ref.blocks[1].w_pre, ref.w_last)):
        q, k, v, g = b.project(h)
        o = pairs(q, k, v, b.log_a)[0].reshape(g.shape)
        y = (rms(o, b.d_v, head_eps) * b.w_head * ACT["silu"](g)) @ b.w_o.t()
        s = s + rms(y, y.shape[-1], eps) * b.w_post * b.scale
        h = rms(s, s.shape[-1], eps) * after
    with torch.no_grad():
        got, states = net(x[:, :50].contiguous().to(DEV))
        assert rel(got, h[:, :50]) <= OUT[torch.float32]
        for t in range(50, 60):
            assert rel(net.step(x[:, t].contiguous().to(DEV), states), h[:, t]) <= OUT[torch.float32]
