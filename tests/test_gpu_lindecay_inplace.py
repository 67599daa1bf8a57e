"""GPU tests of outputs in the place of inputs: o over v (allowed), and the refusals."""
import pytest
import torch

from test_gpu_lindecay import draw, on_gpu, sml  # noqa: F401  (sml is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,H,hpg,dk,dv,dtype", [
    (2, 500, 90, 1, 64, 72, torch.bfloat16),   # units cut between SMs
    (1, 4100, 2, 2, 128, 128, torch.bfloat16),  # segments, two column tiles
    (2, 1300, 2, 1, 40, 72, torch.float32),
    (2, 40, 4, 2, 64, 64, torch.float32),
])
def test_o_in_the_place_of_v(sml, B, T, H, hpg, dk, dv, dtype):  # noqa: F811
    d = on_gpu(draw(B, T, H, hpg, dk, dv, dtype, seed=T, lengths=[T] + [T // 2] * (B - 1)))
    args = dict(lengths=d["lengths"], state_in=d["state_in"])
    want = sml.lindecay_fwd(d["q"], d["k"], d["v"], d["log_a"], **args)
    got = sml.lindecay_fwd(d["q"], d["k"], d["v"], d["log_a"], o=d["v"], **args)
    assert got.data_ptr() == d["v"].data_ptr() and torch.equal(got, want)


def test_outputs_in_the_place_of_what_is_still_read(sml):  # noqa: F811
    d = on_gpu(draw(2, 64, 4, 1, 64, 64, torch.bfloat16))
    for name in ("q", "k"):
        with pytest.raises(sml.LogLinearError, match="LL_ERR_SHAPE"):
            sml.lindecay_fwd(d["q"], d["k"], d["v"], d["log_a"], o=d[name])
    y = torch.randn((4, 64), device=d["q"].device)
    w, out = torch.ones(64, device=y.device), torch.empty_like(y)
    with pytest.raises(sml.LogLinearError, match="LL_ERR_SHAPE"):
        sml.blocknorm_fwd(y, w_pre=w, x_new=out, h=out)
