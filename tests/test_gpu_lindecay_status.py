"""GPU test: a timeout that some other call has left in the device's status word, not yet read,
is not taken for one of lindecay's own."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("B,T,H,hpg,dk,dv", [
    (2, 2000, 90, 1, 128, 64),   # units cut between SMs, which wait for one another
    (1, 6000, 4, 2, 64, 64),     # segments
    (2, 700, 48, 4, 64, 64),     # heads that take turns
])
def test_another_calls_timeout(B, T, H, hpg, dk, dv):
    import structured_mask_linear_gb300 as sml

    g = torch.Generator().manual_seed(T)
    shapes = [(B, T, H // hpg, dk)] * 2 + [(B, T, H, dv)] * 2
    q, k, v, dO = ((torch.randn(s, generator=g) * 0.125).to(DEV, torch.bfloat16) for s in shapes)
    la = -torch.rand(H, generator=g).to(DEV)

    def run():
        st = torch.full((B, H, dk, dv), float("nan"), device=DEV)
        o = torch.full_like(v, float("nan"))
        sml.lindecay_fwd(q, k, v, la, state_out=st, o=o)
        return [o, st, *sml.lindecay_bwd(q, k, v, la, dO)]

    assert sml.loglinear_check_status() == 0
    want = run()
    assert sml.loglinear_check_status() == 0
    sml.loglinear_selftest_wait_timeout(1000)
    got = run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert sml.loglinear_check_status() == 7  # LL_ERR_TIMEOUT: the self-test's, still to be read
    assert sml.loglinear_check_status() == 0
