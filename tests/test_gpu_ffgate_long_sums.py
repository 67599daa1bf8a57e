"""GPU tests of the feed-forward block's weight gradients over very many rows, in bf16.

The tensor cores cut their sums off instead of rounding them, towards 0: an addition of 16 products by half of 2^-23 of
the sum on average, n / 16 of them.  Sums that several items share are shorter by as much.  What is seen here is the
mean of the error towards 0, in standard deviations of the gradient, in which the results' roundings (2^-8 / sqrt 3 at
the most, of either sign) are averaged over all values: five times their 2^-9 / sqrt(values) is left to them.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def sml():
    import structured_mask_linear_gb300 as m

    m.lib()
    return m


def lost(sml, R, D, F):
    """The mean error towards 0 of both weights' gradients of x^T dm, and what roundings may make of it."""
    g = torch.Generator(device=DEV).manual_seed(R)
    x, dm = (torch.randn((R, n), generator=g, device=DEV, dtype=torch.bfloat16) for n in (D, F))
    one, w = torch.ones_like(dm), torch.zeros((F, D), dtype=torch.bfloat16, device=DEV)
    got = sml.ffgate_bwd(dm, x, w, w, one, one, act="identity", need=(0, 1, 1))
    assert torch.equal(got.dw_gate, got.dw_up)
    want = torch.zeros((F, D), dtype=torch.float64, device=DEV)
    for s in range(0, R, 1 << 18):
        want += dm[s:s + (1 << 18)].double().t() @ x[s:s + (1 << 18)].double()
    e = (got.dw_gate.double() - want) * -want.sign() / want.std()
    return float(e.mean()), 5 * 2.0 ** -9 / (F * D) ** 0.5


@pytest.mark.parametrize("R,D,F", [(1 << 20, 64, 64), (1 << 20, 256, 256)])
def test_both_weights_sums_are_shared(sml, R, D, F):
    """Two tiles and 76 pairs of CTAs: at most a 38th of the rows in an item, and twice that leaves room."""
    got, noise = lost(sml, R, D, F)
    assert got <= 2 * (R / 38 / 16) * 2.0 ** -24 + noise, got
