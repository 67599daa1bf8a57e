"""GPU tests of the feed-forward block's weight gradients over very many rows, in bf16.

The tensor cores cut their sums off instead of rounding them, towards 0: an addition of 16 products by half of 2^-23 of
its binade on average, 0.72 of 2^-24 of it, n / 16 of them while a random sum grows as their root: 0.48 n / 16 2^-24 of the
whole at most.  Sums that several items share are shorter by as much.  What is seen here is the
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


def test_sums_of_many_tiles_are_not_longer_than_131072_values(sml):
    """81 tiles: more than there are pairs of CTAs, so that sharing them saves no time.  (One sum loses 8.4e-4.)"""
    got, noise = lost(sml, 1 << 20, 2304, 2304)
    assert got <= 0.5 * ((1 << 17) / 16) * 2.0 ** -24 + noise, got


@pytest.mark.parametrize("D", [1 << 18, (1 << 18) + 8])
def test_long_rows(sml, D):
    """The forward's sums, of which a tile has two parts or three."""
    g = torch.Generator(device=DEV).manual_seed(D)
    x, wg, wu = (torch.randn((n, D), generator=g, device=DEV) for n in (40, 64, 64))
    x, wg, wu = x.bfloat16(), (wg * D ** -0.5).bfloat16(), (wu * D ** -0.5).bfloat16()
    gate, up = (torch.full((40, 64), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    sml.ffgate_fwd(x, wg, wu, gate=gate, up=up)
    for y, w in ((gate, wg), (up, wu)):
        want = x.double() @ w.double().t()
        assert float((y.double() - want).norm() / want.norm()) <= 2.0 ** -8 + 2.0 ** -12
