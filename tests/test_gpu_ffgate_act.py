"""GPU tests of the feed-forward block's activations and their slopes, value by value, far from 0 as well.

Weights of ones on the diagonal hand the gates through, and a value of 1 in x is every up's: gates are multiples of
2^-4 below 96 (11 bits), exact in every form of the products.  fp32, relative: the exponential 2^-22, a sum,
a reciprocal 2^-23, one to three products of 2^-24: 2^-20.  gelu's erfc takes its argument z = x / sqrt 2 rounded to
2^-24 twice, which moves it by 2 z^2 of that, x^2 2^-23: from -5 on 2^-18 in all.  A slope's two terms may cancel:
relative to their sizes.  bf16: half a step, 2^-8, and what 32 bits lose beside it (an exponential of |x| 2^-24).  Numbers below the
smallest normal one, 2^-126, have fewer bits than that, or are 0: as much beside everything.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float32
LEAST = 2.0 ** -126
TOL = {("silu", FP): 2.0 ** -20, ("sigmoid", FP): 2.0 ** -20, ("gelu", FP): 2.0 ** -18}
LOW = {"silu": -80, "sigmoid": -80, "gelu": -5}


@pytest.fixture(scope="module")
def sml():
    import structured_mask_linear_gb300 as m

    m.lib()
    return m


def tol(act, dtype):
    return TOL.get((act, dtype), 2.0 ** -8 + 2.0 ** -16)


def draw(rows, F, act, dtype, seed):
    """Gates, every fourth in -20..20; multiples of 2^-4, which bf16 holds up to 16, of 1 above."""
    g = torch.Generator().manual_seed(seed)
    n = torch.rand((rows, F), generator=g) * (96 - LOW[act]) + LOW[act]
    n[:, ::4] = (torch.rand((rows, (F + 3) // 4), generator=g) * 40 - 20).clamp(min=LOW[act])
    n = (n * 16).round() / 16
    return torch.where(n.abs() < 16, n, n.round()) if dtype == BF else n


def value_and_slope(z, act):
    """In 64 bits; the slope's size is that of its terms."""
    if act == "gelu":
        c, e = 0.5 * torch.erfc(-z / math.sqrt(2)), z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        return z * c, c + e, c + e.abs()
    s, rest = 1 / (1 + torch.exp(-z)), 1 / (1 + torch.exp(z))
    if act == "sigmoid":
        return s, s * rest, s * rest
    return z * s, s * (1 + z * rest), s * (1 + z.abs() * rest)


# rows and columns for each way through: streamed weights, narrow tiles, shared sums, whole tiles
@pytest.mark.parametrize("rows,F,D", [(1, 64, 72), (7, 200, 208), (16, 72, 80), (40, 64, 72), (40, 72, 8192), (2500, 1288, 1296)])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("act", ["silu", "sigmoid", "gelu"])
def test_values(sml, act, dtype, rows, F, D):
    gate = draw(rows, F, act, dtype, rows + F)
    x = torch.zeros(rows, D)
    x[:, :F], x[:, F] = gate, 1
    w_gate, w_up = torch.eye(F, D), torch.zeros(F, D)
    w_up[:, F] = 1
    m = sml.ffgate_fwd(*(t.to(dtype).to(DEV) for t in (x, w_gate, w_up)), act=act).double().cpu()
    want = value_and_slope(gate.double(), act)[0]
    assert ((m - want).abs() <= tol(act, dtype) * want.abs() + LEAST).all(), float(((m - want) / want.abs().clamp(min=1e-30)).abs().max())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("act", ["silu", "sigmoid", "gelu"])
def test_slopes(sml, act, dtype):
    rows, F = 300, 256
    gate = draw(rows, F, act, dtype, 3).to(dtype).to(DEV)
    one, eye = torch.ones_like(gate), torch.eye(F, dtype=dtype, device=DEV)
    got = sml.ffgate_bwd(one, torch.zeros_like(gate), eye, torch.zeros_like(eye), gate, one, act=act, need=(1, 0, 0)).dx
    _, want, size = value_and_slope(gate.double().cpu(), act)
    # bf16 rounds the slope (half a step of it), fp32 its terms
    bound = 2.0 ** -8 * want.abs() + 2.0 ** -16 * size if dtype == BF else tol(act, dtype) * size
    assert ((got.double().cpu() - want).abs() <= bound + LEAST).all(), float(((got.double().cpu() - want) / size).abs().max())
