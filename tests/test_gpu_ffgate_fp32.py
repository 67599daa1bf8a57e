"""GPU tests of the feed-forward block in fp32 at its own precision, against the 64-bit form of decoder_ref.

Tolerances, as relative 2-norms.
Projections.  Two fp16 parts hold a value to 2^-23, and the product of the low parts that is left out is at most 2^-22;
both independent from value to value.  The tensor cores cut their sums off, by half of 2^-23 on average and always
downwards, and in a run of 128 values 16 of the additions are of full size: 2^-20.  Runs add up with roundings of
2^-24, sqrt(D / 128) of them: below 2^-21 for D up to 8192.  Up to 8 rows sums are fp32's own, of D / 32 values in a
row, in all roundings: below these.  Together less than 2^-19; a sum of 8192 values left to the tensor cores loses
2^-15.6, operands of two bf16 parts lose 2^-17.8.
m passes on both projections' errors: 2^-18.
Gradients, from the projections as they are given: three bf16 parts (2^-24 of a value and six products), runs of 64
values with 4 additions of full size, 2^-22, up to 256 runs added up, 2^-20, slopes of 2^-20: 2^-19.
"""
import pytest
import torch

from decoder_ref import ffgate, ffgate_bwd, rel
from test_gpu_ffgate import DEV, FP, draw

pytestmark = pytest.mark.gpu
PROJECTION, M, GRAD = 2.0 ** -19, 2.0 ** -18, 2.0 ** -19


@pytest.fixture(scope="module")
def sml():
    import structured_mask_linear_gb300 as m

    m.lib()
    return m


SIZES = [(1, 2048, 520), (8, 8192, 40), (5, 264, 136), (9, 72, 136), (33, 1024, 520), (128, 512, 264), (257, 200, 264),
         (700, 520, 72), (300, 8192, 136), (40, 8192, 72),  # long sums of the projections, shared ones
         (8200, 72, 136), (12000, 136, 24),                  # of the weights' gradients
         (257, 72, 8192), (30, 112, 5000),                   # of dx
         (1003, 1024, 2816), (2500, 264, 1288)]


@pytest.mark.parametrize("R,D,F", SIZES)
def test_sums_and_operands(sml, R, D, F):
    for act in ("silu", "gelu") if R < 1000 else ("sigmoid",):
        a = draw(R, D, F, FP, seed=R + D)
        c, w = {n: v.to(DEV) for n, v in a.items()}, {n: v.double().to(DEV) for n, v in a.items()}
        g, u = (torch.full((R, F), float("nan"), device=DEV) for _ in range(2))
        m = sml.ffgate_fwd(c["x"], c["w_gate"], c["w_up"], act=act, gate=g, up=u)
        want = [t.cpu() for t in ffgate(w["x"], w["w_gate"], w["w_up"], act)]
        for name, x, y, tol in zip(("m", "gate", "up"), (m, g, u), want, (M, PROJECTION, PROJECTION)):
            assert rel(x, y) <= tol, (name, rel(x, y))
        got = sml.ffgate_bwd(c["dm"], c["x"], c["w_gate"], c["w_up"], g, u, act=act)
        want = [t.cpu() for t in ffgate_bwd(w["dm"], w["x"], w["w_gate"], w["w_up"], g.double(), u.double(), act)]
        for name, x, y in zip(got._fields, got, want):
            assert rel(x, y) <= GRAD, (name, rel(x, y))


@pytest.mark.parametrize("k", [0, 10, 16, 17, 18, 24, 30])
@pytest.mark.parametrize("side", ["x", "weights"])
def test_values_far_below_their_rows_largest(sml, side, k):
    """One column of x (or of the weights) of 2^k, met by zeros: of every other value at most 2^-39 2^k goes
    missing, or 2^-23 of itself; beside that each result is within PROJECTION of its two rows' norms."""
    R, D, F = 40, 264, 72
    a = draw(R, D, F, FP, seed=13)
    x, w = a["x"], a["w_gate"]
    big, other = (x, w) if side == "x" else (w, x)
    big[:, 7], other[:, 7] = 2.0 ** k, 0
    g, u = (torch.empty((R, F), device=DEV) for _ in range(2))
    sml.ffgate_fwd(x.to(DEV), w.to(DEV), a["w_up"].to(DEV), gate=g, up=u)
    x, w = x.double(), w.double()
    want = x @ w.t()
    rest = big.double().clone()
    rest[:, 7] = 0
    largest = big.double().abs().amax(1)
    lost = 2.0 ** -39 * (largest[:, None] * x.abs().sum(1)[None] if side == "weights" else largest[:, None] * w.abs().sum(1)[None])
    norms = rest.norm(dim=1)[:, None] * other.double().norm(dim=1)[None]
    bound = lost + PROJECTION * norms
    if side == "weights":
        bound = bound.t()
    assert ((g.double().cpu() - want).abs() <= bound).all()


def test_one_value_at_a_time(sml):
    """What a single value of x keeps, read through weights of ones on the diagonal: 2^-23 of it, or 2^-39 of the row's
    largest, which is just above a power of two and just below one."""
    D = 256
    g = torch.Generator().manual_seed(2)
    x = torch.randn((64, D), generator=g) * torch.exp2(torch.randint(-45, 0, (64, D), generator=g).float())
    x = x.clamp(-1, 1)
    x[:, 0] = torch.where(torch.arange(64) % 2 == 0, torch.tensor(1.0), torch.tensor(1.9999))
    eye = torch.eye(D)
    gate, up = (torch.empty((64, D), device=DEV) for _ in range(2))
    sml.ffgate_fwd(x.to(DEV), eye.to(DEV), eye.to(DEV), gate=gate, up=up)
    bound = torch.maximum(2.0 ** -23 * x.double().abs(), 2.0 ** -39 * x.double().abs().amax(1, keepdim=True))
    assert ((gate.double().cpu() - x.double()).abs() <= bound).all()
