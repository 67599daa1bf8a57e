"""GPU tests of the block norm's gradients where an rsqrt is far from 1: rows of zeros, tiny and
huge rows under an epsilon of almost nothing, and rows of a single value.

Tolerance, row by row (their magnitudes differ by 30 orders): fp32 arithmetic as in
test_gpu_blocknorm, 2^-17 of the row's RMS and of the value, and one rounding to bf16 (8 significant
bits: 2^-8 of the value) where that is the type.  Weights' gradients: 2^-17 in relative L2, on rows of like magnitude.
"""
import pytest
import torch

from lindecay_ref import rel, rms

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32 = 2.0 ** -17
EPS = 1e-30


@pytest.fixture(scope="module")
def sml():
    import structured_mask_linear_gb300 as m

    m.lib()
    return m


def near(got, want, what):
    u = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    got, want = got.double().cpu(), want.double()
    assert torch.isfinite(got).all(), what
    scale = want.square().mean(-1, keepdim=True).sqrt()
    # what is below the smallest normal number may be flushed or lose digits
    worst = ((got - want).abs() - (u + F32) * want.abs() - F32 * scale).max()
    assert float(worst) <= 2.0 ** -126, (what, float(worst))


def norm_grad(x, u, group):
    """Gradient of sum(u x r) by x, r = rsqrt(mean over the group of x^2 + eps), in 64 bits.  For a
    group of one the two terms cancel but for the epsilon, in 64 bits too: the difference itself."""
    z, v = (t.reshape(t.shape[0], -1, group) for t in (x, u))
    r = torch.rsqrt(z.square().mean(-1, keepdim=True) + EPS)
    g = v * EPS * r ** 3 if group == 1 else r * (v - z * r * (v * z * r).mean(-1, keepdim=True))
    return g.reshape(x.shape)


def grads(group, has, x, D):
    """Every gradient from the formulas, in 64 bits."""
    w = {n: t.double() for n, t in x.items()}
    dx, out = w["dx_new"], {}
    if "w_pre" in has:
        out["dw_pre"] = (w["dh"] * rms(w["x_new"], D, EPS)).sum(0)
        dx = dx + norm_grad(w["x_new"], w["dh"] * w["w_pre"], D)
    out["dx"] = dx
    if "y" in has:
        yn, gate, sig = rms(w["y"], group, EPS), w["gate"], torch.sigmoid(w["gate"])
        dm = dx * w["scale"] if "scale" in has else dx
        dn = dm * gate * sig
        out["dscale"] = (dx * gate * sig * yn * w["w_post"]).sum(0)
        out["dgate"] = dm * yn * w["w_post"] * (sig * (1 + gate * (1 - sig)))
        out["dw_post"] = (dn * yn).sum(0)
        out["dy"] = norm_grad(w["y"], dn * w["w_post"], group)
    return out


def draw(R, D, dtype, size):
    g = torch.Generator().manual_seed(D)
    x = {n: torch.randn((R, D), generator=g) for n in ("y", "gate", "x_new", "dx_new", "dh")}
    for n in ("y", "x_new"):
        x[n] = x[n] * size
    x = {n: t.to(dtype) for n, t in x.items()}
    for n, a in (("w_post", 1.0), ("scale", 0.5), ("w_pre", 1.0)):
        x[n] = a + 0.1 * torch.randn(D, generator=g)
    return x


def check(sml, R, D, group, dtype, has, size, dx_new=True):
    x = draw(R, D, dtype, size)
    if not dx_new:
        x["dx_new"] = torch.zeros_like(x["dx_new"])
    a = {n: x[n].to(DEV) if n in has else None for n in ("y", "gate", "w_post", "scale", "w_pre")}
    pre = "w_pre" in has
    got = sml.blocknorm_bwd(x["dx_new"].to(DEV) if dx_new else None, a["y"], a["w_post"],
                            dh=x["dh"].to(DEV) if pre else None, x_new=x["x_new"].to(DEV) if pre else None,
                            gate=a["gate"], scale=a["scale"], w_pre=a["w_pre"], group=group, eps=EPS)
    torch.cuda.synchronize()
    assert sml.loglinear_check_status() == 0
    want = grads(group or D, has, x, D)
    for name, g in got._asdict().items():
        if g is None:
            continue
        what = f"{name} {R}x{D}/{group} {dtype} {size}"
        if name.startswith("dw") or name == "dscale":
            assert rel(g, want[name]) <= F32, what
        else:
            near(g, want[name], what)


DTYPES = [torch.bfloat16, torch.float32]
JOINT, HEADS = ("y", "gate", "w_post", "scale", "w_pre"), ("y", "gate", "w_post")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("has", [JOINT, HEADS], ids=["joint", "heads"])
# the row, groups of lanes, columns apart, groups value by value, groups of one, the widest rows
@pytest.mark.parametrize("D,group", [(256, None), (512, 64), (100, None), (96, 48), (64, 1), (9000, None)])
@pytest.mark.parametrize("size", [0.0, 1e-25, 1e-18, 1e-14, 1.0, 1e15])
def test_extreme_rows(sml, size, D, group, has, dtype):
    """rsqrt from 1e15 (of an epsilon alone) to 1e-15: its cube is outside of fp32, the gradient is
    not."""
    check(sml, 5, D, group, dtype, has, size)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", [1e-15, 1e-3, 1.0])
def test_norm_of_a_single_value(sml, size, dtype):
    """x rsqrt(x^2 + eps): what is left of its gradient is eps (x^2 + eps)^(-3/2)."""
    check(sml, 40, 1, None, dtype, ("w_pre",), size, dx_new=False)


def test_norm_of_a_single_value_at_the_usual_epsilon(sml):
    g = torch.Generator().manual_seed(2)
    x, dh, w = torch.randn((50, 1), generator=g), torch.randn((50, 1), generator=g), torch.full((1,), 1.25)
    got = sml.blocknorm_bwd(None, dh=dh.to(DEV), x_new=x.to(DEV), w_pre=w.to(DEV), eps=1e-6)
    near(got.dx, dh.double() * 1.25 * 1e-6 * (x.double().square() + 1e-6) ** -1.5, "dx")
