"""GPU tests of the block norm (blocknorm_fwd, _bwd) against the 64-bit form of lindecay_ref.

Tolerances: everything is computed in fp32 and rounded once.  bf16 results are within the
cast, u = 2^-8 of the value, plus fp32 arithmetic.  fp32 arithmetic: a mean of squares over D
values is summed by threads of at most 32 values and then in a tree (under 64 roundings of
2^-24), the rsqrt, the activation and the products add less than 16 more: 2^-17 of a value's
scale, taken as its tensor's RMS.  Weight gradients add up at most R rows in fp32 one after
the other, whose roundings are independent: 2^-17 in relative L2 for the R here.
"""
import pytest
import torch

from lindecay_ref import ACT, block, rel, rms

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32 = 2.0 ** -17


@pytest.fixture(scope="module")
def sml():
    import structured_mask_linear_gb300 as m

    m.lib()
    return m


def draw(R, D, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = {n: (torch.randn((R, D), generator=g) * (2.0 if n.startswith("x") else 1.0)).to(dtype)
         for n in ("y", "x", "gate", "x_new", "dx_new", "dh")}
    for n, a in (("w_post", 1.0), ("scale", 0.5), ("w_pre", 1.0)):
        x[n] = a + 0.1 * torch.randn(D, generator=g)
    return x


def near(got, want, what=""):
    got, w = got.double().cpu(), want.detach().double()
    assert got.shape == w.shape and torch.isfinite(got).all(), what
    u = 2.0 ** -8 if got is not None and want is not None and what.endswith("bf16") else 0.0
    scale = float(w.square().mean().sqrt())
    worst = float(((got - w).abs() - (u + F32) * w.abs()).max())
    assert worst <= F32 * scale, (what, worst, scale)


PARTS = {  # which arguments a call has
    "joint": ("y", "x", "gate", "w_post", "scale", "w_pre"),
    "no gate": ("y", "x", "w_post", "scale", "w_pre"),
    "heads": ("y", "gate", "w_post"),
    "heads, no gate": ("y", "w_post"),
    "residual alone": ("y", "x", "gate"),
    "no weights, norm after": ("y", "x", "gate", "w_pre"),
    "before the first block": ("x", "w_pre"),
}


def check(sml, R, D, group, dtype, parts, act="silu", eps=1e-6, seed=0):
    x = draw(R, D, dtype, seed)
    has = PARTS[parts]
    a = {n: x[n].to(DEV) if n in has else None for n in ("y", "x", "gate", "w_post", "scale", "w_pre")}
    kw = dict(group=group, act=act, eps=eps)
    xn, h = sml.blocknorm_fwd(**a, **kw)
    w = {n: x[n].double() if n in has else None for n in a}
    tag = f" {parts} {R}x{D}/{group} {act} {'bf16' if dtype == torch.bfloat16 else 'f32'}"
    if "y" in has:
        ref = block(w["y"], w["w_post"], w["x"], w["gate"], w["scale"], group, act, eps)
        near(xn, ref, "x'" + tag)
    else:
        ref = w["x"]
        assert xn is a["x"]
    if "w_pre" in has:
        near(h, rms(ref, D, eps) * w["w_pre"], "h" + tag)
    else:
        assert h is None
    # gradients, x' as stored drawn apart: only its norm reads it
    pre = "w_pre" in has
    d = {n: x[n].to(DEV) for n in ("dx_new", "dh", "x_new")}
    got = sml.blocknorm_bwd(d["dx_new"], a["y"], a["w_post"], dh=d["dh"] if pre else None,
                            x_new=d["x_new"] if pre else None, gate=a["gate"], scale=a["scale"], w_pre=a["w_pre"],
                            residual="x" in has, **kw)
    torch.cuda.synchronize()
    assert sml.loglinear_check_status() == 0
    want = {}
    dx = x["dx_new"].double()
    if pre:
        v, wp = x["x_new"].double().requires_grad_(), x["w_pre"].double().requires_grad_()
        gx, want["dw_pre"] = torch.autograd.grad((rms(v, D, eps) * wp * x["dh"].double()).sum(), [v, wp])
        dx = dx + gx
    if "x" in has:
        want["dx"] = dx
    if "y" in has:
        need = {n: w[n].clone().requires_grad_() for n in ("y", "gate", "w_post", "scale") if w[n] is not None}
        m = block(need["y"], need.get("w_post"), None, need.get("gate"), need.get("scale"), group, act, eps)
        want.update(zip(["d" + n for n in need], torch.autograd.grad((m * dx).sum(), list(need.values()))))
    for name, g in got._asdict().items():
        assert (g is None) == (name not in want), (name, parts)
        if g is None:
            continue
        if name in ("dx", "dy", "dgate"):
            near(g, want[name], name + tag)
        else:
            assert rel(g, want[name]) <= F32, name + tag


DTYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("parts", list(PARTS))
def test_arguments(sml, parts, dtype):
    check(sml, 33, 512, None, dtype, parts)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,D", [(1, 8), (1, 2048), (3, 264), (700, 1000), (65, 4096), (9, 4104), (5, 8192), (3, 16384),
                                 (1, 1), (2, 7), (50, 333), (2, 16383), (1300, 128), (2500, 96)])
def test_sizes(sml, R, D, dtype):
    check(sml, R, D, None, dtype, "joint", seed=D)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,group", [(512, 8), (512, 64), (2048, 256), (96, 32), (96, 48), (96, 4), (1024, 512),
                                     (105, 21), (640, 1), (4096, 1)])
@pytest.mark.parametrize("parts", ["heads", "joint"])
def test_groups(sml, D, group, parts, dtype):
    check(sml, 40, D, group, dtype, parts, seed=group)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", sorted(ACT))
@pytest.mark.parametrize("D", [256, 100])
def test_activations(sml, act, D, dtype):
    check(sml, 20, D, None, dtype, "joint", act=act)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [256, 99])
def test_zero_rows_and_extreme_gates(sml, D, dtype):
    """Rows of zeros (a head whose mask left nothing) norm to zeros with finite gradients; gates
    far out saturate."""
    x = draw(6, D, dtype)
    x["y"][2] = 0
    x["gate"][3], x["gate"][4] = 1e4, -1e4
    a = {n: x[n].to(DEV) for n in ("y", "x", "gate", "w_post", "scale", "w_pre")}
    xn, h = sml.blocknorm_fwd(**a)
    assert torch.equal(xn[2], a["x"][2]) and torch.isfinite(h).all()
    assert torch.equal(xn[4], a["x"][4])  # silu(-1e4) = 0
    g = sml.blocknorm_bwd(x["dx_new"].to(DEV), a["y"], a["w_post"], gate=a["gate"], scale=a["scale"])
    assert all(torch.isfinite(t).all() for t in g if t is not None)
    assert (g.dgate[2] == 0).all()
    zero = {n: torch.zeros_like(t) for n, t in a.items()}
    xn, h = sml.blocknorm_fwd(zero["y"], x=zero["x"], w_pre=a["w_pre"])
    assert (xn == 0).all() and (h == 0).all()


@pytest.mark.parametrize("D", [256, 100])
def test_in_place(sml, D):
    """x' may take the place of x, y or the gate."""
    x = draw(30, D, torch.bfloat16)
    a = {n: x[n].to(DEV) for n in ("y", "x", "gate", "w_post", "scale", "w_pre")}
    want, wh = sml.blocknorm_fwd(**a)
    for name in ("x", "y", "gate"):
        b = {n: t.clone() for n, t in a.items()}
        xn, h = sml.blocknorm_fwd(**b, x_new=b[name])
        assert xn.data_ptr() == b[name].data_ptr() and torch.equal(xn, want) and torch.equal(h, wh)


def test_gradient_against_differences(sml):
    """<gradient, direction> against central differences of the 64-bit form, x' included."""
    R, D, group = 12, 128, 32
    x = draw(R, D, torch.float32)
    w = {n: x[n].double() for n in x}

    def loss(v):
        xn = block(v["y"], v["w_post"], v["x"], v["gate"], v["scale"], group, "silu", 1e-6)
        return float((xn * w["dx_new"]).sum() + (rms(xn, D, 1e-6) * v["w_pre"] * w["dh"]).sum())

    a = {n: x[n].to(DEV) for n in ("y", "x", "gate", "w_post", "scale", "w_pre")}
    xn, _ = sml.blocknorm_fwd(**a, group=group)
    g = sml.blocknorm_bwd(x["dx_new"].to(DEV), a["y"], a["w_post"], dh=x["dh"].to(DEV), x_new=xn, gate=a["gate"],
                          scale=a["scale"], w_pre=a["w_pre"], group=group)
    gen = torch.Generator().manual_seed(3)
    for name in ("x", "y", "gate", "w_post", "scale", "w_pre"):
        d = torch.randn(w[name].shape, generator=gen, dtype=torch.float64)
        ends = [loss({**w, name: w[name] + s * 1e-5 * d}) for s in (1.0, -1.0)]
        grad = getattr(g, "d" + name).double().cpu()
        assert abs(float((grad * d).sum()) - (ends[0] - ends[1]) / 2e-5) <= 4 * F32 * float(grad.norm()), name


def test_repeated_calls_agree_bitwise(sml):
    x = draw(3000, 512, torch.bfloat16)
    d = {n: t.to(DEV) for n, t in x.items()}
    run = lambda: sml.blocknorm_bwd(d["dx_new"], d["y"], d["w_post"], dh=d["dh"], x_new=d["x_new"],  # noqa: E731
                                    gate=d["gate"], scale=d["scale"], w_pre=d["w_pre"])
    assert all(torch.equal(a, b) for a, b in zip(run(), run()))


def test_batched_shapes_and_stream(sml):
    """Leading sizes are rows; on a stream of the caller's."""
    x = draw(24, 64, torch.bfloat16)
    y, gate, w = (x[n].to(DEV) for n in ("y", "gate", "w_post"))
    want, _ = sml.blocknorm_fwd(y, w, gate=gate)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = sml.blocknorm_fwd(y.view(2, 3, 4, 64), w, gate=gate.view(2, 3, 4, 64), stream=s)
    s.synchronize()
    assert got.shape == (2, 3, 4, 64) and torch.equal(got.view(24, 64), want)


def test_refusals(sml):
    x = {n: t.to(DEV) for n, t in draw(4, 64, torch.bfloat16).items()}
    with pytest.raises(ValueError, match="y or x is required"):
        sml.blocknorm_fwd()
    with pytest.raises(ValueError, match="nothing to compute"):
        sml.blocknorm_fwd(x=x["x"])
    with pytest.raises(ValueError, match="without y"):
        sml.blocknorm_fwd(x=x["x"], gate=x["gate"], w_pre=x["w_pre"])
    with pytest.raises(ValueError, match="act must be one of"):
        sml.blocknorm_fwd(x["y"], gate=x["gate"], act="relu")
    with pytest.raises(ValueError, match="gate must have shape"):
        sml.blocknorm_fwd(x["y"], gate=x["gate"][:2])
    with pytest.raises(TypeError, match="w_post must be torch.float32"):
        sml.blocknorm_fwd(x["y"], x["w_post"].to(torch.bfloat16))
    with pytest.raises(ValueError, match="contiguous"):
        sml.blocknorm_fwd(x["y"].t().contiguous().t())
    with pytest.raises(ValueError, match="at least one row"):
        sml.blocknorm_fwd(x["y"][:0])
    for kw in (dict(group=48), dict(group=0), dict(group=-64), dict(eps=-1.0), dict(eps=float("nan"))):
        with pytest.raises(sml.LogLinearError, match="LL_ERR_SHAPE"):
            sml.blocknorm_fwd(x["y"], **kw)
    with pytest.raises(sml.LogLinearError, match="LL_ERR_SHAPE"):
        sml.blocknorm_fwd(torch.zeros((1, 16392), device=DEV))
    with pytest.raises(ValueError, match="go together"):
        sml.blocknorm_bwd(x["dx_new"], x["y"], dh=x["dh"])
    with pytest.raises(ValueError, match="dx_new or dh is required"):
        sml.blocknorm_bwd(None, x["y"])
    odd = torch.zeros(4 * 64 + 1, device=DEV, dtype=torch.bfloat16)[1:].view(4, 64)
    with pytest.raises(sml.LogLinearError, match="LL_ERR_ALIGN"):
        sml.blocknorm_fwd(odd)
    assert sml.loglinear_check_status() == 0
