"""GPU tests of the gated recurrence where a token keeps all but fp32's smallest numbers of the state."""
import pytest
import torch

from decoder_ref import gatescan, gatescan_bwd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def sml():
    import structured_mask_linear_gb300 as m

    m.lib()
    return m


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("mix", ["rms", "lerp", "none"])
@pytest.mark.parametrize("D", [64, 66, 5])
def test_decays_down_to_the_smallest_numbers(sml, mix, D, dtype):
    """Every r from -84 to -92, where sigmoid(r) goes from normal numbers to none, and decays from 1 to 1e-3 of
    it.  1 - a^2 below 2^-126 counts as 0.  What that leaves out: n, at most 2^-63, of 60 tokens' sums g, below
    60 * 4 + 4 < 2^8, times x below 4 (2^-53 in dx, di and dr); and in ddecay a slope s / n = sqrt(s / (2 decay)),
    with 2 decay s < 2^-126 at most 2^-64 / decay < 2^-54, times g x of 60 tokens, 2^16: 2^-38.  Beside that the
    formulas' 2^-16 and the cast, of the largest value: sums cancel."""
    g = torch.Generator().manual_seed(D)
    T = 60
    n = lambda *s: torch.randn(s, generator=g).clamp(-4, 4)  # noqa: E731
    x, dh, i = (n(1, T, D).to(dtype) for _ in range(3))
    r = torch.linspace(-84, -92, T)[None, :, None].expand(1, T, D).to(dtype).contiguous()
    decay = 10.0 ** torch.linspace(0, -3, D)
    s0 = n(1, D)
    c = [t.to(DEV) for t in (x, r, decay, i, dh, s0)]
    h = sml.gatescan_fwd(c[0], c[1], c[2], i=c[3], mix=mix, state_in=c[5])
    want, _ = gatescan(x.double(), r.double(), decay.double(), i.double(), mix, None, s0.double())
    cast = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0

    def close(a, b, tol, lost):
        return torch.isfinite(a).all() and float((a.double().cpu() - b).abs().max()) <= tol * float(b.abs().max()) + lost

    assert close(h, want, cast + 2.0 ** -16, 2.0 ** -53)
    got = sml.gatescan_bwd(c[4], c[0], c[1], c[2], h, i=c[3], mix=mix, state_in=c[5])
    want = gatescan_bwd(dh.double(), x.double(), r.double(), decay.double(), h.double().cpu(), i.double(), mix, None, s0.double())
    for name, a, b in zip(("dx", "dr", "di"), got, want):
        assert close(a, b, cast + 2.0 ** -16, 2.0 ** -53), name
    assert close(got.ddecay, want[3], 2.0 ** -16, 2.0 ** -38)


@pytest.mark.parametrize("decay", [0.0, 1e-45, 1e-40, 1e-38, 1.2e-38, 1e-36])
def test_decays_that_are_next_to_nothing(sml, decay):
    x = torch.ones((2, 70, 64), device=DEV)
    d = torch.full((64,), decay, device=DEV)
    h = sml.gatescan_fwd(x, x, d)
    got = sml.gatescan_bwd(x, x, x, d, h)
    for t in (h, got.dx, got.dr):
        assert torch.isfinite(t).all() and float(t.abs().max()) < 1e-15
    assert torch.isfinite(got.ddecay).all()
