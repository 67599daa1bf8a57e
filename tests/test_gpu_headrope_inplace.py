"""GPU tests of the gradients of the head norms with rotation in the place of what comes in, and in tensors of
the caller's."""
import pytest
import torch

from test_gpu_headrope import DEV, draw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sml():
    import structured_mask_linear_gb300 as m

    m.lib()
    return m


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("norm", ["rms", "none"])
@pytest.mark.parametrize("layout", ["half", "inter"])
@pytest.mark.parametrize("lead,Gq,Gk,d,rot", [((4, 300), 6, 3, 128, 64), ((2, 37), 16, 16, 128, 128), ((3000,), 3, 1, 8, 8),
                                              ((1,), 24, 24, 128, 128), ((5, 7), 3, 2, 33, 6), ((400,), 2, 0, 80, 20)])
def test_gradients_in_the_place_of_what_comes_in(sml, lead, Gq, Gk, d, rot, layout, norm, dtype):
    c = {n: v.to(DEV) for n, v in draw(lead, Gq, Gk, d, rot, dtype, seed=d).items()}
    kw = dict(w_q=c["w_q"], w_k=c.get("w_k"), inv_freq=c["inv_freq"], positions=c["positions"], layout=layout, norm=norm)
    want = sml.headrope_bwd(c["dq"], c["q"], c.get("dk"), c.get("k"), **kw)
    dq, dk = c["dq"].clone(), c["dk"].clone() if Gk else None
    before = dq._version
    got = sml.headrope_bwd(dq, c["q"], dk, c.get("k"), dq=dq, dk=dk, **kw)
    assert got.dq is dq and got.dk is dk and dq._version > before
    for n, x, y in zip(got._fields, got, want):
        assert (x is None) == (y is None) and (x is None or torch.equal(x, y)), n
    other = torch.full_like(dq, float("nan"))
    got = sml.headrope_bwd(c["dq"], c["q"], c.get("dk"), c.get("k"), dq=other, **kw)
    assert got.dq is other and torch.equal(other, want.dq)


def test_refusals(sml):
    q, k = torch.zeros(2, 3, 4, 64, device=DEV), torch.zeros(2, 3, 2, 64, device=DEV)
    other = torch.zeros_like(k)
    for call, err in ((lambda: sml.headrope_bwd(q, q, dq=k), ValueError), (lambda: sml.headrope_bwd(q, q, dk=k), ValueError),
                      (lambda: sml.headrope_bwd(q, q, dq=q.bfloat16()), TypeError),
                      (lambda: sml.headrope_bwd(q, q, other, k, dk=torch.zeros_like(q)), ValueError),
                      (lambda: sml.headrope_bwd(q, q, q.clone(), q.clone(), dq=other.new_zeros(q.shape), dk=q), sml.LogLinearError)):
        with pytest.raises(err):
            call()
