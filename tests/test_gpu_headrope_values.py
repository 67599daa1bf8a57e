"""GPU tests of the head norms with rotation on values that are not finite: they stay where they are,
as far as the formula goes."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LOST = [float("nan"), float("inf"), float("-inf")]


@pytest.fixture(scope="module")
def sml():
    import structured_mask_linear_gb300 as m

    m.lib()
    return m


def alike(a, b):
    return (a == b) | (a.isnan() & b.isnan())


# (72, 24): 9 lanes' worth in 16; (33, 6), (10, 2), (7, 2): value by value, an odd one left over
DIMS = [(64, 16), (72, 24), (128, 64), (33, 6), (10, 2), (7, 2), (8, 0)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["half", "inter"])
@pytest.mark.parametrize("d,rot", DIMS)
def test_past_the_rotated_part_a_value_is_its_own(sml, d, rot, layout, dtype):
    """Without a norm what is not rotated goes out as it came, and its gradient too."""
    g = torch.Generator().manual_seed(d)
    q, dq = (torch.randn((3, 2, d), generator=g).to(dtype).to(DEV) for _ in range(2))
    kw = dict(inv_freq=sml.rope_frequencies(rot) if rot else None, layout=layout, norm="none",
              positions=torch.tensor([5, 0, 1 << 20], dtype=torch.int32, device=DEV) if rot else None)
    base = sml.headrope_fwd(q, **kw)[0], sml.headrope_bwd(dq, q, **kw).dq
    for n in range(rot, d):
        x, dy = q.clone(), dq.clone()
        x[1, 0, n] = dy[1, 0, n] = LOST[n % 3]
        y, dx = sml.headrope_fwd(x, **kw)[0], sml.headrope_bwd(dy, q, **kw).dq
        for got, was, want in ((y, base[0], x[1, 0, n]), (dx, base[1], dy[1, 0, n])):
            same = alike(got, was)
            assert alike(got[1, 0, n], want) and int((~same).sum()) == 1 and not same[1, 0, n], n


@pytest.mark.parametrize("d,rot", [(64, 16), (64, 0), (33, 6), (128, 128)])
@pytest.mark.parametrize("weights", [False, True])
def test_without_a_norm_x_has_no_part_in_its_gradient(sml, d, rot, weights):
    """dx = R^-1 dy w: an infinity in x reaches the weight's gradient alone."""
    g = torch.Generator().manual_seed(d)
    q, dq = (torch.randn((3, 2, d), generator=g).to(DEV) for _ in range(2))
    kw = dict(w_q=torch.rand(d, generator=g).to(DEV) if weights else None, norm="none",
              inv_freq=sml.rope_frequencies(rot) if rot else None,
              positions=torch.tensor([5, 0, 1 << 20], dtype=torch.int32, device=DEV) if rot else None)
    base = sml.headrope_bwd(dq, q, **kw)
    x = q.clone()
    x[1, 0, d // 2], x[2, 1, 0], x[0, 0, d - 1] = LOST[0], LOST[1], LOST[2]
    got = sml.headrope_bwd(dq, x, **kw)
    assert torch.equal(got.dq, base.dq)
    if weights:
        keep = torch.ones(d, dtype=torch.bool)
        keep[[0, d // 2, d - 1]] = False
        assert torch.equal(got.dw_q[keep.to(DEV)], base.dw_q[keep.to(DEV)]) and not torch.isfinite(got.dw_q[~keep.to(DEV)]).any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["half", "inter"])
@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("d,rot", [(128, 64), (128, 128), (64, 16), (80, 40), (33, 6)])
def test_under_a_norm(sml, d, rot, norm, layout, dtype):
    """An infinity makes its head's inverse norm 0: the others become 0, and it NaN, with the value that it turns
    with.  An infinite dy past the rotated part reaches its own weight's gradient and its head alone."""
    from decoder_ref import headrope

    g = torch.Generator().manual_seed(d)
    q, dq = (torch.randn((3, 4, d), generator=g).to(dtype) for _ in range(2))
    p = torch.tensor([5, 3, 1 << 20], dtype=torch.int32)
    w, f = 1 + 0.3 * torch.rand(d, generator=g), sml.rope_frequencies(rot, device="cpu")
    kw = dict(w_q=w.to(DEV), inv_freq=f.to(DEV), positions=p.to(DEV), layout=layout, norm=norm)
    for n in {0, rot // 2, rot - 1, rot % d, (rot + 4) % d, d - 1}:
        x = q.clone()
        x[1, 2, n] = LOST[1 + n % 2]
        y = sml.headrope_fwd(x.to(DEV), **kw)[0].cpu()
        want = headrope(x.double(), w.double(), f, p, layout, norm, 1e-6)
        assert torch.equal(y.isnan(), want.isnan()) and int(y.isnan().sum()) == (2 if n < rot else 1), n
        assert not y[1, 2].nan_to_num().any() and torch.isfinite(y[[0, 2]]).all()
    base = sml.headrope_bwd(dq.to(DEV), q.to(DEV), **kw)
    for n in range(rot, d, 5):
        dy = dq.clone()
        dy[1, 2, n] = LOST[n % 3]
        got = sml.headrope_bwd(dy.to(DEV), q.to(DEV), **kw)
        other = torch.ones((3, 4), dtype=torch.bool)
        other[1, 2] = False
        assert torch.equal(got.dq[other.to(DEV)], base.dq[other.to(DEV)]) and not torch.isfinite(got.dq[1, 2]).any(), n
        own = torch.arange(d, device=DEV) == n
        assert not torch.isfinite(got.dw_q[own]).any() and torch.equal(got.dw_q[~own], base.dw_q[~own]), n
