"""GPU tests of the gated recurrence with the final states in the place of the first ones, and h in that of
an input, where several CTAs share a sequence."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def sml():
    import structured_mask_linear_gb300 as m

    m.lib()
    return m


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,D", [(1, 1, 64), (1, 57, 8), (1, 120, 64), (2, 450, 16), (1, 1000, 2048), (3, 2000, 40), (1, 130, 2050)])
def test_states_that_take_the_place_of_those_before(sml, B, T, D, dtype):
    """Every CTA of a sequence begins from state_in, and one writes state_out."""
    g = torch.Generator().manual_seed(T)
    x, r = (torch.randn((B, T, D), generator=g).to(dtype).to(DEV) for _ in range(2))
    d, first = torch.rand(D, generator=g).to(DEV), torch.randn((B, D), generator=g).to(DEV)
    last = torch.empty_like(first)
    want = sml.gatescan_fwd(x, r, d, state_in=first, state_out=last)
    for _ in range(20):
        st, y = first.clone(), x.clone()
        h = sml.gatescan_fwd(y, r, d, state_in=st, state_out=st, h=y)
        assert torch.equal(h, want) and torch.equal(st, last)
