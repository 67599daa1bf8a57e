"""CPU test: a stack with rotary heads does not guess where a sequence that goes on is."""
import pytest
import torch

from structured_mask_linear_gb300.block import DecayStack

SIZE = dict(layers=2, width=32, heads=2, groups=1, d_k=16, d_v=16, dtype=torch.float32, device="cpu")


def test_states_without_a_start_are_refused():
    net = DecayStack(**SIZE, rotary=8)
    with pytest.raises(ValueError, match="first position"):
        net(torch.zeros(2, 3, 32), states=net.states(2))


@pytest.mark.parametrize("kw,rotary", [({}, 8), (dict(start=torch.zeros(2, dtype=torch.int32), states=2), 8), (dict(states=2), 0)])
def test_where_there_is_nothing_to_guess_the_call_goes_on(kw, rotary):
    """As far as the first kernel, which wants a CUDA device."""
    net = DecayStack(**SIZE, rotary=rotary)
    if "states" in kw:
        kw = {**kw, "states": net.states(2)}
    with pytest.raises(ValueError, match="CUDA device"):
        net(torch.zeros(2, 3, 32), **kw)
