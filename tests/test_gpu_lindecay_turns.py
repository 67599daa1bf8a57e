"""GPU tests of lindecay's gradients where the heads of a group take turns over several blocks of
chunks: three or more heads a group and more than 16 chunks of 128 tokens.  Tolerances as in
test_gpu_lindecay; the 64-bit form is differentiated group by group, on the GPU."""
import pytest
import torch

from lindecay_ref import rel
from parity_util import assert_parity
from test_gpu_lindecay import DEV, REL_STATE, draw, ref_grads, run_bwd, sml  # noqa: F401  (sml is a fixture)

pytestmark = pytest.mark.gpu


def group_grads(x, g, hpg):
    """ref_grads of one group's heads."""
    heads = slice(g * hpg, (g + 1) * hpg)
    y = {"q": x["q"][:, :, g:g + 1], "k": x["k"][:, :, g:g + 1], "v": x["v"][:, :, heads], "dO": x["dO"][:, :, heads],
         "log_a": x["log_a"][heads], "lengths": x["lengths"], "state_in": x["state_in"][:, heads],
         "dstate_out": x["dstate_out"][:, heads]}
    with torch.device(DEV):
        return [t.cpu() for t in ref_grads({n: None if t is None else t.to(DEV) for n, t in y.items()})]


@pytest.mark.parametrize("B,T,H,hpg,dk,dv,lengths", [
    (1, 2049, 3, 3, 64, 64, None),               # one token in the second block; few units: segments
    (2, 2200, 8, 4, 64, 40, [2200, 2100]),
    (1, 4500, 5, 5, 40, 64, None),               # three blocks
    (3, 2200, 6, 3, 128, 64, [2200, 0, 2060]),   # two widths
    (2, 2300, 60, 5, 64, 72, [2300, 2049]),      # more units than SMs: units cut between two SMs
    (1, 2176, 80, 4, 32, 128, None),             # the second block one whole chunk
])
def test_blocks_of_a_groups_turns(sml, B, T, H, hpg, dk, dv, lengths):  # noqa: F811
    x = draw(B, T, H, hpg, dk, dv, torch.bfloat16, seed=T, lengths=lengths)
    got = run_bwd(sml, x)
    ref = [group_grads(x, g, hpg) for g in range(H // hpg)]
    for i, name in enumerate(("dq", "dk", "dv", "dstate_in")):
        want = torch.cat([r[i] for r in ref], 1 if name == "dstate_in" else 2)
        if name == "dstate_in":
            assert rel(got[i], want) <= REL_STATE, name
        else:
            assert_parity(got[i].double().cpu().numpy(), want.numpy(), name, got[i].dtype)
