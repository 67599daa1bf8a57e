"""GPU test of the rotation's angles at every position, against exact rational arithmetic.

Tolerance: the frequency is held in steps of 2^-64 turns, at most 2^31 of them, and 32 bits of a turn are used:
1.5 * 2^-32 turns, 2^-28.7 radians; what is left is at most an eighth of a turn and rounded to fp32, 2^-28 turns,
2^-25.3 radians; sine and cosine are off by a step of a number below 1, 2^-24.  Together 1.5 * 2^-24:
2^-23, whatever the position and the frequency.
"""
import math
from fractions import Fraction

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TURN = 2 * Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)


@pytest.mark.parametrize("layout", ["half", "inter"])
@pytest.mark.parametrize("f", [1.0, 0.5, 3e-6, 1e-12, 123.456, -0.37, 65537.0, 2.0 ** 33 * 1.1, -2.0 ** 55 * 1.7, 2.0 ** 62 * 1.9, 1e-42, 0.0])
def test_angles(f, layout):
    import structured_mask_linear_gb300 as sml

    far = (1 << 31) - 1
    g = torch.Generator().manual_seed(1)
    p = torch.cat([torch.tensor([0, 1, -1, 2, far, -far, -far - 1, far - 1, far // 3, 1 << 24, (1 << 24) + 1]),
                   torch.randint(-far, far, (500,), generator=g)]).to(torch.int32)
    q = torch.tensor([1.0, 0.0]).expand(len(p), 1, 2).contiguous()
    f32 = torch.tensor([f])
    got, _ = sml.headrope_fwd(q.to(DEV), inv_freq=f32.to(DEV), positions=p.to(DEV), norm="none", layout=layout)
    exact = Fraction(float(f32[0])) / TURN
    for pos, (c, s) in zip(p.tolist(), got[:, 0].double().cpu().tolist()):
        turns = exact * pos
        angle = float((turns - math.floor(turns)) * TURN)
        assert abs(c - math.cos(angle)) <= 2.0 ** -23 and abs(s - math.sin(angle)) <= 2.0 ** -23, pos
