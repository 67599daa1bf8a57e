"""GPU tests of the gated recurrence over every way a call can be laid out: 1, 2 or 4 groups a warp, one CTA or
several on a sequence, a single step or many, with every mix and with and without an input gate, against the
64-bit forms of decoder_ref (run on the GPU).  Tolerances as in test_gpu_gatescan."""
import pytest
import torch

from decoder_ref import gatescan, gatescan_bwd, rel
from test_gpu_gatescan import BWD, CAST, DEV, FWD, draw, up

pytestmark = pytest.mark.gpu

# On a whole GPU (CTAs on a sequence x steps): bf16 forward, backward; fp32 forward, backward
SHAPES = [(1, 1000, 16),    # 4 groups 5 x 1, 4 groups 5 x 2; 4 groups 5 x 2
          (1, 2000, 512),   # 2 groups 6 x 3, 4 groups 6 x 3; 4 groups 6 x 3
          (2, 600, 1024),   # 2 groups 5 x 1, 2 groups 6 x 2; 2 groups 6 x 2, 1 or 2 groups
          (2, 1500, 2048),  # 1 group 7 x 4, 7 x 7; 1 group 7 x 7, 4 x 12
          (4, 500, 2560),   # 1 group 3 x 3, 8 x 2; 1 or 2 groups, 8 x 2 and 3 x 3
          (4, 700, 4096),   # 2 groups 2 x 3, 1 group 2 x 11; 1 group 2 x 11, 1 x 22
          (4, 4000, 40),    # 4 groups 6 x 3, 8 x 5; 4 groups 8 x 5
          (3, 1501, 1000),  # 4 groups 7 x 1, 1 group 8 x 6; 1 group 8 x 6, 2 groups 3 x 9
          (32, 130, 2048),  # 1 group 1 x 3, 1 x 5; 1 x 5
          (4, 700, 8192)]   # 2 groups 1 x 6, 1 group 2 x 11; 1 group 2 x 11


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("mix", ["rms", "lerp", "none"])
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_layouts(B, T, D, mix, gate, dtype):
    import structured_mask_linear_gb300 as sml

    c = up(draw(B, T, D, dtype, gate, ragged=B % 2 == 1 and B > 1, seed=T + D))
    w = {n: None if v is None else v if n == "lengths" else v.double() for n, v in c.items()}
    st, ds = (torch.full((B, D), float("nan"), device=DEV) for _ in range(2))
    h = sml.gatescan_fwd(c["x"], c["r"], c["decay"], i=c["i"], mix=mix, lengths=c["lengths"], state_in=c["state_in"],
                         state_out=st)
    got = sml.gatescan_bwd(c["dh"], c["x"], c["r"], c["decay"], h, i=c["i"], mix=mix, lengths=c["lengths"],
                           state_in=c["state_in"], dstate_out=c["dstate_out"], dstate_in=ds)
    with torch.device(DEV):
        want, last = gatescan(w["x"], w["r"], w["decay"], w["i"], mix, w["lengths"], w["state_in"])
        dx, dr, di, dd, d0 = gatescan_bwd(w["dh"], w["x"], w["r"], w["decay"], h.double(), w["i"], mix, w["lengths"],
                                          w["state_in"], w["dstate_out"])
    assert rel(h, want.cpu()) <= FWD + CAST[dtype] and rel(st, last.cpu()) <= FWD
    for name, x, y, tol in (("dx", got.dx, dx, CAST[dtype]), ("dr", got.dr, dr, CAST[dtype]), ("di", got.di, di, CAST[dtype]),
                            ("ddecay", got.ddecay, dd, 0.0), ("dstate_in", ds, d0, 0.0)):
        assert (x is None) == (y is None), name
        if x is not None:
            assert rel(x, y.cpu()) <= BWD + tol, (name, rel(x, y.cpu()))
    assert sml.loglinear_check_status() == 0
