"""GPU test of lindecay on a stream that may use only some of the SMs (a green context's): the calls
whose CTAs hand states to one another need every SM at once, and take another plan there."""
import ctypes

import pytest
import torch

from lindecay_ref import rel

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class DevResource(ctypes.Structure):
    """cuda.h's CUdevResource: a type, 92 bytes, and a union of 48 that starts with the SM count."""

    _fields_ = [("type", ctypes.c_int), ("pad", ctypes.c_ubyte * 92), ("sm_count", ctypes.c_uint),
                ("rest", ctypes.c_ubyte * 44)]


@pytest.fixture
def part_stream():
    """A stream on about half of the SMs."""
    torch.zeros(1, device=DEV)  # the primary context
    cu = ctypes.CDLL("libcuda.so.1")

    def call(name, *args):
        f = getattr(cu, name, None)
        code = -1 if f is None else f(*args)
        if code != 0:
            pytest.skip(f"{name}: {code}")

    u32, ref = ctypes.c_uint, ctypes.byref
    whole, part, left = DevResource(), DevResource(), DevResource()
    call("cuDeviceGetDevResource", 0, ref(whole), 1)
    groups = u32(1)
    call("cuDevSmResourceSplitByCount", ref(part), ref(groups), ref(whole), ref(left), u32(0),
         u32(whole.sm_count // 2 // 8 * 8))
    assert part.sm_count < whole.sm_count
    desc, green, stream = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
    call("cuDevResourceGenerateDesc", ref(desc), ref(part), u32(1))
    call("cuGreenCtxCreate", ref(green), desc, 0, u32(1))
    call("cuGreenCtxStreamCreate", ref(stream), green, u32(1), 0)
    yield stream.value
    torch.cuda.synchronize()
    cu.cuStreamDestroy_v2(stream)
    cu.cuGreenCtxDestroy(green)


def test_on_part_of_the_sms(part_stream):
    import structured_mask_linear_gb300 as sml

    B, T, H, d = 2, 500, 90, 64  # 180 units for 152 SMs: units cut between two SMs
    g = torch.Generator().manual_seed(0)
    q, k, v, dO = ((torch.randn((B, T, H, d), generator=g) * 0.125).to(DEV, torch.bfloat16) for _ in range(4))
    la = -torch.rand(H, generator=g).to(DEV)
    shape = sml.LLShape(B, T, H, 1, d, d, 0, 0, sml.LL_BF16)
    ws = [torch.empty(n(shape), dtype=torch.uint8, device=DEV) for n in
          (sml.lindecay_fwd_workspace_bytes, sml.lindecay_bwd_workspace_bytes)]
    st, want_st, o = torch.empty((B, H, d, d), device=DEV), torch.empty((B, H, d, d), device=DEV), torch.empty_like(v)
    want = sml.lindecay_fwd(q, k, v, la, state_out=want_st)
    grads = sml.lindecay_bwd(q, k, v, la, dO)
    torch.cuda.synchronize()
    sml.lindecay_fwd(q, k, v, la, state_out=st, o=o, workspace=ws[0], stream=part_stream)
    torch.cuda.synchronize()
    # the two plans add the same terms up in another order; bf16 outputs may round the other way
    assert rel(o, want.double().cpu()) <= 2.0 ** -8 and rel(st, want_st.double().cpu()) <= 2.0 ** -16
    got = sml.lindecay_bwd(q, k, v, la, dO, workspace=ws[1], stream=part_stream)
    torch.cuda.synchronize()
    for a, b in zip(got, grads):
        assert rel(a, b.double().cpu()) <= 2.0 ** -8
    assert sml.loglinear_check_status() == 0
