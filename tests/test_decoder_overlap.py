"""CPU tests of the boundary of the gated recurrence and of the head norms with rotation: an output in the
place of what is still read, or of another output, is refused before any CUDA call."""
import ctypes

import pytest

import structured_mask_linear_gb300 as sml
from structured_mask_linear_gb300 import _build

FAKE = 0x10000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    _build.build()
    return sml.lib()


def call(f, shape, names, tail=(), **k):
    at = {a: FAKE + 16 * n for n, a in enumerate(names)}
    at.update({a: at[b] for a, b in k.items()})
    return f(ctypes.byref(shape), *[at[a] for a in names], *tail, None)


SCAN = ("x", "r", "i", "decay", "lengths", "state_in", "h", "state_out")
STEP = ("x", "r", "i", "decay", "states", "h")
HEADS = ("q", "k", "w_q", "w_k", "inv_freq", "positions", "q_out", "k_out")
BACK = ("dq_out", "dk_out", "q", "k", "w_q", "w_k", "inv_freq", "positions", "dq", "dk", "dw_q", "dw_k")


def test_gatescan(L):
    s = sml.GatescanShape(batch=2, T=1, dim=64, mix=0, dtype=sml.LL_F32)
    for o, others in (("h", ("decay", "lengths", "state_in", "state_out")), ("state_out", ("x", "r", "i", "decay", "lengths", "h"))):
        for q in others:
            assert call(L.gatescan_fwd, s, SCAN, **{o: q}) == 2, (o, q)
    for o, others in (("states", ("x", "r", "i", "decay", "h")), ("h", ("decay", "states"))):
        for q in others:
            assert call(L.gatescan_decode_step, s, STEP, **{o: q}) == 2, (o, q)


def test_headrope(L):
    s = sml.HeadropeShape(rows=1, T=1, q_heads=1, k_heads=1, dim=64, rot=64, layout=0, norm=1, eps=1e-6, scale_q=1.0,
                          scale_k=1.0, dtype=sml.LL_F32)
    shared = ("w_q", "w_k", "inv_freq", "positions")
    for o in ("q_out", "k_out"):
        for q in shared:
            assert call(L.headrope_fwd, s, HEADS, **{o: q}) == 2, (o, q)
    for o in ("dq", "dk", "dw_q", "dw_k"):
        for q in shared + ("q", "k", "dq_out", "dk_out") * o.startswith("dw"):
            assert call(L.headrope_bwd, s, BACK, (FAKE, 1 << 40), **{o: q}) == 2, (o, q)
    assert call(L.headrope_bwd, s, BACK, (FAKE, 1 << 40), dw_q="dw_k") == 2
    assert call(L.headrope_bwd, s, BACK, (FAKE, 1 << 40), dw_q="dq") == 2
