"""CPU tests of the head-decay attention's and the block norm's boundary: exports, argument
counts, checks that come before any CUDA call, and the binding's build."""
import ctypes
import os
import re

import pytest
import torch

import structured_mask_linear_gb300 as sml
from structured_mask_linear_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    _build.build()
    return sml.lib()


def prototypes():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "loglinear.h")).read(), flags=re.S)
    return dict(re.findall(r"\b((?:lindecay|blocknorm)_\w+)\s*\(([^)]*)\)\s*;", text))


def test_exports_and_argument_counts(L):
    protos = prototypes()
    assert {"lindecay_fwd", "lindecay_bwd", "lindecay_decode_step", "blocknorm_fwd", "blocknorm_bwd"} <= set(protos)
    for name, params in protos.items():
        assert len(getattr(L, name).argtypes) == params.count(",") + 1, name


def shape(**kw):
    d = dict(batch=2, T=100, heads=4, heads_per_group=2, d_k=128, d_v=64, chunk=0, levels=0, dtype=sml.LL_BF16)
    d.update(kw)
    return sml.LLShape(**d)


BAD = [(dict(d_k=4), 2), (dict(d_k=136), 2), (dict(d_v=12), 2), (dict(d_v=256), 2), (dict(batch=0), 2), (dict(T=0), 2),
       (dict(heads=3), 2), (dict(heads_per_group=0), 2), (dict(dtype=9), 3), (dict(batch=1 << 20), 2)]


@pytest.mark.parametrize("kw,code", BAD)
def test_lindecay_shapes(L, kw, code):
    s = ctypes.byref(shape(**kw))
    assert L.lindecay_fwd_workspace_bytes(s) == 0 and L.lindecay_bwd_workspace_bytes(s) == 0
    assert L.lindecay_fwd(s, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, FAKE, 1 << 40, None) == code
    assert L.lindecay_bwd(s, *[FAKE] * 4, None, None, FAKE, None, *[FAKE] * 3, None, FAKE, 1 << 40, None) == code
    if kw != dict(T=0):  # a step has no T
        assert L.lindecay_decode_step(s, *[FAKE] * 6, None) == code


def test_lindecay_pointers(L):
    s = ctypes.byref(shape())
    fwd = lambda **k: L.lindecay_fwd(s, *[k.get(n, FAKE) for n in ("q", "k", "v", "la")], None,  # noqa: E731
                                     k.get("s_in"), k.get("o", FAKE), k.get("s_out"), k.get("ws", FAKE), 1 << 40, None)
    for n in ("q", "k", "v", "la", "o"):
        assert fwd(**{n: None}) == 1
    for n in ("q", "k", "v", "o", "s_in", "s_out"):
        assert fwd(**{n: FAKE + 8}) == 4
    assert L.lindecay_fwd(None, *[FAKE] * 4, None, None, FAKE, None, FAKE, 1 << 40, None) == 1
    # one state's buffer is not read and written by the same backward call
    assert L.lindecay_bwd(s, *[FAKE] * 4, None, FAKE, FAKE, None, *[FAKE] * 3, FAKE, FAKE, 1 << 40, None) == 2
    assert L.lindecay_bwd(s, *[FAKE] * 4, None, None, FAKE, FAKE, *[FAKE] * 3, FAKE, FAKE, 1 << 40, None) == 2


def test_lindecay_workspace(L):
    """A short prompt needs none; few heads and a long sequence need segments' states."""
    s = ctypes.byref(shape(T=1))
    assert L.lindecay_fwd_workspace_bytes(s) == 16
    s = ctypes.byref(shape(T=100000))
    need = L.lindecay_fwd_workspace_bytes(s)
    assert need > 16
    assert L.lindecay_fwd(s, *[FAKE] * 4, None, None, FAKE, None, FAKE, need - 1, None) == 5
    assert L.lindecay_fwd(s, *[FAKE] * 4, None, None, FAKE, None, None, need, None) == 5
    assert L.lindecay_fwd(s, *[FAKE] * 4, None, None, FAKE, None, FAKE + 8, need, None) == 4


def bn(**kw):
    d = dict(rows=5, dim=64, group=64, act=1, eps=1e-6, dtype=sml.LL_BF16)
    d.update(kw)
    return ctypes.byref(sml.BlocknormShape(**d))


@pytest.mark.parametrize("kw,code", [(dict(rows=0), 2), (dict(rows=1 << 31), 2), (dict(dim=0), 2), (dict(dim=16392), 2),
                                     (dict(group=48), 2), (dict(group=0), 2), (dict(act=3), 2), (dict(eps=-1.0), 2),
                                     (dict(eps=float("nan")), 2), (dict(dtype=5), 3), (dict(dim=8192, group=1), 2)])
def test_blocknorm_shapes(L, kw, code):
    assert L.blocknorm_bwd_workspace_bytes(bn(**kw)) == 0
    assert L.blocknorm_fwd(bn(**kw), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None) == code
    assert L.blocknorm_bwd(bn(**kw), *[FAKE] * 15, 1 << 40, None) == code


def test_blocknorm_pointers(L):
    f = lambda **k: L.blocknorm_fwd(bn(), *[k.get(n) for n in  # noqa: E731
                                            ("x", "y", "gate", "w_post", "scale", "w_pre", "x_new", "h")], None)
    assert f() == 1
    assert f(y=FAKE) == 1                                # no place for x'
    assert f(x=FAKE) == 1                                # nothing to compute
    assert f(x=FAKE, h=FAKE, gate=FAKE) == 1             # a gate without y
    assert f(y=FAKE, x_new=FAKE, w_pre=FAKE) == 1        # a weight for an h that is not asked for
    assert f(y=FAKE + 2, x_new=FAKE) == 4
    names = ("dx_new", "dh", "x_new", "y", "gate", "w_post", "scale", "w_pre", "dx", "dy", "dgate", "dw_post", "dscale",
             "dw_pre", "ws")
    b = lambda n=1 << 40, **k: L.blocknorm_bwd(bn(), *[k.get(m) for m in names], n, None)  # noqa: E731
    assert b() == 1
    assert b(dh=FAKE, y=FAKE, dy=FAKE, ws=FAKE) == 1     # dh without x'
    assert b(dx_new=FAKE, y=FAKE, ws=FAKE) == 1          # no place for dy
    assert b(dx_new=FAKE, y=FAKE, dy=FAKE, dw_post=FAKE, ws=FAKE) == 1  # the gradient of a weight that is not there
    assert b(dx_new=FAKE, y=FAKE, dy=FAKE) == 5
    assert b(100, dx_new=FAKE, y=FAKE, dy=FAKE, ws=FAKE) == 5
    assert b(dx_new=FAKE + 2, y=FAKE, dy=FAKE, ws=FAKE) == 4


def test_binding_refuses_before_cuda(L):
    z = torch.zeros(1, 4, 2, 8)
    with pytest.raises(ValueError, match="must be on a CUDA device"):
        sml.lindecay_fwd(z, z, z, torch.zeros(2))
    with pytest.raises(ValueError, match="k is required"):
        sml.lindecay_fwd(z, None, z, torch.zeros(2))
    with pytest.raises(ValueError, match="dimensions"):
        sml.lindecay_decode_step(z, z, z, torch.zeros(2), z)
    with pytest.raises(ValueError, match="must be on a CUDA device"):
        sml.blocknorm_fwd(z)


def test_parts_are_handed_over_only_while_they_are_short(L):
    """A CTA waits (for 2 s at most) until another one has left a part's state.  The part's time goes
    by its chunks and by the heads that are summed over them: gradients of 8 heads a group hand
    states over, which their workspace holds, up to 2^21 tokens, and beyond that no more."""
    need = [L.lindecay_bwd_workspace_bytes(ctypes.byref(shape(batch=1, heads=128, heads_per_group=8, d_k=8, d_v=8, T=1 << e)))
            for e in (20, 21, 22, 23)]
    assert need[0] == need[1] > need[2] == need[3]


def test_workspace_of_summed_heads(L):
    """Two heads a group run side by side and need no place for their sums; more take turns: 32 KB a
    chunk of 128 tokens for each of the CTAs, at most 16 chunks, and 32 KB a head for the states
    that wait where 16 chunks are not all."""
    need = lambda **kw: L.lindecay_bwd_workspace_bytes(ctypes.byref(shape(d_k=64, d_v=64, **kw)))  # noqa: E731
    tile = 128 * 64 * 4
    assert need(batch=1, heads=4, heads_per_group=2, T=3) == 16
    # items: dq and dk per group, dv per head
    assert need(batch=1, heads=4, heads_per_group=4, T=3) == (1 + 1 + 4) * 1 * tile
    assert need(batch=1, heads=6, heads_per_group=3, T=200) == (2 + 2 + 6) * 2 * tile
    assert need(batch=152, heads=3, heads_per_group=3, T=2048) == 152 * 16 * tile
    assert need(batch=152, heads=3, heads_per_group=3, T=2049) == 152 * (16 + 3) * tile


def test_outputs_in_the_place_of_what_is_still_read(L):
    """Refused, where a call would give wrong results without a word."""
    s = ctypes.byref(shape(T=1, heads=2, heads_per_group=1, d_k=64, d_v=64))
    at = [FAKE * (i + 1) for i in range(16)]
    fwd = lambda o: L.lindecay_fwd(s, *at[:4], None, None, o, None, at[8], 0, None)  # noqa: E731
    assert fwd(at[0]) == 2 and fwd(at[1]) == 2
    bwd = lambda dq, dk, dv: L.lindecay_bwd(s, *at[:4], None, None, at[4], None, dq, dk, dv, None, at[8], 0, None)  # noqa: E731
    places = at[5:8]
    for i in range(3):
        for taken in (*at[:3], at[4], places[(i + 1) % 3]):
            assert bwd(*places[:i], taken, *places[i + 1:]) == 2
    assert L.blocknorm_fwd(bn(), None, at[0], None, None, None, None, at[1], at[1], None) == 2
