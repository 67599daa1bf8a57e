"""GPU tests of the head-decay linear attention (lindecay_fwd, _bwd, _decode_step) against
the 64-bit forms of lindecay_ref.

Tolerances, from the kernels' roundings (unit roundoff of bf16: u = 2^-8):
* bf16 outputs: the masked products P, the state as an operand and the result are each
  rounded to bf16 once, independent errors of at most u (about 0.42 u in the mean square).
  The package's parity bar covers them: relative L2 1e-2, largest error 5e-2 RMS beyond the
  cast's own.
* fp32 states of the bf16 path: w_j z_j enters as two bf16 parts, what is left of a term is
  below 2^-15 and in the mean square below u^2 / 2 = 2^-17; the sums are fp32.  Relative L2
  2^-16.
* fp32 path: products in three tf32 steps leave 2^-22 of a term, sums of up to four steps
  truncate at 2^-23 twelve times at most: 12 x 2^-23 + 2^-22 < 2^-19 relative L2.
* differences: the 64-bit forward's central difference over a step of 1e-5 is exact to about
  1e-9; the fp32 gradient's bound applies.
"""
import pytest
import torch

from lindecay_ref import lindecay, pairs, rel
from parity_util import assert_parity

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
REL_STATE, REL_F32 = 2.0 ** -16, 2.0 ** -19


@pytest.fixture(scope="module")
def sml():
    import structured_mask_linear_gb300 as m

    m.lib()
    return m


def draw(B, T, H, hpg, dk, dv, dtype, seed=0, lengths=None, state=True, log_a=None):
    """Inputs on the CPU: 64-bit copies of what the kernels get."""
    g = torch.Generator().manual_seed(seed)
    G = H // hpg
    x = {"q": (B, T, G, dk), "k": (B, T, G, dk), "v": (B, T, H, dv), "dO": (B, T, H, dv)}
    x = {n: (torch.randn(s, generator=g) * (1.0 if n == "dO" else dk ** -0.5)).to(dtype) for n, s in x.items()}
    x["log_a"] = -torch.rand(H, generator=g) if log_a is None else torch.as_tensor(log_a, dtype=torch.float32)
    x["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    for n in ("state_in", "dstate_out"):
        x[n] = torch.randn((B, H, dk, dv), generator=g) * dk ** -0.5 if state else None
    return x


def wide(x, *names):
    return [None if x[n] is None else x[n] if n == "lengths" else x[n].double() for n in names]


def on_gpu(x):
    return {n: None if t is None else t.to(DEV) for n, t in x.items()}


def run_fwd(sml, x):
    d = on_gpu(x)
    B, _, H, dv = x["v"].shape
    st = torch.full((B, H, x["q"].shape[3], dv), float("nan"), device=DEV)
    o = sml.lindecay_fwd(d["q"], d["k"], d["v"], d["log_a"], lengths=d["lengths"], state_in=d["state_in"], state_out=st)
    torch.cuda.synchronize()
    assert sml.loglinear_check_status() == 0
    return o, st


def run_bwd(sml, x):
    d = on_gpu(x)
    ds = None if d["state_in"] is None else torch.full_like(d["state_in"], float("nan"))
    g = sml.lindecay_bwd(d["q"], d["k"], d["v"], d["log_a"], d["dO"], lengths=d["lengths"], state_in=d["state_in"],
                         dstate_out=d["dstate_out"], dstate_in=ds)
    torch.cuda.synchronize()
    assert sml.loglinear_check_status() == 0
    return [*g, ds]


def check_fwd(sml, x, what=""):
    o, st = run_fwd(sml, x)
    ref_o, ref_st = pairs(*wide(x, "q", "k", "v", "log_a", "lengths", "state_in"))
    if x["q"].dtype == torch.bfloat16:
        assert_parity(o.double().cpu().numpy(), ref_o.numpy(), what, o.dtype)
        assert rel(st, ref_st) <= REL_STATE, what
    else:
        assert rel(o, ref_o) <= REL_F32 and rel(st, ref_st) <= REL_F32, what
    return o, st


def ref_grads(x):
    q, k, v, la, n, s0, dO, dS = wide(x, "q", "k", "v", "log_a", "lengths", "state_in", "dO", "dstate_out")
    need = [t.requires_grad_() for t in (q, k, v) + (() if s0 is None else (s0,))]
    o, st = pairs(q, k, v, la, n, s0)
    loss = (o * dO).sum() + (0.0 if dS is None else (st * dS).sum())
    grads = list(torch.autograd.grad(loss, need, allow_unused=True))
    grads = [torch.zeros_like(t) if g is None else g for g, t in zip(grads, need)]
    return grads if s0 is not None else grads + [None]


def check_bwd(sml, x, what=""):
    got, ref = run_bwd(sml, x), ref_grads(x)
    for name, g, r in zip(("dq", "dk", "dv", "dstate_in"), got, ref):
        if r is None:
            continue
        if name == "dstate_in" and g.dtype == torch.float32 and x["q"].dtype == torch.bfloat16:
            assert rel(g, r) <= REL_STATE, (what, name)
        elif g.dtype == torch.bfloat16:
            assert_parity(g.double().cpu().numpy(), r.numpy(), f"{what} {name}", g.dtype)
        else:
            assert rel(g, r) <= REL_F32, (what, name)
    return got


DTYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 127, 128, 129, 300])
def test_lengths_of_sequence(sml, T, dtype):
    x = draw(2, T, 4, 2, 64, 64, dtype, seed=T)
    check_fwd(sml, x)
    check_bwd(sml, x)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dk,dv,H,hpg", [(8, 8, 1, 1), (16, 72, 2, 1), (40, 96, 6, 3), (128, 64, 4, 2), (64, 128, 4, 4),
                                         (128, 128, 3, 1), (72, 24, 8, 8), (104, 120, 10, 5)])
def test_head_layouts(sml, dk, dv, H, hpg, dtype):
    x = draw(2, 270, H, hpg, dk, dv, dtype, seed=dk + dv)
    check_fwd(sml, x)
    check_bwd(sml, x)


@pytest.mark.parametrize("dtype", DTYPES)
def test_without_states(sml, dtype):
    x = draw(1, 200, 2, 1, 64, 64, dtype, state=False)
    check_fwd(sml, x)
    check_bwd(sml, x)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hpg", [1, 2, 3])
def test_ragged_rows_with_garbage_padding(sml, dtype, hpg):
    """Rows of length 0, 1, inside a chunk, at a chunk's end, all; lengths outside [0, T] are
    clamped.  NaN and infinities past a row's length reach nothing, and zeros are written
    there."""
    T = 300
    lengths = [0, 1, 77, 128, 200, 256, 300, -5, 999]
    x = draw(len(lengths), T, 6, hpg, 64, 72, dtype, seed=3, lengths=lengths)
    clean = {n: t for n, t in x.items()}
    for i, n in enumerate(lengths):
        n = min(max(n, 0), T)
        for j, name in enumerate(("q", "k", "v", "dO")):
            x[name] = x[name].clone()
            x[name][i, n:] = float("nan") if (i + j) % 2 else float("inf")
    o, st = run_fwd(sml, x)
    co, cst = check_fwd(sml, clean)
    assert torch.equal(o, co) and torch.equal(st, cst)
    assert all((o[i, min(max(n, 0), T):] == 0).all() for i, n in enumerate(lengths))
    assert torch.equal(st[0].cpu(), x["state_in"][0])
    for g, c in zip(run_bwd(sml, x), check_bwd(sml, clean)):
        assert torch.equal(g, c)


@pytest.mark.parametrize("dtype", DTYPES)
def test_decays(sml, dtype):
    """No decay, hardly any, strong, so strong that a token is gone at the next, and values
    outside the range (which count as its ends)."""
    la = [0.0, -1e-4, -0.5, -3.0, -40.0, -1000.0, float("-inf"), 2.0]
    x = draw(1, 400, len(la), 1, 64, 64, dtype, log_a=la)
    for h in range(len(la)):  # head by head: their magnitudes differ by orders
        y = {n: (t[:, :, h:h + 1].contiguous() if t is not None and n in ("q", "k", "v", "dO") else
                 t[:, h:h + 1].contiguous() if t is not None and "state" in n else t) for n, t in x.items()}
        y["log_a"] = x["log_a"][h:h + 1]
        check_fwd(sml, y, f"log_a {la[h]}")
        check_bwd(sml, y, f"log_a {la[h]}")


@pytest.mark.parametrize("B,T,H,hpg,dk,dv", [
    (1, 4100, 2, 1, 64, 64),     # few heads: segments, a state pass and a prefix over them
    (2, 1500, 2, 2, 128, 72),    # the same with a group's heads summed in the gradients
    (2, 500, 90, 1, 64, 64),     # more units than SMs: units cut between two SMs
    (3, 390, 104, 2, 40, 128),
    (2, 333, 128, 4, 128, 64),   # gradients in two widths
    (1, 260, 180, 3, 64, 40),
])
def test_schedules(sml, B, T, H, hpg, dk, dv):
    """Every way in which the work is shared out, ragged rows among them."""
    n = [T] + [T // 3] * (B - 1)
    x = draw(B, T, H, hpg, dk, dv, torch.bfloat16, seed=H, lengths=n)
    check_fwd(sml, x)
    check_bwd(sml, x)


def test_fp32_segments(sml):
    x = draw(1, 1300, 2, 2, 40, 72, torch.float32, seed=9)
    check_fwd(sml, x)
    check_bwd(sml, x)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,hpg", [(97, 1), (150, 2)])
def test_gradient_against_differences(sml, dtype, T, hpg):
    """<gradient, direction> against the forward's central difference in 64 bits, for each input
    alone.  With bf16 the gradient's own rounding is let through (relative to the norms)."""
    x = draw(2, T, 4, hpg, 24, 40, dtype, seed=T, lengths=[T, T - 20])
    got = run_bwd(sml, x)
    q, k, v, la, n, s0, dO, dS = wide(x, "q", "k", "v", "log_a", "lengths", "state_in", "dO", "dstate_out")
    base = [q, k, v, s0]
    g = torch.Generator().manual_seed(1)
    for i, (name, grad) in enumerate(zip(("q", "k", "v", "state_in"), got)):
        d = torch.randn(base[i].shape, generator=g, dtype=torch.float64)
        loss = []
        for sign in (1.0, -1.0):
            a = list(base)
            a[i] = a[i] + sign * 1e-5 * d
            o, st = lindecay(a[0], a[1], a[2], la, n, a[3])
            loss.append(float((o * dO).sum() + (st * dS).sum()))
        want = (loss[0] - loss[1]) / 2e-5
        have = float((grad.double().cpu() * d).sum())
        tol = 1e-2 if grad.dtype == torch.bfloat16 else REL_STATE if dtype == torch.bfloat16 else REL_F32
        assert abs(have - want) <= 4 * tol * float(grad.double().norm()), name


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dk,dv,hpg", [(128, 64, 2), (64, 64, 1), (40, 24, 3), (8, 128, 1)])
def test_prompt_then_single_tokens(sml, dk, dv, hpg, dtype):
    """A prompt's state continues token by token, and in a further prompt from a state that is
    updated in place."""
    T, more = 150, 6
    x = draw(2, T + more, 2 * hpg, hpg, dk, dv, dtype, seed=dk)
    d = on_gpu(x)
    cut = lambda n, a, b: d[n][:, a:b].contiguous()  # noqa: E731
    st = d["state_in"].clone()
    o = [sml.lindecay_fwd(cut("q", 0, 90), cut("k", 0, 90), cut("v", 0, 90), d["log_a"], state_in=st, state_out=st)]
    o.append(sml.lindecay_fwd(cut("q", 90, T), cut("k", 90, T), cut("v", 90, T), d["log_a"], state_in=st, state_out=st))
    for t in range(T, T + more):
        o.append(sml.lindecay_decode_step(*(d[n][:, t].contiguous() for n in ("q", "k", "v")), d["log_a"], st)[:, None])
    torch.cuda.synchronize()
    assert sml.loglinear_check_status() == 0
    ref_o, ref_st = lindecay(*wide(x, "q", "k", "v", "log_a", "lengths", "state_in"))
    o = torch.cat(o, 1)
    if dtype == torch.bfloat16:
        assert_parity(o.double().cpu().numpy(), ref_o.numpy(), "", o.dtype)
        assert rel(st, ref_st) <= REL_STATE
    else:
        assert rel(o, ref_o) <= REL_F32 and rel(st, ref_st) <= REL_F32


def test_states_past_32_bits(sml):
    """More than 2^31 state elements: the last batch row's states are found and updated."""
    B, H, d = 2100, 64, 128
    st = torch.zeros((B, H, d, d), device=DEV)
    assert st.numel() > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(0)
    q, k, v = (torch.randn((B, H, d), generator=g, device=DEV).to(torch.bfloat16) for _ in range(3))
    la = torch.full((H,), -0.25, device=DEV)
    st[-1] = 1.0
    o = sml.lindecay_decode_step(q, k, v, la, st)
    want = torch.exp(la.double())[:, None, None] + k[-1].double()[:, :, None] * v[-1].double()[:, None, :]
    assert rel(st[-1], want.cpu()) <= 2.0 ** -22
    assert_parity(o[-1].double().cpu().numpy(), (q[-1].double()[:, :, None] * want).sum(1).cpu().numpy(), "", o.dtype)


def test_sequence_past_32_bits(sml):
    """More than 2^31 elements in v and o: the last tokens of the last head."""
    T, H, d = 270_000, 64, 128
    assert T * H * d > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(0)
    q, k, v = (torch.empty((1, T, H, d), device=DEV, dtype=torch.bfloat16).normal_(generator=g) for _ in range(3))
    la = torch.full((H,), -0.5, device=DEV)
    st = torch.empty((1, H, d, d), device=DEV)
    o = sml.lindecay_fwd(q, k, v, la, state_out=st)
    torch.cuda.synchronize()
    assert sml.loglinear_check_status() == 0
    # 300 tokens back a term has decayed by e^-150
    tail = [t[:, -400:, -2:].double().cpu() for t in (q, k, v)]
    ref_o, ref_st = lindecay(*tail, la[-2:].double().cpu())
    assert_parity(o[:, -100:, -2:].double().cpu().numpy(), ref_o[:, -100:].numpy(), "", o.dtype)
    assert rel(st[:, -2:], ref_st) <= REL_STATE


def test_repeated_calls_agree_bitwise(sml):
    """A group's heads add up in order: no result varies between calls."""
    x = draw(2, 700, 48, 4, 64, 64, torch.bfloat16, seed=5)
    a, b = run_bwd(sml, x), run_bwd(sml, x)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    a, b = run_fwd(sml, x), run_fwd(sml, x)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_other_stream_and_given_buffers(sml):
    """On a stream of the caller's, into its buffers and workspace."""
    x = draw(2, 400, 90, 1, 64, 64, torch.bfloat16, seed=6)
    want, _ = run_fwd(sml, x)
    d = on_gpu(x)
    shape = sml.LLShape(2, 400, 90, 1, 64, 64, 0, 0, sml.LL_BF16)
    ws = torch.empty(max(16, sml.lindecay_fwd_workspace_bytes(shape)), dtype=torch.uint8, device=DEV).fill_(0xFF)
    o = torch.empty_like(d["v"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sml.lindecay_fwd(d["q"], d["k"], d["v"], d["log_a"], state_in=d["state_in"], o=o, workspace=ws, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert got.data_ptr() == o.data_ptr() and torch.equal(o, want)
    with torch.cuda.stream(s):
        got = sml.lindecay_fwd(d["q"], d["k"], d["v"], d["log_a"], state_in=d["state_in"])
    s.synchronize()
    assert torch.equal(got, want)
    with pytest.raises(sml.LogLinearError, match="LL_ERR_WORKSPACE"):
        sml.lindecay_fwd(d["q"], d["k"], d["v"], d["log_a"], workspace=ws[:64])


def test_graph_capture(sml):
    x = on_gpu(draw(2, 300, 90, 1, 64, 64, torch.bfloat16, seed=7))
    o = torch.empty_like(x["v"])
    want = sml.lindecay_fwd(x["q"], x["k"], x["v"], x["log_a"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sml.lindecay_fwd(x["q"], x["k"], x["v"], x["log_a"], o=o)
    for _ in range(3):
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)
    assert sml.loglinear_check_status() == 0


def test_refusals(sml):
    x = on_gpu(draw(2, 64, 4, 2, 64, 64, torch.bfloat16, lengths=[3, 64]))
    a = [x["q"], x["k"], x["v"], x["log_a"]]
    bad = lambda i, t: a[:i] + [t] + a[i + 1:]  # noqa: E731
    with pytest.raises(ValueError, match="contiguous"):
        sml.lindecay_fwd(*bad(1, x["k"].transpose(1, 2).contiguous().transpose(1, 2)))
    with pytest.raises(TypeError, match="k must be torch.bfloat16"):
        sml.lindecay_fwd(*bad(1, x["k"].float()))
    with pytest.raises(TypeError, match="unsupported dtype"):
        sml.lindecay_fwd(*(t.half() for t in a[:3]), x["log_a"])
    with pytest.raises(ValueError, match="k must have shape"):
        sml.lindecay_fwd(*bad(1, x["k"][:, :32].contiguous()))
    with pytest.raises(ValueError, match="log_a must have shape"):
        sml.lindecay_fwd(*bad(3, x["log_a"][:2].contiguous()))
    with pytest.raises(ValueError, match="log_a is on cpu"):
        sml.lindecay_fwd(*bad(3, x["log_a"].cpu()))
    with pytest.raises(ValueError, match="do not divide"):
        sml.lindecay_fwd(*(t[:, :, :3].contiguous() if t.dim() == 4 else t for t in bad(0, x["v"])[:2]), *a[2:])
    with pytest.raises(TypeError, match="lengths must be torch.int32"):
        sml.lindecay_fwd(*a, lengths=x["lengths"].long())
    with pytest.raises(ValueError, match="state_in must have shape"):
        sml.lindecay_fwd(*a, state_in=x["state_in"][:1])
    with pytest.raises(ValueError, match="dO is required"):
        sml.lindecay_bwd(*a, None)
    with pytest.raises(TypeError, match="must be a tensor"):
        sml.lindecay_fwd(*bad(2, 3.0))
    wide_heads = torch.zeros((1, 8, 1, 136), device=DEV, dtype=torch.bfloat16)
    with pytest.raises(sml.LogLinearError, match="LL_ERR_SHAPE"):
        sml.lindecay_fwd(wide_heads, wide_heads, wide_heads, torch.zeros(1, device=DEV))
    with pytest.raises(sml.LogLinearError, match="LL_ERR_SHAPE"):  # it may still be read there
        sml.lindecay_bwd(*a, x["dO"], dstate_out=x["dstate_out"], dstate_in=x["dstate_out"])
    odd = torch.zeros(2 * 64 * 4 * 64 + 1, device=DEV, dtype=torch.bfloat16)[1:].view(2, 64, 4, 64)
    with pytest.raises(sml.LogLinearError, match="LL_ERR_ALIGN"):
        sml.lindecay_fwd(*bad(2, odd))
    assert sml.loglinear_check_status() == 0


def test_memory_of_a_call_on_a_given_stream(sml):
    """A result allocated by a call on another stream does not take the place of memory that
    the current stream still has to read."""
    d = on_gpu(draw(1, 30000, 4, 1, 64, 64, torch.bfloat16, seed=7))
    s = torch.cuda.Stream()
    first = sml.lindecay_fwd(d["q"], d["k"], d["v"], d["log_a"])
    torch.ones_like(d["v"]).sum(dtype=torch.float32)
    torch.cuda._sleep(100)  # every kernel is loaded: nothing below waits for that
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    pending = torch.ones_like(d["v"])
    torch.cuda._sleep(50_000_000)  # some 25 ms, ahead of the sum
    total = pending.sum(dtype=torch.float32)
    del pending
    o = sml.lindecay_fwd(d["q"], d["k"], d["v"], d["log_a"], stream=s)
    s.synchronize()
    assert torch.equal(o, first)
    assert float(total) == d["v"].numel()
