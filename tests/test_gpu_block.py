"""GPU tests of the stack of decay-attention blocks (block.py): a prompt and single tokens
against the whole sequence, and every gradient against a plain 64-bit form.

Tolerances (relative L2).  fp32: an operator is exact to 2^-21, a product over up to 192
terms to 2^-20, of independent errors; two blocks are some 20 of them one after the other,
and a norm can pass an error on larger by the ratio of its input's scale to the error's
share of it: 2^-14 for outputs, 2^-13 for gradients, which run through both directions.
bf16: each block rounds eight tensors to 2^-9, independently, which two blocks add up to
2^-9 sqrt(16) = 2^-7; 2^-6 leaves the products' own. Gradients round as many again: 2^-4.
"""
import copy

import pytest
import torch

from lindecay_ref import ACT, pairs, rel, rms

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
OUT = {torch.float32: 2.0 ** -14, torch.bfloat16: 2.0 ** -6}
GRAD = {torch.float32: 2.0 ** -13, torch.bfloat16: 2.0 ** -4}
SIZE = dict(layers=2, width=192, heads=4, groups=2, d_k=40, d_v=48)


def stack(dtype, **kw):
    from structured_mask_linear_gb300.block import DecayStack

    torch.manual_seed(3)
    return DecayStack(**{**SIZE, **kw}, dtype=dtype, device=DEV)


def plain(net, x, lengths=None, states=None):
    """The same stack in 64 bits on the CPU (net: a double copy)."""
    n = len(net.blocks)
    h, after = rms(x, x.shape[-1], 1e-6) * net.blocks[0].w_pre, []
    for i, b in enumerate(net.blocks):
        q, k, v, g = b.project(h)
        o, s = pairs(q, k, v, b.log_a, lengths, None if states is None else states[i])
        after.append(s)
        o = o.reshape(g.shape)
        y = (rms(o, b.d_v, 1.0) * b.w_head * ACT["silu"](g)) @ b.w_o.t()
        x = x + rms(y, y.shape[-1], 1e-6) * b.w_post * b.scale
        h = rms(x, x.shape[-1], 1e-6) * (net.blocks[i + 1].w_pre if i + 1 < n else net.w_last)
    return h, after


def draw(B, T, dtype, seed=0):
    return torch.randn((B, T, SIZE["width"]), generator=torch.Generator().manual_seed(seed)).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,prompt", [(140, 133), (5, 1), (3, 0)])
def test_prompt_then_tokens_is_the_whole_sequence(dtype, T, prompt):
    net, x = stack(dtype), draw(2, T, dtype)
    want, _ = plain(copy.deepcopy(net).double().cpu(), x.double())
    x = x.to(DEV)
    with torch.no_grad():
        if prompt:
            h, states = net(x[:, :prompt].contiguous())
            assert rel(h, want[:, :prompt]) <= OUT[dtype]
        else:
            states = [torch.zeros((2, b.heads, b.d_k, b.d_v), device=DEV) for b in net.blocks]
        for t in range(prompt, T):
            assert rel(net.step(x[:, t].contiguous(), states), want[:, t]) <= OUT[dtype], t


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ragged_prompts_go_on_where_each_ends(dtype):
    net, x = stack(dtype), draw(3, 150, dtype)
    n = torch.tensor([150, 0, 37], dtype=torch.int32)
    ref = copy.deepcopy(net).double().cpu()
    nxt = draw(3, 1, dtype, seed=1)
    with torch.no_grad():
        _, states = net(x.to(DEV), n.to(DEV))
        got = net.step(nxt[:, 0].to(DEV), states)
        for b in range(3):
            row = torch.cat([x[b:b + 1, :int(n[b])], nxt[b:b + 1]], 1).double()
            assert rel(got[b], plain(ref, row)[0][0, -1]) <= OUT[dtype], b


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_states", [False, True])
def test_gradients_of_every_weight(dtype, with_states):
    net, x = stack(dtype), draw(2, 131, dtype)
    w = draw(2, 131, dtype, seed=2)
    ref = copy.deepcopy(net).double().cpu()
    shape = (2, SIZE["heads"], SIZE["d_k"], SIZE["d_v"])
    s0 = [torch.randn(shape, generator=torch.Generator().manual_seed(9 + i)) for i in range(2)] if with_states else None

    xd = x.to(DEV).requires_grad_()
    sd = [s.to(DEV).requires_grad_() for s in s0] if with_states else None
    h, after = net(xd, states=sd)
    loss = (h.float() * w.to(DEV).float()).sum() + (sum(s.square().sum() for s in after) if with_states else 0.0)
    loss.backward()
    xr = x.double().requires_grad_()
    sr = [s.double().requires_grad_() for s in s0] if with_states else None
    h, after = plain(ref, xr, states=sr)
    loss = (h * w.double()).sum() + (sum(s.square().sum() for s in after) if with_states else 0.0)
    loss.backward()
    torch.cuda.synchronize()
    assert rel(xd.grad, xr.grad) <= GRAD[dtype]
    for (name, p), q in zip(net.named_parameters(), ref.parameters()):
        assert rel(p.grad, q.grad) <= GRAD[dtype], name
    for i in range(2 if with_states else 0):
        assert rel(sd[i].grad, sr[i].grad) <= GRAD[dtype], i


def test_on_another_stream_and_again():
    """The same bits on a stream of the caller's, and at every repetition."""
    net, x = stack(torch.bfloat16), draw(2, 260, torch.bfloat16).to(DEV)

    def run():
        net.zero_grad(set_to_none=True)
        h, _ = net(x)
        h.float().square().sum().backward()
        return [h.detach()] + [p.grad.clone() for b in net.blocks for p in (b.w_pre, b.w_head, b.w_post, b.scale)]

    first = run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        second = run()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, second))


def test_refuses_heads_that_do_not_share_evenly():
    with pytest.raises(ValueError):
        stack(torch.float32, heads=5)
