"""Blocks of decoders, as layers: the operators under autograd (first derivatives, backward; a second one
and forward mode raise), and a stack of blocks that trains, takes a prompt and generates token by token.

A block holds one norm before it, projections, a mixer of tokens, a norm of each head under the
gate, the projection back, and a norm after it under a learned scale:

    q, k, v, g = h W_q, h W_k, h W_v, h W_g
    q, k       = norm and rotation of each head        headrope (if asked for)
    o          = lindecay(q, k, v)                     state S (d_k x d_v) per head
    u          = silu(g) * norm_head(o) * w_head       blocknorm: "heads"
    x'         = x + scale * norm(u W_o) * w_post      blocknorm: both of these
    h'         = norm(x') * w_pre'                     in one pass, w_pre' of what comes next

The mixer may instead be a recurrence per channel, o = gatescan(h W_x, h W_r, h W_i) with a decay
that is learned.  Behind the mixer a block may have a feed-forward half, y = ffgate(h') W_down,
between the same two norms.

The norms' epsilons are arguments, to be those that a model was trained with.  For training from
the start q begins smaller by sqrt(d_k), so that a product q k v begins at a mean square of 1,
and that is the head norm's epsilon unless another is given.  A sequence's first outputs are
(q_0 k_0) v_0 alone, and where q_0 k_0 happens to be near zero a norm with a small epsilon would
make one token's gradient the whole sum, and a rounding of q or k a large share of it (7 % of a
weight's gradient in bf16, against 1 %).  Only the projections are library products; the rest is
three kernels per block going forward and three calls going back (a feed-forward half: two and
two more).  Decays of the attention are constants of the model, as log_a.
"""
from __future__ import annotations

import math
from typing import List, Optional, Sequence, Tuple

import torch
from torch import nn
from torch.autograd import forward_ad
from torch.nn import functional as F

from . import (MIXES, blocknorm_bwd, blocknorm_fwd, ffgate_bwd, ffgate_fwd, gatescan_bwd, gatescan_decode_step, gatescan_fwd,
               headrope_bwd, headrope_fwd, lindecay_bwd, lindecay_decode_step, lindecay_fwd, rope_frequencies)


class _FirstOrder(torch.autograd.Function):
    """A backward's gradients, made part of the graph of what they depend on, where they refuse to
    be differentiated.  The library's calls return tensors without history: with create_graph they
    would pass for constants, and a loss over them would lose its gradient without a word."""

    @staticmethod
    def forward(ctx, name, n, *tensors):  # n gradients, then what they depend on
        ctx.name = name
        return tuple(None if t is None else t.clone() for t in tensors[:n])

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError(f"{ctx.name} has no second derivative: its gradients cannot be differentiated")


def _first_order(name, grads, *inputs):
    return _FirstOrder.apply(name, len(grads), *grads, *inputs) if torch.is_grad_enabled() else grads


def _constant(*tensors):
    """Whether nothing can be derived from a call on these: grad mode is off, and none carries a tangent, which
    no_grad leaves to it (and which the functions below refuse)."""
    if torch.is_grad_enabled():
        return False
    # outside of forward mode, where every token of a generation is, there is no need to ask each tensor
    return getattr(forward_ad, "_current_level", 0) < 0 or all(
        t is None or forward_ad.unpack_dual(t).tangent is None for t in tensors)


class _Lindecay(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_a, lengths, state_in):
        B, H = v.shape[0], v.shape[2]
        state_out = torch.empty((B, H, k.shape[3], v.shape[3]), dtype=torch.float32, device=v.device)
        o = lindecay_fwd(q, k, v, log_a, lengths=lengths, state_in=state_in, state_out=state_out)
        ctx.save_for_backward(q, k, v, log_a, lengths, state_in)
        ctx.set_materialize_grads(False)
        return o, state_out

    @staticmethod
    def backward(ctx, dO, dstate_out):
        q, k, v, log_a, lengths, state_in = ctx.saved_tensors
        dO = torch.zeros_like(v) if dO is None else dO.contiguous()
        dstate_out = None if dstate_out is None else dstate_out.contiguous()
        dstate_in = torch.empty_like(state_in) if ctx.needs_input_grad[5] else None
        grads = lindecay_bwd(q, k, v, log_a, dO, lengths=lengths, state_in=state_in, dstate_out=dstate_out,
                             dstate_in=dstate_in)
        dq, dk, dv, dstate_in = _first_order("lindecay", (*grads, dstate_in), q, k, v, state_in, dO, dstate_out)
        return dq, dk, dv, None, None, dstate_in


class _Blocknorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, w_post, x, gate, scale, w_pre, group, act, eps):
        x_new, h = blocknorm_fwd(y, w_post, x, gate, scale, w_pre, group=group, act=act, eps=eps)
        ctx.save_for_backward(y, w_post, gate, scale, w_pre, None if h is None else x_new)
        ctx.args = dict(group=group, act=act, eps=eps, residual=x is not None)
        ctx.set_materialize_grads(False)
        if y is None:  # x' is x: not an output of this call
            return None, h
        return x_new, h

    @staticmethod
    def backward(ctx, dx_new, dh):
        y, w_post, gate, scale, w_pre, x_new = ctx.saved_tensors
        if dh is None:  # nothing came back through the norm after
            x_new = w_pre = None
        if dx_new is None and dh is None:
            return (None,) * 9
        g = blocknorm_bwd(None if dx_new is None else dx_new.contiguous(), y, w_post,
                          None if dh is None else dh.contiguous(), x_new, gate, scale, w_pre, **ctx.args)
        g = _first_order("blocknorm", (g.dy, g.dw_post, g.dx, g.dgate, g.dscale, g.dw_pre), dx_new, dh, y, w_post,
                         x_new, gate, scale, w_pre)
        return (*g, None, None, None)


class _Gatescan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, r, decay, i, mix, lengths, state_in):
        state_out = torch.empty((x.shape[0], x.shape[2]), dtype=torch.float32, device=x.device)
        h = gatescan_fwd(x, r, decay, i=i, mix=mix, lengths=lengths, state_in=state_in, state_out=state_out)
        ctx.save_for_backward(x, r, decay, i, h, lengths, state_in)
        ctx.mix = mix
        ctx.set_materialize_grads(False)
        return h, state_out

    @staticmethod
    def backward(ctx, dh, dstate_out):
        x, r, decay, i, h, lengths, state_in = ctx.saved_tensors
        dh = torch.zeros_like(x) if dh is None else dh.contiguous()
        dstate_out = None if dstate_out is None else dstate_out.contiguous()
        dstate_in = torch.empty_like(state_in) if ctx.needs_input_grad[6] else None
        g = gatescan_bwd(dh, x, r, decay, h, i=i, mix=ctx.mix, lengths=lengths, state_in=state_in, dstate_out=dstate_out,
                         dstate_in=dstate_in)
        dx, dr, ddecay, di, dstate_in = _first_order("gatescan", (g.dx, g.dr, g.ddecay, g.di, dstate_in), x, r, decay, i,
                                                     h, state_in, dh, dstate_out)
        return dx, dr, ddecay, di, None, None, dstate_in


class _Headrope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, w_q, w_k, inv_freq, positions, args):
        ctx.save_for_backward(q, k, w_q, w_k, inv_freq, positions)
        ctx.args = args
        ctx.set_materialize_grads(False)
        return headrope_fwd(q, k, w_q=w_q, w_k=w_k, inv_freq=inv_freq, positions=positions, **args)

    @staticmethod
    def backward(ctx, dq, dk):
        q, k, w_q, w_k, inv_freq, positions = ctx.saved_tensors
        if dq is None and dk is None:
            return (None,) * 7
        dq = torch.zeros_like(q) if dq is None else dq.contiguous()
        dk = None if k is None else torch.zeros_like(k) if dk is None else dk.contiguous()
        g = headrope_bwd(dq, q, dk, k, w_q=w_q, w_k=w_k, inv_freq=inv_freq, positions=positions, **ctx.args)
        g = _first_order("headrope", tuple(g), dq, dk, q, k, w_q, w_k)
        return (*g, None, None, None)


class _Ffgate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, act):
        keep = any(ctx.needs_input_grad)
        gate, up = (x.new_empty((*x.shape[:-1], w_gate.shape[0])) if keep else None for _ in range(2))
        m = ffgate_fwd(x, w_gate, w_up, act=act, gate=gate, up=up)
        ctx.save_for_backward(x, w_gate, w_up, gate, up)
        ctx.act = act
        return m

    @staticmethod
    def backward(ctx, dm):
        x, w_gate, w_up, gate, up = ctx.saved_tensors
        g = ffgate_bwd(dm.contiguous(), x, w_gate, w_up, gate, up, act=ctx.act, need=ctx.needs_input_grad[:3])
        return (*_first_order("ffgate", tuple(g), dm, x, w_gate, w_up), None)


def gatescan(x, r, decay, i=None, mix="rms", lengths=None, state_in=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """gatescan_fwd under autograd (first derivatives): h and the final states."""
    return _Gatescan.apply(x, r, decay, i, mix, lengths, state_in)


def headrope(q, k=None, w_q=None, w_k=None, inv_freq=None, positions=None, layout="half", norm="rms", eps=1e-6, scale_q=1.0,
             scale_k=1.0):
    """headrope_fwd under autograd (first derivatives): q and k.  Frequencies, positions and scales
    are constants: an inv_freq that asks for a gradient, which there is none of, is refused."""
    if inv_freq is not None and inv_freq.requires_grad and torch.is_grad_enabled():
        raise ValueError("inv_freq is a constant of headrope, which has no gradient for it: detach it")
    if _constant(q, k, w_q, w_k, inv_freq):
        return headrope_fwd(q, k, w_q=w_q, w_k=w_k, inv_freq=inv_freq, positions=positions, layout=layout, norm=norm, eps=eps,
                            scale_q=scale_q, scale_k=scale_k)
    return _Headrope.apply(q, k, w_q, w_k, inv_freq, positions,
                           dict(layout=layout, norm=norm, eps=eps, scale_q=scale_q, scale_k=scale_k))


def ffgate(x, w_gate, w_up, act="silu"):
    """ffgate_fwd under autograd (first derivatives)."""
    if _constant(x, w_gate, w_up):
        return ffgate_fwd(x, w_gate, w_up, act=act)
    return _Ffgate.apply(x, w_gate, w_up, act)


def lindecay(q, k, v, log_a, lengths=None, state_in=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """lindecay_fwd under autograd (first derivatives): o and the final states.  log_a and lengths
    are constants: a log_a that asks for a gradient, which there is none of, is refused."""
    if log_a.requires_grad and torch.is_grad_enabled():
        raise ValueError("log_a is a constant of lindecay, which has no gradient for it: detach it")
    return _Lindecay.apply(q, k, v, log_a, lengths, state_in)


def blocknorm(y=None, w_post=None, x=None, gate=None, scale=None, w_pre=None, group=None, act="silu", eps=1e-6):
    """blocknorm_fwd under autograd (first derivatives): (x', h)."""
    if _constant(y, w_post, x, gate, scale, w_pre):
        return blocknorm_fwd(y, w_post, x, gate, scale, w_pre, group=group, act=act, eps=eps)
    x_new, h = _Blocknorm.apply(y, w_post, x, gate, scale, w_pre, group, act, eps)
    return (x if y is None else x_new), h


def head_decays(heads: int, shortest: float = 8.0, longest: float = 2048.0) -> torch.Tensor:
    """log_a (heads,) of half-lives spread evenly in the logarithm, in tokens."""
    step = (longest / shortest) ** (1.0 / max(heads - 1, 1))
    return torch.tensor([-math.log(2.0) / (shortest * step ** h) for h in range(heads)], dtype=torch.float32)


def _product(n_out, n_in, dtype, device, shrink=1):
    w = torch.empty((n_out, n_in), dtype=dtype, device=device)
    return nn.Parameter(w.normal_(0.0, (n_in * shrink) ** -0.5))


def _weight(n, value, device):
    return nn.Parameter(torch.full((n,), value, dtype=torch.float32, device=device))


class DecayBlock(nn.Module):
    """One block's weights, and what it does between its two norms.  rotary: how many values of
    each head of q and k turn with the position; qk_norm ("rms" or "l2"): a norm of those heads
    before, with weights and the epsilon qk_eps.  ff: width of its feed-forward half."""

    def __init__(self, width: int, heads: int, groups: int, d_k: int, d_v: int, dtype=torch.bfloat16, device="cuda",
                 head_eps: float = 1.0, rotary: int = 0, qk_norm: str = "none", ff: int = 0, ff_act: str = "silu",
                 base: float = 10000.0, qk_eps: float = 1e-6):
        super().__init__()
        if heads <= 0 or groups <= 0 or heads % groups:
            raise ValueError(f"heads ({heads}) must be a multiple of groups ({groups})")
        self.heads, self.groups, self.d_k, self.d_v, self.head_eps = heads, groups, d_k, d_v, head_eps
        product = lambda n_out, n_in, shrink=1: _product(n_out, n_in, dtype, device, shrink)  # noqa: E731
        weight = lambda n, value: _weight(n, value, device)  # noqa: E731
        self.w_q, self.w_k = product(groups * d_k, width, shrink=d_k), product(groups * d_k, width)
        self.w_v, self.w_g = product(heads * d_v, width), product(heads * d_v, width)
        self.w_o = product(width, heads * d_v)
        self.w_pre, self.w_head = weight(width, 1.0), weight(heads * d_v, 1.0)
        self.w_post, self.scale = weight(width, 1.0), weight(width, 0.5)
        self.register_buffer("log_a", head_decays(heads).to(device))
        self.qk_norm, self.qk_eps, self.rotary = qk_norm, qk_eps, rotary
        if qk_norm != "none":  # q begins smaller by sqrt(d_k), as without the norm
            self.w_q_norm, self.w_k_norm = weight(d_k, d_k ** -0.5 if qk_norm == "rms" else 1.0), weight(d_k, 1.0)
        if rotary:
            self.register_buffer("inv_freq", rope_frequencies(rotary, base, device=device), persistent=False)
        _feed_forward(self, width, ff, ff_act, product, weight)

    def state(self, batch: int):
        """States in front of a sequence."""
        return torch.zeros((batch, self.heads, self.d_k, self.d_v), dtype=torch.float32, device=self.w_q.device)

    def project(self, h):
        """q, k, v by head, and the gate, for any leading sizes."""
        n = h.shape[:-1]
        return (F.linear(h, self.w_q).view(*n, self.groups, self.d_k),
                F.linear(h, self.w_k).view(*n, self.groups, self.d_k),
                F.linear(h, self.w_v).view(*n, self.heads, self.d_v), F.linear(h, self.w_g))

    def place(self, q, k, positions):
        """q and k under their norm and rotation, where the block has one."""
        if self.qk_norm == "none" and not self.rotary:
            return q, k
        w_q, w_k = (None, None) if self.qk_norm == "none" else (self.w_q_norm, self.w_k_norm)
        return headrope(q, k, w_q, w_k, self.inv_freq if self.rotary else None, positions, norm=self.qk_norm,
                        eps=self.qk_eps)

    def mix(self, h, lengths, state, positions):
        """The heads' outputs, the gate, and the states after."""
        q, k, v, g = self.project(h)
        q, k = self.place(q, k, positions)
        o, s = lindecay(q, k, v, self.log_a, lengths, state)
        return o, g, s

    def mix_token(self, h, state, positions):
        """mix() of one token; the states move on in place."""
        q, k, v, g = self.project(h)
        q, k = self.place(q, k, positions)
        return lindecay_decode_step(q, k, v, self.log_a, state), g

    def back(self, o, g):
        """From the heads' outputs to the block's, ahead of the norm after it."""
        u, _ = blocknorm(o.reshape(g.shape), self.w_head, gate=g, group=self.d_v, eps=self.head_eps)
        return F.linear(u, self.w_o)


class ScanBlock(nn.Module):
    """A block whose mixer is a gated recurrence over `channels`, in `heads` groups for the norm
    under the gate.  Decays begin at half-lives from 8 to 2048 tokens (at gates of one half) and are
    learned, as log_decay."""

    def __init__(self, width: int, channels: int, heads: int, dtype=torch.bfloat16, device="cuda", head_eps: float = 1e-6,
                 mix: str = "rms", ff: int = 0, ff_act: str = "silu"):
        super().__init__()
        if heads <= 0 or channels % heads:
            raise ValueError(f"channels ({channels}) must be a multiple of heads ({heads})")
        if mix not in MIXES:
            raise ValueError(f"mix must be one of {sorted(MIXES)}, got {mix!r}")
        self.channels, self.d_v, self.head_eps, self.mixing = channels, channels // heads, head_eps, mix
        product = lambda n_out, n_in, shrink=1: _product(n_out, n_in, dtype, device, shrink)  # noqa: E731
        weight = lambda n, value: _weight(n, value, device)  # noqa: E731
        self.w_x, self.w_r, self.w_i = (product(channels, width) for _ in range(3))
        self.w_g, self.w_o = product(channels, width), product(width, channels)
        self.w_pre, self.w_head = weight(width, 1.0), weight(channels, 1.0)
        self.w_post, self.scale = weight(width, 1.0), weight(width, 0.5)
        self.log_decay = nn.Parameter(torch.log(-2.0 * head_decays(channels)).to(device))
        _feed_forward(self, width, ff, ff_act, product, weight)

    def state(self, batch: int):
        """States in front of a sequence."""
        return torch.zeros((batch, self.channels), dtype=torch.float32, device=self.w_x.device)

    def mix(self, h, lengths, state, positions):
        x, r, i, g = (F.linear(h, w) for w in (self.w_x, self.w_r, self.w_i, self.w_g))
        o, s = gatescan(x, r, self.log_decay.exp(), i, self.mixing, lengths, state)
        return o, g, s

    def mix_token(self, h, state, positions):
        x, r, i, g = (F.linear(h, w) for w in (self.w_x, self.w_r, self.w_i, self.w_g))
        return gatescan_decode_step(x, r, self.log_decay.exp(), state, i_t=i, mix=self.mixing), g

    back = DecayBlock.back


def _feed_forward(block, width, ff, act, product, weight):
    """The weights of a block's feed-forward half (ff 0: it has none)."""
    block.ff, block.ff_act = ff, act
    if ff:
        block.w_gate, block.w_up, block.w_down = product(ff, width), product(ff, width), product(width, ff)
        block.w_ff_pre, block.w_ff_post, block.ff_scale = weight(width, 1.0), weight(width, 1.0), weight(width, 0.5)


class DecayStack(nn.Module):
    """Blocks on a residual stream.  forward() for training and prompts, step() for a token.  eps: of
    the norms over the stream and over a block's output; head_eps: of the norm of each head, in blocks of
    both kinds (none given: 1 in DecayBlocks, 1e-6 in ScanBlocks).
    rotary, qk_norm, qk_eps, ff: of every block, as DecayBlock has them; recurrent: which blocks (by index)
    are ScanBlocks, of `channels` channels (width unless given) with n(a) as `mix` says."""

    def __init__(self, layers: int, width: int, heads: int, groups: int, d_k: int, d_v: int, dtype=torch.bfloat16,
                 device="cuda", eps: float = 1e-6, head_eps: Optional[float] = None, rotary: int = 0, qk_norm: str = "none", ff: int = 0,
                 ff_act: str = "silu", recurrent: Sequence[int] = (), channels: int = 0, base: float = 10000.0,
                 mix: str = "rms", qk_eps: float = 1e-6):
        super().__init__()
        if any(not 0 <= i < layers for i in recurrent):
            raise ValueError(f"recurrent blocks {tuple(recurrent)} are not among {layers}")
        self.eps, self.rotary = eps, rotary
        self.blocks = nn.ModuleList(
            ScanBlock(width, channels or width, heads, dtype, device, 1e-6 if head_eps is None else head_eps, mix, ff, ff_act)
            if i in recurrent else
            DecayBlock(width, heads, groups, d_k, d_v, dtype, device, 1.0 if head_eps is None else head_eps, rotary, qk_norm, ff,
                       ff_act, base, qk_eps)
            for i in range(layers))
        self.w_last = nn.Parameter(torch.ones(width, dtype=torch.float32, device=device))

    def _after(self, i):
        return self.blocks[i + 1].w_pre if i + 1 < len(self.blocks) else self.w_last

    def _joint(self, i, y, x):
        """From block i's mixer (its output y) to the next block's input: (x', h')."""
        b = self.blocks[i]
        if b.ff:
            x, h = blocknorm(y, b.w_post, x, scale=b.scale, w_pre=b.w_ff_pre, eps=self.eps)
            y = F.linear(ffgate(h, b.w_gate, b.w_up, b.ff_act), b.w_down)
            return blocknorm(y, b.w_ff_post, x, scale=b.ff_scale, w_pre=self._after(i), eps=self.eps)
        return blocknorm(y, b.w_post, x, scale=b.scale, w_pre=self._after(i), eps=self.eps)

    def states(self, batch: int) -> List[torch.Tensor]:
        """The blocks' states in front of `batch` sequences, for step()."""
        return [b.state(batch) for b in self.blocks]

    def forward(self, x, lengths: Optional[torch.Tensor] = None, states: Optional[List[torch.Tensor]] = None,
                start: Optional[torch.Tensor] = None):
        """x (B, T, width), lengths (B,) int32 and the blocks' states before it (none: zero).
        start (B,) int32: each row's first position, for rotary, which asks for it where states are given
        (none: 0).
        Returns the stream under its last norm and the states after each row's length."""
        positions = None
        if self.rotary and states is not None and start is None:
            raise ValueError("a stack with rotary heads that goes on from states needs each row's first position")
        if self.rotary and start is not None:
            positions = start[:, None] + torch.arange(x.shape[1], dtype=torch.int32, device=x.device)
        _, h = blocknorm(x=x, w_pre=self.blocks[0].w_pre if len(self.blocks) else self.w_last, eps=self.eps)
        after = []
        for i, b in enumerate(self.blocks):
            o, g, s = b.mix(h, lengths, None if states is None else states[i], positions)
            after.append(s)
            x, h = self._joint(i, b.back(o, g), x)
        return h, after

    @torch.no_grad()
    def step(self, x_t, states: List[torch.Tensor], positions: Optional[torch.Tensor] = None):
        """One token of every row: x_t (B, width); the states move on in place.  positions (B,) int32:
        how many tokens each row has before this one; rotary asks for them."""
        if self.rotary and positions is None:
            raise ValueError("a stack with rotary heads needs each row's position")
        _, h = blocknorm(x=x_t, w_pre=self.blocks[0].w_pre if len(self.blocks) else self.w_last, eps=self.eps)
        for i, b in enumerate(self.blocks):
            o, g = b.mix_token(h, states[i], positions)
            x_t, h = self._joint(i, b.back(o, g), x_t)
        return h
