"""Linear attention with per-head decay, as layers: the operators under autograd (first
derivatives; a second one raises), and a stack of blocks that trains, takes a prompt and
generates token by token.

A block holds one norm before it, four projections, the attention, a norm of each head under
the gate, the projection back, and a norm after it under a learned scale:

    q, k, v, g = h W_q, h W_k, h W_v, h W_g
    o          = lindecay(q, k, v)                     state S (d_k x d_v) per head
    u          = silu(g) * norm_head(o) * w_head       blocknorm: "heads"
    x'         = x + scale * norm(u W_o) * w_post      blocknorm: both of these
    h'         = norm(x') * w_pre'                     in one pass, w_pre' of the next block

The norms' epsilons are arguments, to be those that a model was trained with.  For training from
the start q begins smaller by sqrt(d_k), so that a product q k v begins at a mean square of 1,
and that is the head norm's epsilon unless another is given.  A sequence's first outputs are
(q_0 k_0) v_0 alone, and where q_0 k_0 happens to be near zero a norm with a small epsilon would
make one token's gradient the whole sum, and a rounding of q or k a large share of it (7 % of a
weight's gradient in bf16, against 1 %).  Only the projections are library products; the rest is
three kernels per block going forward and three calls going back.  Decays are constants of the
model, as log_a.
"""
from __future__ import annotations

import math
from typing import List, Optional, Tuple

import torch
from torch import nn
from torch.nn import functional as F

from . import blocknorm_bwd, blocknorm_fwd, lindecay_bwd, lindecay_decode_step, lindecay_fwd


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


def lindecay(q, k, v, log_a, lengths=None, state_in=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """lindecay_fwd under autograd (first derivatives): o and the final states.  log_a and lengths
    are constants: a log_a that asks for a gradient, which there is none of, is refused."""
    if log_a.requires_grad and torch.is_grad_enabled():
        raise ValueError("log_a is a constant of lindecay, which has no gradient for it: detach it")
    return _Lindecay.apply(q, k, v, log_a, lengths, state_in)


def blocknorm(y=None, w_post=None, x=None, gate=None, scale=None, w_pre=None, group=None, act="silu", eps=1e-6):
    """blocknorm_fwd under autograd (first derivatives): (x', h)."""
    x_new, h = _Blocknorm.apply(y, w_post, x, gate, scale, w_pre, group, act, eps)
    return (x if y is None else x_new), h


def head_decays(heads: int, shortest: float = 8.0, longest: float = 2048.0) -> torch.Tensor:
    """log_a (heads,) of half-lives spread evenly in the logarithm, in tokens."""
    step = (longest / shortest) ** (1.0 / max(heads - 1, 1))
    return torch.tensor([-math.log(2.0) / (shortest * step ** h) for h in range(heads)], dtype=torch.float32)


class DecayBlock(nn.Module):
    """One block's weights, and what it does between its two norms."""

    def __init__(self, width: int, heads: int, groups: int, d_k: int, d_v: int, dtype=torch.bfloat16, device="cuda",
                 head_eps: float = 1.0):
        super().__init__()
        if heads <= 0 or groups <= 0 or heads % groups:
            raise ValueError(f"heads ({heads}) must be a multiple of groups ({groups})")
        self.heads, self.groups, self.d_k, self.d_v, self.head_eps = heads, groups, d_k, d_v, head_eps

        def product(n_out, n_in, shrink=1):
            w = torch.empty((n_out, n_in), dtype=dtype, device=device)
            return nn.Parameter(w.normal_(0.0, (n_in * shrink) ** -0.5))

        def weight(n, value):
            return nn.Parameter(torch.full((n,), value, dtype=torch.float32, device=device))

        self.w_q, self.w_k = product(groups * d_k, width, shrink=d_k), product(groups * d_k, width)
        self.w_v, self.w_g = product(heads * d_v, width), product(heads * d_v, width)
        self.w_o = product(width, heads * d_v)
        self.w_pre, self.w_head = weight(width, 1.0), weight(heads * d_v, 1.0)
        self.w_post, self.scale = weight(width, 1.0), weight(width, 0.5)
        self.register_buffer("log_a", head_decays(heads).to(device))

    def project(self, h):
        """q, k, v by head, and the gate, for any leading sizes."""
        n = h.shape[:-1]
        return (F.linear(h, self.w_q).view(*n, self.groups, self.d_k),
                F.linear(h, self.w_k).view(*n, self.groups, self.d_k),
                F.linear(h, self.w_v).view(*n, self.heads, self.d_v), F.linear(h, self.w_g))

    def back(self, o, g):
        """From the heads' outputs to the block's, ahead of the norm after it."""
        u, _ = blocknorm(o.reshape(g.shape), self.w_head, gate=g, group=self.d_v, eps=self.head_eps)
        return F.linear(u, self.w_o)


class DecayStack(nn.Module):
    """Blocks on a residual stream.  forward() for training and prompts, step() for a token.  eps: of
    the norms over the stream and over a block's output; head_eps: of the norm of each head."""

    def __init__(self, layers: int, width: int, heads: int, groups: int, d_k: int, d_v: int, dtype=torch.bfloat16,
                 device="cuda", eps: float = 1e-6, head_eps: float = 1.0):
        super().__init__()
        self.eps = eps
        self.blocks = nn.ModuleList(DecayBlock(width, heads, groups, d_k, d_v, dtype, device, head_eps)
                                    for _ in range(layers))
        self.w_last = nn.Parameter(torch.ones(width, dtype=torch.float32, device=device))

    def _after(self, i):
        return self.blocks[i + 1].w_pre if i + 1 < len(self.blocks) else self.w_last

    def forward(self, x, lengths: Optional[torch.Tensor] = None, states: Optional[List[torch.Tensor]] = None):
        """x (B, T, width), lengths (B,) int32 and the blocks' states before it (none: zero).
        Returns the stream under its last norm and the states after each row's length."""
        _, h = blocknorm(x=x, w_pre=self.blocks[0].w_pre if len(self.blocks) else self.w_last, eps=self.eps)
        after = []
        for i, b in enumerate(self.blocks):
            q, k, v, g = b.project(h)
            o, s = lindecay(q, k, v, b.log_a, lengths, None if states is None else states[i])
            after.append(s)
            x, h = blocknorm(b.back(o, g), b.w_post, x, scale=b.scale, w_pre=self._after(i), eps=self.eps)
        return h, after

    @torch.no_grad()
    def step(self, x_t, states: List[torch.Tensor]):
        """One token of every row: x_t (B, width); the states move on in place."""
        _, h = blocknorm_fwd(x=x_t, w_pre=self.blocks[0].w_pre if len(self.blocks) else self.w_last, eps=self.eps)
        for i, b in enumerate(self.blocks):
            q, k, v, g = b.project(h)
            y = b.back(lindecay_decode_step(q, k, v, b.log_a, states[i]), g)
            x_t, h = blocknorm_fwd(y, b.w_post, x_t, scale=b.scale, w_pre=self._after(i), eps=self.eps)
        return h
