"""Plain 64-bit forms of the head-decay linear attention and of the block norm (torch, CPU),
for the tests of their kernels.  The attention is there twice, as the recurrence token by
token and as the masked product over all pairs (which test_lindecay_ref holds against each
other); gradients come from differentiating these forms."""
import torch


def pairs(q, k, v, log_a, lengths=None, state_in=None):
    """lindecay() as masked products over all pairs of tokens."""
    B, T, G, _ = q.shape
    H = v.shape[2]
    n = torch.full((B,), T) if lengths is None else lengths.long().clamp(0, T)
    t = torch.arange(T)
    on = (t < n[:, None])[:, :, None, None]
    q, k = (x.repeat_interleave(H // G, 2) for x in (q, k))
    q, k, v = (torch.where(on, x, torch.zeros_like(x)).transpose(1, 2) for x in (q, k, v))  # (B, H, T, .)
    la = log_a.clamp(-1000.0, 0.0)

    def power(e):  # g^e (H, *e.shape), 0 where e < 0
        e = e.to(q.dtype)
        return torch.exp(la.view(-1, *[1] * e.dim()) * e.clamp(min=0)) * (e >= 0)

    o = ((q @ k.transpose(-1, -2)) * power(t[:, None] - t[None, :])) @ v
    left = power(n[:, None] - 1 - t[None, :]).transpose(0, 1)  # (B, H, T)
    S = (k * left[..., None]).transpose(-1, -2) @ v
    if state_in is not None:
        o = o + (q * power(t + 1)[None, :, :, None]) @ state_in
        S = S + power(n).t()[..., None, None] * state_in
    o = o.transpose(1, 2)
    return torch.where(on, o, torch.zeros_like(o)), S


def lindecay(q, k, v, log_a, lengths=None, state_in=None):
    """o (B, T, H, d_v) and the final states (B, H, d_k, d_v); zeros past a row's length."""
    B, T, G, _ = q.shape
    H = v.shape[2]
    q, k = (x.repeat_interleave(H // G, 2) for x in (q, k))
    g = torch.exp(log_a.clamp(-1000.0, 0.0))[None, :, None, None]
    S = torch.zeros(B, H, q.shape[3], v.shape[3], dtype=q.dtype) if state_in is None else state_in
    n = torch.full((B,), T) if lengths is None else lengths.long().clamp(0, T)
    out = []
    for t in range(T):
        on = (t < n)[:, None, None, None]
        kv = k[:, t, :, :, None] * v[:, t, :, None, :]
        S = torch.where(on, g * S + torch.where(on, kv, torch.zeros_like(kv)), S)
        o = (q[:, t, :, :, None] * S).sum(-2)
        out.append(torch.where(on[..., 0], o, torch.zeros_like(o)))
    return torch.stack(out, 1), S


ACT = {"identity": lambda x: x, "silu": lambda x: x * torch.sigmoid(x), "sigmoid": torch.sigmoid}


def rms(x, group, eps):
    z = x.reshape(*x.shape[:-1], -1, group)
    return (z * torch.rsqrt(z.square().mean(-1, keepdim=True) + eps)).reshape(x.shape)


def block(y, w_post, x, gate, scale, group, act, eps):
    """x' of the block norm."""
    m = rms(y, group or y.shape[-1], eps)
    if w_post is not None:
        m = m * w_post
    if gate is not None:
        m = m * ACT[act](gate)
    if scale is not None:
        m = m * scale
    return m if x is None else x + m


def rel(got, want):
    got, want = got.double().cpu(), want.double()
    assert torch.isfinite(got).all()
    n = float(want.norm())
    return float((got - want).norm()) / n if n else float((got - want).norm())
