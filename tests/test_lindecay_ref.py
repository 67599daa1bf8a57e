"""Pins of the plain forms that the kernels of the head-decay attention are tested against."""
import pytest
import torch

from lindecay_ref import lindecay, pairs


@pytest.mark.parametrize("T,G,H,lengths,state", [(1, 1, 1, None, False), (7, 2, 4, None, True), (33, 1, 3, [0, 33, 12], True),
                                                 (20, 2, 2, [20, 1, -3], False)])
def test_recurrence_and_pairs_agree(T, G, H, lengths, state):
    g = torch.Generator().manual_seed(T)
    B = 3
    draw = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    q, k, v = draw(B, T, G, 5), draw(B, T, G, 5), draw(B, T, H, 4)
    la = -torch.rand(H, generator=g, dtype=torch.float64)
    n = None if lengths is None else torch.tensor(lengths)
    s0 = draw(B, H, 5, 4) if state else None
    for a, b in zip(lindecay(q, k, v, la, n, s0), pairs(q, k, v, la, n, s0)):
        assert torch.allclose(a, b, rtol=1e-12, atol=1e-12)


def test_no_decay_is_a_running_sum():
    """log_a = 0: o_t = q_t . sum over s <= t of k_s v_s^T; log_a = -inf: only s = t."""
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn((1, 9, 2, 3), generator=g, dtype=torch.float64) for _ in range(3))
    run = torch.cumsum(k[..., :, None] * v[..., None, :], 1)
    o, st = lindecay(q, k, v, torch.zeros(2, dtype=torch.float64))
    assert torch.allclose(o, (q[..., None] * run).sum(-2)) and torch.allclose(st, run[:, -1])
    o, _ = lindecay(q, k, v, torch.full((2,), float("-inf"), dtype=torch.float64))
    assert torch.allclose(o, (q * k).sum(-1, keepdim=True) * v)
