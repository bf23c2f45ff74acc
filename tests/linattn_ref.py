"""Linear attention with a decay for each head in 64 bits, token after token, and the sums of
absolute values that bound the rounding of any order of evaluation."""
from __future__ import annotations

import torch


def recurrence(q, k, v, g, start, scale):
    """One sequence: q, k [T][G][N], v [T][H][P], g [T][H] or None, start [H][P][N].  Returns o,
    the last state, and for both the same recurrence on absolute values."""
    T, H = v.shape[:2]
    share = H // q.shape[1]
    q, k = (x.double().repeat_interleave(share, 1) for x in (q, k))
    v, s = v.double(), start.double().clone()
    mag = s.abs()
    o, om = torch.zeros(v.shape, dtype=torch.float64), torch.zeros(v.shape, dtype=torch.float64)
    for t in range(T):
        lam = torch.ones(H, 1, 1, dtype=torch.float64) if g is None else g[t].double().exp()[:, None, None]
        write = v[t][:, :, None] * k[t][:, None, :]
        s = torch.where(lam == 0, 0.0, lam * s) + write
        mag = torch.where(lam == 0, 0.0, lam * mag) + write.abs()
        o[t] = scale * (s * q[t][:, None, :]).sum(-1)
        om[t] = abs(scale) * (mag * q[t].abs()[:, None, :]).sum(-1)
    return o, s, om, mag


def inputs(gen, tokens, H, G, P, dtype, N=128):
    """q, k, v, g of the distributions a layer sees: heads of strong, moderate and weak decay in turn."""
    q, k = (torch.randn(tokens, G, N, generator=gen) / N ** 0.5 for _ in range(2))
    v = torch.randn(tokens, H, P, generator=gen)
    band = torch.tensor((0.325, 0.0325, 0.00325)).repeat(H)[:H]
    g = -(torch.randn(tokens, H, generator=gen) * 0.7).exp() * band
    return q.to(dtype), k.to(dtype), v.to(dtype), g
