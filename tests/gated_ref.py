"""The gated recurrence and its gradient in 64 bits, token after token, with first-order bounds of
what fp32 evaluation of the same formulas may be off by.

u = 2^-24 is half a step of fp32.  A decay is an exponential of a rounded product, off by
(2|g| + 4)u of itself; a sigmoid adds a sum, a reciprocal and a product, (2|g| + 8)u.  The factor on
the input comes from a polynomial, 3.3u of itself as it is evaluated, or from g = -1/2 (for a^2: -1/4) on from a
difference that is at least 0.39 of its larger side, ((2|g| + 4)a + 1)u / (1 - a) <= 8.7u, half of 17u with the
root and 2u of its own: 10u and less.  Every token then adds a rounding of the product and of the sum, and an evaluation in
pieces one more of each piece's decay: the state's error runs through the same recurrence,
  E_t = a E_(t-1) + u ((2|g| + 12) a M_(t-1) + 14 |s x| + 3 M_t),  M the recurrence on absolute values,
which holds for any grouping of the products.  The gradient's recurrence is the same one backwards.

A decay below 2^-126 = 1.2e-38, the smallest normal number of fp32 (exp(-90) = 8e-40), may become zero, as the
exponential does not return subnormal numbers: every decay and slope is off by FLUSH = 2^-126 besides, times what it multiplies.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
FLUSH = 2.0 ** -126
LOG, SIGMOID = 0, 1
PLAIN, COMPLEMENT, NORM = 0, 1, 2


def gates(g, gate, input):
    """a, s and their derivatives along g, in 64 bits."""
    g = g.double()
    if gate == LOG:
        a, rest, both = g.exp(), -torch.expm1(g), -torch.expm1(2 * g)
        da = a
    else:
        a, rest = torch.sigmoid(g), torch.sigmoid(-g)
        both, da = rest * (1 + a), a * rest
    if input == PLAIN:
        return a, torch.ones_like(a), da, torch.zeros_like(a)
    if input == COMPLEMENT:
        return a, rest, da, -da
    s = both.clamp(min=0).sqrt()
    return a, s, da, torch.where(s > 0, -a * da / torch.where(s > 0, s, 1.0), 0.0)


def _reach(g):
    """2|g| + 12, nothing where the decay is zero anyway."""
    g = g.double().abs()
    return torch.where(g > 200, 0.0, 2 * g + 12)


def scan(x, g, start, gate, input):
    """One sequence [T][C] from start [C]: the states [T + 1][C] (the first is start) and their bounds."""
    T = x.shape[0]
    a, s, _, _ = gates(g, gate, input)
    write = s * x.double()
    h, m, e = (torch.zeros(T + 1, x.shape[1], dtype=torch.float64) for _ in range(3))
    h[0], m[0] = start.double(), start.double().abs()
    reach = _reach(g) * a
    for t in range(T):
        h[t + 1] = a[t] * h[t] + write[t]
        m[t + 1] = a[t] * m[t] + write[t].abs()
        e[t + 1] = a[t] * e[t] + FLUSH * m[t] + U * (reach[t] * m[t] + 14 * write[t].abs() + 3 * m[t + 1])
    return h, m, e


def gradient(x, g, do, dlast, start, gate, input):
    """(dx, dg, dfirst) and their bounds, of one sequence."""
    T = x.shape[0]
    a, s, da, ds = gates(g, gate, input)
    h, m, e = scan(x, g, start, gate, input)
    x, do = x.double(), do.double()
    d, dm, de = dlast.double().clone(), dlast.double().abs(), torch.zeros_like(dlast, dtype=torch.float64)
    dx, dg, ex, eg = (torch.zeros_like(x) for _ in range(4))
    reach = _reach(g)
    for t in reversed(range(T)):
        d, dm = d + do[t], dm + do[t].abs()
        de = de + 3 * U * dm
        dx[t], ex[t] = s[t] * d, s[t] * (de + 12 * U * dm)
        slope = da[t] * h[t] + ds[t] * x[t]
        size = da[t].abs() * m[t] + ds[t].abs() * x[t].abs()
        dg[t] = d * slope
        eg[t] = de * size + dm * (da[t].abs() * e[t] + U * (2 * reach[t] + 30) * size + FLUSH * (m[t] + x[t].abs()))
        d, dm, de = a[t] * d, a[t] * dm, a[t] * de + (U * (reach[t] * a[t] + a[t]) + FLUSH) * dm
    return (dx, dg, d), (ex, eg, de)


def inputs(gen, tokens, channels, dtype, gate):
    """x and g of the distributions a layer sees: channels of strong, moderate and weak decay in turn."""
    x = torch.randn(tokens, channels, generator=gen).to(dtype)
    if gate == LOG:
        band = torch.tensor((0.325, 0.0325, 0.00325)).repeat(channels)[:channels]
        g = -(torch.randn(tokens, channels, generator=gen) * 0.7).exp() * band
    else:
        g = torch.randn(tokens, channels, generator=gen) * 1.5 + torch.linspace(0, 6, channels)
    return x, g.to(dtype)


def rounding(dtype, value):
    """Half a step of the type, and of its smallest numbers."""
    if dtype == torch.float32:
        return 1e-37
    return torch.finfo(dtype).eps / 2 * value.abs() + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
