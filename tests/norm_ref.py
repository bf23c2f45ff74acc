"""The group norm with an activation and its gradient in 64 bits, with first-order bounds of what fp32
evaluation may be off by.

u = 2^-24 is half a step of fp32.  A sigmoid is off by (2|v| + 8)u of itself.  A sum over a group is off by K u
of the sum of absolute values, K = width/64 + 16 additions one after the other at most, whatever the lanes hold; a sum over
tokens by (tokens + 64)u of it.  Errors of what enters a formula are carried on by its derivatives.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
SILU, GATE_OUTPUT, GATE_INPUT = range(3)


def _swish(v):
    s = torch.sigmoid(v)
    slope = s * (1 + v * (1 - s))
    size = s * (1 + v.abs())
    return v * s, slope, (v * s).abs() * (2 * v.abs() + 10) * U, size * (2 * v.abs() + 14) * U


def norm(x, z, weight, bias, act, center, eps, dy=None):
    """x, z, dy [T][G][W], weight, bias [G][W] or None.  A dict of values and a dict of bounds."""
    T, _, W = x.shape
    K = W / 64 + 16
    x = x.double()
    one = torch.ones(x.shape[1:], dtype=torch.float64)
    w = one if weight is None else weight.double()
    b = 0 * one if bias is None else bias.double()
    mean = lambda v: v.mean(-1, keepdim=True)  # noqa: E731
    if z is not None:
        z = z.double()
        sz, slope_z, e_sz, e_slope_z = _swish(z)
    u, eu = x, torch.zeros_like(x)
    if act == GATE_INPUT:
        u = x * sz
        eu = x.abs() * e_sz + u.abs() * U
    c, ec = u, eu
    if center:
        c = u - mean(u)
        ec = eu + mean(eu) + K * U * mean(u.abs()) + U * c.abs()
    var = mean(c * c)
    r = (var + eps).rsqrt()
    er = r * (0.5 * (2 * mean(c.abs() * ec) + K * U * var) / (var + eps) + 4 * U)
    m, em = c * r, ec * r + c.abs() * er + U * (c * r).abs()
    n = m * w + b
    en = w.abs() * em + 2 * U * (n.abs() + (m * w).abs())
    if act == SILU:
        y, slope_n, ey, e_slope_n = _swish(n)
        ey = ey + 1.1 * en
    elif act == GATE_OUTPUT:
        y, ey = n * sz, en * sz.abs() + n.abs() * e_sz + U * (n * sz).abs()
    else:
        y, ey = n, en
    out, err = dict(y=y), dict(y=ey)
    if dy is None:
        return out, err
    dy = dy.double()
    if act == SILU:
        dn, edn = dy * slope_n, dy.abs() * (e_slope_n + 0.5 * en)
    elif act == GATE_OUTPUT:
        dn, edn = dy * sz, dy.abs() * (e_sz + 2 * U * sz.abs())
        out["dz"] = dy * n * slope_z
        err["dz"] = dy.abs() * (en * slope_z.abs() + n.abs() * (e_slope_z + 3 * U * slope_z.abs()))
    else:
        dn, edn = dy, torch.zeros_like(dy)
    Kt = T + 64
    out["dweight"], err["dweight"] = (dn * m).sum(0), (edn * m.abs() + dn.abs() * em + Kt * U * (dn * m).abs()).sum(0)
    out["dbias"], err["dbias"] = dn.sum(0), (edn + Kt * U * dn.abs()).sum(0)
    dm, edm = dn * w, edn * w.abs() + U * (dn * w).abs()
    m2 = mean(dm * m)
    em2 = mean(edm * m.abs() + dm.abs() * em) + K * U * mean((dm * m).abs())
    m1, em1 = torch.zeros_like(m2), torch.zeros_like(m2)
    if center:
        m1, em1 = mean(dm), mean(edm) + K * U * mean(dm.abs())
    inner = dm - m1 - m * m2
    du = r * inner
    edu = er * inner.abs() + r * (edm + em1 + m.abs() * em2 + em * m2.abs() + 4 * U * (dm.abs() + m1.abs() + (m * m2).abs()))
    if act == GATE_INPUT:
        out["dx"], err["dx"] = du * sz, edu * sz.abs() + du.abs() * (e_sz + U * sz.abs())
        out["dz"] = du * x * slope_z
        err["dz"] = x.abs() * (edu * slope_z.abs() + du.abs() * (e_slope_z + 3 * U * slope_z.abs()))
    else:
        out["dx"], err["dx"] = du, edu
    return out, err
