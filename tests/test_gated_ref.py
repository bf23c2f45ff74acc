"""The gated recurrence's 64-bit reference against differences and torch's differentiation (CPU)."""
import itertools

import pytest
import torch

from tests import gated_ref as ref


@pytest.mark.parametrize("gate,input", itertools.product((0, 1), (0, 1, 2)))
def test_gradient_against_differences(gate, input):
    gen = torch.Generator().manual_seed(3 * gate + input)
    T, C = 9, 7
    x, g = (t.double() for t in ref.inputs(gen, T, C, torch.float64, gate))
    do, dlast, start = (torch.randn(*s, generator=gen, dtype=torch.float64) for s in ((T, C), (C,), (C,)))

    def loss(x, g, start):
        h = ref.scan(x, g, start, gate, input)[0]
        return float((h[1:] * do).sum() + (h[-1] * dlast).sum())

    grads, _ = ref.gradient(x, g, do, dlast, start, gate, input)
    for i, (t, grad) in enumerate(zip((x, g, start), grads)):
        way = torch.randn(t.shape, generator=gen, dtype=torch.float64)
        step = 1e-6 * (g.abs() if t is g and gate == 0 else 1.0)  # log gates stay below zero
        up, down = ([x, g, start], [x, g, start])
        up[i], down[i] = t + step * way, t - step * way
        slope = (loss(*up) - loss(*down)) / 2e-6
        want = float((grad * way * (step / 1e-6)).sum())
        # the quotient's own error: 1e-12 of the third derivative's size and 2^-52 of the loss over the step
        assert abs(slope - want) <= 1e-7 * (1 + float((grad * way).abs().sum())), (i, slope, want)


@pytest.mark.parametrize("gate,input", itertools.product((0, 1), (0, 1, 2)))
def test_gradient_against_differentiation(gate, input):
    gen = torch.Generator().manual_seed(10 + 3 * gate + input)
    T, C = 21, 5
    x, g = (t.double().requires_grad_() for t in ref.inputs(gen, T, C, torch.float64, gate))
    do, dlast = torch.randn(T, C, generator=gen, dtype=torch.float64), torch.randn(C, generator=gen, dtype=torch.float64)
    start = torch.randn(C, generator=gen, dtype=torch.float64).requires_grad_()
    a = g.exp() if gate == 0 else torch.sigmoid(g)
    s = (torch.ones_like(a), 1 - a, (1 - a * a).sqrt())[input]
    h, total = start, 0.0
    for t in range(T):
        h = a[t] * h + s[t] * x[t]
        total = total + (h * do[t]).sum()
    want = torch.autograd.grad(total + (h * dlast).sum(), (x, g, start))
    got, _ = ref.gradient(x.detach(), g.detach(), do, dlast, start.detach(), gate, input)
    for w, v in zip(want, got):
        torch.testing.assert_close(v, w, rtol=1e-9, atol=1e-10)
