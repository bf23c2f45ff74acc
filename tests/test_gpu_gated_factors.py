"""GPU: the factor on the input by itself, read out by single tokens of ones on states of zeros, against expm1 and the sigmoid
in 64 bits; and gates of a norm whose sigmoid is below fp32's smallest normal number.

u = 2^-24 is half a step of fp32.  The hardware's exponential, reciprocal and root are off by a step, 2u, a product or sum by u.
exp(x) of a rounded product is off by |x| u for the product, a quarter of it for the constant log2(e), and 2u: (2|x| + 4)u.
  log, 1 - a:       for g > -1/2 a polynomial fitted to 1.8u of itself, 3.3u as it is evaluated (4u here); below, a difference of one
                    and a: ((2|g| + 4) a + 1)u / (1 - a)
  log, norm:        the same of 1 - a a for g > -1/4, else ((2 (2|g| + 4) + 1) a^2 + 1)u / (1 - a^2); half of it through the root, 2u
                    of its own
  sigmoid, 1 - a:   e / (1 + e), e = exp(-g): what e is off by counts 1 / (1 + e) times, sum, reciprocal and product 4u; one
                    from e = 2^24 on, which is u off; an exponential below 2^-126 is zero
  sigmoid, norm:    half of what 1 - a, 1 + a and their product are off by, 2u of the root; where 1 - a is zero, 2^-62.5"""
import sys

import pytest
import torch

from tests import norm_ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mamba_decode_amd as ssq
    from tests.test_gpu_gated import state_of

U, FLUSH = 2.0 ** -24, 2.0 ** -126


def exact(g, gate, input):
    """The factor in 64 bits, and what it may be off by."""
    far = 2 * g.abs() + 4
    if gate == 0:
        y = g if input == 1 else 2 * g
        rest, kept = -torch.expm1(y), y.exp()
        off = torch.where(y > -0.5, 4.0, ((far if input == 1 else 2 * far + 1) * kept + 1) / rest) * U
        return (rest, off * rest) if input == 1 else (rest.sqrt(), (off / 2 + 2 * U) * rest.sqrt())
    a, rest = torch.sigmoid(g), torch.sigmoid(-g)
    off = (far * a + 4) * U  # 1 / (1 + e) = a
    if input == 1:
        return rest, off * rest + FLUSH
    up = 1 + a
    s = (rest * up).sqrt()
    both = off + (a / up * (far * rest + 3) + 2) * U
    return s, (both / 2 + 2 * U) * s + torch.where(rest < 1.001 * FLUSH, 2.0 ** -62.5, 0.0)


@pytest.mark.parametrize("gate,input", [(0, 1), (0, 2), (1, 1), (1, 2)])
def test_factor_on_the_input(gate, input):
    print("factor", gate, input, file=sys.stderr, flush=True)
    gen = torch.Generator().manual_seed(gate * 2 + input)
    n, C = 64, 4096
    size = torch.exp(torch.empty(n, C, dtype=torch.float64).uniform_(-14.0, 4.8, generator=gen)).float()  # 1e-6 to 120
    size[0] = torch.linspace(0.2, 0.6, C)
    size[1] = torch.linspace(16.0, 18.0, C)
    size[2] = torch.linspace(86.5, 89.5, C)
    g = -size if gate == 0 else torch.where(torch.rand(n, C, generator=gen) < 0.5, size, -size)
    st, x, o = state_of(torch.zeros(n, C)), torch.ones(n, C, device="cuda"), torch.zeros(n, C, device="cuda")
    ssq.ssq_gated_step(st, x, g.cuda(), o, gate=gate, input=input)
    want, off = exact(g.double(), gate, input)
    bad = ~((o.cpu().double() - want).abs() <= 1.001 * off)  # first order
    assert not bad.any(), (int(bad.sum()), g[bad][:4].tolist(), o.cpu()[bad][:4].tolist(), want[bad][:4].tolist())


@pytest.mark.parametrize("act", [1, 2])
def test_far_gates_of_a_norm(act):
    """z of -80 to -104: its sigmoid may be zero below 2^-126, so silu(z) is off by |z| 2^-126 besides what norm_ref bounds."""
    print("far gates of a norm", act, file=sys.stderr, flush=True)
    gen = torch.Generator().manual_seed(act)
    shape = (50, 2, 264)
    x = torch.randn(shape, generator=gen)
    z = torch.empty(shape).uniform_(-104.0, -80.0, generator=gen)
    if act == 2:  # groups of such gates alone would be zero beside eps
        z[..., ::3] = torch.randn(shape, generator=gen)[..., ::3]
    y = torch.zeros(shape, device="cuda")
    ssq.ssq_group_norm(x.cuda(), y, z=z.cuda(), act=act)
    want, bound = norm_ref.norm(x, z, None, None, act, True, 1e-5)
    flushed = 1.001 * FLUSH * z.double().abs() * (z < -87.3)
    if act == 1:
        c = x.double() - x.double().mean(-1, keepdim=True)
        n = c * (c.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
        more = flushed * n.abs() * 1.001
    else:  # u moves by x times as much, its mean and its deviation with it, r <= 1 / sqrt(1e-5) = 317 times each
        more = 317 * 4 * (flushed * x.double().abs()).amax(-1, keepdim=True)
    assert ((y.cpu().double() - want["y"]).abs() <= bound["y"] + more).all()
