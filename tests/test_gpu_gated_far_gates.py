"""GPU: sigmoid gates where the decay is near and below fp32's smallest normal number, 2^-126 = sigmoid(-87.34), and where
exp(-g) passes fp32's largest, at -88.72: the decay may be zero there, what remains for the input is one.

Tolerances: the reference's own bounds (tests/gated_ref.py), which let a decay be off by 2^-126 and the factor on the input
by 14 * 2^-24 of itself, and half a step of the outputs' type.  From g = 87.34 on it is 1 - a that is below 2^-126, and
the interface lets it, and 1 - a^2, be zero: FLUSHED below."""
import sys

import pytest
import torch

from tests import gated_ref as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mamba_decode_amd as ssq
    from tests.test_gpu_gated import case, check, cu_of, state_of, values_of

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
# around 2^-126, inside the interval, around the overflow, behind it; and around exp(-g) = 2^24, where 1 - a rounds to 1
FAR = (-87.0, -87.25, -87.3125, -87.375, -87.5, -88.0, -88.5, -88.6875, -88.75, -89.0, -104.0, -16.5, -16.625, -16.75, -17.5, 87.5, 88.5, 104.0)


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def far(g, gen):
    pick = torch.randint(0, len(FAR) + 6, g.shape, generator=gen)
    for i, v in enumerate(FAR):
        g = torch.where(pick == i, torch.tensor(v).to(g.dtype), g)
    return g.contiguous()


def flushed(g, input):
    """What the factor on the input and its slope are off by where 1 - a is below 2^-126 and taken as zero.

    An exponential below 2^-126 is zero, and with it 1 - a = e a.  COMPLEMENT: the factor is 1 - a itself, off by less than
    2^-126.  NORM: the factor is sqrt((1 - a)(1 + a)) < sqrt(2 * 2^-126) = 2^-62.5, and its slope a^2 s / (1 + a) <= s / 2,
    as a <= 1.  Where 1 - a is 2^-126 or more, so is 1 - a^2 = (1 - a)(1 + a), and nothing is flushed.  The border and the
    bounds are 1.001 times as far, as the exponential is off by (2 * 87.4 + 4) * 2^-24 = 1.07e-5 of itself."""
    there = torch.sigmoid(-g.double()) < 1.001 * ref.FLUSH
    most = {0: 0.0, 1: 1.001 * ref.FLUSH, 2: 1.001 * 2.0 ** -62.5}[input]
    return torch.where(there, most, 0.0)


@pytest.fixture
def with_flushed(monkeypatch):
    """The reference's bounds with FLUSHED carried on by the same recurrences."""
    plain_scan, plain_gradient = ref.scan, ref.gradient

    def scan(x, g, start, gate, input):
        h, m, e = plain_scan(x, g, start, gate, input)
        a, off = ref.gates(g, gate, input)[0], flushed(g, input) * x.double().abs()
        more = torch.zeros_like(e)
        for t in range(x.shape[0]):
            more[t + 1] = a[t] * more[t] + off[t]
        return h, m, e + more

    def gradient(x, g, do, dlast, start, gate, input):
        values, (ex, eg, de) = plain_gradient(x, g, do, dlast, start, gate, input)  # its scan is the one above
        a, off = ref.gates(g, gate, input)[0], flushed(g, input)
        dm = dlast.double().abs()
        for t in reversed(range(x.shape[0])):
            dm = dm + do[t].double().abs()
            ex[t] += off[t] * dm
            eg[t] += off[t] * dm * x[t].double().abs()
            dm = a[t] * dm
        return values, (ex, eg, de)

    monkeypatch.setattr(ref, "scan", scan)
    monkeypatch.setattr(ref, "gradient", gradient)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("input", [0, 1, 2])
@pytest.mark.parametrize("channels,lens", [(40, [130, 65]), (2600, [35, 0, 20]), (72, [2300])])
def test_scan_and_gradient(with_flushed, dtype, input, channels, lens):
    say("far", dtype, input, channels, lens)
    case(dtype, 1, input, channels, lens, gates=far, seed=input + channels)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("input", [0, 1, 2])
def test_tokens(with_flushed, dtype, input):
    say("far token", dtype, input)
    gen = torch.Generator().manual_seed(60 + input)
    n, C = 4, 264
    x, g = ref.inputs(gen, n, C, dtype, 1)
    g = far(g, gen)
    start = torch.randn(n, C, generator=gen)
    st, o = state_of(start), torch.zeros_like(x).cuda()
    ssq.ssq_gated_step(st, x.cuda(), g.cuda(), o, gate=1, input=input)
    state = values_of(st)
    for i in range(n):
        h, m, e = ref.scan(x[i:i + 1], g[i:i + 1], start[i], 1, input)
        check(o[i:i + 1], h[1:], e[1:], dtype, ("o", i))
        check(state[i][None], h[1:], e[1:], F32, ("state", i))


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("input", [1, 2])
def test_a_forgotten_state_leaves_the_input(dtype, input):
    """Gates of -87.5 to -89: every output is its input and every gradient its output's, to a last step of the factor."""
    say("far, all of them", dtype, input)
    gen = torch.Generator().manual_seed(70 + input)
    T, C = 50, 64
    x, do = (torch.randn(T, C, generator=gen).to(dtype).cuda() for _ in range(2))
    g = torch.tensor((-87.5, -88.0, -88.5, -89.0)).repeat(T * C // 4).view(T, C).to(dtype).cuda()
    o, dx, dg = (torch.zeros_like(x) for _ in range(3))
    ck = torch.empty(ssq.ssq_gated_checkpoint_rows(1, T), C, device="cuda")
    ssq.ssq_gated_scan(None, x, g, o, cu_of([T]), gate=1, input=input, checkpoints=ck)
    ssq.ssq_gated_scan_backward(ck, x, g, do, dx, dg, cu_of([T]), gate=1, input=input)
    # the factor is one to 14 * 2^-24 of itself; nothing but it and a rounding stands between
    eps = 14 * 2.0 ** -24 + (0 if dtype == F32 else torch.finfo(dtype).eps / 2)
    for got, want in ((o, x), (dx, do)):
        assert ((got.double() - want.double()).abs() <= eps * want.double().abs()).all()
