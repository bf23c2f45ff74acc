"""GPU: how exact linear attention on prompts is, beyond what its other tests ask.

Bounds, each relative to the sum of the absolute values of a result's terms, which the reference
computes beside it.  A product's operand that stands as two bf16 terms is off by 2^-16: 2^-8 of it is
left by the first rounding, and 2^-8 of that by the second.  An output meets that three times at
most: the decayed scores as v meets them or the state as q reads it, and what a part of a split
sequence writes into its own state.  Sums and decays are fp32 or wider, by ``sum_bound``.  The
output is rounded once to its type, half a step of the value."""
import math
import sys

import pytest
import torch

from tests import linattn_ref as ref
from tests.test_gpu_linattn import BF, F32, HF, cu_of, state_of, sum_bound, values_of

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mamba_decode_amd as ssq


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def run(q, k, v, g, lens, G, start, scale):
    st = state_of(start, G)
    o = torch.zeros_like(v).cuda()
    ssq.ssq_linattn_prefill(st, q.cuda(), k.cuda(), v.cuda(), g.cuda(), o, cu_of(lens), scale=scale)
    o, state, at, want = o.cpu(), values_of(st), 0, []
    for i, n in enumerate(lens):
        want.append(ref.recurrence(*(x[at:at + n] for x in (q, k, v, g)), start[i], scale))
        at += n
    return o, state, want


def check_rounded_once(o, wo, om, T, where, pairs=3):
    tol = om * (pairs * 2.0 ** -16 + sum_bound(T)) * 1.01 + wo.abs() * (torch.finfo(o.dtype).eps / 2) + torch.finfo(o.dtype).tiny
    off = (o.double() - wo).abs() / tol
    assert (off <= 1).all(), f"{where}: {int((off > 1).sum())} of {off.numel()} outputs off, the worst {off.max():.1f} times its bound"


@pytest.mark.parametrize("H,G,P,lens", [(24, 1, 64, [300, 77]), (2, 2, 128, [2000]), (40, 4, 48, [64, 130, 1, 65, 200, 90, 16]),
                                        (1, 1, 16, [1000, 33])])
def test_outputs_of_bf16_prompts_are_rounded_once(H, G, P, lens):
    """Scores that meet v in bf16 alone are off by 2^-8 each, many steps of an output whose terms cancel."""
    say("rounded once", H, G, P, lens)
    gen = torch.Generator().manual_seed(H + P)
    q, k, v, g = ref.inputs(gen, sum(lens), H, G, P, BF)
    o, _, want = run(q, k, v, g, lens, G, torch.randn(len(lens), H, P, 128, generator=gen), 0.3)
    at, off, once, norm = 0, 0.0, 0.0, 0.0
    for n, (wo, _, om, _) in zip(lens, want):
        check_rounded_once(o[at:at + n], wo, om, n, f"{n} tokens")
        off += (o[at:at + n].double() - wo).square().sum().item()
        once += (wo.to(BF).double() - wo).square().sum().item()
        norm += wo.square().sum().item()
        at += n
    # what comes before the rounding adds to it in squares: 2^-16 of terms whose sum of absolute values is some
    # 10 times the result, against 2^-9.2 of the result itself, is less than 1% of it
    say(f"  off by {math.sqrt(off / norm):.6f}, one rounding {math.sqrt(once / norm):.6f}")
    assert math.sqrt(off) <= 1.02 * math.sqrt(once)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("T", [16, 47, 300])
def test_decays_behind_tokens_that_forget(dtype, T):
    """A decay between two tokens is the difference of two sums of log decays.  Behind 13 tokens that
    forget all (e^-128 is 0) these are some -2400 in powers of two: rounded to fp32 each is off by up
    to 2^-13, and the decay by as much of itself, where 2^-22 is asked.  Of the three tokens that
    follow each writes the opposite of the one before it, so that an output is little but the
    difference of their decays.  Nothing comes through a state: scores alone stand as two terms."""
    say("behind tokens that forget", dtype, T)
    gen = torch.Generator().manual_seed(T)
    H, G, P = 12, 2, 64
    q, _, v, _ = ref.inputs(gen, T, H, G, P, dtype)
    q[:] = q[:1]
    t = torch.arange(T)
    for i in (14, 15):
        v[t % 16 == i] = -v[t % 16 == i - 1][: int((t % 16 == i).sum())]
    g = -0.01 * torch.rand(T, H, generator=gen)
    g[t % 16 < 13] -= 150.0
    o, _, want = run(q, q, v, g, [T], G, torch.zeros(1, H, P, 128), 1.0)
    wo, _, om, _ = want[0]
    if dtype == F32:
        off = (o.double() - wo).abs() / (sum_bound(T) * om)
        assert (off <= 1).all(), f"the worst {off.max():.1f} times its bound"
    else:
        check_rounded_once(o, wo, om, T, "behind tokens that forget", pairs=1)


def off_by(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("H,G,P,T", [(24, 1, 64, 700), (3, 1, 32, 2000), (60, 4, 64, 320)])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_norms(dtype, H, G, P, T):
    """Errors of many roundings, in the 2-norm.  A chain of n fp32 additions is off by 2^-24 * sqrt(n/3)
    of its running value; a state takes some 8 a chunk, whose weights its decay bounds to the last
    hundred or so, a score or S q 32, an output twice that: 2e-7 for 40, 3e-7 for 80, and twice it
    taken.  A state that is written as two bf16 terms would be off by 2.6e-6 (the rms of a rounding
    to bf16 is 0.0016 of a value, and the second term's is that of 0.0023/1.4 of it)."""
    gen = torch.Generator().manual_seed(T)
    q, k, v, g = ref.inputs(gen, T, H, G, P, dtype)
    n = 5 if H == 60 else 1
    lens = [T // n] * n
    o, state, want = run(q, k, v, g, lens, G, torch.randn(n, H, P, 128, generator=gen), 0.3)
    ws, wo = torch.stack([w[1] for w in want]), torch.cat([w[0] for w in want])
    so, oo = off_by(state, ws), off_by(o, wo)
    say("norms", dtype, H, G, P, T, f"state {so:.2e}, o {oo:.2e}")
    assert so <= 4e-7
    if dtype == F32:
        assert oo <= 6e-7
    else:
        assert oo <= 1.02 * off_by(wo.to(dtype), wo)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("H,lens", [(3, [900, 1, 70]), (90, [65, 0, 130, 1]), (2, [5])])
def test_log_decays_in_a_wider_row(dtype, H, lens):
    """g as a slice of a wider tensor, whose other columns and rows behind the last sequence are NaN."""
    say("wide decays", dtype, H, lens)
    gen = torch.Generator().manual_seed(H)
    T, P = sum(lens), 16
    q, k, v, g = ref.inputs(gen, T, H, 1, P, dtype)
    start = torch.randn(len(lens), H, P, 128, generator=gen)
    want, same = run(q, k, v, g, lens, 1, start, 0.3)[:2]
    wide = torch.full((T + 9, H + 7), math.nan, device="cuda")
    wide[:T, 3:H + 3] = g.cuda()
    st, o = state_of(start, 1), torch.zeros_like(v).cuda()
    ssq.ssq_linattn_prefill(st, q.cuda(), k.cuda(), v.cuda(), wide[:T, 3:H + 3], o, cu_of(lens), scale=0.3)
    assert torch.equal(o.cpu(), want) and torch.equal(values_of(st), same)
