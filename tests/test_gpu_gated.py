"""GPU: the gated recurrence, its gradient and its single token against the recurrence in 64 bits.

Tolerances: the reference's own bounds of fp32 evaluation (tests/gated_ref.py) and half a step of the outputs' type."""
import itertools
import sys

import numpy as np
import pytest
import torch

from tests import gated_ref as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mamba_decode_amd as ssq

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
SENTINEL = 7.0
MODES = list(itertools.product((0, 1), (0, 1, 2)))


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def state_of(values):
    B, C = values.shape
    desc = ssq.make_desc(ssq.SSQ_GATED, "fp32", B, 1, 1, C)
    storage = torch.zeros(ssq.ssq_state_bytes(desc), dtype=torch.uint8, device="cuda")
    return ssq.ssq_alloc_state(desc, storage, values.float().cuda().contiguous())


def values_of(state):
    out = torch.empty(state.desc.batch, state.desc.row_len, device="cuda")
    ssq.ssq_dequant(state, out)
    return out.cpu()


def cu_of(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")


def check(got, want, bound, dtype, where):
    tol = bound + ref.rounding(dtype, want.abs() + bound)
    bad = ~((got.cpu().double() - want).abs() <= tol)
    assert not bad.any(), f"{where}: off at {bad.nonzero()[:4].tolist()}, {int(bad.sum())} of {bad.numel()}"


def sliced(t, at=8, wide=24):
    """The same values as a slice of wider rows."""
    if t is None:
        return None
    big = torch.full((t.shape[0], t.shape[1] + wide), SENTINEL, dtype=t.dtype, device="cuda")
    big[:, at:at + t.shape[1]] = t
    return big[:, at:at + t.shape[1]]


def case(dtype, gate, input, channels, lens, tail=0, slots=None, fresh=None, batch=None, slices=False, seed=0, gates=None,
         stateless=False, backward=True):
    gen = torch.Generator().manual_seed(seed)
    n, T = len(lens), sum(lens) + tail
    x, g = ref.inputs(gen, T, channels, dtype, gate)
    if gates is not None:
        g = gates(g, gen)
    batch = batch or max(n, 1)
    start = torch.randn(batch, channels, generator=gen)
    do, dlast = torch.randn(T, channels, generator=gen).to(dtype), torch.randn(n, channels, generator=gen)
    st = None if stateless else state_of(start)
    slot_t = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
    fresh_t = None if fresh is None else torch.tensor(fresh, dtype=torch.uint8, device="cuda")
    place = sliced if slices else (lambda t: t.cuda())
    dev = [place(t) for t in (x, g, do)]
    o, dx, dg = (place(torch.full_like(x, SENTINEL)) for _ in range(3))
    ck = torch.full((ssq.ssq_gated_checkpoint_rows(n, T), channels), SENTINEL, device="cuda")
    dfirst = torch.full((n, channels), SENTINEL, device="cuda")
    cu = cu_of(lens)
    how = dict(gate=gate, input=input, slots=slot_t)
    ssq.ssq_gated_scan(st, dev[0], dev[1], o, cu, fresh=fresh_t, checkpoints=ck if backward else None, **how)
    if backward:
        ssq.ssq_gated_scan_backward(ck, dev[0], dev[1], dev[2], dx, dg, cu, dlast=dlast.cuda(), dfirst=dfirst, state=st, **how)
    torch.cuda.synchronize()
    o, dx, dg, dfirst, ck = (t.cpu() for t in (o, dx, dg, dfirst, ck))
    state = None if stateless else values_of(st)
    named, at, rows = set(), 0, set()
    for i, L in enumerate(lens):
        slot = i if slots is None else slots[i]
        s = slice(at, at + L)
        where = (dtype, gate, input, channels, lens, i)
        if not stateless and not 0 <= slot < batch:  # left out
            for t in (o, dx, dg):
                assert (t[s] == SENTINEL).all(), where
            assert (dfirst[i] == SENTINEL).all()
            at += L
            continue
        zero = stateless or (fresh is not None and fresh[i])
        h0 = torch.zeros(channels) if zero else start[slot]
        h, m, e = ref.scan(x[s], g[s], h0, gate, input)
        check(o[s], h[1:], e[1:], dtype, ("o", where))
        if not stateless:
            named.add(slot)
            check(state[slot][None], h[-1:], e[-1:], F32, ("state", where))
        if backward:
            first = at // 16 + i
            chunks = (L + 15) // 16
            check(ck[first:first + chunks], h[:L:16], e[:L:16], F32, ("checkpoints", where))
            rows |= set(range(first, first + chunks))
            grads, bounds = ref.gradient(x[s], g[s], do[s], dlast[i], h0, gate, input)
            check(dx[s], grads[0], bounds[0], dtype, ("dx", where))
            check(dg[s], grads[1], bounds[1], dtype, ("dg", where))
            check(dfirst[i], grads[2], bounds[2], F32, ("dfirst", where))
        at += L
    if T > at:
        assert (o[at:] == SENTINEL).all() and (dx[at:] == SENTINEL).all() and (dg[at:] == SENTINEL).all()
    for r in set(range(ck.shape[0])) - rows:
        assert (ck[r] == SENTINEL).all(), r
    if not stateless:
        for b in set(range(batch)) - named:
            assert torch.equal(state[b], start[b]), b


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("gate,input", MODES)
def test_modes(dtype, gate, input):
    say("modes", dtype, gate, input)
    case(dtype, gate, input, 200, [300, 0, 1, 77], tail=5, seed=gate * 3 + input, fresh=[0, 1, 0, 1])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("channels", [8, 16, 24, 40, 64, 128, 136, 264, 520, 1544])
@pytest.mark.parametrize("lens", [[1], [15], [16], [17], [0], [33, 0, 64, 1, 31], [513]])
def test_sizes(dtype, channels, lens):
    say("sizes", dtype, channels, lens)
    case(dtype, 0, 2, channels, lens, tail=len(lens), seed=channels)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("lens", [[2049], [1500, 3, 700, 0, 129, 64], [5000], [4100, 1], [40] * 40])
def test_lengths(dtype, lens):
    say("lengths", dtype, lens)
    case(dtype, 1, 1, 72, lens, tail=3, seed=len(lens))
    case(dtype, 0, 0, 72, lens, seed=len(lens), stateless=True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("slots,fresh", [([3, 0, 4], None), ([4, -1, 0], [0, 1, 1]), ([5, 2, 7], [1, 0, 0])])
def test_slots(dtype, slots, fresh):
    say("slots", dtype, slots)
    for gate, input in ((0, 1), (1, 2)):
        case(dtype, gate, input, 136, [50, 200, 16], slots=slots, fresh=fresh, batch=5, seed=7, slices=True)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("gate,input", MODES)
def test_gates_that_forget_and_keep(dtype, gate, input):
    """-infinity, the type's lowest value and large ones forget; zero (log) or +infinity (sigmoid) keep everything."""
    say("forget", dtype, gate, input)

    def gates(g, gen):
        pick = torch.randint(0, 24, g.shape, generator=gen)
        for i, v in enumerate((-torch.inf, torch.finfo(dtype).min, -90.0, 0.0 if gate == 0 else torch.inf, -0.0, -1e-4, -0.5, -0.25)):
            g = torch.where(pick == i, torch.tensor(v, dtype=dtype), g)
        return g.contiguous()

    case(dtype, gate, input, 40, [130, 65], gates=gates, seed=gate * 3 + input + 50)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("gate,input", MODES)
def test_tokens(dtype, gate, input):
    say("step", dtype, gate, input)
    gen = torch.Generator().manual_seed(gate * 3 + input)
    for channels, slots, batch in ((8, None, 1), (200, [2, 0, 5, -1, 6, 1], 6), (2056, None, 3)):
        n = batch if slots is None else len(slots)
        x, g = ref.inputs(gen, n, channels, dtype, gate)
        start = torch.randn(batch, channels, generator=gen)
        st, o = state_of(start), sliced(torch.full_like(x, SENTINEL))
        slot_t = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
        ssq.ssq_gated_step(st, sliced(x), sliced(g), o, gate=gate, input=input, slots=slot_t)
        o, state = o.cpu(), values_of(st)
        for i in range(n):
            slot = i if slots is None else slots[i]
            if not 0 <= slot < batch:
                assert (o[i] == SENTINEL).all()
                continue
            h, m, e = ref.scan(x[i:i + 1], g[i:i + 1], start[slot], gate, input)
            check(o[i:i + 1], h[1:], e[1:], dtype, ("o", channels, i))
            check(state[slot][None], h[1:], e[1:], F32, ("state", channels, i))
        for b in set(range(batch)) - set(range(n) if slots is None else slots):
            assert torch.equal(state[b], start[b])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_prompt_and_tokens_are_one_sequence(dtype):
    """A prompt in one call, in two calls that go on from the state, and token after token."""
    say("prompt and tokens", dtype)
    gen = torch.Generator().manual_seed(8)
    C, T = 264, 90
    x, g = ref.inputs(gen, T, C, dtype, 0)
    start = torch.randn(1, C, generator=gen)
    h, m, e = ref.scan(x, g, start[0], 0, 2)
    xd, gd = x.cuda(), g.cuda()
    for cuts in ([T], [40, 50], [17, 73], [1] * T):
        st, o = state_of(start), torch.zeros_like(xd)
        at = 0
        for n in cuts:
            s = slice(at, at + n)
            if n == 1:
                ssq.ssq_gated_step(st, xd[s], gd[s], o[s], input=2)
            else:
                ssq.ssq_gated_scan(st, xd[s], gd[s], o[s], cu_of([n]), input=2)
            at += n
        check(o, h[1:], e[1:], dtype, cuts[:2])
        check(values_of(st), h[-1:], e[-1:], F32, cuts[:2])


def test_offsets_are_clamped():
    say("clamped")
    gen = torch.Generator().manual_seed(11)
    C, T = 24, 40
    x, g = ref.inputs(gen, T, C, F32, 0)
    start = torch.randn(3, C, generator=gen)
    st, o = state_of(start), torch.full_like(x, SENTINEL).cuda()
    cu = torch.tensor([-5, 10, 4, 1 << 30], dtype=torch.int32, device="cuda")  # 0..10, none, 4..40
    ssq.ssq_gated_scan(st, x.cuda(), g.cuda(), o, cu)
    state = values_of(st)
    for i, (a, b) in enumerate(((0, 10), (10, 10), (4, 40))):
        h, m, e = ref.scan(x[a:b], g[a:b], start[i], 0, 0)
        check(state[i][None], h[-1:], e[-1:], F32, i)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_nothing_is_read_that_is_not_asked_for(dtype):
    """NaN around and between sequences, in the states of fresh and unnamed slots, in one sequence and in one channel."""
    say("NaN around", dtype)
    gen = torch.Generator().manual_seed(20)
    C, T = 72, 400
    x, g = (t.cuda() for t in ref.inputs(gen, T, C, dtype, 1))
    do = torch.randn(T, C, generator=gen).to(dtype).cuda()
    start = torch.randn(5, C, generator=gen)
    cu = torch.tensor([10, 100, 101, 330], dtype=torch.int32, device="cuda")
    slots = torch.tensor([2, 4, 0], dtype=torch.int32, device="cuda")
    fresh = torch.tensor([1, 0, 0], dtype=torch.uint8, device="cuda")
    results = []
    for dirty in (False, True):
        st = state_of(start)
        if dirty:
            for t in (x, g, do):
                t[:10] = t[330:] = t[100:101] = torch.nan
                t[150, 7] = torch.nan
            st.regions()[0][1:4] = torch.nan
        o, dx, dg = (torch.zeros_like(x) for _ in range(3))
        ck = torch.full((ssq.ssq_gated_checkpoint_rows(3, T), C), torch.nan, device="cuda")
        dfirst = torch.zeros(3, C, device="cuda")
        ssq.ssq_gated_scan(st, x, g, o, cu, gate=1, input=2, slots=slots, fresh=fresh, checkpoints=ck)
        ssq.ssq_gated_scan_backward(ck, x, g, do, dx, dg, cu, gate=1, input=2, dfirst=dfirst, state=st, slots=slots)
        results.append([t.cpu() for t in (o, dx, dg)] + [dfirst.cpu(), values_of(st)])
    keep = torch.ones(T, C, dtype=torch.bool)
    keep[100] = False
    keep[101:330, 7] = False
    for a, b in zip(results[0][:3], results[1][:3]):
        assert torch.equal(a[keep], b[keep])
    other = torch.arange(C) != 7
    for a, b in zip(results[0][3:], results[1][3:]):
        assert torch.equal(a[0], b[0]) or a.shape[0] == 5
    assert torch.equal(results[0][3][2, other], results[1][3][2, other])
    assert torch.equal(results[0][4][2], results[1][4][2]) and torch.equal(results[0][4][0, other], results[1][4][0, other])
    assert results[1][4][[1, 3]].isnan().all()


@pytest.mark.parametrize("gate,input", MODES)
def test_gradient_against_differences(gate, input):
    """The kernel's fp32 gradients along random directions against difference quotients of the 64-bit recurrence."""
    say("differences", gate, input)
    gen = torch.Generator().manual_seed(30 + gate * 3 + input)
    T, C = 100, 16
    x, g = ref.inputs(gen, T, C, F32, gate)
    do, dlast, start = torch.randn(T, C, generator=gen), torch.randn(1, C, generator=gen), torch.randn(1, C, generator=gen)
    st = state_of(start)
    o, dx, dg = (torch.empty_like(x).cuda() for _ in range(3))
    ck, dfirst = torch.empty(ssq.ssq_gated_checkpoint_rows(1, T), C, device="cuda"), torch.empty(1, C, device="cuda")
    ssq.ssq_gated_scan(st, x.cuda(), g.cuda(), o, cu_of([T]), gate=gate, input=input, checkpoints=ck)
    ssq.ssq_gated_scan_backward(ck, x.cuda(), g.cuda(), do.cuda(), dx, dg, cu_of([T]), gate=gate, input=input, dlast=dlast.cuda(),
                                dfirst=dfirst)

    def loss(x, g, h):
        h = ref.scan(x, g, h, gate, input)[0]
        return float((h[1:] * do).sum() + (h[-1] * dlast[0]).sum())

    base = [x.double(), g.double(), start[0].double()]
    for i, grad in enumerate((dx, dg, dfirst[0])):
        way = torch.randn(base[i].shape, generator=gen, dtype=torch.float64)
        way = way * (base[1].abs() if i == 1 and gate == 0 else 1.0)
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + 1e-6 * way, base[i] - 1e-6 * way
        slope = (loss(*up) - loss(*down)) / 2e-6
        terms = grad.cpu().double() * way
        # gradients in fp32 from at most T tokens' chains: 2^-24 of each term some hundred times
        assert abs(slope - float(terms.sum())) <= 3e-5 * float(terms.abs().sum()) + 1e-6, (i, slope, float(terms.sum()))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_a_graph(dtype):
    """Prompt, gradient and token captured, replayed with eager work between, every replay against eager calls."""
    say("graph", dtype)
    gen = torch.Generator().manual_seed(40)
    C, lens = 520, [700, 33]
    T = sum(lens)
    cu = cu_of(lens)
    x, g = (t.cuda() for t in ref.inputs(gen, T, C, dtype, 0))
    do = torch.randn(T, C, generator=gen).to(dtype).cuda()
    start = torch.randn(2, C, generator=gen)
    st = state_of(start)
    o, dx, dg = (torch.zeros_like(x) for _ in range(3))
    ck, dfirst = torch.empty(ssq.ssq_gated_checkpoint_rows(2, T), C, device="cuda"), torch.empty(2, C, device="cuda")
    ws = torch.empty(max(256, ssq.ssq_gated_workspace(C, 2, T)), dtype=torch.uint8, device="cuda")

    def run():
        ssq.ssq_gated_scan(st, x, g, o, cu, input=2, checkpoints=ck, workspace=ws)
        ssq.ssq_gated_scan_backward(ck, x, g, do, dx, dg, cu, input=2, dfirst=dfirst, workspace=ws)
        ssq.ssq_gated_step(st, x[:2], g[:2], o[:2], input=2)

    def results():
        return [t.clone() for t in (o, dx, dg, dfirst, st.regions()[0])]

    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        run()
    torch.cuda.synchronize()
    st.regions()[0].copy_(start)
    eager = []
    for _ in range(3):
        run()
        eager.append(results())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    st.regions()[0].copy_(start)
    for want in eager:
        for t in (o, dx, dg, dfirst):
            t.fill_(SENTINEL)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(results(), want):
            assert torch.equal(a, b)


def test_two_calls_at_once():
    say("two at once")
    gen = torch.Generator().manual_seed(21)
    C, T = 136, 3000
    cases = [[t.cuda() for t in ref.inputs(gen, T, C, dtype, 1)] + [torch.randn(1, C, generator=gen)] for dtype in (BF, F32, BF)]
    cu = cu_of([T])

    def run(i, out, stream=None):
        x, g, start = cases[i]
        st, o, dx, dg = out
        ck = torch.empty(ssq.ssq_gated_checkpoint_rows(1, T), C, device="cuda")
        for _ in range(3):
            ssq.ssq_gated_scan(st, x, g, o, cu, gate=1, input=1, checkpoints=ck, stream=stream)
            ssq.ssq_gated_scan_backward(ck, x, g, x, dx, dg, cu, gate=1, input=1, stream=stream)
        return ck

    fresh = lambda c: (state_of(c[2]), *(torch.zeros_like(c[0]) for _ in range(3)))  # noqa: E731
    want = []
    for i, c in enumerate(cases):
        out = fresh(c)
        run(i, out)
        want.append([values_of(out[0])] + [t.cpu() for t in out[1:]])
    outs, streams = [fresh(c) for c in cases], [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    keep = [run(i, outs[i], s) for i, s in enumerate(streams)]
    torch.cuda.synchronize()
    for w, out in zip(want, outs):
        assert torch.equal(w[0], values_of(out[0])) and all(torch.equal(a, b.cpu()) for a, b in zip(w[1:], out[1:]))
    del keep


def test_refusals():
    say("refusals")
    C, T = 24, 6
    st = state_of(torch.ones(2, C))
    t = lambda *s, d=BF: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    x, cu = t(T, C), cu_of([4, 2])
    ck = t(ssq.ssq_gated_checkpoint_rows(2, T), C, d=F32)
    before = st.storage.clone()
    bad = (ValueError, TypeError, ssq.SsqError)

    def refused(call, *a, **kw):
        with pytest.raises(bad):
            call(*a, **kw)

    o = t(T, C)
    for kw in (dict(x=t(T, C, d=torch.float64)), dict(g=t(T, C, d=HF)), dict(g=t(T, 16)), dict(g=t(5, C)), dict(o=t(T, C).cpu()),
               dict(cu=torch.tensor([0, 6], device="cuda")), dict(x=t(T, 2 * C)[:, ::2]), dict(o=t(1, C).expand(T, C)),
               dict(slots=t(3, d=torch.int32)), dict(fresh=t(1, d=torch.uint8)), dict(gate=2), dict(input=3), dict(gate=-1),
               dict(gate=1 << 32), dict(checkpoints=ck[:1]), dict(checkpoints=ck.double()), dict(cu=cu_of([2, 2, 2])),
               dict(x=t(T, C + 4)[:, :C], g=x, o=o), dict(stream=type("S", (), dict(cuda_stream=0, device=torch.device("cuda", 1)))())):
        a = dict(x=x, g=x, o=o, cu=cu) | kw
        refused(ssq.ssq_gated_scan, st, a.pop("x"), a.pop("g"), a.pop("o"), a.pop("cu"), **a)
    refused(ssq.ssq_gated_scan, None, x, x, o, cu, slots=t(2, d=torch.int32))
    refused(ssq.ssq_gated_scan, None, x, x, o, cu, fresh=t(2, d=torch.uint8))
    refused(ssq.ssq_gated_scan, None, t(T, 20), t(T, 20), t(T, 20), cu)  # channels not a multiple of 8
    refused(ssq.ssq_gated_scan, st, t(T, 16), t(T, 16), t(T, 16), cu)    # the state has 24
    refused(ssq.ssq_gated_step, st, x, x, o)                             # six rows, two sequences
    refused(ssq.ssq_gated_step, st, x[:2], x[:2], o[:2], slots=t(3, d=torch.int32))
    other = ssq.ssq_alloc_state(ssq.make_desc(ssq.SSQ_MAMBA2, "fp32", 2, 1, 16))
    refused(ssq.ssq_gated_step, other, x[:2], x[:2], o[:2])
    refused(ssq.ssq_linattn_step, st, t(2, 1, 128), t(2, 1, 128), t(2, 1, 16), None, t(2, 1, 16))
    grad = ssq.ssq_gated_scan_backward
    for kw in (dict(do=t(T, 16)), dict(dx=t(T, C, d=F32)), dict(dg=t(5, C)), dict(dlast=t(2, C)), dict(dfirst=t(1, C, d=F32)),
               dict(ck=ck[1:]), dict(ck=ck.cpu()), dict(slots=t(2, d=torch.int32)), dict(cu=cu_of([1, 2, 3]), state=st)):
        a = dict(ck=ck, do=x, dx=t(T, C), dg=t(T, C), cu=cu) | kw
        refused(grad, a.pop("ck"), x, x, a.pop("do"), a.pop("dx"), a.pop("dg"), a.pop("cu"), **a)
    for fmt, H, P, C2 in (("int8_sym", 1, 1, 24), ("fp32", 2, 1, 24), ("fp32", 1, 16, 24), ("fp32", 1, 1, 20), ("fp32", 1, 1, (1 << 20) + 8)):
        refused(ssq.ssq_alloc_state, ssq.make_desc(ssq.SSQ_GATED, fmt, 2, H, P, C2))
    gone = state_of(torch.ones(2, C))
    gone.free()  # not the same as no state
    refused(ssq.ssq_gated_scan, gone, x, x, o, cu)
    refused(ssq.ssq_gated_scan_backward, ck, x, x, x, t(T, C), t(T, C), cu, state=gone)
    refused(ssq.ssq_gated_step, gone, x[:2], x[:2], o[:2])
    torch.cuda.synchronize()
    assert torch.equal(st.storage, before) and (o == 0).all()


@pytest.mark.parametrize("nseq,tokens", [(0, 0), (0, 9), (2, 0)])
def test_empty_calls(nseq, tokens):
    say("empty", nseq, tokens)
    C = 24
    start = torch.randn(2, C, generator=torch.Generator().manual_seed(1))
    st = state_of(start)
    x = torch.zeros(tokens, C, device="cuda")
    cu = torch.zeros(nseq + 1, dtype=torch.int32, device="cuda")
    ck = torch.zeros(ssq.ssq_gated_checkpoint_rows(nseq, tokens), C, device="cuda")
    fresh = torch.tensor([1, 0][:nseq], dtype=torch.uint8, device="cuda")
    o, dx, dg = (torch.full_like(x, SENTINEL) for _ in range(3))
    ssq.ssq_gated_scan(st, x, x, o, cu, fresh=fresh, checkpoints=ck)
    dlast, dfirst = torch.ones(nseq, C, device="cuda"), torch.zeros(nseq, C, device="cuda")
    ssq.ssq_gated_scan_backward(ck, x, x, x, dx, dg, cu, dlast=dlast, dfirst=dfirst)
    got = values_of(st)
    assert torch.equal(got[1], start[1]) and torch.equal(got[0], start[0] * (0 if nseq else 1))
    assert (dfirst == 1).all() and (o == SENTINEL).all() and (dx == SENTINEL).all()
    ssq.ssq_gated_step(st, x[:0], x[:0], x[:0])


def test_a_gated_state_is_a_state_like_the_others():
    """It follows its beams and reads back; calls of other kinds refuse it."""
    say("state")
    start = torch.randn(6, 40, generator=torch.Generator().manual_seed(2))
    st = state_of(start)
    other = ssq.ssq_alloc_state(ssq.make_desc(ssq.SSQ_MAMBA2, "int8_sym", 6, 2, 16))
    ssq.ssq_state_reorder([st, other], torch.tensor([[1, 1, 0], [2, 0, 0]], dtype=torch.int32, device="cuda"))
    assert torch.equal(values_of(st), start[[1, 1, 0, 5, 3, 3]])
    with pytest.raises(ssq.SsqError):
        ssq.ssq_set_rounding(st, ssq.SSQ_ROUND_STOCHASTIC)
    f = torch.zeros(1 << 12, device="cuda")
    p = f.data_ptr()
    assert ssq.lib.ssq_decode_step(st.handle, p, p, p, p, p, p, p, 0, None) == ssq.SSQ_ERR_KIND_MISMATCH
    assert ssq.lib.ssq_delta_step(st.handle, p, p, p, p, p, p, 0, None) == ssq.SSQ_ERR_KIND_MISMATCH
    owned = ssq.ssq_alloc_state(ssq.make_desc(ssq.SSQ_GATED, "fp32", 3, 1, 1, 40))
    assert (values_of(owned) == 0).all()
