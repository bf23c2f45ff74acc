"""GPU: linear attention with a decay for each head, prompts and single tokens, against the
recurrence in 64 bits.

Tolerances.  An output of a half type is rounded once, by half a step of its type relative to
the value.  Between, the chunked form may round its decayed scores and its copy of the state to
bf16, half a step of 2^-8 relative to each term: at most 2^-8 of the sum of the terms' absolute
values, which the reference computes beside each output.  The state and fp32 outputs are sums in
fp32 of n = T + 256 terms at most, each rounding 2^-24 of the sum of absolute values, and decays
are exponentials in fp32 of sums taken wider: 2^-22 of a term.  n*2^-24 is the worst order; the
bound taken is that of a tree or of chained blocks of 64 and 128, (64 + 128 + T/64 + 8)*2^-24.
"""
import sys

import numpy as np
import pytest
import torch

from tests import linattn_ref as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mamba_decode_amd as ssq
    from tests import parity as par

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
SENTINEL = 7.0


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def state_of(values, G, fmt="fp32"):
    B, H, P, N = values.shape
    desc = ssq.make_desc(ssq.SSQ_MAMBA2, fmt, B, H, P, N, G)
    storage = torch.zeros(ssq.ssq_state_bytes(desc), dtype=torch.uint8, device="cuda")
    return ssq.ssq_alloc_state(desc, storage, values.float().cuda().contiguous())


def values_of(state):
    d = state.desc
    out = torch.empty(d.batch, d.nheads, d.rows_per_head, d.row_len, device="cuda")
    ssq.ssq_dequant(state, out)
    return out.cpu()


def sum_bound(T):
    return (64 + 128 + T / 64 + 8) * 2.0 ** -24 + 2.0 ** -22


def check_o(o, want, mag, T, dtype, where):
    tol = sum_bound(T) * mag
    if dtype != F32:
        tol = tol + mag * 2.0 ** -8 + want.abs() * (torch.finfo(dtype).eps / 2) + torch.finfo(dtype).tiny
    bad = (o.double() - want).abs() > tol
    assert not bad.any(), f"{where}: o off at {bad.nonzero()[:4].tolist()}, {int(bad.sum())} of {bad.numel()}"


def check_state(got, want, mag, T, where):
    bad = (got.double() - want).abs() > sum_bound(T) * mag + 1e-38
    assert not bad.any(), f"{where}: state off at {bad.nonzero()[:4].tolist()}, {int(bad.sum())} of {bad.numel()}"


def cu_of(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")


def prefill_case(dtype, H, G, P, lens, tail=0, packed=False, slots=None, fresh=None, g_kind="drawn", seed=0, scale=0.3,
                 batch=None):
    gen = torch.Generator().manual_seed(seed)
    T = sum(lens) + tail
    q, k, v, g = ref.inputs(gen, T, H, G, P, dtype)
    if g_kind == "none":
        g = None
    elif g_kind == "constant":
        g = g[:1].expand(T, H)
    elif g_kind == "forget":  # the state forgotten at some tokens, by -inf, the lowest value and a large one
        at = torch.rand(T, H, generator=gen)
        g = torch.where(at < 0.05, -torch.inf, torch.where(at < 0.1, torch.finfo(F32).min, torch.where(at < 0.15, -200.0, g)))
    elif g_kind == "zero":
        g = torch.zeros(T, H)
    n = len(lens)
    batch = batch or n
    start = torch.randn(batch, H, P, 128, generator=gen)
    st = state_of(start, G)
    if packed:  # slices of one projection's output, wider than they are
        row = torch.cat([x.reshape(T, -1) for x in (q, k, v)] + [torch.zeros(T, 24, dtype=dtype)], 1).cuda()
        dq, dk = row[:, :G * 128].view(T, G, 128), row[:, G * 128:2 * G * 128].view(T, G, 128)
        dv = row[:, 2 * G * 128:2 * G * 128 + H * P].view(T, H, P)
        do = torch.full((T, H * P + 16), SENTINEL, dtype=dtype, device="cuda")[:, 8:8 + H * P].view(T, H, P)
    else:
        dq, dk, dv = q.cuda(), k.cuda(), v.cuda()
        do = torch.full((T, H, P), SENTINEL, dtype=dtype, device="cuda")
    if g is None:
        dg = None
    elif g_kind == "constant":
        dg = g[:1].cuda().expand(T, H)
    else:
        dg = g.cuda()
    dslots = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
    dfresh = None if fresh is None else torch.tensor(fresh, dtype=torch.uint8, device="cuda")
    ssq.ssq_linattn_prefill(st, dq, dk, dv, dg, do, cu_of(lens), slots=dslots, fresh=dfresh, scale=scale)
    torch.cuda.synchronize()
    o, state = do.cpu(), values_of(st)
    seen, at = set(), 0
    for i, n_i in enumerate(lens):
        slot = i if slots is None else slots[i]
        span = slice(at, at + n_i)
        at += n_i
        where = f"sequence {i} of {n_i} tokens"
        if not 0 <= slot < batch:
            assert (o[span] == SENTINEL).all(), where
            continue
        seen.add(slot)
        begin = torch.zeros_like(start[slot]) if fresh is not None and fresh[i] else start[slot]
        wo, ws, om, sm = ref.recurrence(q[span], k[span], v[span], None if g is None else g[span], begin, scale)
        check_o(o[span], wo, om, n_i, dtype, where)
        check_state(state[slot], ws, sm, n_i, where)
        if n_i == 0:
            assert torch.equal(state[slot], begin)
    assert (o[at:] == SENTINEL).all(), "rows behind the last sequence"
    for s in set(range(batch)) - seen:
        assert torch.equal(state[s], start[s]), f"slot {s} is nobody's"


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("H,G,P", [(24, 1, 64), (4, 2, 16), (3, 3, 48), (2, 1, 128), (6, 2, 80), (1, 1, 192)])
def test_prompts(dtype, H, G, P):
    say("prompts", dtype, H, G, P)
    prefill_case(dtype, H, G, P, [5, 0, 64, 1, 130, 63, 65], tail=3, seed=H + P)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 255, 513, 1000, 2049])
def test_lengths(dtype, T):
    say("lengths", dtype, T)
    prefill_case(dtype, 4, 2, 64, [T], seed=T, fresh=[1] if T % 2 else None)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_slots_fresh_and_padding(dtype):
    say("slots", dtype)
    prefill_case(dtype, 6, 2, 64, [70, 3, 0, 200, 0, 9], tail=70, slots=[5, 0, 7, 2, 3, 1], fresh=[1, 0, 1, 0, 0, 1], batch=9)
    prefill_case(dtype, 2, 1, 32, [4, 100, 6, 50], slots=[-1, 2, 1 << 30, 0], batch=3, seed=1)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_slices_of_one_projection(dtype):
    say("strides", dtype)
    prefill_case(dtype, 8, 2, 64, [100, 29], tail=2, packed=True)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("kind", ["none", "constant", "forget", "zero"])
def test_decays(dtype, kind):
    say("decays", dtype, kind)
    prefill_case(dtype, 6, 1, 64, [300, 77], g_kind=kind, seed=5)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_few_heads_and_a_long_prompt(dtype):
    """The sequence is split into parts here: one head, thousands of tokens, beside short ones."""
    say("long", dtype)
    prefill_case(dtype, 1, 1, 64, [5000, 1, 700], seed=3)
    prefill_case(dtype, 3, 1, 128, [3000, 0, 65], fresh=[1, 1, 0], seed=4, tail=5)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_heads(dtype):
    """Enough heads and sequences that none is split."""
    say("many heads", dtype)
    prefill_case(dtype, 96, 4, 64, [40, 130, 0, 64, 90, 1, 33, 128, 200, 3], seed=6)


def test_a_prompt_in_two_calls_is_the_prompt():
    say("two calls")
    gen = torch.Generator().manual_seed(8)
    H, G, P, T = 4, 1, 64, 300
    q, k, v, g = (x.cuda() for x in ref.inputs(gen, T, H, G, P, F32))
    start = torch.randn(1, H, P, 128, generator=gen)
    one, two = state_of(start, G), state_of(start, G)
    o1, o2 = torch.empty_like(v), torch.empty_like(v)
    ssq.ssq_linattn_prefill(one, q, k, v, g, o1, cu_of([T]))
    for a, b in ((0, 101), (101, T)):
        ssq.ssq_linattn_prefill(two, q[a:b], k[a:b], v[a:b], g[a:b], o2[a:b], cu_of([b - a]))
    wo, ws, om, sm = ref.recurrence(q.cpu(), k.cpu(), v.cpu(), g.cpu(), start[0], 1.0)
    for o, st in ((o1, one), (o2, two)):
        check_o(o.cpu(), wo, om, T, F32, "two calls")
        check_state(values_of(st)[0], ws, sm, T, "two calls")


@pytest.mark.parametrize("fmt", ["int8_sym", "int8_asym", "int4_sym", "int4_asym"])
def test_prompts_into_a_quantized_state(fmt):
    """The recurrence starts from the reconstructed rows, and the rows it leaves are refit and
    rounded once: the bytes are those of a state made from the fp32 call's result."""
    say("quantized", fmt)
    gen = torch.Generator().manual_seed(9)
    H, G, P, lens = 6, 2, 48, [70, 0, 33, 0, 1]
    q, k, v, g = (x.cuda() for x in ref.inputs(gen, sum(lens), H, G, P, BF))
    start = torch.randn(7, H, P, 128, generator=gen)
    slots = torch.tensor([3, 0, 6, 2, 5], dtype=torch.int32, device="cuda")
    fresh = torch.tensor([1, 0, 0, 1, 0], dtype=torch.bool, device="cuda")
    st = state_of(start, G, fmt)
    before = st.storage.clone()
    f32 = state_of(values_of(st), G)
    o, of = torch.zeros_like(v), torch.zeros_like(v)
    ssq.ssq_linattn_prefill(f32, q, k, v, g, of, cu_of(lens), slots=slots, fresh=fresh)
    ssq.ssq_linattn_prefill(st, q, k, v, g, o, cu_of(lens), slots=slots, fresh=fresh)
    assert torch.equal(o, of)
    want = state_of(values_of(f32), G, fmt)
    got, exp, old = (par.read_gpu_state(s, fmt) if isinstance(s, ssq.State) else s for s in (st, want, None))
    rows = H * P
    moved = np.zeros(7, bool)
    moved[[3, 6, 2, 5]] = True
    for name in ("code", "scale", "zero"):
        if got.get(name) is None:
            continue
        a, b = (x[name].reshape(7, -1) for x in (got, exp))
        assert np.array_equal(a[moved], b[moved]), name
    codes, scale, zero = st.regions()
    prev = ssq.State(None, st.desc, st.layout, before)
    pc, ps, pz = prev.regions()
    still = torch.tensor(~moved).repeat_interleave(rows)
    assert torch.equal(codes.cpu()[still], pc.cpu()[still]) and torch.equal(scale.cpu()[still], ps.cpu()[still])


def test_stochastic_rounding_of_a_prompt():
    """One draw of uniforms at the state's next token, which moves on by one."""
    say("stochastic prompt")
    gen = torch.Generator().manual_seed(10)
    H, P, T, fmt = 4, 64, 70, "int8_asym"
    q, k, v, g = (x.cuda() for x in ref.inputs(gen, T, H, 1, P, BF))
    st, f32 = state_of(torch.zeros(1, H, P, 128), 1, fmt), state_of(torch.zeros(1, H, P, 128), 1)
    ssq.ssq_set_rounding(st, ssq.SSQ_ROUND_STOCHASTIC, 77, 5)
    o = torch.empty_like(v)
    ssq.ssq_linattn_prefill(f32, q, k, v, g, o, cu_of([T]))
    ssq.ssq_linattn_prefill(st, q, k, v, g, o, cu_of([T]))
    assert ssq.ssq_get_rounding(st)[2] == 6
    import oracle
    rows = H * P
    codes, scale, zero = st.regions()
    got = par.read_gpu_state(st, fmt)
    h = values_of(f32).reshape(rows, 128).numpy()
    # the grid is round-to-nearest's; each code is one of the two neighbours of the exact value
    near = oracle.make_state(fmt, rows, 128, h)
    assert np.array_equal(got["scale"], near.scale) and np.array_equal(got["zero"], near.zero)
    inv = (np.float32(1) / near.scale).astype(np.float64).reshape(rows, 1)
    exact = h.astype(np.float64) * inv + near.zero.reshape(rows, 1)
    code = got["code"].reshape(rows, 128)
    assert (np.abs(code - exact) <= 1.0 + 1e-6).all() and not np.array_equal(code, near.code.reshape(rows, 128))


# ----------------------------------------------------------------------------- single tokens


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("H,G,P,n", [(24, 1, 64, 1), (4, 2, 16, 5), (3, 3, 48, 2), (2, 1, 128, 9), (6, 2, 80, 3)])
def test_tokens(dtype, H, G, P, n):
    say("tokens", dtype, H, G, P, n)
    gen = torch.Generator().manual_seed(n)
    B = n + 3
    q, k, v, g = ref.inputs(gen, n, H, G, P, dtype)
    g[0, 0] = -torch.inf
    start = torch.randn(B, H, P, 128, generator=gen)
    st = state_of(start, G)
    slots = torch.randperm(B, generator=gen)[:n].tolist()
    if n > 2:
        slots[1] = -1
    o = torch.full(v.shape, SENTINEL, dtype=dtype, device="cuda")
    ssq.ssq_linattn_step(st, q.cuda(), k.cuda(), v.cuda(), g.cuda(), o,
                         slots=torch.tensor(slots, dtype=torch.int32, device="cuda"), scale=0.3)
    o, state = o.cpu(), values_of(st)
    for i, s in enumerate(slots):
        if s < 0:
            assert (o[i] == SENTINEL).all()
            continue
        wo, ws, om, sm = ref.recurrence(q[i:i + 1], k[i:i + 1], v[i:i + 1], g[i:i + 1], start[s], 0.3)
        tol = om[0] * 130 * 2.0 ** -24
        if dtype != F32:
            tol = tol + wo[0].abs() * (torch.finfo(dtype).eps / 2) + torch.finfo(dtype).tiny
        assert ((o[i].double() - wo[0]).abs() <= tol).all(), i
        assert ((state[s].double() - ws).abs() <= sm * 3 * 2.0 ** -24).all(), i
    for s in set(range(B)) - set(slots):
        assert torch.equal(state[s], start[s])


@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("sr", [False, True])
@pytest.mark.parametrize("fmt", ["int8_sym", "int8_asym", "int4_sym", "int4_asym", "fp32"])
def test_tokens_are_the_decode_step(fmt, sr, pre):
    """With the same decay in every sequence the step is the Mamba-2 decode step with dt = 1 and
    D = 0: the same bytes in the state, and o in another order of summation."""
    say("decode step", fmt, sr, pre)
    if fmt == "fp32" and sr:
        pytest.skip("the fp32 state is not rounded")
    gen = torch.Generator().manual_seed(11)
    B, H, G, P = 5, 6, 2, 48
    start = torch.randn(B, H, P, 128, generator=gen)
    start[1, 2] = 1000.0 + 1e-3 * torch.randn(P, 128, generator=gen)  # rows far from zero: the slow path
    start[2, 1] = 0.0
    one, two = state_of(start, G, fmt), state_of(start, G, fmt)
    if sr:
        for s in (one, two):
            ssq.ssq_set_rounding(s, ssq.SSQ_ROUND_STOCHASTIC, 123, 9)
    readout = ssq.SSQ_READ_PRE_QUANT if pre else ssq.SSQ_READ_POST_QUANT
    A = -torch.rand(H, generator=gen)
    dt, D = torch.ones(B, H), torch.zeros(H)
    for t in range(3):
        q, k, v, _ = ref.inputs(gen, B, H, G, P, F32)
        if t == 2:
            v[2, 1] = 0.0  # a row of zeros
        y, o = torch.empty(B, H, P, device="cuda"), torch.empty(B, H, P, device="cuda")
        ssq.ssq_decode_step(one, v.cuda(), dt.cuda(), A.cuda(), k.cuda(), q.cuda(), D.cuda(), y, readout)
        ssq.ssq_linattn_step(two, q.cuda(), k.cuda(), v.cuda(), A.cuda().expand(B, H), o, readout=readout)
        assert torch.equal(one.storage, two.storage), t
        mag = (values_of(two).abs() * q.repeat_interleave(H // G, 1).abs()[:, :, None]).sum(-1).double()
        # pre-rounding values differ from the stored ones by a code's step at most: twice the sum covers them
        assert ((o.cpu().double() - y.cpu().double()).abs() <= 2 * 130 * 2.0 ** -24 * (mag + mag.mean())).all(), t


@pytest.mark.parametrize("fmt", ["int8_asym", "int4_asym", "int4_sym"])
def test_tokens_of_a_large_batch(fmt):
    """Enough rows that a wave takes 32 or 64 of them: the same bytes as in small calls."""
    say("large batch", fmt)
    gen = torch.Generator(device="cuda").manual_seed(17)
    for P in (64, 32):
        B, H = 4096 * 64 // (32 * P), 32
        start = torch.randn(B, H, P, 128, device="cuda", generator=gen)
        one, two = state_of(start, 1, fmt), state_of(start, 1, fmt)
        q, k, v, g = (x.cuda() for x in ref.inputs(torch.Generator().manual_seed(18), B, H, 1, P, BF))
        o, o2 = torch.empty_like(v), torch.empty_like(v)
        ssq.ssq_linattn_step(one, q, k, v, g, o)
        for i in range(0, B, 16):
            slots = torch.arange(i, i + 16, dtype=torch.int32, device="cuda")
            ssq.ssq_linattn_step(two, q[i:i + 16], k[i:i + 16], v[i:i + 16], g[i:i + 16], o2[i:i + 16], slots=slots)
        assert torch.equal(one.storage, two.storage) and torch.equal(o, o2)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_tokens_of_half_types_on_a_quantized_state(dtype):
    """Half-type inputs are exact in fp32: the bytes are those of the same values in fp32."""
    say("half step", dtype)
    gen = torch.Generator().manual_seed(12)
    B, H, G, P = 3, 4, 1, 64
    start = torch.randn(B, H, P, 128, generator=gen)
    for fmt in ("int8_asym", "int4_sym"):
        one, two = state_of(start, G, fmt), state_of(start, G, fmt)
        q, k, v, g = (x.cuda() for x in ref.inputs(gen, B, H, G, P, dtype))
        o, of = torch.empty_like(v), torch.empty_like(v, dtype=F32)
        ssq.ssq_linattn_step(one, q, k, v, g, o)
        ssq.ssq_linattn_step(two, q.float(), k.float(), v.float(), g, of)
        assert torch.equal(one.storage, two.storage) and torch.equal(o, of.to(dtype))


def test_step_after_step_is_the_prompt():
    say("steps are the prompt")
    gen = torch.Generator().manual_seed(13)
    H, G, P, T = 4, 2, 64, 20
    q, k, v, g = (x.cuda() for x in ref.inputs(gen, T, H, G, P, F32))
    start = torch.randn(1, H, P, 128, generator=gen)
    st = state_of(start, G)
    o = torch.empty_like(v)
    for t in range(T):
        ssq.ssq_linattn_step(st, q[t:t + 1], k[t:t + 1], v[t:t + 1], g[t:t + 1], o[t:t + 1])
    wo, ws, om, sm = ref.recurrence(q.cpu(), k.cpu(), v.cpu(), g.cpu(), start[0], 1.0)
    check_o(o.cpu(), wo, om, T, F32, "steps")
    check_state(values_of(st)[0], ws, sm, T, "steps")


# ----------------------------------------------------------------------------- calls


def test_captured_and_replayed_and_on_another_stream():
    say("graph")
    gen = torch.Generator().manual_seed(14)
    H, G, P, lens = 4, 1, 64, [500, 0, 77]
    q, k, v, g = (x.cuda() for x in ref.inputs(gen, sum(lens), H, G, P, BF))
    start = torch.randn(3, H, P, 128, generator=gen)
    cu = cu_of(lens)
    for fmt in ("fp32", "int8_asym"):
        st = state_of(start, G, fmt)
        begin = st.storage.clone()
        o, o1 = torch.zeros_like(v), torch.zeros(3, H, P, dtype=BF, device="cuda")

        def both():
            ssq.ssq_linattn_prefill(st, q, k, v, g, o, cu)
            ssq.ssq_linattn_step(st, q[:3], k[:3], v[:3], g[:3], o1)

        both()
        torch.cuda.synchronize()
        want = [x.clone() for x in (st.storage, o, o1)]
        side = torch.cuda.Stream()
        st.storage.copy_(begin)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            both()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((st.storage, o, o1), want))
        st.storage.copy_(begin)
        o.zero_()
        torch.cuda.synchronize()
        ssq.ssq_linattn_prefill(st, q, k, v, g, o, cu, stream=side)  # named, not the current one
        torch.cuda.synchronize()
        assert torch.equal(o, want[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            both()
        for _ in range(3):
            st.storage.copy_(begin)
            o.zero_()
            o1.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip((st.storage, o, o1), want))


def test_empty_calls():
    say("empty")
    st = state_of(torch.ones(2, 2, 16, 128), 1)
    e = lambda *s: torch.empty(*s, dtype=BF, device="cuda")  # noqa: E731
    g = torch.empty(0, 2, device="cuda")
    ssq.ssq_linattn_step(st, e(0, 1, 128), e(0, 1, 128), e(0, 2, 16), g, e(0, 2, 16))
    ssq.ssq_linattn_prefill(st, e(0, 1, 128), e(0, 1, 128), e(0, 2, 16), g, e(0, 2, 16), cu_of([]))
    ssq.ssq_linattn_prefill(st, e(0, 1, 128), e(0, 1, 128), e(0, 2, 16), g, e(0, 2, 16), cu_of([0, 0]),
                            fresh=torch.tensor([0, 1], dtype=torch.uint8, device="cuda"))
    got = values_of(st)
    assert (got[0] == 1).all() and (got[1] == 0).all()


def test_offsets_outside_the_tensors_are_clamped():
    say("clamped offsets")
    gen = torch.Generator().manual_seed(15)
    H, P, T = 2, 32, 40
    q, k, v, g = ref.inputs(gen, T, H, 1, P, BF)
    start = torch.randn(3, H, P, 128, generator=gen)
    st = state_of(start, 1)
    o = torch.zeros_like(v).cuda()
    cu = torch.tensor([-5, 10, 4, 1 << 30], dtype=torch.int32, device="cuda")  # 0..10, none, 4..40
    ssq.ssq_linattn_prefill(st, q.cuda(), k.cuda(), v.cuda(), g.cuda(), o, cu)
    state = values_of(st)
    for i, (a, b) in enumerate(((0, 10), (10, 10), (4, 40))):
        _, ws, _, sm = ref.recurrence(q[a:b], k[a:b], v[a:b], g[a:b], start[i], 1.0)
        check_state(state[i], ws, sm, b - a, f"sequence {i}")


@pytest.mark.parametrize("heads", [1, 40])
def test_rows_before_the_first_sequence(heads):
    say("rows before", heads)
    gen = torch.Generator().manual_seed(16)
    P, T, a, b = 64, 2000, 700, 1900
    q, k, v, g = ref.inputs(gen, T, heads, 1, P, BF)
    st = state_of(torch.zeros(2, heads, P, 128), 1)
    o = torch.full_like(v, SENTINEL).cuda()
    cu = torch.tensor([a, a + 300, b], dtype=torch.int32, device="cuda")
    ssq.ssq_linattn_prefill(st, q.cuda(), k.cuda(), v.cuda(), g.cuda(), o, cu)
    o, state = o.cpu(), values_of(st)
    assert (o[:a] == SENTINEL).all() and (o[b:] == SENTINEL).all()
    for i, s in enumerate((slice(a, a + 300), slice(a + 300, b))):
        wo, ws, om, sm = ref.recurrence(q[s], k[s], v[s], g[s], torch.zeros(heads, P, 128), 1.0)
        check_o(o[s], wo, om, 1200, BF, i)
        check_state(state[i], ws, sm, 1200, i)


def test_refusals():
    st = state_of(torch.zeros(2, 4, 32, 128), 2)
    t = lambda *s, d=BF: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    q, v, g, cu = t(6, 2, 128), t(6, 4, 32), t(6, 4, d=F32), cu_of([4, 2])
    before = st.storage.clone()

    def refused(kind, call, *a, **kw):
        with pytest.raises(kind):
            call(*a, **kw)

    run, step = ssq.ssq_linattn_prefill, ssq.ssq_linattn_step
    for kw in (dict(q=t(6, 1, 128)), dict(v=t(6, 4, 48)), dict(k=t(5, 2, 128)), dict(k=t(6, 2, 128, d=HF)),
               dict(g=t(6, 4)), dict(cu=torch.tensor([0, 6], device="cuda")), dict(q=t(6, 2, 256)[..., ::2]),
               dict(q=t(6, 2, 128).cpu()), dict(o=t(6, 2, 32).expand(6, 2, 32)), dict(q=t(6, 4, 128)[:, ::2])):
        x = dict(q=q, k=q, v=v, g=g, o=t(6, 4, 32), cu=cu) | kw
        refused(ValueError, run, st, x["q"], x["k"], x["v"], x["g"], x["o"], x["cu"])
    o = t(6, 4, 32)
    refused(ssq.SsqError, run, st, torch.zeros(6 * 257 + 1, dtype=BF, device="cuda")[1:].view(6, 257)[:, :256].view(6, 2, 128), q, v, g, o, cu)
    refused(ssq.SsqError, run, st, q, q, v, g, o, cu_of([2, 2, 2]))  # more sequences than the state holds
    refused(ssq.SsqError, run, st, q, q, v, g, o[:1].expand(6, 4, 32), cu)  # o's rows overlap
    refused(ssq.SsqError, step, st, q, q, v, g, o)  # six rows, two sequences
    refused(ssq.SsqError, step, st, q[:2], q[:2], v[:2], g[:2], o[:2], readout=5)
    refused(ValueError, step, st, q[:2], q[:2], v[:2], g[:2], o[:2], slots=t(3, d=torch.int32))
    delta = ssq.ssq_alloc_state(ssq.make_desc(ssq.SSQ_DELTA, "fp32", 2, 4, 128, 128))
    refused(ssq.SsqError, step, delta, q[:2], q[:2], v[:2], g[:2], o[:2])
    quant = state_of(torch.zeros(2, 4, 32, 128), 2, "int8_sym")
    refused(ssq.SsqError, run, quant, q, q, v, g, o, cu, workspace=t(256, d=torch.uint8))
    # more state rows, or more tokens, than one launch covers: refused whatever the slots say
    io = ssq._linattn_io(st, q, q, v, g, o, 1.0, 6, torch.cuda.current_device())
    slots = torch.full((8,), -1, dtype=torch.int32, device="cuda")
    ws = t(256, d=torch.uint8)
    for n, T in (((1 << 26) // 128 + 1, 6), (1, 0x7FFFFF80), (1, 1 << 40)):
        assert ssq.lib.ssq_linattn_workspace(st.handle, n, T) == ssq._SIZE_MAX
        assert ssq.lib.ssq_linattn_prefill(st.handle, io, n, T, cu.data_ptr(), slots.data_ptr(), None, ws.data_ptr(), 256,
                                           None) == ssq.SSQ_ERR_UNSUPPORTED
    assert ssq.lib.ssq_linattn_step(st.handle, io, (1 << 29) // 128 + 1, slots.data_ptr(), 0, None) == ssq.SSQ_ERR_UNSUPPORTED
    assert ssq.ssq_linattn_workspace(st, 0, 0x7FFFFF7F) == 0
    torch.cuda.synchronize()
    assert torch.equal(st.storage, before)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("fmt", ["fp32", "int8_asym"])
def test_nothing_is_read_that_is_not_asked_for(dtype, fmt):
    """NaN in the rows before, between and behind the sequences, in the states of fresh and unnamed
    slots and in one sequence: every other sequence has the result of a clean call."""
    say("NaN around", dtype, fmt)
    gen = torch.Generator().manual_seed(20)
    H, G, P, T = 4, 2, 48, 400
    q, k, v, g = (x.cuda() for x in ref.inputs(gen, T, H, G, P, dtype))
    start = torch.randn(5, H, P, 128, generator=gen)
    # tokens 10..100, 100..101 (the bad one), 101..330; 0..10 and 330..400 are padding
    cu = torch.tensor([10, 100, 101, 330], dtype=torch.int32, device="cuda")
    slots = torch.tensor([2, 4, 0], dtype=torch.int32, device="cuda")
    fresh = torch.tensor([1, 0, 0], dtype=torch.uint8, device="cuda")
    clean, dirty = state_of(start, G, fmt), state_of(start, G, fmt)
    want, got = torch.zeros_like(v), torch.zeros_like(v)
    ssq.ssq_linattn_prefill(clean, q, k, v, g, want, cu, slots=slots, fresh=fresh)
    for x in (q, k, v, g):
        x[:10] = x[330:] = x[100:101] = torch.nan
    for part in (dirty.regions()[0] if fmt == "fp32" else dirty.regions()[1],):
        rows = part.view(torch.float32).view(5, -1)
        rows[1] = rows[2] = rows[3] = torch.nan
    ssq.ssq_linattn_prefill(dirty, q, k, v, g, got, cu, slots=slots, fresh=fresh)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[100] = False
    assert torch.equal(got[keep], want[keep])
    a, b = values_of(clean), values_of(dirty)
    assert torch.equal(a[[0, 2]], b[[0, 2]])
    assert b[[1, 3]].isnan().all()


def test_two_calls_at_once():
    """Two prompts and a token on three states and streams, each with its own workspace."""
    say("two at once")
    gen = torch.Generator().manual_seed(21)
    H, P, T = 8, 64, 1500
    cases = []
    for dtype in (BF, F32, BF):
        q, k, v, g = (x.cuda() for x in ref.inputs(gen, T, H, 1, P, dtype))
        start = torch.randn(1, H, P, 128, generator=gen)
        cases.append((q, k, v, g, start))
    cu = cu_of([T])

    def run(i, st, o, stream=None):
        q, k, v, g, _ = cases[i]
        for _ in range(3):
            ssq.ssq_linattn_prefill(st, q, k, v, g, o, cu, stream=stream)
            ssq.ssq_linattn_step(st, q[:1], k[:1], v[:1], g[:1], o[:1], stream=stream)

    want = []
    for i, c in enumerate(cases):
        st, o = state_of(c[4], 1), torch.zeros_like(c[2])
        run(i, st, o)
        want.append((values_of(st), o.cpu()))
    streams = [torch.cuda.Stream() for _ in cases]
    states, outs = [state_of(c[4], 1) for c in cases], [torch.zeros_like(c[2]) for c in cases]
    torch.cuda.synchronize()
    for i, s in enumerate(streams):
        run(i, states[i], outs[i], stream=s)
    torch.cuda.synchronize()
    for w, st, o in zip(want, states, outs):
        assert torch.equal(w[0], values_of(st)) and torch.equal(w[1], o.cpu())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,H,G", [(2, 140, 2), (7, 40, 8), (31, 12, 1), (64, 5, 5), (65, 4, 2), (130, 3, 1)])
def test_sequences_of_every_length_that_fill_the_card(dtype, n, H, G):
    """Whole sequences, taken in the order of their lengths up to 64 of them: equal lengths, empty
    ones, ones that are skipped, the longest anywhere."""
    say("order of lengths", dtype, n, H)
    gen = torch.Generator().manual_seed(n)
    lens = [(0, 1, 64, 65, 5)[i % 5] if i % 2 else int(torch.randint(0, 130, (1,), generator=gen)) for i in range(n)]
    lens[n // 2] = 200
    slots = torch.randperm(n + 2, generator=gen)[:n].tolist()
    if n > 2:
        slots[1] = -1
        slots[n - 1] = n + 2
    prefill_case(dtype, H, G, 16, lens, tail=3, slots=slots, fresh=[i % 3 == 0 for i in range(n)], seed=n, batch=n + 2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[1025], [0, 700, 0], [0], [193, 192, 191], [0, 5, 900, 64, 0], [3, 4000], [2600, 0, 0, 0, 1],
                                  [8000, 10, 0, 200, 1]])
def test_parts_joined_by_those_who_need_them_and_by_a_launch(dtype, lens):
    """Sequences of few heads, in one part, a few and many, with empty ones, fresh and not."""
    say("parts", dtype, lens)
    n = len(lens)
    for fresh in ([0] * n, [1] * n, [i % 2 for i in range(n)]):
        prefill_case(dtype, 2, 1, 32, lens, tail=2, slots=list(range(n, 0, -1)), fresh=fresh, seed=sum(lens), batch=n + 1)
