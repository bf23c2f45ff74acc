"""GPU: beam selection against a stable sort in 64 bits, and states that follow their beams.

Scores: one rounding to fp32 (2^-24 of the value) and a softmax sum in fp32 of exponentials with
a few units of error each: 2^-20 of the sum, as much of its logarithm's argument, absolutely."""
import itertools
import math
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mamba_decode_amd as ssq

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def reference(logits, scores, finished, n, pad):
    b, m, v = logits.shape
    x = logits.double()
    x = torch.where(x.isnan(), -math.inf, x)
    top = x.amax(-1, keepdim=True)
    rel = torch.where(x == -math.inf, -math.inf, x - torch.where(top == -math.inf, 0.0, top))
    logp = rel - rel.exp().sum(-1, keepdim=True).log()
    logp = torch.where(x == -math.inf, -math.inf, logp)
    if finished is not None:
        only = torch.full_like(logp, -math.inf)
        only[..., pad] = 0.0
        logp = torch.where(finished.bool()[..., None], only, logp)
    alive = scores > -math.inf
    s = torch.where(alive[..., None], scores.double()[..., None] + logp, -math.inf).view(b, m * v)
    val, at = s.sort(dim=-1, descending=True, stable=True)
    if val.shape[1] < n:
        val = torch.cat([val, torch.full((b, n - val.shape[1]), -math.inf, dtype=val.dtype)], 1)
        at = torch.cat([at, torch.zeros(b, n - at.shape[1], dtype=at.dtype)], 1)
    val, at = val[:, :n], at[:, :n]
    none = val == -math.inf
    return val, torch.where(none, -1, at % v), torch.where(none, torch.arange(n) % m, at // v)


def select(logits, scores, n, finished=None, pad=0, **kw):
    b = logits.shape[0]
    out = (torch.full((b, n), 9.0, device="cuda"), torch.full((b, n), -7, dtype=torch.int32, device="cuda"),
           torch.full((b, n), -7, dtype=torch.int32, device="cuda"))
    ssq.ssq_beam_select(logits, scores, *out, finished=finished, pad_token=pad, **kw)
    return out


def check(logits, scores, n, finished=None, pad=0):
    out = [x.cpu() for x in select(logits, scores, n, finished, pad)]
    want = reference(logits.cpu(), scores.cpu(), None if finished is None else finished.cpu(), n, pad)
    none = want[0] == -math.inf
    assert torch.equal(out[0] == -math.inf, none)
    off = (out[0].double() - want[0])[~none].abs()
    assert (off <= want[0][~none].abs() * 2.0 ** -23 + 2.0 ** -19).all(), off.max()
    assert torch.equal(out[1].long(), want[1]), (out[1], want[1])
    assert torch.equal(out[2].long(), want[2]), (out[2], want[2])


def draw(gen, b, m, v, dtype, spread=3.0):
    return (torch.randn(b, m, v, generator=gen) * spread).to(dtype).cuda(), (-10 * torch.rand(b, m, generator=gen)).cuda()


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("b,m,v", [(1, 4, 50280), (3, 8, 1000), (2, 1, 300), (1, 5, 8193), (2, 16, 32001), (1, 2, 150001),
                                   (1, 32, 7000), (3, 3, 17), (1, 1, 1), (2, 4, 3)])
def test_selection(dtype, b, m, v):
    say("selection", dtype, b, m, v)
    gen = torch.Generator().manual_seed(v)
    logits, scores = draw(gen, b, m, v, dtype)
    for n in sorted({1, m, 2 * m}):
        check(logits, scores, n)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_ties_go_to_the_lower_token(dtype):
    say("ties", dtype)
    gen = torch.Generator().manual_seed(1)
    for v in (40, 9000, 20000):
        logits = torch.randint(-1, 2, (2, 4, v), generator=gen).to(dtype).cuda()
        check(logits, torch.tensor([[0.0, -5.0, -0.25, -9.0]] * 2).cuda(), 8)
        check(torch.full((1, 4, v), -0.5, dtype=dtype, device="cuda"), torch.tensor([[-1.0, -2.0, -3.0, -4.0]]).cuda(), 8)
    # signed zeros are equal; equal beams: the lower beam first
    z = torch.zeros(1, 3, 5000, dtype=dtype)
    z[..., ::2] = -0.0
    check(z.cuda(), torch.zeros(1, 3).cuda(), 6)


def test_descending_rows():
    """Rows sorted against the lanes: a lane then holds many of the best."""
    say("descending")
    for v, m in ((30000, 16), (70000, 32)):
        x = torch.arange(v, 0, -1).float()[None, None].repeat(1, m, 1) * 1e-3
        for rows in (x, x.flip(-1), x.view(1, m, 10, -1).transpose(-1, -2).reshape(1, m, v)):
            check(rows.contiguous().cuda(), -torch.arange(m).float()[None].cuda() * 0.37, 2 * m)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_masks(dtype):
    say("masks", dtype)
    gen = torch.Generator().manual_seed(2)
    low = torch.finfo(dtype).min
    for v in (100, 20000):
        logits, scores = draw(gen, 6, 4, v, dtype)
        keep = torch.rand(v, generator=gen).cuda() < 0.02
        keep[3] = True
        logits[0].masked_fill_(~keep, -math.inf)
        logits[1].masked_fill_(~keep, low)
        logits[2, :, 4:] = -math.inf          # 16 candidates
        logits[2, 1] = -math.inf              # a beam with none
        logits[3] = -math.inf                 # a request with none
        logits[4, :3] = low                   # nothing but the lowest value: all equal
        logits[5, :, ::2] = math.nan
        scores[0, 2] = -math.inf
        scores[2, 3] = -math.inf
        check(logits, scores, 8)
        finished = torch.zeros(6, 4, dtype=torch.bool, device="cuda")
        finished[0, 1] = finished[2, 1] = finished[3, 0] = finished[1, 3] = True
        finished[2, 3] = True                 # finished and dead
        logits[1, 3] = math.nan               # the logits of a finished beam do not count
        check(logits, scores, 8, finished, pad=2)


def test_rows_at_any_stride_and_alignment():
    say("strides")
    gen = torch.Generator().manual_seed(3)
    for dtype in (BF, F32):
        for shift, width in itertools.product((0, 1, 3, 7), (1003, 1008, 1001)):
            big = (torch.randn(8 * width + 8, generator=gen) * 3).to(dtype).cuda()
            rows = big[shift:shift + 8 * width].view(2, 4, width)[:, :, :1001]
            check(rows, (-10 * torch.rand(2, 4, generator=gen)).cuda(), 8)


def test_calls():
    say("calls")
    gen = torch.Generator().manual_seed(4)
    logits, scores = draw(gen, 3, 4, 9000, BF)
    want = [x.clone() for x in select(logits, scores, 4)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = select(logits, scores, 4)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = select(logits, scores, 4, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got[1], want[1])
    out = select(logits, scores, 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssq.ssq_beam_select(logits, scores, *out)
    for _ in range(3):
        for x in out:
            x.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    select(logits[:0], scores[:0], 4)  # no request


def test_select_refusals():
    x, s = torch.zeros(2, 4, 50, device="cuda"), torch.zeros(2, 4, device="cuda")
    for call in (lambda: select(x, s, 9), lambda: select(x, s, 4, pad=50), lambda: select(x, s, 4, pad=-1),
                 lambda: select(x[:, :, :0], s, 4), lambda: select(torch.zeros(1, 33, 5, device="cuda"), torch.zeros(1, 33, device="cuda"), 4),
                 lambda: select(x[:, :1].expand(2, 4, 50), s, 4),
                 lambda: select(x, s, 4, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((ssq.SsqError, ValueError)):
            call()
    for call in (lambda: select(x[..., ::2], s, 4), lambda: select(x.double(), s, 4), lambda: select(x, s[:1], 4),
                 lambda: select(x, s.double(), 4), lambda: select(x, s, 4, finished=s), lambda: select(x.cpu(), s, 4)):
        with pytest.raises(ValueError):
            call()


# ----------------------------------------------------------------------------- states follow

KINDS = [("mamba2", f) for f in ("fp32", "int8_sym", "int8_asym", "int4_sym", "int4_asym")] + \
        [("delta", f) for f in ("fp32", "int8_asym", "int4_sym", "damp")]


def filled(kind, fmt, batch, H=3, P=48, seed=0):
    desc = ssq.make_desc(ssq.SSQ_MAMBA2, fmt, batch, H, P) if kind == "mamba2" else ssq.make_desc(ssq.SSQ_DELTA, fmt, batch, 2, 128)
    storage = torch.zeros(ssq.ssq_state_bytes(desc), dtype=torch.uint8, device="cuda")
    st = ssq.ssq_alloc_state(desc, storage)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    storage.random_(0, 256, generator=gen)
    return st


def parts_of(st, storage):
    """The arrays of a state by sequence, as bytes, and the token counter."""
    lay, d = st.layout, st.desc
    rows = int(lay.rows)
    low = rows // 128 * (128 - ssq.SSQ_DAMP_NHI) if d.format == ssq.SSQ_DAMP else rows
    spans = [(0, low * lay.row_bytes)]
    spans += [(o, 4 * low) for o in (lay.scale_offset, lay.zero_offset) if o]
    if lay.hi_offset:
        spans.append((lay.hi_offset, (rows - low) * 256))
    return [storage[a:a + n].view(d.batch, -1) for a, n in spans]


def check_reorder(states, parents):
    before = [s.storage.clone() for s in states]
    ssq.ssq_state_reorder(states if len(states) > 1 else states[0], parents)
    groups, beams = parents.shape
    own = torch.arange(beams, device="cuda")
    p = torch.where((parents < 0) | (parents >= beams), own, parents).long()
    frm = (p + beams * torch.arange(groups, device="cuda")[:, None]).view(-1)
    for s, b in zip(states, before):
        want = b.clone()
        for x, y in zip(parts_of(s, want), parts_of(s, b)):
            x.copy_(y[frm])
        assert torch.equal(s.storage, want), (s.desc.kind, s.desc.format, beams)


@pytest.mark.parametrize("kind,fmt", KINDS)
def test_reorder(kind, fmt):
    say("reorder", kind, fmt)
    gen = torch.Generator(device="cuda").manual_seed(5)
    for groups, beams in ((1, 2), (3, 3), (2, 5), (4, 4), (2, 8), (1, 16), (1, 17), (1, 32), (3, 1)):
        st = filled(kind, fmt, groups * beams, seed=beams)
        i = torch.arange(beams, device="cuda").repeat(groups, 1)
        for p in (torch.randint(0, beams, (groups, beams), device="cuda", generator=gen), i, i.flip(1), i * 0, i * 0 + beams - 1,
                  torch.where(i % 2 == 0, -1, beams), i - 1):
            check_reorder([st], p.to(torch.int32))


def test_reorder_of_all_layers():
    say("layers")
    gen = torch.Generator(device="cuda").manual_seed(6)
    states = [filled(*KINDS[i % len(KINDS)], 8, H=1 + i % 5, P=16 * (1 + i % 4), seed=i) for i in range(70)]
    check_reorder(states, torch.randint(0, 4, (2, 4), device="cuda", generator=gen).to(torch.int32))
    ssq.ssq_state_reorder([], torch.zeros(2, 4, dtype=torch.int32, device="cuda"))


def test_reorder_in_a_graph_and_on_a_stream():
    say("reorder graph")
    states = [filled("mamba2", "int4_asym", 8, seed=i) for i in range(3)]
    begin = [s.storage.clone() for s in states]
    parents = torch.tensor([[1, 1, 0, 2], [3, 0, 0, 3]], dtype=torch.int32, device="cuda")
    check_reorder(states, parents)
    want = [s.storage.clone() for s in states]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssq.ssq_state_reorder(states, parents)
    for _ in range(3):
        for s, b in zip(states, begin):
            s.storage.copy_(b)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s.storage, w) for s, w in zip(states, want))
    for s, b in zip(states, begin):
        s.storage.copy_(b)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ssq.ssq_state_reorder(states, parents, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(s.storage, w) for s, w in zip(states, want))


def test_reorder_refusals():
    st, other = filled("mamba2", "fp32", 8), filled("mamba2", "fp32", 4)
    p = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    before = st.storage.clone()
    for call in (lambda: ssq.ssq_state_reorder([st, st], p), lambda: ssq.ssq_state_reorder([st, other], p),
                 lambda: ssq.ssq_state_reorder(st, p[:1]), lambda: ssq.ssq_state_reorder(st, p.long()),
                 lambda: ssq.ssq_state_reorder(st, p.cpu()), lambda: ssq.ssq_state_reorder(st, p.view(-1)),
                 lambda: ssq.ssq_state_reorder(st, torch.zeros(4, 4, dtype=torch.int32, device="cuda")[::2])):
        with pytest.raises((ssq.SsqError, ValueError)):
            call()
    torch.cuda.synchronize()
    assert torch.equal(st.storage, before)


@pytest.mark.parametrize("m,v,n", [(32, 131071, 64), (32, 70000, 17), (20, 40000, 33), (17, 9000, 34), (16, 300, 32), (32, 5, 64)])
def test_many_beams(m, v, n):
    """Waves with two beams, lists longer than 16, dead and finished beams among them, and ties."""
    say("many beams", m, v, n)
    gen = torch.Generator().manual_seed(m + v)
    logits, scores = draw(gen, 2, m, v, BF)
    logits[1] = torch.randint(-2, 3, (m, v), generator=gen).to(BF).cuda()  # ties between tokens
    logits[1, 3:] = logits[1, 2]                                           # and between beams
    scores[1] = -1.5
    for dead in (m - 1, 0, m // 2):
        scores[0, dead] = -math.inf
        finished = torch.zeros(2, m, dtype=torch.bool, device="cuda")
        finished[:, 1::5] = True
        check(logits, scores, n)
        check(logits, scores, n, finished, pad=4)
    scores[0] = -math.inf
    scores[0, m - 2] = 0.0
    check(logits, scores, n)
