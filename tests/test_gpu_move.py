"""GPU: moves between sequences of states, byte for byte against the same moves one after the other."""
import random
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

from tests.test_gpu_beam import KINDS, parts_of  # noqa: E402

if torch.cuda.is_available():
    import mamba_decode_amd as ssq

ALL = KINDS + [("gated", "fp32")]


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def filled(kind, fmt, batch, H=3, P=48, seed=0):
    desc = {"mamba2": lambda: ssq.make_desc(ssq.SSQ_MAMBA2, fmt, batch, H, P), "delta": lambda: ssq.make_desc(ssq.SSQ_DELTA, fmt, batch, 2, 128),
            "gated": lambda: ssq.make_desc(ssq.SSQ_GATED, "fp32", batch, 1, 1, 8 * H * P)}[kind]()
    storage = torch.zeros(ssq.ssq_state_bytes(desc), dtype=torch.uint8, device="cuda")
    st = ssq.ssq_alloc_state(desc, storage)
    storage.random_(0, 256, generator=torch.Generator(device="cuda").manual_seed(seed))
    return st


def rows_of(st, storage):
    if st.desc.kind == ssq.SSQ_GATED:
        return [storage[: st.rows * st.layout.row_bytes].view(st.desc.batch, -1)]
    return parts_of(st, storage)


def check(states, moves, sources=None):
    want, pools = [s.storage.clone() for s in states], [s.storage.clone() for s in sources or []]
    batch, many = states[0].desc.batch, (sources or states)[0].desc.batch
    for l, s in enumerate(states):
        here = rows_of(s, want[l])
        there = rows_of(sources[l], pools[l]) if sources else here
        for to, frm in moves:
            if 0 <= to < batch and -1 <= frm < many:
                for x, y in zip(here, there):
                    x[to] = y[frm] if frm >= 0 else 0
    to, frm = (torch.tensor([m[i] for m in moves], dtype=torch.int32, device="cuda") for i in (0, 1))
    ssq.ssq_state_move(states if len(states) > 1 else states[0], to, frm, sources=sources if sources is None or len(sources) > 1 else sources[0])
    for s, w in zip(states, want):
        assert torch.equal(s.storage, w), (s.desc.kind, s.desc.format, moves[:8])
    for s, p in zip(sources or [], pools):
        assert torch.equal(s.storage, p)


@pytest.mark.parametrize("kind,fmt", ALL)
def test_moves(kind, fmt):
    say("moves", kind, fmt)
    st = filled(kind, fmt, 12, seed=1)
    for moves in ([(0, 5)], [(i, 0) for i in range(1, 12)], [(3, -1), (7, -1)], [(1, 2), (3, 4), (5, -1), (6, 4)],
                  [(4, 4)], [(-1, 3), (12, 2), (2, 12), (2, -2), (5, 6), (1 << 30, 1), (1, -(1 << 31))], []):
        check([st], moves)


@pytest.mark.parametrize("kind,fmt", [("mamba2", "int4_asym"), ("gated", "fp32"), ("delta", "damp")])
def test_moves_that_depend_on_each_other(kind, fmt):
    """Chains, exchanges through a third place, compaction in order, sources freed later, a place written twice."""
    say("chains", kind, fmt)
    for n in (9, 40):
        last = n - 1
        for moves in ([(0, 1), (1, 2), (2, 3)], [(3, 2), (2, 1), (1, 0)], [(last, 0), (0, 1), (1, last)], [(i, i + 1) for i in range(last)],
                      [(i + 1, i) for i in range(last)], [(1, 0), (0, -1)], [(0, -1), (1, 0)], [(5, 1), (5, 2), (5, 5), (6, 5)],
                      [(i, j) for i, j in enumerate(sorted(random.Random(n).sample(range(n), n // 2)))] + [(i, -1) for i in range(n // 2, n)],
                      [(2, 2), (3, 2), (2, -1), (4, 2)]):
            check([filled(kind, fmt, n, seed=n)], moves)


def test_drawn_moves():
    say("drawn")
    r = random.Random(3)
    for i in range(40):
        kind, fmt = ALL[i % len(ALL)]
        b = r.choice((1, 2, 5, 17, 33))
        st = filled(kind, fmt, b, H=1 + i % 4, P=16 * (1 + i % 3), seed=i)
        n = r.choice((1, 3, b, 2 * b, 70, 300))
        if i % 3 == 0:  # disjoint places
            order = r.sample(range(b), b)
            half = max(1, b // 2)
            moves = [(t, r.choice(order[half:] + [-1])) for t in order[:half]]
        else:
            moves = [(r.randrange(-1, b + 1), r.randrange(-2, b + 1)) for _ in range(n)]
        check([st], moves)


def test_all_layers_and_another_pool():
    say("layers")
    r = random.Random(4)
    mk = lambda b, s: [filled(*ALL[i % len(ALL)], b, H=1 + i % 5, P=16 * (1 + i % 4), seed=s + i) for i in range(50)]  # noqa: E731
    states, pool = mk(8, 0), mk(5, 100)
    check(states, [(r.randrange(8), r.randrange(-1, 5)) for _ in range(12)], sources=pool)
    check(states, [(i, (i * 3) % 5) for i in range(8)], sources=pool)
    check(states, [(7, 0), (6, 1), (5, -1)])
    check(states, [(i, i + 1) for i in range(7)])
    check([states[0]], [(1, 4)], sources=[pool[0]])
    ssq.ssq_state_move([], torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"))


def test_many_moves_and_sequences():
    say("many")
    r = random.Random(5)
    st = filled("gated", "fp32", 5000, H=1, P=1)
    check([st], [(i, 4999 - i) for i in range(2000)])
    check([st], [(r.randrange(5000), r.randrange(-1, 5000)) for _ in range(400)])
    big = filled("gated", "fp32", (1 << 18) + 100, H=1, P=1)  # more sequences than the parallel form keeps track of
    check([big], [(0, 1 << 18), ((1 << 18) + 99, 0), (5, -1), (6, 5)])


def test_in_a_graph_and_on_a_stream():
    say("graph")
    states = [filled("mamba2", "int4_asym", 8, seed=i) for i in range(3)]
    begin = [s.storage.clone() for s in states]
    to, frm = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([1, 2, 5, 6], [0, 0, -1, 5]))
    ssq.ssq_state_move(states, to, frm)
    want = [s.storage.clone() for s in states]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssq.ssq_state_move(states, to, frm)
    for way in (graph.replay, graph.replay, graph.replay, lambda: ssq.ssq_state_move(states, to, frm, stream=torch.cuda.Stream())):
        for s, b in zip(states, begin):
            s.storage.copy_(b)
        torch.cuda.synchronize()
        way()
        torch.cuda.synchronize()
        assert all(torch.equal(s.storage, w) for s, w in zip(states, want))


def test_counters_and_rounding_stay():
    say("counters")
    st = filled("mamba2", "int8_asym", 4)
    ssq.ssq_set_rounding(st, ssq.SSQ_ROUND_STOCHASTIC, seed=5, step=77)
    check([st], [(0, 1), (2, -1)])
    assert ssq.ssq_get_rounding(st) == (ssq.SSQ_ROUND_STOCHASTIC, 5, 77)


def test_refusals():
    say("refusals")
    st, other, less = filled("mamba2", "fp32", 8), filled("mamba2", "fp32", 4), filled("mamba2", "fp32", 8, H=2)
    quant, gated = filled("mamba2", "int8_sym", 8), filled("gated", "fp32", 8)
    i = torch.zeros(4, dtype=torch.int32, device="cuda")
    before = st.storage.clone()
    same = ssq.ssq_alloc_state(st.desc, torch.zeros_like(st.storage))
    for a, kw in (((st, i, i[:3]), {}), ((st, i.long(), i), {}), ((st, i.cpu(), i), {}), ((st, i.view(2, 2), i), {}), (([st, st], i, i), {}),
                  (([st, other], i, i), {}), ((st, i, i), dict(sources=st)), ((st, i, i), dict(sources=quant)), ((st, i, i), dict(sources=gated)),
                  ((st, i, i), dict(sources=less)), ((st, i, i), dict(sources=[same, same])), (([st, less], i, i), dict(sources=[same, other])),
                  ((st, i, i), dict(sources=[])), ((st, torch.zeros(65536, dtype=torch.int32, device="cuda"), torch.zeros(65536, dtype=torch.int32, device="cuda")), {}),
                  ((st, i, i), dict(stream=type("S", (), dict(cuda_stream=0, device=torch.device("cuda", 1)))()))):
        with pytest.raises((ssq.SsqError, ValueError, TypeError)):
            ssq.ssq_state_move(*a, **kw)
    torch.cuda.synchronize()
    assert torch.equal(st.storage, before)
