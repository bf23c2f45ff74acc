"""GPU: the gated recurrence, the group norm and the moves of states as a program uses them together; every way in which a
scan's call is split; tensors and states past 4 GiB; graphs that share a workspace.

Tolerances: the references' own bounds (tests/gated_ref.py, tests/norm_ref.py); a later operator is compared on what the earlier
one really left."""
import random
import sys

import pytest
import torch

from tests import gated_ref as ref
from tests import norm_ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mamba_decode_amd as ssq
    from tests.test_gpu_gated import case, check, cu_of, state_of, values_of

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def index(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_serving_a_layer(dtype):
    """Two prefixes are read into a pool, forked to the requests' slots, go on with prompts of their own, then token by token,
    their beams reordered, the pool compacted and freed in between; the outputs are normalised and gated."""
    say("serving", dtype)
    gen = torch.Generator().manual_seed(1)
    r = random.Random(1)
    C, groups, slots = 264, 3, 8
    x, g = ref.inputs(gen, 400, C, dtype, 1)
    z = torch.randn(400, C, generator=gen).to(dtype)
    xd, gd, zd = (t.cuda() for t in (x, g, z))
    w, b = torch.randn(groups, C // groups, generator=gen) * 0.2 + 1, torch.randn(groups, C // groups, generator=gen) * 0.1
    how = dict(gate=1, input=2)
    layers = 2  # the same layer twice: the moves go over both
    prefixes = [state_of(torch.zeros(2, C)) for _ in range(layers)]
    pool = [state_of(torch.randn(slots, C, generator=gen)) for _ in range(layers)]
    used = 0
    path = {}  # the tokens that each slot has read

    def rows(n):
        nonlocal used
        s = list(range(used, used + n))
        used += n
        return s

    def close(paths_of_rows, o, rows_used):
        """o of the rows, each behind its path, and the gated norm of it."""
        for i, p in zip(range(len(rows_used)), paths_of_rows):
            h, m, e = ref.scan(x[p], g[p], torch.zeros(C), 1, 2)
            check(o[i:i + 1], h[-1:], e[-1:], dtype, ("o", rows_used[i]))
        y = torch.empty_like(o)
        shape = (len(rows_used), groups, C // groups)
        ssq.ssq_group_norm(o.view(shape), y.view(shape), weight=w.cuda(), bias=b.cuda(), z=zd[rows_used].view(shape), act=ssq.SSQ_ACT_GATE_OUTPUT)
        want, bound = norm_ref.norm(o.cpu().view(shape), z[rows_used].view(shape), w, b, 1, True, 1e-5)
        check(y.view(shape), want["y"], bound["y"], dtype, "y")

    a = [rows(33), rows(50)]
    o = torch.empty(83, C, dtype=dtype, device="cuda")
    for st in prefixes:
        ssq.ssq_gated_scan(st, xd[:83], gd[:83], o, cu_of([33, 50]), fresh=index([1, 1]).to(torch.uint8), **how)
    close(a, o[[32, 82]], [p[-1] for p in a])
    live = {0: 0, 3: 0, 5: 1, 6: 1}
    ssq.ssq_state_move(pool, index(list(live) + [1, 2, 4, 7]), index(list(live.values()) + [-1] * 4), sources=prefixes)
    path = {s: list(a[p]) for s, p in live.items()}
    own = {s: rows(r.choice((1, 17, 40))) for s in live}
    order = list(live)
    flat = [t for s in order for t in own[s]]
    o = torch.empty(len(flat), C, dtype=dtype, device="cuda")
    for st in pool:
        ssq.ssq_gated_scan(st, xd[flat], gd[flat], o, cu_of([len(own[s]) for s in order]), slots=index(order), **how)
    ends = torch.tensor([len(own[s]) for s in order]).cumsum(0) - 1
    for s in order:
        path[s] += own[s]
    close([path[s] for s in order], o[ends.cuda()], [own[s][-1] for s in order])
    ssq.ssq_state_move(pool, index([0, 1, 2, 3, 4, 5, 6]), index([0, 3, 5, 6, -1, -1, -1]))  # compacted in their order
    path = {i: path[s] for i, s in enumerate(order)}
    for step in range(3):
        new = rows(4)
        o = torch.empty(4, C, dtype=dtype, device="cuda")
        for st in pool:
            ssq.ssq_gated_step(st, xd[new], gd[new], o, slots=index([0, 1, 2, 3]), **how)
        for i in range(4):
            path[i] = path[i] + [new[i]]
        close([path[i] for i in range(4)], o, new)
        parents = [[r.randrange(4) for _ in range(4)], [0, 1, 2, 3]]
        ssq.ssq_state_reorder(pool, index(parents))
        path = {i: path[parents[0][i]] for i in range(4)}
    for st in pool:
        got = values_of(st)
        for i in range(4):
            h, m, e = ref.scan(x[path[i]], g[path[i]], torch.zeros(C), 1, 2)
            check(got[i][None], h[-1:], e[-1:], F32, ("slot", i))
        assert (got[4:7] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_training_a_layer(dtype):
    """Scan, norm with its gate, both gradients."""
    say("training", dtype)
    gen = torch.Generator().manual_seed(2)
    C, groups, lens = 144, 2, [90, 0, 333, 1]
    T = sum(lens)
    shape = (T, groups, C // groups)
    x, g = ref.inputs(gen, T, C, dtype, 0)
    z, dy = (torch.randn(shape, generator=gen).to(dtype) for _ in range(2))
    w, b = torch.randn(shape[1:], generator=gen) * 0.2 + 1, torch.randn(shape[1:], generator=gen) * 0.1
    xd, gd, zd, dyd, wd, bd = (t.cuda() for t in (x, g, z, dy, w, b))
    o, do, dx, dg = (torch.empty_like(xd) for _ in range(4))
    y, dz = torch.empty_like(zd), torch.empty_like(zd)
    dw, db, dfirst = torch.empty_like(wd), torch.empty_like(bd), torch.empty(len(lens), C, device="cuda")
    ck = torch.empty(ssq.ssq_gated_checkpoint_rows(len(lens), T), C, device="cuda")
    how = dict(weight=wd, bias=bd, z=zd, act=ssq.SSQ_ACT_GATE_INPUT, center=False)
    ssq.ssq_gated_scan(None, xd, gd, o, cu_of(lens), input=2, checkpoints=ck)
    ssq.ssq_group_norm(o.view(shape), y, **how)
    ssq.ssq_group_norm_backward(dyd, o.view(shape), do.view(shape), dz=dz, dweight=dw, dbias=db, **how)
    ssq.ssq_gated_scan_backward(ck, xd, gd, do, dx, dg, cu_of(lens), input=2, dfirst=dfirst)
    want, bound = norm_ref.norm(o.cpu().view(shape), z, w, b, 2, False, 1e-5, dy)
    for k, t in dict(y=y, dx=do.view(shape), dz=dz, dweight=dw, dbias=db).items():
        check(t, want[k], bound[k], F32 if k in ("dweight", "dbias") else dtype, k)
    at = 0
    for i, n in enumerate(lens):
        s = slice(at, at + n)
        h, m, e = ref.scan(x[s], g[s], torch.zeros(C), 0, 2)
        check(o[s], h[1:], e[1:], dtype, ("o", i))
        grads, bounds = ref.gradient(x[s], g[s], do.cpu()[s], torch.zeros(C), torch.zeros(C), 0, 2)
        for t, v, k, d in zip((dx[s], dg[s], dfirst[i]), grads, bounds, (dtype, dtype, F32)):
            check(t, v, k, d, i)
        at += n


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,channels", [(310, 8), (70, 520), (64, 640), (50, 256), (24, 1032), (3, 2056), (1, 4200), (65, 264), (2, 1160)])
def test_every_way_of_splitting(dtype, n, channels):
    """Rows of 256, 128 and 64 bytes, whole sequences in the order of their lengths and not, with empty and skipped ones."""
    say("splits", dtype, n, channels)
    r = random.Random(n)
    lens = [r.choice((0, 1, 5, 16, 40)) for _ in range(n)]
    lens[n // 2] = 300
    slots = r.sample(range(n + 2), n)
    if n > 2:
        slots[1], slots[n - 1] = -1, n + 2
    case(dtype, 0, 2, channels, lens, tail=2, slots=slots, fresh=[i % 3 == 0 for i in range(n)], batch=n + 2, seed=n)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens,channels", [([1200, 0, 2000], 40), ([700, 1300, 64, 1], 24), ([0, 2100], 136), ([1100], 1000)])
def test_parts(dtype, lens, channels):
    say("parts", dtype, lens, channels)
    n = len(lens)
    assert ssq.ssq_gated_workspace(channels, n, sum(lens) + 1) > 0
    case(dtype, 1, 1, channels, lens, tail=1, slots=list(range(n, 0, -1)), fresh=[i % 2 for i in range(n)], batch=n + 1, seed=n)
    case(dtype, 0, 2, channels, lens, seed=n, slices=True)


@pytest.mark.parametrize("dtype,lens,channels", [(BF, [1100], 4104), (F32, [1030], 2056), (F32, [2700, 0, 1500], 1080), (BF, [2700, 1], 2600)])
def test_parts_of_the_gradient_alone(dtype, lens, channels):
    """Sizes whose scan takes sequences whole and whose gradient takes them in parts."""
    say("parts of the gradient", dtype, lens, channels)
    n = len(lens)
    assert ssq.ssq_gated_workspace(channels, n, sum(lens) + 3) > 0
    case(dtype, 0, 1, channels, lens, tail=3, slots=list(range(n, 0, -1)), fresh=[i % 2 for i in range(n)], batch=n + 1, seed=n)


def test_past_4_gib():
    """Rows that lie 2^18 elements apart, so that the last ones begin behind 2^32 bytes."""
    say("past 4 GiB")
    gen = torch.Generator().manual_seed(3)
    T, C, wide = 8300, 40, 1 << 18
    x, g = ref.inputs(gen, T, C, BF, 0)
    do = torch.randn(T, C, generator=gen).to(BF)
    big = torch.zeros(T, wide, dtype=BF, device="cuda")
    dev = [big[:, 64 * i: 64 * i + C] for i in range(6)]
    for t, v in zip(dev, (x, g, do)):
        t.copy_(v)
    lens = [300, 8000]
    ck = torch.empty(ssq.ssq_gated_checkpoint_rows(2, T), C, device="cuda")
    ssq.ssq_gated_scan(None, dev[0], dev[1], dev[3], cu_of(lens), input=1, checkpoints=ck)
    ssq.ssq_gated_scan_backward(ck, dev[0], dev[1], dev[2], dev[4], dev[5], cu_of(lens), input=1)
    s = slice(300, T)
    h, m, e = ref.scan(x[s], g[s], torch.zeros(C), 0, 1)
    check(dev[3][s], h[1:], e[1:], BF, "o")
    grads, bounds = ref.gradient(x[s], g[s], do[s], torch.zeros(C), torch.zeros(C), 0, 1)
    check(dev[4][s], grads[0], bounds[0], BF, "dx")
    check(dev[5][s], grads[1], bounds[1], BF, "dg")
    st = state_of(torch.zeros(T, C))
    ssq.ssq_gated_step(st, dev[0], dev[1], dev[3], input=1)
    h, m, e = ref.scan(x[-1:], g[-1:], torch.zeros(C), 0, 1)
    check(dev[3][-1:], h[1:], e[1:], BF, "token")
    x3, z3 = x.view(T, 1, C), g.view(T, 1, C)
    n3 = [t.unflatten(1, (1, C)) for t in dev]
    w = torch.ones(1, C, device="cuda")
    dw = torch.empty_like(w)
    ssq.ssq_group_norm(n3[0], n3[3], weight=w, z=n3[1], act=1)
    ssq.ssq_group_norm_backward(n3[2], n3[0], n3[4], weight=w, z=n3[1], dz=n3[5], dweight=dw, act=1)
    want, bound = norm_ref.norm(x3, z3, w.cpu(), None, 1, True, 1e-5, do.view(T, 1, C))
    for k, t in dict(y=n3[3], dx=n3[4], dz=n3[5]).items():
        check(t, want[k], bound[k], BF, k)
    check(dw, want["dweight"], bound["dweight"], F32, "dweight")
    del big, dev, n3
    st = ssq.ssq_alloc_state(ssq.make_desc(ssq.SSQ_GATED, "fp32", 1100, 1, 1, 1 << 20), torch.empty(1100 << 22, dtype=torch.uint8, device="cuda"))
    rows = st.regions()[0]
    for i in (3, 500, 1099):
        rows[i] = i
    ssq.ssq_state_move(st, index([1098, 1, 1099]), index([3, 1099, -1]))
    assert (rows[1098] == 3).all() and (rows[1] == 1099).all() and (rows[1099] == 0).all() and (rows[500] == 500).all()


def test_graphs_that_share_a_workspace():
    """Two captured calls with one workspace, replayed in turn with eager calls between."""
    say("shared workspace")
    gen = torch.Generator().manual_seed(4)
    C, T = 40, 3000
    ws = torch.empty(max(ssq.ssq_gated_workspace(C, 1, T), ssq.ssq_group_norm_workspace(2, 64, 500)), dtype=torch.uint8, device="cuda")
    x, g = (t.cuda() for t in ref.inputs(gen, T, C, BF, 0))
    do = torch.randn(T, C, generator=gen).to(BF).cuda()
    o, dx, dg = (torch.zeros_like(x) for _ in range(3))
    ck = torch.empty(ssq.ssq_gated_checkpoint_rows(1, T), C, device="cuda")
    n = torch.randn(500, 2, 64, generator=gen).cuda()
    dn, dw, db = torch.empty_like(n), torch.empty(2, 64, device="cuda"), torch.empty(2, 64, device="cuda")
    cu = cu_of([T])

    def scan():
        ssq.ssq_gated_scan(None, x, g, o, cu, checkpoints=ck, workspace=ws)
        ssq.ssq_gated_scan_backward(ck, x, g, do, dx, dg, cu, workspace=ws)

    def norm():
        ssq.ssq_group_norm_backward(n, n, dn, dweight=dw, dbias=db, workspace=ws)

    outs = (o, dx, dg, dn, dw, db)
    scan(), norm()
    want = [t.clone() for t in outs]
    graphs = []
    for f in (scan, norm):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f()
        graphs.append(graph)
    for _ in range(3):
        for t in outs:
            t.fill_(7)
        torch.cuda.synchronize()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        norm(), scan()


@pytest.mark.parametrize("gate", [0, 1])
def test_long_decays_do_not_drift(gate):
    """A channel that keeps nearly everything over 20000 tokens: the distance from 64 bits, relative to the state's size, stays
    below what 2^-24 a token in one direction would leave, by a factor of 20."""
    say("drift", gate)
    gen = torch.Generator().manual_seed(5)
    T, C = 20000, 8
    x = torch.randn(T, C, generator=gen)
    g = torch.full((T, C), -1e-5 if gate == 0 else 11.5)
    o = torch.empty_like(x).cuda()
    ssq.ssq_gated_scan(None, x.cuda(), g.cuda(), o, cu_of([T]), gate=gate)
    h, m, e = ref.scan(x, g, torch.zeros(C), gate, 0)
    off = (o.cpu().double() - h[1:]).abs().max(0).values / m[-1]
    assert (off < T * 2.0 ** -24 / 20).all(), off
