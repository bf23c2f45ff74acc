"""GPU: the group norm with an activation and its gradient against the formulas in 64 bits.

Tolerances: the reference's own bounds of fp32 evaluation (tests/norm_ref.py) and half a step of the outputs' type."""
import itertools
import sys

import pytest
import torch

from tests import norm_ref as ref
from tests.gated_ref import rounding

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mamba_decode_amd as ssq

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
SENTINEL = 7.0
MODES = list(itertools.product((0, 1, 2), (True, False)))


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def check(got, want, bound, dtype, where):
    bad = ~((got.cpu().double() - want).abs() <= bound + rounding(dtype, want.abs() + bound))
    assert not bad.any(), f"{where}: off at {bad.nonzero()[:4].tolist()}, {int(bad.sum())} of {bad.numel()}"


def sliced(t):
    """The same values as a slice of wider rows."""
    big = torch.full((t.shape[0], t.shape[1] + 2, t.shape[2]), SENTINEL, dtype=t.dtype, device="cuda")
    big[:, 1:-1] = t
    return big[:, 1:-1]


def inputs(gen, shape, dtype, act, offset=1.0):
    x = (torch.randn(shape, generator=gen) * 1.5 + offset * torch.randn(shape[1:], generator=gen)).to(dtype)
    z = None if act == ref.SILU else torch.randn(shape, generator=gen).to(dtype)
    w, b = torch.randn(shape[1:], generator=gen) * 0.3 + 1, torch.randn(shape[1:], generator=gen) * 0.2
    return x, z, w, b, torch.randn(shape, generator=gen).to(dtype)


def run(x, z, w, b, dy, act, center, eps=1e-5, place=lambda t: t.cuda(), params=(True, True), **kw):
    x, z, dy = (None if t is None else place(t) for t in (x, z, dy))
    w, b = (None if t is None else t.cuda() for t in (w, b))
    y, dx = (place(torch.full(x.shape, SENTINEL, dtype=x.dtype)) for _ in range(2))
    dz = None if z is None else place(torch.full(x.shape, SENTINEL, dtype=x.dtype))
    dw, db = (torch.full(x.shape[1:], SENTINEL, device="cuda") if p else None for p in params)
    how = dict(weight=w, bias=b, z=z, act=act, center=center, eps=eps, **kw)
    ssq.ssq_group_norm(x, y, **how)
    ssq.ssq_group_norm_backward(dy, x, dx, dz=dz, dweight=dw, dbias=db, **how)
    return dict(y=y, dx=dx, dz=dz, dweight=dw, dbias=db)


def case(shape, dtype, act, center, seed=0, affine=(True, True), **kw):
    gen = torch.Generator().manual_seed(seed)
    x, z, w, b, dy = inputs(gen, shape, dtype, act)
    w, b = (t if a else None for t, a in zip((w, b), affine))
    got = run(x, z, w, b, dy, act, center, **kw)
    want, bound = ref.norm(x, z, w, b, act, center, kw.get("eps", 1e-5), dy)
    for k, v in want.items():
        if got[k] is not None:
            check(got[k], v, bound[k], F32 if k in ("dweight", "dbias") else dtype, (k, shape, dtype, act, center))


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("act,center", MODES)
def test_modes(dtype, act, center):
    say("modes", dtype, act, center)
    case((37, 3, 72), dtype, act, center, seed=act)
    case((5, 2, 1000), dtype, act, center, seed=act, place=sliced)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("groups,width", [(1, 8), (7, 8), (5, 16), (3, 24), (9, 32), (2, 40), (32, 64), (3, 128), (1, 136), (2, 256), (3, 264),
                                          (2, 512), (1, 520), (2, 1024), (1, 1032), (1, 2048), (3, 2056), (1, 4104), (2, 8192), (1, 16384)])
def test_widths(dtype, groups, width):
    say("widths", dtype, groups, width)
    for tokens in (1, 6):
        case((tokens, groups, width), dtype, 2, True, seed=width)
        case((tokens, groups, width), dtype, 0, False, seed=width)


@pytest.mark.parametrize("tokens,groups,width", [(1000, 1, 8), (700, 5, 64), (515, 32, 64), (300, 2, 1024), (129, 1, 4104), (2500, 3, 16), (70, 1, 16384)])
def test_many_tokens(tokens, groups, width):
    say("tokens", tokens, groups, width)
    case((tokens, groups, width), BF, 1, True, seed=tokens)
    case((tokens, groups, width), F32, 2, False, seed=tokens)


@pytest.mark.parametrize("act,center", MODES)
def test_without_parameters(act, center):
    say("no parameters", act, center)
    for affine, params in (((False, False), (True, True)), ((True, False), (False, True)), ((False, True), (True, False)), ((True, True), (False, False))):
        case((9, 3, 136), F32, act, center, seed=1, affine=affine, params=params)


@pytest.mark.parametrize("center", [True, False])
def test_rows_without_spread(center):
    """Constant groups, zero groups, a group far from zero, gates of the type's lowest value."""
    say("no spread", center)
    gen = torch.Generator().manual_seed(4)
    for dtype in (BF, F32):
        for act in (0, 1, 2):
            x, z, w, b, dy = inputs(gen, (8, 4, 200), dtype, act)
            x[0], x[1, 1], x[2, 2] = 0, 3.0, -0.5
            x[3] = x[3] * 2.0 ** -10 + 100
            if z is not None:
                z[4], z[5, :, ::3] = torch.finfo(dtype).min, torch.finfo(dtype).min
                z[6], z[7, 1] = 0, 60.0
            got = run(x, z, w, b, dy, act, center, eps=1e-3)
            want, bound = ref.norm(x, z, w, b, act, center, 1e-3, dy)
            for k, v in want.items():
                check(got[k], v, torch.nan_to_num(bound[k], nan=0.0, posinf=0.0) if k in ("y", "dz") else bound[k],
                      F32 if k in ("dweight", "dbias") else dtype, (k, dtype, act, center))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_nothing_else_is_read_or_written(dtype):
    """NaN in one group of one token reaches no other group of any token, nor other channels' parameters."""
    say("NaN", dtype)
    gen = torch.Generator().manual_seed(5)
    for act, shape in ((2, (40, 5, 64)), (1, (33, 2, 2056)), (0, (21, 9, 8))):
        x, z, w, b, dy = inputs(gen, shape, dtype, act)
        clean = run(x, z, w, b, dy, act, True, place=sliced)
        x[7, 1, 3] = torch.nan
        dirty = run(x, z, w, b, dy, act, True, place=sliced)
        keep = torch.ones(shape[:2], dtype=torch.bool, device="cuda")
        keep[7, 1] = False
        for k in ("y", "dx", "dz"):
            if clean[k] is not None:
                assert torch.equal(clean[k][keep], dirty[k][keep]), k
                whole = clean[k]._base
                assert (whole[:, 0] == SENTINEL).all() and (whole[:, -1] == SENTINEL).all()
        other = torch.arange(shape[1]) != 1
        for k in ("dweight", "dbias"):
            assert torch.equal(clean[k][other.cuda()], dirty[k][other.cuda()]), k


@pytest.mark.parametrize("act,center", MODES)
def test_gradient_against_differences(act, center):
    """fp32 gradients along random directions against difference quotients of the formulas in 64 bits."""
    say("differences", act, center)
    gen = torch.Generator().manual_seed(6 + act)
    x, z, w, b, dy = inputs(gen, (4, 3, 48), F32, act)
    got = run(x, z, w, b, dy, act, center, eps=1e-2)
    leaves = dict(dx=x, dz=z, dweight=w, dbias=b)
    for k, leaf in leaves.items():
        if leaf is None:
            continue
        way = torch.randn(leaf.shape, generator=gen, dtype=torch.float64)

        def loss(step):
            v = {n: (t if n != k else t.double() + step * way) for n, t in leaves.items()}
            return float((ref.norm(v["dx"], v["dz"], v["dweight"], v["dbias"], act, center, 1e-2)[0]["y"] * dy).sum())

        slope = (loss(1e-6) - loss(-1e-6)) / 2e-6
        terms = got[k].cpu().double() * way
        # fp32 gradients of groups of 48: 2^-24 of each term some tens of times
        assert abs(slope - float(terms.sum())) <= 1e-5 * float(terms.abs().sum()) + 1e-6, (k, slope, float(terms.sum()))


def test_no_tokens():
    for act in (0, 2):
        x = torch.empty(0, 2, 16, device="cuda")
        got = run(x, None if act == 0 else x, None, None, x, act, True)
        assert (got["dweight"] == 0).all() and (got["dbias"] == 0).all()


def test_in_a_graph_and_on_a_stream():
    say("graph")
    gen = torch.Generator().manual_seed(9)
    x, z, w, b, dy = (t.cuda() for t in inputs(gen, (300, 4, 136), BF, 2))
    y, dx, dz = (torch.zeros_like(x) for _ in range(3))
    dw, db = torch.zeros_like(w), torch.zeros_like(b)
    ws = torch.empty(max(256, ssq.ssq_group_norm_workspace(4, 136, 300)), dtype=torch.uint8, device="cuda")
    how = dict(weight=w, bias=b, z=z, act=2)

    def call(**kw):
        ssq.ssq_group_norm(x, y, **how, **kw)
        ssq.ssq_group_norm_backward(dy, x, dx, dz=dz, dweight=dw, dbias=db, workspace=ws, **how, **kw)

    call()
    want = [t.clone() for t in (y, dx, dz, dw, db)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        for t in (y, dx, dz, dw, db):
            t.fill_(SENTINEL)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, dx, dz, dw, db), want))
    for t in (y, dx, dz, dw, db):
        t.fill_(SENTINEL)
    torch.cuda.synchronize()
    call(stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((y, dx, dz, dw, db), want))


def test_refusals():
    say("refusals")
    t = lambda *s, d=BF: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    x, w = t(6, 2, 16), t(2, 16, d=F32)
    bad = (ValueError, TypeError, ssq.SsqError)

    def refused(call, *a, **kw):
        with pytest.raises(bad):
            call(*a, **kw)

    out = t(6, 2, 16)
    for kw in (dict(x=t(6, 32)), dict(x=t(6, 2, 16, d=torch.float64)), dict(y=t(6, 2, 16, d=HF)), dict(y=t(5, 2, 16)), dict(z=x), dict(act=1),
               dict(act=3, z=x), dict(act=2, z=t(6, 2, 8)), dict(weight=w[0]), dict(weight=w.bfloat16()), dict(bias=t(16, 2, d=F32).t()),
               dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(x=t(6, 2, 12), y=t(6, 2, 12)),
               dict(x=t(1, 1, 16392), y=t(1, 1, 16392)), dict(x=t(1, 65, 16384), y=t(1, 65, 16384)), dict(y=t(6, 2, 16).cpu()),
               dict(x=t(6, 2, 32)[..., :16]), dict(x=t(1, 2, 16).expand(6, 2, 16)), dict(act=1 << 32)):
        a = dict(x=x, y=out) | kw
        refused(ssq.ssq_group_norm, a.pop("x"), a.pop("y"), **a)
    for kw in (dict(dy=t(5, 2, 16)), dict(dx=t(6, 2, 16, d=F32)), dict(dz=t(6, 2, 16)), dict(act=2, z=x), dict(dweight=t(2, 16)), dict(dbias=t(16, d=F32)),
               dict(workspace=t(0, d=torch.uint8)), dict(workspace=t(1 << 20, d=torch.uint8)[8:])):
        a = dict(dy=x, x=x, dx=out) | dict(dweight=t(2, 16, d=F32)) | kw
        refused(ssq.ssq_group_norm_backward, a.pop("dy"), a.pop("x"), a.pop("dx"), **a)
    torch.cuda.synchronize()
    assert (out == 0).all()
