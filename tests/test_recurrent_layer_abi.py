"""Host: sizes and argument checks of the gated recurrence, the group norm and the moves of states.  No kernel is
launched: every call here is rejected, or covers nothing."""
import ctypes

import pytest

import mamba_decode_amd as ssq

L = ssq.lib
P = 0x10000  # a pointer that nothing follows
INVALID, UNSUPPORTED = ssq.SSQ_ERR_INVALID_ARG, ssq.SSQ_ERR_UNSUPPORTED


def test_layout_of_a_gated_state():
    lay = ssq.ssq_state_layout(ssq.make_desc(ssq.SSQ_GATED, "fp32", 5, 1, 1, 1544))
    assert (lay.rows, lay.row_bytes, lay.codes_offset) == (5, 1544 * 4, 0)
    assert (lay.scale_offset, lay.zero_offset, lay.hi_offset, lay.counter_offset) == (0, 0, 0, 0)
    assert lay.total_bytes == (5 * 1544 * 4 + 255) // 256 * 256


@pytest.mark.parametrize("fmt,shape,status", [
    ("fp32", (2, 1, 1, 12, 1), UNSUPPORTED), ("fp32", (2, 1, 1, (1 << 20) + 8, 1), UNSUPPORTED), ("int8_sym", (2, 1, 1, 16, 1), UNSUPPORTED),
    ("damp", (2, 1, 1, 16, 1), UNSUPPORTED), ("fp32", (2, 2, 1, 16, 1), INVALID), ("fp32", (2, 1, 16, 16, 1), INVALID),
    ("fp32", (2, 2, 1, 16, 2), INVALID), ("fp32", (0, 1, 1, 16, 1), INVALID), ("fp32", (2, 1, 1, 0, 1), INVALID)])
def test_bad_descriptions_of_gated_states(fmt, shape, status):
    batch, heads, rows, channels, groups = shape
    d = ssq.make_desc(ssq.SSQ_GATED, fmt, batch, heads, rows, channels, groups)
    assert ssq.ssq_state_bytes(d) == 0
    lay = ssq.ssq_layout()
    assert L.ssq_state_layout(ctypes.byref(d), ctypes.byref(lay)) == status


def test_checkpoint_rows():
    assert ssq.ssq_gated_checkpoint_rows(3, 100) == 6 + 3
    assert ssq.ssq_gated_checkpoint_rows(0, 0) == 0
    for n, t in ((-1, 5), (1, -1), (1, 1 << 31), (1, 1 << 62)):
        assert L.ssq_gated_checkpoint_rows(n, t) == -1
    with pytest.raises(ValueError):
        ssq.ssq_gated_checkpoint_rows(1, 1 << 64)


def test_workspaces():
    assert ssq.ssq_gated_workspace(8, 0, 0) == 0 and ssq.ssq_gated_workspace(2048, 24, 16800) == 0
    assert ssq.ssq_gated_workspace(64, 1, 100000) > 0
    for c, n, t in ((0, 1, 1), (12, 1, 1), (8, -1, 1), (8, 1, -1), ((1 << 20) + 8, 1, 1), (1 << 20, 65, 1), (8, 1 << 23, 1), (8, 1, 0x7FFFFF80)):
        assert L.ssq_gated_workspace(c, n, t) == ssq._SIZE_MAX, (c, n, t)
    assert ssq.ssq_group_norm_workspace(8, 1024, 0) == 0 and ssq.ssq_group_norm_workspace(8, 1024, 8192) > 0
    for g, w, t in ((0, 8, 1), (1, 12, 1), (1, 16392, 1), (65, 16384, 1), (1, 8, -1), (2, 8, (1 << 30) + 1)):
        assert L.ssq_group_norm_workspace(g, w, t) == ssq._SIZE_MAX, (g, w, t)
    # sizes that a program meets never need more than it expects: sums of the parts, of the workgroups along the tokens
    for c in (8, 64, 256, 2048, 8192):
        for n in (1, 3, 100):
            for t in (1, 1000, 100000, 3000000):
                assert ssq.ssq_gated_workspace(c, n, t) <= 64 << 20


def gated(**kw):
    return ssq.ssq_gated_io(*(dict(dtype=0, gate=0, input=0, channels=16, x=P, g=P, o=P, x_stride=16, g_stride=16, o_stride=16) | kw).values())


def scan(io, nseq=1, tokens=4, cu=P, slots=None, fresh=None, ck=None, ws=None, nws=0):
    return L.ssq_gated_scan(None, io, nseq, tokens, cu, slots, fresh, ck, ws, nws, None)


@pytest.mark.parametrize("kw,call,status", [
    (dict(dtype=3), {}, INVALID), (dict(gate=2), {}, INVALID), (dict(gate=-1), {}, INVALID), (dict(input=3), {}, INVALID),
    (dict(channels=0), {}, INVALID), (dict(channels=12), {}, UNSUPPORTED), (dict(channels=-8), {}, INVALID),
    (dict(x=None), {}, INVALID), (dict(g=None), {}, INVALID), (dict(o=None), {}, INVALID), (dict(x=P + 8), {}, INVALID),
    (dict(x_stride=8), {}, INVALID), (dict(g_stride=18), {}, INVALID), (dict(o_stride=-16), {}, INVALID), (dict(o_stride=(1 << 23) + 8), {}, UNSUPPORTED),
    (dict(dtype=1, x_stride=20), {}, INVALID), ({}, dict(nseq=-1), INVALID), ({}, dict(tokens=-1), INVALID), ({}, dict(tokens=0x7FFFFF80), UNSUPPORTED),
    ({}, dict(nseq=(1 << 22) + 1), UNSUPPORTED), ({}, dict(cu=None), INVALID), ({}, dict(cu=P + 2), INVALID), ({}, dict(slots=P), INVALID),
    ({}, dict(fresh=P), INVALID), ({}, dict(ck=P + 8), INVALID), ({}, dict(tokens=100000), INVALID),
    ({}, dict(tokens=100000, ws=P, nws=64), INVALID), ({}, dict(tokens=100000, ws=P + 64, nws=1 << 40), INVALID)])
def test_scans_are_checked(kw, call, status):
    assert scan(gated(**kw), **call) == status
    assert ssq.ssq_last_error()


def test_calls_of_nothing():
    assert scan(gated(), nseq=0, cu=None) == ssq.SSQ_OK
    assert scan(gated(x=None, g=None, o=None), nseq=0, tokens=0) == ssq.SSQ_OK
    assert L.ssq_group_norm(norm(x=None), None, 16, 0, None) == ssq.SSQ_OK
    assert L.ssq_state_move(None, None, 0, None, None, 5, None) == ssq.SSQ_OK
    assert L.ssq_gated_scan(None, None, 1, 4, P, None, None, None, None, 0, None) == INVALID
    assert L.ssq_gated_step(None, gated(), 1, None, None) == INVALID


@pytest.mark.parametrize("kw,call,status", [
    (dict(dtype=-1), {}, INVALID), (dict(channels=20), {}, UNSUPPORTED), (dict(dout=None), {}, INVALID), (dict(dx=None), {}, INVALID), (dict(dg=P + 4), {}, INVALID),
    (dict(dx_stride=8), {}, INVALID), (dict(dlast=P + 8), {}, INVALID), (dict(dfirst=P + 8), {}, INVALID), ({}, dict(ck=None), INVALID), ({}, dict(ck=P + 8), INVALID),
    ({}, dict(cu=None), INVALID), ({}, dict(slots=P), INVALID), ({}, dict(tokens=100000), INVALID)])
def test_gradients_are_checked(kw, call, status):
    io = dict(dtype=0, gate=0, input=0, channels=16, x=P, g=P, dout=P, dx=P, dg=P, x_stride=16, g_stride=16, dout_stride=16, dx_stride=16,
              dg_stride=16, dlast=None, dfirst=None) | kw
    a = dict(tokens=4, cu=P, slots=None, ck=P) | call
    assert L.ssq_gated_scan_backward(None, ssq.ssq_gated_grad(*io.values()), 1, a["tokens"], a["cu"], a["slots"], a["ck"], None, 0, None) == status
    assert L.ssq_gated_scan_backward(None, None, 1, 4, P, None, P, None, 0, None) == INVALID


def norm(**kw):
    return ssq.ssq_norm_io(*(dict(dtype=0, act=0, center=1, groups=2, width=8, eps=1e-5, weight=None, bias=None, x=P, z=None, x_stride=16,
                                  z_stride=0) | kw).values())


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=5), INVALID), (dict(act=3), INVALID), (dict(groups=0), INVALID), (dict(width=-8), INVALID), (dict(width=12), UNSUPPORTED),
    (dict(width=16392), UNSUPPORTED), (dict(groups=1 << 20), UNSUPPORTED), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=-1e-5), INVALID), (dict(eps=1e-39), INVALID), (dict(eps=float("inf")), INVALID), (dict(x=None), INVALID), (dict(x=P + 8), INVALID),
    (dict(x_stride=8), INVALID), (dict(x_stride=1 << 24), UNSUPPORTED), (dict(z=P, z_stride=16), INVALID), (dict(act=1), INVALID),
    (dict(act=2, z=P, z_stride=8), INVALID), (dict(weight=P + 4), INVALID), (dict(bias=P + 4), INVALID)])
def test_norms_are_checked(kw, status):
    assert L.ssq_group_norm(norm(**kw), P, 16, 4, None) == status
    grad = ssq.ssq_norm_grad(P, P, None if kw.get("act", 0) == 0 else P, P, P, 16, 16, 16)
    assert L.ssq_group_norm_backward(norm(**kw), grad, 4, P, 1 << 30, None) == status


def test_gradients_of_norms_are_checked():
    ok = dict(dy=P, dx=P, dz=None, dweight=P, dbias=P, dy_stride=16, dx_stride=16, dz_stride=16)
    call = lambda io, ws=P, n=1 << 30, **kw: L.ssq_group_norm_backward(io, ssq.ssq_norm_grad(*(ok | kw).values()), 4, ws, n, None)  # noqa: E731
    for kw in (dict(dy=None), dict(dx=None), dict(dx=P + 4), dict(dy_stride=8), dict(dz=P), dict(dweight=P + 8), dict(dbias=P + 8),
               dict(ws=None), dict(ws=P + 128), dict(n=16)):
        assert call(norm(), **kw) == INVALID, kw
    assert call(norm(act=1, z=P, z_stride=16)) == INVALID  # dz is missing
    assert L.ssq_group_norm_backward(norm(), None, 4, P, 1 << 30, None) == INVALID
    assert L.ssq_group_norm(None, P, 16, 4, None) == INVALID
    assert L.ssq_group_norm(norm(), None, 16, 4, None) == INVALID and L.ssq_group_norm(norm(), P, 8, 4, None) == INVALID
    assert L.ssq_group_norm(norm(), P, 16, -1, None) == INVALID and L.ssq_group_norm(norm(), P, 16, 1 << 31, None) == UNSUPPORTED


def test_moves_are_checked():
    states = (ctypes.c_void_p * 1)(None)
    for args in ((None, None, 1, P, P, 1), (states, None, -1, P, P, 1), (states, None, 1025, P, P, 1), (states, None, 1, P, P, -1),
                 (states, None, 1, P, P, 65536), (states, None, 1, None, P, 1), (states, None, 1, P, None, 1), (states, None, 1, P + 2, P, 1),
                 (states, None, 1, P, P, 1), (states, states, 1, P, P, 1)):
        assert L.ssq_state_move(*args, None) == INVALID, args
