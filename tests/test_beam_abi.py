"""The C ABI of linear attention, beam selection and reordering on the host: refusals that come
before any device call, and workspace sizes.  No kernel is launched (no GPU needed)."""
import ctypes

import pytest
import torch

import mamba_decode_amd as ssq

L = ssq.lib
BAD = ssq.SSQ_ERR_INVALID_ARG


def desc(**kw):
    d = dict(dtype=ssq.SSQ_DTYPE_BF16, batch=2, beams=4, vocab=100, nselect=8, pad_token=0, row_stride=100) | kw
    return ssq.ssq_beam_desc(*(d[n] for n, _ in ssq.ssq_beam_desc._fields_))


@pytest.mark.parametrize("kw", [dict(dtype=3), dict(dtype=-1), dict(batch=-1), dict(beams=0), dict(beams=33), dict(vocab=0),
                                dict(nselect=0), dict(nselect=9), dict(pad_token=-1), dict(pad_token=100),
                                dict(row_stride=99), dict(row_stride=1 << 60)])
def test_beam_descriptions(kw):
    d = desc(**kw)
    assert ssq.ssq_beam_workspace(d) == 0
    vp = ctypes.c_void_p
    assert L.ssq_beam_select(ctypes.byref(d), vp(4096), vp(4096), None, vp(4096), vp(4096), vp(4096), vp(4096), 1 << 30,
                             None) == BAD
    assert ssq.ssq_last_error()


def test_beam_rows_of_one_launch():
    d = desc(batch=1 << 22)
    assert ssq.ssq_beam_workspace(d) == 0
    vp = ctypes.c_void_p
    assert L.ssq_beam_select(ctypes.byref(d), vp(4096), vp(4096), None, vp(4096), vp(4096), vp(4096), vp(4096), 1 << 40,
                             None) == ssq.SSQ_ERR_UNSUPPORTED
    assert ssq.ssq_beam_workspace(desc(batch=(1 << 22) - 1)) > 0


def test_beam_arguments():
    vp = ctypes.c_void_p
    d = desc()
    need = ssq.ssq_beam_workspace(d)
    assert need > 0
    ok = [vp(4096), vp(4096), None, vp(4096), vp(4096), vp(4096), vp(4096), need, None]
    for i, bad in ((0, None), (0, vp(4097)), (1, None), (1, vp(4098)), (3, None), (4, None), (5, vp(4097)), (6, None),
                   (6, vp(4096 + 16)), (7, need - 1)):
        args = list(ok)
        args[i] = bad
        assert L.ssq_beam_select(ctypes.byref(d), *args) == BAD, i
    assert L.ssq_beam_select(None, *ok) == BAD
    assert L.ssq_beam_select(ctypes.byref(desc(batch=0)), *([None] * 7), 0, None) == ssq.SSQ_OK


def test_workspace_grows_with_the_batch():
    sizes = [ssq.ssq_beam_workspace(desc(batch=b, vocab=200000, row_stride=200000)) for b in (1, 2, 64)]
    assert sizes[0] < sizes[1] < sizes[2]


def test_null_states():
    io = ssq.ssq_linattn_io()
    assert L.ssq_linattn_workspace(None, 1, 1) == ctypes.c_size_t(-1).value
    assert L.ssq_linattn_prefill(None, ctypes.byref(io), 0, 0, None, None, None, None, 0, None) == BAD
    assert L.ssq_linattn_step(None, ctypes.byref(io), 0, None, 0, None) == BAD
    vp = ctypes.c_void_p
    none = (vp * 1)(None)
    assert L.ssq_state_reorder(None, 0, None, 4, None) == ssq.SSQ_OK
    for args in ((None, 1, vp(4096), 4), (none, 1, None, 4), (none, 1, vp(4096), 4), (none, -1, vp(4096), 4),
                 (none, 1025, vp(4096), 4), (none, 1, vp(4096), 0), (none, 1, vp(4096), 33), (none, 1, vp(4098), 4)):
        assert L.ssq_state_reorder(*args, None) == BAD, args


def test_tensors_of_the_host_are_refused():
    if torch.cuda.is_available():
        pytest.skip("the message of a machine without a GPU")
    x = torch.zeros(1, 2, 5)
    with pytest.raises((ValueError, RuntimeError)):
        ssq.ssq_beam_select(x, x[..., 0], x[0], x[0], x[0])
    with pytest.raises((ValueError, RuntimeError)):
        ssq.ssq_state_reorder([], torch.zeros(1, 2, dtype=torch.int32))
