"""Python binding of ``libssq.so``: the quantized recurrent-state update on MI355X.

Argument marshalling only.  Every step of the path runs in the HIP kernels
behind the C ABI of ``include/ssq.h``; PyTorch supplies device memory (tensor
data pointers) and the stream (``torch.cuda.current_stream()``).  The binding
checks that tensors have the dtype, device, contiguity and size that the
state's description implies, so that the kernels never see a short buffer.

Importing this package fails loudly if the library has not been built
(``python -m mamba_decode_amd.build``): there is no fallback path.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch  # imported first: the library binds to the HIP runtime torch has loaded

_HERE = os.path.dirname(os.path.abspath(__file__))
# SSQ_LIBRARY names another build of the same sources (the host tests' sanitized build)
LIB_PATH = os.environ.get("SSQ_LIBRARY") or os.path.join(_HERE, "libssq.so")

# ssq_status
SSQ_OK, SSQ_ERR_INVALID_ARG, SSQ_ERR_UNSUPPORTED, SSQ_ERR_KIND_MISMATCH, SSQ_ERR_ALLOC, SSQ_ERR_DEVICE = range(6)
# ssq_format
SSQ_FP32, SSQ_INT8_SYM, SSQ_INT8_ASYM, SSQ_INT4_SYM, SSQ_INT4_ASYM, SSQ_DAMP = range(6)
SSQ_DAMP_NHI = 16
# ssq_kind
SSQ_MAMBA2, SSQ_DELTA, SSQ_GATED = range(3)
# ssq_readout
SSQ_READ_POST_QUANT, SSQ_READ_PRE_QUANT = 0, 1
# ssq_dtype
SSQ_DTYPE_FP32, SSQ_DTYPE_BF16, SSQ_DTYPE_FP16 = range(3)
SSQ_MAX_BEAMS = 32
# ssq_gate, ssq_input
SSQ_GATE_LOG, SSQ_GATE_SIGMOID = 0, 1
SSQ_INPUT_PLAIN, SSQ_INPUT_COMPLEMENT, SSQ_INPUT_NORM = range(3)
SSQ_GATED_CHUNK = 16
# ssq_act
SSQ_ACT_SILU, SSQ_ACT_GATE_OUTPUT, SSQ_ACT_GATE_INPUT = range(3)
# ssq_rounding
SSQ_ROUND_NEAREST, SSQ_ROUND_STOCHASTIC = 0, 1

FORMAT_NAMES = {"fp32": SSQ_FP32, "int8_sym": SSQ_INT8_SYM, "int8_asym": SSQ_INT8_ASYM,
                "int4_sym": SSQ_INT4_SYM, "int4_asym": SSQ_INT4_ASYM, "damp": SSQ_DAMP}
FORMAT_BITS = {SSQ_FP32: 32, SSQ_INT8_SYM: 8, SSQ_INT8_ASYM: 8, SSQ_INT4_SYM: 4, SSQ_INT4_ASYM: 4, SSQ_DAMP: 8}


class SsqError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: {detail} (status {status})")
        self.status = status


class ssq_desc(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("format", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("nheads", ctypes.c_int32), ("ngroups", ctypes.c_int32),
                ("rows_per_head", ctypes.c_int32), ("row_len", ctypes.c_int32)]


class ssq_layout(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_size_t), ("row_bytes", ctypes.c_size_t),
                ("codes_offset", ctypes.c_size_t), ("scale_offset", ctypes.c_size_t),
                ("zero_offset", ctypes.c_size_t), ("total_bytes", ctypes.c_size_t),
                ("hi_offset", ctypes.c_size_t), ("counter_offset", ctypes.c_size_t)]


class ssq_linattn_io(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("scale", ctypes.c_float), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("g", ctypes.c_void_p), ("o", ctypes.c_void_p), ("q_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64), ("g_stride", ctypes.c_int64),
                ("o_stride", ctypes.c_int64)]


class ssq_beam_desc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("batch", ctypes.c_int32), ("beams", ctypes.c_int32),
                ("vocab", ctypes.c_int32), ("nselect", ctypes.c_int32), ("pad_token", ctypes.c_int32),
                ("row_stride", ctypes.c_int64)]


_i32, _i64, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p


class ssq_gated_io(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("gate", _i32), ("input", _i32), ("channels", _i32), ("x", _vp), ("g", _vp), ("o", _vp),
                ("x_stride", _i64), ("g_stride", _i64), ("o_stride", _i64)]


class ssq_gated_grad(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("gate", _i32), ("input", _i32), ("channels", _i32), ("x", _vp), ("g", _vp), ("dout", _vp),
                ("dx", _vp), ("dg", _vp), ("x_stride", _i64), ("g_stride", _i64), ("dout_stride", _i64), ("dx_stride", _i64),
                ("dg_stride", _i64), ("dlast", _vp), ("dfirst", _vp)]


class ssq_norm_io(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("act", _i32), ("center", _i32), ("groups", _i32), ("width", _i32), ("eps", ctypes.c_float),
                ("weight", _vp), ("bias", _vp), ("x", _vp), ("z", _vp), ("x_stride", _i64), ("z_stride", _i64)]


class ssq_norm_grad(ctypes.Structure):
    _fields_ = [("dy", _vp), ("dx", _vp), ("dz", _vp), ("dweight", _vp), ("dbias", _vp), ("dy_stride", _i64),
                ("dx_stride", _i64), ("dz_stride", _i64)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -m mamba_decode_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, f32p = ctypes.c_void_p, ctypes.c_void_p
    st = ctypes.c_int
    dp = ctypes.POINTER(ssq_desc)
    L.ssq_state_bytes.argtypes = [dp]
    L.ssq_state_bytes.restype = ctypes.c_size_t
    L.ssq_state_layout.argtypes = [dp, ctypes.POINTER(ssq_layout)]
    L.ssq_state_layout.restype = st
    L.ssq_alloc_state.argtypes = [dp, vp, f32p, vp, ctypes.POINTER(ctypes.c_void_p)]
    L.ssq_alloc_state.restype = st
    L.ssq_free_state.argtypes = [vp]
    L.ssq_free_state.restype = st
    L.ssq_state_info.argtypes = [vp, dp, ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ssq_layout)]
    L.ssq_state_info.restype = st
    L.ssq_decode_step.argtypes = [vp, f32p, f32p, f32p, f32p, f32p, f32p, f32p, ctypes.c_int32, vp]
    L.ssq_decode_step.restype = st
    L.ssq_scan.argtypes = [vp, ctypes.c_int32, f32p, f32p, f32p, f32p, f32p, f32p, f32p, ctypes.c_int32, vp]
    L.ssq_scan.restype = st
    L.ssq_delta_step.argtypes = [vp, f32p, f32p, f32p, f32p, f32p, f32p, ctypes.c_int32, vp]
    L.ssq_delta_step.restype = st
    L.ssq_dequant.argtypes = [vp, f32p, vp]
    L.ssq_dequant.restype = st
    L.ssq_stream_copy.argtypes = [vp, vp, ctypes.c_size_t, vp]
    L.ssq_stream_copy.restype = st
    L.ssq_status_string.argtypes = [ctypes.c_int32]
    L.ssq_status_string.restype = ctypes.c_char_p
    L.ssq_last_error.argtypes = []
    L.ssq_last_error.restype = ctypes.c_char_p
    L.ssq_prefill.argtypes = [vp, ctypes.c_int32, ctypes.c_int32, f32p, f32p, f32p, f32p, f32p, f32p, f32p,
                              ctypes.c_int32, vp]
    L.ssq_prefill.restype = st
    L.ssq_kda_step.argtypes = [vp, f32p, f32p, f32p, f32p, f32p, f32p, ctypes.c_int32, vp]
    L.ssq_kda_step.restype = st
    u64 = ctypes.c_uint64
    L.ssq_set_rounding.argtypes = [vp, ctypes.c_int32, u64, u64, vp]
    L.ssq_set_rounding.restype = st
    L.ssq_get_rounding.argtypes = [vp, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(u64), ctypes.POINTER(u64), vp]
    L.ssq_get_rounding.restype = st
    iop = ctypes.POINTER(ssq_linattn_io)
    L.ssq_linattn_workspace.argtypes = [vp, ctypes.c_int32, ctypes.c_int64]
    L.ssq_linattn_workspace.restype = ctypes.c_size_t
    L.ssq_linattn_prefill.argtypes = [vp, iop, ctypes.c_int32, ctypes.c_int64, vp, vp, vp, vp, ctypes.c_size_t, vp]
    L.ssq_linattn_prefill.restype = st
    L.ssq_linattn_step.argtypes = [vp, iop, ctypes.c_int32, vp, ctypes.c_int32, vp]
    L.ssq_linattn_step.restype = st
    bdp = ctypes.POINTER(ssq_beam_desc)
    L.ssq_beam_workspace.argtypes = [bdp]
    L.ssq_beam_workspace.restype = ctypes.c_size_t
    L.ssq_beam_select.argtypes = [bdp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    L.ssq_beam_select.restype = st
    L.ssq_state_reorder.argtypes = [ctypes.POINTER(vp), ctypes.c_int32, vp, ctypes.c_int32, vp]
    L.ssq_state_reorder.restype = st
    size = ctypes.c_size_t
    L.ssq_state_move.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(vp), _i32, vp, vp, _i32, vp]
    L.ssq_state_move.restype = st
    L.ssq_gated_checkpoint_rows.argtypes = [_i32, _i64]
    L.ssq_gated_checkpoint_rows.restype = _i64
    L.ssq_gated_workspace.argtypes = [_i32, _i32, _i64]
    L.ssq_gated_workspace.restype = size
    L.ssq_gated_scan.argtypes = [vp, ctypes.POINTER(ssq_gated_io), _i32, _i64, vp, vp, vp, vp, vp, size, vp]
    L.ssq_gated_scan.restype = st
    L.ssq_gated_scan_backward.argtypes = [vp, ctypes.POINTER(ssq_gated_grad), _i32, _i64, vp, vp, vp, vp, size, vp]
    L.ssq_gated_scan_backward.restype = st
    L.ssq_gated_step.argtypes = [vp, ctypes.POINTER(ssq_gated_io), _i32, vp, vp]
    L.ssq_gated_step.restype = st
    L.ssq_group_norm.argtypes = [ctypes.POINTER(ssq_norm_io), vp, _i64, _i64, vp]
    L.ssq_group_norm.restype = st
    L.ssq_group_norm_workspace.argtypes = [_i32, _i32, _i64]
    L.ssq_group_norm_workspace.restype = size
    L.ssq_group_norm_backward.argtypes = [ctypes.POINTER(ssq_norm_io), ctypes.POINTER(ssq_norm_grad), _i64, vp, size, vp]
    L.ssq_group_norm_backward.restype = st
    return L


lib = _load()


def ssq_status_string(status: int) -> str:
    return lib.ssq_status_string(status).decode()


def ssq_last_error() -> str:
    return lib.ssq_last_error().decode()


def _check(status: int, where: str):
    if status != SSQ_OK:
        raise SsqError(status, where, ssq_last_error() or ssq_status_string(status))


def make_desc(kind: int, fmt, batch: int, nheads: int, rows_per_head: int, row_len: int = 128,
              ngroups: int = 1) -> ssq_desc:
    if isinstance(fmt, str):
        fmt = FORMAT_NAMES[fmt]
    return ssq_desc(kind, fmt, batch, nheads, ngroups, rows_per_head, row_len)


def ssq_state_bytes(desc: ssq_desc) -> int:
    return int(lib.ssq_state_bytes(ctypes.byref(desc)))


def ssq_state_layout(desc: ssq_desc) -> ssq_layout:
    lay = ssq_layout()
    _check(lib.ssq_state_layout(ctypes.byref(desc), ctypes.byref(lay)), "ssq_state_layout")
    return lay


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dev(t: torch.Tensor, name: str, numel, dtype=torch.float32) -> ctypes.c_void_p:
    """Device pointer of a tensor; ``numel`` None skips the size check (the call is rejected by
    the library anyway, e.g. for a state of the other kind)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
    return ctypes.c_void_p(t.data_ptr())


class State:
    """A state handle plus the torch tensor that holds its storage (if torch allocated it)."""

    def __init__(self, handle: ctypes.c_void_p, desc: ssq_desc, layout: ssq_layout, storage):
        self.handle = handle
        self.desc = desc
        self.layout = layout
        self.storage = storage  # torch uint8 tensor, or None when the library owns the memory

    @property
    def rows(self) -> int:
        return int(self.layout.rows)

    def regions(self):
        """(codes, scale, zero) views of a torch-held storage: codes [rows][row_bytes] uint8
        (fp32 format: [rows][row_len] float32), scale/zero [rows] float32 or None."""
        if self.storage is None:
            raise ValueError("the library owns this state's memory; pass a torch storage to view it")
        L, s = self.layout, self.storage
        n = self.rows
        if self.desc.format == SSQ_DAMP:  # the uint8 rows only; hi_region() holds the half rows
            n = n // self.desc.rows_per_head * (self.desc.rows_per_head - SSQ_DAMP_NHI)
        if self.desc.format == SSQ_FP32:
            codes = s[: n * L.row_bytes].view(torch.float32).view(n, self.desc.row_len)
            return codes, None, None
        codes = s[: n * L.row_bytes].view(n, L.row_bytes)
        scale = s[L.scale_offset: L.scale_offset + 4 * n].view(torch.float32)
        zero = s[L.zero_offset: L.zero_offset + 4 * n].view(torch.float32) if L.zero_offset else None
        return codes, scale, zero

    def hi_region(self):
        """Two-tier state: the half rows [mats][16][row_len] as float16 (a view of the storage)."""
        L, s, d = self.layout, self.storage, self.desc
        mats = self.rows // d.rows_per_head
        nb = mats * SSQ_DAMP_NHI * d.row_len * 2
        return s[L.hi_offset: L.hi_offset + nb].view(torch.float16).view(mats, SSQ_DAMP_NHI, d.row_len)

    def free(self):
        if self.handle is not None:
            _check(lib.ssq_free_state(self.handle), "ssq_free_state")
            self.handle = None

    def __del__(self):
        try:
            if self.handle is not None and lib is not None:
                lib.ssq_free_state(self.handle)
                self.handle = None
        except Exception:
            pass


def ssq_alloc_state(desc: ssq_desc, storage: torch.Tensor | None = None, init: torch.Tensor | None = None,
                    stream=None) -> State:
    """Create a state (zero, or ``init`` quantized).  ``storage``: a uint8 CUDA tensor of at least
    ``ssq_state_bytes(desc)`` bytes that outlives the state, or None for library-owned memory."""
    layout = ssq_state_layout(desc)
    sp = None
    if storage is not None:
        if not storage.is_cuda or storage.dtype != torch.uint8 or not storage.is_contiguous():
            raise ValueError("storage must be a contiguous uint8 CUDA tensor")
        if storage.numel() < layout.total_bytes:
            raise ValueError(f"storage has {storage.numel()} bytes, needs {layout.total_bytes}")
        sp = ctypes.c_void_p(storage.data_ptr())
    ip = None
    if init is not None:
        ip = _dev(init, "init", int(layout.rows) * desc.row_len)
    h = ctypes.c_void_p()
    _check(lib.ssq_alloc_state(ctypes.byref(desc), sp, ip, _stream(stream), ctypes.byref(h)), "ssq_alloc_state")
    return State(h, desc, layout, storage)


def ssq_free_state(state: State):
    state.free()


def ssq_state_info(state: State):
    """(desc, storage device pointer, layout) of a state."""
    d, lay, ptr = ssq_desc(), ssq_layout(), ctypes.c_void_p()
    _check(lib.ssq_state_info(state.handle, ctypes.byref(d), ctypes.byref(ptr), ctypes.byref(lay)),
           "ssq_state_info")
    return d, ptr.value, lay


def ssq_set_rounding(state: State, mode: int, seed: int = 0, step: int = 0, stream=None):
    """Round the state's codes to nearest or stochastically (seed; the next token is written to the
    state's counter on ``stream``)."""
    _check(lib.ssq_set_rounding(state.handle, mode, seed, step, _stream(stream)), "ssq_set_rounding")


def ssq_get_rounding(state: State, stream=None):
    """(mode, seed, next token) of a state; the token is read from the device on ``stream``."""
    m, sd, sp = ctypes.c_int32(), ctypes.c_uint64(), ctypes.c_uint64()
    _check(lib.ssq_get_rounding(state.handle, ctypes.byref(m), ctypes.byref(sd), ctypes.byref(sp), _stream(stream)),
           "ssq_get_rounding")
    return m.value, sd.value, sp.value


def _sizes(state: State, kind: int, *sizes):
    return sizes if state.desc.kind == kind else (None,) * len(sizes)


def ssq_decode_step(state: State, x, dt, A, B, C, D, y, readout: int = SSQ_READ_POST_QUANT, stream=None):
    d = state.desc
    rows, bh, bc, nh = _sizes(state, SSQ_MAMBA2, d.batch * d.nheads * d.rows_per_head, d.batch * d.nheads,
                              d.batch * d.ngroups * d.row_len, d.nheads)
    _check(lib.ssq_decode_step(state.handle, _dev(x, "x", rows), _dev(dt, "dt", bh), _dev(A, "A", nh),
                               _dev(B, "B", bc), _dev(C, "C", bc), _dev(D, "D", nh), _dev(y, "y", rows),
                               readout, _stream(stream)), "ssq_decode_step")


def ssq_scan(state: State, T: int, x, dt, A, B, C, D, y, readout: int = SSQ_READ_POST_QUANT, stream=None):
    d = state.desc
    Tn = max(int(T), 0)
    xs, dts, bcs, nh = _sizes(state, SSQ_MAMBA2, d.batch * d.nheads * d.rows_per_head * Tn,
                              d.batch * Tn * d.nheads, d.batch * Tn * d.ngroups * d.row_len, d.nheads)
    _check(lib.ssq_scan(state.handle, T, _dev(x, "x", xs), _dev(dt, "dt", dts), _dev(A, "A", nh),
                        _dev(B, "B", bcs), _dev(C, "C", bcs), _dev(D, "D", nh), _dev(y, "y", xs),
                        readout, _stream(stream)), "ssq_scan")


def ssq_prefill(state: State, T: int, chunk: int, x, dt, A, B, C, D, y, readout: int = SSQ_READ_POST_QUANT,
                stream=None):
    d = state.desc
    Tn = max(int(T), 0)
    xs, dts, bcs, nh = _sizes(state, SSQ_MAMBA2, d.batch * d.nheads * d.rows_per_head * Tn,
                              d.batch * Tn * d.nheads, d.batch * Tn * d.ngroups * d.row_len, d.nheads)
    _check(lib.ssq_prefill(state.handle, T, chunk, _dev(x, "x", xs), _dev(dt, "dt", dts), _dev(A, "A", nh),
                           _dev(B, "B", bcs), _dev(C, "C", bcs), _dev(D, "D", nh), _dev(y, "y", xs),
                           readout, _stream(stream)), "ssq_prefill")


def ssq_delta_step(state: State, q, k, v, alpha, beta, o, readout: int = SSQ_READ_POST_QUANT, stream=None):
    d = state.desc
    bh = d.batch * d.nheads
    nk, nv, nb = _sizes(state, SSQ_DELTA, bh * d.rows_per_head, bh * d.row_len, bh)
    _check(lib.ssq_delta_step(state.handle, _dev(q, "q", nk), _dev(k, "k", nk), _dev(v, "v", nv),
                              _dev(alpha, "alpha", nb), _dev(beta, "beta", nb), _dev(o, "o", nv), readout,
                              _stream(stream)), "ssq_delta_step")


def ssq_kda_step(state: State, q, k, v, alpha, beta, o, readout: int = SSQ_READ_POST_QUANT, stream=None):
    d = state.desc
    bh = d.batch * d.nheads
    nk, nv, nb = _sizes(state, SSQ_DELTA, bh * d.rows_per_head, bh * d.row_len, bh)
    _check(lib.ssq_kda_step(state.handle, _dev(q, "q", nk), _dev(k, "k", nk), _dev(v, "v", nv),
                            _dev(alpha, "alpha", nk), _dev(beta, "beta", nb), _dev(o, "o", nv), readout,
                            _stream(stream)), "ssq_kda_step")


def ssq_dequant(state: State, out, stream=None):
    _check(lib.ssq_dequant(state.handle, _dev(out, "out", state.rows * state.desc.row_len), _stream(stream)),
           "ssq_dequant")


def ssq_stream_copy(dst, src, nbytes: int | None = None, stream=None):
    """Copy ``nbytes`` (default: all of ``src``) from one CUDA tensor to another with the
    library's streaming copy kernel."""
    for name, t in (("dst", dst), ("src", src)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    n = src.numel() * src.element_size() if nbytes is None else int(nbytes)
    if n > src.numel() * src.element_size() or n > dst.numel() * dst.element_size():
        raise ValueError("nbytes exceeds a tensor")
    _check(lib.ssq_stream_copy(ctypes.c_void_p(dst.data_ptr()), ctypes.c_void_p(src.data_ptr()), n, _stream(stream)),
           "ssq_stream_copy")


_DTYPES = {torch.float32: SSQ_DTYPE_FP32, torch.bfloat16: SSQ_DTYPE_BF16, torch.float16: SSQ_DTYPE_FP16}

# The calls below are short enough on the device that their checks count: one function sees to a
# tensor's dtype, device, shape and layout and says what is wrong only if something is.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_get_device = getattr(torch._C, "_cuda_getDevice", None)


def _current_device() -> int:
    if _get_device is not None and torch.cuda.is_initialized():
        return _get_device()
    return torch.cuda.current_device()



def _stream_ptr(stream, dev: int) -> int:
    if stream is None:
        return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream
    if not hasattr(stream, "cuda_stream"):
        return int(stream)
    if getattr(getattr(stream, "device", None), "index", dev) != dev:  # its kernels would run there, on this device's memory
        raise ValueError("stream must be one of the current CUDA device")
    return stream.cuda_stream


def _refuse(t, name: str, dtype, shape, dev: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current CUDA device")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, is {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has the shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _ptr(t, name: str, dtype, shape, dev: int):
    """Device pointer of a contiguous tensor of this dtype and shape on device ``dev``."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev or t.shape != shape
            or not t.is_contiguous()):
        _refuse(t, name, dtype, shape, dev)
    return t.data_ptr()


def _flags(t, name: str, shape, dev: int):
    """The same of uint8 or bool flags, or None."""
    if t is None:
        return None
    return _ptr(t, name, torch.bool if isinstance(t, torch.Tensor) and t.dtype is torch.bool else torch.uint8, shape, dev)


def _tokens(t, name: str, dtype, shape, dev: int):
    """Pointer and stride between tokens of a [tokens][heads][width] or [tokens][heads] tensor whose tokens are packed."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        _refuse(t, name, dtype, shape, dev)
    if t.is_contiguous():
        return t.data_ptr(), math.prod(shape[1:])
    want = 1
    for n, s in zip(reversed(shape[1:]), reversed(t.stride()[1:])):
        if n != 1 and s != want:
            raise ValueError(f"the heads of {name} must be packed within a token")
        want *= n
    return t.data_ptr(), t.stride(0) if shape[0] > 1 else want


def _workspace(given, need: int, stream, dev: int):
    """Device memory for one call on ``stream``: the caller's, or torch's, which is reused in the stream's order."""
    if given is not None:
        return given, _ptr(given, "workspace", torch.uint8, given.shape, dev), given.numel()
    if need == 0:
        return None, None, 0
    if stream is None:
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    else:
        with torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream))):
            ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    return ws, ws.data_ptr(), need


def _int32(x, name: str) -> int:
    """A number that ctypes would otherwise take modulo 2^32."""
    if not -0x80000000 <= x <= 0x7FFFFFFF:
        raise ValueError(f"{name} is {x}, which 32 bits do not hold")
    return x


def _linattn_io(state: State, q, k, v, g, o, scale: float, tokens: int, dev: int):
    d = state.desc
    if d.kind != SSQ_MAMBA2:
        raise SsqError(SSQ_ERR_KIND_MISMATCH, "linear attention", "it runs on an SSQ_MAMBA2 state")
    dtype = q.dtype if isinstance(q, torch.Tensor) else None
    if dtype not in _DTYPES:
        raise ValueError("q must be a float32, bfloat16 or float16 tensor")
    keys, values = (tokens, d.ngroups, d.row_len), (tokens, d.nheads, d.rows_per_head)
    qp, qs = _tokens(q, "q", dtype, keys, dev)
    kp, ks = _tokens(k, "k", dtype, keys, dev)
    vp, vs = _tokens(v, "v", dtype, values, dev)
    op, os_ = _tokens(o, "o", dtype, values, dev)
    gp, gs = (None, 0) if g is None else _tokens(g, "g", torch.float32, values[:2], dev)
    if tokens == 0:  # no row is read: any stride serves
        qs = ks = keys[1] * keys[2]
        vs = os_ = values[1] * values[2]
    return ssq_linattn_io(_DTYPES[dtype], scale, qp, kp, vp, gp, op, qs, ks, vs, gs, os_)


def ssq_linattn_workspace(state: State, nseq: int, tokens: int) -> int:
    """Bytes of workspace ``ssq_linattn_prefill`` needs for these sizes."""
    if tokens >= 1 << 63:
        raise ValueError("tokens is more than 63 bits hold")
    n = lib.ssq_linattn_workspace(state.handle, _int32(nseq, "nseq"), tokens)
    if n == _SIZE_MAX:
        raise ValueError("linear attention runs on an SSQ_MAMBA2 state, sizes must not be negative")
    return n


_SIZE_MAX = ctypes.c_size_t(-1).value


def ssq_linattn_prefill(state: State, q, k, v, g, o, cu_seqlens, slots=None, fresh=None, scale: float = 1.0,
                        workspace: torch.Tensor | None = None, stream=None):
    """Ragged prompts through linear attention with a decay for each head.

    q, k ``[tokens, ngroups, 128]``, v, o ``[tokens, nheads, P]`` (float32, bfloat16 or float16; any stride between
    tokens that is a multiple of 16 bytes and not below a token's row), g ``[tokens, nheads]`` float32 log decays or
    None, cu_seqlens int32 ``[nseq + 1]``, slots int32 ``[nseq]`` or None, fresh uint8 or bool ``[nseq]`` or None; all
    on the device.  ``workspace``: uint8, at least ``ssq_linattn_workspace`` bytes, or None to take it from torch."""
    dev = torch.cuda.current_device()
    tokens = q.shape[0] if isinstance(q, torch.Tensor) and q.dim() else 0
    io = _linattn_io(state, q, k, v, g, o, scale, tokens, dev)
    nseq = cu_seqlens.numel() - 1 if isinstance(cu_seqlens, torch.Tensor) else 0
    if nseq < 0:
        raise ValueError("cu_seqlens has nseq + 1 entries")
    cu = _ptr(cu_seqlens, "cu_seqlens", torch.int32, (nseq + 1,), dev)
    sp = None if slots is None else _ptr(slots, "slots", torch.int32, (nseq,), dev)
    fp = _flags(fresh, "fresh", (nseq,), dev)
    on = _stream_ptr(stream, dev)
    ws, wp, wn = _workspace(workspace, ssq_linattn_workspace(state, nseq, tokens), stream, dev)
    _check(lib.ssq_linattn_prefill(state.handle, io, nseq, tokens, cu, sp, fp, wp, wn, on), "ssq_linattn_prefill")


def ssq_linattn_step(state: State, q, k, v, g, o, slots=None, scale: float = 1.0, readout: int = SSQ_READ_POST_QUANT,
                     stream=None):
    """One token of linear attention for ``nseq = q.shape[0]`` sequences: row i of the tensors (as in
    ``ssq_linattn_prefill``) is sequence ``slots[i]`` of the state, or sequence i without slots."""
    dev = torch.cuda.current_device()
    nseq = q.shape[0] if isinstance(q, torch.Tensor) and q.dim() else 0
    io = _linattn_io(state, q, k, v, g, o, scale, nseq, dev)
    sp = None if slots is None else _ptr(slots, "slots", torch.int32, (nseq,), dev)
    _check(lib.ssq_linattn_step(state.handle, io, _int32(nseq, "nseq"), sp, _int32(readout, "readout"),
                                _stream_ptr(stream, dev)), "ssq_linattn_step")


def ssq_beam_workspace(desc: ssq_beam_desc) -> int:
    """Bytes of workspace ``ssq_beam_select`` needs, 0 for an invalid description."""
    return lib.ssq_beam_workspace(desc)


def ssq_beam_select(logits, scores, out_scores, out_tokens, out_parents, finished=None, pad_token: int = 0,
                    workspace: torch.Tensor | None = None, stream=None):
    """The best ``out_scores.shape[1]`` continuations of every request over its beams and the vocabulary.

    logits ``[batch, beams, vocab]`` (float32, bfloat16 or float16; the beams any stride apart), scores
    ``[batch, beams]`` float32, out_scores float32, out_tokens and out_parents int32 ``[batch, nselect]``, finished
    uint8 or bool ``[batch, beams]`` or None."""
    dev = torch.cuda.current_device()
    if not isinstance(logits, torch.Tensor) or logits.dtype not in _DTYPES or logits.dim() != 3:
        raise ValueError("logits must be a float32, bfloat16 or float16 tensor [batch, beams, vocab]")
    if logits.get_device() != dev:
        raise ValueError("logits must be on the current CUDA device")
    b, m, v = logits.shape
    row = v
    if not logits.is_contiguous():
        s = logits.stride()
        row = s[1] if m > 1 else s[0] if b > 1 else v
        if v > 1 and s[2] != 1 or b > 1 and s[0] != m * row:
            raise ValueError("the rows of logits must be contiguous and evenly spaced")
    n = out_scores.shape[1] if isinstance(out_scores, torch.Tensor) and out_scores.dim() == 2 else 0
    sp = _ptr(scores, "scores", torch.float32, (b, m), dev)
    fp = _flags(finished, "finished", (b, m), dev)
    osp = _ptr(out_scores, "out_scores", torch.float32, (b, n), dev)
    otp = _ptr(out_tokens, "out_tokens", torch.int32, (b, n), dev)
    opp = _ptr(out_parents, "out_parents", torch.int32, (b, n), dev)
    d = ssq_beam_desc(_DTYPES[logits.dtype], _int32(b, "batch"), _int32(m, "beams"), _int32(v, "vocab"),
                      _int32(n, "nselect"), _int32(pad_token, "pad_token"), row)
    on = _stream_ptr(stream, dev)
    ws, wp, wn = _workspace(workspace, lib.ssq_beam_workspace(d), stream, dev)
    _check(lib.ssq_beam_select(d, logits.data_ptr(), sp, fp, osp, otp, opp, wp, wn, on), "ssq_beam_select")


def ssq_state_reorder(states, parents, stream=None):
    """States follow their beams: of every group of ``parents.shape[1]`` consecutive sequences, sequence j becomes
    what sequence ``parents[group, j]`` of the group was.  ``states``: a State or a sequence of them (the layers of a
    model), each of ``parents.numel()`` sequences; parents int32 ``[groups, beams]``."""
    dev = torch.cuda.current_device()
    states = [states] if isinstance(states, State) else states
    if not isinstance(parents, torch.Tensor) or parents.dim() != 2:
        raise ValueError("parents must be a tensor [groups, beams]")
    p = _ptr(parents, "parents", torch.int32, parents.shape, dev)
    batch = parents.numel()
    for s in states:
        if s.desc.batch != batch:
            raise ValueError(f"a state has {s.desc.batch} sequences, parents names {batch}")
    n = len(states)
    _check(lib.ssq_state_reorder(_handles(states), n, p, parents.shape[1], _stream_ptr(stream, dev)), "ssq_state_reorder")


def _handles(states):
    return (ctypes.c_void_p * max(1, len(states)))(*[s.handle for s in states])


def ssq_state_move(states, to, from_, sources=None, stream=None):
    """Moves between sequences, one after the other: sequence ``to[i]`` of every state becomes what sequence ``from_[i]``
    of its source is then, or the zero state where ``from_[i]`` is -1.  ``states``: a State or a sequence of them (the
    layers of a model); ``sources``: the same number of States of another pool, None for the states themselves; to,
    from_: int32 ``[nmoves]`` on the device."""
    dev = _current_device()
    states = [states] if isinstance(states, State) else states
    sources = [sources] if isinstance(sources, State) else sources
    if sources is not None and len(sources) != len(states):
        raise ValueError(f"{len(states)} states have {len(sources)} sources")
    n = to.numel() if isinstance(to, torch.Tensor) else 0
    tp = _ptr(to, "to", torch.int32, (n,), dev)
    fp = _ptr(from_, "from_", torch.int32, (n,), dev)
    _check(lib.ssq_state_move(_handles(states), None if sources is None else _handles(sources), len(states), tp, fp,
                              _int32(n, "nmoves"), _stream_ptr(stream, dev)), "ssq_state_move")


def _rows(t, name: str, dtype, shape, dev: int):
    """Pointer and stride between tokens of a [tokens][channels] tensor whose tokens are packed."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        _refuse(t, name, dtype, shape, dev)
    between, within = t.stride()
    if within != 1 and shape[1] != 1:
        raise ValueError(f"the channels of {name} must be packed within a token")
    return t.data_ptr(), between if shape[0] > 1 else shape[1]


def _token_rows(t, name: str):
    """dtype and shape of a [tokens][channels] tensor."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES or t.dim() != 2:
        raise ValueError(f"{name} must be a float32, bfloat16 or float16 tensor [tokens, channels]")
    return t.dtype, t.shape


def ssq_gated_checkpoint_rows(nseq: int, tokens: int) -> int:
    """Rows of the float32 checkpoints ``[rows, channels]`` that ``ssq_gated_scan`` writes for its gradient."""
    if tokens >= 1 << 63:
        raise ValueError("tokens is more than 63 bits hold")
    n = lib.ssq_gated_checkpoint_rows(_int32(nseq, "nseq"), tokens)
    if n < 0:
        raise ValueError("sizes must not be negative or more than a call takes")
    return n


def ssq_gated_workspace(channels: int, nseq: int, tokens: int) -> int:
    """Bytes of workspace ``ssq_gated_scan`` and ``ssq_gated_scan_backward`` need for these sizes."""
    if tokens >= 1 << 63:
        raise ValueError("tokens is more than 63 bits hold")
    n = lib.ssq_gated_workspace(_int32(channels, "channels"), _int32(nseq, "nseq"), tokens)
    if n == _SIZE_MAX:
        raise ValueError(ssq_last_error())
    return n


def _sequences(cu_seqlens, slots, dev: int):
    nseq = cu_seqlens.numel() - 1 if isinstance(cu_seqlens, torch.Tensor) else 0
    if nseq < 0:
        raise ValueError("cu_seqlens has nseq + 1 entries")
    cu = _ptr(cu_seqlens, "cu_seqlens", torch.int32, (nseq + 1,), dev)
    return nseq, cu, None if slots is None else _ptr(slots, "slots", torch.int32, (nseq,), dev)


def _gated_io(x, g, o, gate: int, input: int, dev: int):
    dtype, shape = _token_rows(x, "x")
    xp, xs = _rows(x, "x", dtype, shape, dev)
    gp, gs = _rows(g, "g", dtype, shape, dev)
    op, os_ = _rows(o, "o", dtype, shape, dev)
    return shape[0], ssq_gated_io(_DTYPES[dtype], _int32(gate, "gate"), _int32(input, "input"), _int32(shape[1], "channels"),
                                  xp, gp, op, xs, gs, os_)


def _state_handle(state: State | None):
    """The handle of a state that may be left out; a freed one is not one left out."""
    if state is not None and state.handle is None:
        raise ValueError("the state has been freed")
    return None if state is None else state.handle


def ssq_gated_scan(state: State | None, x, g, o, cu_seqlens, gate: int = SSQ_GATE_LOG, input: int = SSQ_INPUT_PLAIN,
                   slots=None, fresh=None, checkpoints=None, workspace: torch.Tensor | None = None, stream=None):
    """A gated linear recurrence over ragged sequences: ``h = a h + s x`` in every channel, ``o = h``.

    x, g, o ``[tokens, channels]`` (float32, bfloat16 or float16; any stride between tokens that is a multiple of 16
    bytes and not below a token's row), cu_seqlens int32 ``[nseq + 1]``, slots int32 ``[nseq]`` or None, fresh uint8 or
    bool ``[nseq]`` or None; all on the device.  ``state``: an SSQ_GATED state, or None to start from zero.
    ``checkpoints``: float32 ``[ssq_gated_checkpoint_rows(nseq, tokens), channels]`` for the gradient, or None.
    ``workspace``: uint8, at least ``ssq_gated_workspace`` bytes, or None to take it from torch."""
    dev = _current_device()
    tokens, io = _gated_io(x, g, o, gate, input, dev)
    nseq, cu, sp = _sequences(cu_seqlens, slots, dev)
    fp = _flags(fresh, "fresh", (nseq,), dev)
    cp = None
    if checkpoints is not None:
        cp = _ptr(checkpoints, "checkpoints", torch.float32, (ssq_gated_checkpoint_rows(nseq, tokens), io.channels), dev)
    on = _stream_ptr(stream, dev)
    ws, wp, wn = _workspace(workspace, ssq_gated_workspace(io.channels, nseq, tokens), stream, dev)
    _check(lib.ssq_gated_scan(_state_handle(state), io, nseq, tokens, cu, sp, fp, cp, wp, wn, on),
           "ssq_gated_scan")


def ssq_gated_scan_backward(checkpoints, x, g, do, dx, dg, cu_seqlens, gate: int = SSQ_GATE_LOG,
                            input: int = SSQ_INPUT_PLAIN, dlast=None, dfirst=None, state: State | None = None, slots=None,
                            workspace: torch.Tensor | None = None, stream=None):
    """Gradients of ``ssq_gated_scan`` (the same x, g, cu_seqlens, gate, input, state and slots, and the checkpoints that
    it wrote): dx and dg from do, the gradient of o (all shaped and strided as x).  dlast: float32 ``[nseq, channels]``,
    the gradient of the last states, or None; dfirst: the same of the states the sequences started from is written."""
    dev = _current_device()
    dtype, shape = _token_rows(x, "x")
    tokens, channels = shape
    ptrs, strides = zip(*[_rows(t, name, dtype, shape, dev)
                          for t, name in ((x, "x"), (g, "g"), (do, "do"), (dx, "dx"), (dg, "dg"))])
    nseq, cu, sp = _sequences(cu_seqlens, slots, dev)
    ends = [None if t is None else _ptr(t, name, torch.float32, (nseq, channels), dev)
            for t, name in ((dlast, "dlast"), (dfirst, "dfirst"))]
    io = ssq_gated_grad(_DTYPES[dtype], _int32(gate, "gate"), _int32(input, "input"), _int32(channels, "channels"), *ptrs,
                        *strides, *ends)
    cp = _ptr(checkpoints, "checkpoints", torch.float32, (ssq_gated_checkpoint_rows(nseq, tokens), channels), dev)
    on = _stream_ptr(stream, dev)
    ws, wp, wn = _workspace(workspace, ssq_gated_workspace(channels, nseq, tokens), stream, dev)
    _check(lib.ssq_gated_scan_backward(_state_handle(state), io, nseq, tokens, cu, sp, cp, wp, wn, on),
           "ssq_gated_scan_backward")


def ssq_gated_step(state: State, x, g, o, gate: int = SSQ_GATE_LOG, input: int = SSQ_INPUT_PLAIN, slots=None, stream=None):
    """One token of the gated recurrence for ``nseq = x.shape[0]`` sequences: row i of the tensors (as in
    ``ssq_gated_scan``) is sequence ``slots[i]`` of the state, or sequence i without slots."""
    dev = _current_device()
    nseq, io = _gated_io(x, g, o, gate, input, dev)
    sp = None if slots is None else _ptr(slots, "slots", torch.int32, (nseq,), dev)
    _check(lib.ssq_gated_step(state.handle, io, _int32(nseq, "nseq"), sp, _stream_ptr(stream, dev)), "ssq_gated_step")


def ssq_group_norm_workspace(groups: int, width: int, tokens: int) -> int:
    """Bytes of workspace ``ssq_group_norm_backward`` needs."""
    if tokens >= 1 << 63:
        raise ValueError("tokens is more than 63 bits hold")
    n = lib.ssq_group_norm_workspace(_int32(groups, "groups"), _int32(width, "width"), tokens)
    if n == _SIZE_MAX:
        raise ValueError(ssq_last_error())
    return n


def _norm_io(x, z, weight, bias, act: int, center: bool, eps: float, dev: int):
    if not isinstance(x, torch.Tensor) or x.dtype not in _DTYPES or x.dim() != 3:
        raise ValueError("x must be a float32, bfloat16 or float16 tensor [tokens, groups, width]")
    shape = x.shape
    xp, xs = _tokens(x, "x", x.dtype, shape, dev)
    zp, zs = (None, 0) if z is None else _tokens(z, "z", x.dtype, shape, dev)
    tokens, groups, width = shape
    if tokens == 0:  # no row is read: any stride serves
        xs = zs = groups * width
    wp = None if weight is None else _ptr(weight, "weight", torch.float32, shape[1:], dev)
    bp = None if bias is None else _ptr(bias, "bias", torch.float32, shape[1:], dev)
    return ssq_norm_io(_DTYPES[x.dtype], _int32(act, "act"), 1 if center else 0, _int32(groups, "groups"), _int32(width, "width"),
                       eps, wp, bp, xp, zp, xs, zs)


def ssq_group_norm(x, y, weight=None, bias=None, z=None, act: int = SSQ_ACT_SILU, center: bool = True, eps: float = 1e-5,
                   stream=None):
    """Group norm with an activation, channels last: every token's groups normalised by themselves.

    x, z, y ``[tokens, groups, width]`` (float32, bfloat16 or float16; any stride between tokens that is a multiple of 16
    bytes and not below a token's row), z None for SSQ_ACT_SILU; weight, bias ``[groups, width]`` float32 or None.
    ``center``: mean and variance, else the root mean square alone."""
    dev = _current_device()
    io = _norm_io(x, z, weight, bias, act, center, eps, dev)
    tokens, row = x.shape[0], io.groups * io.width
    yp, ys = _tokens(y, "y", x.dtype, x.shape, dev)
    _check(lib.ssq_group_norm(io, yp, ys if tokens else row, tokens, _stream_ptr(stream, dev)), "ssq_group_norm")


def ssq_group_norm_backward(dy, x, dx, weight=None, bias=None, z=None, dz=None, dweight=None, dbias=None,
                            act: int = SSQ_ACT_SILU, center: bool = True, eps: float = 1e-5,
                            workspace: torch.Tensor | None = None, stream=None):
    """Gradients of ``ssq_group_norm`` (the same x, z, weight, bias, act, center and eps): dx and dz from dy (all shaped
    and strided as x), and dweight and dbias, float32 ``[groups, width]``, where they are given."""
    dev = _current_device()
    io = _norm_io(x, z, weight, bias, act, center, eps, dev)
    tokens, groups, width = x.shape
    row = groups * width
    pairs = [(None, row) if t is None and name == "dz" else _tokens(t, name, x.dtype, x.shape, dev)
             for t, name in ((dy, "dy"), (dx, "dx"), (dz, "dz"))]
    wp, bp = (None if t is None else _ptr(t, name, torch.float32, x.shape[1:], dev) for t, name in ((dweight, "dweight"), (dbias, "dbias")))
    strides = [s if tokens else row for _, s in pairs]
    grad = ssq_norm_grad(*(p for p, _ in pairs), wp, bp, *strides)
    on = _stream_ptr(stream, dev)
    ws, wsp, wn = _workspace(workspace, ssq_group_norm_workspace(groups, width, tokens), stream, dev)
    _check(lib.ssq_group_norm_backward(io, grad, tokens, wsp, wn, on), "ssq_group_norm_backward")
