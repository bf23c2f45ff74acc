// ssq_api.cpp -- the C ABI of include/ssq.h: argument validation, state
// layout and ownership, launch configuration and error reporting.  Every
// argument is checked before anything is enqueued, so a rejected call changes
// nothing; kernels run asynchronously on the caller's stream.
#include "ssq.h"

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <new>
#include <string>

#include "ssq_internal.h"
#include "ssq_ops.h"

struct ssq_state {
    ssq_desc desc;
    ssq_layout lay;
    void* storage;
    bool owned;
    int device;
    int32_t rounding; // ssq_rounding
    uint64_t sr_seed; // stochastic rounding: generator seed (the next token is in the storage)
};

namespace {

thread_local std::string g_last_error;

ssq_status fail(ssq_status st, const std::string& msg)
{
    g_last_error = msg;
    return st;
}

ssq_status ok()
{
    g_last_error.clear();
    return SSQ_OK;
}

bool fmt_valid(int f) { return f >= SSQ_FP32 && f <= SSQ_DAMP; }
bool fmt_quant(int f) { return f != SSQ_FP32; }
bool fmt_asym(int f) { return f == SSQ_INT8_ASYM || f == SSQ_INT4_ASYM || f == SSQ_DAMP; }
int fmt_bits(int f)
{
    return f == SSQ_FP32 ? 32 : (f == SSQ_INT8_SYM || f == SSQ_INT8_ASYM || f == SSQ_DAMP ? 8 : 4);
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

bool mul_ok(size_t a, size_t b, size_t* out)
{
    if (a != 0 && b > SIZE_MAX / a) return false;
    *out = a * b;
    return true;
}

ssq_status check_desc(const ssq_desc* d, ssq_layout* lay)
{
    if (!d) return fail(SSQ_ERR_INVALID_ARG, "desc is NULL");
    if (d->kind != SSQ_MAMBA2 && d->kind != SSQ_DELTA && d->kind != SSQ_GATED) return fail(SSQ_ERR_INVALID_ARG, "unknown state kind");
    if (!fmt_valid(d->format)) return fail(SSQ_ERR_INVALID_ARG, "unknown format");
    if (d->batch <= 0 || d->nheads <= 0 || d->ngroups <= 0 || d->rows_per_head <= 0 || d->row_len <= 0)
        return fail(SSQ_ERR_INVALID_ARG, "every dimension must be positive");
    if (d->nheads % d->ngroups != 0) return fail(SSQ_ERR_INVALID_ARG, "ngroups must divide nheads");
    if (d->kind == SSQ_DELTA && d->ngroups != 1) return fail(SSQ_ERR_INVALID_ARG, "a delta state has ngroups == 1");
    if (d->kind == SSQ_GATED) {
        if (d->nheads != 1 || d->rows_per_head != 1)
            return fail(SSQ_ERR_INVALID_ARG, "a gated state has nheads == ngroups == rows_per_head == 1");
        if (d->format != SSQ_FP32) return fail(SSQ_ERR_UNSUPPORTED, "a gated state is fp32");
        if (d->row_len % 8 != 0 || d->row_len > ssq::kMaxChannels)
            return fail(SSQ_ERR_UNSUPPORTED, "a gated state has a multiple of 8 channels, 2^20 at most");
    } else if (d->row_len != 128) {
        return fail(SSQ_ERR_UNSUPPORTED, "kernels are built for row_len == 128");
    }
    if (d->kind == SSQ_MAMBA2 && d->rows_per_head % 16 != 0)
        return fail(SSQ_ERR_UNSUPPORTED, "Mamba-2 kernels need rows_per_head to be a multiple of 16");
    if (d->kind == SSQ_DELTA && d->rows_per_head != 128)
        return fail(SSQ_ERR_UNSUPPORTED, "delta kernels are built for dk == 128");
    if (d->format == SSQ_DAMP && d->kind != SSQ_DELTA)
        return fail(SSQ_ERR_UNSUPPORTED, "the two-tier format is a delta-rule state");

    ssq_layout l;
    size_t rows;
    if (!mul_ok((size_t)d->batch, (size_t)d->nheads, &rows) || !mul_ok(rows, (size_t)d->rows_per_head, &rows))
        return fail(SSQ_ERR_INVALID_ARG, "state size overflows size_t");
    const int bits = fmt_bits(d->format);
    l.rows = rows;
    l.row_bytes = (size_t)d->row_len * (size_t)bits / 8;
    // the two-tier format keeps its uint8 rows in codes/scale/zero and the half rows apart
    size_t qrows = rows, hi_bytes = 0;
    if (d->format == SSQ_DAMP) {
        const size_t mats = rows / (size_t)d->rows_per_head;
        qrows = mats * (size_t)(d->rows_per_head - SSQ_DAMP_NHI);
        hi_bytes = mats * SSQ_DAMP_NHI * (size_t)d->row_len * 2;
    }
    size_t codes_bytes, meta_bytes;
    if (!mul_ok(qrows, l.row_bytes, &codes_bytes) || !mul_ok(qrows, 4, &meta_bytes) || codes_bytes > SIZE_MAX / 2)
        return fail(SSQ_ERR_INVALID_ARG, "state size overflows size_t");
    l.codes_offset = 0;
    size_t end = align256(codes_bytes);
    l.scale_offset = 0;
    l.zero_offset = 0;
    if (fmt_quant(d->format)) {
        l.scale_offset = end;
        end = align256(end + meta_bytes);
        if (fmt_asym(d->format)) {
            l.zero_offset = end;
            end = align256(end + meta_bytes);
        }
    }
    l.hi_offset = 0;
    if (hi_bytes) {
        l.hi_offset = end;
        end = align256(end + hi_bytes);
    }
    // quantized formats: the stochastic-rounding token counter
    l.counter_offset = 0;
    if (fmt_quant(d->format)) {
        l.counter_offset = end;
        end = align256(end + 8);
    }
    l.total_bytes = end;
    if (lay) *lay = l;
    return SSQ_OK;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// compute units of a device, cached (read-only after the first query)
int num_cus(int dev)
{
    static std::atomic<int> cache[64];
    if (dev < 0 || dev >= 64) return 256;
    int v = cache[dev].load(std::memory_order_relaxed);
    if (v > 0) return v;
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) n = 256;
    cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

ssq_status from_hip(hipError_t e, const char* what)
{
    if (e == hipSuccess) return ok();
    return fail(SSQ_ERR_DEVICE, std::string(what) + ": " + hipGetErrorString(e));
}

ssq_status check_device(const ssq_state* st)
{
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return from_hip(e, "hipGetDevice");
    if (dev != st->device) return fail(SSQ_ERR_INVALID_ARG, "the state lives on another device than the current one");
    return SSQ_OK;
}

uint8_t* codes_ptr(const ssq_state* st) { return (uint8_t*)st->storage + st->lay.codes_offset; }
float* scale_ptr(const ssq_state* st)
{
    return fmt_quant(st->desc.format) ? (float*)((uint8_t*)st->storage + st->lay.scale_offset) : nullptr;
}
float* zero_ptr(const ssq_state* st)
{
    return fmt_asym(st->desc.format) ? (float*)((uint8_t*)st->storage + st->lay.zero_offset) : nullptr;
}
uint64_t* counter_ptr(const ssq_state* st)
{
    return fmt_quant(st->desc.format) ? (uint64_t*)((uint8_t*)st->storage + st->lay.counter_offset) : nullptr;
}
uint16_t* hi_ptr(const ssq_state* st)
{
    return st->desc.format == SSQ_DAMP ? (uint16_t*)((uint8_t*)st->storage + st->lay.hi_offset) : nullptr;
}
// rows of the state that are rounded to a grid (the counter space of stochastic rounding)
int64_t grid_rows(const ssq_state* st)
{
    if (st->desc.format != SSQ_DAMP) return (int64_t)st->lay.rows;
    return (int64_t)(st->lay.rows / 128) * (128 - SSQ_DAMP_NHI);
}

// a gated state's numbers, which are fp32 as they stand; a launch stays below 2^32 work-items
hipError_t copy_state(void* dst, const void* src, size_t bytes, hipStream_t st)
{
    const size_t most = (size_t)1 << 35;
    for (size_t at = 0; at < bytes; at += most) {
        const hipError_t e = ssq::launch_stream_copy((uint8_t*)dst + at, (const uint8_t*)src + at,
                                                     (int64_t)(bytes - at < most ? bytes - at : most), st);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

#define SSQ_REQUIRE(cond, status, msg)            \
    do {                                           \
        if (!(cond)) return fail((status), (msg)); \
    } while (0)

} // namespace

extern "C" {

size_t ssq_state_bytes(const ssq_desc* desc)
{
    ssq_layout l;
    if (check_desc(desc, &l) != SSQ_OK) return 0;
    return l.total_bytes;
}

ssq_status ssq_state_layout(const ssq_desc* desc, ssq_layout* layout)
{
    SSQ_REQUIRE(layout, SSQ_ERR_INVALID_ARG, "layout is NULL");
    ssq_status s = check_desc(desc, layout);
    return s == SSQ_OK ? ok() : s;
}

ssq_status ssq_alloc_state(const ssq_desc* desc, void* storage, const float* init, void* stream, ssq_state** out)
{
    SSQ_REQUIRE(out, SSQ_ERR_INVALID_ARG, "out is NULL");
    ssq_layout lay;
    ssq_status s = check_desc(desc, &lay);
    if (s != SSQ_OK) return s;
    SSQ_REQUIRE(aligned(storage, 256), SSQ_ERR_INVALID_ARG, "storage must be 256-byte aligned");
    SSQ_REQUIRE(aligned(init, 16), SSQ_ERR_INVALID_ARG, "init must be 16-byte aligned");
    if (!storage) {
        const char* hook = std::getenv("SSQ_TEST_FAIL_ALLOC");
        if (hook && hook[0] == '1') return fail(SSQ_ERR_ALLOC, "allocation failure forced by SSQ_TEST_FAIL_ALLOC");
    }
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return from_hip(e, "hipGetDevice");

    ssq_state* st = new (std::nothrow) ssq_state;
    SSQ_REQUIRE(st, SSQ_ERR_ALLOC, "out of host memory");
    st->desc = *desc;
    st->lay = lay;
    st->device = dev;
    st->owned = false;
    st->storage = storage;
    st->rounding = SSQ_ROUND_NEAREST;
    st->sr_seed = 0;
    if (!storage) {
        void* p = nullptr;
        e = hipMalloc(&p, lay.total_bytes);
        if (e != hipSuccess || !p) {
            (void)hipGetLastError();
            delete st;
            return fail(SSQ_ERR_ALLOC, std::string("hipMalloc: ") + hipGetErrorString(e));
        }
        st->storage = p;
        st->owned = true;
    }
    hipStream_t hs = (hipStream_t)stream;
    // every byte of the storage is written: zero first (padding, the token counter), then the
    // quantized rows of `init`
    e = ssq::launch_zero_fill(st->storage, lay.total_bytes, hs);
    if (e == hipSuccess && init && desc->kind == SSQ_GATED) {
        e = copy_state(st->storage, init, lay.rows * lay.row_bytes, hs);
    } else if (e == hipSuccess && init) {
        ssq::QArgs a{};
        a.codes = codes_ptr(st);
        a.scale = scale_ptr(st);
        a.zero = zero_ptr(st);
        a.h32 = (float*)codes_ptr(st);
        a.hi = hi_ptr(st);
        a.in = init;
        a.rows = (int64_t)lay.rows;
        e = desc->format == SSQ_DAMP ? ssq::launch_damp_rows(a, false, hs)
                                     : ssq::launch_rows(desc->format, a, false, hs);
    }
    if (e != hipSuccess) {
        if (st->owned) (void)hipFree(st->storage);
        delete st;
        return from_hip(e, "state initialisation launch");
    }
    *out = st;
    return ok();
}

ssq_status ssq_free_state(ssq_state* st)
{
    if (!st) return ok();
    hipError_t e = hipSuccess;
    if (st->owned) e = hipFree(st->storage);
    delete st;
    return from_hip(e, "hipFree");
}

ssq_status ssq_state_info(const ssq_state* st, ssq_desc* desc, void** storage, ssq_layout* layout)
{
    SSQ_REQUIRE(st, SSQ_ERR_INVALID_ARG, "state is NULL");
    if (desc) *desc = st->desc;
    if (storage) *storage = st->storage;
    if (layout) *layout = st->lay;
    return ok();
}

// the stochastic-rounding arguments of the next call on a state (the launcher sets the
// call's wave count and the tokens it consumes)
static ssq::SrArgs sr_args(const ssq_state* st)
{
    ssq::SrArgs r{};
    r.on = st->rounding == SSQ_ROUND_STOCHASTIC;
    r.seed = st->sr_seed;
    r.rows = grid_rows(st);
    r.ctr = counter_ptr(st);
    return r;
}

// after a stochastically rounded call's step kernels: the state's next token moves on
static ssq_status advance(const ssq_state* st, uint64_t tokens, hipStream_t stream)
{
    if (st->rounding != SSQ_ROUND_STOCHASTIC) return ok();
    return from_hip(ssq::launch_advance_counter(counter_ptr(st), tokens, stream), "token counter launch");
}

ssq_status ssq_set_rounding(ssq_state* st, int32_t mode, uint64_t seed, uint64_t step, void* stream)
{
    SSQ_REQUIRE(st, SSQ_ERR_INVALID_ARG, "state is NULL");
    SSQ_REQUIRE(mode == SSQ_ROUND_NEAREST || mode == SSQ_ROUND_STOCHASTIC, SSQ_ERR_INVALID_ARG,
                "unknown rounding mode");
    SSQ_REQUIRE(mode == SSQ_ROUND_NEAREST || fmt_quant(st->desc.format), SSQ_ERR_UNSUPPORTED,
                "the fp32 state is not rounded");
    SSQ_REQUIRE(mode == SSQ_ROUND_STOCHASTIC || step == 0 || fmt_quant(st->desc.format), SSQ_ERR_UNSUPPORTED,
                "the fp32 state has no token counter");
    ssq_status s = check_device(st);
    if (s != SSQ_OK) return s;
    if (fmt_quant(st->desc.format)) {
        s = from_hip(ssq::launch_set_counter(counter_ptr(st), step, (hipStream_t)stream), "token counter launch");
        if (s != SSQ_OK) return s;
    }
    st->rounding = mode;
    st->sr_seed = seed;
    return ok();
}

ssq_status ssq_get_rounding(const ssq_state* st, int32_t* mode, uint64_t* seed, uint64_t* step, void* stream)
{
    SSQ_REQUIRE(st, SSQ_ERR_INVALID_ARG, "state is NULL");
    uint64_t next = 0;
    if (step && fmt_quant(st->desc.format)) {
        ssq_status s = check_device(st);
        if (s != SSQ_OK) return s;
        hipError_t e = hipMemcpyAsync(&next, counter_ptr(st), sizeof next, hipMemcpyDeviceToHost, (hipStream_t)stream);
        if (e == hipSuccess) e = hipStreamSynchronize((hipStream_t)stream);
        if (e != hipSuccess) return from_hip(e, "reading the token counter");
    }
    if (mode) *mode = st->rounding;
    if (seed) *seed = st->sr_seed;
    if (step) *step = next;
    return ok();
}

static ssq_status fill_m2(ssq_state* st, const float* x, const float* dt, const float* A, const float* B,
                          const float* C, const float* D, float* y, int32_t readout, ssq::M2Args* a)
{
    SSQ_REQUIRE(st, SSQ_ERR_INVALID_ARG, "state is NULL");
    SSQ_REQUIRE(st->desc.kind == SSQ_MAMBA2, SSQ_ERR_KIND_MISMATCH, "a Mamba-2 call on a state of another kind");
    SSQ_REQUIRE(x && dt && A && B && C && D && y, SSQ_ERR_INVALID_ARG, "an input or output pointer is NULL");
    SSQ_REQUIRE(aligned(x, 4) && aligned(dt, 4) && aligned(A, 4) && aligned(D, 4) && aligned(y, 4),
                SSQ_ERR_INVALID_ARG, "x, dt, A, D and y must be 4-byte aligned");
    SSQ_REQUIRE(aligned(B, 16) && aligned(C, 16), SSQ_ERR_INVALID_ARG, "B and C must be 16-byte aligned");
    SSQ_REQUIRE(readout == SSQ_READ_POST_QUANT || readout == SSQ_READ_PRE_QUANT, SSQ_ERR_INVALID_ARG,
                "unknown readout");
    ssq_status s = check_device(st);
    if (s != SSQ_OK) return s;
    *a = ssq::M2Args{};
    a->codes = codes_ptr(st);
    a->scale = scale_ptr(st);
    a->zero = zero_ptr(st);
    a->h32 = (float*)codes_ptr(st);
    a->x = x;
    a->dt = dt;
    a->A = A;
    a->Bm = B;
    a->Cm = C;
    a->D = D;
    a->y = y;
    a->Bsz = st->desc.batch;
    a->H = st->desc.nheads;
    a->G = st->desc.ngroups;
    a->P = st->desc.rows_per_head;
    a->T = 1;
    return SSQ_OK;
}

ssq_status ssq_decode_step(ssq_state* st, const float* x, const float* dt, const float* A, const float* B,
                           const float* C, const float* D, float* y, int32_t readout, void* stream)
{
    ssq::M2Args a;
    ssq_status s = fill_m2(st, x, dt, A, B, C, D, y, readout, &a);
    if (s != SSQ_OK) return s;
    a.sr = sr_args(st);
    s = from_hip(ssq::launch_m2_step(st->desc.format, a, readout == SSQ_READ_PRE_QUANT, num_cus(st->device),
                                     (hipStream_t)stream),
                 "decode step launch");
    return s == SSQ_OK ? advance(st, 1, (hipStream_t)stream) : s;
}

ssq_status ssq_scan(ssq_state* st, int32_t T, const float* x, const float* dt, const float* A, const float* B,
                    const float* C, const float* D, float* y, int32_t readout, void* stream)
{
    ssq::M2Args a;
    ssq_status s = fill_m2(st, x, dt, A, B, C, D, y, readout, &a);
    if (s != SSQ_OK) return s;
    SSQ_REQUIRE(T > 0, SSQ_ERR_INVALID_ARG, "T must be positive");
    a.T = T;
    a.sr = sr_args(st);
    s = from_hip(ssq::launch_m2_scan(st->desc.format, a, readout == SSQ_READ_PRE_QUANT, num_cus(st->device),
                                     (hipStream_t)stream),
                 "scan launch");
    return s == SSQ_OK ? advance(st, (uint64_t)T, (hipStream_t)stream) : s;
}

ssq_status ssq_prefill(ssq_state* st, int32_t T, int32_t chunk, const float* x, const float* dt, const float* A,
                       const float* B, const float* C, const float* D, float* y, int32_t readout, void* stream)
{
    ssq::M2Args a;
    ssq_status s = fill_m2(st, x, dt, A, B, C, D, y, readout, &a);
    if (s != SSQ_OK) return s;
    SSQ_REQUIRE(T > 0, SSQ_ERR_INVALID_ARG, "T must be positive");
    SSQ_REQUIRE(chunk > 0, SSQ_ERR_INVALID_ARG, "chunk must be positive");
    a.T = T;
    a.sr = sr_args(st);
    s = from_hip(ssq::launch_m2_prefill(st->desc.format, a, chunk, readout == SSQ_READ_PRE_QUANT, num_cus(st->device),
                                        (hipStream_t)stream),
                 "prefill launch");
    return s == SSQ_OK ? advance(st, (uint64_t)T, (hipStream_t)stream) : s;
}

static ssq_status delta_common(ssq_state* st, const float* q, const float* k, const float* v, const float* alpha,
                               const float* beta, float* o, int32_t readout, void* stream, bool kda)
{
    SSQ_REQUIRE(st, SSQ_ERR_INVALID_ARG, "state is NULL");
    SSQ_REQUIRE(st->desc.kind == SSQ_DELTA, SSQ_ERR_KIND_MISMATCH, "a delta-rule call on a state of another kind");
    SSQ_REQUIRE(q && k && v && alpha && beta && o, SSQ_ERR_INVALID_ARG, "an input or output pointer is NULL");
    SSQ_REQUIRE(aligned(q, 4) && aligned(k, 4) && aligned(alpha, 4) && aligned(beta, 4) && aligned(o, 4),
                SSQ_ERR_INVALID_ARG, "q, k, alpha, beta and o must be 4-byte aligned");
    SSQ_REQUIRE(aligned(v, 16), SSQ_ERR_INVALID_ARG, "v must be 16-byte aligned");
    SSQ_REQUIRE(readout == SSQ_READ_POST_QUANT || readout == SSQ_READ_PRE_QUANT, SSQ_ERR_INVALID_ARG,
                "unknown readout");
    ssq_status s = check_device(st);
    if (s != SSQ_OK) return s;
    ssq::DeltaArgs a{};
    a.codes = codes_ptr(st);
    a.scale = scale_ptr(st);
    a.zero = zero_ptr(st);
    a.h32 = (float*)codes_ptr(st);
    a.q = q;
    a.k = k;
    a.v = v;
    a.alpha = alpha;
    a.beta = beta;
    a.o = o;
    a.nmat = (int64_t)st->desc.batch * st->desc.nheads;
    a.kda = kda ? 1 : 0;
    a.sr = sr_args(st);
    a.hi = hi_ptr(st);
    if (st->desc.format == SSQ_DAMP) {
        SSQ_REQUIRE(!kda, SSQ_ERR_UNSUPPORTED, "the two-tier state takes the scalar-decay step only");
        s = from_hip(ssq::launch_damp_step(a, readout == SSQ_READ_PRE_QUANT, (hipStream_t)stream),
                     "two-tier delta step launch");
    } else {
        s = from_hip(ssq::launch_delta_step(st->desc.format, a, readout == SSQ_READ_PRE_QUANT, (hipStream_t)stream),
                     kda ? "KDA step launch" : "delta step launch");
    }
    return s == SSQ_OK ? advance(st, 1, (hipStream_t)stream) : s;
}

ssq_status ssq_delta_step(ssq_state* st, const float* q, const float* k, const float* v, const float* alpha,
                          const float* beta, float* o, int32_t readout, void* stream)
{
    return delta_common(st, q, k, v, alpha, beta, o, readout, stream, false);
}

ssq_status ssq_kda_step(ssq_state* st, const float* q, const float* k, const float* v, const float* alpha,
                        const float* beta, float* o, int32_t readout, void* stream)
{
    return delta_common(st, q, k, v, alpha, beta, o, readout, stream, true);
}

ssq_status ssq_dequant(const ssq_state* st, float* out, void* stream)
{
    SSQ_REQUIRE(st, SSQ_ERR_INVALID_ARG, "state is NULL");
    SSQ_REQUIRE(out, SSQ_ERR_INVALID_ARG, "out is NULL");
    SSQ_REQUIRE(aligned(out, 16), SSQ_ERR_INVALID_ARG, "out must be 16-byte aligned");
    ssq_status s = check_device(st);
    if (s != SSQ_OK) return s;
    if (st->desc.kind == SSQ_GATED)
        return from_hip(copy_state(out, st->storage, st->lay.rows * st->lay.row_bytes, (hipStream_t)stream),
                        "dequant launch");
    ssq::QArgs a{};
    a.codes = codes_ptr(st);
    a.scale = scale_ptr(st);
    a.zero = zero_ptr(st);
    a.h32 = (float*)codes_ptr(st);
    a.out = out;
    a.rows = (int64_t)st->lay.rows;
    a.hi = hi_ptr(st);
    if (st->desc.format == SSQ_DAMP)
        return from_hip(ssq::launch_damp_rows(a, true, (hipStream_t)stream), "dequant launch");
    return from_hip(ssq::launch_rows(st->desc.format, a, true, (hipStream_t)stream), "dequant launch");
}

ssq_status ssq_stream_copy(void* dst, const void* src, size_t bytes, void* stream)
{
    SSQ_REQUIRE(dst && src, SSQ_ERR_INVALID_ARG, "dst and src must not be NULL");
    SSQ_REQUIRE(aligned(dst, 16) && aligned(src, 16), SSQ_ERR_INVALID_ARG, "dst and src must be 16-byte aligned");
    SSQ_REQUIRE(bytes % 16 == 0, SSQ_ERR_INVALID_ARG, "bytes must be a multiple of 16");
    SSQ_REQUIRE(bytes <= ((size_t)1 << 40), SSQ_ERR_INVALID_ARG, "bytes must not exceed 2^40");
    const uintptr_t s = (uintptr_t)src, d = (uintptr_t)dst;
    SSQ_REQUIRE(d + bytes <= s || s + bytes <= d, SSQ_ERR_INVALID_ARG, "dst and src must not overlap");
    return from_hip(ssq::launch_stream_copy(dst, src, (int64_t)bytes, (hipStream_t)stream), "copy launch");
}

// ---------------------------------------------------------------------------
// linear attention
// ---------------------------------------------------------------------------
constexpr int64_t kMostTokens = 0x7FFFFF80 - 1; // of a prompt call

static bool dtype_valid(int d) { return d >= SSQ_DTYPE_FP32 && d <= SSQ_DTYPE_FP16; }

static ssq_status fill_linattn(ssq_state* st, const ssq_linattn_io* io, int32_t nseq, int64_t tokens,
                               const int32_t* slots, int64_t most_rows, ssq::LinArgs* a)
{
    SSQ_REQUIRE(st && io, SSQ_ERR_INVALID_ARG, "state or io is NULL");
    SSQ_REQUIRE(st->desc.kind == SSQ_MAMBA2, SSQ_ERR_KIND_MISMATCH, "linear attention runs on an SSQ_MAMBA2 state");
    SSQ_REQUIRE(dtype_valid(io->dtype), SSQ_ERR_INVALID_ARG, "unknown dtype");
    SSQ_REQUIRE(nseq >= 0 && tokens >= 0, SSQ_ERR_INVALID_ARG, "nseq and tokens must not be negative");
    SSQ_REQUIRE(nseq <= most_rows / ((int64_t)st->desc.nheads * st->desc.rows_per_head), SSQ_ERR_UNSUPPORTED,
                "the call covers too many state rows");
    SSQ_REQUIRE(slots || nseq <= st->desc.batch, SSQ_ERR_INVALID_ARG, "without slots nseq must not exceed the batch");
    SSQ_REQUIRE(tokens == 0 || (io->q && io->k && io->v && io->o), SSQ_ERR_INVALID_ARG,
                "an input or output pointer is NULL");
    SSQ_REQUIRE(aligned(io->q, 16) && aligned(io->k, 16) && aligned(io->v, 16) && aligned(io->o, 16),
                SSQ_ERR_INVALID_ARG, "q, k, v and o must be 16-byte aligned");
    SSQ_REQUIRE(aligned(io->g, 4) && aligned(slots, 4), SSQ_ERR_INVALID_ARG, "g and slots must be 4-byte aligned");
    const int64_t unit = io->dtype == SSQ_DTYPE_FP32 ? 4 : 8; // elements in 16 bytes
    SSQ_REQUIRE(io->q_stride % unit == 0 && io->k_stride % unit == 0 && io->v_stride % unit == 0 && io->o_stride % unit == 0,
                SSQ_ERR_INVALID_ARG, "the strides of q, k, v and o must be multiples of 16 bytes");
    const int64_t row = (int64_t)st->desc.nheads * st->desc.rows_per_head, kv_row = (int64_t)st->desc.ngroups * 128;
    SSQ_REQUIRE(io->q_stride >= kv_row && io->k_stride >= kv_row && io->v_stride >= row && io->o_stride >= row && io->g_stride >= 0,
                SSQ_ERR_INVALID_ARG, "a stride is shorter than a token's row");
    // a chunk's offsets stay below 2^31 bytes
    const int64_t most = (int64_t)1 << 23;
    SSQ_REQUIRE(io->q_stride <= most && io->k_stride <= most && io->v_stride <= most && io->g_stride <= most && io->o_stride <= most,
                SSQ_ERR_UNSUPPORTED, "strides must not exceed 2^23 elements");
    ssq_status s = check_device(st);
    if (s != SSQ_OK) return s;
    *a = ssq::LinArgs{};
    if (fmt_quant(st->desc.format)) a->codes = codes_ptr(st);
    else a->h32 = (float*)codes_ptr(st);
    a->scale = scale_ptr(st);
    a->zero = zero_ptr(st);
    a->q = io->q;
    a->k = io->k;
    a->v = io->v;
    a->g = io->g;
    a->o = io->o;
    a->qs = io->q_stride;
    a->ks = io->k_stride;
    a->vs = io->v_stride;
    a->gs = io->g_stride;
    a->os = io->o_stride;
    a->slots = slots;
    a->tokens = tokens;
    a->nseq = nseq;
    a->batch = st->desc.batch;
    a->H = st->desc.nheads;
    a->G = st->desc.ngroups;
    a->P = st->desc.rows_per_head;
    a->oscale = io->scale;
    a->sr = sr_args(st);
    return SSQ_OK;
}

size_t ssq_linattn_workspace(const ssq_state* st, int32_t nseq, int64_t tokens)
{
    if (!st || st->desc.kind != SSQ_MAMBA2 || nseq < 0 || tokens < 0 || tokens > kMostTokens ||
        nseq > ssq::kMaxPrefillRows / ((int64_t)st->desc.nheads * st->desc.rows_per_head))
        return (size_t)-1;
    return ssq::linattn_workspace(st->desc.format, nseq, tokens, st->desc.nheads, st->desc.rows_per_head,
                                  num_cus(st->device));
}

ssq_status ssq_linattn_prefill(ssq_state* st, const ssq_linattn_io* io, int32_t nseq, int64_t tokens,
                               const int32_t* cu_seqlens, const int32_t* slots, const uint8_t* fresh, void* workspace,
                               size_t workspace_bytes, void* stream)
{
    ssq::LinArgs a;
    ssq_status s = fill_linattn(st, io, nseq, tokens, slots, ssq::kMaxPrefillRows, &a);
    if (s != SSQ_OK) return s;
    SSQ_REQUIRE(nseq == 0 || cu_seqlens, SSQ_ERR_INVALID_ARG, "cu_seqlens is NULL");
    SSQ_REQUIRE(aligned(cu_seqlens, 4), SSQ_ERR_INVALID_ARG, "cu_seqlens must be 4-byte aligned");
    SSQ_REQUIRE(tokens <= kMostTokens, SSQ_ERR_UNSUPPORTED, "a call takes fewer than 2^31-128 tokens");
    const size_t need = ssq_linattn_workspace(st, nseq, tokens);
    SSQ_REQUIRE(need == 0 || (workspace && workspace_bytes >= need), SSQ_ERR_INVALID_ARG, "the workspace is too small");
    SSQ_REQUIRE(aligned(workspace, 256), SSQ_ERR_INVALID_ARG, "the workspace must be 256-byte aligned");
    if (nseq == 0) return ok();
    a.cu = cu_seqlens;
    a.fresh = fresh;
    s = from_hip(ssq::launch_linattn_prefill(st->desc.format, io->dtype, a, workspace, num_cus(st->device),
                                             (hipStream_t)stream),
                 "linear attention prefill launch");
    return s == SSQ_OK ? advance(st, 1, (hipStream_t)stream) : s;
}

ssq_status ssq_linattn_step(ssq_state* st, const ssq_linattn_io* io, int32_t nseq, const int32_t* slots,
                            int32_t readout, void* stream)
{
    ssq::LinArgs a;
    ssq_status s = fill_linattn(st, io, nseq, nseq, slots, ssq::kMaxStepRows, &a);
    if (s != SSQ_OK) return s;
    SSQ_REQUIRE(readout == SSQ_READ_POST_QUANT || readout == SSQ_READ_PRE_QUANT, SSQ_ERR_INVALID_ARG,
                "unknown readout");
    if (nseq == 0) return ok();
    s = from_hip(ssq::launch_linattn_step(st->desc.format, io->dtype, a, readout == SSQ_READ_PRE_QUANT,
                                          (hipStream_t)stream),
                 "linear attention step launch");
    return s == SSQ_OK ? advance(st, 1, (hipStream_t)stream) : s;
}

// ---------------------------------------------------------------------------
// beam search
// ---------------------------------------------------------------------------
static ssq_status check_beam(const ssq_beam_desc* d)
{
    SSQ_REQUIRE(d, SSQ_ERR_INVALID_ARG, "desc is NULL");
    SSQ_REQUIRE(dtype_valid(d->dtype), SSQ_ERR_INVALID_ARG, "unknown dtype");
    SSQ_REQUIRE(d->batch >= 0 && d->vocab > 0, SSQ_ERR_INVALID_ARG, "batch must not be negative, vocab positive");
    SSQ_REQUIRE(d->beams > 0 && d->beams <= SSQ_MAX_BEAMS, SSQ_ERR_INVALID_ARG, "beams must be 1 .. SSQ_MAX_BEAMS");
    SSQ_REQUIRE(d->nselect > 0 && d->nselect <= 2 * d->beams, SSQ_ERR_INVALID_ARG, "nselect must be 1 .. 2*beams");
    SSQ_REQUIRE(d->pad_token >= 0 && d->pad_token < d->vocab, SSQ_ERR_INVALID_ARG, "pad_token must be 0 .. vocab-1");
    SSQ_REQUIRE(d->row_stride >= d->vocab, SSQ_ERR_INVALID_ARG, "row_stride must be at least vocab");
    const int64_t rows = (int64_t)d->batch * d->beams;
    SSQ_REQUIRE(rows <= ssq::kMaxBlocks, SSQ_ERR_UNSUPPORTED, "batch * beams must be below 2^24");
    SSQ_REQUIRE(d->row_stride <= ((int64_t)1 << 59) / (rows > 0 ? rows : 1), SSQ_ERR_INVALID_ARG,
                "row_stride is too large");
    return SSQ_OK;
}

size_t ssq_beam_workspace(const ssq_beam_desc* d)
{
    if (check_beam(d) != SSQ_OK) return 0;
    return ssq::beam_workspace(d->batch, d->beams, d->vocab, d->nselect);
}

ssq_status ssq_beam_select(const ssq_beam_desc* d, const void* logits, const float* scores, const uint8_t* finished,
                           float* out_scores, int32_t* out_tokens, int32_t* out_parents, void* workspace,
                           size_t workspace_bytes, void* stream)
{
    ssq_status s = check_beam(d);
    if (s != SSQ_OK) return s;
    if (d->batch == 0) return ok();
    SSQ_REQUIRE(logits && scores && out_scores && out_tokens && out_parents, SSQ_ERR_INVALID_ARG,
                "an input or output pointer is NULL");
    SSQ_REQUIRE(aligned(logits, d->dtype == SSQ_DTYPE_FP32 ? 4 : 2), SSQ_ERR_INVALID_ARG,
                "the logits must be aligned to their element");
    SSQ_REQUIRE(aligned(scores, 4) && aligned(out_scores, 4) && aligned(out_tokens, 4) && aligned(out_parents, 4),
                SSQ_ERR_INVALID_ARG, "scores and outputs must be 4-byte aligned");
    SSQ_REQUIRE(workspace && aligned(workspace, 256) && workspace_bytes >= ssq_beam_workspace(d), SSQ_ERR_INVALID_ARG,
                "the workspace is too small or not 256-byte aligned");
    ssq::BeamArgs a{};
    a.logits = logits;
    a.scores = scores;
    a.finished = finished;
    a.out_scores = out_scores;
    a.out_tokens = out_tokens;
    a.out_parents = out_parents;
    a.ws = workspace;
    a.row_stride = d->row_stride;
    a.batch = d->batch;
    a.beams = d->beams;
    a.vocab = d->vocab;
    a.nselect = d->nselect;
    a.pad = d->pad_token;
    return from_hip(ssq::launch_beam_select(d->dtype, a, (hipStream_t)stream), "beam selection launch");
}

// the arrays of a state and each sequence's bytes in them; 4 at most
static int state_parts(const ssq_state* st, ssq::ReorderPart* parts)
{
    const int64_t rows = (int64_t)(st->lay.rows / (size_t)st->desc.batch);
    const int64_t low = st->desc.format == SSQ_DAMP ? rows / 128 * (128 - SSQ_DAMP_NHI) : rows;
    int n = 0;
    parts[n++] = {codes_ptr(st), low * (int64_t)st->lay.row_bytes};
    if (scale_ptr(st)) parts[n++] = {(uint8_t*)scale_ptr(st), low * 4};
    if (zero_ptr(st)) parts[n++] = {(uint8_t*)zero_ptr(st), low * 4};
    if (hi_ptr(st)) parts[n++] = {(uint8_t*)hi_ptr(st), (rows - low) * 256};
    return n;
}

static bool share_memory(const ssq_state* a, const ssq_state* b)
{
    const uintptr_t p = (uintptr_t)a->storage, q = (uintptr_t)b->storage;
    return p < q + b->lay.total_bytes && q < p + a->lay.total_bytes;
}

ssq_status ssq_state_reorder(ssq_state* const* states, int32_t nstates, const int32_t* parents, int32_t beams,
                             void* stream)
{
    constexpr int kMost = 1024; // states of one call
    SSQ_REQUIRE(nstates >= 0 && nstates <= kMost, SSQ_ERR_INVALID_ARG, "nstates must be 0 .. 1024");
    if (nstates == 0) return ok();
    SSQ_REQUIRE(states && parents, SSQ_ERR_INVALID_ARG, "states or parents is NULL");
    SSQ_REQUIRE(aligned(parents, 4), SSQ_ERR_INVALID_ARG, "parents must be 4-byte aligned");
    SSQ_REQUIRE(beams > 0 && beams <= SSQ_MAX_BEAMS, SSQ_ERR_INVALID_ARG, "beams must be 1 .. SSQ_MAX_BEAMS");
    ssq::ReorderPart parts[4 * kMost];
    int n = 0;
    for (int i = 0; i < nstates; ++i) {
        const ssq_state* st = states[i];
        SSQ_REQUIRE(st, SSQ_ERR_INVALID_ARG, "a state is NULL");
        SSQ_REQUIRE(st->desc.batch == states[0]->desc.batch, SSQ_ERR_INVALID_ARG, "the states differ in their batch");
        SSQ_REQUIRE(st->desc.batch % beams == 0, SSQ_ERR_INVALID_ARG, "beams must divide the batch");
        const ssq_status s = check_device(st);
        if (s != SSQ_OK) return s;
        // two handles over the same bytes would move them twice at once
        for (int j = 0; j < i; ++j)
            SSQ_REQUIRE(!share_memory(st, states[j]), SSQ_ERR_INVALID_ARG, "two of the states share memory");
        // rows are ordered by sequence, and a sequence's rows are a multiple of 16 (a gated state's channels of 8): its
        // bytes in every array are a multiple of 16
        const int64_t rows = (int64_t)(st->lay.rows / (size_t)st->desc.batch);
        n += state_parts(st, parts + n);
        SSQ_REQUIRE(ssq::reorder_blocks(rows * (int64_t)st->lay.row_bytes, st->desc.batch / beams) <= ssq::kMaxBlocks,
                    SSQ_ERR_UNSUPPORTED, "a state has too many bytes for each beam");
    }
    if (beams == 1) return ok();
    return from_hip(ssq::launch_reorder(parts, n, parents, beams, states[0]->desc.batch / beams, (hipStream_t)stream),
                    "state reorder launch");
}

// ---------------------------------------------------------------------------
// moves between sequences
// ---------------------------------------------------------------------------
ssq_status ssq_state_move(ssq_state* const* states, ssq_state* const* sources, int32_t nstates, const int32_t* to,
                          const int32_t* from, int32_t nmoves, void* stream)
{
    constexpr int kMost = 1024; // states of one call
    SSQ_REQUIRE(nstates >= 0 && nstates <= kMost, SSQ_ERR_INVALID_ARG, "nstates must be 0 .. 1024");
    SSQ_REQUIRE(nmoves >= 0 && nmoves <= ssq::kMaxMoves, SSQ_ERR_INVALID_ARG, "nmoves must be 0 .. 65535");
    if (nstates == 0 || nmoves == 0) return ok();
    SSQ_REQUIRE(states && to && from, SSQ_ERR_INVALID_ARG, "states, to or from is NULL");
    SSQ_REQUIRE(aligned(to, 4) && aligned(from, 4), SSQ_ERR_INVALID_ARG, "to and from must be 4-byte aligned");
    for (int i = 0; i < nstates; ++i) {
        const ssq_state* st = states[i];
        const ssq_state* src = sources ? sources[i] : st;
        SSQ_REQUIRE(st && src, SSQ_ERR_INVALID_ARG, "a state is NULL");
        SSQ_REQUIRE(st->desc.batch == states[0]->desc.batch, SSQ_ERR_INVALID_ARG, "the states differ in their batch");
        ssq_status s = check_device(st);
        if (s != SSQ_OK) return s;
        if (sources) {
            SSQ_REQUIRE(src->desc.batch == sources[0]->desc.batch, SSQ_ERR_INVALID_ARG, "the sources differ in their batch");
            SSQ_REQUIRE(src->desc.kind == st->desc.kind, SSQ_ERR_KIND_MISMATCH, "a source is of another kind");
            SSQ_REQUIRE(src->desc.format == st->desc.format && src->desc.nheads == st->desc.nheads &&
                            src->desc.rows_per_head == st->desc.rows_per_head && src->desc.row_len == st->desc.row_len,
                        SSQ_ERR_INVALID_ARG, "a source is of another format or size");
            s = check_device(src);
            if (s != SSQ_OK) return s;
        }
        for (int j = 0; j < nstates; ++j) {
            SSQ_REQUIRE(j >= i || !share_memory(st, states[j]), SSQ_ERR_INVALID_ARG, "two of the states share memory");
            SSQ_REQUIRE(!sources || !sources[j] || !share_memory(st, sources[j]), SSQ_ERR_INVALID_ARG,
                        "a state and a source share memory");
        }
        ssq::ReorderPart d[4];
        const int m = state_parts(st, d);
        for (int j = 0; j < m; ++j)
            SSQ_REQUIRE(d[j].bytes <= ssq::kMaxBlocks * ssq::kColumnBytes, SSQ_ERR_UNSUPPORTED,
                        "a state has too many bytes for each sequence");
    }
    // all of them checked; a launch's arrays at a time, as the callers' stacks may be small
    ssq::MovePart parts[ssq::kMoveParts];
    int n = 0;
    for (int i = 0; i < nstates; ++i) {
        ssq::ReorderPart d[4], f[4];
        const int m = state_parts(states[i], d);
        (void)state_parts((sources ? sources : states)[i], f);
        for (int j = 0; j < m; ++j) {
            parts[n++] = {d[j].p, f[j].p, d[j].bytes};
            if (n < ssq::kMoveParts && !(i == nstates - 1 && j == m - 1)) continue;
            const hipError_t e = ssq::launch_move(parts, n, to, from, nmoves, states[0]->desc.batch,
                                                  (sources ? sources : states)[0]->desc.batch, !sources, (hipStream_t)stream);
            if (e != hipSuccess) return from_hip(e, "state move launch");
            n = 0;
        }
    }
    return ok();
}

// ---------------------------------------------------------------------------
// gated linear recurrence
// ---------------------------------------------------------------------------
// one tensor of [tokens][channels]
static ssq_status check_rows(const void* p, int64_t stride, int dtype, int64_t channels, int64_t tokens, const char* name)
{
    const int64_t unit = dtype == SSQ_DTYPE_FP32 ? 4 : 8; // elements in 16 bytes
    SSQ_REQUIRE(p || tokens == 0, SSQ_ERR_INVALID_ARG, std::string(name) + " is NULL");
    SSQ_REQUIRE(aligned(p, 16) && stride % unit == 0, SSQ_ERR_INVALID_ARG,
                std::string(name) + " must be 16-byte aligned, its stride a multiple of 16 bytes");
    SSQ_REQUIRE(stride >= channels, SSQ_ERR_INVALID_ARG, std::string(name) + ": a stride is shorter than a token's row");
    SSQ_REQUIRE(stride <= ((int64_t)1 << 23), SSQ_ERR_UNSUPPORTED, "strides must not exceed 2^23 elements");
    return SSQ_OK;
}

#define SSQ_TRY(call)                      \
    do {                                   \
        const ssq_status s_ = (call);      \
        if (s_ != SSQ_OK) return s_;       \
    } while (0)

static ssq_status check_gated(const ssq_state* st, int dtype, int gate, int input, int channels, int32_t nseq,
                              int64_t tokens, const int32_t* slots, int64_t most)
{
    SSQ_REQUIRE(!st || st->desc.kind == SSQ_GATED, SSQ_ERR_KIND_MISMATCH, "the gated recurrence runs on an SSQ_GATED state");
    SSQ_REQUIRE(dtype_valid(dtype), SSQ_ERR_INVALID_ARG, "unknown dtype");
    SSQ_REQUIRE(gate == SSQ_GATE_LOG || gate == SSQ_GATE_SIGMOID, SSQ_ERR_INVALID_ARG, "unknown gate");
    SSQ_REQUIRE(input >= SSQ_INPUT_PLAIN && input <= SSQ_INPUT_NORM, SSQ_ERR_INVALID_ARG, "unknown input factor");
    SSQ_REQUIRE(channels > 0, SSQ_ERR_INVALID_ARG, "channels must be positive");
    SSQ_REQUIRE(channels % 8 == 0 && channels <= ssq::kMaxChannels, SSQ_ERR_UNSUPPORTED,
                "channels must be a multiple of 8, 2^20 at most");
    SSQ_REQUIRE(!st || st->desc.row_len == channels, SSQ_ERR_INVALID_ARG, "the state has another number of channels");
    SSQ_REQUIRE(nseq >= 0 && tokens >= 0, SSQ_ERR_INVALID_ARG, "nseq and tokens must not be negative");
    SSQ_REQUIRE(tokens <= kMostTokens, SSQ_ERR_UNSUPPORTED, "a call takes fewer than 2^31-128 tokens");
    SSQ_REQUIRE(nseq <= most / channels && nseq <= ssq::kMaxGatedSeqs, SSQ_ERR_UNSUPPORTED,
                "the call covers too many sequences and channels");
    SSQ_REQUIRE(st || !slots, SSQ_ERR_INVALID_ARG, "slots without a state");
    SSQ_REQUIRE(!st || slots || nseq <= st->desc.batch, SSQ_ERR_INVALID_ARG, "without slots nseq must not exceed the batch");
    SSQ_REQUIRE(aligned(slots, 4), SSQ_ERR_INVALID_ARG, "slots must be 4-byte aligned");
    return SSQ_OK;
}

static ssq_status check_gated_workspace(int channels, int32_t nseq, int64_t tokens, const void* workspace, size_t bytes)
{
    const size_t need = ssq_gated_workspace(channels, nseq, tokens);
    SSQ_REQUIRE(need == 0 || (workspace && bytes >= need), SSQ_ERR_INVALID_ARG, "the workspace is too small");
    SSQ_REQUIRE(aligned(workspace, 256), SSQ_ERR_INVALID_ARG, "the workspace must be 256-byte aligned");
    return SSQ_OK;
}

static ssq_status fill_gated(const ssq_state* st, const ssq_gated_io* io, int32_t nseq, int64_t tokens, const int32_t* slots,
                             int64_t most, ssq::GatedArgs* a)
{
    SSQ_REQUIRE(io, SSQ_ERR_INVALID_ARG, "io is NULL");
    SSQ_TRY(check_gated(st, io->dtype, io->gate, io->input, io->channels, nseq, tokens, slots, most));
    SSQ_TRY(check_rows(io->x, io->x_stride, io->dtype, io->channels, tokens, "x"));
    SSQ_TRY(check_rows(io->g, io->g_stride, io->dtype, io->channels, tokens, "g"));
    SSQ_TRY(check_rows(io->o, io->o_stride, io->dtype, io->channels, tokens, "o"));
    if (st) SSQ_TRY(check_device(st));
    *a = ssq::GatedArgs{};
    a->x = io->x;
    a->g = io->g;
    a->o = io->o;
    a->xs = io->x_stride;
    a->gs = io->g_stride;
    a->os = io->o_stride;
    a->h = st ? (float*)codes_ptr(st) : nullptr;
    a->slots = slots;
    a->tokens = tokens;
    a->nseq = nseq;
    a->batch = st ? st->desc.batch : 0;
    a->channels = io->channels;
    return SSQ_OK;
}

int64_t ssq_gated_checkpoint_rows(int32_t nseq, int64_t tokens)
{
    if (nseq < 0 || tokens < 0 || tokens > kMostTokens) return -1;
    return tokens / SSQ_GATED_CHUNK + nseq;
}

size_t ssq_gated_workspace(int32_t channels, int32_t nseq, int64_t tokens)
{
    if (check_gated(nullptr, SSQ_DTYPE_FP32, SSQ_GATE_LOG, SSQ_INPUT_PLAIN, channels, nseq, tokens, nullptr,
                    ssq::kMaxGatedRows) != SSQ_OK)
        return (size_t)-1;
    return ssq::gated_workspace(channels, nseq, tokens);
}

ssq_status ssq_gated_scan(ssq_state* st, const ssq_gated_io* io, int32_t nseq, int64_t tokens, const int32_t* cu_seqlens,
                          const int32_t* slots, const uint8_t* fresh, float* checkpoints, void* workspace,
                          size_t workspace_bytes, void* stream)
{
    ssq::GatedArgs a;
    SSQ_TRY(fill_gated(st, io, nseq, tokens, slots, ssq::kMaxGatedRows, &a));
    SSQ_REQUIRE(st || !fresh, SSQ_ERR_INVALID_ARG, "fresh without a state");
    SSQ_REQUIRE(nseq == 0 || cu_seqlens, SSQ_ERR_INVALID_ARG, "cu_seqlens is NULL");
    SSQ_REQUIRE(aligned(cu_seqlens, 4), SSQ_ERR_INVALID_ARG, "cu_seqlens must be 4-byte aligned");
    SSQ_REQUIRE(aligned(checkpoints, 16), SSQ_ERR_INVALID_ARG, "checkpoints must be 16-byte aligned");
    SSQ_TRY(check_gated_workspace(io->channels, nseq, tokens, workspace, workspace_bytes));
    if (nseq == 0) return ok();
    a.cu = cu_seqlens;
    a.fresh = fresh;
    a.ckpt = checkpoints;
    return from_hip(ssq::launch_gated_scan(io->dtype, io->gate, io->input, a, workspace, (hipStream_t)stream),
                    "gated scan launch");
}

ssq_status ssq_gated_scan_backward(const ssq_state* st, const ssq_gated_grad* io, int32_t nseq, int64_t tokens,
                                   const int32_t* cu_seqlens, const int32_t* slots, const float* checkpoints,
                                   void* workspace, size_t workspace_bytes, void* stream)
{
    SSQ_REQUIRE(io, SSQ_ERR_INVALID_ARG, "io is NULL");
    SSQ_TRY(check_gated(st, io->dtype, io->gate, io->input, io->channels, nseq, tokens, slots, ssq::kMaxGatedRows));
    SSQ_TRY(check_rows(io->x, io->x_stride, io->dtype, io->channels, tokens, "x"));
    SSQ_TRY(check_rows(io->g, io->g_stride, io->dtype, io->channels, tokens, "g"));
    SSQ_TRY(check_rows(io->dout, io->dout_stride, io->dtype, io->channels, tokens, "dout"));
    SSQ_TRY(check_rows(io->dx, io->dx_stride, io->dtype, io->channels, tokens, "dx"));
    SSQ_TRY(check_rows(io->dg, io->dg_stride, io->dtype, io->channels, tokens, "dg"));
    SSQ_REQUIRE(nseq == 0 || cu_seqlens, SSQ_ERR_INVALID_ARG, "cu_seqlens is NULL");
    SSQ_REQUIRE(aligned(cu_seqlens, 4), SSQ_ERR_INVALID_ARG, "cu_seqlens must be 4-byte aligned");
    SSQ_REQUIRE(checkpoints || tokens == 0 || nseq == 0, SSQ_ERR_INVALID_ARG, "checkpoints is NULL");
    SSQ_REQUIRE(aligned(checkpoints, 16) && aligned(io->dlast, 16) && aligned(io->dfirst, 16), SSQ_ERR_INVALID_ARG,
                "checkpoints, dlast and dfirst must be 16-byte aligned");
    SSQ_TRY(check_gated_workspace(io->channels, nseq, tokens, workspace, workspace_bytes));
    if (nseq == 0) return ok();
    ssq::GatedArgs a{};
    a.x = io->x;
    a.g = io->g;
    a.dout = io->dout;
    a.dx = io->dx;
    a.dg = io->dg;
    a.dlast = io->dlast;
    a.dfirst = io->dfirst;
    a.xs = io->x_stride;
    a.gs = io->g_stride;
    a.dos = io->dout_stride;
    a.dxs = io->dx_stride;
    a.dgs = io->dg_stride;
    a.ckpt = const_cast<float*>(checkpoints);
    a.cu = cu_seqlens;
    a.slots = slots;
    a.tokens = tokens;
    a.nseq = nseq;
    a.batch = st ? st->desc.batch : 0;
    a.channels = io->channels;
    return from_hip(ssq::launch_gated_backward(io->dtype, io->gate, io->input, a, workspace, (hipStream_t)stream),
                    "gated scan gradient launch");
}

ssq_status ssq_gated_step(ssq_state* st, const ssq_gated_io* io, int32_t nseq, const int32_t* slots, void* stream)
{
    ssq::GatedArgs a;
    SSQ_REQUIRE(st, SSQ_ERR_INVALID_ARG, "state is NULL");
    SSQ_TRY(fill_gated(st, io, nseq, nseq, slots, ssq::kMaxGatedStep, &a));
    if (nseq == 0) return ok();
    return from_hip(ssq::launch_gated_step(io->dtype, io->gate, io->input, a, (hipStream_t)stream), "gated step launch");
}

// ---------------------------------------------------------------------------
// group norm
// ---------------------------------------------------------------------------
static ssq_status check_norm_size(int64_t groups, int64_t width, int64_t tokens)
{
    SSQ_REQUIRE(groups > 0 && width > 0 && tokens >= 0, SSQ_ERR_INVALID_ARG,
                "groups and width must be positive, tokens not negative");
    SSQ_REQUIRE(width % 8 == 0 && width <= ssq::kMaxNormWidth, SSQ_ERR_UNSUPPORTED, "width must be a multiple of 8, 16384 at most");
    SSQ_REQUIRE(groups * width <= ssq::kMaxChannels, SSQ_ERR_UNSUPPORTED, "a token has 2^20 channels at most");
    SSQ_REQUIRE(tokens <= ((int64_t)1 << 31) / groups, SSQ_ERR_UNSUPPORTED, "tokens * groups must not exceed 2^31");
    return SSQ_OK;
}

static ssq_status fill_norm(const ssq_norm_io* io, int64_t tokens, ssq::NormArgs* a)
{
    SSQ_REQUIRE(io, SSQ_ERR_INVALID_ARG, "io is NULL");
    SSQ_REQUIRE(dtype_valid(io->dtype), SSQ_ERR_INVALID_ARG, "unknown dtype");
    SSQ_REQUIRE(io->act >= SSQ_ACT_SILU && io->act <= SSQ_ACT_GATE_INPUT, SSQ_ERR_INVALID_ARG, "unknown activation");
    SSQ_TRY(check_norm_size(io->groups, io->width, tokens));
    SSQ_REQUIRE(io->eps >= 1.17549435e-38f && io->eps < 1e30f, SSQ_ERR_INVALID_ARG, "eps must be a positive number");
    const int64_t row = (int64_t)io->groups * io->width;
    SSQ_TRY(check_rows(io->x, io->x_stride, io->dtype, row, tokens, "x"));
    if (io->act == SSQ_ACT_SILU) SSQ_REQUIRE(!io->z, SSQ_ERR_INVALID_ARG, "SSQ_ACT_SILU has no z");
    else SSQ_TRY(check_rows(io->z, io->z_stride, io->dtype, row, tokens, "z"));
    SSQ_REQUIRE(aligned(io->weight, 16) && aligned(io->bias, 16), SSQ_ERR_INVALID_ARG, "weight and bias must be 16-byte aligned");
    *a = ssq::NormArgs{};
    a->x = io->x;
    a->z = io->z;
    a->weight = io->weight;
    a->bias = io->bias;
    a->xs = io->x_stride;
    a->zs = io->z_stride;
    a->tokens = tokens;
    a->groups = io->groups;
    a->width = io->width;
    a->eps = io->eps;
    a->center = io->center != 0;
    return SSQ_OK;
}

ssq_status ssq_group_norm(const ssq_norm_io* io, void* y, int64_t y_stride, int64_t tokens, void* stream)
{
    ssq::NormArgs a;
    SSQ_TRY(fill_norm(io, tokens, &a));
    SSQ_TRY(check_rows(y, y_stride, io->dtype, (int64_t)io->groups * io->width, tokens, "y"));
    if (tokens == 0) return ok();
    a.y = y;
    a.ys = y_stride;
    return from_hip(ssq::launch_group_norm(io->dtype, io->act, a, (hipStream_t)stream), "group norm launch");
}

size_t ssq_group_norm_workspace(int32_t groups, int32_t width, int64_t tokens)
{
    if (check_norm_size(groups, width, tokens) != SSQ_OK) return (size_t)-1;
    return ssq::norm_workspace(groups, width, tokens);
}

ssq_status ssq_group_norm_backward(const ssq_norm_io* io, const ssq_norm_grad* grad, int64_t tokens, void* workspace,
                                   size_t workspace_bytes, void* stream)
{
    ssq::NormArgs a;
    SSQ_TRY(fill_norm(io, tokens, &a));
    SSQ_REQUIRE(grad, SSQ_ERR_INVALID_ARG, "grad is NULL");
    const int64_t row = (int64_t)io->groups * io->width;
    SSQ_TRY(check_rows(grad->dy, grad->dy_stride, io->dtype, row, tokens, "dy"));
    SSQ_TRY(check_rows(grad->dx, grad->dx_stride, io->dtype, row, tokens, "dx"));
    if (io->act == SSQ_ACT_SILU) SSQ_REQUIRE(!grad->dz, SSQ_ERR_INVALID_ARG, "SSQ_ACT_SILU has no dz");
    else SSQ_TRY(check_rows(grad->dz, grad->dz_stride, io->dtype, row, tokens, "dz"));
    SSQ_REQUIRE(aligned(grad->dweight, 16) && aligned(grad->dbias, 16), SSQ_ERR_INVALID_ARG,
                "dweight and dbias must be 16-byte aligned");
    const size_t need = ssq_group_norm_workspace(io->groups, io->width, tokens);
    SSQ_REQUIRE(need == 0 || (workspace && workspace_bytes >= need), SSQ_ERR_INVALID_ARG, "the workspace is too small");
    SSQ_REQUIRE(aligned(workspace, 256), SSQ_ERR_INVALID_ARG, "the workspace must be 256-byte aligned");
    a.dy = grad->dy;
    a.dx = grad->dx;
    a.dz = grad->dz;
    a.dweight = grad->dweight;
    a.dbias = grad->dbias;
    a.dys = grad->dy_stride;
    a.dxs = grad->dx_stride;
    a.dzs = grad->dz_stride;
    a.ws = (float*)workspace;
    return from_hip(ssq::launch_group_norm_backward(io->dtype, io->act, a, (hipStream_t)stream), "group norm gradient launch");
}

const char* ssq_status_string(int32_t status)
{
    switch (status) {
    case SSQ_OK: return "SSQ_OK";
    case SSQ_ERR_INVALID_ARG: return "SSQ_ERR_INVALID_ARG: invalid argument";
    case SSQ_ERR_UNSUPPORTED: return "SSQ_ERR_UNSUPPORTED: size or format not supported by the kernels";
    case SSQ_ERR_KIND_MISMATCH: return "SSQ_ERR_KIND_MISMATCH: call does not match the state kind";
    case SSQ_ERR_ALLOC: return "SSQ_ERR_ALLOC: device allocation failed";
    case SSQ_ERR_DEVICE: return "SSQ_ERR_DEVICE: HIP runtime error";
    }
    return "unknown ssq_status";
}

const char* ssq_last_error(void) { return g_last_error.c_str(); }

} // extern "C"
