// ssq_linattn_step.hip -- linear attention with a decay for each head, one token: the
// recurrent form, for any subset of a state's sequences, gfx950.
//
//   h'_pn = fma(exp(g), h_pn, fl(v_p*k_n)),   o_p = scale * sum_n q_n h'_pn
//
// on rows of 128 key entries, fp32 or quantized (then reconstructed, refit and rounded as
// every state step does it).  The state is read and written once: bytes bound it.
//
// A wave takes 16, 32 or 64 rows of one head (P is a multiple of 16), so that q, k and the decay
// of its (sequence, head) serve all of them and its o is one run of elements.  All of its rows are
// in flight before the first is worked on.
#include "ssq_ops_device.h"

namespace ssq {

// lanes per row: 16 bytes a lane and load.  A row of fp32 takes 16 lanes, each with the
// entries 4l .. 4l+3 and 64+4l .. 64+4l+3, so that an instruction covers 256 contiguous bytes of
// each row and the non-temporal hint pays on its loads and stores: 240 sequences of 128 heads
// (2.02 GB) take 332 us with it, 6.1 TB/s, and 377 us without.
template <int F>
constexpr int linattn_lpr()
{
    return F == FP32 ? 16 : (Traits<F>::bits == 8 ? 8 : 4);
}

// int4 holds 32 entries of q, k and the row in registers: three waves per SIMD by decree (168
// registers, no spill) against two, 256 sequences of 128 heads asymmetric 91 us against 105.
template <int F, bool SR>
constexpr int linattn_step_waves()
{
    return F != FP32 && Traits<F>::bits == 4 && !SR ? 3 : 1;
}

template <int F, int DT, int ROWS, bool PRE, bool SR>
__global__ __launch_bounds__(256, (linattn_step_waves<F, SR>())) void k_linattn_step(LinArgs a, int64_t units)
{
    constexpr int LPR = linattn_lpr<F>(), E = 128 / LPR, RPW = 64 / LPR, K = ROWS / RPW;
    static_assert(K <= LPR, "a lane of each row stores one output");
    constexpr int NW = F == FP32 ? E : E * Traits<F>::bits / 32;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t unit = (int64_t)blockIdx.x * 4 + wave;
    if (unit >= units) return;
    const int parts = a.P / ROWS;
    const int part = (int)(unit % parts);
    const int64_t ih = unit / parts;
    const int head = (int)(ih % a.H);
    const int seq = (int)(ih / a.H);
    const int slot = a.slots ? a.slots[seq] : seq;
    if (slot < 0 || slot >= a.batch) return;
    const int lane = threadIdx.x & 63, sub = lane % LPR, grp = lane / LPR;
    const int64_t row0 = ((int64_t)slot * a.H + head) * a.P + part * ROWS;
    const int kvh = head / (a.H / a.G);

    uint32_t w[K][NW];
    float rs[K], rz[K];
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int64_t row = row0 + i * RPW + grp;
        if constexpr (F == FP32) {
            const float* p = a.h32 + row * 128 + 4 * sub;
            load_words<4>(p, w[i]);
            load_words<4>(p + 64, w[i] + 4);
        } else {
            load_words<NW>(a.codes + row * (128 * Traits<F>::bits / 8) + sub * (4 * NW), w[i]);
            rs[i] = a.scale[row];
            rz[i] = Traits<F>::asym ? a.zero[row] : 0.0f;
        }
    }
    float k[E], q[E];
    const void* kp = elem_ptr<DT>(a.k, seq * a.ks + kvh * 128);
    const void* qp = elem_ptr<DT>(a.q, seq * a.qs + kvh * 128);
    if constexpr (F == FP32) {
        load_elems<DT, 4>(elem_ptr<DT>(kp, 4 * sub), k);
        load_elems<DT, 4>(elem_ptr<DT>(kp, 64 + 4 * sub), k + 4);
        load_elems<DT, 4>(elem_ptr<DT>(qp, 4 * sub), q);
        load_elems<DT, 4>(elem_ptr<DT>(qp, 64 + 4 * sub), q + 4);
    } else {
        load_elems<DT, E>(elem_ptr<DT>(kp, E * sub), k);
        load_elems<DT, E>(elem_ptr<DT>(qp, E * sub), q);
    }
    const int64_t v0 = seq * a.vs + (int64_t)head * a.P + part * ROWS;
    float v[K];
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = load_elem<DT>(a.v, v0 + i * RPW + grp);
    const float lam = a.g ? (float)exp((double)a.g[seq * a.gs + head]) : 1.0f;
    uint64_t ctr = 0;
    if constexpr (SR) ctr = sr_token(a.sr) * (uint64_t)a.sr.rows;

    float out = 0.0f;
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int64_t row = row0 + i * RPW + grp;
        float h[E];
        float acc = 0.0f;
        if constexpr (F == FP32) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                h[e] = __builtin_fmaf(lam, __uint_as_float(w[i][e]), v[i] * k[e]);
                acc = __builtin_fmaf(q[e], h[e], acc);
                w[i][e] = __float_as_uint(h[e]);
            }
            float* p = a.h32 + row * 128 + 4 * sub;
            store_words<4>(p, w[i]);
            store_words<4>(p + 64, w[i] + 4);
            acc = group_sum<LPR>(acc);
        } else {
            float d[E];
            unpack_codes<F, E>(w[i], d);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float c = Traits<F>::asym ? d[e] - rz[i] : d[e];
                h[e] = __builtin_fmaf(lam, rs[i] * c, v[i] * k[e]);
                if constexpr (PRE) acc = __builtin_fmaf(q[e], h[e], acc);
            }
            RowGrid g;
            const uint64_t ctr0 = SR ? (ctr + (uint64_t)row) * 128 + (uint64_t)(E * sub) : 0;
            const bool fast = refit_row<F, E, LPR, SR>(h, g, a.sr.seed, ctr0);
            uint32_t ow[NW];
            pack_codes<F, E>(h, ow);
            store_words<NW>(a.codes + row * (128 * Traits<F>::bits / 8) + sub * (4 * NW), ow);
            if (sub == 0) {
                a.scale[row] = g.s;
                if constexpr (Traits<F>::asym) a.zero[row] = g.z;
            }
            if constexpr (!PRE) {
                // fl(c' - z') of the new row: exact against Mr on the fast path
                if (fast) {
#pragma unroll
                    for (int e = 0; e < E; ++e) acc = __builtin_fmaf(q[e], h[e] - g.Mr, acc);
                } else {
#pragma unroll
                    for (int e = 0; e < E; ++e) acc = __builtin_fmaf(q[e], (h[e] - kMagic) - g.z, acc);
                }
            }
            acc = group_sum<LPR>(acc);
            if constexpr (!PRE) acc *= g.s;
        }
        if (sub == i) out = acc; // lane (grp, i) keeps the row that it stores
    }
    if (sub < K) store_elem<DT>(a.o, seq * a.os + (int64_t)head * a.P + part * ROWS + sub * RPW + grp, a.oscale * out);
}

template <int F, int DT, int ROWS>
static hipError_t launch_step_rows(const LinArgs& a, bool pre, hipStream_t st)
{
    const int64_t units = (int64_t)a.nseq * a.H * (a.P / ROWS);
    const int64_t blocks = (units + 3) / 4;
    const dim3 grid((unsigned)blocks), wg(256);
    if constexpr (F == FP32) {
        hipLaunchKernelGGL((k_linattn_step<F, DT, ROWS, true, false>), grid, wg, 0, st, a, units);
    } else if (a.sr.on) {
        if (pre) hipLaunchKernelGGL((k_linattn_step<F, DT, ROWS, true, true>), grid, wg, 0, st, a, units);
        else hipLaunchKernelGGL((k_linattn_step<F, DT, ROWS, false, true>), grid, wg, 0, st, a, units);
    } else {
        if (pre) hipLaunchKernelGGL((k_linattn_step<F, DT, ROWS, true, false>), grid, wg, 0, st, a, units);
        else hipLaunchKernelGGL((k_linattn_step<F, DT, ROWS, false, false>), grid, wg, 0, st, a, units);
    }
    return hipGetLastError();
}

// More rows a wave once that leaves 4096 waves, 4 on each SIMD: q, k and the decay, an exponential
// in double, are then made for fewer waves.  256 sequences of 128 heads (2.1 M rows): int4
// asymmetric 146 us at 16 rows, 91 at 64; int8 asymmetric 141 at 16, 111 at 32, 117 at 64.  61
// sequences of 32 heads, int8: 12.2 us at 16 rows, 14.6 at 64.
// Of the same rows with fp32 inputs the Mamba-2 decode step, whose waves run on with loads an iteration
// ahead, takes 75 us in int4 (here 98 symmetric, 128 asymmetric; 87 and 90 with bf16 inputs) and 108 in
// int8 asymmetric (here 111); the floor is 46-49 and 89.  Stochastic rounding: 145-149 us in all formats.
template <int F, int DT>
static hipError_t launch_step_fd(const LinArgs& a, bool pre, hipStream_t st)
{
    constexpr int64_t kWaves = 4096;
    if constexpr (F != FP32) {
        const int64_t rows = (int64_t)a.nseq * a.H * a.P;
        if constexpr (Traits<F>::bits == 4)
            if (a.P % 64 == 0 && rows / 64 >= kWaves) return launch_step_rows<F, DT, 64>(a, pre, st);
        if (a.P % 32 == 0 && rows / 32 >= kWaves) return launch_step_rows<F, DT, 32>(a, pre, st);
    }
    return launch_step_rows<F, DT, 16>(a, pre, st);
}

template <int F>
static hipError_t launch_step_f(int dtype, const LinArgs& a, bool pre, hipStream_t st)
{
    switch (dtype) {
    case DT_FP32: return launch_step_fd<F, DT_FP32>(a, pre, st);
    case DT_BF16: return launch_step_fd<F, DT_BF16>(a, pre, st);
    case DT_FP16: return launch_step_fd<F, DT_FP16>(a, pre, st);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_linattn_step(int fmt, int dtype, const LinArgs& a, bool pre, hipStream_t st)
{
    switch (fmt) {
    case FP32: return launch_step_f<FP32>(dtype, a, pre, st);
    case INT8_SYM: return launch_step_f<INT8_SYM>(dtype, a, pre, st);
    case INT8_ASYM: return launch_step_f<INT8_ASYM>(dtype, a, pre, st);
    case INT4_SYM: return launch_step_f<INT4_SYM>(dtype, a, pre, st);
    case INT4_ASYM: return launch_step_f<INT4_ASYM>(dtype, a, pre, st);
    }
    return hipErrorInvalidValue;
}

} // namespace ssq
