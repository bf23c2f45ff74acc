// ssq_linattn_step.hip -- linear attention with a decay for each head, one token: the
// recurrent form, for any subset of a state's sequences, gfx950.
//
//   h'_pn = fma(exp(g), h_pn, fl(v_p*k_n)),   o_p = scale * sum_n q_n h'_pn
//
// on rows of 128 key entries, fp32 or quantized (then reconstructed, refit and rounded as
// every state step does it).  The state is read and written once: bytes bound it.
//
// A wave takes 16 rows of one head (P is a multiple of 16), so that every wave has whole
// rows of one (sequence, head) and its o is one run of 16 elements.
#include "ssq_ops_device.h"

namespace ssq {

constexpr int kStepRows = 16;

// lanes per row: 16 bytes a lane and load.  A row of fp32 takes 16 lanes, each with the
// entries 4l .. 4l+3 and 64+4l .. 64+4l+3, so that an instruction covers 256 contiguous bytes of
// each row and the non-temporal hint pays on its loads and stores: 240 sequences of 128 heads
// (2.02 GB) take 332 us with it, 6.1 TB/s, and 377 us without.
template <int F>
constexpr int linattn_lpr()
{
    return F == FP32 ? 16 : (Traits<F>::bits == 8 ? 8 : 4);
}

template <int F, int DT, bool PRE, bool SR>
__global__ __launch_bounds__(256) void k_linattn_step(LinArgs a, int64_t units)
{
    constexpr int LPR = linattn_lpr<F>(), E = 128 / LPR, RPW = 64 / LPR, K = kStepRows / RPW;
    constexpr int NW = F == FP32 ? E : E * Traits<F>::bits / 32;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t unit = (int64_t)blockIdx.x * 4 + wave;
    if (unit >= units) return;
    const int parts = a.P / kStepRows;
    const int part = (int)(unit % parts);
    const int64_t ih = unit / parts;
    const int head = (int)(ih % a.H);
    const int seq = (int)(ih / a.H);
    const int slot = a.slots ? a.slots[seq] : seq;
    if (slot < 0 || slot >= a.batch) return;
    const int lane = threadIdx.x & 63, sub = lane % LPR, grp = lane / LPR;
    const int64_t row0 = ((int64_t)slot * a.H + head) * a.P + part * kStepRows;
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
    const int64_t v0 = seq * a.vs + (int64_t)head * a.P + part * kStepRows;
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
#pragma unroll
                for (int e = 0; e < E; ++e)
                    acc = __builtin_fmaf(q[e], fast ? h[e] - g.Mr : (h[e] - kMagic) - g.z, acc);
            }
            acc = group_sum<LPR>(acc);
            if constexpr (!PRE) acc *= g.s;
        }
        if (sub == i) out = acc; // lane (grp, i) keeps the row that it stores
    }
    if (sub < K) store_elem<DT>(a.o, seq * a.os + (int64_t)head * a.P + part * kStepRows + sub * RPW + grp, a.oscale * out);
}

template <int F, int DT>
static hipError_t launch_step_fd(const LinArgs& a, bool pre, hipStream_t st)
{
    const int64_t units = (int64_t)a.nseq * a.H * (a.P / kStepRows);
    const int64_t blocks = (units + 3) / 4;
    if (blocks > kMaxBlocks) return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks), wg(256);
    if constexpr (F == FP32) {
        hipLaunchKernelGGL((k_linattn_step<F, DT, true, false>), grid, wg, 0, st, a, units);
    } else if (a.sr.on) {
        if (pre) hipLaunchKernelGGL((k_linattn_step<F, DT, true, true>), grid, wg, 0, st, a, units);
        else hipLaunchKernelGGL((k_linattn_step<F, DT, false, true>), grid, wg, 0, st, a, units);
    } else {
        if (pre) hipLaunchKernelGGL((k_linattn_step<F, DT, true, false>), grid, wg, 0, st, a, units);
        else hipLaunchKernelGGL((k_linattn_step<F, DT, false, false>), grid, wg, 0, st, a, units);
    }
    return hipGetLastError();
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
