// ssq_linattn_prefill.hip -- linear attention with a decay for each head over ragged prompts.
//
// A wave takes four rows of one (sequence, head) from the first token to the last: 16 lanes a
// row, 8 entries a lane, the recurrence in fp32.
#include "ssq_ops_device.h"

namespace ssq {

// sequence i of the call: its slot, or -1 if it is skipped, and its tokens
struct SeqSpan {
    int slot;
    int64_t begin, end;
};

__device__ __forceinline__ SeqSpan seq_span(const LinArgs& a, int i)
{
    SeqSpan s;
    s.slot = a.slots ? a.slots[i] : i;
    if (s.slot < 0 || s.slot >= a.batch) s.slot = -1;
    const int64_t b = a.cu[i], e = a.cu[i + 1];
    s.begin = b < 0 ? 0 : (b > a.tokens ? a.tokens : b);
    s.end = e < s.begin ? s.begin : (e > a.tokens ? a.tokens : e);
    return s;
}

// quantized states: the rows a call reads, reconstructed into `h32` [nseq][H*P][128], and the
// rows it leaves, refit and rounded from there
template <int F, bool SR>
__global__ __launch_bounds__(256) void k_linattn_rows(LinArgs a, int64_t units, bool store)
{
    constexpr int LPR = Traits<F>::bits == 8 ? 8 : 4, E = 128 / LPR, RPW = 64 / LPR;
    constexpr int NW = E * Traits<F>::bits / 32;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t unit = (int64_t)blockIdx.x * 4 + wave;
    if (unit >= units) return;
    const int64_t per_seq = (int64_t)a.H * a.P / RPW;
    const int seq = (int)(unit / per_seq);
    const SeqSpan s = seq_span(a, seq);
    const bool fresh = a.fresh && a.fresh[seq];
    // an empty sequence that goes on keeps its codes; a fresh one starts from zero
    if (s.slot < 0 || (!fresh && s.begin == s.end) || (fresh && !store)) return;
    const int lane = threadIdx.x & 63, sub = lane % LPR;
    const int64_t r = (unit % per_seq) * RPW + lane / LPR;
    const int64_t row = (int64_t)s.slot * a.H * a.P + r;
    float* p = a.h32 + ((int64_t)seq * a.H * a.P + r) * 128 + E * sub;
    float h[E];
    uint32_t w[NW];
    uint8_t* c = a.codes + row * (128 * Traits<F>::bits / 8) + sub * (4 * NW);
    if (!store) {
        load_words<NW>(c, w);
        unpack_codes<F, E>(w, h);
        const float sc = a.scale[row], z = Traits<F>::asym ? a.zero[row] : 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) h[e] = sc * (Traits<F>::asym ? h[e] - z : h[e]);
        store_f32<E>(p, h);
        return;
    }
    load_f32<E>(p, h);
    RowGrid g;
    const uint64_t ctr0 = SR ? (sr_token(a.sr) * (uint64_t)a.sr.rows + (uint64_t)row) * 128 + (uint64_t)(E * sub) : 0;
    refit_row<F, E, LPR, SR>(h, g, a.sr.seed, ctr0);
    pack_codes<F, E>(h, w);
    store_words<NW>(c, w);
    if (sub == 0) {
        a.scale[row] = g.s;
        if constexpr (Traits<F>::asym) a.zero[row] = g.z;
    }
}

// where the fp32 rows of sequence i are: the state itself, or the copy of a quantized one
__device__ __forceinline__ float* seq_rows(const LinArgs& a, int seq, int slot)
{
    return a.h32 + (int64_t)(a.codes ? seq : slot) * a.H * a.P * 128;
}

template <int DT>
__global__ __launch_bounds__(256) void k_linattn_scan(LinArgs a, int64_t units)
{
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t unit = (int64_t)blockIdx.x * 4 + wave;
    if (unit >= units) return;
    const int parts = a.P / 4;
    const int part = (int)(unit % parts), head = (int)(unit / parts % a.H), seq = (int)(unit / parts / a.H);
    const SeqSpan s = seq_span(a, seq);
    const bool fresh = a.fresh && a.fresh[seq];
    if (s.slot < 0 || (!fresh && s.begin == s.end)) return;
    const int lane = threadIdx.x & 63, sub = lane & 15, r = part * 4 + lane / 16;
    const int kvh = head / (a.H / a.G);
    float* p = seq_rows(a, seq, s.slot) + ((int64_t)head * a.P + r) * 128 + 8 * sub;
    float h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = 0.0f;
    if (!fresh) load_f32<8>(p, h);
    for (int64_t t = s.begin; t < s.end; ++t) {
        float k[8], q[8], acc = 0.0f;
        load_elems<DT, 8>(elem_ptr<DT>(a.k, t * a.ks + kvh * 128 + 8 * sub), k);
        load_elems<DT, 8>(elem_ptr<DT>(a.q, t * a.qs + kvh * 128 + 8 * sub), q);
        const float v = load_elem<DT>(a.v, t * a.vs + (int64_t)head * a.P + r);
        const float lam = a.g ? (float)exp((double)a.g[t * a.gs + head]) : 1.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            h[e] = __builtin_fmaf(lam, h[e], v * k[e]);
            acc = __builtin_fmaf(q[e], h[e], acc);
        }
        acc = group_sum<16>(acc);
        if (sub == 0) store_elem<DT>(a.o, t * a.os + (int64_t)head * a.P + r, a.oscale * acc);
    }
    store_f32<8>(p, h);
}

size_t linattn_workspace(int fmt, int nseq, int64_t tokens, int H, int P, int num_cus)
{
    (void)tokens;
    (void)num_cus;
    return fmt == FP32 ? 0 : (size_t)nseq * H * P * 512;
}

template <int F>
static hipError_t launch_state_rows(const LinArgs& a, bool store, hipStream_t st)
{
    constexpr int RPW = Traits<F>::bits == 8 ? 8 : 16;
    const int64_t units = (int64_t)a.nseq * a.H * a.P / RPW, blocks = (units + 3) / 4;
    if (blocks > kMaxBlocks) return hipErrorInvalidValue;
    if (a.sr.on) hipLaunchKernelGGL((k_linattn_rows<F, true>), dim3((unsigned)blocks), dim3(256), 0, st, a, units, store);
    else hipLaunchKernelGGL((k_linattn_rows<F, false>), dim3((unsigned)blocks), dim3(256), 0, st, a, units, store);
    return hipGetLastError();
}

static hipError_t state_rows(int fmt, const LinArgs& a, bool store, hipStream_t st)
{
    switch (fmt) {
    case FP32: return hipSuccess;
    case INT8_SYM: return launch_state_rows<INT8_SYM>(a, store, st);
    case INT8_ASYM: return launch_state_rows<INT8_ASYM>(a, store, st);
    case INT4_SYM: return launch_state_rows<INT4_SYM>(a, store, st);
    case INT4_ASYM: return launch_state_rows<INT4_ASYM>(a, store, st);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_linattn_prefill(int fmt, int dtype, const LinArgs& args, void* ws, int num_cus, hipStream_t st)
{
    (void)num_cus;
    LinArgs a = args;
    if (fmt == FP32) a.codes = nullptr;
    else a.h32 = static_cast<float*>(ws);
    hipError_t e = state_rows(fmt, a, false, st);
    if (e != hipSuccess) return e;
    const int64_t units = (int64_t)a.nseq * a.H * a.P / 4, blocks = (units + 3) / 4;
    if (blocks > kMaxBlocks) return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks), wg(256);
    switch (dtype) {
    case DT_FP32: hipLaunchKernelGGL(k_linattn_scan<DT_FP32>, grid, wg, 0, st, a, units); break;
    case DT_BF16: hipLaunchKernelGGL(k_linattn_scan<DT_BF16>, grid, wg, 0, st, a, units); break;
    case DT_FP16: hipLaunchKernelGGL(k_linattn_scan<DT_FP16>, grid, wg, 0, st, a, units); break;
    default: return hipErrorInvalidValue;
    }
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    return state_rows(fmt, a, true, st);
}

} // namespace ssq
