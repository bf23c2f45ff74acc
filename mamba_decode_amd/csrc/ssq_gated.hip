// ssq_gated.hip -- a gated linear recurrence, h_t = a_t h_(t-1) + s_t x_t in every channel, over
// ragged sequences, its gradient and its single-token form, gfx950.
//
// A run of tokens takes a state h to A h + B, A the product of its decays and B what it makes of a state of zero, and runs
// compose: (A2, B2) after (A1, B1) is (A2 A1, A2 B1 + B2).  A lane holds 16 tokens of a few channels in registers and finds
// their (A, B); the lanes of a slice of channels meet in LDS, each learns the state before its tokens and goes over them again,
// from registers.  The tiles of a sequence follow each other in one workgroup, the loads of the next one under way
// meanwhile.  So x and g are read once and o is written once.  The gradient goes through the tiles from the end, dh_t = do_t +
// a_(t+1) dh_(t+1), and computes the states of a lane's tokens again from the one before them, which the scan keeps in fp32.
//
// Bytes bound it where enough workgroups have whole cache lines: 8 packed sequences, 8925 tokens in all, 4096 channels, bf16,
// 56 + 84 us (585 MB in the two, 4.2 TB/s); 8192 tokens of 8192 channels (403 MB, rows of half lines) 98 us; a token
// of 240 sequences of 8192 channels (27 MB) 7 us, 2 us of a launch among them.
#include <type_traits>

#include "ssq_gated_device.h"

namespace ssq {

constexpr int kGroupSlices = 16; // fewer are not dealt to the XCDs in groups

// The tile of a workgroup: a slice of channels, LC lanes of CPL channels (4 bytes of x), and W
// waves x 64/LC groups of lanes along the tokens, each with a chunk of 16 tokens in registers.
template <int DT, int LC_, int W_>
struct Tile {
    static constexpr int LC = LC_, W = W_, K = kGatedChunk;
    static constexpr int SIZE = DT == DT_FP32 ? 4 : 2, CPL = 4 / SIZE, S = LC * CPL;
    static constexpr int TL = 64 / LC, SEGS = W * TL, WAVE_TOKENS = TL * K, TOKENS = SEGS * K;
    static_assert(TL <= 4, "a wave's rows stay below 2^31 bytes at the largest stride");
    int wave, tl, c, ch; // wave, group of lanes, first channel within the slice and of all
    uint32_t bad;        // beyond every descriptor's bytes where the lane's channels are none

    __device__ __forceinline__ Tile(int slice, int channels)
    {
        wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
        const int lane = threadIdx.x & 63;
        tl = lane / LC;
        c = lane % LC * CPL;
        ch = slice * S + c;
        bad = ch < channels ? 0u : kNowhere;
    }
    __device__ __forceinline__ int seg() const { return wave * TL + tl; }
    // The wave's rows from token t0 of a tensor on, `left` of them at most.  A row's offset is the scalar one of its load or store,
    // which the range check of these descriptors counts in.
    __device__ __forceinline__ Rsrc rows(const void* p, int64_t t0, int64_t stride, int64_t left, int channels) const
    {
        const int64_t n = left < WAVE_TOKENS ? left : WAVE_TOKENS;
        const uint32_t bytes = n > 0 ? (uint32_t)((n - 1) * stride * SIZE) + (uint32_t)channels * SIZE : 0u;
        return uniform_rsrc((uint64_t)p + (uint64_t)(t0 * stride * SIZE), bytes);
    }
    // the wave's checkpoints, from chunk j of a sequence on, and the lane's place in them
    __device__ __forceinline__ Rsrc checkpoints(const float* p, int64_t row, int64_t left, int channels) const
    {
        const int64_t chunks = (left + K - 1) / K, n = chunks < TL ? chunks : TL;
        return uniform_rsrc((uint64_t)p + (uint64_t)(row * channels * 4), p && left > 0 ? (uint32_t)(n * channels * 4) : 0u);
    }
    __device__ __forceinline__ uint32_t checkpoint(int channels) const { return ((uint32_t)tl * (uint32_t)channels + (uint32_t)ch) * 4u | bad; }
    __device__ __forceinline__ uint32_t at(int64_t stride) const { return ((uint32_t)(tl * K) * (uint32_t)stride + (uint32_t)ch) * SIZE | bad; }
    __device__ __forceinline__ void load(Rsrc r, int64_t stride, uint32_t* v) const
    {
        const uint32_t off = at(stride), step = (uint32_t)stride * SIZE;
#pragma unroll
        for (int j = 0; j < K; ++j) v[j] = __builtin_amdgcn_raw_buffer_load_b32(r, off, j * step, 0);
    }
    __device__ __forceinline__ void store(Rsrc r, int64_t stride, int j, uint32_t v) const
    {
        __builtin_amdgcn_raw_buffer_store_b32(v, r, at(stride), (uint32_t)j * (uint32_t)stride * SIZE, kAuxStore);
    }
    static __device__ __forceinline__ float get(uint32_t w, int e)
    {
        if constexpr (CPL == 1) return __uint_as_float(w);
        else return to_f32<DT>(e ? w >> 16 : w & 0xFFFFu);
    }
    static __device__ __forceinline__ uint32_t put(const float* v)
    {
        if constexpr (CPL == 1) return __float_as_uint(v[0]);
        else return pack_elems<DT>(v[0], v[1]);
    }
};

// Slice of workgroup i of a sequence (workgroups go to the 8 XCDs in turn): each XCD takes neighbouring slices, whose rows
// share cache lines where they are half a line or not aligned to lines, and all XCDs take part in each sequence.
__device__ __forceinline__ int slice_of(int i, int slices)
{
    return slices < kGroupSlices ? i : i % 8 * (slices / 8) + i / 8;
}

// WHOLE: a workgroup takes a sequence from its start to its end.  PART_SUM, PART_OUT: it takes a part of one, first
// what the part does to a state (product of its decays, and the state from zero), then the outputs, from the
// state that the parts before leave.
enum Stage { WHOLE, PART_SUM, PART_OUT };

// the r-th longest of 64 sequences or fewer, of equal ones the first first
__device__ __forceinline__ int longest(const GatedArgs& a, int r)
{
    const int lane = threadIdx.x & 63;
    const int len = lane < a.nseq ? (int)gated_span(a, lane).len : -1;
    int rank = 0;
    for (int i = 0; i < a.nseq; ++i) {
        const int other = __builtin_amdgcn_readlane(len, i);
        rank += other > len || (other == len && i < lane);
    }
    return __builtin_ctzll(__ballot(lane < a.nseq && rank == r));
}

// What a workgroup works on.  More whole sequences than run at once are taken from the longest on, so that what is left for
// the end is short (24 sequences of up to 1040 tokens, 2048 channels: 49 us, 58 in the call's order).
struct GatedWork {
    int seq, part, slice;
};
template <int STAGE>
__device__ __forceinline__ GatedWork gated_work(const GatedArgs& a)
{
    const int j = (int)(blockIdx.x / a.slices), i = (int)(blockIdx.x % a.slices);
    GatedWork w{j / a.parts, j % a.parts, slice_of(i, a.slices)};
    if (STAGE == WHOLE && a.nseq > 1 && a.nseq <= 64 && gridDim.x > 256) w.seq = longest(a, w.seq);
    return w;
}

// Gates of tokens that are not there keep the state: a log gate reads 0, a sigmoid's gets infinity.
template <int DT, int GATE, class T>
__device__ __forceinline__ void keep_absent(const T& t, int64_t left, uint32_t* rg)
{
    if constexpr (GATE == GATE_SIGMOID) {
        if (left < T::WAVE_TOKENS) { // the wave's; the same in all lanes
#pragma unroll
            for (int j = 0; j < T::K; ++j)
                if (t.tl * T::K + j >= left) rg[j] = DT == DT_FP32 ? 0x7F800000u : DT == DT_BF16 ? 0x7F807F80u : 0x7C007C00u;
        }
    }
}

// What the lanes of a slice carry from segment to segment of a tile: s_a, s_b hold what a segment does to a state, s_h
// receives the state before each; `product` goes on over all of them.
template <int SEGS, int S, bool BACK, bool SUM>
struct Carry {
    float (*s_a)[S];
    float (*s_b)[S];
    float (*s_h)[S];
    __device__ __forceinline__ void along(float& h, float& product) const
    {
#pragma unroll
        for (int k = 0; k < SEGS; ++k) {
            const int i = BACK ? SEGS - 1 - k : k;
            if (!SUM) s_h[i][threadIdx.x] = h;
            h = __builtin_fmaf(s_a[i][threadIdx.x], h, s_b[i][threadIdx.x]);
            if (SUM) product *= s_a[i][threadIdx.x];
        }
    }
};

template <int DT, int GATE, int INPUT, int LC, int W>
struct Scan {
    using T = Tile<DT, LC, W>;
    static constexpr int K = T::K, CPL = T::CPL;
    // product of the decays, and the state from zero, behind each token
    float through[K][CPL], own[K][CPL];

    static __device__ __forceinline__ void load(const GatedArgs& a, const T& t, const Span& sp, int64_t base, int64_t end, uint32_t* rg, uint32_t* rx)
    {
        const int64_t t0 = base + t.wave * T::WAVE_TOKENS, left = end - t0;
        t.load(t.rows(a.g, sp.begin + t0, a.gs, left, a.channels), a.gs, rg);
        t.load(t.rows(a.x, sp.begin + t0, a.xs, left, a.channels), a.xs, rx);
    }
    __device__ __forceinline__ void sums(const T& t, int64_t left, uint32_t* rg, const uint32_t* rx, float (*s_a)[T::S], float (*s_b)[T::S])
    {
        keep_absent<DT, GATE>(t, left, rg);
#pragma unroll
        for (int j = 0; j < K; ++j)
#pragma unroll
            for (int e = 0; e < CPL; ++e) {
                const GateValue v = gate_value<GATE, INPUT>(T::get(rg[j], e));
                const float in = v.s * T::get(rx[j], e);
                through[j][e] = j ? through[j - 1][e] * v.a : v.a;
                own[j][e] = j ? __builtin_fmaf(v.a, own[j - 1][e], in) : in;
            }
#pragma unroll
        for (int e = 0; e < CPL; ++e) {
            s_a[t.seg()][t.c + e] = through[K - 1][e];
            s_b[t.seg()][t.c + e] = own[K - 1][e];
        }
    }
    __device__ __forceinline__ void outputs(const GatedArgs& a, const T& t, const Span& sp, int seq, int64_t base, int64_t end, float (*s_h)[T::S])
    {
        const int64_t t0 = base + t.wave * T::WAVE_TOKENS, row = sp.begin / K + seq + t0 / K;
        float before[CPL];
        uint32_t ck[CPL];
#pragma unroll
        for (int e = 0; e < CPL; ++e) {
            before[e] = s_h[t.seg()][t.c + e];
            ck[e] = __float_as_uint(before[e]);
        }
        buf_store_words<CPL, 0>(t.checkpoints(a.ckpt, row, end - t0, a.channels), t.checkpoint(a.channels), 0u, ck);
        const Rsrc ro = t.rows(a.o, sp.begin + t0, a.os, end - t0, a.channels);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            float o[CPL];
#pragma unroll
            for (int e = 0; e < CPL; ++e) o[e] = __builtin_fmaf(through[j][e], before[e], own[j][e]);
            t.store(ro, a.os, j, T::put(o));
        }
    }
};

// 3 waves a SIMD: one workgroup of 8 waves on a unit at a time.  Two of them in 128 registers are slower: 24 ragged sequences of
// 2048 channels 58 us (49), 8 packed ones, 8925 tokens, 4096 channels 67 (57); so are three workgroups of 4 waves, 53 and 62.
template <int DT, int GATE, int INPUT, int STAGE, int LC, int W>
__global__ __launch_bounds__(W * 64, 3) void k_gated_scan(GatedArgs a)
{
    using T = Tile<DT, LC, W>;
    constexpr int K = T::K, S = T::S;
    __shared__ float s_a[T::SEGS][S], s_b[T::SEGS][S], s_h[T::SEGS][S];
    const GatedWork work = gated_work<STAGE>(a);
    const int seq = work.seq, slot = gated_slot(a, seq);
    if (slot < 0) return;
    const Span sp = gated_span(a, seq);
    const int64_t begin = STAGE == WHOLE ? 0 : work.part * a.part_tokens;
    const bool last = STAGE == WHOLE || begin + a.part_tokens >= sp.len;
    if (work.part > 0 && begin >= sp.len) return;
    if (STAGE == PART_SUM && last) return;
    const int64_t end = last ? sp.len : begin + a.part_tokens;
    if (work.slice * S >= a.channels) return;
    const T t(work.slice, a.channels);
    const int mine = work.slice * S + threadIdx.x; // the channel that this thread carries along the chunks
    const bool carrier = threadIdx.x < S && mine < a.channels;
    float* state = a.h && carrier ? a.h + (int64_t)slot * a.channels + mine : nullptr;
    const int64_t pitch = (int64_t)a.nseq * a.parts * a.channels;
    float* sums = a.sums + (int64_t)seq * a.parts * a.channels + mine;
    float h = 0.0f, product = 1.0f;
    if (work.part == 0) {
        // the first of several parts has its start from the sums, as the last one overwrites the state
        if (STAGE == PART_OUT && !last) h = carrier ? sums[0] : 0.0f;
        else if (state && !(a.fresh && a.fresh[seq])) h = *state;
        if (STAGE == PART_SUM && carrier) sums[0] = h;
    } else if (STAGE == PART_OUT && carrier) {
        h = sums[pitch];
#pragma unroll 8
        for (int p = 1; p < work.part; ++p) h = __builtin_fmaf(sums[(int64_t)p * a.channels], h, sums[pitch + (int64_t)p * a.channels]);
    }
    const Carry<T::SEGS, S, false, STAGE == PART_SUM> carry{s_a, s_b, s_h};
    Scan<DT, GATE, INPUT, LC, W> scan;
    uint32_t rx[K], rg[K], nx[K], ng[K];
    scan.load(a, t, sp, begin, end, ng, nx);
    for (int64_t base = begin; base < end; base += T::TOKENS) {
#pragma unroll
        for (int j = 0; j < K; ++j) {
            rx[j] = nx[j];
            rg[j] = ng[j];
        }
        scan.load(a, t, sp, base + T::TOKENS, end, ng, nx); // nothing, behind the end
        scan.sums(t, end - base - t.wave * T::WAVE_TOKENS, rg, rx, s_a, s_b);
        __syncthreads();
        if (threadIdx.x < S) carry.along(h, product);
        __syncthreads();
        if constexpr (STAGE != PART_SUM) scan.outputs(a, t, sp, seq, base, end, s_h);
    }
    if constexpr (STAGE == PART_SUM) {
        if (carrier) {
            if (work.part) sums[(int64_t)work.part * a.channels] = product;
            sums[pitch + (int64_t)work.part * a.channels] = h;
        }
    } else if (state && last) {
        *state = h;
    }
}

template <int DT, int GATE, int INPUT, int STAGE, int LC, int W>
struct Back {
    using T = Tile<DT, LC, W>;
    static constexpr int K = T::K, CPL = T::CPL;
    // each token's decay, factor, and the slope of its state along its gate; gradients of its output
    float va[K][CPL], vs[K][CPL], slope[K][CPL];
    uint32_t dy[K];
    struct Raw {
        uint32_t x[K], g[K], d[K], s[CPL];
    };

    static __device__ __forceinline__ void load(const GatedArgs& a, const T& t, const Span& sp, int seq, int64_t base, int64_t end, Raw* r)
    {
        const int64_t t0 = base + t.wave * T::WAVE_TOKENS, left = end - t0;
        t.load(t.rows(a.g, sp.begin + t0, a.gs, left, a.channels), a.gs, r->g);
        t.load(t.rows(a.dout, sp.begin + t0, a.dos, left, a.channels), a.dos, r->d);
        if constexpr (STAGE == PART_SUM) return;
        t.load(t.rows(a.x, sp.begin + t0, a.xs, left, a.channels), a.xs, r->x);
        buf_load_words<CPL, 0>(t.checkpoints(a.ckpt, sp.begin / K + seq + t0 / K, left, a.channels), t.checkpoint(a.channels), 0u, r->s);
    }
    __device__ __forceinline__ void sums(const T& t, int64_t left, Raw* r, float (*s_a)[T::S], float (*s_b)[T::S])
    {
        keep_absent<DT, GATE>(t, left, r->g);
#pragma unroll
        for (int e = 0; e < CPL; ++e) {
            float h = STAGE == PART_SUM ? 0.0f : __uint_as_float(r->s[e]), p = 1.0f, back = 0.0f;
#pragma unroll
            for (int j = 0; j < K; ++j) {
                const GateSlope v = gate_slope<GATE, INPUT>(T::get(r->g[j], e));
                if constexpr (STAGE != PART_SUM) {
                    const float x = T::get(r->x[j], e);
                    slope[j][e] = __builtin_fmaf(v.da, h, v.ds * x);
                    h = __builtin_fmaf(v.a, h, v.s * x);
                    vs[j][e] = v.s;
                }
                va[j][e] = v.a;
                p *= v.a;
            }
#pragma unroll
            for (int j = K - 1; j >= 0; --j) back = va[j][e] * (T::get(r->d[j], e) + back);
            s_a[t.seg()][t.c + e] = p;
            s_b[t.seg()][t.c + e] = back;
        }
#pragma unroll
        for (int j = 0; j < K; ++j) dy[j] = r->d[j];
    }
    __device__ __forceinline__ void outputs(const GatedArgs& a, const T& t, const Span& sp, int64_t base, int64_t end, float (*s_h)[T::S])
    {
        const int64_t t0 = base + t.wave * T::WAVE_TOKENS;
        float back[CPL];
#pragma unroll
        for (int e = 0; e < CPL; ++e) back[e] = s_h[t.seg()][t.c + e];
        const Rsrc rdx = t.rows(a.dx, sp.begin + t0, a.dxs, end - t0, a.channels);
        const Rsrc rdg = t.rows(a.dg, sp.begin + t0, a.dgs, end - t0, a.channels);
#pragma unroll
        for (int j = K - 1; j >= 0; --j) {
            float dx[CPL], dg[CPL];
#pragma unroll
            for (int e = 0; e < CPL; ++e) {
                const float dh = T::get(dy[j], e) + back[e];
                dx[e] = vs[j][e] * dh;
                dg[e] = slope[j][e] * dh;
                back[e] = va[j][e] * dh;
            }
            t.store(rdx, a.dxs, j, T::put(dx));
            t.store(rdg, a.dgs, j, T::put(dg));
        }
    }
};

// Backwards through the chunks.  PART_SUM: what a part makes of the gradient behind it.
// 2 waves a SIMD: a third would spill (8925 packed tokens, 4096 channels: 288 us, 83 without).
template <int DT, int GATE, int INPUT, int STAGE, int LC, int W>
__global__ __launch_bounds__(W * 64, STAGE == PART_SUM ? 3 : 2) void k_gated_backward(GatedArgs a)
{
    using T = Tile<DT, LC, W>;
    constexpr int S = T::S;
    __shared__ float s_a[T::SEGS][S], s_b[T::SEGS][S], s_h[T::SEGS][S];
    const GatedWork work = gated_work<STAGE>(a);
    const int seq = work.seq;
    if (gated_slot(a, seq) < 0) return;
    const Span sp = gated_span(a, seq);
    const int64_t begin = STAGE == WHOLE ? 0 : work.part * a.part_tokens;
    if (work.part > 0 && begin >= sp.len) return;
    if (STAGE == PART_SUM && work.part == 0) return;
    const int64_t end = STAGE == WHOLE || begin + a.part_tokens >= sp.len ? sp.len : begin + a.part_tokens;
    if (work.slice * S >= a.channels) return;
    const T t(work.slice, a.channels);
    const int mine = work.slice * S + threadIdx.x;
    const bool carrier = threadIdx.x < S && mine < a.channels;
    const int64_t edge = (int64_t)seq * a.channels + mine, pitch = (int64_t)a.nseq * a.parts * a.channels;
    float* sums = a.sums + (int64_t)seq * a.parts * a.channels + mine;
    float d = 0.0f, product = 1.0f; // gradient of the state behind the tokens that are left
    if (STAGE != PART_SUM && carrier) {
        if (a.dlast) d = a.dlast[edge];
        if constexpr (STAGE == PART_OUT) {
            const int n = (int)((sp.len + a.part_tokens - 1) / a.part_tokens);
#pragma unroll 8
            for (int p = n - 1; p > work.part; --p) d = __builtin_fmaf(sums[(int64_t)p * a.channels], d, sums[pitch + (int64_t)p * a.channels]);
        }
    }
    const Carry<T::SEGS, S, true, STAGE == PART_SUM> carry{s_a, s_b, s_h};
    Back<DT, GATE, INPUT, STAGE, LC, W> back;
    typename Back<DT, GATE, INPUT, STAGE, LC, W>::Raw r;
    int64_t base = end > begin ? begin + (end - begin - 1) / T::TOKENS * T::TOKENS : begin - T::TOKENS;
    back.load(a, t, sp, seq, base, base >= begin ? end : base, &r);
    for (; base >= begin; base -= T::TOKENS) {
        back.sums(t, end - base - t.wave * T::WAVE_TOKENS, &r, s_a, s_b);
        back.load(a, t, sp, seq, base - T::TOKENS, base > begin ? end : base - T::TOKENS, &r); // nothing, before the first
        __syncthreads();
        if (threadIdx.x < S) carry.along(d, product);
        __syncthreads();
        if constexpr (STAGE != PART_SUM) back.outputs(a, t, sp, base, end, s_h);
    }
    if constexpr (STAGE == PART_SUM) {
        if (carrier) {
            sums[(int64_t)work.part * a.channels] = product;
            sums[pitch + (int64_t)work.part * a.channels] = d;
        }
    } else if (carrier && a.dfirst && work.part == 0) {
        a.dfirst[edge] = d;
    }
}

// One token: a thread takes 8 channels of a sequence, 16 bytes of x and g and 32 of the state: one read and one write of each,
// no wait between waves (one sequence of 2048 channels takes 2 us, a launch's time).
template <int DT, int GATE, int INPUT>
__global__ __launch_bounds__(256) void k_gated_step(GatedArgs a, uint32_t threads)
{
    const uint32_t i = blockIdx.x * 256 + threadIdx.x, per = (uint32_t)a.channels / 8;
    if (i >= threads) return;
    const int seq = (int)(i / per), c = (int)(i % per) * 8;
    const int slot = gated_slot(a, seq);
    if (slot < 0) return;
    float g[8], x[8];
    uint32_t h[8];
    float* state = a.h + (int64_t)slot * a.channels + c;
    load_words<8>(state, h);
    load_elems<DT, 8>(elem_ptr<DT>(a.g, seq * a.gs + c), g);
    load_elems<DT, 8>(elem_ptr<DT>(a.x, seq * a.xs + c), x);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const GateValue v = gate_value<GATE, INPUT>(g[e]);
        h[e] = __float_as_uint(__builtin_fmaf(v.a, __uint_as_float(h[e]), v.s * x[e]));
    }
    store_words<8>(state, h);
    if constexpr (DT == DT_FP32) {
        store_words<8>(static_cast<float*>(a.o) + seq * a.os + c, h);
    } else {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = pack_elems<DT>(__uint_as_float(h[2 * e]), __uint_as_float(h[2 * e + 1]));
        store_words<4>(static_cast<uint16_t*>(a.o) + seq * a.os + c, o);
    }
}

// f(dtype, gate, input) with the three as constants
template <class F>
static hipError_t with_gate(int dtype, int gate, int input, F f)
{
    const auto in = [&](auto dt, auto ga) {
        switch (input) {
        case IN_PLAIN: return f(dt, ga, std::integral_constant<int, IN_PLAIN>{});
        case IN_COMPLEMENT: return f(dt, ga, std::integral_constant<int, IN_COMPLEMENT>{});
        case IN_NORM: return f(dt, ga, std::integral_constant<int, IN_NORM>{});
        }
        return hipErrorInvalidValue;
    };
    const auto ga = [&](auto dt) {
        return gate == GATE_LOG ? in(dt, std::integral_constant<int, GATE_LOG>{}) : in(dt, std::integral_constant<int, GATE_SIGMOID>{});
    };
    switch (dtype) {
    case DT_FP32: return ga(std::integral_constant<int, DT_FP32>{});
    case DT_BF16: return ga(std::integral_constant<int, DT_BF16>{});
    case DT_FP16: return ga(std::integral_constant<int, DT_FP16>{});
    }
    return hipErrorInvalidValue;
}

// How a call is split.  More waves, more registers and loads further ahead change no time, wider rows do: as if a compute unit
// had some 512 cache lines under way whatever its waves do (inferred from times, no counter shows it), so that rows of 64 bytes,
// half a line each, come at half the rate of whole lines; and a workgroup's tiles follow each other.  So: enough workgroups to
// fill the card, and then rows as wide as they can be.  bf16, scan + gradient in us:
//   300 workgroups of 256-byte rows   24 sequences of up to 1040 tokens, 2048 channels      49 (128-byte rows 57)
//   192 of 128-byte rows              8 of up to 1846 tokens, 4096 channels         57 + 83 (256-byte rows 60 + 95)
//   64-byte rows                      8192 tokens, 8192 channels                    98 (128-byte rows 120)
//   parts of 128-byte rows            8192 tokens, 2048 channels                    40 + 58 (whole 71 + 156)
// Parts cost a second pass over what they read, and a launch; whole sequences take as long as the longest of them.  So parts are for
// few workgroups of 64-byte rows, fewer in the scan, which has less to do beside that pass, and not for short sequences.  In us,
// whole and in parts:
//   scan      128 workgroups   1 of 4096: 37, 44;  1 of 2048: 21, 21;  0, 1, 1299 and 2588 tokens: 26, 18
//             192              1 of 2048: 21, 35;  the four 27, 22
//   gradient  128              1 of 4096: 75, 55;  the four 39, 19
//             192              1 of 4096: 86, 70;  1 of 2048: 35, 35
//             256              1 of 8192: 180, 192;  the four 42, 27;  8 of 0 to 1316 tokens 19, 25
//   either    32 to 192        1 of 1024: 11 to 14, 14 to 20, and the gradient 15 to 19, 15 to 20
// Whether several sequences are of one length is not known here: they count as uneven, as the ones above are.  The scan's limits
// are from sequences of up to 4096 tokens and know no length: one of 8192 tokens of 4096 channels still runs whole, on half of
// the units (89 us; its bytes take 31 at a copy's rate).
constexpr int kPartLanes = 32;
struct GatedPlan {
    int lc;             // lanes across the channels
    int slices, parts;  // parts 1: whole sequences
    int64_t part_tokens;
};
static GatedPlan gated_plan(bool back, int cpl, int channels, int nseq, int64_t tokens)
{
    const auto slices = [&](int lc) { return (channels + lc * cpl - 1) / (lc * cpl); };
    const auto wgs = [&](int lc) { return (int64_t)nseq * slices(lc); };
    const auto whole = [&](int lc) { return GatedPlan{lc, slices(lc), 1, 0}; };
    if (nseq == 0) return whole(64);
    if (wgs(64) >= 300) return whole(64);
    if (wgs(32) >= 192) return whole(32);
    const int64_t mean = (tokens + nseq - 1) / nseq, tile = (back ? 4 : 8) * 64 / kPartLanes * kGatedChunk;
    const int64_t few = !back ? (nseq == 1 ? 127 : 159) : mean / 4 < 224 ? mean / 4 : nseq == 1 ? 224 : 256;
    if (mean <= (nseq == 1 ? 1024 : 512) || wgs(16) > few) return whole(16);
    const int64_t want = (512 + wgs(kPartLanes) - 1) / wgs(kPartLanes); // parts of a sequence of the mean length
    GatedPlan p{kPartLanes, slices(kPartLanes), 1, ((mean + want - 1) / want + tile - 1) / tile * tile};
    p.parts = (int)((tokens + p.part_tokens - 1) / p.part_tokens);
    return p;
}

size_t gated_workspace(int channels, int nseq, int64_t tokens)
{
    size_t most = 0;
    for (int i = 0; i < 4; ++i) {
        const GatedPlan p = gated_plan(i & 1, 1 + i / 2, channels, nseq, tokens);
        const size_t n = p.parts > 1 ? (size_t)nseq * p.parts * channels * 8 : 0;
        if (n > most) most = n;
    }
    return most;
}

template <int DT, int GATE, int INPUT, bool BACK, int STAGE, int LC, int W>
static hipError_t launch_gated(const GatedArgs& a, hipStream_t st)
{
    const dim3 grid((unsigned)((int64_t)a.nseq * a.slices * a.parts)), wg(W * 64);
    if constexpr (BACK) hipLaunchKernelGGL((k_gated_backward<DT, GATE, INPUT, STAGE, LC, W>), grid, wg, 0, st, a);
    else hipLaunchKernelGGL((k_gated_scan<DT, GATE, INPUT, STAGE, LC, W>), grid, wg, 0, st, a);
    return hipGetLastError();
}

template <bool BACK>
static hipError_t launch_gated(int dtype, int gate, int input, const GatedArgs& args, void* ws, hipStream_t st)
{
    return with_gate(dtype, gate, input, [&](auto dt, auto ga, auto in) {
        constexpr int DT = decltype(dt)::value, GA = decltype(ga)::value, IN = decltype(in)::value;
        const GatedPlan p = gated_plan(BACK, DT == DT_FP32 ? 1 : 2, args.channels, args.nseq, args.tokens);
        GatedArgs a = args;
        a.slices = p.slices < kGroupSlices ? p.slices : (p.slices + 7) / 8 * 8; // those beyond the channels end at once
        a.parts = p.parts;
        a.part_tokens = p.part_tokens;
        a.sums = (float*)ws;
        if (p.parts > 1) {
            constexpr int W = BACK ? 4 : 8; // gradient of 32768 tokens, 256 channels: 29 us, 8 waves 36; scan 29 and 25
            // what a part makes of a gradient is its decays' doing alone
            const hipError_t e = launch_gated<DT, GA, BACK ? IN_PLAIN : IN, BACK, PART_SUM, kPartLanes, W>(a, st);
            return e != hipSuccess ? e : launch_gated<DT, GA, IN, BACK, PART_OUT, kPartLanes, W>(a, st);
        }
        if (p.lc == 64) return launch_gated<DT, GA, IN, BACK, WHOLE, 64, 8>(a, st);
        if (p.lc == 32) return launch_gated<DT, GA, IN, BACK, WHOLE, 32, 8>(a, st);
        // gradient of 8 sequences, 6312 tokens, 1024 channels: 20 us, 4 waves 24; scan of 8192 tokens, 8192 channels: 105 and 100
        return launch_gated<DT, GA, IN, BACK, WHOLE, 16, BACK ? 8 : 4>(a, st);
    });
}

hipError_t launch_gated_scan(int dtype, int gate, int input, const GatedArgs& a, void* ws, hipStream_t st)
{
    return launch_gated<false>(dtype, gate, input, a, ws, st);
}

hipError_t launch_gated_backward(int dtype, int gate, int input, const GatedArgs& a, void* ws, hipStream_t st)
{
    return launch_gated<true>(dtype, gate, input, a, ws, st);
}

hipError_t launch_gated_step(int dtype, int gate, int input, const GatedArgs& a, hipStream_t st)
{
    const int64_t n = (int64_t)a.nseq * (a.channels / 8);
    const dim3 grid((unsigned)((n + 255) / 256)), wg(256);
    return with_gate(dtype, gate, input, [&](auto dt, auto ga, auto in) {
        hipLaunchKernelGGL((k_gated_step<decltype(dt)::value, decltype(ga)::value, decltype(in)::value>), grid, wg, 0, st, a, (uint32_t)n);
        return hipGetLastError();
    });
}

} // namespace ssq
