// ssq_linattn_prefill.hip -- linear attention with a decay for each head over ragged prompts,
// gfx950: chunks of tokens on the matrix cores, bf16 products for bf16 tensors and fp32 products
// for fp32 and fp16 ones.
#include <cstddef>

#include "ssq_ops_device.h"

namespace ssq {

// sequence i of the call: its slot, or -1 if it is skipped, and its tokens (below 2^31)
struct SeqSpan {
    int slot, begin, end;
};

__device__ __forceinline__ SeqSpan seq_span(const LinArgs& a, int i)
{
    const int most = (int)a.tokens;
    SeqSpan s;
    s.slot = a.slots ? a.slots[i] : i;
    if (s.slot < 0 || s.slot >= a.batch) s.slot = -1;
    s.begin = min(max(a.cu[i], 0), most);
    s.end = min(max(a.cu[i + 1], s.begin), most);
    return s;
}
// the same where i is the wave's: in scalar registers
__device__ __forceinline__ SeqSpan seq_span_uniform(const LinArgs& a, int i)
{
    SeqSpan s = seq_span(a, i);
    s.slot = __builtin_amdgcn_readfirstlane(s.slot);
    s.begin = __builtin_amdgcn_readfirstlane(s.begin);
    s.end = __builtin_amdgcn_readfirstlane(s.end);
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

// ---------------------------------------------------------------------------
// bf16: chunks of 64 tokens on the matrix cores
// ---------------------------------------------------------------------------
// With c_i the sum of a chunk's g up to token i, S the state before it:
//   o_i = scale * (exp(c_i) S q_i + sum_{j<=i} exp(c_i - c_j) (q_i.k_j) v_j)
//   S'  = exp(c_last) S + sum_j (exp(c_last - c_j) v_j) k_j^T
// Every exponent is a difference that is not positive, so nothing overflows; sums of g are taken
// in double, since they are subtracted from each other.
//
// A workgroup of four waves runs one span of tokens for 64 columns of one head.  A wave owns 16
// of them and keeps their state, 16 x 128 fp32, in registers, laid out as a matrix product leaves
// it: lane (g, c) = (lane/16, lane%16) holds column c and the key entries 32g .. 32g+31, which is
// at once the operand of the next S q (any order of the summed index serves, if both operands
// have it).  Each wave also has the scores of 16 keys; they meet the other waves through LDS, the
// first terms in a place of their own and the second ones, once q has been read, in q's: room for
// both would cost the third workgroup of a compute unit.  The barrier between is behind the state's
// products, so that few waves wait there (24 ragged prompts of 32 heads 80 us, 84 with it in front of
// them; 72 with one term, and outputs off by as much again as their rounding).
//
// What bounds it: the chain of each wave and what the waves of a SIMD can issue.  One prompt of 8192
// tokens on 128 heads of 64 takes 203 us: 63 for the parts' own states, 140 for the outputs, which
// join them (the 310 MB that have to move take 47 us as a copy, the 47 GFLOP 37 us as a large matrix
// product).  In the last the matrix pipes are busy 30% of the cycles and vector instructions (decays,
// roundings to bf16 and their remainders, addresses), at 4 cycles each, take 41%; in the rest the
// three waves of a SIMD wait for LDS and at barriers.  Three workgroups of 64 columns on a compute
// unit, 12 waves, against two of 128 columns (two tiles a wave, each fragment of q and k read once for
// both): the ragged prompts, when scores had one term, 84 us against 99, since what one wave waits for
// the others fill.  HBM is not a bound: those prompts move 159 MB in 82 us.
constexpr int kChunk = 64;
constexpr int kCols = 64;
constexpr int kPitch = 136;      // bf16 of a row of 128 in LDS: 16-byte reads of 16 rows fall in different banks
constexpr int kColPitch = 72;    // the same of a row of 64 ...
constexpr int kScorePitch = 40;  // ... and of 32
constexpr double kLog2e = 1.4426950408889634;
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// A block of 4 rows x 16 columns per 16 lanes, lane i naming four columns of row i/4; lane i
// receives column i of the four rows.
__device__ __forceinline__ bf16x4 lds_read_tr(const __bf16* p)
{
    typedef __attribute__((address_space(3))) i16x4* lds_ptr;
    return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)p));
}
__device__ __forceinline__ bf16x8 join4(bf16x4 a, bf16x4 b)
{
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// two values rounded to nearest, ties to even, in one instruction; and back
__device__ __forceinline__ bf16x2 to_bf16(float x, float y)
{
    return __builtin_convertvector(f32x2{x, y}, bf16x2);
}
__device__ __forceinline__ f32x2 from_bf16(bf16x2 v)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    return f32x2{__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u)};
}

// Decays of a chunk.  r_i is the sum of g, in powers of two, over the tokens of i's tile of 16 up
// to i, c_i the sum over the chunk.
struct alignas(16) ReadDecay {
    float r[kChunk], rlo[kChunk]; // r_i as two floats (behind tokens that forget it is some -2000, and
                                  // one would be off by 2^-13): scores on the diagonal decay by exp2(r_i - r_j) ...
    float row[kChunk]; // ... and off it by scale * exp2(r_i) ...
    float col[96];     // ... times exp2(c - c_j) with c before the tile of i: 16 keys for tile 1, 32 for 2, 48 for 3
    float in[kChunk];  // scale * exp2(c_i)
};
struct alignas(16) WriteDecay {
    float out[kChunk];  // exp2(c_last - c_i)
    float keep, change; // exp2(c_last) x = keep*x + change*x, keep 0 or 1: exact near 1
};

// 53,152 bytes: three workgroups on a compute unit
struct alignas(16) ChunkLds {
    __bf16 k[kChunk][kPitch];
    __bf16 v[kChunk][kColPitch];
    WriteDecay w[2]; // of this chunk and the next
    union {
        __bf16 q[kChunk][kPitch];
        __bf16 low[kChunk][kColPitch]; // once q has been read: what p01 and p23 leave of the scores
    };
    __bf16 p01[32][kScorePitch]; // decayed scores, [query][key]: the queries 0 .. 31 have no later keys
    __bf16 p23[32][kColPitch];
    ReadDecay d;
};
constexpr size_t kStateLds = offsetof(ChunkLds, q); // what the parts' own states take

// exp2 of the double x, rounded to a few units of fp32 for any size of x
__device__ __forceinline__ float exp2_of(double x)
{
    const float h = (float)x;
    return __builtin_amdgcn_exp2f(h) * (1.0f + 0.6931472f * (float)(x - (double)h));
}

// x with the double of another lane added, or 0 where the row mask or the row's end leaves none
template <int CTRL, int ROWS>
__device__ __forceinline__ double add_dpp(double x)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xF, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xF, true);
    return x + __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ double readlane_d(double x, int lane)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane), hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// A decay of 2^c as keep*x + change*x.  From 1/2 up the change, exp(y) - 1 of y = c ln 2, is
// taken by itself, as the exponential's series (to y^10: the rest is below 2^-26 of it), so that
// the same decay, chunk after chunk, does not add up one rounding of a number next to 1.
__device__ __forceinline__ float2 decay_of(double c)
{
    const float y = fmaxf((float)(c * 0.6931471805599453), -0.6931472f);
    float p = 1.0f / 3628800.0f;
    p = __builtin_fmaf(p, y, 1.0f / 362880.0f);
    p = __builtin_fmaf(p, y, 1.0f / 40320.0f);
    p = __builtin_fmaf(p, y, 1.0f / 5040.0f);
    p = __builtin_fmaf(p, y, 1.0f / 720.0f);
    p = __builtin_fmaf(p, y, 1.0f / 120.0f);
    p = __builtin_fmaf(p, y, 1.0f / 24.0f);
    p = __builtin_fmaf(p, y, 1.0f / 6.0f);
    p = __builtin_fmaf(p, y, 0.5f);
    const bool near = c > -1.0;
    return make_float2(near ? 1.0f : 0.0f, near ? __builtin_fmaf(p * y, y, y) : exp2_of(c));
}

// the log decay g in powers of two: 2^-184 is 0 in fp32, and so is all that passes such a token
__device__ __forceinline__ double log2_decay(float g)
{
    return (double)fmaxf(g, -128.0f) * kLog2e;
}
// sums along the rows of 16 lanes, from those to the sums of all lanes up to this one
__device__ __forceinline__ double row_sums(double x)
{
    x = add_dpp<0x111, 0xF>(x); // from 1, 2, 4 and 8 lanes before
    x = add_dpp<0x112, 0xF>(x);
    x = add_dpp<0x114, 0xF>(x);
    return add_dpp<0x118, 0xF>(x);
}
__device__ __forceinline__ double wave_sums(double r)
{
    r = add_dpp<0x142, 0xA>(r); // the last lane of the row before to rows 1 and 3
    return add_dpp<0x143, 0xC>(r); // lane 31 to rows 2 and 3
}

// One wave's share of a chunk's decays; lane = token, g its log decay (0 behind the span's end).
__device__ __forceinline__ void chunk_decays(int wave, float g, float scale, int lane, ReadDecay& d, WriteDecay& w)
{
    const double r = row_sums(log2_decay(g)), c = wave_sums(r);
    if (wave == 0) {
        const float hi = (float)r;
        d.r[lane] = hi;
        d.rlo[lane] = (float)(r - (double)hi);
        d.row[lane] = scale * exp2_of(r);
    } else if (wave == 1) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (lane < 16 * (i + 1)) d.col[8 * i * (i + 1) + lane] = exp2_of(readlane_d(c, 16 * i + 15) - c);
    } else if (wave == 2) {
        d.in[lane] = scale * exp2_of(c);
        if (lane == 63) {
            const float2 e = decay_of(c);
            w.keep = e.x;
            w.change = e.y;
        }
    } else {
        w.out[lane] = exp2_of(readlane_d(c, 63) - c);
    }
}

enum { WHOLE = 0, PART_STATE = 1, PART_OUT = 2 };

// Terms of bf16 that stand for an fp32 operand, each leaving 2^-8 of what the one before left.  The
// state as S q reads it and the decayed scores as v meets them: two, off by 2^-16 of each term of an
// output, so that o is exact to its own rounding (one term would add an error as large as that
// rounding, and many times it where the terms of an output cancel).  The decayed values that
// are added to a state which is kept: three, all 24 bits (two leave 2e-6 of the state, as much as
// a chain of fp32 sums; 128 heads x 8192 tokens take 7% less time with them); two where the state
// only serves to the end of a part.
constexpr int kReadTerms = 2;
template <int MODE>
constexpr int write_terms() { return MODE == PART_OUT ? 2 : 3; }

struct ChunkArgs {
    LinArgs a;
    float* part_state;  // [parts][H*P][128], with `fold` also [nseq]: the states before the call
    float2* part_decay; // [parts][H]: keep, change
    int64_t parts;      // places of parts
    int part_tokens;    // a multiple of kChunk
    int fold;           // the parts' outputs join the states themselves
    int items;          // sequences, or parts at most
    int blocks;         // column blocks
    int run, runs;      // blocks on an XCD together, and such runs in `blocks`
    int bins;           // runs that the compute units take side by side; 0: sequences in their order
};

// the place of a sequence's first part among all parts: sequences follow each other, each ending in a part of its own
__device__ __forceinline__ int64_t first_part(const ChunkArgs& c, int64_t begin, int seq)
{
    return begin / c.part_tokens + seq;
}

// a descriptor of the wave's: without the readfirstlanes the compiler would loop over its lanes' values
__device__ __forceinline__ Rsrc wave_rsrc(const void* base, uint32_t bytes)
{
    const uint64_t b = (uint64_t)base;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)b), hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32));
    return make_rsrc((const void*)(((uint64_t)hi << 32) | lo), (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes));
}

// What a workgroup does: a block of columns of a sequence, or of a part of one.
struct Work {
    int block, item, seq, slot;
    bool fresh, last;   // last, part: of a sequence's parts
    int64_t part;
    int64_t begin, end; // tokens
};

template <int MODE>
__device__ __forceinline__ bool find_work(const ChunkArgs& c, Work& w)
{
    const LinArgs& a = c.a;
    // Workgroups go to the 8 XCDs in turn.  Runs of `run` blocks, which share keys, are dealt to
    // the XCDs, so that an XCD's L2 reads those keys once.
    // Whole sequences, up to 64 of them (a lane ranks each), are taken from the longest to the
    // shortest, and every other row of the runs that lie side by side the other way round, so that
    // the workgroups that share a compute unit have about the same work: 24 ragged prompts of 32
    // heads 79 us, in their own order 85; 64 of 24 heads, to 3000 tokens, 365 and 436; of one
    // length, where it serves nothing, 79 either way.
    const unsigned at = blockIdx.x / 8;
    unsigned deal = at / c.run * 8 + blockIdx.x % 8;
    if (deal >= (unsigned)c.items * c.runs) return false;
    if (MODE == WHOLE && c.bins) { // every other row of bins from its end
        const unsigned row = deal / c.bins, pos = deal % c.bins;
        if (row % 2 && (row + 1) * c.bins <= (unsigned)c.items * c.runs) deal = row * c.bins + c.bins - 1 - pos;
    }
    w.block = (int)(deal % c.runs * c.run + at % c.run);
    w.item = (int)(deal / c.runs);
    if (w.block >= c.blocks) return false;
    w.seq = w.item;
    if (MODE == WHOLE && c.bins) { // the item-th longest sequence
        const int lane = threadIdx.x & 63;
        uint32_t key = 0;
        if (lane < a.nseq) {
            const SeqSpan s = seq_span(a, lane);
            key = s.slot < 0 ? lane : (uint32_t)(s.end - s.begin + 63) / 64 * 64 + lane;
        }
        int rank = 0;
        for (int j = 0; j < a.nseq; j += 8)
#pragma unroll
            for (int i = 0; i < 8; ++i) rank += (uint32_t)__builtin_amdgcn_readlane((int)key, j + i) > key;
        w.seq = __builtin_amdgcn_readfirstlane((int)__builtin_ctzll(__ballot(lane < a.nseq && rank == w.item)));
    }
    if constexpr (MODE != WHOLE) { // the last sequence whose first part is not behind the item
        int lo = 0, hi = a.nseq - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            const SeqSpan m = seq_span_uniform(a, mid);
            if (first_part(c, m.begin, mid) <= w.item) lo = mid;
            else hi = mid - 1;
        }
        w.seq = lo;
    }
    const SeqSpan span = seq_span_uniform(a, w.seq);
    w.slot = span.slot;
    if (span.slot < 0) return false;
    w.fresh = a.fresh && __builtin_amdgcn_readfirstlane((int)a.fresh[w.seq]);
    w.begin = span.begin;
    w.end = span.end;
    if constexpr (MODE == WHOLE) return w.begin < w.end || w.fresh;
    const int64_t part = (int64_t)w.item - first_part(c, span.begin, w.seq);
    w.part = part;
    w.last = true;
    if (MODE == PART_OUT && c.fold && part == 0 && w.begin == w.end) return w.fresh; // its state is zeroed
    w.begin += part * c.part_tokens;
    if (part < 0 || w.begin >= w.end) return false; // a place of no part
    if (w.end > w.begin + c.part_tokens) {
        w.end = w.begin + c.part_tokens;
        w.last = false;
    }
    return true;
}

// A wave's 16 columns of a state are 8 vectors a lane, vector u the entries 32g + 4u .. 32g + 4u + 3
// of column l16: in rows in a state, one vector after the other in a part's.
struct Tile {
    float* rows; // + 4 floats a vector
    float* part; // of place 0, + 256 floats a vector
    int64_t place; // floats from one place to the next
    const float2* decay; // of place 0, + H
};
__device__ __forceinline__ Tile tile_of(const ChunkArgs& c, const Work& w, int head, int64_t col, int lane)
{
    const LinArgs& a = c.a;
    Tile t;
    t.rows = seq_rows(a, w.seq, w.slot) + (col + (lane & 15)) * 128 + 32 * (lane >> 4);
    t.part = c.part_state + col * 128 + lane * 4;
    t.place = (int64_t)a.H * a.P * 128;
    t.decay = c.part_decay + head;
    return t;
}
__device__ __forceinline__ void load_tile(const float* p, int step, f32x4 (&x)[8])
{
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = *reinterpret_cast<const f32x4*>(p + u * step);
}
__device__ __forceinline__ void store_tile(float* p, int step, const f32x4 (&x)[8])
{
#pragma unroll
    for (int u = 0; u < 8; ++u) *reinterpret_cast<f32x4*>(p + u * step) = x[u];
}
// the state x behind a part with this decay and this own state
__device__ __forceinline__ f32x4 pass_part(f32x4 x, float2 d, f32x4 own)
{
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = __builtin_fmaf(x[r], d.y, x[r] * d.x) + own[r];
    return x;
}

// The state that a workgroup starts from.  With `fold` the parts' own states are joined here, part 0's
// already with the sequence's state before the call, and the last part leaves the state behind them.
template <int MODE>
__device__ __forceinline__ void first_state(const ChunkArgs& c, const Work& w, const Tile& t, f32x4 (&x)[8])
{
    if constexpr (MODE == WHOLE) {
        if (!w.fresh) load_tile(t.rows, 4, x);
        return;
    }
    // the join's state, the state before the call, or part 0's
    const int64_t first = w.item - w.part;
    const int64_t from = !c.fold ? w.item : w.part == 0 ? c.parts + w.seq : first;
    if (!(c.fold && w.part == 0 && w.fresh)) load_tile(t.part + from * t.place, 256, x);
    if (!c.fold) return;
    for (int64_t p = first + 1; p < w.item; ++p) {
        f32x4 own[8];
        load_tile(t.part + p * t.place, 256, own);
        const float2 d = t.decay[p * c.a.H];
#pragma unroll
        for (int u = 0; u < 8; ++u) x[u] = pass_part(x[u], d, own[u]);
    }
    if (!w.last) return;
    if (w.begin == w.end) { // an empty sequence, which is fresh
#pragma unroll
        for (int u = 0; u < 8; ++u) *reinterpret_cast<f32x4*>(t.rows + 4 * u) = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        return;
    }
    f32x4 own[8];
    load_tile(t.part + w.item * t.place, 256, own);
    const float2 d = w.part > 0 ? t.decay[w.item * c.a.H] : float2{0.0f, 0.0f}; // part 0 has the state before it
#pragma unroll
    for (int u = 0; u < 8; ++u) *reinterpret_cast<f32x4*>(t.rows + 4 * u) = pass_part(x[u], d, own[u]);
}
// what PART_STATE leaves: its own state, part 0's with the state before the call, which is kept aside
__device__ __forceinline__ void leave_part(const ChunkArgs& c, const Work& w, const Tile& t, float2 d, f32x4 (&x)[8])
{
    if (c.fold && w.part == 0 && !w.fresh) {
        f32x4 s0[8];
        load_tile(t.rows, 4, s0);
        store_tile(t.part + (c.parts + w.seq) * t.place, 256, s0);
#pragma unroll
        for (int u = 0; u < 8; ++u) *reinterpret_cast<f32x4*>(t.part + w.item * t.place + u * 256) = pass_part(s0[u], d, x[u]);
    } else {
        store_tile(t.part + w.item * t.place, 256, x);
    }
}

template <int MODE>
__global__ __launch_bounds__(256, MODE == PART_STATE ? 4 : 3) void k_linattn_chunk(ChunkArgs c)
{
    __shared__ alignas(16) uint8_t lds[MODE == PART_STATE ? kStateLds : sizeof(ChunkLds)];
    ChunkLds& s = *reinterpret_cast<ChunkLds*>(lds);
    const LinArgs& a = c.a;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    Work work;
    if (!find_work<MODE>(c, work)) return;
    const int block = work.block, item = work.item;
    const int64_t begin = work.begin, end = work.end;
    const int per_head = (a.P + kCols - 1) / kCols;
    const int head = block / per_head, p0 = block % per_head * kCols;
    const int cols = min(kCols, a.P - p0);                 // a multiple of 16
    const int64_t col0 = (int64_t)head * a.P + p0;         // of v and o, and the row of the state
    const int kvh = head / (a.H / a.G);
    const bool have = wave * 16 < cols;                    // a wave without columns runs on zeros and stores nothing

    const __bf16* qp = static_cast<const __bf16*>(a.q) + kvh * 128;
    const __bf16* kp = static_cast<const __bf16*>(a.k) + kvh * 128;
    const __bf16* vp = static_cast<const __bf16*>(a.v) + col0;
    __bf16* op = static_cast<__bf16*>(a.o) + col0;

    // n-tile t: entries 32g + 4t .. 32g + 4t + 3 of column l16.  A sequence's state is in rows, a
    // part's as the registers hold it.
    f32x4 S[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) S[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (have && MODE != PART_STATE) first_state<MODE>(c, work, tile_of(c, work, head, col0 + wave * 16, lane), S);
    if constexpr (MODE != PART_STATE) { // the scores above the diagonal's tiles stay zero
        constexpr int words = (sizeof(s.p01) + sizeof(s.p23)) / 4;
        for (int i = tid; i < words; i += 256) reinterpret_cast<uint32_t*>(s.p01)[i] = 0;
    }

    // Tiles come and go through buffer descriptors that end with the span: rows behind it read 0
    // and are not written.  16 pieces of 16 bytes a row of q and k, 8 of v.
    const uint32_t piece = tid & 15, prow = tid >> 4, vpiece = tid & 7, vrow = tid >> 3;
    const uint32_t q_row = (uint32_t)a.qs * 2, k_row = (uint32_t)a.ks * 2, v_row = (uint32_t)a.vs * 2, o_row = (uint32_t)a.os * 2, g_row = (uint32_t)a.gs * 4;
    const uint32_t q_off = prow * q_row + piece * 16, k_off = prow * k_row + piece * 16;
    constexpr uint32_t kNone = 0x80000000u; // behind every range
    const uint32_t v_off = (int)vpiece * 8 < cols ? vrow * v_row + vpiece * 16 : kNone;
    const uint32_t o_off = have ? l16 * o_row + wave * 32 + 8 * g : kNone;
    u32x4 rq[4], rk[4], rv[2];
    float rg = 0.0f;
    // offsets are added up where they are used: kept for the whole loop they would cost the registers that it lacks
    auto here = [](uint32_t x) {
        asm volatile("" : "+v"(x));
        return x;
    };
    auto rows_of = [&](int64_t t0) { return (uint32_t)(end - t0 < kChunk ? end - t0 : kChunk) - 1; };
    auto fetch_q = [&](int64_t t0) {
        const Rsrc bq = wave_rsrc(qp + t0 * a.qs, rows_of(t0) * q_row + 256);
        const uint32_t at = here(q_off);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if constexpr (MODE != PART_STATE) rq[i] = __builtin_amdgcn_raw_buffer_load_b128(bq, at + 16 * i * q_row, 0, 0);
    };
    auto fetch = [&](int64_t t0) {
        const Rsrc bk = wave_rsrc(kp + t0 * a.ks, rows_of(t0) * k_row + 256);
        const Rsrc bv = wave_rsrc(vp + t0 * a.vs, rows_of(t0) * v_row + cols * 2);
        const uint32_t k_at = here(k_off), v_at = here(v_off);
        // without g an empty range, which reads 0 (two descriptors to choose from would cost 3% of ragged prompts)
        const Rsrc bg = wave_rsrc((const void*)((uint64_t)a.g + (uint64_t)(t0 * a.gs + head) * 4), a.g ? rows_of(t0) * g_row + 4 : 0);
        const uint32_t g_at = (uint32_t)lane <= rows_of(t0) ? lane * g_row : kNone; // a stride of 0 has no row behind the span
        rg = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(bg, g_at, 0, 0));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            rk[i] = __builtin_amdgcn_raw_buffer_load_b128(bk, k_at + 16 * i * k_row, 0, 0);
            if (i < 2) rv[i] = __builtin_amdgcn_raw_buffer_load_b128(bv, v_at + 32 * i * v_row, 0, 0);
        }
    };
    // PART_STATE runs from the last chunk to the first, so that what is summed need not decay:
    // `after` is the decay of the chunks behind.
    double after = 0.0;
    auto decays = [&](int buf) {
        if constexpr (MODE == PART_STATE) {
            const double sum = wave_sums(row_sums(log2_decay(rg))), last = readlane_d(sum, 63);
            if (wave == 0) s.w[buf].out[lane] = exp2_of(after + (last - sum));
            after += last;
        } else {
            chunk_decays(wave, rg, a.oscale, lane, s.d, s.w[buf]);
        }
    };
    const int64_t chunks = (end - begin + kChunk - 1) / kChunk;
    auto start = [&](int64_t n) { return begin + (MODE == PART_STATE ? chunks - 1 - n : n) * kChunk; };
    if (chunks > 0) { // an empty sequence has no row that a descriptor could end with
        fetch(start(0));
        fetch_q(start(0));
        decays(0);
    }
    int buf = 0;
    for (int64_t n = 0; n < chunks; ++n, buf ^= 1) {
        const int64_t t0 = start(n);
        const WriteDecay& sw = s.w[buf];
        __syncthreads(); // the previous chunk has been read
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (MODE != PART_STATE) *reinterpret_cast<u32x4*>(&s.q[prow + 16 * i][piece * 8]) = rq[i];
            *reinterpret_cast<u32x4*>(&s.k[prow + 16 * i][piece * 8]) = rk[i];
            if (i < 2) *reinterpret_cast<u32x4*>(&s.v[vrow + 32 * i][vpiece * 8]) = rv[i];
        }
        __syncthreads();
        const bool more = n + 1 < chunks;
        if (more) fetch(start(n + 1));

        f32x4 O[4]; // query tile i: columns 4g .. 4g+3, query l16
        if constexpr (MODE != PART_STATE) {
            // S q, the state as a sum of bf16, and the scores of this wave's 16 keys, which use the
            // same fragments of q (rows keys, columns queries; those above the diagonal for nothing)
            f32x4 A[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) A[i] = O[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                __builtin_amdgcn_sched_barrier(0); // one step's fragments at a time: more would not fit the registers
                const bf16x8 kk = *reinterpret_cast<const bf16x8*>(&s.k[wave * 16 + l16][g * 32 + ks * 8]);
                bf16x8 qq[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) qq[i] = *reinterpret_cast<const bf16x8*>(&s.q[i * 16 + l16][g * 32 + ks * 8]);
                bf16x8 term[kReadTerms];
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    f32x2 v = {S[2 * ks + e / 4][e % 4], S[2 * ks + e / 4][e % 4 + 1]};
#pragma unroll
                    for (int j = 0; j < kReadTerms; ++j) {
                        const bf16x2 h = to_bf16(v.x, v.y);
                        const f32x2 f = from_bf16(h);
                        term[j][e] = h.x;
                        term[j][e + 1] = h.y;
                        v.x -= f.x;
                        v.y -= f.y;
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) A[i] = mfma(kk, qq[i], A[i]);
#pragma unroll
                for (int j = 0; j < kReadTerms; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) O[i] = mfma(term[j], qq[i], O[i]);
            }
            const int kj = wave * 16 + g * 4;
            bf16x4 low[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int qi = i * 16 + l16;
                f32x4 w;
                low[i] = bf16x4{};
                if (i < wave) continue;
                if (i == wave) {
                    const f32x4 rj = *reinterpret_cast<const f32x4*>(&s.d.r[kj]), lj = *reinterpret_cast<const f32x4*>(&s.d.rlo[kj]);
                    const float ri = s.d.r[qi], li = s.d.rlo[qi];
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        w[r] = kj + r <= qi ? A[i][r] * (a.oscale * __builtin_amdgcn_exp2f((ri - rj[r]) + (li - lj[r]))) : 0.0f;
                } else {
                    w = A[i] * s.d.row[qi] * *reinterpret_cast<const f32x4*>(&s.d.col[8 * i * (i - 1) + kj]);
                }
                const bf16x2 w01 = to_bf16(w.x, w.y), w23 = to_bf16(w.z, w.w);
                __bf16* const p = i < 2 ? &s.p01[qi][kj] : &s.p23[qi - 32][kj];
                *reinterpret_cast<bf16x4*>(p) = __builtin_shufflevector(w01, w23, 0, 1, 2, 3);
                const f32x2 f01 = from_bf16(w01), f23 = from_bf16(w23);
                low[i] = __builtin_shufflevector(to_bf16(w.x - f01.x, w.y - f01.y), to_bf16(w.z - f23.x, w.w - f23.y), 0, 1, 2, 3);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) O[i] *= s.d.in[i * 16 + l16];
            __syncthreads(); // the scores are written, q and the decays that they took are read
#pragma unroll
            for (int i = 0; i < 4; ++i) // a tile above the diagonal that shares a product with one on it is zero
                if (i >= (wave & ~1)) *reinterpret_cast<bf16x4*>(&s.low[i * 16 + l16][kj]) = low[i];
        }
        if (more) fetch_q(start(n + 1)); // not sooner: its registers are S q's operands till here
        bf16x8 vf[2]; // this wave's columns of v: column l16, tokens 32*kb + 8g .. +7
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            const int row = kb * 32 + g * 8 + (l16 >> 2), col = wave * 16 + 4 * (l16 & 3);
            vf[kb] = join4(lds_read_tr(&s.v[row][col]), lds_read_tr(&s.v[row + 4][col]));
        }
        if constexpr (MODE != PART_STATE) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                O[i] = mfma(vf[0], *reinterpret_cast<const bf16x8*>(i < 2 ? &s.p01[i * 16 + l16][g * 8] : &s.p23[i * 16 - 32 + l16][g * 8]), O[i]);
#pragma unroll
            for (int i = 2; i < 4; ++i)
                O[i] = mfma(vf[1], *reinterpret_cast<const bf16x8*>(&s.p23[i * 16 - 32 + l16][32 + g * 8]), O[i]);
        }
        if (MODE != PART_OUT || more) { // the next part has its own state
            // the state: decayed, and the chunk's writes with v's decay, as a sum of bf16
            if constexpr (MODE != PART_STATE) {
                const float change = sw.change;
                if (__builtin_amdgcn_readfirstlane(__float_as_int(sw.keep)) != 0) {
#pragma unroll
                    for (int t = 0; t < 8; ++t)
#pragma unroll
                        for (int r = 0; r < 4; ++r) S[t][r] = __builtin_fmaf(S[t][r], change, S[t][r]);
                } else {
#pragma unroll
                    for (int t = 0; t < 8; ++t) S[t] *= change;
                }
            }
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                const float* od = &sw.out[kb * 32 + g * 8];
                const f32x4 o0 = *reinterpret_cast<const f32x4*>(od), o1 = *reinterpret_cast<const f32x4*>(od + 4);
                const float oe[8] = {o0.x, o0.y, o0.z, o0.w, o1.x, o1.y, o1.z, o1.w};
                bf16x8 term[write_terms<MODE>()];
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    f32x2 v = from_bf16(bf16x2{vf[kb][e], vf[kb][e + 1]});
                    v.x *= oe[e];
                    v.y *= oe[e + 1];
#pragma unroll
                    for (int j = 0; j < write_terms<MODE>(); ++j) {
                        const bf16x2 h = to_bf16(v.x, v.y);
                        const f32x2 f = from_bf16(h);
                        term[j][e] = h.x;
                        term[j][e + 1] = h.y;
                        v.x -= f.x;
                        v.y -= f.y;
                    }
                }
                const int row = kb * 32 + g * 8 + (l16 >> 2), col = (l16 & 3) * 32;
#pragma unroll
                for (int t = 0; t < 8; t += 4) {
                    bf16x8 kf[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        kf[u] = join4(lds_read_tr(&s.k[row][col + 4 * (t + u)]), lds_read_tr(&s.k[row + 4][col + 4 * (t + u)]));
#pragma unroll
                    for (int j = 0; j < write_terms<MODE>(); ++j)
#pragma unroll
                        for (int u = 0; u < 4; ++u) S[t + u] = mfma(kf[u], term[j], S[t + u]);
                }
            }
        }
        if constexpr (MODE != PART_STATE) {
            __syncthreads(); // the scores' second terms are written
#pragma unroll
            for (int i = 0; i < 4; ++i) O[i] = mfma(vf[0], *reinterpret_cast<const bf16x8*>(&s.low[i * 16 + l16][g * 8]), O[i]);
#pragma unroll
            for (int i = 2; i < 4; ++i) O[i] = mfma(vf[1], *reinterpret_cast<const bf16x8*>(&s.low[i * 16 + l16][32 + g * 8]), O[i]);
            const uint32_t last = (uint32_t)(end - t0 < kChunk ? end - t0 : kChunk) - 1;
            const Rsrc bo = wave_rsrc(op + t0 * a.os, last * o_row + cols * 2);
            const uint32_t o_at = here(o_off);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const u32x2 w4 = {__builtin_bit_cast(uint32_t, to_bf16(O[i].x, O[i].y)), __builtin_bit_cast(uint32_t, to_bf16(O[i].z, O[i].w))};
                __builtin_amdgcn_raw_buffer_store_b64(w4, bo, o_at + i * 16 * o_row, 0, 0);
            }
        }
        if (more) decays(buf ^ 1);
    }
    if (have && MODE != PART_OUT) {
        const Tile tile = tile_of(c, work, head, col0 + wave * 16, here(lane)); // not addresses kept through the loop
        if constexpr (MODE == WHOLE) store_tile(tile.rows, 4, S);
        else leave_part(c, work, tile, decay_of(after), S);
    }
    if constexpr (MODE == PART_STATE) {
        if (tid == 0 && p0 == 0) c.part_decay[(int64_t)item * a.H + head] = decay_of(after);
    }
}

// ---------------------------------------------------------------------------
// fp32 and fp16: chunks of 32 tokens, every product on the fp32 matrix instruction
// ---------------------------------------------------------------------------
// The same mathematics with nothing rounded below fp32: bf16 products would need three terms of
// each operand, six products and as many instructions to split them.  The instruction sums four
// products at a sixteenth of the bf16 rate, so a chunk is half as long, which halves its scores.
// A workgroup of four waves has 64 columns of one head; a lane's 32 state entries are 32g + 8r + t
// of column l16, so that its key and query operands are 16-byte reads.
constexpr int kWideChunk = 32;
constexpr int kWidePitch = 132;     // floats of a row of 128 in LDS
constexpr int kWideColPitch = 68;   // of 64
constexpr int kWideScorePitch = 36; // of 32

struct alignas(16) WideDecay {
    float r[kWideChunk], rlo[kWideChunk]; // sums of g, in powers of two, along tiles of 16, as two floats
    float row[kWideChunk];                // scale * exp2(r_i)
    float col[16];                        // exp2(c_15 - c_j)
    float in[kWideChunk];                 // scale * exp2(c_i)
    float out[kWideChunk];                // exp2(c_last - c_i), in PART_STATE with what follows the chunk
    float keep, change;
};
struct alignas(16) WideLds {
    float q[kWideChunk][kWidePitch], k[kWideChunk][kWidePitch];
    float v[kWideChunk][kWideColPitch];
    float p[kWideChunk][kWideScorePitch];
    WideDecay d[2];
};

__device__ __forceinline__ f32x4 mfma_f32(float a, float b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

template <int MODE, int DT>
__global__ __launch_bounds__(256, 2) void k_linattn_wide(ChunkArgs c)
{
    using T = typename Elem<DT>::T;
    constexpr int SIZE = sizeof(T), PER = 16 / SIZE; // elements in 16 bytes
    __shared__ WideLds s;
    __shared__ float2 part_decay;
    const LinArgs& a = c.a;
    Work work;
    if (!find_work<MODE>(c, work)) return;
    const int64_t begin = work.begin, end = work.end;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int per_head = (a.P + kCols - 1) / kCols;
    const int head = work.block / per_head, p0 = work.block % per_head * kCols;
    const int cols = min(kCols, a.P - p0);         // a multiple of 16
    const bool have = wave * 16 < cols;            // a wave without columns runs on zeros and stores nothing
    const int64_t col0 = (int64_t)head * a.P + p0; // of v and o, and the row of the state
    const int kvh = head / (a.H / a.G);
    const T* qp = static_cast<const T*>(a.q) + kvh * 128;
    const T* kp = static_cast<const T*>(a.k) + kvh * 128;
    const T* vp = static_cast<const T*>(a.v) + col0;
    T* op = static_cast<T*>(a.o) + col0;

    f32x4 S[8]; // S[t][r]: entry 32g + 8r + t of column l16
#pragma unroll
    for (int t = 0; t < 8; ++t) S[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (have && MODE != PART_STATE) {
        f32x4 x[8] = {};
        first_state<MODE>(c, work, tile_of(c, work, head, col0 + wave * 16, lane), x);
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[u % 2 * 4 + e][u / 2] = x[u][e];
    }

    // rows of 128 (q, k) and of 64 (v) in pieces of 16 bytes
    constexpr int QP = 128 / PER, QR = 256 / QP, NQ = kWideChunk / QR;
    constexpr int VP = 64 / PER, VR = 256 / VP, NV = kWideChunk / VR;
    const uint32_t qpiece = tid % QP, qrow = tid / QP, vpiece = tid % VP, vrow = tid / VP;
    const uint32_t q_row = (uint32_t)a.qs * SIZE, k_row = (uint32_t)a.ks * SIZE, v_row = (uint32_t)a.vs * SIZE, o_row = (uint32_t)a.os * SIZE;
    const uint32_t q_off = qrow * q_row + qpiece * 16, k_off = qrow * k_row + qpiece * 16;
    constexpr uint32_t kNone = 0x80000000u; // behind every range
    const uint32_t v_off = (int)(vpiece * PER) < cols ? vrow * v_row + vpiece * 16 : kNone;
    const uint32_t o_off = have ? l16 * o_row + (wave * 16 + 4 * g) * SIZE : kNone;
    u32x4 rq[NQ], rk[NQ], rv[NV];
    float rg = 0.0f;
    auto fetch = [&](int64_t t0) {
        const uint32_t last = (uint32_t)(end - t0 < kWideChunk ? end - t0 : kWideChunk) - 1;
        const Rsrc bq = wave_rsrc(qp + t0 * a.qs, last * q_row + 128 * SIZE);
        const Rsrc bk = wave_rsrc(kp + t0 * a.ks, last * k_row + 128 * SIZE);
        const Rsrc bv = wave_rsrc(vp + t0 * a.vs, last * v_row + cols * SIZE);
        rg = 0.0f;
        if (wave == 3 && a.g && lane < kWideChunk && t0 + lane < end) rg = a.g[(t0 + lane) * a.gs + head];
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            if constexpr (MODE != PART_STATE) rq[i] = __builtin_amdgcn_raw_buffer_load_b128(bq, q_off + QR * i * q_row, 0, 0);
            rk[i] = __builtin_amdgcn_raw_buffer_load_b128(bk, k_off + QR * i * k_row, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) rv[i] = __builtin_amdgcn_raw_buffer_load_b128(bv, v_off + VR * i * v_row, 0, 0);
    };
    auto put = [&](float* to, u32x4 w) { // 16 bytes as floats
        if constexpr (DT == DT_FP32) {
            *reinterpret_cast<u32x4*>(to) = w;
        } else {
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<f32x4*>(to + 4 * i) = f32x4{to_f32<DT>(ws[2 * i] & 0xFFFFu), to_f32<DT>(ws[2 * i] >> 16),
                                                              to_f32<DT>(ws[2 * i + 1] & 0xFFFFu), to_f32<DT>(ws[2 * i + 1] >> 16)};
        }
    };
    // the last wave has no scores and makes the decays, a chunk's while the one before it is run
    double after = 0.0; // PART_STATE runs from the last chunk to the first: the decay of those behind
    auto decays = [&](int buf) {
        if (wave != 3) return;
        WideDecay& d = s.d[buf];
        const double r = row_sums(log2_decay(rg)), sum = wave_sums(r), last = readlane_d(sum, 63);
        if constexpr (MODE == PART_STATE) {
            if (lane < kWideChunk) d.out[lane] = exp2_of(after + (last - sum));
            after += last;
        } else if (lane < kWideChunk) {
            const float hi = (float)r;
            d.r[lane] = hi;
            d.rlo[lane] = (float)(r - (double)hi);
            d.row[lane] = a.oscale * exp2_of(r);
            if (lane < 16) d.col[lane] = exp2_of(readlane_d(sum, 15) - sum);
            d.in[lane] = a.oscale * exp2_of(sum);
            d.out[lane] = exp2_of(last - sum);
            if (lane == 0) {
                const float2 e = decay_of(last);
                d.keep = e.x;
                d.change = e.y;
            }
        }
    };
    const int64_t chunks = (end - begin + kWideChunk - 1) / kWideChunk;
    auto start = [&](int64_t n) { return begin + (MODE == PART_STATE ? chunks - 1 - n : n) * kWideChunk; };
    if (chunks > 0) { // an empty sequence has no row that a descriptor could end with
        fetch(start(0));
        decays(0);
    }
    int buf = 0;
    for (int64_t n = 0; n < chunks; ++n, buf ^= 1) {
        const int64_t t0 = start(n);
        const WideDecay& d = s.d[buf];
        __syncthreads(); // the previous chunk has been read
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            if constexpr (MODE != PART_STATE) put(&s.q[qrow + QR * i][qpiece * PER], rq[i]);
            put(&s.k[qrow + QR * i][qpiece * PER], rk[i]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) put(&s.v[vrow + VR * i][vpiece * PER], rv[i]);
        __syncthreads();
        const bool more = n + 1 < chunks;
        if (more) fetch(start(n + 1));

        f32x4 O[2]; // query tile i: columns 4g .. 4g+3, query l16
        if constexpr (MODE != PART_STATE) {
            // S q, and the scores of one tile: (queries, keys) = (0, 0), (1, 0), (1, 1) of the first three waves
            const int qt = wave == 0 ? 0 : 1, kt = wave == 2 ? 1 : 0;
            f32x4 A = {0.0f, 0.0f, 0.0f, 0.0f};
            O[0] = O[1] = A;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int n0 = 32 * g + 8 * r + 4 * h;
                    const f32x4 q0 = *reinterpret_cast<const f32x4*>(&s.q[l16][n0]);
                    const f32x4 q1 = *reinterpret_cast<const f32x4*>(&s.q[16 + l16][n0]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        O[0] = mfma_f32(S[4 * h + e][r], q0[e], O[0]);
                        O[1] = mfma_f32(S[4 * h + e][r], q1[e], O[1]);
                    }
                    if (wave < 3) { // rows keys, columns queries
                        const f32x4 kk = *reinterpret_cast<const f32x4*>(&s.k[kt * 16 + l16][n0]);
                        const f32x4 qq = qt ? q1 : q0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) A = mfma_f32(kk[e], qq[e], A);
                    }
                }
            if (wave < 3) {
                const int qi = qt * 16 + l16, kj = kt * 16 + 4 * g;
                f32x4 w;
                if (qt == kt) {
                    const f32x4 rj = *reinterpret_cast<const f32x4*>(&d.r[kj]), lj = *reinterpret_cast<const f32x4*>(&d.rlo[kj]);
                    const float ri = d.r[qi], li = d.rlo[qi];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = kj + e <= qi ? A[e] * (a.oscale * __builtin_amdgcn_exp2f((ri - rj[e]) + (li - lj[e]))) : 0.0f;
                } else {
                    w = A * d.row[qi] * *reinterpret_cast<const f32x4*>(&d.col[kj]);
                }
                *reinterpret_cast<f32x4*>(&s.p[qi][kj]) = w;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) O[i] *= d.in[i * 16 + l16];
            __syncthreads(); // the scores are written
        }
        float vf[2][4]; // v of column l16, tokens 16h + 4g .. +3
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) vf[h][e] = s.v[16 * h + 4 * g + e][wave * 16 + l16];
        if constexpr (MODE != PART_STATE) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int h = 0; h <= i; ++h) {
                    const f32x4 p = *reinterpret_cast<const f32x4*>(&s.p[i * 16 + l16][16 * h + 4 * g]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) O[i] = mfma_f32(vf[h][e], p[e], O[i]);
                }
            const uint32_t last = (uint32_t)(end - t0 < kWideChunk ? end - t0 : kWideChunk) - 1;
            const Rsrc bo = wave_rsrc(op + t0 * a.os, last * o_row + cols * SIZE);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if constexpr (DT == DT_FP32) {
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, O[i]), bo, o_off + i * 16 * o_row, 0, 0);
                } else {
                    typedef T t4 __attribute__((ext_vector_type(4)));
                    const t4 w = {(T)O[i].x, (T)O[i].y, (T)O[i].z, (T)O[i].w};
                    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, w), bo, o_off + i * 16 * o_row, 0, 0);
                }
            }
        }
        if (MODE == PART_OUT && !more) break; // the next part has its own state
        if constexpr (MODE != PART_STATE) {
            const float keep = d.keep, change = d.change;
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[t][r] = __builtin_fmaf(S[t][r], change, S[t][r] * keep);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4 od = *reinterpret_cast<const f32x4*>(&d.out[16 * h + 4 * g]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float w = vf[h][e] * od[e];
                const float* kr = &s.k[16 * h + 4 * g + e][8 * l16];
                const f32x4 k0 = *reinterpret_cast<const f32x4*>(kr), k1 = *reinterpret_cast<const f32x4*>(kr + 4);
#pragma unroll
                for (int t = 0; t < 8; ++t) S[t] = mfma_f32(t < 4 ? k0[t & 3] : k1[t & 3], w, S[t]);
            }
        }
        if (more) decays(buf ^ 1);
    }
    if constexpr (MODE == PART_STATE) { // the part's decay, which wave 3 has
        if (wave == 3 && lane == 0) {
            part_decay = decay_of(after);
            if (p0 == 0) c.part_decay[(int64_t)work.item * a.H + head] = part_decay;
        }
        __syncthreads();
    }
    if (have && MODE != PART_OUT) {
        f32x4 x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[u][e] = S[u % 2 * 4 + e][u / 2];
        const Tile tile = tile_of(c, work, head, col0 + wave * 16, lane);
        if constexpr (MODE == WHOLE) store_tile(tile.rows, 4, x);
        else leave_part(c, work, tile, part_decay, x);
    }
}

// The states before each part, from the parts' own, and the state after the last: a thread has
// four entries of one (sequence, head).
__global__ __launch_bounds__(256) void k_linattn_join(ChunkArgs c, int64_t units)
{
    const LinArgs& a = c.a;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= units) return;
    const int64_t per_seq = (int64_t)a.H * a.P * 32;
    const int seq = (int)(i / per_seq);
    const int64_t e = i % per_seq;
    const int head = (int)(e / ((int64_t)a.P * 32));
    const SeqSpan span = seq_span(a, seq);
    const bool fresh = a.fresh && a.fresh[seq];
    if (span.slot < 0 || (span.begin == span.end && !fresh)) return;
    // the parts' order within a tile of 16 columns: n-tile, then lane
    const int lane = e & 63, t = e >> 6 & 7;
    const int64_t row = (e >> 9) * 16 + (lane & 15);
    f32x4* state = reinterpret_cast<f32x4*>(seq_rows(a, seq, span.slot) + row * 128 + 32 * (lane >> 4) + 4 * t);
    f32x4 S = {0.0f, 0.0f, 0.0f, 0.0f};
    if (!fresh) S = *state;
    const int64_t n = (span.end - span.begin + c.part_tokens - 1) / c.part_tokens;
    const int64_t p0 = first_part(c, span.begin, seq);
    f32x4* part = reinterpret_cast<f32x4*>(c.part_state) + p0 * per_seq + e;
    const float2* decay = c.part_decay + p0 * a.H + head;
    constexpr int AHEAD = 8; // parts in flight
    for (int64_t p = 0; p < n; p += AHEAD) {
        f32x4 own[AHEAD];
        float2 d[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (p + k < n) {
                own[k] = part[(p + k) * per_seq];
                d[k] = decay[(p + k) * a.H];
            }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (p + k < n) {
                part[(p + k) * per_seq] = S;
#pragma unroll
                for (int r = 0; r < 4; ++r) S[r] = __builtin_fmaf(S[r], d[k].y, S[r] * d[k].x) + own[k][r];
            }
    }
    *state = S;
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------
struct ChunkPlan {
    int blocks;      // of 64 columns of a head
    int part_tokens; // 0: sequences are not split
    int64_t nparts;
    bool fold;       // the parts' outputs join the states
};

// Sequences are split where they and the blocks do not give every compute unit a workgroup (24
// ragged bf16 prompts of 32 heads, as 384 workgroups of twice the columns and with scores in one
// term: 99 us whole and 162 us split), into as many parts as there can be workgroups at once (three
// prompts of 32 heads of 128, bf16: 75 us for three workgroups a unit, 82 us for two; 16000 tokens of
// 24 heads 88 and 99), of three chunks at least (2048 tokens of 24 heads: 33.4 us, 34.6 in parts of
// two, 31.5 of four; 512 tokens 20.3, 25.5 of four).
// Few parts are joined by those who need them, each from the parts before it, more by a launch of
// its own: 512 tokens of 24 heads 20.3 us against 25.5, three prompts of 32 heads of 128 75 against
// 85; but 16000 tokens, 32 parts, 112 against 88.  Only the sum of the parts is known here: where
// four sequences or more share it, 32 are few (five fp32 prompts, 21 parts, 52.7 us against 56.9),
// unless one of them has nearly all (16000 tokens beside three of one: 115 us).
static ChunkPlan chunk_plan(int dtype, int nseq, int64_t tokens, int H, int P, int num_cus)
{
    ChunkPlan p;
    const int chunk = dtype == DT_BF16 ? kChunk : kWideChunk;
    p.blocks = H * ((P + kCols - 1) / kCols);
    p.part_tokens = 0;
    p.nparts = 0;
    p.fold = false;
    const int64_t chunks = (tokens + chunk - 1) / chunk;
    const int64_t slots = (dtype == DT_BF16 ? 3 : 2) * (int64_t)num_cus; // workgroups at once
    if (nseq > 0 && chunks > 2 && nseq * (int64_t)p.blocks < num_cus) {
        int64_t per = (chunks * p.blocks + slots - 1) / slots;
        if (per < 3) per = 3;
        p.part_tokens = (int)(per * chunk);
        p.nparts = tokens / p.part_tokens + nseq;
        p.fold = (tokens + p.part_tokens - 1) / p.part_tokens <= (nseq < 4 ? 16 : 32);
    }
    return p;
}

static size_t align256(size_t n) { return (n + 255) / 256 * 256; }

static int64_t part_places(const ChunkPlan& p, int nseq) { return p.nparts + (p.fold ? nseq : 0); }

static size_t parts_bytes(const ChunkPlan& p, int nseq, int H, int P)
{
    return (size_t)part_places(p, nseq) * H * P * 512 + align256((size_t)p.nparts * H * sizeof(float2));
}

size_t linattn_workspace(int fmt, int nseq, int64_t tokens, int H, int P, int num_cus)
{
    size_t parts = 0; // of the type that takes most
    for (int dtype : {DT_FP32, DT_BF16, DT_FP16}) {
        const size_t n = parts_bytes(chunk_plan(dtype, nseq, tokens, H, P, num_cus), nseq, H, P);
        if (n > parts) parts = n;
    }
    return (fmt == FP32 ? 0 : (size_t)nseq * H * P * 512) + parts;
}

template <int MODE>
static hipError_t launch_chunk(int dtype, ChunkArgs c, int64_t items, int num_cus, hipStream_t st)
{
    const LinArgs& a = c.a;
    // all the blocks of a key head, fewer where that would leave XCDs without work
    const int share = c.blocks / a.G;
    int cut = (int)((32 + items * a.G - 1) / (items * a.G));
    if (cut > share) cut = share;
    c.items = (int)items;
    c.run = (share + cut - 1) / cut;
    c.runs = (c.blocks + c.run - 1) / c.run;
    c.bins = 0;
    if (MODE == WHOLE && a.nseq > 1 && a.nseq <= 64) c.bins = 8 * (num_cus / 8 > c.run ? num_cus / 8 / c.run : 1);
    const int64_t blocks = (items * c.runs + 7) / 8 * 8 * c.run;
    const dim3 grid((unsigned)blocks), wg(256);
    if (dtype == DT_FP32) {
        hipLaunchKernelGGL((k_linattn_wide<MODE, DT_FP32>), grid, wg, 0, st, c);
    } else if (dtype == DT_FP16) {
        hipLaunchKernelGGL((k_linattn_wide<MODE, DT_FP16>), grid, wg, 0, st, c);
    } else {
        hipLaunchKernelGGL(k_linattn_chunk<MODE>, grid, wg, 0, st, c);
    }
    return hipGetLastError();
}

static hipError_t launch_chunks(int dtype, const LinArgs& a, void* ws, int num_cus, hipStream_t st)
{
    const ChunkPlan p = chunk_plan(dtype, a.nseq, a.tokens, a.H, a.P, num_cus);
    ChunkArgs c{};
    c.a = a;
    c.blocks = p.blocks;
    if (p.part_tokens == 0) return launch_chunk<WHOLE>(dtype, c, a.nseq, num_cus, st);
    c.part_tokens = p.part_tokens;
    c.part_state = static_cast<float*>(ws);
    c.part_decay = reinterpret_cast<float2*>(c.part_state + part_places(p, a.nseq) * a.H * a.P * 128);
    c.parts = p.nparts;
    c.fold = p.fold;
    hipError_t e = launch_chunk<PART_STATE>(dtype, c, p.nparts, num_cus, st);
    if (e != hipSuccess) return e;
    if (!p.fold) {
        const int64_t units = (int64_t)a.nseq * a.H * a.P * 32, blocks = (units + 255) / 256;
        hipLaunchKernelGGL(k_linattn_join, dim3((unsigned)blocks), dim3(256), 0, st, c, units);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return launch_chunk<PART_OUT>(dtype, c, p.nparts, num_cus, st);
}

template <int F>
static hipError_t launch_state_rows(const LinArgs& a, bool store, hipStream_t st)
{
    constexpr int RPW = Traits<F>::bits == 8 ? 8 : 16;
    const int64_t units = (int64_t)a.nseq * a.H * a.P / RPW, blocks = (units + 3) / 4;
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
    LinArgs a = args;
    if (fmt == FP32) {
        a.codes = nullptr;
    } else {
        a.h32 = static_cast<float*>(ws);
        ws = a.h32 + (int64_t)a.nseq * a.H * a.P * 128;
    }
    hipError_t e = state_rows(fmt, a, false, st);
    if (e != hipSuccess) return e;
    e = launch_chunks(dtype, a, ws, num_cus, st);
    if (e != hipSuccess) return e;
    return state_rows(fmt, a, true, st);
}

} // namespace ssq
