// ssq_beam.hip -- beam search's selection: the best `nselect` of beams x vocabulary by
// score + log softmax, gfx950.
//
//   score(beam, token) = s_beam + (x - m) - log(sum exp(x - m)),  m = max x of the beam
//
// Within a beam the order of scores is the order of the logits, so a beam's candidates are
// its largest logits and the softmax only places beams against each other.  One pass over the
// logits therefore finds both: each workgroup reads one share of a beam's row and leaves the
// share's (m, sum) and its best `nselect` (logit, token) pairs; a second, small kernel joins
// the shares of each beam and then the beams of each request.
//
// Selection works on unique 64-bit keys, the logit's order-preserving bits above the inverted
// token index, so that a larger key is a larger logit or, of equal ones, the lower token; the
// result is a set, independent of the order in which lanes append to it.  A wave holds its
// share of a tile in registers, ranks its lanes' largest keys, and takes the nselect-th of
// those as a threshold: at least nselect elements reach it, and only elements of the nselect
// best lanes can, which bounds the list whatever the values are.
#include "ssq_ops_device.h"

namespace ssq {

constexpr int kBeamMaxShares = 16; // workgroups per row at most
constexpr int kBeamNarrow = 32;    // up to this many candidates a lane holds 32 elements, above 16: the same LDS

// elements a lane holds at once
constexpr int beam_lane_elems(int nselect) { return nselect <= kBeamNarrow ? 32 : 16; }

struct BeamShare {
    float m;   // largest logit, -inf if there is none
    float sum; // sum exp(x - m)
};

// floats in ascending order of an unsigned integer; -0 counts as +0
__device__ __forceinline__ uint32_t order_bits(float x)
{
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t o)
{
    return __uint_as_float((o >> 31) ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ uint64_t beam_key(float x, uint32_t token)
{
    return ((uint64_t)order_bits(x) << 32) | (uint32_t)~token;
}

__device__ __forceinline__ uint64_t shfl_u64(uint64_t v, int lane)
{
    const uint32_t lo = __builtin_amdgcn_ds_bpermute(lane << 2, (int)(uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_ds_bpermute(lane << 2, (int)(uint32_t)(v >> 32));
    return ((uint64_t)hi << 32) | lo;
}

__device__ __forceinline__ float wave_max(float v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}
__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// the n-th largest of the wave's unique keys (0: an absent one); 0 if fewer are present
__device__ __forceinline__ uint64_t wave_nth(uint64_t key, int n)
{
    int rank = 0;
#pragma unroll 8
    for (int i = 0; i < 64; ++i) {
        const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)key, i);
        const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(key >> 32), i);
        rank += (((uint64_t)hi << 32) | lo) > key;
    }
    const uint64_t at = __ballot(key != 0 && rank == n - 1);
    return at ? shfl_u64(key, __builtin_ctzll(at)) : 0;
}

// ---------------------------------------------------------------------------
// one share of one beam's row
// ---------------------------------------------------------------------------
template <int DT, int VPL>
__global__ __launch_bounds__(256) void k_beam_rows(BeamArgs a, BeamShare* shares, uint64_t* best, int nshares)
{
    constexpr int VE = DT == DT_FP32 ? 4 : 8; // elements in 16 bytes
    constexpr int NV = VPL / VE;
    constexpr int TILE = 256 * VPL;           // elements of a workgroup's tile
    extern __shared__ uint64_t lds[];         // two lists of nselect, then 4 * VPL * nselect new keys
    __shared__ int count;
    __shared__ uint64_t wave_thr[4];
    __shared__ BeamShare wave_share[4];
    const int n = a.nselect;
    uint64_t* kept = lds;
    uint64_t* next = lds + n;
    uint64_t* fresh = lds + 2 * n;
    const int row = blockIdx.x / nshares, share = blockIdx.x % nshares;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    BeamShare* out = shares + (int64_t)row * nshares + share;
    uint64_t* out_best = best + ((int64_t)row * nshares + share) * n;
    // a beam without candidates of its own, dead or finished: its share is not read
    if ((a.finished && a.finished[row]) || !(a.scores[row] > -INFINITY)) return;
    using T = typename Elem<DT>::T;
    const T* x = static_cast<const T*>(a.logits) + (int64_t)row * a.row_stride;
    // 16-byte pieces from the row's first aligned address down: `off` elements of piece 0 lie before the row
    const int off = (int)(((uintptr_t)x & 15) / sizeof(T));
    const int64_t pieces = ((int64_t)a.vocab + off + VE - 1) / VE;
    const int64_t tiles = (pieces + TILE / VE - 1) / (TILE / VE);

    float m = -INFINITY, s = 0.0f; // of this lane's elements, m of its wave's
    int nkept = 0;
    for (int64_t t = share; t < tiles; t += nshares) {
        float v[VPL];
        const int64_t p0 = t * (TILE / VE) + wave * (64 * NV) + lane;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t e0 = (p0 + i * 64) * VE - off; // the piece's first element
            if (e0 >= 0 && e0 + VE <= a.vocab) {
                load_elems<DT, VE>(x + e0, v + i * VE);
            } else {
#pragma unroll
                for (int j = 0; j < VE; ++j)
                    v[i * VE + j] = e0 + j >= 0 && e0 + j < a.vocab ? (float)x[e0 + j] : -INFINITY;
            }
        }
        float lm = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            v[i] = fmaxf(v[i], -INFINITY); // a NaN is no candidate
            lm = fmaxf(lm, v[i]);
        }
        const float wm = fmaxf(m, wave_max(lm));
        if (wm > -INFINITY) {
            float part = 0.0f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) part += __expf(v[i] - wm);
            s = s * (m > -INFINITY ? __expf(m - wm) : 0.0f) + part;
            m = wm;
        }
        // the lane's largest key: its first element with the largest logit
        int first = 0;
#pragma unroll
        for (int i = VPL - 1; i >= 0; --i) first = v[i] == lm ? i : first;
        const int64_t fe = (p0 + (first / VE) * 64) * VE - off + first % VE;
        const uint64_t mine = lm > -INFINITY ? beam_key(lm, (uint32_t)fe) : 0;
        const uint64_t nth = wave_nth(mine, n);
        if (lane == 0) wave_thr[wave] = nth;
        if (tid == 0) count = 0;
        for (int i = tid; i < n; i += 256) next[i] = 0;
        __syncthreads();
        // any wave's n-th key is a threshold for all, and so is the n-th of the tiles before
        uint64_t low = nkept == n ? kept[n - 1] : 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) low = wave_thr[i] > low ? wave_thr[i] : low;
        const uint32_t low_hi = (uint32_t)(low >> 32);
        if (mine >= low) { // only these lanes, n of a wave at most, hold keys that reach it
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                if (v[i] > -INFINITY && order_bits(v[i]) >= low_hi) {
                    const uint64_t key = beam_key(v[i], (uint32_t)((p0 + (i / VE) * 64) * VE - off + i % VE));
                    if (key >= low) fresh[atomicAdd(&count, 1)] = key;
                }
            }
        }
        __syncthreads();
        const int c = count; // at most 4 * n * VPL
        for (int i = tid; i < nkept + c; i += 256) {
            const uint64_t key = i < nkept ? kept[i] : fresh[i - nkept];
            int rank = 0;
            for (int j = 0; j < nkept; ++j) rank += kept[j] > key;
            for (int j = 0; j < c; ++j) rank += fresh[j] > key;
            if (rank < n) next[rank] = key;
        }
        nkept = min(n, nkept + c);
        uint64_t* const swap = kept;
        kept = next;
        next = swap;
        __syncthreads(); // the lists are written, and the counter and thresholds have been read
    }
    s = wave_sum(s);
    if (lane == 0) wave_share[wave] = {m, s};
    __syncthreads();
    if (tid == 0) {
        float M = -INFINITY, sum = 0.0f;
        for (int i = 0; i < 4; ++i) M = fmaxf(M, wave_share[i].m);
        for (int i = 0; i < 4; ++i)
            if (wave_share[i].m > -INFINITY) sum += wave_share[i].sum * __expf(wave_share[i].m - M);
        *out = {M, sum};
    }
    for (int i = tid; i < n; i += 256) out_best[i] = i < nkept ? kept[i] : 0;
}

// ---------------------------------------------------------------------------
// the shares of each beam, then the beams of each request
// ---------------------------------------------------------------------------
struct BeamCand {
    double score;
    uint32_t beam, token;
};

__global__ __launch_bounds__(256) void k_beam_join(BeamArgs a, const BeamShare* shares, const uint64_t* best, int nshares)
{
    // LDS: a work list of each wave, the best [n], the beams' lists [beams][n]: scores, tokens
    extern __shared__ uint64_t lds[];
    __shared__ int counts[kMaxBeams];
    const int n = a.nselect, beams = a.beams;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint64_t* work = lds + wave * (kBeamMaxShares * n);
    BeamCand* top = reinterpret_cast<BeamCand*>(lds + 4 * kBeamMaxShares * n);
    double* cand = reinterpret_cast<double*>(top + n);
    uint32_t* tokens = reinterpret_cast<uint32_t*>(cand + beams * n);
    const int64_t request = blockIdx.x;

    for (int b = wave; b < beams; b += 4) {
        const int64_t row = request * beams + b;
        const float score = a.scores[row];
        if (!(score > -INFINITY)) {
            if (lane == 0) counts[b] = 0;
            continue;
        }
        if (a.finished && a.finished[row]) {
            if (lane == 0) {
                counts[b] = 1;
                cand[b * n] = (double)score;
                tokens[b * n] = (uint32_t)a.pad;
            }
            continue;
        }
        BeamShare sh = {-INFINITY, 0.0f};
        if (lane < nshares) sh = shares[row * nshares + lane];
        const float M = wave_max(sh.m);
        if (!(M > -INFINITY)) {
            if (lane == 0) counts[b] = 0;
            continue;
        }
        double sum = sh.m > -INFINITY ? (double)sh.sum * exp((double)sh.m - (double)M) : 0.0;
#pragma unroll
        for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
        const double logz = log(sum);

        const int total = nshares * n; // at most 16 for each lane
        const uint64_t* keys = best + row * total;
        uint64_t k[kBeamMaxShares], mine = 0;
#pragma unroll
        for (int i = 0; i < kBeamMaxShares; ++i) {
            k[i] = lane + 64 * i < total ? keys[lane + 64 * i] : 0;
            mine = k[i] > mine ? k[i] : mine;
        }
        const uint64_t nth = wave_nth(mine, n);
        const uint64_t low = nth ? nth : 1;
        int c = 0;
#pragma unroll
        for (int i = 0; i < kBeamMaxShares; ++i) {
            const uint64_t have = __ballot(k[i] >= low);
            if (k[i] >= low) work[c + __popcll(have & ((1ull << lane) - 1))] = k[i];
            c += __popcll(have);
        }
        wave_lds_sync();
        for (int i = lane; i < c; i += 64) {
            const uint64_t key = work[i];
            int rank = 0;
            for (int j = 0; j < c; ++j) rank += work[j] > key;
            if (rank < n) {
                const double x = (double)order_value((uint32_t)(key >> 32));
                cand[b * n + rank] = (double)score + ((x - (double)M) - logz);
                tokens[b * n + rank] = ~(uint32_t)key;
            }
        }
        if (lane == 0) counts[b] = min(c, n);
        wave_lds_sync(); // the list is read before the next beam's is written
    }
    __syncthreads();
    // A candidate's rank: its place in its own beam's list, and the candidates before it in the
    // others', which are sorted: found by halving.  Of equal scores the lower beam is first.
    int found = 0;
    for (int b = 0; b < beams; ++b) found += counts[b];
    for (int i = tid; i < beams * n; i += 256) {
        const int b = i / n, r = i % n;
        if (r >= counts[b]) continue;
        const double me = cand[i];
        int rank = r;
        for (int o = 0; o < beams && rank < n; ++o) {
            if (o == b) continue;
            int lo = 0, hi = counts[o];
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                const double other = cand[o * n + mid];
                if (other > me || (other == me && o < b)) lo = mid + 1;
                else hi = mid;
            }
            rank += lo;
        }
        if (rank < n) top[rank] = {me, (uint32_t)b, tokens[i]};
    }
    __syncthreads();
    for (int j = tid; j < n; j += 256) {
        const bool have = j < found;
        const int64_t at = request * n + j;
        a.out_scores[at] = have ? (float)top[j].score : -INFINITY;
        a.out_tokens[at] = have ? (int32_t)top[j].token : -1;
        a.out_parents[at] = have ? (int32_t)top[j].beam : j % beams;
    }
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------
static int beam_shares(int vocab, int nselect)
{
    // one tile for a workgroup, and no more shares than the join takes
    const int tile = 256 * beam_lane_elems(nselect);
    const int64_t tiles = ((int64_t)vocab + 7 + tile - 1) / tile;
    return tiles < kBeamMaxShares ? (int)tiles : kBeamMaxShares;
}

size_t beam_workspace(int dtype, int batch, int beams, int vocab, int nselect)
{
    (void)dtype;
    const size_t shares = (size_t)batch * beams * beam_shares(vocab, nselect);
    return (shares * sizeof(BeamShare) + 255) / 256 * 256 + shares * nselect * sizeof(uint64_t);
}

template <int DT, int VPL>
static hipError_t launch_rows_of(const BeamArgs& a, BeamShare* shares, uint64_t* best, int nshares, hipStream_t st)
{
    const int64_t blocks = (int64_t)a.batch * a.beams * nshares;
    if (blocks > kMaxBlocks) return hipErrorInvalidValue;
    const size_t lds = (size_t)(2 + 4 * VPL) * a.nselect * sizeof(uint64_t);
    hipLaunchKernelGGL((k_beam_rows<DT, VPL>), dim3((unsigned)blocks), dim3(256), lds, st, a, shares, best, nshares);
    return hipGetLastError();
}

template <int DT>
static hipError_t launch_beam_dt(const BeamArgs& a, hipStream_t st)
{
    const int nshares = beam_shares(a.vocab, a.nselect);
    const size_t rows = (size_t)a.batch * a.beams * nshares;
    BeamShare* shares = static_cast<BeamShare*>(a.ws);
    uint64_t* best = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(a.ws) + (rows * sizeof(BeamShare) + 255) / 256 * 256);
    hipError_t e = a.nselect <= kBeamNarrow ? launch_rows_of<DT, beam_lane_elems(1)>(a, shares, best, nshares, st)
                                            : launch_rows_of<DT, beam_lane_elems(2 * kMaxBeams)>(a, shares, best, nshares, st);
    if (e != hipSuccess) return e;
    // at most 32 KiB of work lists and 25 KiB of candidates
    const size_t lds = 4 * (size_t)kBeamMaxShares * a.nselect * sizeof(uint64_t) +
                       (size_t)a.nselect * (sizeof(BeamCand) + a.beams * (sizeof(double) + sizeof(uint32_t)));
    hipLaunchKernelGGL(k_beam_join, dim3((unsigned)a.batch), dim3(256), lds, st, a, shares, best, nshares);
    return hipGetLastError();
}

hipError_t launch_beam_select(int dtype, const BeamArgs& a, hipStream_t st)
{
    switch (dtype) {
    case DT_FP32: return launch_beam_dt<DT_FP32>(a, st);
    case DT_BF16: return launch_beam_dt<DT_BF16>(a, st);
    case DT_FP16: return launch_beam_dt<DT_FP16>(a, st);
    }
    return hipErrorInvalidValue;
}

} // namespace ssq
