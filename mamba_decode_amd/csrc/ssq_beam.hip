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
// result is a set, independent of the order in which lanes append to it.  A wave runs over tiles
// of its row with the best nselect keys so far in LDS, and looks further at a tile only where a
// lane's maximum passes the last of them.  The elements that do, or in a first tile those that
// reach the nselect-th largest of the lanes' maxima (found to a few thousandths of their range by
// halving: any value that nselect lanes reach serves), go into a short list; the list and the
// kept keys are ranked together.  Where the list runs over (rows in order, or many equal logits),
// the tile is taken in pieces of 16 elements a lane with an exact threshold, which bounds the list
// whatever the values are.
#include "ssq_ops_device.h"

namespace ssq {

constexpr int kBeamMaxShares = 16; // workgroups per row at most
constexpr int kBeamLane = 32; // elements a lane holds at once
constexpr int kBeamPiece = 16;

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

// the n-th largest of the wave's unique keys (0: an absent one); 0 if fewer are present.
// `room`: 64 keys of LDS of the wave's own.
__device__ __forceinline__ uint64_t wave_nth(uint64_t key, int n, uint64_t* room)
{
    const int lane = threadIdx.x & 63;
    room[lane] = key;
    wave_lds_sync();
    int rank = 0;
    const ulonglong2* all = reinterpret_cast<const ulonglong2*>(room);
#pragma unroll 8
    for (int i = 0; i < 32; ++i) {
        const ulonglong2 two = all[i];
        rank += (two.x > key) + (two.y > key);
    }
    wave_lds_sync();
    const uint64_t at = __ballot(key != 0 && rank == n - 1);
    return at ? shfl_u64(key, __builtin_ctzll(at)) : 0;
}

// keys larger than `key` among list[0 .. count)
__device__ __forceinline__ int keys_above(const uint64_t* list, int count, uint64_t key)
{
    int above = 0;
    for (int j = 0; j < count; ++j) above += list[j] > key;
    return above;
}

// ---------------------------------------------------------------------------
// one share of one beam's row
// ---------------------------------------------------------------------------
// LDS of a wave: two lists of n, then the new keys: n of a piece's lanes may have them all, and
// wave_nth takes 64
__host__ __device__ constexpr int beam_list_keys(int n) { return kBeamPiece * n > 64 ? kBeamPiece * n : 64; }
__host__ __device__ constexpr int beam_wave_keys(int n) { return 2 * n + beam_list_keys(n); }

// A value that at least n of the lanes' values reach, close below the n-th largest.
__device__ __forceinline__ float wave_threshold(float v, int n)
{
    const uint32_t o = order_bits(v);
    const uint32_t top = order_bits(group_max<16>(v)), bottom = order_bits(group_min<16>(v));
    uint32_t hi = 0, lo = 0xFFFFFFFFu;
#pragma unroll
    for (int r = 0; r < 64; r += 16) {
        const uint32_t t = __builtin_amdgcn_readlane((int)top, r), b = __builtin_amdgcn_readlane((int)bottom, r);
        hi = t > hi ? t : hi;
        lo = b < lo ? b : lo;
    }
    for (int i = 0; i < 14 && lo < hi; ++i) {
        const uint32_t mid = lo + (hi - lo) / 2 + 1;
        if (__popcll(__ballot(o >= mid)) >= n) lo = mid;
        else hi = mid - 1;
    }
    return order_value(lo);
}

template <int DT>
__global__ __launch_bounds__(256) void k_beam_rows(BeamArgs a, BeamShare* shares, uint64_t* best, int nshares)
{
    constexpr int VPL = kBeamLane;
    constexpr int VE = DT == DT_FP32 ? 4 : 8; // elements in 16 bytes
    constexpr int NV = VPL / VE;
    constexpr int TILE = 64 * VPL;            // elements of a wave's tile
    extern __shared__ __align__(16) uint64_t lds[];
    __shared__ BeamShare wave_share[4];
    __shared__ int wave_kept[4];
    const int n = a.nselect;
    const int row = blockIdx.x / nshares, share = blockIdx.x % nshares;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // a beam without candidates of its own, dead or finished: its share is not read
    if ((a.finished && a.finished[row]) || !(a.scores[row] > -INFINITY)) return;
    uint64_t* const mine = lds + wave * beam_wave_keys(n);
    uint64_t* kept = mine;
    uint64_t* next = mine + n;
    uint64_t* const fresh = mine + 2 * n;
    using T = typename Elem<DT>::T;
    const T* x = static_cast<const T*>(a.logits) + (int64_t)row * a.row_stride;
    // 16-byte pieces from the row's first aligned address down: `off` elements of piece 0 lie before the row
    const int off = (int)(((uintptr_t)x & 15) / sizeof(T));
    const int64_t pieces = ((int64_t)a.vocab + off + VE - 1) / VE;
    const int64_t tiles = (pieces + TILE / VE - 1) / (TILE / VE);

    float m = -INFINITY, s = 0.0f; // of this lane's elements
    int nkept = 0;
    float last = -INFINITY;        // the n-th best so far; -inf while there are fewer
    auto merge = [&](int c) { // the new keys and the kept ones: the best n are kept
        wave_lds_sync();
        for (int i = lane; i < nkept + c; i += 64) {
            const uint64_t key = i < nkept ? kept[i] : fresh[i - nkept];
            const int rank = keys_above(kept, nkept, key) + keys_above(fresh, c, key);
            if (rank < n) next[rank] = key;
        }
        wave_lds_sync();
        nkept = min(n, nkept + c);
        uint64_t* const swap = kept;
        kept = next;
        next = swap;
        if (nkept == n) last = order_value((uint32_t)(kept[n - 1] >> 32));
    };
    for (int64_t t = share * 4 + wave; t < tiles; t += 4 * nshares) {
        float v[VPL];
        const int64_t p0 = t * (TILE / VE) + lane;
        auto token = [&](int i) { return (uint32_t)((p0 + (i / VE) * 64) * VE - off + i % VE); };
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
        const float wm = fmaxf(m, lm), shift = wm > -INFINITY ? wm : 0.0f; // exp(-inf - 0) is 0
        float part = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) part += __expf(v[i] - shift);
        s = s * __expf(m - shift) + part;
        m = wm;
        // tiles come in the order of their tokens: an element equal to the last kept one comes behind it
        if (!__ballot(lm > last)) continue;
        const int room = beam_list_keys(n);
        const float reach = nkept == n ? order_value(order_bits(last) + 1) : wave_threshold(lm, n);
        const float low_value = fmaxf(reach, -3.4028234663852886e38f); // -inf is no candidate
        int c = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const bool take = v[i] >= low_value;
            const uint64_t who = __ballot(take);
            if (who) {
                const int at = c + __popcll(who & ((1ull << lane) - 1));
                if (take && at < room) fresh[at] = beam_key(v[i], token(i));
                c += __popcll(who);
            }
        }
        if (c <= room) {
            merge(c);
            continue;
        }
#pragma unroll
        for (int i0 = 0; i0 < VPL; i0 += kBeamPiece) {
            // the lane's largest key: its first element with the largest logit
            float pm = -INFINITY;
            uint32_t first = 0;
#pragma unroll
            for (int i = i0 + kBeamPiece - 1; i >= i0; --i) {
                first = v[i] >= pm ? token(i) : first;
                pm = fmaxf(pm, v[i]);
            }
            const uint64_t top = pm > -INFINITY ? beam_key(pm, first) : 0;
            const uint64_t nth = wave_nth(top, n, fresh), floor = nkept == n ? kept[n - 1] : 1;
            const uint64_t low = nth > floor ? nth : floor;
            c = 0;
#pragma unroll
            for (int i = i0; i < i0 + kBeamPiece; ++i) { // of n lanes at most
                const uint64_t key = v[i] > -INFINITY ? beam_key(v[i], token(i)) : 0;
                const uint64_t who = __ballot(key >= low);
                if (key >= low) fresh[c + __popcll(who & ((1ull << lane) - 1))] = key;
                c += __popcll(who);
            }
            merge(c);
        }
    }
    // the four waves' lists, each copied to its place at the front of the wave's LDS
    const float wm = wave_max(m);
    s = wave_sum(m > -INFINITY ? s * __expf(m - wm) : 0.0f);
    if (kept != mine) {
        for (int i = lane; i < nkept; i += 64) mine[i] = kept[i];
    }
    if (lane == 0) {
        wave_share[wave] = {wm, s};
        wave_kept[wave] = nkept;
    }
    __syncthreads();
    uint64_t* out_best = best + ((int64_t)row * nshares + share) * n;
    int found = 0;
    for (int w = 0; w < 4; ++w) found += wave_kept[w];
    for (int i = tid; i < 4 * n; i += 256) {
        const int w = i / n, r = i % n;
        if (r >= wave_kept[w]) continue;
        const uint64_t key = lds[w * beam_wave_keys(n) + r];
        int rank = r;
        for (int o = 0; o < 4; ++o)
            if (o != w) rank += keys_above(lds + o * beam_wave_keys(n), wave_kept[o], key);
        if (rank < n) out_best[rank] = key;
    }
    for (int i = found + tid; i < n; i += 256) out_best[i] = 0;
    if (tid == 0) {
        float M = -INFINITY, sum = 0.0f;
        for (int i = 0; i < 4; ++i) M = fmaxf(M, wave_share[i].m);
        for (int i = 0; i < 4; ++i)
            if (wave_share[i].m > -INFINITY) sum += wave_share[i].sum * __expf(wave_share[i].m - M);
        shares[(int64_t)row * nshares + share] = {M, sum};
    }
}

// ---------------------------------------------------------------------------
// the shares of each beam, then the beams of each request
// ---------------------------------------------------------------------------
// a wave's work list: the keys of all shares, and at least the 64 of wave_nth
__host__ __device__ constexpr int beam_join_keys(int nshares, int n) { return nshares * n > 64 ? nshares * n : 64; }

struct BeamCand {
    double score;
    uint32_t beam, token;
};

// a wave for each beam, up to 16
__global__ __launch_bounds__(1024) void k_beam_join(BeamArgs a, const BeamShare* shares, const uint64_t* best, int nshares)
{
    // LDS: a work list of each wave, the best [n], the beams' lists [beams][n]: scores, tokens
    extern __shared__ __align__(16) uint64_t lds[];
    __shared__ int counts[kMaxBeams];
    const int n = a.nselect, beams = a.beams;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int waves = blockDim.x >> 6, room = beam_join_keys(nshares, n);
    uint64_t* work = lds + wave * room;
    BeamCand* top = reinterpret_cast<BeamCand*>(lds + waves * room);
    double* cand = reinterpret_cast<double*>(top + n);
    uint32_t* tokens = reinterpret_cast<uint32_t*>(cand + beams * n);
    const int64_t request = blockIdx.x;

    for (int b = wave; b < beams; b += waves) {
        const int64_t row = request * beams + b;
        const float score = a.scores[row];
        const int total = nshares * n; // at most 16 for each lane
        const uint64_t* keys = best + row * total;
        BeamShare sh = {-INFINITY, 0.0f};
        if (lane < nshares) sh = shares[row * nshares + lane];
        uint64_t k[kBeamMaxShares], mine = 0; // of a dead or finished beam never written, and not used
#pragma unroll
        for (int i = 0; i < kBeamMaxShares; ++i) {
            k[i] = lane + 64 * i < total ? keys[lane + 64 * i] : 0;
            mine = k[i] > mine ? k[i] : mine;
        }
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
        const float M = wave_max(sh.m);
        if (!(M > -INFINITY)) {
            if (lane == 0) counts[b] = 0;
            continue;
        }
        const double logz = log((double)wave_sum(sh.m > -INFINITY ? sh.sum * __expf(sh.m - M) : 0.0f));
        const uint64_t nth = wave_nth(mine, n, work);
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
            const int rank = keys_above(work, c, key);
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
    for (int i = tid; i < beams * n; i += blockDim.x) {
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
    for (int j = tid; j < n; j += blockDim.x) {
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
// Workgroups of a row: enough of all rows to fill the card (1024), no more than there are tiles of
// four waves, nor than the join takes.
static int beam_shares(int64_t rows, int vocab)
{
    const int tile = 256 * kBeamLane;
    const int64_t tiles = ((int64_t)vocab + 7 + tile - 1) / tile;
    int64_t shares = (1024 + rows - 1) / (rows > 0 ? rows : 1);
    if (shares > tiles) shares = tiles;
    return (int)(shares < kBeamMaxShares ? shares : kBeamMaxShares);
}

size_t beam_workspace(int batch, int beams, int vocab, int nselect)
{
    const size_t shares = (size_t)batch * beams * beam_shares((int64_t)batch * beams, vocab);
    return (shares * sizeof(BeamShare) + 255) / 256 * 256 + shares * nselect * sizeof(uint64_t);
}

template <int DT>
static hipError_t launch_rows_of(const BeamArgs& a, BeamShare* shares, uint64_t* best, int nshares, hipStream_t st)
{
    const int64_t blocks = (int64_t)a.batch * a.beams * nshares;
    const size_t lds = 4 * (size_t)beam_wave_keys(a.nselect) * sizeof(uint64_t); // 34 KiB at most
    hipLaunchKernelGGL(k_beam_rows<DT>, dim3((unsigned)blocks), dim3(256), lds, st, a, shares, best, nshares);
    return hipGetLastError();
}

template <int DT>
static hipError_t launch_beam_dt(const BeamArgs& a, hipStream_t st)
{
    const int nshares = beam_shares((int64_t)a.batch * a.beams, a.vocab);
    const size_t rows = (size_t)a.batch * a.beams * nshares;
    BeamShare* shares = static_cast<BeamShare*>(a.ws);
    uint64_t* best = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(a.ws) + (rows * sizeof(BeamShare) + 255) / 256 * 256);
    const hipError_t e = launch_rows_of<DT>(a, shares, best, nshares, st);
    if (e != hipSuccess) return e;
    // the waves' lists within 32 KiB, at most 26 KiB of candidates
    const size_t list = (size_t)beam_join_keys(nshares, a.nselect) * sizeof(uint64_t);
    int waves = a.beams < 16 ? a.beams : 16;
    while (waves * list > 32768) --waves;
    const size_t lds = waves * list + (size_t)a.nselect * (sizeof(BeamCand) + a.beams * (sizeof(double) + sizeof(uint32_t)));
    hipLaunchKernelGGL(k_beam_join, dim3((unsigned)a.batch), dim3(64 * waves), lds, st, a, shares, best, nshares);
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
