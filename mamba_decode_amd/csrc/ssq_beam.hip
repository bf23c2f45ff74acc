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
// halving: any value that nselect lanes reach serves), go into a short list, and the list and the
// kept keys together give the kept ones: ranked by counting up to 64 of them, else sorted across
// the lanes and merged, 64 at a time (counting costs their square: 32 x 32 beams of 32000 with
// nselect 64 took 351 us that way, 44 so).  Where the list runs over (rows in order, or many equal logits),
// the tile is taken in pieces of 16 elements a lane with an exact threshold, which bounds the list
// whatever the values are.
//
// What bounds it: 32 x 8 beams of 131071 in fp32 (134 MB) take 27 us, 5.0 TB/s, in the pass and 6
// us in the join; a wave's loads of 2048 elements wait for the tile before (fetched a tile ahead
// they need 32 registers more, three waves a SIMD for four: 40 us in fp32; 3% gained in bf16).
// 4 x 50280 take 6.4 and 4.6 us, mostly the latency of two launches.
#include "ssq.h"
#include "ssq_ops_device.h"

namespace ssq {

constexpr int kBeamMaxShares = 16; // workgroups per row at most
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

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t x)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true);
}
// the value of lane ^ D
template <int D>
__device__ __forceinline__ uint32_t xor_u32(uint32_t x)
{
    if constexpr (D == 1) return dpp_u32<0xB1>(x);
    else if constexpr (D == 2) return dpp_u32<0x4E>(x);
    else if constexpr (D == 3) return dpp_u32<0x1B>(x);
    else if constexpr (D == 4) return dpp_u32<0x141>(dpp_u32<0x1B>(x));
    else if constexpr (D == 7) return dpp_u32<0x141>(x);
    else if constexpr (D == 8) return dpp_u32<0x128>(x);
    else if constexpr (D == 15) return dpp_u32<0x140>(x);
    else if constexpr (D == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false); // rows 0 0 2 2 and 1 1 3 3
        return threadIdx.x & 16 ? r[0] : r[1];
    } else if constexpr (D == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false); // the low half twice, the high half twice
        return threadIdx.x & 32 ? r[0] : r[1];
    } else if constexpr (D == 31) return xor_u32<16>(xor_u32<15>(x));
    else return xor_u32<32>(xor_u32<31>(x));
}

// What is sorted: a key, or a candidate of which one with an equal score comes first by its place.
struct BeamTop {
    uint64_t score; // order bits of the double, 0: none
    uint32_t place; // beam, and rank in the beam's list
};
__device__ __forceinline__ bool before(uint64_t a, uint64_t b) { return a > b; }
__device__ __forceinline__ bool before(BeamTop a, BeamTop b)
{
    return a.score > b.score || (a.score == b.score && a.place < b.place);
}
template <int D>
__device__ __forceinline__ uint64_t other_lane(uint64_t v)
{
    return ((uint64_t)xor_u32<D>((uint32_t)(v >> 32)) << 32) | xor_u32<D>((uint32_t)v);
}
template <int D>
__device__ __forceinline__ BeamTop other_lane(BeamTop v)
{
    return {other_lane<D>(v.score), xor_u32<D>(v.place)};
}

// One step of a sorting network over the wave's lanes: of lane and lane ^ D the one without bit
// UPPER keeps what comes first.
template <int D, int UPPER, typename K>
__device__ __forceinline__ void exchange(K& v)
{
    const K o = other_lane<D>(v);
    if (before(o, v) != ((threadIdx.x & UPPER) != 0)) v = o;
}
// lanes that first rise and then fall, or the other way round, into order
template <int N, typename K>
__device__ __forceinline__ void settle(K& v)
{
    if constexpr (N >= 32) exchange<32, 32>(v);
    if constexpr (N >= 16) exchange<16, 16>(v);
    if constexpr (N >= 8) exchange<8, 8>(v);
    if constexpr (N >= 4) exchange<4, 4>(v);
    if constexpr (N >= 2) exchange<2, 2>(v);
    if constexpr (N >= 1) exchange<1, 1>(v);
}
// the wave's keys in descending order
__device__ __forceinline__ uint64_t wave_sort(uint64_t v)
{
    exchange<1, 1>(v);
    exchange<3, 2>(v);
    settle<1>(v);
    exchange<7, 4>(v);
    settle<2>(v);
    exchange<15, 8>(v);
    settle<4>(v);
    exchange<31, 16>(v);
    settle<8>(v);
    exchange<63, 32>(v);
    settle<16>(v);
    return v;
}
// the 64 first of two lists, one in descending order and one in ascending order, in descending order
template <typename K>
__device__ __forceinline__ K wave_merge(K v, K ascending)
{
    if (before(ascending, v)) v = ascending;
    settle<32>(v);
    return v;
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

// 16 bytes of logits, aligned to their element
template <int DT>
__device__ __forceinline__ void load_piece(const typename Elem<DT>::T* p, float* v)
{
    u32x4 w;
    __builtin_memcpy(&w, p, sizeof(w));
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (DT == DT_FP32) {
            v[j] = __uint_as_float(ws[j]);
        } else {
            v[2 * j] = to_f32<DT>(ws[j] & 0xFFFFu);
            v[2 * j + 1] = to_f32<DT>(ws[j] >> 16);
        }
    }
}

template <int DT, int VPL>
__global__ __launch_bounds__(256) void k_beam_rows(BeamArgs a, BeamShare* shares, uint64_t* best, int nshares)
{
    constexpr int VE = DT == DT_FP32 ? 4 : 8; // elements in 16 bytes
    constexpr int NV = VPL / VE;
    constexpr int TILE = 64 * VPL;            // elements of a wave's tile
    extern __shared__ __align__(16) uint64_t lds[];
    __shared__ BeamShare wave_share[4];
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
    // 16-byte pieces from the row's start, whatever its alignment: rows of equal logits have equal sums
    const int64_t pieces = ((int64_t)a.vocab + VE - 1) / VE;
    const int64_t tiles = (pieces + TILE / VE - 1) / (TILE / VE);

    // of this lane's elements; the sum over tiles is a double: a lane of the longest rows has thousands of
    // them, and one rounding to fp32 after the other, of alike addends, has a drift (2e-5 at 2^28 tokens)
    float m = -INFINITY;
    double s = 0.0;
    int nkept = 0;
    float last = -INFINITY;        // the n-th best so far; -inf while there are fewer
    auto merge = [&](int c) { // the new keys and the kept ones: the best n are kept
        wave_lds_sync();
        if (nkept + c > 64) {
            uint64_t top = lane < nkept ? kept[lane] : 0;
            for (int i = 0; i < c; i += 64) top = wave_merge(top, ~wave_sort(i + lane < c ? ~fresh[i + lane] : ~0ull));
            if (lane < n) kept[lane] = top;
        } else {
            const uint64_t key = lane < nkept ? kept[lane] : lane < nkept + c ? fresh[lane - nkept] : 0;
            const int rank = keys_above(kept, nkept, key) + keys_above(fresh, c, key);
            if (key && rank < n) next[rank] = key;
            uint64_t* const swap = kept;
            kept = next;
            next = swap;
        }
        wave_lds_sync();
        nkept = min(n, nkept + c);
        if (nkept == n) last = order_value((uint32_t)(kept[n - 1] >> 32));
    };
    for (int64_t t = share * 4 + wave; t < tiles; t += 4 * nshares) {
        float v[VPL];
        const int64_t p0 = t * (TILE / VE) + lane;
        auto token = [&](int i) { return (uint32_t)((p0 + (i / VE) * 64) * VE + i % VE); };
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t e0 = (p0 + i * 64) * VE; // the piece's first element
            if (e0 + VE <= a.vocab) {
                load_piece<DT>(x + e0, v + i * VE);
            } else {
#pragma unroll
                for (int j = 0; j < VE; ++j)
                    v[i * VE + j] = e0 + j < a.vocab ? (float)x[e0 + j] : -INFINITY;
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
        s = s * (double)__expf(m - shift) + (double)part;
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
    // the four waves' lists, each at the front of the wave's LDS, 0 behind its last key
    const float wm = wave_max(m);
    const float of_wave = wave_sum(m > -INFINITY ? (float)s * __expf(m - wm) : 0.0f);
    wave_lds_sync();
    uint64_t top = lane < nkept ? kept[lane] : 0;
    wave_lds_sync();
    if (lane < n) mine[lane] = top;
    if (lane == 0) wave_share[wave] = {wm, of_wave};
    __syncthreads();
    if (wave != 0) return;
    for (int w = 1; w < 4; ++w) top = wave_merge(top, 63 - lane < n ? lds[w * beam_wave_keys(n) + 63 - lane] : 0);
    if (lane < n) best[((int64_t)row * nshares + share) * n + lane] = top;
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
// order bits of a double, and the double
__device__ __forceinline__ uint64_t order_bits64(double x)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, x + 0.0);
    return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ double order_value64(uint64_t o)
{
    return __builtin_bit_cast(double, (o >> 63) ? o ^ (1ull << 63) : ~o);
}

// LDS of the join: each wave's list [n], scores and places, and the tokens of all beams [beams][n]
__host__ __device__ constexpr size_t beam_join_lds(int waves, int beams, int n)
{
    return (size_t)waves * n * (sizeof(uint64_t) + sizeof(uint32_t)) + (size_t)beams * n * sizeof(uint32_t);
}

// A workgroup of a request, a wave of a beam (of two from 17 beams up).  A wave joins the lists of
// its beam's shares into the beam's candidates, a lane each, and its beams into one list; then the
// waves' lists are joined in pairs.  Lists of up to 16 are sorted, 64 keys of several shares at a
// time; longer ones are merged one by one (28 steps of a network for 64 keys, or 7 for a share:
// 32 beams of 131071 with nselect 64, 16 shares each, take 21 us, 55 sorted).
__global__ __launch_bounds__(1024) void k_beam_join(BeamArgs a, const BeamShare* shares, const uint64_t* best, int nshares)
{
    extern __shared__ __align__(16) uint64_t lds[];
    const int n = a.nselect, beams = a.beams;
    const int tid = threadIdx.x, lane = tid & 63, waves = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    uint64_t* const scores = lds;
    uint32_t* const places = reinterpret_cast<uint32_t*>(lds + waves * n);
    uint32_t* const tokens = places + waves * n;
    const int64_t request = blockIdx.x;

    BeamTop top = {0, 0};
    for (int b = wave; b < beams; b += waves) {
        const int64_t row = request * beams + b;
        const float score = a.scores[row];
        const bool finished = a.finished && a.finished[row];
        if (!(score > -INFINITY)) continue;
        BeamTop mine = {0, (uint32_t)(b * n + lane)};
        uint32_t token = (uint32_t)a.pad;
        if (finished) {
            if (lane == 0) mine.score = order_bits64((double)score);
        } else {
            const int total = nshares * n;
            const uint64_t* keys = best + row * total;
            BeamShare sh = {-INFINITY, 0.0f};
            if (lane < nshares) sh = shares[row * nshares + lane];
            uint64_t k[kBeamMaxShares];
            uint64_t key;
            if (n > 16) { // each share's list, in order, by itself
#pragma unroll
                for (int i = 0; i < kBeamMaxShares; ++i) {
                    const int r = i == 0 ? lane : 63 - lane; // the first from its front, the others from their ends
                    k[i] = i < nshares && r < n ? keys[i * n + r] : 0;
                }
                key = k[0];
#pragma unroll
                for (int i = 1; i < kBeamMaxShares; ++i)
                    if (i < nshares) key = wave_merge(key, k[i]);
            } else { // 64 keys of several shares at a time, at most four times
#pragma unroll
                for (int i = 0; i < 4; ++i) k[i] = lane + 64 * i < total ? keys[lane + 64 * i] : 0;
                key = wave_sort(k[0]);
#pragma unroll
                for (int i = 1; i < 4; ++i)
                    if (64 * i < total) key = wave_merge(key, ~wave_sort(~k[i]));
            }
            const float M = wave_max(sh.m);
            if (!(M > -INFINITY)) continue;
            const double logz = log((double)wave_sum(sh.m > -INFINITY ? sh.sum * __expf(sh.m - M) : 0.0f));
            if (key && lane < n) {
                const double x = (double)order_value((uint32_t)(key >> 32));
                mine.score = order_bits64((double)score + ((x - (double)M) - logz));
                token = ~(uint32_t)key;
            }
        }
        if (lane < n) tokens[b * n + lane] = token;
        // this list from its end: its places are above those of the wave's beams before it
        const BeamTop end = other_lane<63>(mine);
        top = b == wave ? mine : wave_merge(top, end);
    }
    auto leave = [&]() {
        if (lane < n) {
            scores[wave * n + lane] = top.score;
            places[wave * n + lane] = top.place;
        }
    };
    leave();
    for (int step = 1; step < waves; step *= 2) {
        __syncthreads();
        if (wave % (2 * step) == 0 && wave + step < waves) {
            BeamTop end = {0, 0};
            if (63 - lane < n) end = {scores[(wave + step) * n + 63 - lane], places[(wave + step) * n + 63 - lane]};
            top = wave_merge(top, end);
            leave();
        }
    }
    __syncthreads();
    if (wave == 0 && lane < n) {
        const int64_t at = request * n + lane;
        const bool have = top.score != 0;
        a.out_scores[at] = have ? (float)order_value64(top.score) : -INFINITY;
        a.out_tokens[at] = have ? (int32_t)tokens[top.place] : -1;
        a.out_parents[at] = have ? (int32_t)(top.place / n) : lane % beams;
    }
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------
// Elements a lane holds at once: 32, or 16 where all of the logits are in flight at once that way
// and the card is not full (4 x 50280 bf16: 12.9 us against 13.8; 64 x 50280 fp32 15.9 against 15.1,
// 8 x 131071 bf16 22.7 against 21.5, 256 x 131071 fp32 45 against 40; 64 of them: 15.5 and 48).
// Workgroups of a row: enough of all rows to fill the card (1024: of 256 x 131071 40 us, 48 for
// 512 and 43 for 2048), no more than there are tiles of four waves, nor than the join takes.
struct BeamPlan {
    int lane, shares;
};
static BeamPlan beam_plan(int64_t rows, int vocab)
{
    auto tiles = [&](int lane) { return ((int64_t)vocab + 256 * lane - 1) / (256 * lane); };
    if (tiles(16) <= kBeamMaxShares && rows * tiles(16) <= 512) return {16, (int)tiles(16)};
    int64_t shares = (1024 + rows - 1) / (rows > 0 ? rows : 1);
    if (shares > tiles(32)) shares = tiles(32);
    return {32, (int)(shares < kBeamMaxShares ? shares : kBeamMaxShares)};
}

size_t beam_workspace(int batch, int beams, int vocab, int nselect)
{
    const size_t shares = (size_t)batch * beams * beam_plan((int64_t)batch * beams, vocab).shares;
    return (shares * sizeof(BeamShare) + 255) / 256 * 256 + shares * nselect * sizeof(uint64_t);
}

template <int DT, int VPL>
static hipError_t launch_rows_of(const BeamArgs& a, BeamShare* shares, uint64_t* best, int nshares, hipStream_t st)
{
    const int64_t blocks = (int64_t)a.batch * a.beams * nshares;
    const size_t lds = 4 * (size_t)beam_wave_keys(a.nselect) * sizeof(uint64_t); // 36 KiB at most
    static_assert(4 * beam_wave_keys(2 * SSQ_MAX_BEAMS) * sizeof(uint64_t) == 36 * 1024, "a launch takes up to 64 KiB");
    hipLaunchKernelGGL((k_beam_rows<DT, VPL>), dim3((unsigned)blocks), dim3(256), lds, st, a, shares, best, nshares);
    return hipGetLastError();
}

template <int DT>
static hipError_t launch_beam_dt(const BeamArgs& a, hipStream_t st)
{
    const BeamPlan plan = beam_plan((int64_t)a.batch * a.beams, a.vocab);
    const int nshares = plan.shares;
    const size_t rows = (size_t)a.batch * a.beams * nshares;
    BeamShare* shares = static_cast<BeamShare*>(a.ws);
    uint64_t* best = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(a.ws) + (rows * sizeof(BeamShare) + 255) / 256 * 256);
    const hipError_t e = plan.lane == 16 ? launch_rows_of<DT, 16>(a, shares, best, nshares, st)
                                         : launch_rows_of<DT, 32>(a, shares, best, nshares, st);
    if (e != hipSuccess) return e;
    const int waves = a.beams < 16 ? a.beams : 16;
    const size_t lds = beam_join_lds(waves, a.beams, a.nselect); // 20 KiB at most
    static_assert(beam_join_lds(16, SSQ_MAX_BEAMS, 2 * SSQ_MAX_BEAMS) == 20 * 1024, "a launch takes up to 64 KiB");
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
