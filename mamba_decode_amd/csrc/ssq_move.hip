// ssq_move.hip -- moves between sequences of states, for many arrays in one launch, gfx950.
//
// A thread owns one 16-byte column of an array.  A workgroup looks first whether any move reads or writes what
// another one writes, on a bitmap of the destinations in LDS.  If none does, the moves are dealt to the
// workgroups of a column; else the first of them takes them all in their order, each thread its own column, so
// that a sequence may be the source of one move and the destination of another one.
//
// Bytes bound it.  48 int4 layers (453 MB read and written): 8 sequences forked to 56 places, one source's places next to
// each other in the list, 78-81 us, 5.6-5.8 TB/s (sources in turn 103 us: the list's order is kept), 32 copied to 32 others 69 us,
// 6.6 TB/s, 56 freed 77 us, a chain of 63 one after the other 187 us.  Loads keep their lines for the next workgroup that
// forks the same source (with the non-temporal hint 98, 133 and 84 us), stores have the hint (without it 100 and 95 us).
// Every workgroup goes through the whole list to see whether moves meet, which is what bounds long lists of small sequences: 4000
// moves of 2048 fp32 channels 26 us (bytes 10), 65535 of them 1.1 ms (165 us), 65535 of 64 channels 0.9 ms (5 us).
#include "ssq_ops_device.h"

namespace ssq {

struct MoveArgs {
    uint8_t* dst[kMoveParts];
    const uint8_t* src[kMoveParts];
    uint32_t n16[kMoveParts];   // 16-byte pieces of a sequence
    uint32_t first[kMoveParts]; // the first workgroup of each array
    const int32_t* to;
    const int32_t* from;
    int nparts, nmoves, batch, sources;
    bool inside; // sources and destinations are the same arrays
};
constexpr int kMoveBitmap = 1 << 18; // sequences
constexpr int kMoveWorkgroups = 8192;

struct Move {
    int to, from;
};
// the i-th move, to -1 if it is left out or moves nothing
__device__ __forceinline__ Move move_at(const MoveArgs& a, int i)
{
    Move m{a.to[i], a.from[i]};
    if (m.to < 0 || m.to >= a.batch || m.from < -1 || m.from >= a.sources || (a.inside && m.to == m.from)) m.to = -1;
    return m;
}

// whether a move reads or writes what another one writes; the same in every workgroup
__device__ __forceinline__ bool moves_meet(const MoveArgs& a)
{
    extern __shared__ uint32_t s_written[];
    __shared__ int s_meet;
    for (int i = threadIdx.x; i < (a.batch + 31) / 32; i += 256) s_written[i] = 0;
    if (threadIdx.x == 0) s_meet = 0;
    __syncthreads();
    bool meet = false;
    for (int i = threadIdx.x; i < a.nmoves; i += 256) {
        const Move m = move_at(a, i);
        if (m.to >= 0) meet = meet || (atomicOr(&s_written[m.to >> 5], 1u << (m.to & 31)) >> (m.to & 31) & 1u);
    }
    __syncthreads();
    if (a.inside)
        for (int i = threadIdx.x; i < a.nmoves; i += 256) {
            const Move m = move_at(a, i);
            if (m.to >= 0 && m.from >= 0) meet = meet || (s_written[m.from >> 5] >> (m.from & 31) & 1u);
        }
    if (meet) s_meet = 1;
    __syncthreads();
    return s_meet != 0;
}

__global__ __launch_bounds__(256) void k_move(MoveArgs a)
{
    constexpr int N = 8; // moves under way
    int lo = 0, hi = a.nparts - 1;
    while (lo < hi) { // the last array whose first workgroup is not behind this one
        const int mid = (lo + hi + 1) >> 1;
        if (a.first[mid] <= blockIdx.x) lo = mid;
        else hi = mid - 1;
    }
    const int64_t bytes = (int64_t)a.n16[lo] * 16;
    const bool meet = a.nmoves > 1 && (a.batch > kMoveBitmap || moves_meet(a));
    if (meet && blockIdx.y) return;
    const int64_t col = (int64_t)(blockIdx.x - a.first[lo]) * kColumnBytes + threadIdx.x * 16;
    const bool there = col < bytes;
    const uint8_t* src = a.src[lo] + col;
    uint8_t* dst = a.dst[lo] + col;
    if (meet) {
        if (!there) return;
        for (int i = 0; i < a.nmoves; ++i) {
            const Move m = move_at(a, i);
            if (m.to < 0) continue;
            u32x4 v = {0, 0, 0, 0};
            if (m.from >= 0) v = *reinterpret_cast<const u32x4*>(src + m.from * bytes);
            *reinterpret_cast<u32x4*>(dst + m.to * bytes) = v;
        }
        return;
    }
    // a run of moves for each workgroup of the column, as one sequence is often forked to places next to each other in the list
    const int per = (a.nmoves + gridDim.y - 1) / gridDim.y, first = blockIdx.y * per, end = first + per < a.nmoves ? first + per : a.nmoves;
    const int lane = threadIdx.x & (N - 1);
    for (int at = first; at < end; at += N) {
        const Move m = at + lane < end ? move_at(a, at + lane) : Move{-1, -1}; // a lane each: one wait for all of them
        u32x4 v[N];
        int to[N];
        int before = -2;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            to[j] = __builtin_amdgcn_readlane(m.to, j);
            const int from = to[j] >= 0 ? __builtin_amdgcn_readlane(m.from, j) : -2;
            if (j && from == before) v[j] = v[j - 1];
            else if (from >= 0 && there) v[j] = *reinterpret_cast<const u32x4*>(src + from * bytes);
            else v[j] = u32x4{0, 0, 0, 0};
            before = from;
        }
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (to[j] >= 0 && there) st_stream(reinterpret_cast<u32x4*>(dst + to[j] * bytes), v[j]);
    }
}

hipError_t launch_move(const MovePart* parts, int nparts, const int32_t* to, const int32_t* from, int nmoves, int batch,
                       int sources, bool inside, hipStream_t st)
{
    for (int at = 0; at < nparts;) {
        MoveArgs a;
        a.to = to;
        a.from = from;
        a.nmoves = nmoves;
        a.batch = batch;
        a.sources = sources;
        a.inside = inside;
        a.nparts = 0;
        int64_t blocks = 0;
        while (at < nparts && a.nparts < kMoveParts) {
            const int64_t n = (parts[at].bytes + kColumnBytes - 1) / kColumnBytes;
            if (blocks + n > kMaxBlocks) break;
            a.dst[a.nparts] = parts[at].dst;
            a.src[a.nparts] = parts[at].src;
            a.n16[a.nparts] = (uint32_t)(parts[at].bytes / 16);
            a.first[a.nparts] = (uint32_t)blocks;
            blocks += n;
            ++a.nparts;
            ++at;
        }
        // workgroups of a column: until the card is full, with some moves for each (8 sequences forked to 56: 81 us; 4096
        // workgroups 4% more, 32768 6%)
        int64_t deal = (nmoves + 3) / 4;
        if (deal > (kMoveWorkgroups + blocks - 1) / blocks) deal = (kMoveWorkgroups + blocks - 1) / blocks;
        if (batch > kMoveBitmap) deal = 1;
        const size_t lds = nmoves > 1 && batch <= kMoveBitmap ? (size_t)(batch + 31) / 32 * 4 : 0;
        hipLaunchKernelGGL(k_move, dim3((unsigned)blocks, (unsigned)deal), dim3(256), lds, st, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

} // namespace ssq
