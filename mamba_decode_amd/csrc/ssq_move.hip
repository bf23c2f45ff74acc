// ssq_move.hip -- moves between sequences of states, for many arrays in one launch, gfx950.
//
// A thread owns one 16-byte column of an array and takes the moves in their order, so that a
// sequence may be the source of one move and the destination of a later one.
#include "ssq_ops_device.h"

namespace ssq {

constexpr int kMoveParts = 120; // arrays in one launch: the kernel's arguments stay below 4 KiB

struct MoveArgs {
    MovePart part[kMoveParts];
    uint32_t first[kMoveParts]; // the first workgroup of each array
    const int32_t* to;
    const int32_t* from;
    int nparts, nmoves, batch, sources;
};

__global__ __launch_bounds__(256) void k_move(MoveArgs a)
{
    int lo = 0, hi = a.nparts - 1;
    while (lo < hi) { // the last array whose first workgroup is not behind this one
        const int mid = (lo + hi + 1) >> 1;
        if (a.first[mid] <= blockIdx.x) lo = mid;
        else hi = mid - 1;
    }
    const MovePart p = a.part[lo];
    const int64_t col = (int64_t)(blockIdx.x - a.first[lo]) * kColumnBytes + threadIdx.x * 16;
    if (col >= p.bytes) return;
    for (int i = 0; i < a.nmoves; ++i) {
        const int to = a.to[i], from = a.from[i];
        if (to < 0 || to >= a.batch || from < -1 || from >= a.sources) continue;
        u32x4 v = {0, 0, 0, 0};
        if (from >= 0) v = *reinterpret_cast<const u32x4*>(p.src + from * p.bytes + col);
        *reinterpret_cast<u32x4*>(p.dst + to * p.bytes + col) = v;
    }
}

hipError_t launch_move(const MovePart* parts, int nparts, const int32_t* to, const int32_t* from, int nmoves, int batch,
                       int sources, bool, hipStream_t st)
{
    for (int at = 0; at < nparts;) {
        MoveArgs a;
        a.to = to;
        a.from = from;
        a.nmoves = nmoves;
        a.batch = batch;
        a.sources = sources;
        a.nparts = 0;
        int64_t blocks = 0;
        while (at < nparts && a.nparts < kMoveParts) {
            const int64_t n = (parts[at].bytes + kColumnBytes - 1) / kColumnBytes;
            if (blocks + n > kMaxBlocks) break;
            a.part[a.nparts] = parts[at];
            a.first[a.nparts] = (uint32_t)blocks;
            blocks += n;
            ++a.nparts;
            ++at;
        }
        hipLaunchKernelGGL(k_move, dim3((unsigned)blocks), dim3(256), 0, st, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

} // namespace ssq
