// ssq_reorder.hip -- states follow their beams: sequence j of a group becomes what sequence
// parents[j] of the group was, in place, for many arrays in one launch, gfx950.
//
// A thread owns one 16-byte column of a group: it reads that column of every sequence that
// another one comes from, then writes the sequences that change.  No other thread touches the
// column, so the move needs no second buffer, no order among threads and each byte is read at
// most once and written at most once; sequences that keep their place are not touched.  Bytes
// bound it: 48 int4 layers of 8 x 4 beams (301 MB) take 50-58 us with the non-temporal hint on
// loads and stores, 5.2-6.0 TB/s, 61-65 us without it on either.
#include "ssq_ops_device.h"

namespace ssq {

constexpr int kMaxParts = 160; // arrays in one launch: the kernel's arguments stay below 4 KiB

struct ReorderArgs {
    ReorderPart part[kMaxParts];
    uint32_t first[kMaxParts]; // the first workgroup of each array
    const int32_t* parents;
    int nparts, beams, groups;
};

template <int BMAX>
__global__ __launch_bounds__(256) void k_reorder(ReorderArgs a)
{
    int lo = 0, hi = a.nparts - 1;
    while (lo < hi) { // the last array whose first workgroup is not behind this one
        const int mid = (lo + hi + 1) >> 1;
        if (a.first[mid] <= blockIdx.x) lo = mid;
        else hi = mid - 1;
    }
    const int64_t bytes = a.part[lo].bytes;
    const uint32_t rel = blockIdx.x - a.first[lo];
    const uint32_t per_group = (uint32_t)((bytes + kColumnBytes - 1) / kColumnBytes);
    const uint32_t group = rel / per_group;
    const int64_t col = (int64_t)(rel % per_group) * kColumnBytes + threadIdx.x * 16;

    const int lane = threadIdx.x & 63;
    const int parent = lane < a.beams ? a.parents[(int64_t)group * a.beams + lane] : -1;
    uint64_t to[BMAX]; // the sequences that come from s and are not s
#pragma unroll
    for (int s = 0; s < BMAX; ++s) to[s] = s < a.beams ? __ballot(parent == s && lane != s) : 0;
    if (col >= bytes) return;
    uint8_t* base = a.part[lo].p + (int64_t)group * a.beams * bytes + col;
    u32x4 v[BMAX];
#pragma unroll
    for (int s = 0; s < BMAX; ++s)
        if (to[s]) v[s] = ld_stream(reinterpret_cast<const u32x4*>(base + s * bytes));
#pragma unroll
    for (int s = 0; s < BMAX; ++s)
        for (uint64_t m = to[s]; m; m &= m - 1) {
            const int j = __builtin_ctzll(m);
            st_stream(reinterpret_cast<u32x4*>(base + j * bytes), v[s]);
        }
}

hipError_t launch_reorder(const ReorderPart* parts, int nparts, const int32_t* parents, int beams, int groups,
                          hipStream_t st)
{
    for (int at = 0; at < nparts;) {
        ReorderArgs a;
        a.parents = parents;
        a.beams = beams;
        a.groups = groups;
        a.nparts = 0;
        int64_t blocks = 0;
        while (at < nparts && a.nparts < kMaxParts) {
            const int64_t n = reorder_blocks(parts[at].bytes, groups); // kMaxBlocks at most
            if (blocks + n > kMaxBlocks) break;
            a.part[a.nparts] = parts[at];
            a.first[a.nparts] = (uint32_t)blocks;
            blocks += n;
            ++a.nparts;
            ++at;
        }
        const dim3 grid((unsigned)blocks), wg(256);
        if (beams <= 4) hipLaunchKernelGGL(k_reorder<4>, grid, wg, 0, st, a);
        else if (beams <= 8) hipLaunchKernelGGL(k_reorder<8>, grid, wg, 0, st, a);
        else if (beams <= 16) hipLaunchKernelGGL(k_reorder<16>, grid, wg, 0, st, a);
        else hipLaunchKernelGGL(k_reorder<32>, grid, wg, 0, st, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

} // namespace ssq
