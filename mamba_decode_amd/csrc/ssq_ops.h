// ssq_ops.h -- argument blocks and launchers of the linear-attention, beam-search and
// state-reordering kernels, shared with the C-ABI layer (not part of the public interface).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssq_internal.h"

namespace ssq {

enum Dtype : int { DT_FP32 = 0, DT_BF16 = 1, DT_FP16 = 2 };

// linear attention on a layer's state
struct LinArgs {
    uint8_t* codes; // quantized formats: [rows][128*bits/8]
    float* scale;   // [rows]
    float* zero;    // [rows] (asymmetric formats)
    float* h32;     // fp32 rows: the state, or a prefill's copy of a quantized one
    const void* q;
    const void* k;
    const void* v;
    const float* g; // nullptr: no decay
    void* o;
    int64_t qs, ks, vs, gs, os; // elements from one token to the next
    const int32_t* cu;          // prefill: [nseq + 1]
    const int32_t* slots;       // nullptr: sequence i is slot i
    const uint8_t* fresh;       // prefill; nullptr: none
    int64_t tokens;
    int nseq, batch, H, G, P;
    float oscale;
    SrArgs sr;
};


// Sizes are refused before anything is enqueued where a launch would have 2^32 work-items or more:
// workgroups of 256, state rows of a token step (16 a wave) and of a prompt (16 a column block, and
// the blocks' runs rounded up at no more than 2.3 blocks for each).
constexpr int64_t kMaxBlocks = (1 << 24) - 1;
constexpr int64_t kMaxStepRows = (int64_t)1 << 29;
constexpr int64_t kMaxPrefillRows = (int64_t)1 << 26;

struct BeamArgs {
    const void* logits;
    const float* scores;
    const uint8_t* finished;
    float* out_scores;
    int32_t* out_tokens;
    int32_t* out_parents;
    void* ws;
    int64_t row_stride;
    int batch, beams, vocab, nselect, pad;
};

// one array of a state with `bytes` (a multiple of 16) for each sequence
struct ReorderPart {
    uint8_t* p;
    int64_t bytes;
};
constexpr int64_t kColumnBytes = 256 * 16; // what a workgroup moves of each sequence of a group
constexpr int64_t reorder_blocks(int64_t bytes, int64_t groups) { return (bytes + kColumnBytes - 1) / kColumnBytes * groups; }

hipError_t launch_linattn_step(int fmt, int dtype, const LinArgs& a, bool pre, hipStream_t st);
size_t linattn_workspace(int fmt, int nseq, int64_t tokens, int H, int P, int num_cus);
hipError_t launch_linattn_prefill(int fmt, int dtype, const LinArgs& a, void* ws, int num_cus, hipStream_t st);
size_t beam_workspace(int batch, int beams, int vocab, int nselect);
hipError_t launch_beam_select(int dtype, const BeamArgs& a, hipStream_t st);
hipError_t launch_reorder(const ReorderPart* parts, int nparts, const int32_t* parents, int beams, int groups,
                          hipStream_t st);

} // namespace ssq
