// ssq_gated_device.h -- the decay and the input's factor of a gated linear recurrence from its
// gate, and their derivatives, in fp32.
#pragma once

#include "ssq_ops_device.h"

namespace ssq {

constexpr float kLog2e = 1.44269504088896341f;

__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// 1 - e^y for y <= 0 without the difference of near numbers: for y > -1/2 the series of
// (1 - e^y) / -y to the term y^7/8!, which leaves 2^-8/9! = 1.1e-8 of it at most.
__device__ __forceinline__ float one_minus_exp(float y, float e)
{
    float p = 1.0f / 40320.0f;
    p = __builtin_fmaf(p, y, 1.0f / 5040.0f);
    p = __builtin_fmaf(p, y, 1.0f / 720.0f);
    p = __builtin_fmaf(p, y, 1.0f / 120.0f);
    p = __builtin_fmaf(p, y, 1.0f / 24.0f);
    p = __builtin_fmaf(p, y, 1.0f / 6.0f);
    p = __builtin_fmaf(p, y, 0.5f);
    p = __builtin_fmaf(p, y, 1.0f);
    return y > -0.5f ? -y * p : 1.0f - e;
}

struct GateValue {
    float a; // decay
    float s; // factor on the input
};
struct GateSlope {
    float a, s, da, ds; // and their derivatives along the gate
};

template <int GATE, int INPUT>
__device__ __forceinline__ GateSlope gate_slope(float g)
{
    GateSlope r;
    float rest; // 1 - a
    if constexpr (GATE == GATE_LOG) {
        r.a = exp_fast(g);
        r.da = r.a;
        rest = INPUT == IN_COMPLEMENT ? one_minus_exp(g, r.a) : 0.0f;
    } else {
        // e <= 1: neither side of the sigmoid is a difference
        const float e = exp_fast(-fabsf(g));
        const float big = __builtin_amdgcn_rcpf(1.0f + e), small = e * big;
        r.a = g >= 0.0f ? big : small;
        rest = g >= 0.0f ? small : big;
        r.da = big * small;
    }
    if constexpr (INPUT == IN_PLAIN) {
        r.s = 1.0f;
        r.ds = 0.0f;
    } else if constexpr (INPUT == IN_COMPLEMENT) {
        r.s = rest;
        r.ds = -r.da;
    } else {
        const float sq = GATE == GATE_LOG ? one_minus_exp(2.0f * g, r.a * r.a) : rest * (1.0f + r.a);
        r.s = __builtin_amdgcn_sqrtf(fmaxf(sq, 0.0f));
        r.ds = r.s > 0.0f ? -r.a * r.da * __builtin_amdgcn_rcpf(r.s) : 0.0f;
    }
    return r;
}

template <int GATE, int INPUT>
__device__ __forceinline__ GateValue gate_value(float g)
{
    const GateSlope r = gate_slope<GATE, INPUT>(g);
    return {r.a, r.s};
}

// a sequence's tokens, within 0 .. tokens whatever cu says
struct Span {
    int64_t begin;
    int64_t len;
};
__device__ __forceinline__ Span gated_span(const GatedArgs& a, int seq)
{
    const int64_t lo = a.cu[seq], hi = a.cu[seq + 1];
    Span s;
    s.begin = lo < 0 ? 0 : lo > a.tokens ? a.tokens : lo;
    const int64_t end = hi < 0 ? 0 : hi > a.tokens ? a.tokens : hi;
    s.len = end > s.begin ? end - s.begin : 0;
    return s;
}

// the sequence's place in the state, -1: left out
__device__ __forceinline__ int gated_slot(const GatedArgs& a, int seq)
{
    if (!a.slots) return seq;
    const int slot = a.slots[seq];
    return slot >= 0 && slot < a.batch ? slot : -1;
}

} // namespace ssq
