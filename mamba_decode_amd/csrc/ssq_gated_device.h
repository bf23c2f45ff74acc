// ssq_gated_device.h -- the decay and the input's factor of a gated linear recurrence from its
// gate, and their derivatives, in fp32.
#pragma once

#include "ssq_ops_device.h"

namespace ssq {

constexpr float kLog2e = 1.44269504088896341f;

__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// 1 - e^(Y g) for g <= 0 and Y = 1 or 2 without the difference of near numbers, e = e^(Y g): for
// y = Y g > -1/2 the polynomial of degree 4 nearest to (1 - e^y) / -y in relative error, fitted to it, which is
// off by 1.8 * 2^-24 with these coefficients and by 3.3 * 2^-24 as it is evaluated in fp32; below, the difference is 0.39 of
// its larger side at least.
template <int Y>
__device__ __forceinline__ float one_minus_exp(float g, float e)
{
    constexpr float y = Y;
    float p = -0.00677103545f * y * y * y * y * y;
    p = __builtin_fmaf(p, g, -0.0410012762f * y * y * y * y);
    p = __builtin_fmaf(p, g, -0.166548151f * y * y * y);
    p = __builtin_fmaf(p, g, -0.499992498f * y * y);
    p = __builtin_fmaf(p, g, -0.999999923f * y);
    float near = g * p;
    asm volatile("" : "+v"(near)); // both sides and a select: a branch around the polynomial would be taken token by token
    return g > -0.5f / y ? near : 1.0f - e;
}

struct GateValue {
    float a; // decay
    float s; // factor on the input
};
struct GateSlope {
    float a, s, da, ds; // and their derivatives along the gate
};

// The sigmoid and one minus it, from e = exp(-g): neither is a difference.  From e = 2^24 on the latter is one to a last
// step, and is not formed from the former: above 2^126 that is subnormal, which the reciprocal returns as zero, and e may
// be infinity.
__device__ __forceinline__ void sigmoid_pair(float g, float* a, float* rest)
{
    const float e = exp_fast(-g);
    *a = __builtin_amdgcn_rcpf(1.0f + e);
    *rest = e < 0x1p24f ? e * *a : 1.0f;
}

template <int GATE, int INPUT>
__device__ __forceinline__ GateSlope gate_slope(float g)
{
    GateSlope r;
    if constexpr (GATE == GATE_LOG) {
        r.a = exp_fast(g);
        r.da = r.a;
        if constexpr (INPUT == IN_COMPLEMENT) {
            r.s = one_minus_exp<1>(g, r.a);
            r.ds = -r.a;
        }
        if constexpr (INPUT == IN_NORM) {
            const float sq = r.a * r.a;
            r.s = __builtin_amdgcn_sqrtf(one_minus_exp<2>(g, sq));
            r.ds = r.s > 0.0f ? -sq * __builtin_amdgcn_rcpf(r.s) : 0.0f;
        }
    } else {
        float rest;
        sigmoid_pair(g, &r.a, &rest);
        r.da = r.a * rest;
        if constexpr (INPUT == IN_COMPLEMENT) {
            r.s = rest;
            r.ds = -r.da;
        }
        if constexpr (INPUT == IN_NORM) { // ds = -a^2 (1 - a) / s = -a^2 s / (1 + a)
            const float up = 1.0f + r.a;
            r.s = __builtin_amdgcn_sqrtf(rest * up);
            r.ds = -r.a * r.a * r.s * __builtin_amdgcn_rcpf(up);
        }
    }
    if constexpr (INPUT == IN_PLAIN) {
        r.s = 1.0f;
        r.ds = 0.0f;
    }
    return r;
}

// what is not used of the slopes is not computed
template <int GATE, int INPUT>
__device__ __forceinline__ GateValue gate_value(float g)
{
    const GateSlope r = gate_slope<GATE, INPUT>(g);
    return {r.a, r.s};
}

// A descriptor of the wave's: without the readfirstlanes the compiler would loop over its lanes' values.  Loads
// through it need no branch for rows that are not there, and where loads ahead stand in no branch the compiler
// counts them instead of waiting for all of them.
__device__ __forceinline__ Rsrc uniform_rsrc(uint64_t base, uint32_t bytes)
{
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)base), hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(base >> 32));
    return make_rsrc((const void*)(((uint64_t)hi << 32) | lo), (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes));
}
constexpr uint32_t kNowhere = 0x80000000u; // an offset beyond every descriptor's bytes

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
