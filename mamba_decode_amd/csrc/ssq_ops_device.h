// ssq_ops_device.h -- device helpers of the linear-attention and beam-search kernels: loads and
// stores of fp32, bf16 and fp16 tensors as fp32 values, and one quantized row's refit.
#pragma once

#include "ssq_device.h"
#include "ssq_ops.h"

namespace ssq {

template <int DT> struct Elem;
template <> struct Elem<DT_FP32> { using T = float; };
template <> struct Elem<DT_BF16> { using T = __bf16; };
template <> struct Elem<DT_FP16> { using T = _Float16; };

template <int DT>
__device__ __forceinline__ float to_f32(uint32_t bits16)
{
    if constexpr (DT == DT_BF16) return __uint_as_float(bits16 << 16);
    else return (float)__builtin_bit_cast(_Float16, (uint16_t)bits16);
}

// E consecutive elements (E a multiple of 4) at an address aligned to min(16, E*size) bytes
template <int DT, int E>
__device__ __forceinline__ void load_elems(const void* p, float* v)
{
    if constexpr (DT == DT_FP32) {
        load_f32<E>(static_cast<const float*>(p), v);
    } else if constexpr (E % 8 == 0) {
#pragma unroll
        for (int i = 0; i < E / 8; ++i) {
            const u32x4 w = static_cast<const u32x4*>(p)[i];
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[8 * i + 2 * j] = to_f32<DT>(ws[j] & 0xFFFFu);
                v[8 * i + 2 * j + 1] = to_f32<DT>(ws[j] >> 16);
            }
        }
    } else {
        static_assert(E == 4, "4 elements or a multiple of 8");
        const u32x2 w = *static_cast<const u32x2*>(p);
        v[0] = to_f32<DT>(w.x & 0xFFFFu);
        v[1] = to_f32<DT>(w.x >> 16);
        v[2] = to_f32<DT>(w.y & 0xFFFFu);
        v[3] = to_f32<DT>(w.y >> 16);
    }
}

template <int DT>
__device__ __forceinline__ float load_elem(const void* p, int64_t i)
{
    return (float)static_cast<const typename Elem<DT>::T*>(p)[i];
}

// one rounding to the nearest value of the type, ties to even
template <int DT>
__device__ __forceinline__ void store_elem(void* p, int64_t i, float v)
{
    static_cast<typename Elem<DT>::T*>(p)[i] = (typename Elem<DT>::T)v;
}

// two of them, in one conversion where the type has one
template <int DT>
__device__ __forceinline__ uint32_t pack_elems(float lo, float hi)
{
    typedef typename Elem<DT>::T T2 __attribute__((ext_vector_type(2)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){lo, hi}, T2));
}

template <int DT>
__device__ __forceinline__ const void* elem_ptr(const void* p, int64_t i)
{
    return static_cast<const typename Elem<DT>::T*>(p) + i;
}

// Refit and round one fp32 row, E entries a lane: h becomes f = 1.5*2^23 + code, g its grid.
// Whole waves only (the choice of path is the wave's).
template <int F, int E, int LPR, bool SR>
__device__ __forceinline__ bool refit_row(float* h, RowGrid& g, uint64_t seed, uint64_t ctr0)
{
    float mn = 0.0f, mx = 0.0f, am = 0.0f;
    if constexpr (Traits<F>::asym) {
        mn = h[0];
        mx = h[0];
#pragma unroll
        for (int e = 1; e < E; ++e) {
            mn = fminf(mn, h[e]);
            mx = fmaxf(mx, h[e]);
        }
        mn = group_min<LPR>(mn);
        mx = group_max<LPR>(mx);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) am = fmaxf(am, fabsf(h[e]));
        am = group_max<LPR>(am);
    }
    const bool fast = __all(refit_fast<F, SR>(mn, mx, am, g));
    if (fast) {
        if constexpr (SR) {
            round_codes_sr<F, E, true>(h, g, seed, ctr0, h);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) h[e] = __builtin_fmaf(h[e], g.inv, g.Mz);
        }
    } else {
        g = refit<F>(mn, mx, am);
        if constexpr (SR) {
            round_codes_sr<F, E, false>(h, g, seed, ctr0, h);
        } else {
            const bool slow_any = Traits<F>::asym && __any(g.slow);
            round_codes<F, E>(h, g, slow_any, h);
        }
    }
    return fast;
}

} // namespace ssq
