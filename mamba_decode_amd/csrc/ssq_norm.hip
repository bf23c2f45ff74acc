// ssq_norm.hip -- group norm with an activation, channels last, and its gradient, gfx950.
#include <type_traits>

#include "ssq_gated_device.h"

namespace ssq {

__device__ __forceinline__ float wave_sum(float v)
{
    v = group_sum<16>(v);
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

__device__ __forceinline__ float sigmoid(float v) { return __builtin_amdgcn_rcpf(1.0f + exp_fast(-v)); }
// by itself, before anything is multiplied with it: 0 for the lowest value of a type
__device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }

// a wave a token and group
template <int DT, int ACT, bool BACK>
__global__ __launch_bounds__(64) void k_norm_rows(NormArgs a, float* sums)
{
    const int64_t token = blockIdx.x / a.groups;
    const int group = blockIdx.x % a.groups;
    const int c0 = group * a.width, lane = threadIdx.x;
    const auto xat = [&](int c) { return load_elem<DT>(a.x, token * a.xs + c0 + c); };
    const auto zat = [&](int c) { return load_elem<DT>(a.z, token * a.zs + c0 + c); };
    const auto uat = [&](int c) {
        if constexpr (ACT != ACT_GATE_INPUT) return xat(c);
        return xat(c) * silu(zat(c));
    };
    float mean = 0.0f, sq = 0.0f;
    if (a.center) {
        for (int c = lane; c < a.width; c += 64) mean += uat(c);
        mean = wave_sum(mean) / a.width;
    }
    for (int c = lane; c < a.width; c += 64) {
        const float d = uat(c) - mean;
        sq = __builtin_fmaf(d, d, sq);
    }
    const float r = 1.0f / sqrtf(wave_sum(sq) / a.width + a.eps);
    const auto weight = [&](int c) { return a.weight ? a.weight[c0 + c] : 1.0f; };
    const auto bias = [&](int c) { return a.bias ? a.bias[c0 + c] : 0.0f; };
    if constexpr (!BACK) {
        for (int c = lane; c < a.width; c += 64) {
            const float n = __builtin_fmaf((uat(c) - mean) * r, weight(c), bias(c));
            float y = n;
            if constexpr (ACT == ACT_SILU) y = silu(n);
            if constexpr (ACT == ACT_GATE_OUTPUT) y = n * silu(zat(c));
            store_elem<DT>(a.y, token * a.ys + c0 + c, y);
        }
        return;
    }
    // gradient of n, and of z where the gate follows
    const auto dn = [&](int c, float n, float* dz) {
        const float dy = load_elem<DT>(a.dy, token * a.dys + c0 + c);
        if constexpr (ACT == ACT_GATE_INPUT) return dy;
        const float v = ACT == ACT_SILU ? n : zat(c), s = sigmoid(v);
        const float slope = s * __builtin_fmaf(v, 1.0f - s, 1.0f);
        if constexpr (ACT == ACT_SILU) return dy * slope;
        *dz = dy * n * slope;
        return dy * (v * s);
    };
    float m1 = 0.0f, m2 = 0.0f;
    for (int c = lane; c < a.width; c += 64) {
        const float m = (uat(c) - mean) * r;
        float dz = 0.0f;
        const float d = dn(c, __builtin_fmaf(m, weight(c), bias(c)), &dz) * weight(c);
        m1 += d;
        m2 = __builtin_fmaf(d, m, m2);
    }
    m1 = a.center ? wave_sum(m1) / a.width : 0.0f;
    m2 = wave_sum(m2) / a.width;
    for (int c = lane; c < a.width; c += 64) {
        const float m = (uat(c) - mean) * r;
        float dz = 0.0f;
        float du = dn(c, __builtin_fmaf(m, weight(c), bias(c)), &dz) * weight(c);
        du = r * (du - m1 - m * m2);
        if constexpr (ACT == ACT_GATE_INPUT) {
            const float z = zat(c), s = sigmoid(z);
            dz = du * xat(c) * s * __builtin_fmaf(z, 1.0f - s, 1.0f);
            du *= z * s;
        }
        store_elem<DT>(a.dx, token * a.dxs + c0 + c, du);
        if constexpr (ACT != ACT_SILU) store_elem<DT>(a.dz, token * a.dzs + c0 + c, dz);
    }
    if (lane == 0) {
        sums[(token * a.groups + group) * 2] = mean;
        sums[(token * a.groups + group) * 2 + 1] = r;
    }
}

// a thread a channel
template <int DT, int ACT>
__global__ __launch_bounds__(64) void k_norm_params(NormArgs a, const float* sums)
{
    const int c = blockIdx.x * 64 + threadIdx.x;
    if (c >= a.groups * a.width) return;
    const float weight = a.weight ? a.weight[c] : 1.0f, bias = a.bias ? a.bias[c] : 0.0f;
    float dw = 0.0f, db = 0.0f;
    for (int64_t token = 0; token < a.tokens; ++token) {
        const float* s = sums + (token * a.groups + c / a.width) * 2;
        float u = load_elem<DT>(a.x, token * a.xs + c), z = 0.0f;
        if constexpr (ACT != ACT_SILU) z = load_elem<DT>(a.z, token * a.zs + c);
        if constexpr (ACT == ACT_GATE_INPUT) u *= silu(z);
        const float m = (u - s[0]) * s[1], n = __builtin_fmaf(m, weight, bias);
        float dn = load_elem<DT>(a.dy, token * a.dys + c);
        if constexpr (ACT == ACT_SILU) dn *= sigmoid(n) * __builtin_fmaf(n, 1.0f - sigmoid(n), 1.0f);
        if constexpr (ACT == ACT_GATE_OUTPUT) dn *= silu(z);
        dw = __builtin_fmaf(dn, m, dw);
        db += dn;
    }
    if (a.dweight) a.dweight[c] = dw;
    if (a.dbias) a.dbias[c] = db;
}

template <class F>
static hipError_t with_act(int dtype, int act, F f)
{
    const auto ac = [&](auto dt) {
        switch (act) {
        case ACT_SILU: return f(dt, std::integral_constant<int, ACT_SILU>{});
        case ACT_GATE_OUTPUT: return f(dt, std::integral_constant<int, ACT_GATE_OUTPUT>{});
        case ACT_GATE_INPUT: return f(dt, std::integral_constant<int, ACT_GATE_INPUT>{});
        }
        return hipErrorInvalidValue;
    };
    switch (dtype) {
    case DT_FP32: return ac(std::integral_constant<int, DT_FP32>{});
    case DT_BF16: return ac(std::integral_constant<int, DT_BF16>{});
    case DT_FP16: return ac(std::integral_constant<int, DT_FP16>{});
    }
    return hipErrorInvalidValue;
}

size_t norm_workspace(int groups, int, int64_t tokens) { return (size_t)tokens * groups * 8; }

hipError_t launch_group_norm(int dtype, int act, const NormArgs& a, hipStream_t st)
{
    const dim3 grid((unsigned)(a.tokens * a.groups)), wg(64);
    return with_act(dtype, act, [&](auto dt, auto ac) {
        hipLaunchKernelGGL((k_norm_rows<decltype(dt)::value, decltype(ac)::value, false>), grid, wg, 0, st, a, nullptr);
        return hipGetLastError();
    });
}

hipError_t launch_group_norm_backward(int dtype, int act, const NormArgs& a, hipStream_t st)
{
    const dim3 grid((unsigned)(a.tokens * a.groups)), wg(64), cols((a.groups * a.width + 63) / 64);
    return with_act(dtype, act, [&](auto dt, auto ac) {
        constexpr int DT = decltype(dt)::value, ACT = decltype(ac)::value;
        if (a.tokens) hipLaunchKernelGGL((k_norm_rows<DT, ACT, true>), grid, wg, 0, st, a, a.ws);
        if (a.dweight || a.dbias) hipLaunchKernelGGL((k_norm_params<DT, ACT>), cols, wg, 0, st, a, a.ws);
        return hipGetLastError();
    });
}

} // namespace ssq
