// ssq_gated.hip -- a gated linear recurrence, h_t = a_t h_(t-1) + s_t x_t in every channel, over
// ragged sequences, its gradient and its single-token form, gfx950.
#include <type_traits>

#include "ssq_gated_device.h"

namespace ssq {

// one thread a sequence and channel, one token after the other
template <int DT, int GATE, int INPUT>
__global__ __launch_bounds__(256) void k_gated_scan(GatedArgs a)
{
    const int c = (int)(blockIdx.x % ((a.channels + 255) / 256)) * 256 + threadIdx.x;
    const int seq = (int)(blockIdx.x / ((a.channels + 255) / 256));
    if (c >= a.channels) return;
    const int slot = gated_slot(a, seq);
    if (slot < 0) return;
    const Span sp = gated_span(a, seq);
    float* state = a.h ? a.h + (int64_t)slot * a.channels + c : nullptr;
    float h = state && !(a.fresh && a.fresh[seq]) ? *state : 0.0f;
    const int64_t row = sp.begin / kGatedChunk + seq;
    for (int64_t t = 0; t < sp.len; ++t) {
        if (a.ckpt && t % kGatedChunk == 0) a.ckpt[(row + t / kGatedChunk) * a.channels + c] = h;
        const GateValue v = gate_value<GATE, INPUT>(load_elem<DT>(a.g, (sp.begin + t) * a.gs + c));
        h = __builtin_fmaf(v.a, h, v.s * load_elem<DT>(a.x, (sp.begin + t) * a.xs + c));
        store_elem<DT>(a.o, (sp.begin + t) * a.os + c, h);
    }
    if (state) *state = h;
}

template <int DT, int GATE, int INPUT>
__global__ __launch_bounds__(256) void k_gated_backward(GatedArgs a)
{
    const int c = (int)(blockIdx.x % ((a.channels + 255) / 256)) * 256 + threadIdx.x;
    const int seq = (int)(blockIdx.x / ((a.channels + 255) / 256));
    if (c >= a.channels) return;
    if (gated_slot(a, seq) < 0) return;
    const Span sp = gated_span(a, seq);
    const int64_t at = (int64_t)seq * a.channels + c;
    float dh = a.dlast ? a.dlast[at] : 0.0f;
    const int64_t row = sp.begin / kGatedChunk + seq;
    for (int64_t j = (sp.len + kGatedChunk - 1) / kGatedChunk - 1; j >= 0; --j) {
        const int n = (int)(sp.len - j * kGatedChunk < kGatedChunk ? sp.len - j * kGatedChunk : kGatedChunk);
        const int64_t t0 = sp.begin + j * kGatedChunk;
        float before[kGatedChunk];
        float h = a.ckpt[(row + j) * a.channels + c];
        for (int i = 0; i < n; ++i) {
            before[i] = h;
            const GateValue v = gate_value<GATE, INPUT>(load_elem<DT>(a.g, (t0 + i) * a.gs + c));
            h = __builtin_fmaf(v.a, h, v.s * load_elem<DT>(a.x, (t0 + i) * a.xs + c));
        }
        for (int i = n - 1; i >= 0; --i) {
            const GateSlope v = gate_slope<GATE, INPUT>(load_elem<DT>(a.g, (t0 + i) * a.gs + c));
            const float x = load_elem<DT>(a.x, (t0 + i) * a.xs + c);
            dh += load_elem<DT>(a.dout, (t0 + i) * a.dos + c);
            store_elem<DT>(a.dx, (t0 + i) * a.dxs + c, v.s * dh);
            store_elem<DT>(a.dg, (t0 + i) * a.dgs + c, dh * __builtin_fmaf(v.da, before[i], v.ds * x));
            dh *= v.a;
        }
    }
    if (a.dfirst) a.dfirst[at] = dh;
}

// One token: a thread takes 8 channels of a sequence.
template <int DT, int GATE, int INPUT>
__global__ __launch_bounds__(256) void k_gated_step(GatedArgs a)
{
    const int per = a.channels / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)a.nseq * per) return;
    const int seq = (int)(i / per), c = (int)(i % per) * 8;
    const int slot = gated_slot(a, seq);
    if (slot < 0) return;
    for (int e = 0; e < 8; ++e) {
        float* state = a.h + (int64_t)slot * a.channels + c + e;
        const GateValue v = gate_value<GATE, INPUT>(load_elem<DT>(a.g, seq * a.gs + c + e));
        const float h = __builtin_fmaf(v.a, *state, v.s * load_elem<DT>(a.x, seq * a.xs + c + e));
        *state = h;
        store_elem<DT>(a.o, seq * a.os + c + e, h);
    }
}

// f(dtype, gate, input) with the three as constants
template <class F>
static hipError_t with_gate(int dtype, int gate, int input, F f)
{
    const auto in = [&](auto dt, auto ga) {
        switch (input) {
        case IN_PLAIN: return f(dt, ga, std::integral_constant<int, IN_PLAIN>{});
        case IN_COMPLEMENT: return f(dt, ga, std::integral_constant<int, IN_COMPLEMENT>{});
        case IN_NORM: return f(dt, ga, std::integral_constant<int, IN_NORM>{});
        }
        return hipErrorInvalidValue;
    };
    const auto ga = [&](auto dt) {
        return gate == GATE_LOG ? in(dt, std::integral_constant<int, GATE_LOG>{}) : in(dt, std::integral_constant<int, GATE_SIGMOID>{});
    };
    switch (dtype) {
    case DT_FP32: return ga(std::integral_constant<int, DT_FP32>{});
    case DT_BF16: return ga(std::integral_constant<int, DT_BF16>{});
    case DT_FP16: return ga(std::integral_constant<int, DT_FP16>{});
    }
    return hipErrorInvalidValue;
}

size_t gated_workspace(int, int, int64_t, int) { return 0; }

hipError_t launch_gated_scan(int dtype, int gate, int input, const GatedArgs& a, void*, int, hipStream_t st)
{
    const dim3 grid((unsigned)((int64_t)a.nseq * ((a.channels + 255) / 256))), wg(256);
    return with_gate(dtype, gate, input, [&](auto dt, auto ga, auto in) {
        hipLaunchKernelGGL((k_gated_scan<decltype(dt)::value, decltype(ga)::value, decltype(in)::value>), grid, wg, 0, st, a);
        return hipGetLastError();
    });
}

hipError_t launch_gated_backward(int dtype, int gate, int input, const GatedArgs& a, void*, int, hipStream_t st)
{
    const dim3 grid((unsigned)((int64_t)a.nseq * ((a.channels + 255) / 256))), wg(256);
    return with_gate(dtype, gate, input, [&](auto dt, auto ga, auto in) {
        hipLaunchKernelGGL((k_gated_backward<decltype(dt)::value, decltype(ga)::value, decltype(in)::value>), grid, wg, 0, st, a);
        return hipGetLastError();
    });
}

hipError_t launch_gated_step(int dtype, int gate, int input, const GatedArgs& a, hipStream_t st)
{
    const int64_t n = (int64_t)a.nseq * (a.channels / 8);
    const dim3 grid((unsigned)((n + 255) / 256)), wg(256);
    return with_gate(dtype, gate, input, [&](auto dt, auto ga, auto in) {
        hipLaunchKernelGGL((k_gated_step<decltype(dt)::value, decltype(ga)::value, decltype(in)::value>), grid, wg, 0, st, a);
        return hipGetLastError();
    });
}

} // namespace ssq
