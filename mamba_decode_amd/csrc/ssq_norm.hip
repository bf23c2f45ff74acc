// ssq_norm.hip -- group norm with an activation, channels last, and its gradient, gfx950.
//
// Each token's groups stand in registers from their one read to their one write: the mean, then the squares of the
// distances from it, then the outputs.  The gradient computes the statistics again from x and z, which it reads
// anyway, and keeps the sums over its tokens for the parameters' gradients; a second launch adds the workgroups' sums
// in their order.  The next token's loads are under way meanwhile.  Bytes bound it: 8192 tokens of 8 groups of 1024 in
// bf16 with a gate take 72 us (403 MB, 5.6 TB/s), 118-120 us (671 MB, 5.6 TB/s) and 5 us for the parameters' second launch.
#include <type_traits>

#include "ssq_gated_device.h"

namespace ssq {

// How the groups lie on the waves.  A lane holds V vectors of 8 channels of a group.  A group takes a
// power of two of lanes of one wave (wpg = 1; then a wave holds `gslots` neighbouring groups of `tokens`
// tokens), or wpg whole waves, up to MAXW.  A workgroup stays on its groups and goes along the tokens, so that weights and the
// sums of their gradients stay in registers.
struct NormPlan {
    int lanes;    // of a group within a wave
    int gslots;   // groups of a token in a wave
    int tokens;   // tokens of a wave at a time
    int gblocks;  // workgroups along the groups
    int tblocks;  // workgroups along the tokens
    int wpg, v;   // waves of a group, vectors of a lane
};

struct NormCall {
    NormArgs a;
    NormPlan p;
};

template <int DT, int V>
struct Vectors {
    static constexpr int SIZE = DT == DT_FP32 ? 4 : 2, NW = 2 * SIZE;
    uint32_t w[V][NW];
    __device__ __forceinline__ void load(Rsrc r, const uint32_t* off)
    {
#pragma unroll
        for (int v = 0; v < V; ++v) buf_load_words<NW, 0>(r, off[v], 0u, w[v]);
    }
    __device__ __forceinline__ float get(int v, int i) const
    {
        if constexpr (DT == DT_FP32) return __uint_as_float(w[v][i]);
        else return to_f32<DT>(i & 1 ? w[v][i / 2] >> 16 : w[v][i / 2] & 0xFFFFu);
    }
};

template <int DT>
__device__ __forceinline__ void store_vector(Rsrc r, uint32_t off, const float* f)
{
    uint32_t w[DT == DT_FP32 ? 8 : 4];
    if constexpr (DT == DT_FP32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(f[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack_elems<DT>(f[2 * i], f[2 * i + 1]);
    }
    buf_store_words<(DT == DT_FP32 ? 8 : 4), kAuxStore>(r, off, 0u, w);
}

// sums over the lanes of a group within a wave; every lane has the sum, in an order that the size alone sets
__device__ __forceinline__ float lane_sum(float v, int lanes)
{
    if (lanes > 1) v += dppf<0xB1>(v);
    if (lanes > 2) v += dppf<0x4E>(v);
    if (lanes > 4) v += dppf<0x141>(v);
    if (lanes > 8) v += dppf<0x140>(v);
    if (lanes > 16) v += __shfl_xor(v, 16);
    if (lanes > 32) v += __shfl_xor(v, 32);
    return v;
}

template <int MAXW>
struct GroupSum {
    float (*buf)[MAXW][2]; // two places in turn: one barrier a sum
    int lanes, wave, wpg, turn;
    __device__ __forceinline__ void operator()(float& x, float& y)
    {
        x = lane_sum(x, lanes);
        y = lane_sum(y, lanes);
        across(x, &y);
    }
    __device__ __forceinline__ void operator()(float& x)
    {
        x = lane_sum(x, lanes);
        across(x, nullptr);
    }
    __device__ __forceinline__ void across(float& x, float* y)
    {
        if constexpr (MAXW > 1) {
            if ((threadIdx.x & 63) == 0) {
                buf[turn][wave][0] = x;
                if (y) buf[turn][wave][1] = *y;
            }
            __syncthreads();
            // A lane reads a wave's sums, each 16 lanes all of them (4096 tokens of 8192 channels, gradient: 70 us, 74 with one
            // wave's after the other).
            const int i = threadIdx.x & (MAXW - 1);
            x = lane_sum(i < wpg ? buf[turn][i][0] : 0.0f, MAXW);
            if (y) *y = lane_sum(i < wpg ? buf[turn][i][1] : 0.0f, MAXW);
            turn ^= 1;
        }
    }
};

__device__ __forceinline__ float sigmoid(float v) { return __builtin_amdgcn_rcpf(1.0f + exp_fast(-v)); }

template <int DT, int ACT, int MAXW, int V, bool BACK>
__global__ __launch_bounds__(MAXW == 1 ? 256 : MAXW * 64) void k_norm(NormCall c)
{
    constexpr bool IN_WAVE = MAXW == 1;
    // Groups of more than 8192 channels leave a lane of 16 waves too few registers for the parameters, the sums of
    // their gradients and loads ahead: the parameters are read again for every token, the sums stand in LDS, each lane its own
    // (2000 tokens of 16000 channels in bf16, gradient: 124 us, 302 us all in registers).  The gated forms still have 8 to 24
    // bytes of scratch a lane (gate after) and 96 to 108 (gate before) at the 128 registers of 16 waves, the one without a gate none.
    constexpr bool LEAN = BACK && MAXW == 16 && V == 2;
    __shared__ float s_grad[LEAN ? 2 * V * 2 : 1][LEAN ? MAXW * 64 : 1][4];
    __shared__ float s_sum[2][MAXW][2];
    const NormArgs& a = c.a;
    const NormPlan& p = c.p;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int gblock = (int)(blockIdx.x % p.gblocks), tblock = (int)(blockIdx.x / p.gblocks);
    const int gi = IN_WAVE ? lane / p.lanes : 0;
    const int group = gblock * p.gslots + gi % p.gslots;
    const int n8 = a.width / 8;
    const float inv = 1.0f / (float)a.width;
    const bool centre = a.center;
    int vec[V];
    bool in[V]; // the vector is one of the group's
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = IN_WAVE ? lane % p.lanes + v * 64 : (int)threadIdx.x + v * p.wpg * 64;
        in[v] = group < a.groups && i < n8;
        vec[v] = i;
    }
    const int64_t c0 = (int64_t)group * a.width;
    float w[V][8], b[V][8], dw[V][8], db[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[v][i] = 1.0f;
            b[v][i] = dw[v][i] = db[v][i] = 0.0f;
        }
    const auto parameters = [&]() {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (in[v]) {
                if (a.weight) load_f32<8>(a.weight + c0 + 8 * vec[v], w[v]);
                if (a.bias) load_f32<8>(a.bias + c0 + 8 * vec[v], b[v]);
            }
    };
    const auto grads = [&](int k, int v, float* f, bool store) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float& s = s_grad[LEAN ? (k * V + v) * 2 + i / 4 : 0][LEAN ? threadIdx.x : 0][i & 3];
            if (store) s = f[i];
            else f[i] = s;
        }
    };
    if constexpr (!LEAN) parameters();
    if constexpr (LEAN)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            grads(0, v, dw[v], true);
            grads(1, v, db[v], true);
        }
    GroupSum<MAXW> sum{s_sum, IN_WAVE ? p.lanes : 64, wave, p.wpg, 0};
    // tokens of this lane: one in every `step`
    const int64_t per = (IN_WAVE ? 4 : 1) * (int64_t)p.tokens, step = per * p.tblocks;
    const int64_t first = tblock * per + (IN_WAVE ? wave * p.tokens : 0); // the wave's
    const int sub = IN_WAVE ? gi / p.gslots : 0;                          // the lane's, from it
    const int64_t rounds = (a.tokens - tblock * per + step - 1) / step;   // the workgroup's

    // the wave's tokens from `token` on of a tensor, and the lane's places in them
    constexpr int SIZE = Vectors<DT, V>::SIZE;
    const auto rows = [&](const void* base, int64_t stride, int64_t token) {
        const int64_t left = a.tokens - token, n = left < p.tokens ? left : p.tokens;
        const uint32_t bytes = n > 0 ? (uint32_t)((n - 1) * stride + (int64_t)a.groups * a.width) * SIZE : 0u;
        return uniform_rsrc((uint64_t)base + (uint64_t)(token * stride * SIZE), bytes);
    };
    const auto places = [&](int64_t stride, uint32_t* off) {
#pragma unroll
        for (int v = 0; v < V; ++v) off[v] = in[v] ? ((uint32_t)sub * (uint32_t)stride + (uint32_t)c0 + 8 * vec[v]) * SIZE : kNowhere;
    };
    uint32_t ox[V], oz[V], ody[V], oo[V], odz[V];
    places(a.xs, ox);
    places(a.zs, oz);
    places(a.dys, ody);
    places(BACK ? a.dxs : a.ys, oo);
    places(a.dzs, odz);
    Vectors<DT, V> x, z, dy, nx, nz, ndy;
    const auto load = [&](int64_t token) {
        nx.load(rows(a.x, a.xs, token), ox);
        if constexpr (ACT != ACT_SILU) nz.load(rows(a.z, a.zs, token), oz);
        if constexpr (BACK) ndy.load(rows(a.dy, a.dys, token), ody);
    };
    load(first);
    int64_t token = first;
    for (int64_t round = 0; round < rounds; ++round, token += step) {
        x = nx;
        z = nz;
        dy = ndy;
        if constexpr (!LEAN) load(token + step); // nothing, behind the last token
        const bool here = token + sub < a.tokens;
        const Rsrc ro = rows(BACK ? a.dx : a.y, BACK ? a.dxs : a.ys, token), rdz = rows(a.dz, a.dzs, token);

        float m[V][8], swish[V][8], slope[V][8]; // u, then its distance from the mean, then normalised; silu(z) and its slope
        float mean = 0.0f, sq = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                m[v][i] = x.get(v, i);
                if constexpr (ACT != ACT_SILU) {
                    const float zz = z.get(v, i), s = sigmoid(zz);
                    swish[v][i] = zz * s; // by itself: 0 for the lowest value of a type
                    if constexpr (BACK) slope[v][i] = s * __builtin_fmaf(zz, 1.0f - s, 1.0f);
                    if constexpr (ACT == ACT_GATE_INPUT) m[v][i] *= swish[v][i];
                }
                mean += m[v][i]; // a vector that is not there is zero
            }
        if (centre) {
            sum(mean);
            mean *= inv;
        } else {
            mean = 0.0f;
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                m[v][i] = in[v] && here ? m[v][i] - mean : 0.0f;
                sq = __builtin_fmaf(m[v][i], m[v][i], sq);
            }
        sum(sq);
        const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(sq, inv, a.eps));
        if constexpr (!BACK) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    y[i] = __builtin_fmaf(m[v][i] * r, w[v][i], b[v][i]);
                    if constexpr (ACT == ACT_SILU) y[i] *= sigmoid(y[i]);
                    if constexpr (ACT == ACT_GATE_OUTPUT) y[i] *= swish[v][i];
                }
                store_vector<DT>(ro, oo[v], y);
            }
        } else {
            float dm[V][8], m1 = 0.0f, m2 = 0.0f;
            if constexpr (LEAN) parameters();
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float dz[8];
                if constexpr (LEAN) {
                    grads(0, v, dw[v], false);
                    grads(1, v, db[v], false);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    m[v][i] *= r;
                    float dn = dy.get(v, i);
                    if constexpr (ACT != ACT_GATE_INPUT) {
                        const float n = __builtin_fmaf(m[v][i], w[v][i], b[v][i]);
                        if constexpr (ACT == ACT_SILU) {
                            const float s = sigmoid(n);
                            dn *= s * __builtin_fmaf(n, 1.0f - s, 1.0f);
                        } else {
                            dz[i] = dn * n * slope[v][i];
                            dn *= swish[v][i];
                        }
                    }
                    dw[v][i] = __builtin_fmaf(dn, m[v][i], dw[v][i]);
                    db[v][i] += dn;
                    dm[v][i] = dn * w[v][i];
                    m1 += dm[v][i];
                    m2 = __builtin_fmaf(dm[v][i], m[v][i], m2);
                }
                if constexpr (LEAN) {
                    grads(0, v, dw[v], true);
                    grads(1, v, db[v], true);
                }
                if constexpr (ACT == ACT_GATE_OUTPUT) store_vector<DT>(rdz, odz[v], dz);
            }
            sum(m1, m2);
            m1 = centre ? m1 * inv : 0.0f;
            m2 *= inv;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float dx[8], dz[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dx[i] = r * (dm[v][i] - m1 - m[v][i] * m2);
                    if constexpr (ACT == ACT_GATE_INPUT) {
                        dz[i] = dx[i] * x.get(v, i) * slope[v][i];
                        dx[i] *= swish[v][i];
                    }
                }
                store_vector<DT>(ro, oo[v], dx);
                if constexpr (ACT == ACT_GATE_INPUT) store_vector<DT>(rdz, odz[v], dz);
            }
            if constexpr (LEAN) load(token + step);
        }
    }
    if constexpr (BACK) {
        if (!a.dweight && !a.dbias) return;
        // the workgroup's sums: over the tokens that a wave had at a time, then over its waves
        const int64_t channels = (int64_t)a.groups * a.width;
        float* part = a.ws + (int64_t)tblock * 2 * channels + c0;
        __shared__ float s_part[IN_WAVE ? 4 : 1][IN_WAVE ? 64 : 1][9];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float t[8];
                if constexpr (LEAN) grads(k, v, t, false);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if constexpr (!LEAN) t[i] = k ? db[v][i] : dw[v][i];
                    if constexpr (IN_WAVE)
                        for (int off = p.lanes * p.gslots; off < 64; off *= 2) t[i] += __shfl_xor(t[i], off);
                }
                bool mine = in[v];
                if constexpr (IN_WAVE) {
                    __syncthreads();
#pragma unroll
                    for (int i = 0; i < 8; ++i) s_part[wave][lane][i] = t[i];
                    __syncthreads();
#pragma unroll
                    for (int i = 0; i < 8; ++i) t[i] = s_part[0][lane][i] + s_part[1][lane][i] + s_part[2][lane][i] + s_part[3][lane][i];
                    mine = mine && wave == 0 && lane < p.lanes * p.gslots;
                }
                if (mine)
#pragma unroll
                    for (int i = 0; i < 8; ++i) part[k * channels + 8 * vec[v] + i] = t[i];
            }
    }
}

// the workgroups' sums of the parameters' gradients, in their order; a wave takes a sixteenth of them
__global__ __launch_bounds__(1024) void k_norm_params(const float* ws, int parts, int channels, float* dweight, float* dbias)
{
    __shared__ float s[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    const int per = (parts + 15) / 16, hi = (wave + 1) * per < parts ? (wave + 1) * per : parts;
    float t = 0.0f;
    if (c < 2 * (int64_t)channels)
#pragma unroll 8
        for (int i = wave * per; i < hi; ++i) t += ws[(int64_t)i * 2 * channels + c];
    s[wave][lane] = t;
    __syncthreads();
    if (wave || c >= 2 * (int64_t)channels) return;
    t = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += s[i][lane];
    if (c < channels) {
        if (dweight) dweight[c] = t;
    } else if (dbias) {
        dbias[c - channels] = t;
    }
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

static NormPlan norm_plan(int groups, int width, int64_t tokens, bool back)
{
    const int n8 = width / 8;
    NormPlan p{};
    // One vector a lane leaves room for more waves, which the barriers of groups of several waves need (8192 tokens of
    // 4096 channels, gradient: 63 us, two vectors 70; 2000 of 8192 in fp32 49 and 58, 4096 of 8192 in bf16 73 and 70);
    // groups of up to 1024 channels stay in one wave, and more than 16 waves there are not.
    p.v = n8 <= 64 || (n8 > 128 && n8 <= 1024) ? 1 : 2;
    p.wpg = (n8 + 64 * p.v - 1) / (64 * p.v);
    p.lanes = 64;
    p.gslots = 1;
    p.tokens = 1;
    if (p.wpg == 1) {
        while (p.lanes / 2 >= n8) p.lanes /= 2;
        while (p.gslots < groups && p.gslots * p.lanes < 64) p.gslots *= 2;
        p.tokens = 64 / (p.lanes * p.gslots);
    }
    p.gblocks = (groups + p.gslots - 1) / p.gslots;
    const int64_t per = (p.wpg == 1 ? 4 : 1) * (int64_t)p.tokens; // tokens of a workgroup at a time
    int64_t blocks = (tokens + per - 1) / per;
    // Waves in all: 16384 (8192 tokens of 8 groups of 1024: 72 us, 4096 waves 75).  The gradient's sums are written once
    // for each workgroup along the tokens: 4096 (120 us; 2048 124, 8192 124), and of groups of several waves whole workgroups
    // of 16 waves on each of 256 units, which from 9 waves on is one (1999 tokens of 4104 channels in fp32, 9 waves: 28 us, 4096
    // waves in all 34; two a unit, which the registers allow, 5 us more, as the sums are written twice as often).
    int64_t most = !back ? 16384 / ((p.wpg == 1 ? 4 : p.wpg) * (int64_t)p.gblocks) : p.wpg == 1 ? 1024 / p.gblocks : 256 * (16 / p.wpg) / p.gblocks;
    if (most < 1) most = 1;
    if (blocks > most) { // as many rounds for all
        const int64_t rounds = (blocks + most - 1) / most;
        blocks = (blocks + rounds - 1) / rounds;
    }
    p.tblocks = (int)blocks;
    return p;
}

size_t norm_workspace(int groups, int width, int64_t tokens)
{
    return (size_t)norm_plan(groups, width, tokens, true).tblocks * groups * width * 8;
}

template <int DT, int ACT, bool BACK>
static hipError_t launch_norm(const NormArgs& a, hipStream_t st)
{
    const NormCall c{a, norm_plan(a.groups, a.width, a.tokens, BACK)};
    const dim3 grid((unsigned)((int64_t)c.p.gblocks * c.p.tblocks)), wg(c.p.wpg == 1 ? 256 : c.p.wpg * 64);
    if (a.tokens) {
        if (c.p.wpg == 1 && c.p.v == 1) hipLaunchKernelGGL((k_norm<DT, ACT, 1, 1, BACK>), grid, wg, 0, st, c);
        else if (c.p.v == 1) hipLaunchKernelGGL((k_norm<DT, ACT, 16, 1, BACK>), grid, wg, 0, st, c);
        else if (c.p.wpg == 1) hipLaunchKernelGGL((k_norm<DT, ACT, 1, 2, BACK>), grid, wg, 0, st, c);
        else hipLaunchKernelGGL((k_norm<DT, ACT, 16, 2, BACK>), grid, wg, 0, st, c);
    }
    if (BACK && (a.dweight || a.dbias)) {
        const int channels = a.groups * a.width;
        hipLaunchKernelGGL(k_norm_params, dim3((2 * channels + 63) / 64), dim3(1024), 0, st, a.ws, c.p.tblocks, channels, a.dweight, a.dbias);
    }
    return hipGetLastError();
}

hipError_t launch_group_norm(int dtype, int act, const NormArgs& a, hipStream_t st)
{
    return with_act(dtype, act, [&](auto dt, auto ac) { return launch_norm<decltype(dt)::value, decltype(ac)::value, false>(a, st); });
}

hipError_t launch_group_norm_backward(int dtype, int act, const NormArgs& a, hipStream_t st)
{
    return with_act(dtype, act, [&](auto dt, auto ac) { return launch_norm<decltype(dt)::value, decltype(ac)::value, true>(a, st); });
}

} // namespace ssq
