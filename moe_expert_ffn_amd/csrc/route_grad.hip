// The router's gradient: that of the softmax weights of route.hip with respect to the logits.
//
// With w the softmax over the experts that take part (those chosen, with renormalize), g[e] the gradient of
// expert e's weight (0 where it was not chosen) and dot = sum_e w[e] g[e]:
//   dlogit[e] = w[e] (g[e] - dot), 0 where e takes no part
// With renormalize w is probs, and the logits are not read.
#include "element.hpp"
#include "half.hpp"

namespace megamoe {

constexpr int kRgBlock = 256;

// Over the lanes of a token, in every one of them.
__device__ __forceinline__ float group_sum(float v, int lanes) {
    for (int off = lanes >> 1; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
    return v;
}

// The logit of an expert that takes part, else -inf.
__device__ __forceinline__ float rg_part(float x, float bias) { return x + bias > -INFINITY ? x : -INFINITY; }
__device__ __forceinline__ float rg_exp(float x, float most) {
    if (!(x > -INFINITY)) return 0.0f;
    return x == most ? 1.0f : __builtin_amdgcn_exp2f((x - most) * 1.4426950408889634f);
}

// `lanes` lanes (a power of two) to a token: lane j has its slot j and eight experts: with PIECES 8 j + 0..7, so that a row is
// read and written 16 bytes at a time, else j + lanes v, for rows that are not whole pieces of 8.  What the slots add to their experts meets the experts in LDS; a slot whose expert an
// earlier slot names leaves its part to that one, so that the order of the sum is fixed.
// 32768 tokens of 256 bf16 logits, 8 slots: 37 MB in 12.9 us, 2.9 TB/s; of 255 17.4 (a wave to a token: 50).  Instructions bound it, not memory (7.4 us):
// VALUs are active in 57% of the cycles, the shuffles over the slots among them.  A wave to a token, four experts a lane and
// each looking through all slots, took 29.7.  128 tokens of 32 fp32 logits: 7.1 us, the call itself.
template <int T, bool PIECES>
__global__ __launch_bounds__(kRgBlock) void route_grad_kernel(RouteGradParams p, int lanes) {
    __shared__ __align__(16) float s_gain[kRgBlock * 8];
    const int tid = threadIdx.x, j = tid & (lanes - 1), group = tid / lanes;
    const size_t t = (size_t)blockIdx.x * (kRgBlock / lanes) + group;
    const bool here = t < (size_t)p.M, mine = here && (PIECES ? 8 * j : j) < p.E;
    float *gain = s_gain + group * lanes * 8;
    float x[8];
    typename Element<T>::Raw raw;
    if (mine && !p.renormalize) {
        if constexpr (PIECES) {
            raw = Element<T>::load_nt(p.logits, t * p.E + 8 * j);
        } else {
#pragma unroll
            for (int v = 0; v < 8; ++v) x[v] = Element<T>::load1(p.logits, t * p.E + min(j + lanes * v, p.E - 1));
        }
    }
    int id = -1;
    float w = 0.0f, g = 0.0f;
    if (here && j < p.top_k) {
        id = p.expert_idx[t * p.top_k + j];
        w = p.probs[t * p.top_k + j];
        g = p.dprobs[t * p.top_k + j];
    }
    if (id < 0 || id >= p.E) {
        id = -1;
        w = g = 0.0f;
    }
#pragma unroll
    for (int v = 0; v < 8; v += 4) *reinterpret_cast<float4 *>(gain + 8 * j + v) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float dot = group_sum(w * g, lanes);
    const float part = p.renormalize ? w * (g - dot) : g;
    float total = 0.0f;
    bool first = id >= 0;
    for (int s = 0; s < p.top_k; ++s) {
        const int at = (tid & (kWave - 1) & ~(lanes - 1)) + s;
        const int other = __shfl(id, at, kWave);
        const float v = __shfl(part, at, kWave);
        if (other == id) {
            total += v;
            first = first && s >= j;
        }
    }
    if (first) gain[id] = total;
    __syncthreads();
    float y[8];
    if constexpr (PIECES) {
#pragma unroll
        for (int v = 0; v < 8; v += 4) {
            const float4 q = *reinterpret_cast<const float4 *>(gain + 8 * j + v);
            y[v] = q.x;
            y[v + 1] = q.y;
            y[v + 2] = q.z;
            y[v + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int v = 0; v < 8; ++v) y[v] = gain[j + lanes * v];
    }
    if (!p.renormalize) {
        float most = -INFINITY, sum = 0.0f;
        if (mine) {
            float b[8] = {};
            if constexpr (PIECES) {
                Element<T>::values(raw, x);
                if (p.bias) Element<kFp32>::values(Element<kFp32>::load(p.bias, 8 * j), b);
            } else if (p.bias) {
#pragma unroll
                for (int v = 0; v < 8; ++v) b[v] = p.bias[min(j + lanes * v, p.E - 1)];
            }
#pragma unroll
            for (int v = 0; v < 8; ++v)
                x[v] = PIECES || j + lanes * v < p.E ? rg_part(x[v], b[v]) : -INFINITY;
        } else {
#pragma unroll
            for (int v = 0; v < 8; ++v) x[v] = -INFINITY;
        }
#pragma unroll
        for (int v = 0; v < 8; ++v) most = fmaxf(most, x[v]);
        for (int off = lanes >> 1; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor(most, off, kWave));
#pragma unroll
        for (int v = 0; v < 8; ++v) {
            x[v] = rg_exp(x[v], most);
            sum += x[v];
        }
        sum = group_sum(sum, lanes);
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int v = 0; v < 8; ++v) y[v] = x[v] == 0.0f ? 0.0f : x[v] * inv * (y[v] - dot);
    }
    if (!mine) return;
    if constexpr (PIECES) {
        Element<T>::store_nt(p.dlogits, t * p.E + 8 * j, y);
    } else {
#pragma unroll
        for (int v = 0; v < 8; ++v)
            if (j + lanes * v < p.E) Element<T>::store1(p.dlogits, t * p.E + j + lanes * v, y[v]);
    }
}

// More than 64 slots, of which no lane has one each: a wave to a token, lane l with the experts l + 64 v, all of them
// looking through all slots.
template <int T>
__global__ __launch_bounds__(64) void route_grad_any_kernel(RouteGradParams p) {
    const size_t t = blockIdx.x;
    const int lane = threadIdx.x;
    float x[4], gain[4] = {}, most = -INFINITY, dot = 0.0f, sum = 0.0f;
    for (int s = 0; s < p.top_k; ++s) {
        const int id = p.expert_idx[t * p.top_k + s];
        if (id >= 0 && id < p.E) dot += p.probs[t * p.top_k + s] * p.dprobs[t * p.top_k + s];
    }
    for (int s = 0; s < p.top_k; ++s) {
        const int id = p.expert_idx[t * p.top_k + s];
        const float w = p.probs[t * p.top_k + s], g = p.dprobs[t * p.top_k + s];
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if (id >= 0 && id < p.E && id == lane + 64 * v) gain[v] += p.renormalize ? w * (g - dot) : g;
    }
    if (!p.renormalize) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int e = lane + 64 * v;
            x[v] = e < p.E ? rg_part(Element<T>::load1(p.logits, t * p.E + e), p.bias ? p.bias[e] : 0.0f) : -INFINITY;
            most = fmaxf(most, x[v]);
        }
        most = wave_max(most);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            x[v] = rg_exp(x[v], most);
            sum += x[v];
        }
        sum = wave_sum(sum);
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int v = 0; v < 4; ++v) gain[v] = x[v] == 0.0f ? 0.0f : x[v] * inv * (gain[v] - dot);
    }
#pragma unroll
    for (int v = 0; v < 4; ++v)
        if (lane + 64 * v < p.E) Element<T>::store1(p.dlogits, t * p.E + lane + 64 * v, gain[v]);
}

template <int T>
static void rg_launch(const RouteGradParams &p, hipStream_t stream) {
    if (p.top_k > kWave) {
        hipLaunchKernelGGL(route_grad_any_kernel<T>, dim3(p.M), dim3(64), 0, stream, p);
        return;
    }
    int lanes = 1;
    while (8 * lanes < p.E || lanes < p.top_k) lanes *= 2;
    const int tokens = kRgBlock / lanes;
    hipLaunchKernelGGL((p.E % 8 == 0 ? route_grad_kernel<T, true> : route_grad_kernel<T, false>),
                       dim3((p.M + tokens - 1) / tokens), dim3(kRgBlock), 0, stream, p, lanes);
}

hipError_t launch_route_grad(const RouteGradParams &p, int type, hipStream_t stream) {
    if (type == kFp32) rg_launch<kFp32>(p, stream);
    else if (type == kFp16) rg_launch<kFp16>(p, stream);
    else rg_launch<kBf16>(p, stream);
    return hipGetLastError();
}

}  // namespace megamoe
