// The router: softmax top-k of a token's logits over the experts, which makes the
// expert_idx and probs that FrontReorder (section 1 of the pto-isa MegaMoE
// overview page) and Unpermute (section 7) take as given.
//
// For token t, score[e] = fp32(logit[t, e]) + bias[e].  An expert whose score is
// NaN or -inf takes no part.  The chosen experts are the top_k largest scores,
// largest first, ties to the lowest index; the weights are a softmax of the
// logits (without the bias) over the chosen experts or over all that take part.
//
// G lanes share a token and hold V consecutive experts each (G * V >= E), so the
// row is read once and stays in registers.  A score becomes an integer key that
// orders like it (0: takes no part), and each of the top_k rounds is an integer
// maximum over the lane's keys and then over the G lanes; the first lane that
// holds it clears its first copy.  Only the indices go through LDS.
#include "common.hpp"
#include "kernels.hpp"

namespace megamoe {

constexpr int kRouteBlock = 256;

template <typename T>
__device__ __forceinline__ float logit_f32(const T *p);
template <>
__device__ __forceinline__ float logit_f32<float>(const float *p) { return *p; }
template <>
__device__ __forceinline__ float logit_f32<_Float16>(const _Float16 *p) { return (float)*p; }
template <>
__device__ __forceinline__ float logit_f32<__bf16>(const __bf16 *p) { return (float)*p; }

template <int G>
__device__ __forceinline__ uint32_t group_max_u32(uint32_t v) {
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)v, off, kWave);
        v = o > v ? o : v;
    }
    return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, kWave));
    return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
    return v;
}

// exp(x - most), 1 at x = most also where both are +inf, 0 for an expert that
// takes no part (x = -inf).  The base-2 exponential is within about 1 ulp, and
// rounding its argument adds a relative error of |x - most| * 2^-24, which
// matters only where the weight itself is small.
__device__ __forceinline__ float soft_weight(float x, float most) {
    if (x == -__builtin_inff()) return 0.0f;
    if (x == most) return 1.0f;
    return __builtin_amdgcn_exp2f((x - most) * 1.4426950408889634f);
}

template <typename T, int G, int V>
__global__ __launch_bounds__(kRouteBlock) void route_topk_kernel(
    const T *__restrict__ logits, const float *__restrict__ bias, int M, int E, int top_k,
    int renormalize, int32_t *__restrict__ expert_idx, float *__restrict__ probs) {
    static_assert(G < 32, "the group mask has one bit a lane");
    constexpr int TOK = kRouteBlock / G;  // tokens of the workgroup
    extern __shared__ uint8_t s_pick[];   // [TOK][top_k] chosen experts, E <= 256
    const int gl = threadIdx.x % G, tok = threadIdx.x / G;
    const int t = blockIdx.x * TOK + tok;
    const bool live = t < M;  // the same for the G lanes of a token
    const T *row = logits + (size_t)(live ? t : M - 1) * E;

    uint32_t key[V];
    float x[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int e = gl * V + j;
        key[j] = 0;
        x[j] = -__builtin_inff();
        if (e < E) {
            const float l = logit_f32(row + e);
            // + 0: -0 and +0 are one score
            const float s = (bias ? l + bias[e] : l) + 0.0f;
            if (s > -__builtin_inff()) {  // false for NaN too
                const uint32_t u = __float_as_uint(s);
                key[j] = (u >> 31) ? ~u : (u | 0x80000000u);
                x[j] = l;
            }
        }
    }

    uint8_t *pick = s_pick + tok * top_k;
    int n = 0;  // experts chosen
    const int lane = threadIdx.x & (kWave - 1);
    for (; n < top_k; ++n) {
        uint32_t mine = key[0];
#pragma unroll
        for (int j = 1; j < V; ++j) mine = key[j] > mine ? key[j] : mine;
        const uint32_t best = group_max_u32<G>(mine);
        if (best == 0) break;  // no expert left: the same for the G lanes of a token
        const uint64_t have = __ballot(mine == best);
        // lanes of this token that hold the best key; the lowest one wins
        const uint32_t group = (uint32_t)(have >> (lane & ~(G - 1))) & ((1u << G) - 1);
        if (__builtin_ctz(group) == gl) {
            int at = 0;
#pragma unroll
            for (int j = V - 1; j >= 0; --j) at = key[j] == best ? j : at;
#pragma unroll
            for (int j = 0; j < V; ++j) key[j] = j == at ? 0 : key[j];
            pick[n] = (uint8_t)(gl * V + at);
        }
    }
    __syncthreads();

    float most = -__builtin_inff(), total = 0.0f;
    if (renormalize) {
        for (int i = gl; i < n; i += G) most = fmaxf(most, logit_f32(row + pick[i]));
        most = group_max<G>(most);
        for (int i = gl; i < n; i += G) total += soft_weight(logit_f32(row + pick[i]), most);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) most = fmaxf(most, x[j]);
        most = group_max<G>(most);
#pragma unroll
        for (int j = 0; j < V; ++j) total += soft_weight(x[j], most);
    }
    total = group_sum<G>(total);
    if (!live) return;
    for (int i = gl; i < top_k; i += G) {
        const size_t o = (size_t)t * top_k + i;
        expert_idx[o] = i < n ? (int)pick[i] : -1;
        probs[o] = i < n ? soft_weight(logit_f32(row + pick[i]), most) / total : 0.0f;
    }
}

template <typename T>
static hipError_t launch_typed(const void *logits, const float *bias, int M, int E, int top_k,
                               int renormalize, int32_t *expert_idx, float *probs,
                               hipStream_t stream) {
#define MEGAMOE_ROUTE(G, V)                                                                     \
    hipLaunchKernelGGL((route_topk_kernel<T, G, V>), dim3((M + kRouteBlock / G - 1) / (kRouteBlock / G)), \
                       dim3(kRouteBlock), kRouteBlock / G * top_k, stream,                        \
                       static_cast<const T *>(logits), bias, M, E, top_k, renormalize, expert_idx, \
                       probs)
    if (E <= 64) MEGAMOE_ROUTE(16, 4);
    else if (E <= 128) MEGAMOE_ROUTE(16, 8);
    else MEGAMOE_ROUTE(16, 16);
#undef MEGAMOE_ROUTE
    return hipGetLastError();
}

hipError_t launch_route(const void *logits, int type, const float *bias, int M, int E, int top_k,
                        int renormalize, int32_t *expert_idx, float *probs, hipStream_t stream) {
    switch (type) {
        case kFp32:
            return launch_typed<float>(logits, bias, M, E, top_k, renormalize, expert_idx, probs,
                                       stream);
        case kFp16:
            return launch_typed<_Float16>(logits, bias, M, E, top_k, renormalize, expert_idx, probs,
                                          stream);
        default:
            return launch_typed<__bf16>(logits, bias, M, E, top_k, renormalize, expert_idx, probs,
                                        stream);
    }
}

}  // namespace megamoe
