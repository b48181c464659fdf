// The router: softmax top-k of a token's logits over the experts, which makes the
// expert_idx and probs that FrontReorder (section 1 of the pto-isa MegaMoE
// overview page) and Unpermute (section 7) take as given.
//
// For token t, score[e] = fp32(logit[t, e]) + bias[e].  An expert whose score is
// NaN or -inf takes no part.  The chosen experts are the top_k largest scores,
// largest first, ties to the lowest index; the weights are a softmax of the
// logits (without the bias) over the chosen experts or over all that take part.
//
// 16 lanes share a token and hold V consecutive experts each (16 V >= E), so the row
// is read once, 16 bytes at a time where rows are aligned, and stays in registers; a
// group goes on to further tokens and keeps the bias.  A score becomes an integer
// key that orders like it (0: takes no part), and each of the top_k rounds is an
// integer maximum over the lane's keys and then, by rotations inside the row of 16
// lanes, over the group; the first lane that holds it clears its first copy.  Only
// the indices go through LDS.  Instruction issue bounds the kernel: 64 lanes to a
// token would take half as long again in lane exchanges, one lane to many experts
// more in clearing.  32768 tokens of 256 bf16 logits, top_k = 8: 14 us, with a
// bias and all experts' weights 16 (64 lanes to a token: 53); one token 3.0.  The next
// token's logits asked for early, or more waves with fewer registers, gave nothing.
#include "common.hpp"
#include "kernels.hpp"

namespace megamoe {

constexpr int kRouteBlock = 256;
constexpr int kRouteLanes = 16;                         // of a token: a DPP row
constexpr int kRouteTokens = kRouteBlock / kRouteLanes; // of a workgroup at a time

__device__ __forceinline__ float logit_f32(float v) { return v; }
__device__ __forceinline__ float logit_f32(_Float16 v) { return (float)v; }
__device__ __forceinline__ float logit_f32(__bf16 v) { return (float)v; }

// The value of the lane N places on in the row of 16 lanes.
template <int N>
__device__ __forceinline__ uint32_t row_rotate(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xf, 0xf, false);
}
template <int N>
__device__ __forceinline__ float row_rotate(float v) {
    return __uint_as_float(row_rotate<N>(__float_as_uint(v)));
}
// Over the row, in every lane of it.
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
    uint32_t o = row_rotate<8>(v);
    v = o > v ? o : v;
    o = row_rotate<4>(v);
    v = o > v ? o : v;
    o = row_rotate<2>(v);
    v = o > v ? o : v;
    o = row_rotate<1>(v);
    return o > v ? o : v;
}
__device__ __forceinline__ float row_max(float v) {
    v = fmaxf(v, row_rotate<8>(v));
    v = fmaxf(v, row_rotate<4>(v));
    v = fmaxf(v, row_rotate<2>(v));
    return fmaxf(v, row_rotate<1>(v));
}
__device__ __forceinline__ float row_sum(float v) {
    v += row_rotate<8>(v);
    v += row_rotate<4>(v);
    v += row_rotate<2>(v);
    return v + row_rotate<1>(v);
}

// exp(x - most), 1 at x = most also where both are +inf, 0 for an expert that
// takes no part (x = -inf).  The base-2 exponential is within about 1 ulp, and
// rounding its argument adds a relative error of |x - most| * 2^-24, which
// matters only where the weight itself is small.
__device__ __forceinline__ float soft_weight(float x, float most) {
    const float w = x == most ? 1.0f : __builtin_amdgcn_exp2f((x - most) * 1.4426950408889634f);
    return x == -__builtin_inff() ? 0.0f : w;
}

// VEC: rows start on 16 bytes and hold a multiple of V experts
template <typename T, int V, bool VEC>
__global__ __launch_bounds__(kRouteBlock) void route_topk_kernel(
    const T *__restrict__ logits, const float *__restrict__ bias, int M, int E, int top_k,
    int renormalize, int32_t *__restrict__ expert_idx, float *__restrict__ probs) {
    extern __shared__ uint8_t s_pick[];  // [kRouteTokens][top_k] chosen experts, E <= 256
    const int gl = threadIdx.x % kRouteLanes, tok = threadIdx.x / kRouteLanes;
    const int lane = threadIdx.x & (kWave - 1);
    uint8_t *pick = s_pick + tok * top_k;
    const float none = -__builtin_inff();
    const bool mine_in = gl * V < E;  // with VEC all of the lane's experts exist, or none

    float add[V] = {};
    if (bias) {
        if constexpr (VEC) {
            typedef float word __attribute__((ext_vector_type(4)));
            if (mine_in)
#pragma unroll
                for (int j = 0; j < V; j += 4)
                    *reinterpret_cast<word *>(add + j) = *reinterpret_cast<const word *>(bias + gl * V + j);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) add[j] = gl * V + j < E ? bias[gl * V + j] : 0.0f;
        }
    }

    for (int t = blockIdx.x * kRouteTokens + tok; t < M; t += gridDim.x * kRouteTokens) {
        const T *row = logits + (size_t)t * E;
        T raw[V];
        if constexpr (VEC) {
            constexpr int W = V * sizeof(T) < 16 ? V * sizeof(T) : 16;
            typedef uint32_t word __attribute__((ext_vector_type(W / 4)));
#pragma unroll
            for (int j = 0; j < (int)(V * sizeof(T) / W); ++j)
                if (mine_in)
                    *(reinterpret_cast<word *>(raw) + j) =
                        __builtin_nontemporal_load(reinterpret_cast<const word *>(row + gl * V) + j);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (gl * V + j < E) raw[j] = row[gl * V + j];
        }
        uint32_t key[V];
        float x[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const bool in = VEC ? mine_in : gl * V + j < E;
            const float l = in ? logit_f32(raw[j]) : none;
            const float s = (l + add[j]) + 0.0f;  // + 0: -0 and +0 are one score
            const bool part = s > none;  // false for NaN too
            const uint32_t u = __float_as_uint(s);
            key[j] = part ? u ^ ((uint32_t)((int)u >> 31) | 0x80000000u) : 0u;
            x[j] = part ? l : none;
        }

        int n = 0;  // experts chosen
        for (; n < top_k; ++n) {
            uint32_t mine = key[0];
#pragma unroll
            for (int j = 1; j < V; ++j) mine = key[j] > mine ? key[j] : mine;
            const uint32_t best = row_max(mine);
            if (best == 0) break;  // no expert left: the same for the lanes of a token
            const uint64_t have = __ballot(mine == best);
            // lanes of this token that hold the best key; the lowest one wins
            const uint32_t group = (uint32_t)(have >> (lane & ~(kRouteLanes - 1))) & 0xffffu;
            if (__builtin_ctz(group) == gl) {
                int at = 0;
#pragma unroll
                for (int j = V - 1; j >= 0; --j) at = key[j] == best ? j : at;
#pragma unroll
                for (int j = 0; j < V; ++j) key[j] = j == at ? 0 : key[j];
                pick[n] = (uint8_t)(gl * V + at);
            }
        }
        // a token's lanes are of one wave: its picks are there once the wave's LDS writes are
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();

        // each lane has the picks gl, gl + 16, ...; their logits are in the caches
        float most = none, total = 0.0f;
        const float first = gl < n ? logit_f32(row[pick[gl]]) : none;
        if (renormalize) {
            for (int i = gl; i < n; i += kRouteLanes)
                most = fmaxf(most, i == gl ? first : logit_f32(row[pick[i]]));
            most = row_max(most);
            for (int i = gl; i < n; i += kRouteLanes)
                total += soft_weight(i == gl ? first : logit_f32(row[pick[i]]), most);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) most = fmaxf(most, x[j]);
            most = row_max(most);
#pragma unroll
            for (int j = 0; j < V; ++j) total += soft_weight(x[j], most);
        }
        total = row_sum(total);
        for (int i = gl; i < top_k; i += kRouteLanes) {
            const size_t o = (size_t)t * top_k + i;
            expert_idx[o] = i < n ? (int)pick[i] : -1;
            probs[o] = i < n ? soft_weight(i == gl ? first : logit_f32(row[pick[i]]), most) / total : 0.0f;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();  // the next token's picks come after these reads
    }
}

template <typename T>
static hipError_t launch_typed(const void *logits, const float *bias, int M, int E, int top_k,
                               int renormalize, int32_t *expert_idx, float *probs,
                               hipStream_t stream) {
    // up to 8 workgroups a CU, each with several rounds of tokens
    const int rounds = (M + kRouteTokens - 1) / kRouteTokens;
    const dim3 grid(rounds < 2048 ? rounds : 2048);
#define MEGAMOE_ROUTE(V, VEC)                                                                   \
    hipLaunchKernelGGL((route_topk_kernel<T, V, VEC>), grid, dim3(kRouteBlock),                 \
                       kRouteTokens * top_k, stream, static_cast<const T *>(logits), bias, M, E, \
                       top_k, renormalize, expert_idx, probs)
    const bool rows16 = (size_t)E * sizeof(T) % 16 == 0;
    if (E <= 64) {
        if (rows16 && E % 4 == 0) MEGAMOE_ROUTE(4, true);
        else MEGAMOE_ROUTE(4, false);
    } else if (E <= 128) {
        if (rows16 && E % 8 == 0) MEGAMOE_ROUTE(8, true);
        else MEGAMOE_ROUTE(8, false);
    } else {
        if (rows16 && E % 16 == 0) MEGAMOE_ROUTE(16, true);
        else MEGAMOE_ROUTE(16, false);
    }
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
