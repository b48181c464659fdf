// What the two kernels of the 16-bit products share.
#pragma once

#include "element.hpp"
#include "half.hpp"

namespace megamoe {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
constexpr int kHgE = 256;

__device__ __forceinline__ int hg_row_end(const HalfGmmParams &p, int e) {
    const int v = e >= 0 ? p.cumsum[e] : 0;
    return v < 0 ? 0 : v > p.R ? p.R : v;
}

// A sorted route and its token: what lies past the valid rows stays in bounds.
__device__ __forceinline__ uint32_t hg_route(const HalfGmmParams &p, int v) { return min(max(v, 0), p.R - 1); }
__device__ __forceinline__ uint32_t hg_token(const HalfGmmParams &p, int v) {
    const uint32_t u = hg_route(p, v);
    return __umulhi(u, p.top_k_inv) + (u & p.one_k);
}

// silu(u) * g for a result that is rounded to 16 bits: the reciprocal's last ulp is not corrected
__device__ __forceinline__ float hg_silu_times(float u, float g) {
    const float d = __builtin_amdgcn_exp2f(u * -1.4426950408889634f) + 1.0f;
    return u * __builtin_amdgcn_rcpf(d) * g;
}

}  // namespace megamoe
