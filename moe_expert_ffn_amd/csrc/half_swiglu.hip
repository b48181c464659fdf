// SwiGLU of 16-bit rows, weighted by their route's probability, and its gradient.
//
// Section 4 of the pto-isa MegaMoE overview page without the quantisation.  The weight that section 7 applies
// when it combines a token's rows is applied here instead: the second product is linear, so the combine
// becomes a plain sum, and the gradient of a weight is a dot product with what is in registers anyway.
//   y = p silu(u) v,  silu(u) = u s,  s = 1 / (1 + exp(-u))
//   du = p dy v s (1 + u (1 - s)),  dv = p dy u s,  dp = sum_i dy u s v
// Memory bounds both, every element passing once, 16 bytes a lane.  Forwards a row is a workgroup's; backwards a wave's,
// as its dot product needs the row's lanes alone.  16384 rows of I = 2048, bf16: forwards 201 MB in 35 us, 5.7 TB/s,
// backwards 335 MB in 58 to 64 us, 5.2 to 5.8 TB/s, a copy's rate.  Five tokens: 7.3 us, the call itself.
#include "element.hpp"
#include "half.hpp"
#include "swiglu_row.hpp"

namespace megamoe {

__device__ __forceinline__ int swiglu_valid(const HalfSwigluParams &p) {
    const int v = p.cumsum[p.E - 1];
    return v < 0 ? 0 : v > p.R ? p.R : v;
}
__device__ __forceinline__ int swiglu_route(const HalfSwigluParams &p, int row) {
    const int v = p.route[row];
    return v < 0 ? 0 : v < p.R ? v : p.R - 1;
}

template <int T>
__global__ __launch_bounds__(256) void half_swiglu_kernel(HalfSwigluParams p) {
    const int row = blockIdx.x;
    if (row >= swiglu_valid(p)) return;
    const float w = p.probs ? p.probs[swiglu_route(p, row)] : 1.0f;
    const size_t in = (size_t)row * 2 * p.I;
    for (int i = threadIdx.x * 8; i < p.I; i += 256 * 8) {
        float u[8], v[8], y[8];
        Element<T>::values(Element<T>::load(p.c, in + i), u);
        Element<T>::values(Element<T>::load(p.c, in + p.I + i), v);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = w * silu_times(u[j], v[j]);
        Element<T>::store(p.y, (size_t)row * p.I + i, y);
    }
}

template <int T>
__global__ __launch_bounds__(64) void half_swiglu_grad_kernel(HalfSwigluParams p) {
    const int row = blockIdx.x;
    if (p.dprobs && threadIdx.x == 0 && p.row_of[row] < 0) p.dprobs[row] = 0.0f;  // route `row` has no row
    if (row >= swiglu_valid(p)) return;
    const int route = swiglu_route(p, row);
    const float w = p.probs ? p.probs[route] : 1.0f;
    const size_t in = (size_t)row * 2 * p.I;
    float dp = 0.0f;
    for (int i = threadIdx.x * 8; i < p.I; i += 64 * 8) {
        float u[8], v[8], d[8], du[8], dv[8];
        Element<T>::values(Element<T>::load(p.c, in + i), u);
        Element<T>::values(Element<T>::load(p.c, in + p.I + i), v);
        Element<T>::values(Element<T>::load(p.dy, (size_t)row * p.I + i), d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = 1.0f / (1.0f + __builtin_amdgcn_exp2f(u[j] * -1.4426950408889634f));
            const float su = u[j] * s, q = w * d[j];
            dp += d[j] * su * v[j];
            du[j] = q * v[j] * (s + su * (1.0f - s));
            dv[j] = q * su;
        }
        Element<T>::store(p.dc, in + i, du);
        Element<T>::store(p.dc, in + p.I + i, dv);
    }
    dp = wave_sum(dp);
    if (p.dprobs && threadIdx.x == 0) p.dprobs[route] = dp;
}

hipError_t launch_half_swiglu(const HalfSwigluParams &p, int type, bool grad, hipStream_t stream) {
    if (grad)
        hipLaunchKernelGGL((type == kBf16 ? half_swiglu_grad_kernel<kBf16> : half_swiglu_grad_kernel<kFp16>),
                           dim3(p.R), dim3(64), 0, stream, p);
    else
        hipLaunchKernelGGL((type == kBf16 ? half_swiglu_kernel<kBf16> : half_swiglu_kernel<kFp16>),
                           dim3(p.R), dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace megamoe
