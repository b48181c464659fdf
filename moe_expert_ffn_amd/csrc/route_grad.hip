// The router's gradient: that of the softmax weights of route.hip with respect to the logits.
//
// With w the softmax over the experts that take part (those chosen, with renormalize), g[e] the gradient of
// expert e's weight (0 where it was not chosen) and dot = sum_e w[e] g[e]:
//   dlogit[e] = w[e] (g[e] - dot), 0 where e takes no part
#include "element.hpp"
#include "half.hpp"

namespace megamoe {

template <int T>
__global__ __launch_bounds__(64) void route_grad_kernel(RouteGradParams p) {
    const size_t t = blockIdx.x;
    const int lane = threadIdx.x;
    float x[4], gain[4] = {}, part[4] = {};
    float most = -INFINITY;
    if (!p.renormalize) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int e = lane + 64 * j;
            x[j] = -INFINITY;
            if (e < p.E) {
                const float v = Element<T>::load1(p.logits, t * p.E + e);
                if (v + (p.bias ? p.bias[e] : 0.0f) > -INFINITY) x[j] = v;
            }
            most = fmaxf(most, x[j]);
        }
        most = wave_max(most);
    }
    float dot = 0.0f;
    for (int s = 0; s < p.top_k; ++s) {
        const int id = p.expert_idx[t * p.top_k + s];
        if (id < 0 || id >= p.E) continue;
        const float w = p.probs[t * p.top_k + s], g = p.dprobs[t * p.top_k + s];
        dot += w * g;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (id == lane + 64 * j) {
                gain[j] += p.renormalize ? w * g : g;
                part[j] += w;
            }
    }
    if (!p.renormalize) {
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            part[j] = x[j] == most ? 1.0f : __builtin_amdgcn_exp2f((x[j] - most) * 1.4426950408889634f);
            if (!(x[j] > -INFINITY)) part[j] = 0.0f;
            sum += part[j];
        }
        sum = wave_sum(sum);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            part[j] = sum > 0.0f ? part[j] / sum : 0.0f;
            gain[j] *= part[j];
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int e = lane + 64 * j;
        if (e < p.E) Element<T>::store1(p.dlogits, t * p.E + e, part[j] == 0.0f ? 0.0f : gain[j] - part[j] * dot);
    }
}

hipError_t launch_route_grad(const RouteGradParams &p, int type, hipStream_t stream) {
    const dim3 grid(p.M), block(64);
    if (type == kFp32) hipLaunchKernelGGL(route_grad_kernel<kFp32>, grid, block, 0, stream, p);
    else if (type == kFp16) hipLaunchKernelGGL(route_grad_kernel<kFp16>, grid, block, 0, stream, p);
    else hipLaunchKernelGGL(route_grad_kernel<kBf16>, grid, block, 0, stream, p);
    return hipGetLastError();
}

}  // namespace megamoe
