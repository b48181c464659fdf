// Internal launch interface of the 16-bit experts and of what training takes.
#pragma once

#include "kernels.hpp"

namespace megamoe {

// Grouped products in 16 bits and their gradients (half_gmm.hip).
enum { kHalfProduct = 0, kHalfRows = 1, kHalfWeights = 2 };
struct HalfGmmParams {
    const uint16_t *a;       // rows: [., K], of kHalfWeights [., M]
    const uint16_t *b;       // weights: [E, N (with swiglu 2 N), K], of kHalfRows [E, K, N]; of kHalfWeights rows [., N]
    const int32_t *route;    // nullable: sorted_route, for gather and probs
    const int32_t *cumsum;   // [E] inclusive row prefix over experts
    const float *probs;      // nullable, with swiglu: the weight of each route
    void *c;                 // [R, N], of kHalfWeights [E, M, N]
    int R, E, M, N, K, top_k;
    uint32_t top_k_inv;      // ceil(2^32 / top_k); 0 for top_k == 1, where
    uint32_t one_k;          // this is ~0, else 0
    int gather;              // 0, 1: row d of a is row route[d] / top_k of the array, 2: of b
    int swiglu, accumulate;
    int c_type;              // kFp32 in kHalfWeights alone
};
// ... of few rows an expert (half_few.hip)
bool half_few_ok(const HalfGmmParams &p);
hipError_t launch_half_few(const HalfGmmParams &p, int type, hipStream_t stream);
// ... of few tiles (half_small.hip)
bool half_small_ok(const HalfGmmParams &p, int kind, int cu_count);
hipError_t launch_half_small(const HalfGmmParams &p, int kind, int type, hipStream_t stream);
hipError_t launch_half_gmm(const HalfGmmParams &p, int kind, int type, int cu_count, hipStream_t stream);

// SwiGLU of 16-bit rows and its gradient (half_swiglu.hip).
struct HalfSwigluParams {
    const uint16_t *c, *dy;                // [R, 2 I], [R, I]
    const int32_t *route, *row_of, *cumsum;
    const float *probs;                    // nullable
    uint16_t *y, *dc;
    float *dprobs;                         // nullable
    int R, E, I;
};
hipError_t launch_half_swiglu(const HalfSwigluParams &p, int type, bool grad, hipStream_t stream);

// The norms around the layer and their gradients (norm.hip).
struct NormParams {
    const void *x, *rows;        // forward: [M, K], [M or R, K]
    const int32_t *row_of;       // nullable: the routes' rows (of `rows`; backwards of `h`)
    const float *w_after, *w_before;
    const void *gate;
    void *s, *r, *h;             // backwards inputs: the rows' sum, r, and the gradient of h
    const void *dr;
    void *dx, *ds, *dgate;
    float *dw_after, *dw_before;
    float *part;                 // backwards: [3][norm_grad_groups][K] sums over some tokens
    int M, K, top_k, R, gate_type, gate_rows, gate_cols, h_type;
    float alpha, eps;
};
int norm_grad_groups(int M, int K);
hipError_t launch_norm(const NormParams &p, int x_type, int rows_type, bool grad, hipStream_t stream);

// The router's gradient (route_grad.hip).
struct RouteGradParams {
    const void *logits;
    const float *bias;  // nullable
    const int32_t *expert_idx;
    const float *probs, *dprobs;
    void *dlogits;
    int M, E, top_k, renormalize;
};
hipError_t launch_route_grad(const RouteGradParams &p, int type, hipStream_t stream);

}  // namespace megamoe
