// Grouped product of MXFP4 rows and MXFP4 weights (the place of GMM1 and GMM2,
// sections 3 and 5 of the pto-isa MegaMoE overview page, with 4-bit experts).
//
// For every row of expert e's group, p[n] = sum_k a[k] * w[e][n][k] over the
// values that codes and block scales stand for, in fp32 on the matrix cores:
// v_mfma_scale_f32_16x16x128_f8f6f4 takes 32 codes of a lane (one block) with
// their scale byte.  GMM1 ends in SwiGLU: column n meets column N + n in the same
// lane's accumulators, and silu(p[n]) * p[N + n] goes out as bf16; GMM2's p goes
// out as fp16.
#include "common.hpp"
#include "kernels.hpp"
#include "swiglu_row.hpp"

namespace megamoe {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

// 16 x 16 x 128 with weights as the first operand: lane l holds output row l & 15
// and the columns 4 (l >> 4) + 0..3.  Of either operand lane l has row l & 15, the
// codes of block l >> 4 and, in the low byte, their scale.
__device__ __forceinline__ v4f mx_mfma(v4i w, int ws, v4i a, int as, v4f acc) {
    const v8i w8 = {w[0], w[1], w[2], w[3], 0, 0, 0, 0}, a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w8, a8, acc, 4, 4, 0, ws, 0, as);
}

// fp32 -> the output element, round to nearest even
template <bool SWIGLU>
__device__ __forceinline__ uint16_t mx_out(float v) {
    return SWIGLU ? (uint16_t)(f2bf_pk(v, 0.0f) & 0xffffu) : f2h(v);
}

// first row and row count of expert e's group, within [0, R]
__device__ __forceinline__ int mx_row_end(const MxGmmParams &p, int e) {
    const int v = e >= 0 ? p.cumsum[e] : 0;
    return v < 0 ? 0 : v > p.R ? p.R : v;
}
__device__ __forceinline__ size_t mx_a_row(const MxGmmParams &p, int d) {
    if (!p.a_route) return d;
    const int r = p.a_route[d];
    return (r < 0 ? 0 : r < p.R ? r : p.R - 1) / p.a_div;
}

// ---------------------------------------------------------------------------
// Few rows per expert: the product streams weights.  One workgroup per expert
// with rows and 16 output columns; its waves split the reduction, each reading
// weights and rows straight into fragments, and the partial sums are added in
// wave order.
constexpr int kMxWaves = 8;
constexpr int kMxThreads = kMxWaves * kWave;

template <bool SWIGLU, int RB>
__global__ __launch_bounds__(kMxThreads) void mxfp4_gmm_stream_kernel(MxGmmParams p) {
    constexpr int F = SWIGLU ? 2 : 1;  // weight fragments of a column group
    constexpr int U = RB > 2 ? 2 : 4;  // K slices a wave has in flight
    __shared__ int s_e;
    __shared__ v4f s_part[kMxWaves][RB * F][kWave];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid >> 6;

    if (tid < kWave) {  // the expert of this workgroup: the blockIdx.y-th with rows
        int any[4], sum = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int e = tid * 4 + j;
            any[j] = e < p.E && mx_row_end(p, e) > mx_row_end(p, e - 1);
            sum += any[j];
        }
        int run = wave_inclusive_scan(sum) - sum;
        if (tid == 0) s_e = -1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (any[j] && run == (int)blockIdx.y) s_e = tid * 4 + j;
            run += any[j];
        }
    }
    __syncthreads();
    const int e = s_e;
    if (e < 0) return;
    const int row0 = mx_row_end(p, e - 1), rows = mx_row_end(p, e) - row0;

    const int ns = p.Kred / 128, n0 = blockIdx.x * 16;
    const int s0 = wave * ns / kMxWaves, s1 = (wave + 1) * ns / kMxWaves;
    const size_t qrow = p.Kred / 2, srow = p.Kred / 32;
    const int r = lane & 15, g = lane >> 4;
    const uint8_t *wq[F], *wsc[F];
#pragma unroll
    for (int f = 0; f < F; ++f) {
        const size_t n = (size_t)e * p.N * F + f * p.N + n0 + r;
        wq[f] = p.w + n * qrow + g * 16;
        wsc[f] = p.w_scale + n * srow + g;
    }
    const v4i zero = {0, 0, 0, 0};

    for (int r0 = 0; r0 < rows; r0 += 16 * RB) {
        const uint8_t *aq[RB], *asc[RB];
        bool in[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            in[b] = r0 + 16 * b + r < rows;
            const size_t d = mx_a_row(p, row0 + (in[b] ? r0 + 16 * b + r : r0));
            aq[b] = p.a + d * qrow + g * 16;
            asc[b] = p.a_scale + d * srow + g;
        }
        v4f acc[RB][F] = {};
        v4i fw[U][F], fa[U][RB];
        int cw[U][F], ca[U][RB];
        auto load = [&](int s) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
#pragma unroll
                for (int f = 0; f < F; ++f) {
                    fw[i][f] = zero;
                    cw[i][f] = 0;
                    if (s + i < s1) {
                        fw[i][f] = __builtin_nontemporal_load(
                            reinterpret_cast<const v4i *>(wq[f] + (size_t)(s + i) * 64));
                        cw[i][f] = wsc[f][(s + i) * 4];
                    }
                }
#pragma unroll
                for (int b = 0; b < RB; ++b) {
                    fa[i][b] = zero;
                    ca[i][b] = 0;
                    if (s + i < s1 && in[b]) {
                        fa[i][b] = *reinterpret_cast<const v4i *>(aq[b] + (size_t)(s + i) * 64);
                        ca[i][b] = asc[b][(s + i) * 4];
                    }
                }
            }
        };
        load(s0);
        for (int s = s0; s < s1; s += U) {
            v4i bw[U][F], ba[U][RB];
            int sw[U][F], sa[U][RB];
#pragma unroll
            for (int i = 0; i < U; ++i) {
#pragma unroll
                for (int f = 0; f < F; ++f) {
                    bw[i][f] = fw[i][f];
                    sw[i][f] = cw[i][f];
                }
#pragma unroll
                for (int b = 0; b < RB; ++b) {
                    ba[i][b] = fa[i][b];
                    sa[i][b] = ca[i][b];
                }
            }
            if (s + U < s1) load(s + U);
#pragma unroll
            for (int i = 0; i < U; ++i)
#pragma unroll
                for (int b = 0; b < RB; ++b)
#pragma unroll
                    for (int f = 0; f < F; ++f)
                        if (s + i < s1) acc[b][f] = mx_mfma(bw[i][f], sw[i][f], ba[i][b], sa[i][b], acc[b][f]);
        }
        __syncthreads();  // the last pass's sums have been read
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int f = 0; f < F; ++f) s_part[wave][b * F + f][lane] = acc[b][f];
        __syncthreads();
        for (int i = tid; i < RB * 256; i += kMxThreads) {  // row i / 16, column i % 16
            const int row = i >> 4, col = i & 15;
            if (r0 + row >= rows) break;
            const int at = (row & 15) + 16 * (col >> 2), b = row >> 4;
            float sum[F];
#pragma unroll
            for (int f = 0; f < F; ++f) {
                sum[f] = 0.0f;
#pragma unroll
                for (int w = 0; w < kMxWaves; ++w)
                    sum[f] += reinterpret_cast<const float *>(&s_part[w][b * F + f][at])[col & 3];
            }
            const float v = SWIGLU ? silu_times(sum[0], sum[F - 1]) : sum[0];
            p.c[(size_t)(row0 + r0 + row) * p.N + n0 + col] = mx_out<SWIGLU>(v);
        }
    }
}

template <bool SWIGLU>
static void launch_stream(const MxGmmParams &p, hipStream_t stream) {
    const dim3 grid(p.N / 16, p.E < p.R ? p.E : p.R), block(kMxThreads);
    const int mean = (p.R + p.E - 1) / p.E;
    if (mean <= 8) hipLaunchKernelGGL((mxfp4_gmm_stream_kernel<SWIGLU, 1>), grid, block, 0, stream, p);
    else if (mean <= 24) hipLaunchKernelGGL((mxfp4_gmm_stream_kernel<SWIGLU, 2>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((mxfp4_gmm_stream_kernel<SWIGLU, 4>), grid, block, 0, stream, p);
}

hipError_t launch_mxfp4_gmm(const MxGmmParams &p, bool swiglu, int cu_count, hipStream_t stream) {
    (void)cu_count;
    if (swiglu) launch_stream<true>(p, stream);
    else launch_stream<false>(p, stream);
    return hipGetLastError();
}

}  // namespace megamoe
