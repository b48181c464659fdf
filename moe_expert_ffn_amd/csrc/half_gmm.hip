// Grouped products of fp16 or bf16 rows and weights, and their gradients (the place of GMM1 and GMM2,
// sections 3 and 5 of the pto-isa MegaMoE overview page, with unquantised experts).
//
// For the rows d of expert e's group, sums in fp32 on the matrix cores:
//   product   c[d, n] = sum_k a[d, k] w[e, n, k]      (w: rows over the reduction)
//   rows      c[d, n] = sum_k a[d, k] w[e, k, n]      (the gradient of a product's rows)
//   weights   c[e, m, n] = sum_d a[d, m] b[d, n]      (the gradient of its weights)
// The rows of a or b may be gathered: row d is row route[d] / top_k of the array.
#include "common.hpp"
#include "element.hpp"
#include "half.hpp"
#include "swiglu_row.hpp"

namespace megamoe {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

__device__ __forceinline__ int half_row_end(const HalfGmmParams &p, int e) {
    const int v = e >= 0 ? p.cumsum[e] : 0;
    return v < 0 ? 0 : v > p.R ? p.R : v;
}

__device__ __forceinline__ uint32_t half_row(const HalfGmmParams &p, bool gathered, int d) {
    if (!gathered) return d;
    const int v = p.route[d];
    const uint32_t u = v < 0 ? 0 : v < p.R ? v : p.R - 1;
    return p.top_k == 1 ? u : __umulhi(u, p.top_k_inv);
}

template <int T>
__device__ __forceinline__ v16f half_mfma(uint4 w, uint4 a, v16f acc) {
    if constexpr (T == kBf16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, w), __builtin_bit_cast(v8bf, a), acc, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, w), __builtin_bit_cast(v8h, a), acc, 0, 0, 0);
}

// A tile of 64 by 64 a workgroup, 32 by 32 a wave, 32 of the reduction at a time through LDS.
constexpr int kHalfTile = 64, kHalfK = 32, kHalfPad = 8;

template <int KIND, int T>
__global__ __launch_bounds__(256) void half_gmm_kernel(HalfGmmParams p, int row_blocks) {
    __shared__ __align__(16) uint16_t s_a[kHalfTile][kHalfK + kHalfPad], s_b[2][kHalfTile][kHalfK + kHalfPad];
    const int e = blockIdx.z, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int first = half_row_end(p, e - 1), rows = max(0, half_row_end(p, e) - first);
    const int n0 = blockIdx.y * kHalfTile;
    const bool swiglu = KIND == kHalfProduct && p.swiglu;
    const int m_end = KIND == kHalfWeights ? p.M : rows, red = KIND == kHalfWeights ? rows : p.K;
    const int wn = swiglu ? 2 * p.N : p.N;
    for (int mb = blockIdx.x; mb * kHalfTile < m_end; mb += row_blocks) {
        const int m0 = mb * kHalfTile;
        v16f acc[2] = {};
        for (int k0 = 0; k0 < red; k0 += kHalfK) {
            __syncthreads();
            // rows with the reduction along them, 8 elements a thread; or the other way round
            auto stage = [&](uint16_t(*s)[kHalfK + kHalfPad], bool along, auto address) {
                if (along) {
                    const int r = tid >> 2, k = (tid & 3) * 8;
                    *reinterpret_cast<uint4 *>(&s[r][k]) = *reinterpret_cast<const uint4 *>(address(r, k0 + k));
                } else {
                    const int k = tid >> 3, r = (tid & 7) * 8;
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (k0 + k < red) v = *reinterpret_cast<const uint4 *>(address(r, k0 + k));
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    for (int j = 0; j < 8; ++j) s[r + j][k] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
                }
            };
            if (KIND == kHalfWeights) {
                stage(s_a, false, [&](int r, int k) {
                    return p.a + (size_t)half_row(p, p.gather == 1, first + k) * p.M + min(m0 + r, p.M - 8);
                });
                stage(s_b[0], false, [&](int r, int k) {
                    return p.b + (size_t)half_row(p, p.gather == 2, first + k) * p.N + min(n0 + r, p.N - 8);
                });
            } else {
                stage(s_a, true, [&](int r, int k) {
                    return p.a + (size_t)half_row(p, p.gather == 1, first + min(m0 + r, rows - 1)) * p.K + k;
                });
                for (int f = 0; f < (swiglu ? 2 : 1); ++f)
                    stage(s_b[f], KIND == kHalfProduct, [&](int r, int k) {
                        const uint16_t *w = p.b + (size_t)e * wn * p.K;
                        return KIND == kHalfProduct ? w + (size_t)(f * p.N + min(n0 + r, p.N - 1)) * p.K + k
                                                    : w + (size_t)k * p.N + min(n0 + r, p.N - 8);
                    });
            }
            __syncthreads();
            const int r = lane & 31, g = lane >> 5;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 a = *reinterpret_cast<const uint4 *>(&s_a[(wave >> 1) * 32 + r][16 * h + 8 * g]);
                for (int f = 0; f < (swiglu ? 2 : 1); ++f)
                    acc[f] = half_mfma<T>(*reinterpret_cast<const uint4 *>(&s_b[f][(wave & 1) * 32 + r][16 * h + 8 * g]), a, acc[f]);
            }
        }
        // lane l holds row l & 31, columns 8 q + 4 (l >> 5) + 0..3
        const int row = m0 + (wave >> 1) * 32 + (lane & 31);
        if (row >= m_end) continue;
        float weight = 1.0f;
        if (swiglu && p.probs) {
            const int v = p.route[first + row];
            weight = p.probs[v < 0 ? 0 : v < p.R ? v : p.R - 1];
        }
        const size_t out = KIND == kHalfWeights ? (size_t)e * p.M + row : (size_t)first + row;
        for (int q = 0; q < 4; ++q)
            for (int v = 0; v < 4; ++v) {
                const int n = n0 + (wave & 1) * 32 + 8 * q + 4 * (lane >> 5) + v;
                if (n >= p.N) continue;
                float y = swiglu ? weight * silu_times(acc[0][4 * q + v], acc[1][4 * q + v]) : acc[0][4 * q + v];
                if (KIND == kHalfWeights && p.accumulate) y += load_value(p.c, p.c_type, out * p.N + n);
                store_value(p.c, p.c_type, out * p.N + n, y);
            }
    }
}

hipError_t launch_half_gmm(const HalfGmmParams &p, int kind, int type, int cu_count, hipStream_t stream) {
    const long long most = kind == kHalfWeights ? p.M : p.R;
    const int row_blocks = (int)((most + kHalfTile - 1) / kHalfTile < 64 ? (most + kHalfTile - 1) / kHalfTile : 64);
    const dim3 grid(row_blocks, (p.N + kHalfTile - 1) / kHalfTile, p.E);
    const bool b = type == kBf16;
    if (kind == kHalfProduct)
        hipLaunchKernelGGL((b ? half_gmm_kernel<kHalfProduct, kBf16> : half_gmm_kernel<kHalfProduct, kFp16>), grid, dim3(256), 0, stream, p, row_blocks);
    else if (kind == kHalfRows)
        hipLaunchKernelGGL((b ? half_gmm_kernel<kHalfRows, kBf16> : half_gmm_kernel<kHalfRows, kFp16>), grid, dim3(256), 0, stream, p, row_blocks);
    else
        hipLaunchKernelGGL((b ? half_gmm_kernel<kHalfWeights, kBf16> : half_gmm_kernel<kHalfWeights, kFp16>), grid, dim3(256), 0, stream, p, row_blocks);
    return hipGetLastError();
}

}  // namespace megamoe
