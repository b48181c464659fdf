// The norms after and before the layer with what lies between them, and their gradients.
//
// For token t, in fp32:
//   s = the rows of its routes, summed (section 7 of the pto-isa MegaMoE overview page, without weights), or row t
//   n = s rstd(s) w_after, or s
//   r = x + alpha gate n, or x
//   h = r rstd(r) w_before
// with rstd(v) = 1 / sqrt(mean v^2 + eps).  Backwards, with G the gradient of r, e = dh w_before and f = alpha gate G w_after:
//   G = dr + rstd(r) (e - r rstd(r)^2 mean(e r)),  dx = G
//   ds = rstd(s) (f - s rstd(s)^2 mean(f s)), or alpha gate G
//   dw_before = sum_t dh r rstd(r),  dw_after = sum_t alpha gate G s rstd(s),  dgate = alpha G n, summed where the gate is broadcast
#include "element.hpp"
#include "half.hpp"

namespace megamoe {

constexpr int kNormSlots = 8;  // rows of a token asked for at a time

// Eight columns of token t: row t, or the sum of its routes' rows (slots in order).
template <int T>
__device__ __forceinline__ void norm_rows(const void *rows, const int32_t *row_of, size_t t, int top_k, int R, int K,
                                          int col, float (&v)[8]) {
    if (!row_of) {
        Element<T>::values(Element<T>::load(rows, t * K + col), v);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    for (int s0 = 0; s0 < top_k; s0 += kNormSlots) {
        int d[kNormSlots];
        typename Element<T>::Raw raw[kNormSlots];
#pragma unroll
        for (int u = 0; u < kNormSlots; ++u) {
            d[u] = s0 + u < top_k ? row_of[t * top_k + s0 + u] : -1;
            if (d[u] >= R) d[u] = -1;
        }
#pragma unroll
        for (int u = 0; u < kNormSlots; ++u)
            if (d[u] >= 0) raw[u] = Element<T>::load_nt(rows, (size_t)d[u] * K + col);
#pragma unroll
        for (int u = 0; u < kNormSlots; ++u) {
            if (d[u] < 0) continue;
            float x[8];
            Element<T>::values(raw[u], x);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += x[j];
        }
    }
}

// The sum of N values each over the threads of a row (whole waves), in every one of them.
template <int N>
__device__ __forceinline__ void norm_sum(float (&v)[N], float *lds, int waves) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if (waves == 1) return;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) lds[wave * N + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = 0.0f;
        for (int w = 0; w < waves; ++w) v[i] += lds[w * N + i];
    }
}

__device__ __forceinline__ void norm_gate(const NormParams &p, size_t t, int col, float (&g)[8]) {
    if (!p.gate) {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = p.alpha;
        return;
    }
    const size_t row = p.gate_rows == 1 ? 0 : t;
    if (p.gate_cols == 1) {
        const float v = p.alpha * load_value(p.gate, p.gate_type, row);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = v;
    } else {
        load_values(p.gate, p.gate_type, row * p.K + col, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] *= p.alpha;
    }
}

// A token a workgroup; a thread has the C columns of 8 that lie blockDim.x * 8 apart, and keeps them: rows, weights and
// outputs pass once.  Memory bounds it: 2048 tokens of 7168 columns, eight bf16 rows each, fp32 stream in and
// out, bf16 out: 408 MB in 84 us, 4.86 TB/s, what a copy reaches.  One token: 8 us, the call itself.
template <int TX, int TB, int C, int THREADS>
__global__ __launch_bounds__(THREADS) void norm_kernel(NormParams p) {
    __shared__ float s_a[16], s_b[16];
    const size_t t = blockIdx.x;
    const int waves = blockDim.x >> 6;
    const float inv_k = 1.0f / (float)p.K;
    float v[C][8], r[C][8];
    float sum[1] = {0.0f};
    if (p.rows) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int col = (threadIdx.x + i * blockDim.x) * 8;
            if (col >= p.K) continue;
            norm_rows<TB>(p.rows, p.row_of, t, p.top_k, p.R, p.K, col, v[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[0] += v[i][j] * v[i][j];
            if (p.s) Element<TB>::store(p.s, t * p.K + col, v[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int col = (threadIdx.x + i * blockDim.x) * 8;
        if (col >= p.K) continue;
        if (p.x) Element<TX>::values(Element<TX>::load(p.x, t * p.K + col), r[i]);
        else
#pragma unroll
            for (int j = 0; j < 8; ++j) r[i][j] = 0.0f;
    }
    if (p.rows) {
        float rstd = 1.0f;
        if (p.w_after) {
            norm_sum(sum, s_a, waves);
            rstd = 1.0f / sqrtf(sum[0] * inv_k + p.eps);
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int col = (threadIdx.x + i * blockDim.x) * 8;
            if (col >= p.K) continue;
            float w[8], g[8];
            norm_gate(p, t, col, g);
            if (p.w_after) Element<kFp32>::values(Element<kFp32>::load(p.w_after, col), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) r[i][j] += g[j] * (p.w_after ? v[i][j] * rstd * w[j] : v[i][j]);
        }
    }
    sum[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int col = (threadIdx.x + i * blockDim.x) * 8;
        if (col >= p.K) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[0] += r[i][j] * r[i][j];
        if (p.r) Element<TX>::store(p.r, t * p.K + col, r[i]);
    }
    if (!p.h) return;
    norm_sum(sum, s_b, waves);
    const float rstd = 1.0f / sqrtf(sum[0] * inv_k + p.eps);
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int col = (threadIdx.x + i * blockDim.x) * 8;
        if (col >= p.K) continue;
        float w[8];
        Element<kFp32>::values(Element<kFp32>::load(p.w_before, col), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] = r[i][j] * rstd * w[j];
        store_values(p.h, p.h_type, t * p.K + col, r[i]);
    }
}

// Backwards.  A workgroup goes on to further tokens and keeps its sums over them for every column; they go to the
// workspace, and a second kernel adds them up in a fixed order.  What it waits for is memory: a token's rows are asked
// for together, and kept as they are stored until both of the token's reductions are done.  Sixteen waves a CU, at 128
// registers of which 24 to 29 spill, hide more of the wait than eight that spill none (112 us for 95 below). 4096 tokens
// of 4096 columns, six bf16 rows each, a gate a column: 365 MB in 92 to 96 us, 3.9 TB/s; the second kernel has 6 us of
// it.  bf16 and the norm before alone: 8192 tokens of 4096 columns 268 MB in 66 us, 4.1 TB/s.  Away from that it is far
// from a copy's rate.  Few tokens: two kernels, one waiting for the other: 64 of 5376 columns 12 us for 3 MB, 390 16 us
// for 17.  Few columns, where a CU has few waves (norm_grad_groups): 8192 tokens of 1024 33 us, 2.0 TB/s, 4000 of 384 16
// us, 0.8.  Above 8192 columns a thread has two or four chunks, and the three sums of each column spill (122 to 210
// registers, 381 to 495): 1000 tokens of 16384 columns 75 us, 1.8 TB/s, of 32768 197 us, 1.3 (with both norms and two
// rows each 130, 1.8, and 398, 1.2).
template <int TX, int TB, int C>
__global__ __launch_bounds__(1024) void norm_grad_kernel(NormParams p) {
    __shared__ float s_a[2][48], s_b[2][32];
    const int waves = blockDim.x >> 6;
    const float inv_k = 1.0f / (float)p.K;
    const bool block = p.s != nullptr, before = p.w_before != nullptr, after = p.w_after != nullptr;
    float wb_sum[C][8] = {}, wa_sum[C][8] = {}, gate_sum[C][8] = {}, one_sum = 0.0f;
    int flip = 0;
    for (size_t t = blockIdx.x; t < (size_t)p.M; t += gridDim.x, flip ^= 1) {
        typename Element<TX>::Raw r_raw[C], dr_raw[C];
        typename Element<TB>::Raw s_raw[C];
        float dh[C][8], sum[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int col = (threadIdx.x + i * blockDim.x) * 8;
            if (col >= p.K) continue;
            if (before) r_raw[i] = Element<TX>::load_nt(p.r, t * p.K + col);
            if (p.dr) dr_raw[i] = Element<TX>::load_nt(p.dr, t * p.K + col);
            if (block) s_raw[i] = Element<TB>::load_nt(p.s, t * p.K + col);
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int col = (threadIdx.x + i * blockDim.x) * 8;
            if (col >= p.K) continue;
            float v[8];
            if (before) {
                float w[8];
                if (p.h_type == kFp32) norm_rows<kFp32>(p.h, p.row_of, t, p.top_k, p.R, p.K, col, dh[i]);
                else if (p.h_type == kFp16) norm_rows<kFp16>(p.h, p.row_of, t, p.top_k, p.R, p.K, col, dh[i]);
                else norm_rows<kBf16>(p.h, p.row_of, t, p.top_k, p.R, p.K, col, dh[i]);
                Element<kFp32>::values(Element<kFp32>::load(p.w_before, col), w);
                Element<TX>::values(r_raw[i], v);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sum[0] += v[j] * v[j];
                    sum[1] += dh[i][j] * w[j] * v[j];
                }
            }
            if (block) {
                Element<TB>::values(s_raw[i], v);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[2] += v[j] * v[j];
            }
        }
        norm_sum(sum, s_a[flip], waves);
        const float rstd_r = 1.0f / sqrtf(sum[0] * inv_k + p.eps);
        const float rstd_s = after ? 1.0f / sqrtf(sum[2] * inv_k + p.eps) : 1.0f;
        const float mean_r = sum[1] * inv_k * rstd_r * rstd_r;
        float dot[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int col = (threadIdx.x + i * blockDim.x) * 8;
            if (col >= p.K) continue;
            float g[8], v[8], w[8];
            if (p.dr) Element<TX>::values(dr_raw[i], g);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] = 0.0f;
            if (before) {
                Element<TX>::values(r_raw[i], v);
                Element<kFp32>::values(Element<kFp32>::load(p.w_before, col), w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    wb_sum[i][j] += dh[i][j] * (v[j] * rstd_r);
                    g[j] += rstd_r * (dh[i][j] * w[j] - v[j] * mean_r);
                }
            }
            Element<TX>::store_nt(p.dx, t * p.K + col, g);
            if (!block) continue;
            Element<TB>::values(s_raw[i], v);
            if (after) Element<kFp32>::values(Element<kFp32>::load(p.w_after, col), w);
            if (p.dgate) {  // the gate's own gradient
                float n[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    n[j] = p.alpha * g[j] * (v[j] * rstd_s * (after ? w[j] : 1.0f));
                    dot[1] += n[j];
                }
                if (p.gate_cols != 1) {
                    if (p.gate_rows == 1)
#pragma unroll
                        for (int j = 0; j < 8; ++j) gate_sum[i][j] += n[j];
                    else store_values(p.dgate, p.gate_type, t * p.K + col, n);
                }
            }
            float gate[8];
            norm_gate(p, t, col, gate);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                g[j] *= gate[j];
                if (after) {
                    wa_sum[i][j] += g[j] * (v[j] * rstd_s);
                    g[j] *= w[j];
                    dot[0] += g[j] * v[j];
                }
                dh[i][j] = g[j];
            }
        }
        if (!block) continue;
        if (after || (p.dgate && p.gate_cols == 1)) norm_sum(dot, s_b[flip], waves);
        if (p.dgate && p.gate_cols == 1) {
            if (p.gate_rows == 1) one_sum += dot[1];
            else if (threadIdx.x == 0) store_value(p.dgate, p.gate_type, t, dot[1]);
        }
        const float mean_s = after ? dot[0] * inv_k * rstd_s * rstd_s : 0.0f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int col = (threadIdx.x + i * blockDim.x) * 8;
            if (col >= p.K) continue;
            float v[8];
            Element<TB>::values(s_raw[i], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) dh[i][j] = rstd_s * (dh[i][j] - v[j] * mean_s);
            Element<TB>::store_nt(p.ds, t * p.K + col, dh[i]);
        }
    }
    const size_t n = gridDim.x;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int col = (threadIdx.x + i * blockDim.x) * 8;
        if (col >= p.K) continue;
        const size_t at = blockIdx.x * (size_t)p.K + col;
        if (before) Element<kFp32>::store(p.part, at, wb_sum[i]);
        if (after) Element<kFp32>::store(p.part, n * p.K + at, wa_sum[i]);
        if (p.dgate && p.gate_rows == 1 && p.gate_cols != 1) Element<kFp32>::store(p.part, 2 * n * p.K + at, gate_sum[i]);
    }
    if (p.dgate && p.gate_rows == 1 && p.gate_cols == 1 && threadIdx.x == 0) p.part[2 * n * p.K + blockIdx.x] = one_sum;
}

// Column blockIdx.x * 64 + lane of vector blockIdx.y: the sum of its n parts, a sixteenth of them a wave, eight
// asked for at a time.
__global__ __launch_bounds__(1024) void norm_columns_kernel(NormParams p, int n) {
    __shared__ float s[16][64];
    const int which = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int cols = which == 2 && p.gate_cols == 1 ? 1 : p.K, col = blockIdx.x * 64 + lane;
    if (which == 0 ? !p.w_before : which == 1 ? !p.w_after : !(p.dgate && p.gate_rows == 1)) return;
    const float *part = p.part + (size_t)which * n * p.K;
    float sum = 0.0f;
    if (col < cols)
        for (int i = wave; i < n; i += 16 * 8) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = i + 16 * u < n ? part[(size_t)(i + 16 * u) * cols + col] : 0.0f;
#pragma unroll
            for (int u = 0; u < 8; ++u) sum += v[u];
        }
    s[wave][lane] = sum;
    __syncthreads();
    if (wave != 0 || col >= cols) return;
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) sum += s[w][lane];
    if (which == 2) store_value(p.dgate, p.gate_type, col, sum);
    else (which ? p.dw_after : p.dw_before)[col] = sum;
}

// Threads to a token, of C columns of 8 each.
static int norm_threads(int K, int C) { return ((K / 8 + C - 1) / C + 63) / 64 * 64; }
static int norm_grad_c(int K) { return K <= 8192 ? 1 : K <= 16384 ? 2 : 4; }

// At most sixteen waves a CU, which their registers allow: nine to sixteen from K = 1152 on, four to eight for a K of
// 1024 and less, whose workgroups are one or two waves.  With 512 workgroups always, of at most 512 threads, 8192 tokens
// of 2048 columns took 113 us for 91, and 4096 of 7168 columns 223 for 209.
int norm_grad_groups(int M, int K) {
    const int threads = norm_threads(K, norm_grad_c(K)), most = threads > 512 ? 256 : threads > 256 ? 512 : 1024;
    return M < most ? M : most;
}

template <int TX, int TB, int C, int THREADS>
static void norm_launch_shape(const NormParams &p, hipStream_t stream) {
    hipLaunchKernelGGL((norm_kernel<TX, TB, C, THREADS>), dim3(p.M), dim3(norm_threads(p.K, C)), 0, stream, p);
}
template <int TX, int TB, int C>
static void norm_grad_launch_shape(const NormParams &p, hipStream_t stream) {
    hipLaunchKernelGGL((norm_grad_kernel<TX, TB, C>), dim3(norm_grad_groups(p.M, p.K)), dim3(norm_threads(p.K, C)), 0,
                       stream, p);
}
template <int TX, int TB>
static void norm_launch(const NormParams &p, bool grad, hipStream_t stream) {
    if (grad) {
        const int c = norm_grad_c(p.K);
        if (c == 1) norm_grad_launch_shape<TX, TB, 1>(p, stream);
        else if (c == 2) norm_grad_launch_shape<TX, TB, 2>(p, stream);
        else norm_grad_launch_shape<TX, TB, 4>(p, stream);
    } else if (p.K <= 4096) {
        norm_launch_shape<TX, TB, 1, 512>(p, stream);
    } else if (p.K <= 8192) {
        norm_launch_shape<TX, TB, 2, 512>(p, stream);
    } else {
        norm_launch_shape<TX, TB, 4, 1024>(p, stream);
    }
}

hipError_t launch_norm(const NormParams &p, int x_type, int rows_type, bool grad, hipStream_t stream) {
    switch (3 * x_type + rows_type) {
        case 0: norm_launch<kFp32, kFp32>(p, grad, stream); break;
        case 1: norm_launch<kFp32, kFp16>(p, grad, stream); break;
        case 2: norm_launch<kFp32, kBf16>(p, grad, stream); break;
        case 3: norm_launch<kFp16, kFp32>(p, grad, stream); break;
        case 4: norm_launch<kFp16, kFp16>(p, grad, stream); break;
        case 5: norm_launch<kFp16, kBf16>(p, grad, stream); break;
        case 6: norm_launch<kBf16, kFp32>(p, grad, stream); break;
        case 7: norm_launch<kBf16, kFp16>(p, grad, stream); break;
        default: norm_launch<kBf16, kBf16>(p, grad, stream); break;
    }
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || !grad) return err;
    if (!p.w_before && !p.w_after && !(p.dgate && p.gate_rows == 1)) return err;
    hipLaunchKernelGGL(norm_columns_kernel, dim3((p.K + 63) / 64, 3), dim3(1024), 0, stream, p,
                       norm_grad_groups(p.M, p.K));
    return hipGetLastError();
}

}  // namespace megamoe
