// The expert layer for a few tokens (M <= 16), in two kernels.
//
// The mathematics and every rounding are those of the five stages (sections 1 and
// 3 to 7 of the pto-isa MegaMoE overview page), so the result equals
// megamoe_forward's bit for bit; what differs is where the stages meet.  With a
// few rows per expert the layer is bound by reading the chosen experts' weights
// once from HBM, and what the staged forward spends on top is launches, tiles
// that are mostly empty and intermediates that travel through memory.
//
// The rows are the distinct (token, expert) pairs, expert-major ("pairs"): at
// most 16 per expert, one row block of v_mfma_i32_16x16x64_i8.  Every workgroup
// finds the pairs by itself from the M * top_k expert ids, so nothing has to
// be sorted beforehand.
//  * few_gmm1_kernel, one workgroup per chosen expert and 16 output columns:
//    quantises its expert's tokens into LDS, multiplies them by the 16 silu and
//    the 16 gate columns with the reduction split over its waves (an exact
//    integer sum), and writes y = silu * gate in fp32 with the largest |y| of
//    its columns.
//  * few_gmm2_kernel, one workgroup per 16 output columns: quantises every
//    pair's y into LDS (the row maximum is that of the 16-column maxima),
//    multiplies each expert's rows by its 16 columns, and combines the slots of
//    every token in order, so no partial result leaves the workgroup.
// A wave reads weights straight from memory into fragments: 16 columns of one
// 64-byte K slice are 1 KB in a row in the packed layout.
#include "common.hpp"
#include "kernels.hpp"
#include "quant_row.hpp"
#include "swiglu_row.hpp"

namespace megamoe {

constexpr int kFewWaves = 8;
constexpr int kFewThreads = kFewWaves * kWave;
constexpr int kFewE = 256;
constexpr int kPackRowsF = 256, kPackBlockF = 256 * 64;  // the packed weights' n-block

// The pairs of a batch: experts by their token sets, numbered expert-major.
struct FewPairs {
    uint32_t mask[kFewE];  // tokens of the expert, one bit each
    int base[kFewE];       // pairs of the experts before it
    int act[kFewE];        // experts with a pair, ascending
    int n_act, n_pair, valid;
};

__device__ __forceinline__ void few_find_pairs(const int32_t *__restrict__ ids, int R, int E,
                                               int top_k, FewPairs &s) {
    const int tid = threadIdx.x;
    for (int e = tid; e < kFewE; e += kFewThreads) s.mask[e] = 0;
    if (tid == 0) s.valid = 0;
    const int id = tid < R ? ids[tid] : -1;  // R <= kFewThreads
    __syncthreads();
    if (id >= 0 && id < E) {
        atomicOr(&s.mask[id], 1u << (tid / top_k));
        atomicAdd(&s.valid, 1);
    }
    __syncthreads();
    if (tid < kWave) {  // four experts a lane; counts of pairs (low) and experts (high) together
        int v[4], sum = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = __popc(s.mask[tid * 4 + j]);
            v[j] = n | (n ? 1 << 16 : 0);
            sum += v[j];
        }
        int run = wave_inclusive_scan(sum) - sum;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s.base[tid * 4 + j] = run & 0xffff;
            if (v[j]) s.act[run >> 16] = tid * 4 + j;
            run += v[j];
        }
        if (tid == kWave - 1) {
            s.n_pair = run & 0xffff;
            s.n_act = run >> 16;
        }
    }
    __syncthreads();
}

__device__ __forceinline__ v4i few_load(const int8_t *p) {
    return __builtin_nontemporal_load(reinterpret_cast<const v4i *>(p));
}

__device__ __forceinline__ v4i few_mfma(v4i w, v4i a, v4i acc) {
    // weights first: lane l holds row l & 15 and the columns 4 (l >> 4) + 0..3
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, a, acc, 0, 0, 0);
}

// ---------------------------------------------------------------------------
__global__ __launch_bounds__(kFewThreads) void few_gmm1_kernel(FewParams p, int row_cap) {
    constexpr int U = 4;  // K slices a wave has in flight
    __shared__ FewPairs s_p;
    __shared__ int s_tok[16];
    __shared__ uint32_t s_red[16][kFewWaves];
    __shared__ float s_scale[16];
    __shared__ v4i s_part[kFewWaves][2][kWave];
    extern __shared__ __align__(16) int8_t s_a[];  // [row_cap][K + 16]

    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid >> 6;
    const int K = p.K, I = p.I, stride = K + 16;
    few_find_pairs(p.expert_idx, p.M * p.top_k, p.E, p.top_k, s_p);
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) *p.err = p.M * p.top_k - s_p.valid;
    if ((int)blockIdx.y >= s_p.n_act) return;
    const int e = s_p.act[blockIdx.y];
    const uint32_t mask = s_p.mask[e];
    const int n = __popc(mask), pair0 = s_p.base[e];
    if (tid < 16 && (mask >> tid & 1)) s_tok[__popc(mask & ((1u << tid) - 1))] = tid;
    __syncthreads();

    const int NB = (2 * I + kPackRowsF - 1) / kPackRowsF;
    const size_t slice = (size_t)p.E * NB * kPackBlockF;
    const int nu = blockIdx.x * 16, ng = I + nu, ns = K / 64;
    const int8_t *we = p.w1p + (size_t)e * NB * kPackBlockF + (lane & 15) * 64 + (lane >> 4) * 16;
    const int8_t *wu = we + (size_t)(nu / kPackRowsF) * kPackBlockF + (nu % kPackRowsF) * 64;
    const int8_t *wg = we + (size_t)(ng / kPackRowsF) * kPackBlockF + (ng % kPackRowsF) * 64;
    const int cnt = (ns - wave + kFewWaves - 1) / kFewWaves;  // slices wave, wave + 8, ...
    const v4i zero = {0, 0, 0, 0};

    for (int r0 = 0; r0 < n; r0 += row_cap) {
        const int m = min(row_cap, n - r0);
        v4i fu[U], fg[U];
        auto load = [&](int i0) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const size_t o = (size_t)(wave + (i0 + i) * kFewWaves) * slice;
                fu[i] = i0 + i < cnt ? few_load(wu + o) : zero;
                fg[i] = i0 + i < cnt ? few_load(wg + o) : zero;
            }
        };
        load(0);  // on their way while the rows are quantised

        for (int i = 0; i < m; ++i) {
            const uint4 *xr = reinterpret_cast<const uint4 *>(p.x + (size_t)s_tok[r0 + i] * K);
            u16x2_t mx = {0, 0};
            for (int c = tid; c < K / 8; c += kFewThreads) mx = absmax_step(mx, xr[c]);
            const uint32_t mb = wave_max_u32(mx[0] > mx[1] ? mx[0] : mx[1]);
            if (lane == 0) s_red[i][wave] = mb;
        }
        __syncthreads();
        for (int i = 0; i < m; ++i) {
            uint32_t mb = 0;
#pragma unroll
            for (int w = 0; w < kFewWaves; ++w) mb = s_red[i][w] > mb ? s_red[i][w] : mb;
            const float amax = h2f((uint16_t)mb);
            const float scale = amax / 127.0f;
            const float inv = amax != 0.0f ? 1.0f / scale : 0.0f;
            const uint4 *xr = reinterpret_cast<const uint4 *>(p.x + (size_t)s_tok[r0 + i] * K);
            for (int c = tid; c < K / 8; c += kFewThreads)
                *reinterpret_cast<uint2 *>(s_a + (size_t)i * stride + c * 8) =
                    quant_chunk8(xr[c], scale, inv);
            if (tid == 0) s_scale[i] = scale;
        }
        __syncthreads();

        v4i au = zero, ag = zero;
        // rows past the group read its first one; their results are not used
        const int8_t *arow = s_a + ((lane & 15) < m ? (lane & 15) : 0) * stride + (lane >> 4) * 16;
        for (int i0 = 0; i0 < cnt; i0 += U) {
            v4i bu[U], bg[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                bu[i] = fu[i];
                bg[i] = fg[i];
            }
            if (i0 + U < cnt) load(i0 + U);
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int ks = min(wave + (i0 + i) * kFewWaves, ns - 1);
                const v4i a = *reinterpret_cast<const v4i *>(arow + ks * 64);
                au = few_mfma(bu[i], a, au);
                ag = few_mfma(bg[i], a, ag);
            }
        }
        s_part[wave][0][lane] = au;
        s_part[wave][1][lane] = ag;
        __syncthreads();
        if (tid < 256) {  // row tid / 16, column tid % 16
            const int row = tid >> 4, col = tid & 15;
            const int at = row + 16 * (col >> 2), v = col & 3;
            int su = 0, sg = 0;
#pragma unroll
            for (int w = 0; w < kFewWaves; ++w) {
                su += reinterpret_cast<const int *>(&s_part[w][0][at])[v];
                sg += reinterpret_cast<const int *>(&s_part[w][1][at])[v];
            }
            const float *sc = p.scale1 + (size_t)e * 2 * I + nu + col;
            const uint16_t hu = f2h(keep_f32((float)su * sc[0]));
            const uint16_t hg = f2h(keep_f32((float)sg * sc[I]));
            const float p1 = s_scale[row < m ? row : 0];
            const float y = silu_times(__builtin_fmaf(h2f(hu), p1, 0.0f),
                                       __builtin_fmaf(h2f(hg), p1, 0.0f));
            float big = fmaxf(0.0f, fabsf(y));  // a NaN is passed over, as in the row's own maximum
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) big = fmaxf(big, __shfl_xor(big, off, kWave));
            if (row < m) {
                const size_t pair = pair0 + r0 + row;
                p.y[pair * I + nu + col] = y;
                if (col == 0) p.ymax[pair * (I / 16) + blockIdx.x] = big;
            }
        }
        __syncthreads();  // s_part, s_a and s_scale are free
    }
}

// ---------------------------------------------------------------------------
__global__ __launch_bounds__(kFewThreads) void few_gmm2_kernel(FewParams p, int row_cap,
                                                               int i_cap) {
    constexpr int U = 8;  // K slices a wave has in flight
    __shared__ FewPairs s_p;
    __shared__ int s_id[kFewThreads];
    __shared__ float s_mul[kFewThreads], s_pts2[kFewThreads];  // by pair
    extern __shared__ __align__(16) int8_t s_dyn[];

    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid >> 6;
    const int K = p.K, I = p.I, R = p.M * p.top_k, stride = i_cap + 16;
    int *s_acc = reinterpret_cast<int *>(s_dyn);  // [R][16], int32 then the row as fp32
    int8_t *s_a = s_dyn + (size_t)R * 64;         // [row_cap][i_cap + 16]
    few_find_pairs(p.expert_idx, R, p.E, p.top_k, s_p);
    for (int i = tid; i < R; i += kFewThreads) s_id[i] = p.expert_idx[i];
    for (int i = tid; i < s_p.n_pair * 16; i += kFewThreads) s_acc[i] = 0;

    const int NB = (K + kPackRowsF - 1) / kPackRowsF;
    const size_t block = (size_t)NB * kPackBlockF, slice = (size_t)p.E * block;
    const int n0 = blockIdx.x * 16;
    const int8_t *w0 = p.w2p + (size_t)(n0 / kPackRowsF) * kPackBlockF + (n0 % kPackRowsF) * 64 +
                       (lane & 15) * 64 + (lane >> 4) * 16;
    const v4i zero = {0, 0, 0, 0};

    for (int a0 = 0; a0 < s_p.n_act;) {
        // the experts from a0 on whose rows fit; one expert always does (16 rows at most)
        const int p0 = s_p.base[s_p.act[a0]];
        int a1 = a0 + 1, p1 = p0 + __popc(s_p.mask[s_p.act[a0]]);
        while (a1 < s_p.n_act) {
            const int q1 = p1 + __popc(s_p.mask[s_p.act[a1]]);
            if (q1 - p0 > row_cap) break;
            p1 = q1;
            ++a1;
        }
        for (int i0 = 0; i0 < I; i0 += i_cap) {
            const int ic = min(i_cap, I - i0), nsl = ic / 64;
            // the wave's share of the group's (expert, K slice) list
            const int T = (a1 - a0) * nsl;
            const int t0 = wave * T / kFewWaves, t1 = (wave + 1) * T / kFewWaves;
            int la = a0 + t0 / nsl, ls = t0 % nsl;  // the next to load
            int ca = la, cs = ls;                   // the next to multiply
            v4i f[U];
            auto load = [&](int t) {
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    f[i] = zero;
                    if (t + i < t1) {
                        f[i] = few_load(w0 + (size_t)(i0 / 64 + ls) * slice + s_p.act[la] * block);
                        if (++ls == nsl) {
                            ls = 0;
                            ++la;
                        }
                    }
                }
            };
            load(t0);
            if (i0 == 0) {  // 16 lanes a pair: the row's maximum and its quantisation step
                for (int pr = p0 + (tid >> 4); pr < p1; pr += kFewThreads / 16) {
                    const float *ym = p.ymax + (size_t)pr * (I / 16);
                    float big = 0.0f;
                    for (int c = tid & 15; c < I / 16; c += 16) big = fmaxf(big, ym[c]);
#pragma unroll
                    for (int off = 1; off < 16; off <<= 1)
                        big = fmaxf(big, __shfl_xor(big, off, kWave));
                    if ((tid & 15) == 0) {
                        s_pts2[pr] = big / 127.0f;
                        s_mul[pr] = big != 0.0f ? 127.0f / big : 0.0f;
                    }
                }
            }
            __syncthreads();  // s_mul written; the last chunk's s_a is free
            for (int i = tid; i < (p1 - p0) * (ic / 4); i += kFewThreads) {
                const int row = i / (ic / 4), c = i % (ic / 4);
                const float4 y = *reinterpret_cast<const float4 *>(p.y + (size_t)(p0 + row) * I +
                                                                   i0 + c * 4);
                const float mul = s_mul[p0 + row];
                // the rounding of swiglu_row_finish: the low bytes of y * mul + 1.5 * 2^23
                const uint32_t b0 = __float_as_uint(keep_f32(y.x * mul) + 12582912.0f);
                const uint32_t b1 = __float_as_uint(keep_f32(y.y * mul) + 12582912.0f);
                const uint32_t b2 = __float_as_uint(keep_f32(y.z * mul) + 12582912.0f);
                const uint32_t b3 = __float_as_uint(keep_f32(y.w * mul) + 12582912.0f);
                *reinterpret_cast<uint32_t *>(s_a + row * stride + c * 4) =
                    __builtin_amdgcn_perm(__builtin_amdgcn_perm(b3, b2, 0x0c0c0400u),
                                          __builtin_amdgcn_perm(b1, b0, 0x0c0c0400u), 0x05040100u);
            }
            __syncthreads();

            v4i acc = zero;
            int e = 0, rows = 0, prow = 0;
            const int8_t *arow = s_a;
            auto open = [&]() {
                e = s_p.act[ca];
                rows = __popc(s_p.mask[e]);
                prow = s_p.base[e];
                arow = s_a + (prow - p0 + ((lane & 15) < rows ? (lane & 15) : 0)) * stride +
                       (lane >> 4) * 16;
            };
            auto flush = [&]() {  // integer sums: the order of the waves does not matter
                if ((lane & 15) < rows) {
                    int *d = s_acc + (prow + (lane & 15)) * 16 + 4 * (lane >> 4);
#pragma unroll
                    for (int v = 0; v < 4; ++v) atomicAdd(d + v, acc[v]);
                }
                acc = zero;
            };
            if (t0 < t1) open();
            for (int t = t0; t < t1; t += U) {
                v4i b[U];
#pragma unroll
                for (int i = 0; i < U; ++i) b[i] = f[i];
                if (t + U < t1) load(t + U);
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    if (t + i >= t1) break;
                    acc = few_mfma(b[i], *reinterpret_cast<const v4i *>(arow + cs * 64), acc);
                    if (++cs == nsl) {
                        flush();
                        cs = 0;
                        if (++ca < a1) open();
                    }
                }
            }
            if (t0 < t1 && cs != 0) flush();
            __syncthreads();  // s_acc complete, s_a free
        }
        a0 = a1;
    }
    __syncthreads();

    // dequantise every pair's 16 columns in place
    for (int i = tid; i < s_p.n_pair * 16; i += kFewThreads) {
        const int pr = i >> 4, col = i & 15;
        int lo = 0, hi = s_p.n_act - 1;  // the pair's expert: the last one that starts at or before it
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_p.base[s_p.act[mid]] <= pr) lo = mid;
            else hi = mid - 1;
        }
        const uint16_t h = f2h(keep_f32((float)s_acc[i] * p.scale2[(size_t)s_p.act[lo] * K + n0 + col]));
        const float g = __builtin_fmaf(h2f(h), s_pts2[pr], 0.0f);
        s_acc[i] = (int)__float_as_uint(bf2f_lo(f2bf_pk(g, 0.0f)));
    }
    __syncthreads();
    if (tid < p.M * 16) {  // slots in order, multiply then add
        const int t = tid >> 4, col = tid & 15;
        float acc = 0.0f;
        for (int s = 0; s < p.top_k; ++s) {
            const int e = s_id[t * p.top_k + s];
            if (e < 0 || e >= p.E) continue;
            const int pr = s_p.base[e] + __popc(s_p.mask[e] & ((1u << t) - 1));
            acc = acc + __uint_as_float((uint32_t)s_acc[pr * 16 + col]) * p.probs[t * p.top_k + s];
        }
        p.out[(size_t)t * K + n0 + col] = (uint16_t)(f2bf_pk(acc, 0.0f) & 0xffffu);
    }
}

// ---------------------------------------------------------------------------
constexpr size_t kFewRowBytes = 56 << 10;  // quantised rows held in LDS: two workgroups fit a CU

bool few_ok(int M, int top_k) { return M <= kFewMaxM && M * top_k <= kFewThreads; }

hipError_t launch_few(const FewParams &p, hipStream_t stream) {
    const int R = p.M * p.top_k;
    const int most = p.E < R ? p.E : R;  // experts with a pair, at most
    // as many of the expert's rows as fit at once (one row of K <= 32768 always does)
    int cap1 = (int)(kFewRowBytes / (p.K + 16));
    cap1 = cap1 < 1 ? 1 : cap1 > p.M ? p.M : cap1;
    hipLaunchKernelGGL(few_gmm1_kernel, dim3(p.I / 16, most), dim3(kFewThreads),
                       (size_t)cap1 * (p.K + 16), stream, p, cap1);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    // rows of at most 2048 elements: at least 16 fit, and no expert has more than M
    const int i_cap = p.I < 2048 ? p.I : 2048;
    int cap2 = (int)(kFewRowBytes / (i_cap + 16));
    cap2 = cap2 > R ? R : cap2;
    hipLaunchKernelGGL(few_gmm2_kernel, dim3(p.K / 16), dim3(kFewThreads),
                       (size_t)R * 64 + (size_t)cap2 * (i_cap + 16), stream, p, cap2, i_cap);
    return hipGetLastError();
}

}  // namespace megamoe
