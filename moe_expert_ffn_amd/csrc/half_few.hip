// Grouped products of 16-bit rows and weights for few rows an expert, where the product streams weights.
//
// p[n] = sum_k a[k] b[e, n, k] as in half_gmm.hip, in tiles of at most 32 NP rows by 128 weight rows (with SwiGLU 64 for
// silu and the 64 of the gate), a quarter of them a wave.  A stage is 64 of the reduction, a whole cache line of
// every row, copied asynchronously into one of three or four slots in LDS, so that two or three are under way while one is
// multiplied; two workgroups fit a CU, so that one copies while the other starts or ends.  The code is short: a workgroup goes through
// it once, and every instruction comes from memory again, as the weights have driven it out of the caches.
// K = 7168, I = 2048, E = 32, top_k = 8, one token: first product with SwiGLU 70 us, 6.7 TB/s of weights (the 256-row
// tiles 114; weights straight into registers, half lines at a time, 114), second product 37 to 40 (the tiles 47).
// A workgroup goes through its whole reduction alone: with few workgroups their stages one after the other are the time, not
// the weights' bytes (65 tokens of 7 experts, top_k = 2, K = 6144, I = 256, SwiGLU: 45 us for 32 MB).
#include "dma.hpp"
#include "half_gmm.hpp"

namespace megamoe {

typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kFewRows = 128;  // weight rows of a workgroup

template <int T>
__device__ __forceinline__ v16f few_mfma(v4i w, v4i a, v16f acc) {
    if constexpr (T == kBf16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, w), __builtin_bit_cast(v8bf, a), acc, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, w), __builtin_bit_cast(v8h, a), acc, 0, 0, 0);
}
template <int T, bool SWIGLU, int NP>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) void half_few_kernel(HalfGmmParams p) {
    constexpr int RB = 32 * NP, COLS = SWIGLU ? kFewRows / 2 : kFewRows, SLOT = (RB + kFewRows) * 128;
    constexpr int COPIES = NP + 4;  // of a stage a wave: of 8 rows each
    constexpr int SLOTS = NP == 1 ? 4 : 3;  // as many as two workgroups a CU have room for
    __shared__ __align__(16) uint8_t s_data[SLOTS * SLOT];
    // the schedule is only looked at here, before the first copies: it lies where they go
    const FewTile t = few_find_tile<RB>(p, blockIdx.x, COLS, *reinterpret_cast<FewSchedule *>(s_data));
    if (t.e < 0) return;
    __syncthreads();
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t ld = 2 * p.K;
    const uint8_t *w = uniform_ptr((const uint8_t *)(p.b + (size_t)t.e * (SWIGLU ? 2 : 1) * p.N * p.K));
    const uint8_t *a = uniform_ptr((const uint8_t *)p.a);
    const uint32_t at = __builtin_amdgcn_readfirstlane(lds_addr(s_data));
    uint32_t va[NP], vw[4];
    int route[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int row = t.row0 + min((wave * NP + i) * 8 + (lane >> 3), t.rows - 1);
        route[i] = p.gather ? p.route[row] : row;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // with SwiGLU a wave's 32 are 16 for silu and the 16 of the gate that go with them
        const int r = (wave * 4 + i) * 8 + (lane >> 3), in = r & 31;
        const int col = t.nblk * COLS + (SWIGLU ? 16 * wave + (in & 15) : r);
        vw[i] = (uint32_t)(min(col, p.N - 1) + (SWIGLU && in >= 16 ? p.N : 0)) * ld + hg_swz(r, lane & 7) * 16;
    }
    auto issue_w = [&](int s) {
        const uint32_t to = at + s % SLOTS * SLOT + RB * 128 + wave * 4096;
#pragma unroll
        for (int i = 0; i < 4; ++i) dma16_nt(uniform_ptr(w + s * 128), vw[i], to + i * 1024);
    };
    auto issue_a = [&](int s) {
        const uint32_t to = at + s % SLOTS * SLOT + wave * (NP * 1024);
#pragma unroll
        for (int i = 0; i < NP; ++i) dma16(uniform_ptr(a + s * 128), va[i], to + i * 1024);
    };
    const int ns = p.K / 64;  // two at least
#pragma unroll
    for (int i = 0; i < NP; ++i)
        va[i] = (p.gather ? hg_token(p, route[i]) : (uint32_t)route[i]) * ld +
                hg_swz((wave * NP + i) * 8 + (lane >> 3), lane & 7) * 16;
#pragma unroll
    for (int s = 0; s < SLOTS - 1; ++s)
        if (s < ns) {
            issue_w(s);
            issue_a(s);
        }
    const int r = lane & 31, g = lane >> 5;
    v16f acc[NP] = {};
#pragma unroll 1
    for (int s = 0; s < ns; ++s) {
        // stage s is there: all but the copies of the two behind it
        if (s + SLOTS - 2 < ns) wait_vmcnt<(SLOTS - 2) * COPIES>();
        else wait_vmcnt<0>();
        __syncthreads();  // and every wave has read stage s - 1, whose slot is free
        if (s + SLOTS - 1 < ns) {
            issue_w(s + SLOTS - 1);
            issue_a(s + SLOTS - 1);
        }
        const uint8_t *q = s_data + s % SLOTS * SLOT + r * 128;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const int place = hg_swz(r, 2 * h + g) * 16;
            const v4i wf = *reinterpret_cast<const v4i *>(q + RB * 128 + wave * 4096 + place);
#pragma unroll
            for (int i = 0; i < NP; ++i)
                acc[i] = few_mfma<T>(wf, *reinterpret_cast<const v4i *>(q + i * 4096 + place), acc[i]);
        }
    }
    // Lane l holds row l & 31 and the columns 8 q + 4 (l >> 5) + 0..3, q = 0..3; lanes l and l + 32 exchange halves of
    // two such groups, so that each stores eight columns in a row.
    constexpr int Q = SWIGLU ? 2 : 4;
    const int n0 = t.nblk * COLS + wave * (COLS / 4);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int row = 32 * i + r;
        float weight = 1.0f;
        if (SWIGLU && p.probs) weight = p.probs[hg_route(p, p.route[t.row0 + min(row, t.rows - 1)])];
        uint2 out[Q];
#pragma unroll
        for (int k = 0; k < Q; ++k) {
            float y[4];
#pragma unroll
            for (int v = 0; v < 4; ++v)
                y[v] = SWIGLU ? weight * hg_silu_times(acc[i][4 * k + v], acc[i][8 + 4 * k + v]) : acc[i][4 * k + v];
            out[k] = make_uint2(Element<T>::pack(y[0], y[1]), Element<T>::pack(y[2], y[3]));
        }
        uint16_t *crow = (uint16_t *)p.c + (size_t)(t.row0 + row) * p.N;
#pragma unroll
        for (int k = 0; k < Q; k += 2) {
            const auto x = __builtin_amdgcn_permlane32_swap(out[k].x, out[k + 1].x, false, false);
            const auto y = __builtin_amdgcn_permlane32_swap(out[k].y, out[k + 1].y, false, false);
            const int col = n0 + 8 * (k + g);
            if (row < t.rows && col < p.N) *reinterpret_cast<uint4 *>(crow + col) = make_uint4(x[0], y[0], x[1], y[1]);
        }
    }
}

// Measured on both sides, this kernel and the 256-row tiles, in us, by mean rows an expert.  K = 7168, I = 2048, E = 32,
// uniform routing: first product with SwiGLU 1 row 250 / 265, 4 284 / 309, 16 280 / 298, 32 288 / 312, 40 293 / 310, 50
// 295 / 305, 64 484 / 321; second product 122 / 137, 152 / 190, 157 / 185, 158 / 171, 161 / 173, 170 / 191, 242 / 185.  K
// = 4096, I = 1408, E = 64, Zipf(1.2) routing, whose largest groups have several times the mean: 28 rows 264 / 286 and
// 137 / 148, 32 rows 269 / 289 and 154 / 162, 36 rows 293 / 292 and 166 / 163, 38 rows 286 / 284 and 162 / 158.  The
// bound is the skewed routing's: even groups would pay up to 64 rows, the second block of rows.
bool half_few_ok(const HalfGmmParams &p) { return (p.R + p.E - 1) / p.E <= 36; }

template <int T, bool SWIGLU, int NP>
static void few_launch(const HalfGmmParams &p, hipStream_t stream) {
    constexpr int RB = 32 * NP, COLS = SWIGLU ? kFewRows / 2 : kFewRows;
    const long long n = ((long long)p.R / RB + (p.E < p.R ? p.E : p.R)) * ((p.N + COLS - 1) / COLS);
    hipLaunchKernelGGL((half_few_kernel<T, SWIGLU, NP>), dim3((unsigned)((n + 7) / 8 * 8)), dim3(256), 0, stream, p);
}

hipError_t launch_half_few(const HalfGmmParams &p, int type, hipStream_t stream) {
    // 32 or 64 rows a tile, us of the first product with SwiGLU and of the second, K = 7168, I = 2048, E = 32: one token
    // 72 / 73 and 40 / 41, mean 1 row 251 / 254 and 123 / 125, 4 rows 299 / 284 and 152 / 156, 16 rows 291 / 280 and 157
    // / 158, 32 rows 413 / 288 and 218 / 158
    const bool one = (p.R + p.E - 1) / p.E <= 16;
#define FEW(T, S)                              \
    if (one) few_launch<T, S, 1>(p, stream);   \
    else few_launch<T, S, 2>(p, stream)
    if (type == kBf16) {
        if (p.swiglu) { FEW(kBf16, true); }
        else { FEW(kBf16, false); }
    } else {
        if (p.swiglu) { FEW(kFp16, true); }
        else { FEW(kFp16, false); }
    }
#undef FEW
    return hipGetLastError();
}

}  // namespace megamoe
