// Grouped products of 16-bit rows and weights, and their rows' gradients, for problems of few tiles: short groups by few
// columns over a long reduction, where a workgroup that goes through all of it alone waits for memory at every stage.
//
// As half_gmm.hip, in tiles of 64 rows by 64 columns (with SwiGLU 32 for silu and the 32 of the gate).  The four waves of a
// tile share the reduction: wave w has its stages w, w + 4, ... of 64, three of them under way in registers, straight
// from memory; the columns of a rows' gradient, which lie across the reduction, go through a place in LDS of
// the wave's own.  The waves' sums meet in LDS and are added in the waves' order.
#include "half_gmm.hpp"

namespace megamoe {

constexpr int kSmallRows = 64, kSmallCols = 64, kSmallStage = 64, kSmallAhead = 3;

template <int KIND, int T, bool SWIGLU>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1))) void half_small_kernel(HalfGmmParams p) {
    constexpr bool ACROSS = KIND == kHalfRows;
    constexpr int F = SWIGLU ? 2 : 1, COLS = kSmallCols / F, J = 4 / F;
    __shared__ __align__(16) uint8_t s_data[4 * 16384];
    // the schedule is only looked at here: it lies where the sums will
    const FewTile t = few_find_tile<kSmallRows>(p, blockIdx.x, COLS, *reinterpret_cast<FewSchedule *>(s_data));
    if (t.e < 0) return;
    __syncthreads();
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const uint32_t ld = 2 * p.K;
    const uint8_t *a = (const uint8_t *)p.a;
    const uint8_t *b = (const uint8_t *)(p.b + (size_t)t.e * F * p.N * p.K);
    uint32_t va[4], vb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = t.row0 + min(16 * i + r, t.rows - 1);
        va[i] = (p.gather ? hg_token(p, p.route[row]) : (uint32_t)row) * ld + 16 * g;
        // N is a multiple of 128: every column is there
        const int col = t.nblk * COLS + 16 * (i % J) + r + i / J * p.N;
        vb[i] = ACROSS ? 0 : (uint32_t)col * ld + 16 * g;
    }
    const uint32_t across = (uint32_t)(lane >> 3) * (2 * p.N) + (t.nblk * kSmallCols + (lane & 7) * 8) * 2;
    struct Stage {
        v4i a[4][2], b[4][2];  // b across: the 8 i + (lane >> 3)-th of the reduction, 8 columns
    } stage[kSmallAhead];
    const int n = (p.K / kSmallStage - wave + 3) / 4;  // the wave's stages
    auto load = [&](Stage &s, int q) {
        const int at = wave + 4 * q;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                s.a[i][h] = *reinterpret_cast<const v4i *>(a + (size_t)at * 128 + va[i] + h * 64);
                s.b[i][h] = ACROSS ? *reinterpret_cast<const v4i *>(b + ((size_t)at * kSmallStage + 8 * (2 * i + h)) * (2 * p.N) + across)
                                   : *reinterpret_cast<const v4i *>(b + (size_t)at * 128 + vb[i] + h * 64);
            }
    };
    v4f acc[4][4] = {};
    HgRead<true> columns;
    columns.lane_places();
    columns.at = s_data + wave * 8192;
    auto multiply = [&](Stage &s) {
        if constexpr (ACROSS) {
            uint8_t *to = s_data + wave * 8192 + (lane >> 3) * 128 + (lane & 1) * 16;
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // the quarters' places as HgRead has them
                const int quarter = ((lane & 7) >> 1) ^ ((lane >> 4 & 1) * 2 + (i & 1));
                *reinterpret_cast<v4i *>(to + i * 1024 + quarter * 32) = s.b[i >> 1][i & 1];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) columns.read(i, h, s.b[i][h]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = hg_mfma<T>(s.b[j][h], s.a[i][h], acc[i][j]);
    };
    if (n > 0) {
#pragma unroll
        for (int d = 0; d < kSmallAhead; ++d) load(stage[d], min(d, n - 1));
#pragma unroll 1
        for (int q = 0; q < n; q += kSmallAhead)
#pragma unroll
            for (int d = 0; d < kSmallAhead; ++d) {
                if (q + d >= n) break;
                multiply(stage[d]);
                load(stage[d], min(q + d + kSmallAhead, n - 1));
            }
    }
    // [wave][fragment][lane]; wave w rounds and stores the rows 16 w + 0..15
    __syncthreads();
    v4f *sums = reinterpret_cast<v4f *>(s_data);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sums[(wave * 16 + 4 * i + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    v4f y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        y[j] = sums[(4 * wave + j) * 64 + lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) y[j] += sums[(w * 16 + 4 * wave + j) * 64 + lane];
    }
    const int row = 16 * wave + r;
    if (row >= t.rows) return;
    float weight = 1.0f;
    if (SWIGLU && p.probs) weight = p.probs[hg_route(p, p.route[t.row0 + row])];
    uint16_t *crow = (uint16_t *)p.c + (size_t)(t.row0 + row) * p.N + t.nblk * COLS + 4 * g;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = SWIGLU ? weight * hg_silu_times(y[j][k], y[(j + 2) & 3][k]) : y[j][k];
        *reinterpret_cast<uint2 *>(crow + 16 * j) = make_uint2(Element<T>::pack(v[0], v[1]), Element<T>::pack(v[2], v[3]));
    }
}

static long long small_tiles(const HalfGmmParams &p) {  // at most
    return ((long long)p.R / kSmallRows + (p.E < p.R ? p.E : p.R)) * (p.N / (kSmallCols / (p.swiglu ? 2 : 1)));
}

// At most two tiles a CU.  Measured on both sides, the 256-row tiles and this kernel, in us, by this many small tiles.  Row
// gradients: R = 12, K = 5120, N = 128 (24 tiles) 72 / 19; R = 1751, K = 6528, N = 384 (264) 124 / 40; R = 24, K = 5376,
// N = 896 (336) 81 / 25; R = 1162, K = 896, N = 384 (432) 22 / 19; R = 600, K = 1280, N = 1920 (510) 27 / 26; more of them: R
// = 1659, K = 256, N = 1408 (1034) 13 / 32.  Products: R = 564, K = 1920, N = 256 (52) 35 / 23; R = 2030, K = 384, N = 384
// (312) 18 / 12; R = 1872, K = 5248, N = 768 (456) 100 / 89; more: R = 3906, K = 768, N = 512 (608) 25 / 28.  Products of
// few rows an expert have a kernel that is faster than both: R = 632, K = 1280, N = 3328 39 / 87.
bool half_small_ok(const HalfGmmParams &p, int kind, int cu_count) {
    return small_tiles(p) <= 2 * cu_count && (kind == kHalfRows || !half_few_ok(p));
}

template <int KIND, int T, bool SWIGLU>
static void small_launch(const HalfGmmParams &p, hipStream_t stream) {
    hipLaunchKernelGGL((half_small_kernel<KIND, T, SWIGLU>), dim3((unsigned)((small_tiles(p) + 7) / 8 * 8)), dim3(256), 0,
                       stream, p);
}

hipError_t launch_half_small(const HalfGmmParams &p, int kind, int type, hipStream_t stream) {
    const bool b = type == kBf16;
    if (kind == kHalfRows) {
        if (b) small_launch<kHalfRows, kBf16, false>(p, stream);
        else small_launch<kHalfRows, kFp16, false>(p, stream);
    } else if (p.swiglu) {
        if (b) small_launch<kHalfProduct, kBf16, true>(p, stream);
        else small_launch<kHalfProduct, kFp16, true>(p, stream);
    } else {
        if (b) small_launch<kHalfProduct, kBf16, false>(p, stream);
        else small_launch<kHalfProduct, kFp16, false>(p, stream);
    }
    return hipGetLastError();
}

}  // namespace megamoe
