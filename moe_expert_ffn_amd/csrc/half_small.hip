// Grouped products of 16-bit rows and weights, and their gradients, for problems of few tiles: short groups by few
// columns over a long reduction, where a workgroup that goes through all of it alone waits for memory at every stage.
//
// As half_gmm.hip, in tiles of 64 rows by 64 columns (with SwiGLU 32 for silu and the 32 of the gate).  The four waves of a
// tile share the reduction: wave w has its stages w, w + 4, ... of 64, two of them under way in registers, straight
// from memory (two workgroups a CU; three stages, with room for one, took up to 1.05 of the time for 70 tiles and
// up to 1.6 for 450 to 1500); operands that lie across the reduction go through a place in LDS of
// the wave's own.  The waves' sums meet in LDS and are added in the waves' order.
#include "half_gmm.hpp"

namespace megamoe {

constexpr int kSmallRows = 64, kSmallCols = 64, kSmallStage = 64, kSmallAhead = 2;

// 64 of the reduction by 64 columns, piece i of a lane being the 8 i + (lane >> 3)-th of the reduction, into a place in
// LDS, their 32-byte quarters as HgRead has them.
__device__ __forceinline__ void small_place(uint8_t *to, const v4i (&pieces)[4][2]) {
    const int lane = threadIdx.x & 63;
    to += (lane >> 3) * 128 + (lane & 1) * 16;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int quarter = ((lane & 7) >> 1) ^ ((lane >> 4 & 1) * 2 + (i & 1));
        *reinterpret_cast<v4i *>(to + i * 1024 + quarter * 32) = pieces[i >> 1][i & 1];
    }
}
__device__ __forceinline__ void small_read(const HgRead<true> &from, v4i (&f)[4][2]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) from.read(i, h, f[i][h]);
}
template <int T>
__device__ __forceinline__ void small_multiply(const v4i (&a)[4][2], const v4i (&b)[4][2], v4f (&acc)[4][4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = hg_mfma<T>(b[j][h], a[i][h], acc[i][j]);
}
// The waves' sums, added in their order: wave w gets those of the rows 16 w + 0..15.
__device__ __forceinline__ void small_join(uint8_t *data, int wave, const v4f (&acc)[4][4], v4f (&y)[4]) {
    const int lane = threadIdx.x & 63;
    v4f *sums = reinterpret_cast<v4f *>(data);  // [wave][fragment][lane]
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sums[(wave * 16 + 4 * i + j) * 64 + lane] = acc[i][j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        y[j] = sums[(4 * wave + j) * 64 + lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) y[j] += sums[(w * 16 + 4 * wave + j) * 64 + lane];
    }
}

template <int KIND, int T, bool SWIGLU>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) void half_small_kernel(HalfGmmParams p) {
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
            small_place(s_data + wave * 8192, s.b);
            small_read(columns, s.b);
        }
        small_multiply<T>(s.a, s.b, acc);
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
    v4f y[4];
    small_join(s_data, wave, acc, y);
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

// The weights' gradient: 64 x 64 of expert e's matrix, both operands across the reduction, which is the group's rows.
template <int T, int GATHER>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) void half_small_weights_kernel(HalfGmmParams p) {
    __shared__ __align__(16) uint8_t s_data[4 * 16384];
    const int nb = p.N / kSmallCols, per_expert = p.M / kSmallRows * nb, total = p.E * per_expert;
    // workgroups go round the XCDs: each XCD takes a run of neighbouring tiles, which share rows
    const int per = (total + 7) / 8, t = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || t >= total) return;
    const int e = t / per_expert, m0 = t % per_expert / nb * kSmallRows, n0 = t % nb * kSmallCols;
    const int first = hg_row_end(p, e - 1), red = max(0, hg_row_end(p, e) - first);
    if (red == 0 && p.accumulate) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t la = 2 * p.M, lb = 2 * p.N;
    const uint8_t *a = (const uint8_t *)p.a + (m0 + (lane & 7) * 8) * 2, *b = (const uint8_t *)p.b + (n0 + (lane & 7) * 8) * 2;
    struct Stage {
        v4i a[4][2], b[4][2];
    } stage[kSmallAhead];
    const int stages = (red + kSmallStage - 1) / kSmallStage, n = (stages - wave + 3) / 4;
    auto row_of = [&](int q, int i) { return first + min((wave + 4 * q) * kSmallStage + 8 * i + (lane >> 3), red - 1); };
    int route[8];  // of the stage that is loaded next
    auto load_routes = [&](int q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) route[i] = p.route[row_of(q, i)];
    };
    auto load = [&](Stage &s, int q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t row = row_of(q, i), token = hg_token(p, route[i]);
            s.a[i >> 1][i & 1] = *reinterpret_cast<const v4i *>(a + (GATHER == 1 ? token : row) * la);
            s.b[i >> 1][i & 1] = *reinterpret_cast<const v4i *>(b + (GATHER == 2 ? token : row) * lb);
        }
    };
    v4f acc[4][4] = {};
    HgRead<true> rows, columns;
    rows.lane_places();
    columns.lane_places();
    rows.at = s_data + wave * 16384;
    columns.at = rows.at + 8192;
    auto multiply = [&](Stage &s, int q) {
        const int left = red - (wave + 4 * q) * kSmallStage - (lane >> 3);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (8 * i >= left) s.a[i >> 1][i & 1] = s.b[i >> 1][i & 1] = v4i{0, 0, 0, 0};  // past the group
        small_place(s_data + wave * 16384, s.a);
        small_place(s_data + wave * 16384 + 8192, s.b);
        small_read(rows, s.a);
        small_read(columns, s.b);
        small_multiply<T>(s.a, s.b, acc);
    };
    if (n > 0) {
        load_routes(0);
#pragma unroll
        for (int d = 0; d < kSmallAhead; ++d) {
            load(stage[d], min(d, n - 1));
            load_routes(min(d + 1, n - 1));
        }
#pragma unroll 1
        for (int q = 0; q < n; q += kSmallAhead)
#pragma unroll
            for (int d = 0; d < kSmallAhead; ++d) {
                if (q + d >= n) break;
                multiply(stage[d], q + d);
                load(stage[d], min(q + d + kSmallAhead, n - 1));
                load_routes(min(q + d + kSmallAhead + 1, n - 1));
            }
    }
    v4f y[4];
    small_join(s_data, wave, acc, y);
    const size_t at = ((size_t)e * p.M + m0 + 16 * wave + (lane & 15)) * p.N + n0 + 4 * (lane >> 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (p.c_type == kFp32) {
            v4f *o = reinterpret_cast<v4f *>((float *)p.c + at + 16 * j);
            *o = p.accumulate ? *o + y[j] : y[j];
        } else {
            typedef Element<T> L;
            uint2 *o = reinterpret_cast<uint2 *>((uint16_t *)p.c + at + 16 * j);
            uint2 old = make_uint2(0, 0);
            if (p.accumulate) old = *o;
            *o = make_uint2(L::pack(L::lo(old.x) + y[j][0], L::hi(old.x) + y[j][1]),
                            L::pack(L::lo(old.y) + y[j][2], L::hi(old.y) + y[j][3]));
        }
    }
}

static long long small_tiles(const HalfGmmParams &p, int kind) {  // at most
    if (kind == kHalfWeights) return (long long)p.E * (p.M / kSmallRows) * (p.N / kSmallCols);
    return ((long long)p.R / kSmallRows + (p.E < p.R ? p.E : p.R)) * (p.N / (kSmallCols / (p.swiglu ? 2 : 1)));
}

// Measured on both sides, the 256-row tiles and this kernel, in us, by the number of small tiles (rows, reduction) at 256
// CUs. Row gradients: 72 tiles (42 rows, 1024) 21 / 9, 150 (342, 4864) 76 / 27, 440 (2312, 768) 21 / 18, 616 (4220, 7040)
// 133 / 107, 656 (10002, 1152) 32 / 32, 728 (1043, 768) 20 / 18, 788 (8919, 5248) 108 / 86, 936 (8182, 384) 20 / 25, 1050
// (6412, 1280) 22 / 32, 1300 (45 rows of 26 experts, 1280) 50 / 38, 1428 (224, 1792) 39 / 44, 1860 (3174, 3840) 84 / 144:
// past the bound this kernel is ahead for a few rows an expert and behind for many.  Weights' gradients, whose rows are
// the reduction: 216 (9548 rows) 38 / 14, 504 (10705) 61 / 29, 672 (132) 15 / 11, 900 (5145) 35 / 33, 1040 (1344) 17 /
// 16, 1064 (21344) 57 / 58, 1200 (15488) 66 / 39, 1280 (63) 14 / 15, 1536 (66) 15 / 16, 2016 (2580) 23 / 37, 2208 (10) 15
// / 24: from the bound to some 1800 either.  Products: 188 (2694, 7552) 141 / 61, 296 (3330, 6784) 127 / 57, 368 (5598,
// 1152) 31 / 29, 450 (4060, 1920) 43 / 39, 468 (816, 1024) 25 / 27, 512 (6645, 896) 27 / 25, 576 (595, 1152) 25 / 29, 640
// (639, 2048) 37 / 39, 728 (5628, 256) 17 / 25, 816 (544, 2432) 47 / 67.  Products of few rows an expert have a kernel
// that is mostly faster than both: 30 us for 632 rows of 18 experts, K = 1280, N = 3328, and 52 here; one token of K =
// 7168, E = 32, top_k = 8, I = 256 37 us and 37 here, its second product 7 and 19, 16 such tokens 46 and 42.
bool half_small_ok(const HalfGmmParams &p, int kind, int cu_count) {
    const long long halves = kind == kHalfProduct ? 4 : kind == kHalfRows ? 5 : 8;  // of tiles, a CU
    return 2 * small_tiles(p, kind) <= halves * cu_count && (kind != kHalfProduct || !half_few_ok(p));
}

template <int KIND, int T, bool SWIGLU>
static void small_launch(const HalfGmmParams &p, hipStream_t stream) {
    hipLaunchKernelGGL((half_small_kernel<KIND, T, SWIGLU>), dim3((unsigned)((small_tiles(p, KIND) + 7) / 8 * 8)), dim3(256), 0,
                       stream, p);
}

hipError_t launch_half_small(const HalfGmmParams &p, int kind, int type, hipStream_t stream) {
    const bool b = type == kBf16;
    if (kind == kHalfWeights) {
        const dim3 grid((unsigned)((small_tiles(p, kind) + 7) / 8 * 8));
        auto kernel = p.gather == 1 ? (b ? half_small_weights_kernel<kBf16, 1> : half_small_weights_kernel<kFp16, 1>)
                                    : (b ? half_small_weights_kernel<kBf16, 2> : half_small_weights_kernel<kFp16, 2>);
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, p);
    } else if (kind == kHalfRows) {
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
