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
#include "dma.hpp"
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

// ---------------------------------------------------------------------------
// Many rows per expert: tiles of 256 rows by 256 weight rows on the matrix cores.
// Four waves, one to a SIMD, each multiply all rows of the tile by 64 of its
// weight rows, so that the time of a tile follows its live rows in steps of 64 and
// no wave idles in a ragged one; 8 x 2 fragments of 32 x 32 sums fill half of the
// register file.  (v_mfma_scale_f32_32x32x64_f8f6f4 ran at 9.3 PFLOP/s from registers,
// the 16x16x128 form at 5.5.)
//
// A stage is 256 of the reduction: 128 bytes of codes, a whole cache line, of 256
// rows and 256 weight rows, copied asynchronously into one of two slots in LDS.
// (Stages of half a line took twice the requests for the same bytes, and the L2's
// request rate bound the kernel.)  The scales of two stages (16 bytes a row)
// travel together, into two buffers.  The barrier between stages s and s + 1 lies
// before the last rows of stage s are multiplied: those are in registers by then,
// so behind it the copies of stage s + 2 start, into the slot of stage s, and the
// first fragments of stage s + 1 are read.
//
// The grid is persistent.  While a tile is multiplied the workgroup looks up its
// next one, and the first two stages of that are copied while this one's sums
// are stored.
constexpr int kMxTile = 256;                    // rows, and weight rows
constexpr int kMxStageBytes = 2 * kMxTile * 128; // rows then weight rows
constexpr int kMxScaleBytes = 2 * kMxTile * 16;
constexpr int kMxTileThreads = 256;
constexpr int kMxE = 256;
constexpr int kMxList = 32;

typedef float v16f __attribute__((ext_vector_type(16)));

// 32 x 32 x 64 with weights as the first operand: lane l holds output row l & 31 and
// the columns 8 q + 4 (l >> 5) + 0..3, q = 0..3.  Of either operand lane l has row
// l & 31 and the codes of block l >> 5; their scale is byte 2 H of the scale word.
template <int H>
__device__ __forceinline__ v16f mx_mfma32(v4i w, int ws, v4i a, int as, v16f acc) {
    const v8i w8 = {w[0], w[1], w[2], w[3], 0, 0, 0, 0}, a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w8, a8, acc, 4, 4, 2 * H, ws, 2 * H, as);
}

// 16-byte chunk c of a 128-byte row: the place without bank conflicts for reads of
// one chunk index of consecutive rows
__device__ __forceinline__ int mx_swz(int row, int c) { return c ^ (row & 7); }

// The tiles, numbered by expert, weight block and row block; an expert's rows are
// split evenly over its row blocks in units of 32.
struct MxSchedule {
    int pre[kMxE + 1];  // tiles of the experts before e
    int first[kMxE], rows[kMxE];
    int total;
};
__device__ __forceinline__ void mx_schedule(const MxGmmParams &p, int NB, int *s_w, MxSchedule &s) {
    const int e = threadIdx.x, lane = e & (kWave - 1), wave = e >> 6;
    const int first = e < p.E ? mx_row_end(p, e - 1) : 0;
    const int rows = e < p.E ? max(0, mx_row_end(p, e) - first) : 0;
    const int tiles = (rows + kMxTile - 1) / kMxTile * NB;
    const int incl = wave_inclusive_scan(tiles);
    if (lane == kWave - 1) s_w[wave] = incl;
    __syncthreads();
    int pre = incl - tiles;
#pragma unroll
    for (int w = 0; w < 4; ++w) pre += w < wave ? s_w[w] : 0;
    s.pre[e] = pre;  // experts past E have no tiles: pre is the total
    s.first[e] = first;
    s.rows[e] = rows;
    if (e == kMxE - 1) s.pre[kMxE] = s.total = pre + tiles;
    __syncthreads();
}

struct MxTile {
    int e, row0, rows, nblk;
};
__device__ __forceinline__ MxTile mx_find_tile(const MxSchedule &s, int t) {  // t < total
    int lo = 0, hi = kMxE - 1;  // the first expert that ends after t
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s.pre[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    const int rows = s.rows[lo], local = t - s.pre[lo];
    const int mb = (rows + kMxTile - 1) / kMxTile, m = local % mb;
    const int nu = (rows + 31) / 32, q = nu / mb, r = nu % mb;
    const int u0 = m * q + min(m, r), u1 = u0 + q + (m < r);
    return MxTile{lo, s.first[lo] + 32 * u0, min(rows, 32 * u1) - 32 * u0, local / mb};
}

// What the copies of a tile need.
struct MxCopies {
    uint32_t voff_a[8], voff_w[8], soff_a, soff_w;  // per lane
    const uint8_t *wq, *ws;                         // the expert's weights and scales
    int ac;                                         // copies of 8 rows a wave makes, 2 for 64 rows
};

struct MxLds {
    uint8_t *data, *scale;
    uint32_t data_at, scale_at;  // their LDS addresses
    int32_t *route;              // [256] A rows of the next tile, as sorted routes
};

template <bool SWIGLU>
__device__ __forceinline__ MxCopies mx_copies(const MxGmmParams &p, const MxTile &t, const MxLds &l) {
    constexpr int F = SWIGLU ? 2 : 1;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t qrow = p.Kred / 2, srow = p.Kred / 32;
    const int n0 = t.nblk * (kMxTile / F);
    // tile weight row r -> weight row of the expert: wave w's 64 are, with SwiGLU, 32 silu
    // columns and the 32 gate columns that go with them
    auto weight_row = [&](int r) {
        const int w = r >> 6, c = r & 63;
        const int col = SWIGLU ? n0 + 32 * w + (c & 31) : n0 + r;
        return min(col, p.N - 1) + (SWIGLU && c >= 32 ? p.N : 0);
    };
    auto data_row = [&](int r) {
        r = min(r, t.rows - 1);
        if (!p.a_route) return t.row0 + r;
        const int v = l.route[r];
        const uint32_t u = v < 0 ? 0 : v < p.R ? v : p.R - 1;
        return p.a_div == 1 ? (int)u : (int)__umulhi(u, p.a_div_inv);
    };
    MxCopies c;
    c.ac = (t.rows + 63) / 64 * 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = (wave * c.ac + i) * 8 + (lane >> 3);
        c.voff_a[i] = (uint32_t)data_row(i < c.ac ? r : 0) * qrow + mx_swz(r, lane & 7) * 16;
        const int n = (wave * 8 + i) * 8 + (lane >> 3);
        c.voff_w[i] = (uint32_t)weight_row(n) * qrow + mx_swz(n, lane & 7) * 16;
    }
    c.soff_a = (uint32_t)data_row(wave * 64 + lane) * srow;
    c.soff_w = (uint32_t)weight_row(wave * 64 + lane) * srow;
    c.wq = uniform_ptr(p.w + (size_t)t.e * p.N * F * qrow);
    c.ws = uniform_ptr(p.w_scale + (size_t)t.e * p.N * F * srow);
    return c;
}

// Where a piece of `size` bytes starts in a row of n: the last one early, so as to end with the
// row (n is not a multiple of it where the reduction is not one of 256, for codes, or 512).
__device__ __forceinline__ int mx_start(int piece, int size, int n) { return min(piece * size, n - size); }

// The copies of stage s: at every second stage 2 of scales, then ac of rows and 8 of
// weight rows.  AC: ac where it is known (0: not).
template <int AC>
__device__ __forceinline__ void mx_issue(const MxGmmParams &p, const MxCopies &c, const MxLds &l, int s) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ac = AC ? AC : c.ac;
    if ((s & 1) == 0) {
        const int start = mx_start(s >> 1, 16, p.Kred / 32);
        const uint32_t at = l.scale_at + ((s >> 1) & 1) * kMxScaleBytes + wave * 1024;
        dma16(uniform_ptr(p.a_scale + start), c.soff_a, at);
        dma16(uniform_ptr(c.ws + start), c.soff_w, at + kMxTile * 16);
    }
    const uint32_t at = l.data_at + (s & 1) * kMxStageBytes;
    const int start = mx_start(s, 128, p.Kred / 2);
    const uint8_t *ga = uniform_ptr(p.a + start), *gw = uniform_ptr(c.wq + start);
#pragma unroll
    for (int i = 0; i < (AC ? AC : 8); ++i)
        if (AC || i < ac) dma16(ga, c.voff_a[i], at + (wave * ac + i) * 1024);
#pragma unroll
    for (int i = 0; i < 8; ++i) dma16(gw, c.voff_w[i], at + kMxTile * 128 + (wave * 8 + i) * 1024);
}

// silu(u) * g for a result that is rounded to bf16: the reciprocal's last ulp is not corrected
__device__ __forceinline__ float mx_silu_times(float u, float g) {
    const float d = __builtin_amdgcn_exp2f(u * -1.4426950408889634f) + 1.0f;
    return u * __builtin_amdgcn_rcpf(d) * g;
}

// One sum out of the accumulation registers.  (Left to the compiler, all 256 are copied
// at once and other values spill.)
__device__ __forceinline__ float mx_sum(float a) {
    float v;
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(a));
    return v;
}

// Multiplies tile t, of at most 32 NP rows, whose first stage is in LDS and whose second is
// under way, and rounds and stores its sums while the first stages of tile `nt` are copied.
// (One body for every NP, with the rows behind conditions, made the compiler move the sums
// between register files.)
template <bool SWIGLU, int NP>
__device__ __forceinline__ void mx_tile(const MxGmmParams &p, const MxTile &t, MxCopies &c,
                                        bool more, const MxTile &nt, const MxLds &l) {
    constexpr int F = SWIGLU ? 2 : 1;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ns = (p.Kred + 255) / 256;
    const bool half = p.Kred % 256 != 0;  // of the last stage's row pieces the second halves alone

    const int r = lane & 31, g = lane >> 5;
    int frag_off[4];  // lane's place in 32 rows of a stage, 64 of the reduction each
#pragma unroll
    for (int h = 0; h < 4; ++h) frag_off[h] = r * 128 + mx_swz(r, 2 * h + g) * 16;
    // LDS addresses of stage s, tile row 0
    auto codes = [&](int s) { return l.data + (s & 1) * kMxStageBytes; };
    auto scales = [&](int s) {
        return l.scale + ((s >> 1) & 1) * kMxScaleBytes + r * 16 + mx_start(s, 8, p.Kred / 32) -
               mx_start(s >> 1, 16, p.Kred / 32);
    };
    // 32 rows of a stage: four fragments, and the rows' eight scale bytes
    auto read = [&](const uint8_t *q, const uint8_t *x, int row, v4i (&f)[4], int (&sc)[2]) {
#pragma unroll
        for (int h = 0; h < 4; ++h)
            f[h] = *reinterpret_cast<const v4i *>(q + row * 128 + frag_off[h]);
        sc[0] = (int)*reinterpret_cast<const uint32_t *>(x + row * 16);
        sc[1] = (int)*reinterpret_cast<const uint32_t *>(x + row * 16 + 4);
    };
    auto read_w = [&](int s, v4i (&f)[2][4], int (&sc)[2][2]) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            read(codes(s), scales(s), kMxTile + wave * 64 + 32 * j, f[j], sc[j]);
    };
    v16f acc[NP][2] = {};
    v4i w[2][4], a[2][4];  // weights of the stage, rows of the two fragments that are multiplied
    int wsc[2][2], asc[2][2];
    auto read_a = [&](const uint8_t *q, const uint8_t *x, int pair, v4i (&f)[2][4], int (&sc)[2][2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) read(q, x, 64 * pair + 32 * i, f[i], sc[i]);
    };
    // Two row fragments by two weight fragments: four sums that take turns, so that no product
    // waits for the one before it.  (With two, the loop ran at half the rate.)
    auto multiply = [&](int pair, int first_half) {  // first_half: 0 or -1
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            asc[i][0] >>= 8 * g;  // the lane's blocks are g and 2 + g of each half
            asc[i][1] >>= 8 * g;
            // Codes of 0 where the first half has been multiplied before.  (A NaN scale makes a
            // NaN of them, but where it did so before.)
            a[i][0] &= first_half;
            a[i][1] &= first_half;
        }
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    v16f &d = acc[2 * pair + i][j];
                    d = h & 1 ? mx_mfma32<1>(w[j][h], wsc[j][h >> 1], a[i][h], asc[i][h >> 1], d)
                              : mx_mfma32<0>(w[j][h], wsc[j][h >> 1], a[i][h], asc[i][h >> 1], d);
                }
        // the sums are wanted here: without this the compiler puts a stage's products together
        // behind its barrier and copies, where the reads no longer overlap them
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) asm volatile("" : "+a"(acc[2 * pair + i][j]));
    };

    // Each pair of fragments is read while the one before is multiplied; a stage's first pair and
    // weights while the stage before multiplies its last.
    read_w(0, w, wsc);
    read_a(codes(0), scales(0), 0, a, asc);
#pragma unroll 1
    for (int s = 0; s < ns; ++s) {
        const uint8_t *q = codes(s), *x = scales(s);
        const int first_half = half && s + 1 == ns ? 0 : -1;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            wsc[j][0] >>= 8 * g;
            wsc[j][1] >>= 8 * g;
        }
        v4i na[2][4];
        int nasc[2][2];
        auto shift = [&]() {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int h = 0; h < 4; ++h) a[i][h] = na[i][h];
                asc[i][0] = nasc[i][0];
                asc[i][1] = nasc[i][1];
            }
        };
#pragma unroll
        for (int pair = 0; pair + 1 < NP / 2; ++pair) {
            read_a(q, x, pair + 1, na, nasc);
            __builtin_amdgcn_sched_barrier(0);
            multiply(pair, first_half);
            __builtin_amdgcn_sched_barrier(0);
            shift();
        }
        v4i nw[2][4] = {};
        int nwsc[2][2] = {};
        if (s + 1 < ns) {
            wait_vmcnt<0>();  // stage s + 1
            __syncthreads();
            if (s + 2 < ns) mx_issue<NP>(p, c, l, s + 2);
            read_w(s + 1, nw, nwsc);
            read_a(codes(s + 1), scales(s + 1), 0, na, nasc);
        }
        __builtin_amdgcn_sched_barrier(0);
        multiply(NP / 2 - 1, first_half);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int h = 0; h < 4; ++h) w[j][h] = nw[j][h];
            wsc[j][0] = nwsc[j][0];
            wsc[j][1] = nwsc[j][1];
        }
        shift();
    }

    if (more) {
        __syncthreads();  // every wave has read the last stage, and the next tile's routes are there
        c = mx_copies<SWIGLU>(p, nt, l);
        mx_issue<0>(p, c, l, 0);
        mx_issue<0>(p, c, l, 1);
    }
    // Four columns a lane, rounded; then lanes l and l + 32 exchange halves of two such groups, so
    // that each holds eight columns in a row and stores 16 bytes.
    constexpr int J = 2 / F;
    uint2 out[NP][J][4];
    // the last product's result is there after 18 wait states
    asm volatile("s_nop 15\n\ts_nop 15");
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        __builtin_amdgcn_sched_barrier(0);  // a few sums at a time leave the accumulators
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float y[4];
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    y[v] = SWIGLU ? mx_silu_times(mx_sum(acc[i][0][4 * k + v]),
                                                  mx_sum(acc[i][1][4 * k + v]))
                                  : mx_sum(acc[i][j][4 * k + v]);
                out[i][j][k] = SWIGLU ? make_uint2(f2bf_pk(y[0], y[1]), f2bf_pk(y[2], y[3]))
                                      : make_uint2(f2h(y[0]) | (uint32_t)f2h(y[1]) << 16,
                                                   f2h(y[2]) | (uint32_t)f2h(y[3]) << 16);
                // rounded here, not in the blocks of the stores: half the registers
                asm volatile("" : "+v"(out[i][j][k].x), "+v"(out[i][j][k].y));
            }
    }
    __builtin_amdgcn_sched_barrier(0);
    const int n0 = t.nblk * (kMxTile / F) + wave * (64 / F);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int row = 32 * i + r;
        uint16_t *crow = p.c + (size_t)(t.row0 + row) * p.N;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
                const auto x = __builtin_amdgcn_permlane32_swap(out[i][j][k].x, out[i][j][k + 1].x, false, false);
                const auto y = __builtin_amdgcn_permlane32_swap(out[i][j][k].y, out[i][j][k + 1].y, false, false);
                const int col = n0 + 32 * j + 8 * (k + g);
                if (row < t.rows && col < p.N)
                    *reinterpret_cast<uint4 *>(crow + col) = make_uint4(x[0], y[0], x[1], y[1]);
            }
    }
    if (more) {
        // The first stage's copies are older than the second's, 10 at least, and than the stores:
        // all but the last two fragments have whole rows, so at least that many were issued,
        // unless columns past N were left out.
        if (n0 + 64 / F <= p.N) wait_vmcnt<10 + (NP - 2) * J * 2>();
        else wait_vmcnt<10>();
        __syncthreads();
    }
}

template <bool SWIGLU>
__global__ __launch_bounds__(kMxTileThreads) __attribute__((amdgpu_waves_per_eu(1, 1))) void
mxfp4_gmm_tile_kernel(MxGmmParams p) {
    constexpr int COLS = kMxTile / (SWIGLU ? 2 : 1);  // output columns of a tile
    __shared__ int s_w[4];
    __shared__ MxSchedule s_s;
    __shared__ MxTile s_t[kMxList];
    __shared__ int32_t s_route[kMxTile];
    __shared__ __align__(16) uint8_t s_data[2 * kMxStageBytes];
    __shared__ __align__(16) uint8_t s_scale[2 * kMxScaleBytes];

    mx_schedule(p, (p.N + COLS - 1) / COLS, s_w, s_s);
    const int total = __builtin_amdgcn_readfirstlane(s_s.total);
    // workgroups go round the XCDs: each XCD takes a run of neighbouring tiles, which share
    // weight and row blocks in its L2
    const int per = (total + 7) / 8, step = gridDim.x >> 3;
    const int t0 = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    const int t1 = min((int)(blockIdx.x & 7) * per + per, total);
    const int n = t0 < t1 ? (t1 - t0 + step - 1) / step : 0;  // tiles of this workgroup
    if (n == 0) return;

    const MxLds l{s_data, s_scale, (uint32_t)__builtin_amdgcn_readfirstlane(lds_addr(s_data)),
                  (uint32_t)__builtin_amdgcn_readfirstlane(lds_addr(s_scale)),
                  s_route};
    const int tid = threadIdx.x;
    const uint32_t route_at =
        __builtin_amdgcn_readfirstlane(lds_addr(s_route) + (tid >> 6) * (kWave * 4));
    auto fetch_routes = [&](const MxTile &x) {
        if (p.a_route) dma4(p.a_route + x.row0 + min(tid, x.rows - 1), route_at);
    };
    // its tiles are looked up kMxList at a time, a lane each
    auto look_up = [&](int k) {
        if (tid < kMxList && k + tid < n) s_t[tid] = mx_find_tile(s_s, t0 + (k + tid) * step);
        __syncthreads();
    };
    auto tile = [&](int k) {
        const MxTile &x = s_t[k % kMxList];
        return MxTile{__builtin_amdgcn_readfirstlane(x.e), __builtin_amdgcn_readfirstlane(x.row0),
                      __builtin_amdgcn_readfirstlane(x.rows), __builtin_amdgcn_readfirstlane(x.nblk)};
    };
    look_up(0);
    MxTile cur = tile(0);
    fetch_routes(cur);
    wait_vmcnt<0>();
    __syncthreads();
    MxCopies c = mx_copies<SWIGLU>(p, cur, l);
    mx_issue<0>(p, c, l, 0);
    mx_issue<0>(p, c, l, 1);  // at least 2 stages
    wait_vmcnt<10>();
    __syncthreads();
    for (int k = 1;; ++k) {
        const bool more = k < n;
        if (more && k % kMxList == 0) look_up(k);  // the last tiles of the list have been read
        const MxTile next = more ? tile(k) : cur;
        if (more) fetch_routes(next);
        if (cur.rows > 192) mx_tile<SWIGLU, 8>(p, cur, c, more, next, l);
        else if (cur.rows > 128) mx_tile<SWIGLU, 6>(p, cur, c, more, next, l);
        else if (cur.rows > 64) mx_tile<SWIGLU, 4>(p, cur, c, more, next, l);
        else mx_tile<SWIGLU, 2>(p, cur, c, more, next, l);
        if (!more) return;
        cur = next;
    }
}

template <bool SWIGLU>
static void launch_tile(const MxGmmParams &p, int cu_count, hipStream_t stream) {
    const int cols = kMxTile / (SWIGLU ? 2 : 1);
    // at most this many tiles; one workgroup fits a CU
    const long long most =
        ((long long)p.R / kMxTile + (p.E < p.R ? p.E : p.R)) * ((p.N + cols - 1) / cols);
    const long long g = most < cu_count ? most : cu_count;
    hipLaunchKernelGGL(mxfp4_gmm_tile_kernel<SWIGLU>, dim3((unsigned)((g + 7) / 8 * 8)),
                       dim3(kMxTileThreads), 0, stream, p);
}

hipError_t launch_mxfp4_gmm(const MxGmmParams &p, bool swiglu, int cu_count, hipStream_t stream) {
    const int mean = (p.R + p.E - 1) / p.E;
    // the tiles' scale copies take 16 bytes of a row
    const bool tiles = mean > 32 && p.Kred >= 512;
    if (swiglu) tiles ? launch_tile<true>(p, cu_count, stream) : launch_stream<true>(p, stream);
    else tiles ? launch_tile<false>(p, cu_count, stream) : launch_stream<false>(p, stream);
    return hipGetLastError();
}

}  // namespace megamoe
