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
// Many rows per expert: 256 x 256 tiles on the matrix cores.  Four waves, one to
// a SIMD, each multiply all rows of the tile by 64 of its columns, so that the
// time of a tile follows its live rows in steps of 32 and no wave idles in a
// ragged one; 16 x 4 fragments of sums fill half of the register file.
//
// A stage is 128 of the reduction: 64 bytes of codes of 256 rows and 256 weight
// rows, copied asynchronously into a ring of four stages in LDS.  The scales of
// four stages (16 bytes a row) travel together, into two buffers.  The barrier
// that publishes stage s + 1 lies in stage s, before its last rows are
// multiplied: behind it the copies of stage s + 3 start (into the slot of stage
// s - 1, which every wave has read) and the first fragments of stage s + 1 are
// read, so that the matrix cores do not wait at a stage's start.
constexpr int kMxTile = 256;                    // rows, and weight rows
constexpr int kMxRing = 4;
constexpr int kMxStageBytes = 2 * kMxTile * 64; // rows then weight rows
constexpr int kMxScaleBytes = 2 * kMxTile * 16;

// 16-byte chunk c of a 64-byte row: the place without bank conflicts for reads of
// one chunk index of 16 consecutive rows by each lane group
__device__ __forceinline__ int mx_swz(int row, int c) { return c ^ ((row >> 1) & 3); }

struct MxTile {
    int e, row0, rows, nblk;
};

// Tile t of the schedule: by expert, weight block, row block, an expert's rows
// split evenly over its row blocks in units of 16.  e = -1 past the last tile.
__device__ __forceinline__ MxTile mx_find_tile(const MxGmmParams &p, int NB, int pid, int (*s_w)[4],
                                               MxTile *s_t) {
    const int e = threadIdx.x, lane = e & (kWave - 1), wave = e >> 6;
    const int first = e < p.E ? mx_row_end(p, e - 1) : 0;
    const int rows = e < p.E ? max(0, mx_row_end(p, e) - first) : 0;
    const int mb = (rows + kMxTile - 1) / kMxTile;
    const int incl = wave_inclusive_scan(mb * NB);
    if (lane == kWave - 1) s_w[0][wave] = incl;
    if (e == 0) s_t->e = -1;
    __syncthreads();
    int pre = incl - mb * NB, total = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        pre += w < wave ? s_w[0][w] : 0;
        total += s_w[0][w];
    }
    // workgroups go round the XCDs: each XCD takes a run of neighbouring tiles, which share
    // weight and row blocks in its L2
    const int per = (total + 7) / 8, at = pid >> 3;
    const int t = (pid & 7) * per + at;
    if (at < per && t >= pre && t < pre + mb * NB) {
        const int local = t - pre, m = local % mb;
        const int nu = (rows + 15) / 16, q = nu / mb, r = nu % mb;
        const int u0 = m * q + min(m, r), u1 = u0 + q + (m < r);
        *s_t = MxTile{e, first + 16 * u0, min(rows, 16 * u1) - 16 * u0, local / mb};
    }
    __syncthreads();
    return *s_t;
}

// One tile of at most 32 NP rows.  (One body for every NP, with the row pairs behind
// conditions, made the compiler move the sums between register files.)
template <bool SWIGLU, int NP>
__device__ __forceinline__ void mx_tile(const MxGmmParams &p, int e, int row0, int rows, int n0,
                                        uint8_t *s_data, uint8_t *s_scale) {
    constexpr int F = SWIGLU ? 2 : 1;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ns = p.Kred / 128;
    const uint32_t qrow = p.Kred / 2, srow = p.Kred / 32;

    // tile weight row r -> weight row of the expert: wave w's 64 are, with SwiGLU, 32 silu
    // columns and the 32 gate columns that go with them
    auto weight_row = [&](int r) {
        const int w = r >> 6, c = r & 63;
        const int col = SWIGLU ? n0 + 32 * w + (c & 31) : n0 + r;
        return min(col, p.N - 1) + (SWIGLU && c >= 32 ? p.N : 0);
    };
    auto data_row = [&](int r) { return (uint32_t)mx_a_row(p, row0 + min(r, rows - 1)); };
    const uint8_t *wq = p.w + (size_t)e * p.N * F * qrow, *ws = p.w_scale + (size_t)e * p.N * F * srow;
    // this wave's copies of a stage: AC of 16 rows and four of 16 weight rows, 1 KB each
    constexpr int AC = NP / 2;
    uint32_t voff_a[AC], voff_w[4];
#pragma unroll
    for (int i = 0; i < AC; ++i) {
        const int r = (wave * AC + i) * 16 + (lane >> 2);
        voff_a[i] = data_row(r) * qrow + mx_swz(r, lane & 3) * 16;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = (wave * 4 + i) * 16 + (lane >> 2);
        voff_w[i] = weight_row(r) * qrow + mx_swz(r, lane & 3) * 16;
    }
    const uint32_t soff_a = data_row(wave * 64 + lane) * srow;
    const uint32_t soff_w = weight_row(wave * 64 + lane) * srow;
    const uint32_t data_lds = __builtin_amdgcn_readfirstlane(lds_addr(s_data));
    const uint32_t scale_lds = __builtin_amdgcn_readfirstlane(lds_addr(s_scale));

    // the 16 scale bytes of stages 4 c .. 4 c + 3; the last ones start early so as to end with the row
    auto scale_start = [&](int c) { return min(16 * c, (int)srow - 16); };
    auto issue = [&](int s) {
        if ((s & 3) == 0) {
            const int c = s >> 2;
            const uint32_t at = scale_lds + (c & 1) * kMxScaleBytes + wave * 1024;
            dma16(p.a_scale + scale_start(c), soff_a, at);
            dma16(ws + scale_start(c), soff_w, at + kMxTile * 16);
        }
        const uint32_t at = data_lds + (s & 3) * kMxStageBytes;
        const uint8_t *ga = p.a + (size_t)s * 64, *gw = wq + (size_t)s * 64;
#pragma unroll
        for (int i = 0; i < AC; ++i) dma16(ga, voff_a[i], at + (wave * AC + i) * 1024);
#pragma unroll
        for (int i = 0; i < 4; ++i) dma16(gw, voff_w[i], at + kMxTile * 64 + (wave * 4 + i) * 1024);
    };

    const int r = lane & 15, g = lane >> 4;
    // lane's place in a fragment of 16 rows, of codes and of scales
    const int frag_off = r * 64 + mx_swz(r, g) * 16, scale_off = r * 16 + g;
    struct Pair {  // two row fragments
        v4i f[2];
        int s[2];
    };
    struct Weights {
        v4i f[4];
        int s[4];
    };
    auto scales = [&](int s) {  // of stage s, of tile row 0
        const int c = s >> 2;
        return s_scale + (c & 1) * kMxScaleBytes + scale_off + 4 * s - scale_start(c);
    };
    auto codes = [&](int s) { return s_data + (s & 3) * kMxStageBytes + frag_off; };
    auto read_w = [&](int s) {
        Weights w;
        const uint8_t *q = codes(s) + (kMxTile + wave * 64) * 64;
        const uint8_t *x = scales(s) + (kMxTile + wave * 64) * 16;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w.f[j] = *reinterpret_cast<const v4i *>(q + 16 * j * 64);
            w.s[j] = x[16 * j * 16];
        }
        return w;
    };
    auto read_a = [&](const uint8_t *q, const uint8_t *x, int pair) {
        Pair a;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            a.f[h] = *reinterpret_cast<const v4i *>(q + (32 * pair + 16 * h) * 64);
            a.s[h] = x[(32 * pair + 16 * h) * 16];
        }
        return a;
    };
    v4f acc[2 * NP][4] = {};
    auto multiply = [&](int pair, const Pair &a, const Weights &w) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[2 * pair + h][j] = mx_mfma(w.f[j], w.s[j], a.f[h], a.s[h], acc[2 * pair + h][j]);
    };

    issue(0);
    issue(1);
    issue(2);  // ns >= 4
    wait_vmcnt<2 * (4 + AC)>();
    __syncthreads();
    // Each pair is read while the one before is multiplied; a stage's first pair and weights while
    // the stage before multiplies its last.
    Weights w = read_w(0);
    Pair a = read_a(codes(0), scales(0), 0);
    for (int s = 0; s < ns; ++s) {
        const uint8_t *q = codes(s), *x = scales(s);
#pragma unroll
        for (int pair = 0; pair + 1 < NP; ++pair) {
            const Pair next = read_a(q, x, pair + 1);
            multiply(pair, a, w);
            a = next;
        }
        Weights w_next = w;
        Pair a_next = a;
        if (s + 1 < ns) {
            // of stage s + 2 its last copies, all but the scales, may be under way still
            if (s + 2 < ns) wait_vmcnt<4 + AC>();
            else wait_vmcnt<0>();
            __syncthreads();
            if (s + 3 < ns) issue(s + 3);
            w_next = read_w(s + 1);
            a_next = read_a(codes(s + 1), scales(s + 1), 0);
        }
        multiply(NP - 1, a, w);
        w = w_next;
        a = a_next;
    }

#pragma unroll
    for (int i = 0; i < 2 * NP; ++i) {
        const int row = 16 * i + r;
        if (row >= rows) continue;
        uint16_t *crow = p.c + (size_t)(row0 + row) * p.N;
#pragma unroll
        for (int j = 0; j < 4 / F; ++j) {
            const int col = n0 + wave * (64 / F) + 16 * j + 4 * g;
            if (col >= p.N) continue;
            uint2 o;
            if (SWIGLU) {
                float y[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) y[v] = silu_times(acc[i][j][v], acc[i][j + 2][v]);
                o = make_uint2(f2bf_pk(y[0], y[1]), f2bf_pk(y[2], y[3]));
            } else {
                o = make_uint2(f2h(acc[i][j][0]) | (uint32_t)f2h(acc[i][j][1]) << 16,
                               f2h(acc[i][j][2]) | (uint32_t)f2h(acc[i][j][3]) << 16);
            }
            *reinterpret_cast<uint2 *>(crow + col) = o;
        }
    }
}

template <bool SWIGLU>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void
mxfp4_gmm_tile_kernel(MxGmmParams p) {
    constexpr int COLS = kMxTile / (SWIGLU ? 2 : 1);  // output columns of a tile
    __shared__ int s_w[1][4];
    __shared__ MxTile s_t;
    __shared__ __align__(16) uint8_t s_data[kMxRing * kMxStageBytes];
    __shared__ __align__(16) uint8_t s_scale[2 * kMxScaleBytes];

    const int NB = (p.N + COLS - 1) / COLS;
    const MxTile tile = mx_find_tile(p, NB, blockIdx.x, s_w, &s_t);
    const int e = __builtin_amdgcn_readfirstlane(tile.e);
    if (e < 0) return;
    const int row0 = __builtin_amdgcn_readfirstlane(tile.row0);
    const int rows = __builtin_amdgcn_readfirstlane(tile.rows);
    const int n0 = __builtin_amdgcn_readfirstlane(tile.nblk) * COLS;
    if (rows > 192) mx_tile<SWIGLU, 8>(p, e, row0, rows, n0, s_data, s_scale);
    else if (rows > 128) mx_tile<SWIGLU, 6>(p, e, row0, rows, n0, s_data, s_scale);
    else if (rows > 64) mx_tile<SWIGLU, 4>(p, e, row0, rows, n0, s_data, s_scale);
    else mx_tile<SWIGLU, 2>(p, e, row0, rows, n0, s_data, s_scale);
}

template <bool SWIGLU>
static void launch_tile(const MxGmmParams &p, hipStream_t stream) {
    const int cols = kMxTile / (SWIGLU ? 2 : 1);
    const long long ub = ((long long)p.R / kMxTile + (p.E < p.R ? p.E : p.R)) * ((p.N + cols - 1) / cols);
    hipLaunchKernelGGL(mxfp4_gmm_tile_kernel<SWIGLU>, dim3((unsigned)((ub + 7) / 8 * 8)), dim3(256), 0,
                       stream, p);
}

hipError_t launch_mxfp4_gmm(const MxGmmParams &p, bool swiglu, int cu_count, hipStream_t stream) {
    (void)cu_count;
    const int mean = (p.R + p.E - 1) / p.E;
    // the tiles' scale copies take 16 bytes of a row
    const bool tiles = mean > 32 && p.Kred >= 512;
    if (swiglu) tiles ? launch_tile<true>(p, stream) : launch_stream<true>(p, stream);
    else tiles ? launch_tile<false>(p, stream) : launch_stream<false>(p, stream);
    return hipGetLastError();
}

}  // namespace megamoe
