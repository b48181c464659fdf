// Grouped product of MXFP4 rows and MXFP4 weights (the place of GMM1 and GMM2,
// sections 3 and 5 of the pto-isa MegaMoE overview page, with 4-bit experts).
//
// For every row of expert e's group, p[n] = sum_k a[k] * w[e][n][k] over the
// values that codes and block scales stand for, in fp32 on the matrix cores:
// v_mfma_scale_f32_32x32x64_f8f6f4 takes 32 codes of a lane (one block) with
// their scale byte.  GMM1 ends in SwiGLU: column n meets column N + n in the same
// lane's accumulators, and silu(p[n]) * p[N + n] goes out as bf16 or, where cq is set,
// rounded to bf16 and then to MXFP4 as mxfp4_quant_kernel does; GMM2's p goes out as fp16.
#include <type_traits>

#include "common.hpp"
#include "dma.hpp"
#include "kernels.hpp"
#include "mxfp4_row.hpp"
#include "swiglu_row.hpp"

namespace megamoe {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

// first row and row count of expert e's group, within [0, R]
__device__ __forceinline__ int mx_row_end(const MxGmmParams &p, int e) {
    const int v = e >= 0 ? p.cumsum[e] : 0;
    return v < 0 ? 0 : v > p.R ? p.R : v;
}

// Both kernels below work through tiles of AR rows by WR weight rows, four waves to a
// tile, each multiplying all of its rows by a quarter of its weight rows with
// v_mfma_scale_f32_32x32x64_f8f6f4.  (From registers that ran at 9.3 PFLOP/s on constant
// operands and 6.5 on random ones, where the card throttles; the 16x16x128 form at 5.5.)
//
// A stage is 256 of the reduction: 128 bytes of codes, a whole cache line, of every
// row, copied asynchronously into LDS.  (Stages of half a line took twice the
// requests for the same bytes.)  The scales of two stages, 16 bytes a row, travel
// together.  Where the reduction ends inside a stage, the last piece of a row starts
// early so as to end with it, and what it holds a second time is multiplied as 0.
constexpr int kMxThreads = 256;
constexpr int kMxE = 256;

template <bool SWIGLU_, int AR_, int WR_>
struct MxGeom {
    static constexpr bool SWIGLU = SWIGLU_;
    static constexpr int AR = AR_, WR = WR_;
    static constexpr int COLS = SWIGLU ? WR / 2 : WR;  // output columns
    static constexpr int WRW = WR / 4;                 // weight rows of a wave
    static constexpr int STAGE = (AR + WR) * 128;      // bytes of a stage: rows, then weight rows
    static constexpr int SCALE = (AR + WR) * 16;       // bytes of two stages' scales
    static constexpr int AC = AR / 32, WC = WR / 32;   // copies of 8 rows a wave makes, at most
    static constexpr int SC = (AR + WR + 255) / 256;   // copies of 64 rows' scales
};

// 32 x 32 x 64 with weights as the first operand: lane l holds output row l & 31 and
// the columns 8 q + 4 (l >> 5) + 0..3, q = 0..3.  Of either operand lane l has row
// l & 31 and the codes of block l >> 5; their scale is byte 2 H of the scale word.
template <int H>
__device__ __forceinline__ v16f mx_mfma32(v4i w, int ws, v4i a, int as, v16f acc) {
    const v8i w8 = {w[0], w[1], w[2], w[3], 0, 0, 0, 0}, a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w8, a8, acc, 4, 4, 2 * H, ws, 2 * H, as);
}

// 16-byte chunk c of a 128-byte row: its place.  LDS has 64 banks, two rows; reads of one chunk
// index of 16 rows in the order of the lanes meet each bank once.
__device__ __forceinline__ int mx_swz(int row, int c) { return c ^ (row >> 1 & 7); }

// The tiles, numbered by expert, weight block and row block; an expert's rows are
// split evenly over its row blocks in units of 32.
struct MxSchedule {
    int pre[kMxE + 1];  // tiles of the experts before e
    int first[kMxE], rows[kMxE];
    int total;
};
template <typename G>
__device__ __forceinline__ void mx_schedule(const MxGmmParams &p, int *s_w, MxSchedule &s) {
    const int e = threadIdx.x, lane = e & (kWave - 1), wave = e >> 6;
    const int first = e < p.E ? mx_row_end(p, e - 1) : 0;
    const int rows = e < p.E ? max(0, mx_row_end(p, e) - first) : 0;
    const int tiles = (rows + G::AR - 1) / G::AR * ((p.N + G::COLS - 1) / G::COLS);
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
template <typename G>
__device__ __forceinline__ MxTile mx_find_tile(const MxSchedule &s, int t) {  // t < total
    int lo = 0, hi = kMxE - 1;  // the first expert that ends after t
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s.pre[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    const int rows = s.rows[lo], local = t - s.pre[lo];
    const int mb = (rows + G::AR - 1) / G::AR, m = local % mb;
    const int nu = (rows + 31) / 32, q = nu / mb, r = nu % mb;
    const int u0 = m * q + min(m, r), u1 = u0 + q + (m < r);
    return MxTile{lo, s.first[lo] + 32 * u0, min(rows, 32 * u1) - 32 * u0, local / mb};
}
__device__ __forceinline__ MxTile mx_uniform(const MxTile &x) {
    return MxTile{__builtin_amdgcn_readfirstlane(x.e), __builtin_amdgcn_readfirstlane(x.row0),
                  __builtin_amdgcn_readfirstlane(x.rows), __builtin_amdgcn_readfirstlane(x.nblk)};
}

struct MxLds {
    uint8_t *data, *scale;
    uint32_t data_at, scale_at;  // their LDS addresses
    int32_t *route;              // [AR] rows of the tile that is copied next, as sorted routes
    uint16_t *most;              // [4][AR] a wave's largest |y| of a row (narrow tiles)
};

// row r of tile t -> row of A; rows past the group are its last one
__device__ __forceinline__ uint32_t mx_data_row(const MxGmmParams &p, const MxTile &t, const MxLds &l,
                                                int r) {
    r = min(r, t.rows - 1);
    if (!p.a_route) return t.row0 + r;
    const int v = l.route[r];
    const uint32_t u = v < 0 ? 0 : v < p.R ? v : p.R - 1;
    return p.a_div == 1 ? u : __umulhi(u, p.a_div_inv);
}
// weight row r of tile t -> weight row of the expert: with SwiGLU a wave's are as many silu
// columns and the gate columns that go with them
template <typename G>
__device__ __forceinline__ uint32_t mx_weight_row(const MxGmmParams &p, const MxTile &t, int r) {
    const int w = r / G::WRW, c = r % G::WRW;
    constexpr int H = G::WRW / 2;
    const int col = t.nblk * G::COLS + (G::SWIGLU ? H * w + c % H : r);
    return min(col, p.N - 1) + (G::SWIGLU && c >= H ? p.N : 0);
}

// What the copies of a tile need.
template <typename G>
struct MxCopies {
    uint32_t voff_a[G::AC], voff_w[G::WC], soff[G::SC];  // per lane
    const uint8_t *wq, *ws;                              // the expert's weights and scales
    int ac;                                              // copies of 8 rows a wave makes
};
// Copy i of scales is of 64 weight rows or, past them, of 64 rows (the last ones again where the
// copies are more).
template <typename G>
__device__ __forceinline__ int mx_scale_copy(int i, int wave) {
    return min(4 * i + wave, (G::AR + G::WR) / 64 - 1);
}
// unit: rows go to the waves 32 * unit at a time
template <typename G>
__device__ __forceinline__ MxCopies<G> mx_copies(const MxGmmParams &p, const MxTile &t, const MxLds &l,
                                                 int unit) {
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t qrow = p.Kred / 2, srow = p.Kred / 32;
    constexpr int F = G::SWIGLU ? 2 : 1;
    MxCopies<G> c;
    c.ac = (t.rows + 32 * unit - 1) / (32 * unit) * unit;
    // a row of 64 bytes: its piece starts 64 bytes early, and what lies there is not its own
    auto place = [&](int r) {
        const int chunk = mx_swz(r, lane & 7);
        return chunk * 16 + (qrow < 128 && chunk < 4 ? 64 : 0);
    };
#pragma unroll
    for (int i = 0; i < G::AC; ++i) {
        const int r = (wave * c.ac + i) * 8 + (lane >> 3);
        c.voff_a[i] = mx_data_row(p, t, l, i < c.ac ? r : 0) * qrow + place(r);
    }
#pragma unroll
    for (int i = 0; i < G::WC; ++i) {
        const int r = (wave * G::WC + i) * 8 + (lane >> 3);
        c.voff_w[i] = mx_weight_row<G>(p, t, r) * qrow + place(r);
    }
#pragma unroll
    for (int i = 0; i < G::SC; ++i) {
        const int k = mx_scale_copy<G>(i, wave);
        c.soff[i] = srow * (k < G::WR / 64 ? mx_weight_row<G>(p, t, 64 * k + lane)
                                           : mx_data_row(p, t, l, 64 * k - G::WR + lane));
    }
    c.wq = uniform_ptr(p.w + (size_t)t.e * p.N * F * qrow);
    c.ws = uniform_ptr(p.w_scale + (size_t)t.e * p.N * F * srow);
    return c;
}

// Where a piece of `size` bytes starts in a row of n: the last one early, so as to end with the row.
__device__ __forceinline__ int mx_start(int piece, int size, int n) { return min(piece * size, n - size); }
// the same for the 16 bytes of two stages' scales, the row's start where it is shorter
__device__ __forceinline__ int mx_scale_start(int s, int n) { return max(0, mx_start(s >> 1, 16, n)); }

// Scales of rows under 16 bytes are all of two stages; a 16-byte copy of the last one would
// pass the buffer's end, so they are read and written word by word, with the first stage.
template <typename G>
__device__ __forceinline__ void mx_short_scales(const MxGmmParams &p, const MxTile &t,
                                                const MxCopies<G> &c, const MxLds &l, int sbuf) {
    const int srow = p.Kred / 32;
    if (srow >= 16) return;
    for (int r = threadIdx.x; r < G::AR + G::WR; r += kMxThreads) {
        const uint8_t *q = r < G::AR ? p.a_scale + (size_t)mx_data_row(p, t, l, r) * srow
                                     : c.ws + (size_t)mx_weight_row<G>(p, t, r - G::AR) * srow;
        for (int k = 0; k < srow; k += 4)
            *reinterpret_cast<uint32_t *>(l.scale + sbuf * G::SCALE + r * 16 + k) = *reinterpret_cast<const uint32_t *>(q + k);
    }
}

// Weights are copied with the non-temporal hint: whoever shares a block of them asks for it at
// the same time.  (K = 7168, I = 2048, E = 32, top_k = 8, gmm1 / gmm2 in us with it and without: 1 token
// 22.8 / - and 25.3, 128 tokens 90 and 95, 512 tokens - / 74 and 81, after other work has filled the
// caches 120 / 91 and 150 / 111; 2048 tokens 319 / 197 and 331 / 206.  Where one expert has a
// dozen row blocks, which pass in two or more rounds, it costs 3%: gmm2 of 4096 skewed tokens 166 and
// 160.)  Scales are not: a copy takes 16 bytes of a line.  (With it 128 tokens took 103.)
//
// The copies of stage s into slot `slot`, and of scales, with every second stage, into scale buffer
// `sbuf`: WC + SC of weight rows and scales, ac of rows.
template <typename G>
struct MxIssueW {
    static constexpr int N = G::WC + G::SC;
    const MxCopies<G> &c;
    const uint8_t *gw, *gs, *ga;
    uint32_t at, scale_at;
    int wave;
    bool scales;
    __device__ __forceinline__ MxIssueW(const MxGmmParams &p, const MxCopies<G> &c_, const MxLds &l, int s,
                                        int slot, int sbuf)
        : c(c_) {
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int srow = p.Kred / 32, start = mx_scale_start(s, srow);
        scales = (s & 1) == 0 && srow >= 16;
        gs = uniform_ptr(c.ws + start);
        ga = uniform_ptr(p.a_scale + start);
        scale_at = l.scale_at + sbuf * G::SCALE;
        gw = uniform_ptr(c.wq + mx_start(s, 128, p.Kred / 2));
        at = l.data_at + slot * G::STAGE + G::AR * 128 + wave * G::WC * 1024;
    }
    __device__ __forceinline__ void copy(int i) const {  // 0 <= i < N
        if (i < G::WC) {
            dma16_nt(gw, c.voff_w[i], at + i * 1024);
        } else if (scales) {
            const int k = mx_scale_copy<G>(i - G::WC, wave);
            const bool w = k < G::WR / 64;
            dma16(uniform_ptr(w ? gs : ga), c.soff[i - G::WC], scale_at + (w ? G::AR + 64 * k : 64 * k - G::WR) * 16);
        }
    }
};
template <typename G, int AC>  // AC: ac where it is known (0: not)
struct MxIssueA {
    static constexpr int N = AC ? AC : G::AC;
    const MxCopies<G> &c;
    const uint8_t *ga;
    uint32_t at;
    int ac;
    __device__ __forceinline__ MxIssueA(const MxGmmParams &p, const MxCopies<G> &c_, const MxLds &l, int s,
                                        int slot)
        : c(c_) {
        ac = AC ? AC : c.ac;
        ga = uniform_ptr(p.a + mx_start(s, 128, p.Kred / 2));
        at = l.data_at + slot * G::STAGE + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * ac * 1024;
    }
    __device__ __forceinline__ void copy(int i) const {  // 0 <= i < N
        if (AC || i < ac) dma16(ga, c.voff_a[i], at + i * 1024);
    }
};
template <typename I>
__device__ __forceinline__ void mx_all(const I &issue, int from = 0, int to = I::N) {
#pragma unroll
    for (int i = from; i < to; ++i) issue.copy(i);
}
template <typename G, int AC>
__device__ __forceinline__ void mx_issue(const MxGmmParams &p, const MxCopies<G> &c, const MxLds &l, int s,
                                         int slot, int sbuf) {
    mx_all(MxIssueW<G>(p, c, l, s, slot, sbuf));
    mx_all(MxIssueA<G, AC>(p, c, l, s, slot));
}

// Reads of a stage in LDS: 32 rows from `row`, four fragments of 64 of the reduction and eight scale bytes.
template <typename G>
struct MxStage {
    const uint8_t *q, *x;
    __device__ __forceinline__ MxStage(const MxGmmParams &p, const MxLds &l, int s, int slot, int sbuf) {
        const int r = threadIdx.x & 31, srow = p.Kred / 32;
        q = l.data + slot * G::STAGE + r * 128;
        x = l.scale + sbuf * G::SCALE + r * 16 + mx_start(s, 8, srow) - mx_scale_start(s, srow);
    }
    __device__ __forceinline__ void codes(int row, int place, v4i &f) const {
        f = *reinterpret_cast<const v4i *>(q + row * 128 + place);
    }
    __device__ __forceinline__ void scales(int row, int (&sc)[2]) const {
        sc[0] = (int)*reinterpret_cast<const uint32_t *>(x + row * 16);
        sc[1] = (int)*reinterpret_cast<const uint32_t *>(x + row * 16 + 4);
    }
    __device__ __forceinline__ void read(int row, const int (&place)[4], v4i (&f)[4], int (&sc)[2]) const {
#pragma unroll
        for (int h = 0; h < 4; ++h) codes(row, place[h], f[h]);
        scales(row, sc);
    }
    // the same for two times 32 rows in ten steps, in the order in which products want them
    __device__ __forceinline__ void step(int k, int row, const int (&place)[4], v4i (&f)[2][4], int (&sc)[2][2]) const {
        if (k < 2) scales(row + 32 * k, sc[k]);
        else codes(row + 32 * (k & 1), place[k / 2 - 1], f[k & 1][k / 2 - 1]);
    }
};

// The larger of the bf16 pairs' absolute values, half by half.
__device__ __forceinline__ uint32_t mx_max2(uint32_t m, uint32_t v) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    const u16x2 a = __builtin_bit_cast(u16x2, m), b = __builtin_bit_cast(u16x2, v & 0x7fff7fffu);
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(a, b));
}
__device__ __forceinline__ uint32_t mx_max_half(uint32_t m) { return max(m & 0xffffu, m >> 16); }
// ... of lanes l and l + 32, in both
__device__ __forceinline__ uint32_t mx_max_swap(uint32_t m) {
    const auto x = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    return max(x[0], x[1]);
}
// codes of two groups of four bf16 columns
__device__ __forceinline__ uint32_t mx_codes(uint2 p, uint2 q, uint32_t b) {
    const float v[8] = {bf2f_lo(p.x), bf2f_hi(p.x), bf2f_lo(p.y), bf2f_hi(p.y),
                        bf2f_lo(q.x), bf2f_hi(q.x), bf2f_lo(q.y), bf2f_hi(q.y)};
    return mx_codes8(v, b);
}

// silu(u) * g for a result that is rounded to bf16: the reciprocal's last ulp is not corrected
__device__ __forceinline__ float mx_silu_times(float u, float g) {
    const float d = __builtin_amdgcn_exp2f(u * -1.4426950408889634f) + 1.0f;
    return u * __builtin_amdgcn_rcpf(d) * g;
}

// ---------------------------------------------------------------------------
// Many rows per expert: tiles of 256 by 256, one wave to a SIMD, so that the time of a
// tile follows its live rows in steps of 64 and no wave idles in a ragged one; 8 x 2
// fragments of 32 x 32 sums fill half of the register file.
//
// The stages alternate between two slots.  A wave multiplies by weight rows that it has
// copied itself, and has all of a stage's in registers when the stage begins: the
// weights of stage s + 2 are copied from then on, and have nearly two stages to come from
// memory.  The barrier between stages s and s + 1 lies before the last rows of stage s
// are multiplied: those are in registers by then, so behind it the rows of stage s + 2 are
// copied, and the first fragments of stage s + 1 are read.
//
// K = 7168, I = 2048, E = 32, top_k = 8, 2048 tokens: gmm1 280 to 320 us between other kernels, 3.0 to
// 3.4 PFLOP/s of the 6.5 above, gmm2 190 to 200; 512 tokens: 107 and 75, 128 tokens gmm1 86 (weights at 5.9
// TB/s).  gmm1 of 2048 tokens alone, call after call, goes from 278 us to 390 as the clock comes down (to 1.8 GHz
// in the mean of twenty calls; 2.0 between other kernels, 2.45 in gmm1 of 128 tokens).  Its matrix cores are busy in 41 to 45%
// of the cycles, LDS in 27 to 30%, a third of those for bank conflicts.  On operands of zero, for which the card keeps its clock,
// it took 254 us where random ones took 329, 209 without the copies and 264 without the products.
// What gave nothing or less: words of later stages fetched ahead into the L2, non-temporal
// stores (gmm2 of 4096 tokens 176 -> 235 us), 64-byte pieces of a row to a store.
//
// The grid is persistent.  While a tile is multiplied the workgroup looks up its
// next one, whose first two stages are copied in this one's last two, so that
// they are there when its sums have been rounded and stored.
constexpr int kMxList = 32;

// One sum out of the accumulation registers.  (Left to the compiler, all 256 are copied
// at once and other values spill.)
__device__ __forceinline__ float mx_sum(float a) {
    float v;
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(a));
    return v;
}

// Multiplies tile t, of at most 32 NP rows, whose first stage is in LDS and whose second is
// under way, starts the copies of tile `nt`, and rounds and stores the sums.  `stores`: at least
// 4 J times as many stores of the tile before have been made since its copies.
// (One body for every NP, with the rows behind conditions, made the compiler move the sums
// between register files.)
template <typename G, int NP>
__device__ __forceinline__ void mx_tile(const MxGmmParams &p, const MxTile &t, MxCopies<G> &c,
                                        bool more, const MxTile &nt, const MxLds &l, int &slot0,
                                        int &sbuf0, int &stores) {
    constexpr bool SWIGLU = G::SWIGLU;
    constexpr int F = SWIGLU ? 2 : 1;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int J = 2 / F;  // column fragments of 32 that a wave stores
    const int ns = (p.Kred + 255) / 256;
    const bool half = p.Kred % 256 != 0;  // of the last stage's row pieces the second halves alone

    const int r = lane & 31, g = lane >> 5;
    int place[4];  // of the lane in a row of a stage, 64 of the reduction each
#pragma unroll
    for (int h = 0; h < 4; ++h) place[h] = mx_swz(r, 2 * h + g) * 16;
    const int wrow = G::AR + wave * 64;
    v16f acc[NP][2] = {};
    v4i w[2][4], a[2][4];  // weights of the stage, rows of the two fragments that are multiplied
    int wsc[2][2], asc[2][2];
    // Two row fragments by two weight fragments: four sums that take turns, so that no product
    // waits for the one before it.  (With two, the loop ran at half the rate.)
    // between(k) comes after the k-th of its 16 products: reads and copies there, one or two at a
    // time, as a batch of either held the products up while it was taken in.
    auto multiply = [&](int pair, int first_half, auto between) {  // first_half: 0 or -1
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            asc[i][0] >>= 8 * g;  // the lane's blocks are g and 2 + g of each half
            asc[i][1] >>= 8 * g;
            // codes of 0, and no NaN for a scale, where the first half is not to be multiplied
            a[i][0] &= first_half;
            a[i][1] &= first_half;
            asc[i][0] &= first_half;
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
                    __builtin_amdgcn_sched_barrier(0);
                    between(4 * h + 2 * i + j);
                    __builtin_amdgcn_sched_barrier(0);
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
    {
        const MxStage<G> st(p, l, 0, slot0, sbuf0);
#pragma unroll
        for (int k = 0; k < 10; ++k) {
            st.step(k, wrow, place, w, wsc);
            st.step(k, 0, place, a, asc);
        }
    }
    // Slots and scale buffers go on from tile to tile.  With four stages or more the next tile's
    // first two are copied in the last two of this one (its routes, asked for before this tile, are
    // there after the second stage's barrier); else after it.
    const bool stream = more && ns >= 4;
    const int sbuf_next = (sbuf0 + (ns + 1) / 2) & 1;
    auto slot = [&](int s) { return (slot0 + s) & 1; };
    auto sbuf = [&](int s) { return (sbuf0 + (s >> 1)) & 1; };
    // Waits for all but the newest NEWER of the wave's copies; in the first stage, whose copies are
    // older than the last tile's stores, not for those either.
    auto wait_copies = [&](int s, auto newer) {
        constexpr int NEWER = newer.value, U = 4 * J;
        if (s > 0 || stores == 0) wait_vmcnt<NEWER>();
        else if (stores == 1) wait_vmcnt<NEWER + U>();
        else if (stores == 2) wait_vmcnt<NEWER + 2 * U>();
        else wait_vmcnt<NEWER + 3 * U>();
    };
    typedef std::integral_constant<int, 0> None;
    typedef std::integral_constant<int, G::WC> Weights;
    typedef std::integral_constant<int, G::WC + G::SC> WeightsScales;
    auto stage = [&](int s, auto copies) {  // copies: stage s + 2 is to be copied
        const MxStage<G> st(p, l, s, slot(s), sbuf(s));
        const int first_half = !copies.value && half && s + 1 == ns ? 0 : -1;
        // the stage's weights are in registers, and their place is free
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        const MxIssueW<G> issue_w(p, c, l, s + 2, slot(s), sbuf(s + 2));
        if constexpr (copies.value) {
            if (NP == 2) mx_all(issue_w);
        } else if (stream) {  // the next tile's first stages instead
            if (s + 2 == ns) c = mx_copies<G>(p, nt, l, 2);
            mx_all(MxIssueW<G>(p, c, l, s + 2 - ns, slot(s), sbuf_next), 0, G::WC);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            wsc[j][0] = wsc[j][0] >> (8 * g) & first_half;
            wsc[j][1] >>= 8 * g;
        }
        v4i na[2][4] = {};
        int nasc[2][2] = {};
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
            multiply(pair, first_half, [&](int k) {
                if (k < 10) st.step(k, 64 * (pair + 1), place, na, nasc);
                if constexpr (copies.value)
                    if (pair == 0 && k < G::WC) issue_w.copy(k);
            });
            // not between products: the compiler moves products down past a branch
            if constexpr (copies.value)
                if (pair == 0) mx_all(issue_w, G::WC);
            shift();
        }
        v4i nw[2][4] = {};
        int nwsc[2][2] = {};
        if (copies.value || s + 1 < ns || stream) {
            // stage s + 1 (of the tiles together)
            if (copies.value && issue_w.scales) wait_copies(s, WeightsScales{});
            else if (copies.value || stream) wait_copies(s, Weights{});
            else wait_copies(s, None{});
            __syncthreads();
        }
        const MxStage<G> next(p, l, min(s + 1, ns - 1), slot(s + 1), sbuf(s + 1));
        auto read_next = [&](int k) {
            if (k < 10) {
                next.step(k, wrow, place, nw, nwsc);
                next.step(k, 0, place, na, nasc);
            }
        };
        if constexpr (copies.value) {
            const MxIssueA<G, NP> issue(p, c, l, s + 2, slot(s));
            multiply(NP / 2 - 1, first_half, [&](int k) {
                read_next(k);
                if (k >= 16 - issue.N) issue.copy(k - (16 - issue.N));
            });
        } else {
            if (stream) {
                // its scales here, as their buffer may be the one that stage ns - 2 has read
                mx_all(MxIssueW<G>(p, c, l, s + 2 - ns, slot(s), sbuf_next), G::WC);
                mx_all(MxIssueA<G, 0>(p, c, l, s + 2 - ns, slot(s)));
            }
            multiply(NP / 2 - 1, first_half, read_next);  // in the last stage nobody looks at what it reads
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int h = 0; h < 4; ++h) w[j][h] = nw[j][h];
            wsc[j][0] = nwsc[j][0];
            wsc[j][1] = nwsc[j][1];
        }
        shift();
    };
#pragma unroll 1
    for (int s = 0; s < ns - 2; ++s) stage(s, std::true_type{});
#pragma unroll 1
    for (int s = max(0, ns - 2); s < ns; ++s) stage(s, std::false_type{});

    slot0 = slot(ns);
    sbuf0 = sbuf_next;
    if (more && !stream) {
        wait_vmcnt<0>();  // the next tile's routes, which a reduction of one stage has not waited for
        __syncthreads();  // and every wave has read the last stage
        c = mx_copies<G>(p, nt, l, 2);
        mx_short_scales<G>(p, nt, c, l, sbuf0);
        mx_issue<G, 0>(p, c, l, 0, slot0, sbuf0);
        if (ns > 1) mx_issue<G, 0>(p, c, l, 1, 1 - slot0, sbuf0);
    }
    // Four columns a lane, rounded; then lanes l and l + 32 exchange halves of two such groups, so
    // that each holds eight columns in a row and stores 16 bytes.
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
    const int n0 = t.nblk * G::COLS + wave * (64 / F);
    if (SWIGLU && p.cq) {
        // Quantised here: a row's 32 columns are one block, of lanes l and l + 32.  Their groups of
        // four columns alternate, so each takes half of both's codes and stores 8 bytes.
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const uint2(&o)[4] = out[i][0];
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) m = mx_max2(mx_max2(m, o[k].x), o[k].y);
            const uint32_t b = mx_scale_byte(mx_max_swap(mx_max_half(m)) << 16);
            const auto w = __builtin_amdgcn_permlane32_swap(mx_codes(o[0], o[1], b),
                                                            mx_codes(o[2], o[3], b), false, false);
            const size_t row = t.row0 + 32 * i + r;
            if (32 * i + r < t.rows && n0 < p.N) {
                *reinterpret_cast<uint2 *>(p.cq + row * (p.N / 2) + n0 / 2 + 8 * g) =
                    make_uint2((w[0] & 0xffffu) | w[1] << 16, w[0] >> 16 | (w[1] & 0xffff0000u));
                if (g == 0) p.cs[row * (p.N / 32) + n0 / 32] = (uint8_t)b;
            }
        }
    } else {
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
    }
    // all but the last two fragments have whole rows: so many stores were made at least
    stores = n0 + 64 / F <= p.N ? NP / 2 - 1 : 0;
    if (more && !stream) {  // the next tile's first stage: the second's copies, 10 at least, are newer
        if (ns == 1) {
            wait_vmcnt<0>();
            stores = 0;
        } else if (stores) {
            wait_vmcnt<10 + (NP - 2) * J * 2>();
        } else {
            wait_vmcnt<10>();
        }
        __syncthreads();
    }
}

template <bool SWIGLU>
__global__ __launch_bounds__(kMxThreads) __attribute__((amdgpu_waves_per_eu(1, 1))) void
mxfp4_gmm_tile_kernel(MxGmmParams p) {
    typedef MxGeom<SWIGLU, 256, 256> G;
    __shared__ int s_w[4];
    __shared__ MxSchedule s_s;
    __shared__ MxTile s_t[kMxList];
    __shared__ int32_t s_route[G::AR];
    __shared__ __align__(16) uint8_t s_data[2 * G::STAGE];
    __shared__ __align__(16) uint8_t s_scale[16 + 2 * G::SCALE];  // a short row's word may start 4 bytes early

    mx_schedule<G>(p, s_w, s_s);
    const int total = __builtin_amdgcn_readfirstlane(s_s.total);
    // workgroups go round the XCDs: each XCD takes a run of neighbouring tiles, which share
    // weight and row blocks in its L2
    const int per = (total + 7) / 8, step = gridDim.x >> 3;
    const int t0 = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    const int t1 = min((int)(blockIdx.x & 7) * per + per, total);
    const int n = t0 < t1 ? (t1 - t0 + step - 1) / step : 0;  // tiles of this workgroup
    if (n == 0) return;

    const MxLds l{s_data, s_scale + 16, (uint32_t)__builtin_amdgcn_readfirstlane(lds_addr(s_data)),
                  (uint32_t)__builtin_amdgcn_readfirstlane(lds_addr(s_scale + 16)), s_route, nullptr};
    const int tid = threadIdx.x;
    const uint32_t route_at =
        __builtin_amdgcn_readfirstlane(lds_addr(s_route) + (tid >> 6) * (kWave * 4));
    auto fetch_routes = [&](const MxTile &x) {
        if (p.a_route) dma4(p.a_route + x.row0 + min(tid, x.rows - 1), route_at);
    };
    // its tiles are looked up kMxList at a time, a lane each
    auto look_up = [&](int k) {
        if (tid < kMxList && k + tid < n) s_t[tid] = mx_find_tile<G>(s_s, t0 + (k + tid) * step);
        __syncthreads();
    };
    look_up(0);
    MxTile cur = mx_uniform(s_t[0]);
    fetch_routes(cur);
    wait_vmcnt<0>();
    __syncthreads();
    MxCopies<G> c = mx_copies<G>(p, cur, l, 2);
    mx_short_scales<G>(p, cur, c, l, 0);
    mx_issue<G, 0>(p, c, l, 0, 0, 0);
    if (p.Kred > 256) {
        mx_issue<G, 0>(p, c, l, 1, 1, 0);
        wait_vmcnt<10>();  // the second stage's copies are 10 at least
    } else {
        wait_vmcnt<0>();
    }
    __syncthreads();
    int slot = 0, sbuf = 0;  // of the first stage of the tile
    int stores = 0;          // see mx_tile
    for (int k = 1;; ++k) {
        const bool more = k < n;
        if (more && k % kMxList == 0) look_up(k);  // the last tiles of the list have been read
        const MxTile next = more ? mx_uniform(s_t[k % kMxList]) : cur;
        if (more) fetch_routes(next);
        if (cur.rows > 192) mx_tile<G, 8>(p, cur, c, more, next, l, slot, sbuf, stores);
        else if (cur.rows > 128) mx_tile<G, 6>(p, cur, c, more, next, l, slot, sbuf, stores);
        else if (cur.rows > 64) mx_tile<G, 4>(p, cur, c, more, next, l, slot, sbuf, stores);
        else mx_tile<G, 2>(p, cur, c, more, next, l, slot, sbuf, stores);
        if (!more) return;
        cur = next;
    }
}

// ---------------------------------------------------------------------------
// Few rows per expert: the product streams weights.  Tiles of at most 64 rows by 128
// weight rows; two workgroups fit a CU, so that one copies while the other looks up its tile,
// waits for its first stage or stores.  Three slots: two stages are under way while one is
// multiplied.  At the sizes above one token takes 22 us and 12 (weights of its eight
// experts at 5.6 TB/s); gmm2 of 128 tokens 55.
template <typename G, int NP>
__device__ __forceinline__ void mx_narrow(const MxGmmParams &p, const MxTile &t, const MxCopies<G> &c,
                                          const MxLds &l) {
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ns = (p.Kred + 255) / 256;
    const int r = lane & 31, g = lane >> 5;
    int place[4];  // of the lane in a row of a stage, 64 of the reduction each
#pragma unroll
    for (int h = 0; h < 4; ++h) place[h] = mx_swz(r, 2 * h + g) * 16;

    v16f acc[NP] = {};
    int slot = 0;
#pragma unroll 1
    for (int s = 0; s < ns; ++s) {
        if (s + 1 < ns) wait_vmcnt<G::WC + NP>();  // all but the last copies of stage s + 1
        else wait_vmcnt<0>();
        __syncthreads();  // and every wave has read stage s - 1, whose slot is the next
        const int free = slot == 0 ? 2 : slot - 1;
        if (s + 2 < ns) mx_issue<G, NP>(p, c, l, s + 2, free, ((s >> 1) + 1) & 1);
        const MxStage<G> st(p, l, s, slot, (s >> 1) & 1);
        v4i w[4], a[NP][4];
        int wsc[2], asc[NP][2];
        st.read(G::AR + wave * 32, place, w, wsc);
#pragma unroll
        for (int i = 0; i < NP; ++i) st.read(32 * i, place, a[i], asc[i]);
        // of the last stage, where the reduction ends in it, the second halves of the pieces alone
        const int first_half = s + 1 == ns && p.Kred % 256 != 0 ? 0 : -1;
        // the lane's blocks are g and 2 + g of each half
        wsc[0] = wsc[0] >> (8 * g) & first_half;
        wsc[1] >>= 8 * g;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            a[i][0] &= first_half;
            a[i][1] &= first_half;
            asc[i][0] = asc[i][0] >> (8 * g) & first_half;
            asc[i][1] >>= 8 * g;
        }
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int i = 0; i < NP; ++i)
                acc[i] = h & 1 ? mx_mfma32<1>(w[h], wsc[h >> 1], a[i][h], asc[i][h >> 1], acc[i])
                               : mx_mfma32<0>(w[h], wsc[h >> 1], a[i][h], asc[i][h >> 1], acc[i]);
        slot = slot == 2 ? 0 : slot + 1;
    }

    // four columns a lane, rounded; lanes l and l + 32 exchange halves as above
    constexpr int GR = G::SWIGLU ? 2 : 4;
    const int n0 = t.nblk * G::COLS + wave * (G::COLS / 4);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        uint2 out[GR];
#pragma unroll
        for (int k = 0; k < GR; ++k) {
            float y[4];
#pragma unroll
            for (int v = 0; v < 4; ++v)
                y[v] = G::SWIGLU ? mx_silu_times(acc[i][4 * k + v], acc[i][8 + 4 * (k & 1) + v])
                                 : acc[i][4 * k + v];
            out[k] = G::SWIGLU ? make_uint2(f2bf_pk(y[0], y[1]), f2bf_pk(y[2], y[3]))
                               : make_uint2(f2h(y[0]) | (uint32_t)f2h(y[1]) << 16,
                                            f2h(y[2]) | (uint32_t)f2h(y[3]) << 16);
        }
        const int row = 32 * i + r;
        if (G::SWIGLU && p.cq) {  // as above, of a block that two waves share
            const uint32_t mine =
                mx_max_swap(mx_max_half(mx_max2(mx_max2(mx_max2(mx_max2(0, out[0].x), out[0].y), out[1].x), out[1].y)));
            if (g == 0) l.most[wave * G::AR + row] = (uint16_t)mine;
            __syncthreads();
            const uint32_t b = mx_scale_byte(max(mine, (uint32_t)l.most[(wave ^ 1) * G::AR + row]) << 16);
            const uint32_t codes = mx_codes(out[0], out[1], b);
            const auto w = __builtin_amdgcn_permlane32_swap(codes, codes, false, false);
            const size_t at = t.row0 + row;
            if (row < t.rows && n0 < p.N) {
                *reinterpret_cast<uint32_t *>(p.cq + at * (p.N / 2) + n0 / 2 + 4 * g) =
                    g ? w[0] >> 16 | (w[1] & 0xffff0000u) : (w[0] & 0xffffu) | w[1] << 16;
                if (g == 0 && !(wave & 1)) p.cs[at * (p.N / 32) + n0 / 32] = (uint8_t)b;
            }
            continue;
        }
        uint16_t *crow = p.c + (size_t)(t.row0 + row) * p.N;
#pragma unroll
        for (int k = 0; k < GR; k += 2) {
            const auto x = __builtin_amdgcn_permlane32_swap(out[k].x, out[k + 1].x, false, false);
            const auto y = __builtin_amdgcn_permlane32_swap(out[k].y, out[k + 1].y, false, false);
            const int col = n0 + 8 * (k + g);
            if (row < t.rows && col < p.N)
                *reinterpret_cast<uint4 *>(crow + col) = make_uint4(x[0], y[0], x[1], y[1]);
        }
    }
}

template <bool SWIGLU>
__global__ __launch_bounds__(kMxThreads) __attribute__((amdgpu_waves_per_eu(2))) void
mxfp4_gmm_narrow_kernel(MxGmmParams p) {
    typedef MxGeom<SWIGLU, 64, 128> G;
    __shared__ int s_w[4];
    __shared__ MxTile s_t;
    __shared__ int32_t s_route[G::AR];
    __shared__ uint16_t s_most[4 * G::AR];
    __shared__ __align__(16) uint8_t s_data[3 * G::STAGE];
    __shared__ __align__(16) uint8_t s_scale[16 + 2 * G::SCALE];  // a short row's word may start 4 bytes early

    // the schedule is only looked at here, before the first copies: it lies where they go
    MxSchedule &s_s = *reinterpret_cast<MxSchedule *>(s_data);
    mx_schedule<G>(p, s_w, s_s);
    // workgroups go round the XCDs: each XCD takes a run of neighbouring tiles
    const int total = __builtin_amdgcn_readfirstlane(s_s.total), per = (total + 7) / 8;
    const int t = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || t >= total) return;
    const int tid = threadIdx.x;
    if (tid == 0) s_t = mx_find_tile<G>(s_s, t);
    __syncthreads();
    const MxTile tile = mx_uniform(s_t);
    const MxLds l{s_data, s_scale + 16, (uint32_t)__builtin_amdgcn_readfirstlane(lds_addr(s_data)),
                  (uint32_t)__builtin_amdgcn_readfirstlane(lds_addr(s_scale + 16)), s_route, s_most};
    if (p.a_route && tid < G::AR) s_route[tid] = p.a_route[tile.row0 + min(tid, tile.rows - 1)];
    __syncthreads();
    const MxCopies<G> c = mx_copies<G>(p, tile, l, 1);
    mx_short_scales<G>(p, tile, c, l, 0);
    mx_issue<G, 0>(p, c, l, 0, 0, 0);
    if (p.Kred > 256) mx_issue<G, 0>(p, c, l, 1, 1, 0);
    if (tile.rows > 32) mx_narrow<G, 2>(p, tile, c, l);
    else mx_narrow<G, 1>(p, tile, c, l);
}

// the tiles of a geometry, at most
template <typename G>
static long long mx_most_tiles(const MxGmmParams &p) {
    return ((long long)p.R / G::AR + (p.E < p.R ? p.E : p.R)) * ((p.N + G::COLS - 1) / G::COLS);
}

template <bool SWIGLU>
static void launch_variant(const MxGmmParams &p, bool narrow, int cu_count, hipStream_t stream) {
    if (narrow) {
        const long long n = (mx_most_tiles<MxGeom<SWIGLU, 64, 128>>(p) + 7) / 8 * 8;
        hipLaunchKernelGGL(mxfp4_gmm_narrow_kernel<SWIGLU>, dim3((unsigned)n), dim3(kMxThreads), 0, stream, p);
    } else {
        const long long n = mx_most_tiles<MxGeom<SWIGLU, 256, 256>>(p);  // one workgroup fits a CU
        hipLaunchKernelGGL(mxfp4_gmm_tile_kernel<SWIGLU>, dim3((unsigned)((n < cu_count ? n : cu_count) + 7) / 8 * 8),
                           dim3(kMxThreads), 0, stream, p);
    }
}

hipError_t launch_mxfp4_gmm(const MxGmmParams &p, bool swiglu, int cu_count, hipStream_t stream) {
    const int mean = (p.R + p.E - 1) / p.E;
    // Measured on both sides, narrow and wide in us, at uniform / Zipf(1.2) routing.  GMM1 at K = 7168,
    // I = 2048, E = 32: mean 2 rows 78 / 63 and 83 / 79, 16 rows 88 / 98 and 90 / 92, 24 rows 92 / 113 and
    // 92 / 97, 32 rows 95 / 114 and 91 / 98; at K = 4096, I = 1408, E = 64: 24 rows 76 / 89 and 81 / 97, 36
    // rows 84 / 99 and 84 / 96.  GMM2, with half as many weight rows to a tile of output: 32 rows 60 / 68 and
    // 59 / 67, 48 rows 63 / 73 and 61 / 79, 64 rows 83 / 81 and 65 / 95.
    const bool narrow = mean <= (swiglu ? 28 : 48);
    if (swiglu) launch_variant<true>(p, narrow, cu_count, stream);
    else launch_variant<false>(p, narrow, cu_count, stream);
    return hipGetLastError();
}

}  // namespace megamoe
