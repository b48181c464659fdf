// Grouped products of fp16 or bf16 rows and weights, and their gradients (the place of GMM1 and GMM2,
// sections 3 and 5 of the pto-isa MegaMoE overview page, with unquantised experts).
//
// For the rows d of expert e's group, sums in fp32 on the matrix cores:
//   product   c[d, n] = sum_k a[d, k] b[e, n, k]
//   rows      c[d, n] = sum_k a[d, k] b[e, k, n]      (the gradient of a product's rows)
//   weights   c[e, m, n] = sum_d a[d, m] b[d, n]      (the gradient of its weights)
// The rows of a or b may be gathered: row d is row route[d] / top_k of the array.  A product
// may end in SwiGLU: columns n and N + n of b meet in the same lane's accumulators.
#include <type_traits>

#include "common.hpp"
#include "dma.hpp"
#include "half_gmm.hpp"

namespace megamoe {

// ---------------------------------------------------------------------------
// Tiles of 256 rows by 256 columns, four waves to a tile and one to a SIMD, each multiplying all of
// its rows by 64 of its columns: 16 x 4 fragments of 16 x 16 sums fill half of the register file, and the time of a
// tile follows its live rows in steps of 64.
//
// A stage is 64 of the reduction, copied asynchronously into one of two slots in LDS, 128 bytes (a whole
// cache line) at a time.  An operand lies there in one of two ways:
//   along    its rows run along the reduction: [256 rows][128 bytes], fragments read 16 bytes a lane;
//   across   its rows run across it: [4 panels][64 of the reduction][64 columns], fragments read by the
//            transposing LDS load, which gives a lane four values of one column.
// Either way the 16-byte pieces are placed so that a fragment's reads meet every LDS bank equally often.
//
// A stage is multiplied 64 rows at a time, in two phases of 32 of the reduction; what a phase multiplies is read from
// LDS during the one before, into the registers that were free by then, so that nothing is moved between registers.
// A wave multiplies by columns that it has copied itself: all of a stage's are in registers after the first
// phase, and from then on those of the stage after the next are copied.  The barrier between two stages lies
// before the last phase of the first: its rows are in registers by then, so behind it the rows of
// the stage after the next are copied, and the first fragments of the next one are read.
//
// The grid is persistent, and the copies run two stages ahead of the products through the workgroup's
// tiles, so that a tile's first stages are there when the tile before has been rounded and stored.
//
// K = 7168, I = 2048, E = 32, top_k = 8, bf16, random operands: first product of 2048 tokens 806 to 850 us, 1130 to 1190
// TFLOP/s, of 16384 tokens 5680, 1355; its row gradient of 2048 tokens 850, its weight gradient 1000 to 1040.  Second product 466,
// 1030 TFLOP/s, as its tiles are 32 stages and end 3.5 times as often.  An
// 8192^3 library product reaches 1390 TFLOP/s here in bf16.  What bounds the products is power: at 2048 tokens the
// card runs them at 1.63 of 2.4 GHz, with the matrix cores busy in 71% of the cycles.  Timed with work left out: without
// copies 1.23 times as fast, the same cache lines copied in every stage 1.06, without stores no faster, without LDS reads
// or barriers no faster.  The weight gradients of short groups are bound by their tiles' ends: of eight
// stages each, at 2.1 GHz with the matrix cores busy in 41%; without stores they take 0.82 of the time.  Slower or
// no faster: eight waves, two to a SIMD, with one stage ahead; copies of dead rows left out by EXEC (7%); waits that
// count the stores in flight; 32 x 32 x 16 products; row blocks in turn over all of an expert's.
constexpr int kHgThreads = 256;
constexpr int kHgTile = 256, kHgK = 64;
constexpr int kHgOperand = kHgTile * kHgK * 2;  // bytes of an operand's stage
constexpr int kHgList = 64;                     // tiles looked up ahead, half of them at a time
constexpr int kHgRing = 8;                      // stages whose routes are kept (weights' gradients)

template <int KIND_, int T_, bool SWIGLU_, int GATHER_ = 0>
struct HgGeom {
    static constexpr int KIND = KIND_, T = T_;
    static constexpr bool SWIGLU = SWIGLU_;
    static constexpr int GATHER = GATHER_;  // weights: HalfGmmParams::gather, 1 or 2
    static constexpr bool WEIGHTS = KIND == kHalfWeights;
    static constexpr bool A_ACROSS = WEIGHTS, B_ACROSS = KIND != kHalfProduct;
    static constexpr int F = SWIGLU ? 2 : 1;
    static constexpr int COLS = kHgTile / F;  // output columns of a tile
    static constexpr int J = 4 / F;           // fragments of 16 columns that a wave stores
};

struct HgTile {
    int e, row0, rows, nblk;  // first output row and how many, block of columns
    int first, red;           // weights: the group's first row; the reduction's length
};

struct HgSchedule {
    int first[kHgE], rows[kHgE];
    int order[kHgE];    // experts, those with the longest tiles first
    int pre[kHgE + 1];  // products: tiles of the experts before the i-th of them
    int total;
};

// Tiles by expert, those whose tiles take longest first: weights: that have most rows; products: most
// rows in a tile.  Weights: every expert has as many tiles.  Products: an expert's rows are split evenly
// over its row blocks in units of 32.
template <typename G>
__device__ __forceinline__ void hg_schedule(const HalfGmmParams &p, int *s_w, HgSchedule &s) {
    const int e = threadIdx.x, lane = e & (kWave - 1), wave = e >> 6;
    const int first = e < p.E ? hg_row_end(p, e - 1) : 0;
    const int rows = e < p.E ? max(0, hg_row_end(p, e) - first) : 0;
    const int blocks = (rows + kHgTile - 1) / kHgTile;
    const int length = G::WEIGHTS || rows == 0 ? rows : (rows + blocks - 1) / blocks;
    s.first[e] = first;
    s.rows[e] = rows;
    s.pre[e] = length;
    __syncthreads();
    int rank = 0;
    for (int i = 0; i < p.E; ++i) {
        const int other = s.pre[i];
        rank += other > length || (other == length && i < e);
    }
    if (e >= p.E) rank = e;
    s.order[rank] = e;
    if constexpr (G::WEIGHTS) {
        if (e == 0) s.total = p.E * ((p.M + kHgTile - 1) / kHgTile) * ((p.N + kHgTile - 1) / kHgTile);
    } else {
        __syncthreads();
        const int tiles = (s.rows[s.order[e]] + kHgTile - 1) / kHgTile * ((p.N + G::COLS - 1) / G::COLS);
        const int incl = wave_inclusive_scan(tiles);
        if (lane == kWave - 1) s_w[wave] = incl;
        __syncthreads();
        int pre = incl - tiles;
#pragma unroll
        for (int w = 0; w < 4; ++w) pre += w < wave ? s_w[w] : 0;
        s.pre[e] = pre;  // experts past E have no tiles: pre is the total
        if (e == kHgE - 1) s.pre[kHgE] = s.total = pre + tiles;
    }
    __syncthreads();
}

// Tile `local` of mb row blocks by nb column blocks: eight row blocks, then the columns, then the next eight: what an
// XCD's workgroups multiply at one time shares most (16 row blocks in turn, us: row gradient 1668 for 1594, product
// 1602 for 1590, weights' gradient of 16 groups of 2048 rows 990 for 975).
__device__ __forceinline__ void hg_block(int local, int mb, int nb, int &m, int &n) {
    const int run = local / (8 * nb), wide = min(8, mb - 8 * run), in = local - 8 * nb * run;
    m = 8 * run + in % wide;
    n = in / wide;
}

template <typename G>
__device__ __forceinline__ HgTile hg_find_tile(const HalfGmmParams &p, const HgSchedule &s, int t) {  // t < total
    const int nb = (p.N + G::COLS - 1) / G::COLS;
    int m, n;
    if constexpr (G::WEIGHTS) {
        const int mb = (p.M + kHgTile - 1) / kHgTile, e = s.order[t / (mb * nb)];
        hg_block(t % (mb * nb), mb, nb, m, n);
        return HgTile{e, m * kHgTile, min(kHgTile, p.M - m * kHgTile), n, s.first[e], s.rows[e]};
    } else {
        int lo = 0, hi = kHgE - 1;  // the first of the order that ends after t
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (s.pre[mid + 1] > t) hi = mid;
            else lo = mid + 1;
        }
        const int e = s.order[lo], rows = s.rows[e], mb = (rows + kHgTile - 1) / kHgTile;
        hg_block(t - s.pre[lo], mb, nb, m, n);
        const int nu = (rows + 31) / 32, q = nu / mb, r = nu % mb;
        const int u0 = m * q + min(m, r), u1 = u0 + q + (m < r);
        return HgTile{e, s.first[e] + 32 * u0, min(rows, 32 * u1) - 32 * u0, n, 0, p.K};
    }
}
__device__ __forceinline__ HgTile hg_uniform(const HgTile &x) {
    return HgTile{__builtin_amdgcn_readfirstlane(x.e), __builtin_amdgcn_readfirstlane(x.row0),
                  __builtin_amdgcn_readfirstlane(x.rows), __builtin_amdgcn_readfirstlane(x.nblk),
                  __builtin_amdgcn_readfirstlane(x.first), __builtin_amdgcn_readfirstlane(x.red)};
}

struct HgLds {
    uint8_t *data;
    uint32_t data_at;  // its LDS address
    int32_t *route;    // products: [2][256] routes of a tile's rows; weights: [kHgRing][64] routes of a stage
    float *weight;     // products with SwiGLU: [3][256] weights of a tile's rows
    uint32_t *row;     // weights: [4][64] byte offsets of a stage's gathered rows, of each wave
    uint32_t route_at, weight_at;
};

// One 16-byte piece a lane into LDS through a buffer: 0 where voff is not within it.
__device__ __forceinline__ void dma16_buffer(v4i rsrc, uint32_t voff, uint32_t lds_base) {
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "buffer_load_dwordx4 %1, %2, 0 offen lds"
        :
        : "s"(lds_base), "v"(voff), "s"(rsrc)
        : "memory", "m0");
}
__device__ __forceinline__ v4i hg_buffer(const void *base, uint32_t bytes) {
    const uint64_t v = (uint64_t)base;
    return v4i{(int)__builtin_amdgcn_readfirstlane((uint32_t)v), (int)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32)),
               (int)__builtin_amdgcn_readfirstlane(bytes), 0x00027000};
}

// Where a lane's pieces of a stage come from.  A wave makes eight copies of each operand: 64 of its rows
// (along) or a panel of 64 of its columns (across).
template <typename G>
struct HgCopies {
    // products: byte offsets in the tile, from pointers that go on from stage to stage
    uint32_t va[8], vb[8];
    const uint8_t *a, *b;
    uint32_t step_b;
    // weights: rows past the group are out of the buffers' bounds and read as 0
    v4i ra, rb;
    uint32_t gathered[2];  // byte of the lane's columns in a gathered row, in even and odd copies
    uint32_t straight[2];  // byte offset of the lane's first row in the other operand, likewise
    int left;              // rows of the group from the stage's first one on
    uint32_t row[8];       // byte offsets of the lane's gathered rows
};

// Byte of a lane's columns in its panel of columns from n0, of n that are a multiple of 128, in even copies; in odd
// ones it is this ^ 32.  The 32-byte quarters of a panel's row change places with its bits 1 and 3: a
// transposing load takes 32 bytes of rows 0..3, 8..11, 16..19 and 24..27, which then meet each bank twice.
__device__ __forceinline__ uint32_t hg_across_column(int n0, int n) {
    const int lane = threadIdx.x & 63, c = lane & 7;  // the lane's row in a copy is lane >> 3
    int col = n0 + ((c >> 1) ^ (lane >> 4 & 1) * 2) * 16 + (c & 1) * 8;
    if (col >= n) col = n - 64 + (col & 63);
    return 2 * (uint32_t)col;
}

// The copies of tile t, the workgroup's k-th, from its first stage on.
template <typename G>
__device__ __forceinline__ void hg_open(const HalfGmmParams &p, const HgTile &t, int k, const HgLds &l, HgCopies<G> &c) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if constexpr (G::WEIGHTS) {
        const uint32_t ca = hg_across_column(t.row0 + wave * 64, p.M);
        const uint32_t cb = hg_across_column(t.nblk * kHgTile + wave * 64, p.N);
        c.left = t.red;
        c.gathered[0] = G::GATHER == 1 ? ca : cb;
        c.gathered[1] = c.gathered[0] ^ 32;
        c.straight[0] = (uint32_t)(lane >> 3) * (2 * (G::GATHER == 1 ? p.N : p.M)) + (G::GATHER == 1 ? cb : ca);
        c.straight[1] = c.straight[0] ^ 32;
        const uint32_t la = 2 * p.M, lb = 2 * p.N, tokens = p.R / p.top_k;
        c.ra = G::GATHER == 1 ? hg_buffer(p.a, tokens * la) : hg_buffer(p.a + (size_t)t.first * p.M, t.red * la);
        c.rb = G::GATHER == 2 ? hg_buffer(p.b, tokens * lb) : hg_buffer(p.b + (size_t)t.first * p.N, t.red * lb);
    } else {
        const uint32_t la = 2 * p.K;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = (wave * 8 + i) * 8 + (lane >> 3), piece = hg_swz(r, lane & 7) * 16;
            const int live = min(r, t.rows - 1);
            const uint32_t row = p.gather ? hg_token(p, l.route[(k & 1) * kHgTile + live]) : (uint32_t)(t.row0 + live);
            c.va[i] = row * la + piece;
            if constexpr (G::B_ACROSS) {
                c.vb[i] = (uint32_t)(8 * i + (lane >> 3)) * (2 * p.N) +
                          (hg_across_column(t.nblk * kHgTile + wave * 64, p.N) ^ (i & 1) * 32);
            } else {
                // with SwiGLU a wave's columns are 32 for silu and the 32 of the gate that go with them
                const int w = r >> 6, in = r & 63;
                const int col = t.nblk * G::COLS + (G::SWIGLU ? 32 * w + (in & 31) : r);
                c.vb[i] = (uint32_t)(min(col, p.N - 1) + (G::SWIGLU && in >= 32 ? p.N : 0)) * la + piece;
            }
        }
        c.a = uniform_ptr((const uint8_t *)p.a);
        c.b = uniform_ptr((const uint8_t *)(p.b + (size_t)t.e * G::F * p.N * p.K));
        c.step_b = G::B_ACROSS ? kHgK * 2 * p.N : kHgK * 2;
    }
}

// weights: the i-th copy's byte offset.  Rows past the group are not within the buffer of the straight
// operand, whose bytes end with the group; a gathered row of theirs lies past the end.
template <typename G>
__device__ __forceinline__ uint32_t hg_offset(const HgCopies<G> &c, int i, int operand, uint32_t ld) {
    return G::GATHER == operand ? c.row[i] + c.gathered[i & 1] : c.straight[i & 1] + (uint32_t)i * (8 * ld);
}

template <typename G>
struct HgIssue {  // the copies of one operand's stage into slot `slot`
    const HalfGmmParams &p;
    const HgCopies<G> &c;
    const uint8_t *base;
    v4i rsrc;
    uint32_t at;
    bool b;
    __device__ __forceinline__ HgIssue(const HalfGmmParams &p_, const HgCopies<G> &c_, const HgLds &l, bool b_, int slot)
        : p(p_), c(c_), b(b_) {
        at = __builtin_amdgcn_readfirstlane(l.data_at + (2 * slot + b) * kHgOperand + (threadIdx.x >> 6) * 8192);
        if constexpr (G::WEIGHTS) {
            const v4i r = b ? c.rb : c.ra;
#pragma unroll
            for (int i = 0; i < 4; ++i) rsrc[i] = __builtin_amdgcn_readfirstlane(r[i]);
        } else {
            base = uniform_ptr(b ? c.b : c.a);
        }
    }
    __device__ __forceinline__ void copy(int i) const {
        if constexpr (G::WEIGHTS) {
            const uint32_t v = b ? hg_offset<G>(c, i, 2, 2 * p.N) : hg_offset<G>(c, i, 1, 2 * p.M);
            dma16_buffer(rsrc, v, at + i * 1024);
        } else if (b) {
            dma16_nt(base, c.vb[i], at + i * 1024);
        } else {
            dma16(base, c.va[i], at + i * 1024);
        }
    }
};
template <typename I>
__device__ __forceinline__ void hg_all(const I &issue) {
#pragma unroll
    for (int i = 0; i < 8; ++i) issue.copy(i);
}

// One sum out of the accumulation registers.  (Left to the compiler, all 256 are copied
// at once and other values spill.)
__device__ __forceinline__ float hg_sum(float a) {
    float v;
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(a));
    return v;
}

template <typename G>
struct HgRun {
    const HalfGmmParams &p;
    const HgLds l;  // (a reference to it was kept in LDS, and its pointers taken for generic ones)
    const HgTile *list;
    int n;             // tiles of this workgroup
    int stage, total;  // of all of the workgroup's: the one that is multiplied next, and how many there are
    HgCopies<G> c;
    int tile_k, left;  // the tile whose stages are copied, and how many of them are left
    int route_k, route_s, route_left;  // weights: the next stage whose routes are copied
    HgRead<G::A_ACROSS> ra;
    HgRead<G::B_ACROSS> rb;
    v4i w[4][2], a[4][2];  // columns of the stage, the 64 rows that are multiplied: of both phases

    __device__ __forceinline__ HgTile tile(int k) const { return hg_uniform(list[k & (kHgList - 1)]); }
    __device__ __forceinline__ static int stages(const HgTile &t) { return (t.red + kHgK - 1) / kHgK; }
    // products: the routes of tile k's rows; weights: those of the workgroup's stage `at`, of 64 rows
    __device__ __forceinline__ void fetch_tile_routes(int k) const {
        if (G::WEIGHTS || !p.route || k >= n) return;
        const HgTile t = tile(k);
        const int tid = threadIdx.x;
        dma4(p.route + t.row0 + min(tid, t.rows - 1),
             __builtin_amdgcn_readfirstlane(l.route_at + ((k & 1) * kHgTile + (tid & ~63)) * 4));
    }
    __device__ __forceinline__ void fetch_stage_routes(int at) {
        if (!G::WEIGHTS || at >= total) return;
        if (route_left == 0) {
            ++route_k;
            route_s = 0;
            route_left = stages(tile(route_k));  // not 0: tiles without stages come last
        }
        if (threadIdx.x < kWave) {
            const HgTile t = tile(route_k);
            dma4(p.route + t.first + min(route_s * kHgK + (int)threadIdx.x, t.red - 1),
                 __builtin_amdgcn_readfirstlane(l.route_at + (at & (kHgRing - 1)) * kHgK * 4));
        }
        ++route_s;
        --route_left;
    }
    __device__ __forceinline__ const uint8_t *slot(int g) const { return l.data + (g & 1) * 2 * kHgOperand; }
    // the first phase's fragments of stage g, in eight steps
    __device__ __forceinline__ void read_first(int g, int k) {
        if (k & 1) {
            ra.at = slot(g);
            ra.read(k >> 1, 0, a[k >> 1][0]);
        } else {
            rb.at = slot(g) + kHgOperand;
            rb.read(4 * __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) + (k >> 1), 0, w[k >> 1][0]);
        }
    }
    // before the copies of a stage, and behind them
    __device__ __forceinline__ void open() {
        if (left > 0) return;
        ++tile_k;
        const HgTile t = tile(tile_k);
        left = stages(t);
        hg_open<G>(p, t, tile_k, l, c);
        if (G::SWIGLU && p.probs) {
            const int tid = threadIdx.x;
            const int v = l.route[(tile_k & 1) * kHgTile + min(tid, t.rows - 1)];
            dma4(p.probs + hg_route(p, v),
                 __builtin_amdgcn_readfirstlane(l.weight_at + (tile_k % 3 * kHgTile + (tid & ~63)) * 4));
        }
        fetch_tile_routes(tile_k + 1);
    }
    __device__ __forceinline__ void close() {
        --left;
        if constexpr (G::WEIGHTS) {
            const uint32_t step = kHgK * 2 * (G::GATHER == 1 ? p.N : p.M);
            c.straight[0] += step;
            c.straight[1] += step;
            c.left -= kHgK;
        } else {
            c.a += kHgK * 2;
            c.b += c.step_b;
        }
    }
    // weights: the byte offsets of the gathered rows of stage `at`, whose copies are next: a row a lane, and through
    // LDS, in a place of the wave's own, to the lanes that copy the row
    __device__ __forceinline__ int read_route(int at) const {
        return l.route[(at & (kHgRing - 1)) * kHgK + (int)(threadIdx.x & 63)];
    }
    __device__ __forceinline__ void place_row(int route) const {
        const uint32_t ld = 2 * (G::GATHER == 1 ? p.M : p.N);
        // an array's bytes end 64 rows below 2^32
        uint32_t v = hg_token(p, route) * ld;
        asm volatile("" : "+v"(v));  // a choice, not a branch: one in a stage undoes its registers
        l.row[threadIdx.x] = (int)(threadIdx.x & 63) < c.left ? v : 0u - 4 * ld;
    }
    __device__ __forceinline__ void read_row(int i) {
        c.row[i] = l.row[(threadIdx.x & ~63) + 8 * i + (int)((threadIdx.x & 63) >> 3)];
    }

    // Multiplies tile t, of at most 32 NP rows, whose first stage is in LDS, copies two stages ahead,
    // and rounds and stores the sums.
    template <int NP>
    __device__ __forceinline__ void multiply_tile(const HgTile &t, int k);
};

template <typename G>
template <int NP>
__device__ __forceinline__ void HgRun<G>::multiply_tile(const HgTile &t, int k) {
    constexpr int T = G::T, J = G::J;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ns = (t.red + kHgK - 1) / kHgK;

    v4f acc[2 * NP][4] = {};
    // between(k) comes after the k-th of its 16 products: reads and copies there, one or two at a time, as a batch
    // of either holds the products up while it is taken in.
    auto phase = [&](int pair, int h, auto between) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v4f &d = acc[4 * pair + i][j];
                d = hg_mfma<T>(w[j][h], a[i][h], d);
                __builtin_amdgcn_sched_barrier(0);
                between(4 * i + j);
                __builtin_amdgcn_sched_barrier(0);
            }
        // the sums are wanted here: without this the compiler puts a stage's products together
        // behind its barrier and copies, where the reads no longer overlap them
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) asm volatile("" : "+a"(acc[4 * pair + i][j]));
    };
    // The copies are spread over a stage, as four waves make them at once and a copy takes longer to be taken in
    // than a product: those of the columns over the phases before the barrier, those of the rows over
    // the one behind it.
    constexpr int LAST = NP / 2 - 1, FROM = G::WEIGHTS ? 8 : 1, EVERY = LAST ? (32 * LAST - FROM) / 8 : 1;
    auto one_stage = [&](auto copies) {  // copies: stage `stage` + 2 is to be copied
        if constexpr (copies.value) open();
        const HgIssue<G> columns(p, c, l, true, stage & 1), rows(p, c, l, false, stage & 1);
        ra.at = slot(stage);
        rb.at = slot(stage) + kHgOperand;
        int route;
#pragma unroll
        for (int pair = 0; pair <= LAST; ++pair) {
            phase(pair, 0, [&](int k) {
                if (k < 8 && !(k & 1)) ra.read(4 * pair + (k >> 1), 1, a[k >> 1][1]);
                if (pair == 0 && k < 8 && (k & 1)) rb.read(4 * wave + (k >> 1), 1, w[k >> 1][1]);
                if constexpr (copies.value) {
                    if (G::WEIGHTS && pair == 0 && k == 8) route = read_route(stage + 2);
                    if (G::WEIGHTS && pair == 0 && k == 14) place_row(route);
                    const int at = 32 * pair + k - 16 - FROM;
                    if (LAST && pair && at >= 0 && at % EVERY == 0 && at / EVERY < 8) columns.copy(at / EVERY);
                }
            });
            if (pair == 0) {
                // the stage's columns are in registers, and their place is free
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                if constexpr (copies.value)
                    if (LAST == 0) hg_all(columns);
            }
            if (pair == LAST && (copies.value || stage + 1 < total)) {
                // all but the columns of the stage after the next
                wait_vmcnt<copies.value ? 8 : 0>();
                __syncthreads();
            }
            phase(pair, 1, [&](int k) {
                if (pair < LAST) {
                    if (k < 8 && !(k & 1)) ra.read(4 * (pair + 1) + (k >> 1), 0, a[k >> 1][0]);
                } else if (k < 8) {
                    read_first(stage + 1, k);
                }
                if constexpr (copies.value) {
                    if (G::WEIGHTS && pair == 0 && k < 8) read_row(k);
                    const int at = 32 * pair + k - FROM;
                    if (LAST && pair < LAST && at >= 0 && at % EVERY == 0 && at / EVERY < 8) columns.copy(at / EVERY);
                    if (pair == LAST && (k & 1)) rows.copy(k >> 1);
                }
            });
        }
        if constexpr (copies.value) {
            close();
            fetch_stage_routes(stage + 4);
        }
        ++stage;
    };
    const int with_copies = min(ns, max(0, total - 2 - stage));
#pragma unroll 1
    for (int s = 0; s < with_copies; ++s) one_stage(std::true_type{});
#pragma unroll 1
    for (int s = with_copies; s < ns; ++s) one_stage(std::false_type{});

    // the last product's result is there after 18 wait states
    asm volatile("s_nop 15\n\ts_nop 15");
    const int r = lane & 15, g = lane >> 4;
    const int n0 = t.nblk * G::COLS + wave * 16 * J;
    const size_t out_row = G::WEIGHTS ? (size_t)t.e * p.M + t.row0 : (size_t)t.row0;
    const bool low = r < 8;
    // Lanes l and l ^ 8 exchange four words: of two pieces of a row, x and y, in lines one after the other, each lane
    // then has one of row r & 7 in x and one of row 8 + (r & 7) in y, so that a store has the whole lines of eight rows.
    auto exchange = [&](v4i &x, v4i &y) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int keep = low ? x[v] : y[v], give = low ? y[v] : x[v];
            const int got = __builtin_amdgcn_update_dpp(0, give, 0x128, 0xf, 0xf, false);  // of lane l ^ 8
            x[v] = low ? keep : got;
            y[v] = low ? got : keep;
        }
    };
    if (G::WEIGHTS && p.c_type == kFp32) {
        // four columns a lane; stored as the 16-bit weights below (64 groups of 384 rows, 4096 x 1408: 490 to 517 us for
        // 572).  Added: 1360 us, as a piece is loaded, waited for with all that is under way, and stored before the next
#pragma unroll
        for (int i = 0; i < 2 * NP; ++i) {
#pragma unroll
            for (int j = 0; j < J; j += 2) {
                __builtin_amdgcn_sched_barrier(0);
                v4i q[2];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int v = 0; v < 4; ++v) q[h][v] = __float_as_int(hg_sum(acc[i][j + h][v]));
                exchange(q[0], q[1]);
                const int col = n0 + 16 * (j + (r >> 3)) + 4 * g;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = 16 * i + 8 * h + (r & 7);
                    if (row >= t.rows || col >= p.N) continue;
                    v4f *o = reinterpret_cast<v4f *>((float *)p.c + (out_row + row) * p.N + col);
                    v4f y = __builtin_bit_cast(v4f, q[h]);
                    if (p.accumulate) y += *o;
                    __builtin_nontemporal_store(y, o);
                }
            }
        }
        return;
    }
    // four columns a lane, added to what is there, a piece after the other as in fp32 (the same groups: 810 us, written 394)
    if (G::WEIGHTS && p.accumulate) {
#pragma unroll
        for (int i = 0; i < 2 * NP; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            const int row = 16 * i + r;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                float y[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) y[v] = hg_sum(acc[i][j][v]);
                const int col = n0 + 16 * j + 4 * g;
                if (row >= t.rows || col >= p.N) continue;
                uint2 *o = reinterpret_cast<uint2 *>((uint16_t *)p.c + (out_row + row) * p.N + col);
                const uint2 old = *o;
                typedef Element<T> L;
                *o = make_uint2(L::pack(L::lo(old.x) + y[0], L::hi(old.x) + y[1]),
                                L::pack(L::lo(old.y) + y[2], L::hi(old.y) + y[3]));
            }
        }
        return;
    }
    // Four columns a lane, rounded; then lanes l and l ^ 16 exchange halves of two such fragments, so
    // that each holds eight columns in a row and stores 16 bytes.  Weights, which are more than the caches hold: lanes
    // l and l ^ 8 exchange such pieces too, so that a store has the whole lines of eight rows, and past the caches
    // (64 groups of 384 rows, 4096 x 1408: 430 us with neither, 413 with one, 400 with both; products of 2048 tokens
    // get no faster: 835 and 840).
#pragma unroll
    for (int pair = 0; pair < NP / 2; ++pair) {
        uint2 out[4][J];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __builtin_amdgcn_sched_barrier(0);  // a few sums at a time leave the accumulators
            const int f = 4 * pair + i;
            const float weight = G::SWIGLU && p.probs ? l.weight[k % 3 * kHgTile + 16 * f + r] : 1.0f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                float y[4];
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    y[v] = G::SWIGLU ? weight * hg_silu_times(hg_sum(acc[f][j][v]), hg_sum(acc[f][(j + 2) & 3][v]))
                                     : hg_sum(acc[f][j][v]);
                out[i][j] = make_uint2(Element<T>::pack(y[0], y[1]), Element<T>::pack(y[2], y[3]));
                // rounded here, not in the blocks of the stores: half the registers
                asm volatile("" : "+v"(out[i][j].x), "+v"(out[i][j].y));
            }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v4i q[J / 2];
#pragma unroll
            for (int j = 0; j < J; j += 2) {
                const auto x = __builtin_amdgcn_permlane16_swap(out[i][j].x, out[i][j + 1].x, false, false);
                const auto y = __builtin_amdgcn_permlane16_swap(out[i][j].y, out[i][j + 1].y, false, false);
                q[j / 2] = v4i{(int)x[0], (int)y[0], (int)x[1], (int)y[1]};
            }
            if constexpr (G::WEIGHTS) exchange(q[0], q[1]);
#pragma unroll
            for (int j = 0; j < J / 2; ++j) {
                const int row = 64 * pair + 16 * i + (G::WEIGHTS ? 8 * j + (r & 7) : r);
                const int half = G::WEIGHTS ? r >> 3 : j;
                const int col = n0 + 32 * half + 16 * (g & 1) + 8 * (g >> 1);
                if (row >= t.rows || col >= p.N) continue;
                v4i *o = reinterpret_cast<v4i *>((uint16_t *)p.c + (out_row + row) * p.N + col);
                if (G::WEIGHTS) __builtin_nontemporal_store(q[j], o);
                else *o = q[j];
            }
        }
    }
}

template <typename G>
__global__ __launch_bounds__(kHgThreads) __attribute__((amdgpu_waves_per_eu(1, 1))) void half_gmm_kernel(HalfGmmParams p) {
    __shared__ int s_w[4];
    __shared__ HgSchedule s_s;
    __shared__ HgTile s_t[kHgList];
    __shared__ int32_t s_route[2 * kHgTile];
    __shared__ uint32_t s_row[G::WEIGHTS ? kHgThreads : 1];
    __shared__ float s_weight[G::SWIGLU ? 3 * kHgTile : 1];
    __shared__ __align__(16) uint8_t s_data[4 * kHgOperand];
    static_assert(kHgRing * kHgK <= 2 * kHgTile, "the ring of routes");

    hg_schedule<G>(p, s_w, s_s);
    const int total = __builtin_amdgcn_readfirstlane(s_s.total), tid = threadIdx.x;
    // Rounds of a tile a workgroup, every other one backwards as tiles get shorter.  Workgroups go round the XCDs: those
    // of an XCD take neighbouring tiles, which share blocks of rows and columns in its L2.  The tiles past whole
    // rounds are an eighth an XCD: where all of an XCD's workgroups have one more and another's none, an
    // XCD's share of the memory's rate is left idle.
    const int groups = gridDim.x >> 3, round = gridDim.x;
    const int rounds = total / round, rest = total - rounds * round;
    auto place = [&](int i, int &xcd, int &in) {
        xcd = i & 1 ? 7 - (blockIdx.x & 7) : blockIdx.x & 7;
        in = i & 1 ? groups - 1 - (blockIdx.x >> 3) : blockIdx.x >> 3;
    };
    auto tile_of = [&](int i) {
        int xcd, in;
        place(i, xcd, in);
        return hg_find_tile<G>(p, s_s, i * round + (i < rounds ? xcd * groups : rest * xcd / 8) + in);
    };
    int n = rounds;
    {
        int xcd, in;
        place(rounds, xcd, in);
        n += in < rest * (xcd + 1) / 8 - rest * xcd / 8;
    }
    if (n == 0) return;
    auto look_up = [&](int k) {  // half of the list, from tile k on
        if (tid < kHgList / 2 && k + tid < n) s_t[(k + tid) & (kHgList - 1)] = tile_of(k + tid);
    };
    look_up(0);
    look_up(kHgList / 2);
    int stages = n * (p.K / kHgK);
    if constexpr (G::WEIGHTS) {  // tiles of experts without rows, the last ones, have none
        if (tid < 4) s_w[tid] = 0;
        __syncthreads();
        int mine = 0;
        for (int i = tid; i < n; i += kHgThreads)
            mine += (tile_of(i).red + kHgK - 1) / kHgK;
        atomicAdd(&s_w[0], mine);  // of integers: in any order
        __syncthreads();
        stages = __builtin_amdgcn_readfirstlane(s_w[0]);
    }
    __syncthreads();

    const HgLds l{s_data, (uint32_t)__builtin_amdgcn_readfirstlane(lds_addr(s_data)), s_route, s_weight, s_row,
                  (uint32_t)__builtin_amdgcn_readfirstlane(lds_addr(s_route)),
                  (uint32_t)__builtin_amdgcn_readfirstlane(lds_addr(s_weight))};
    HgRun<G> run{p, l, s_t, n};
    run.ra.lane_places();
    run.rb.lane_places();
    run.stage = 0;
    run.total = stages;
    run.tile_k = run.route_k = -1;
    run.left = run.route_left = 0;
    // the first routes, then the first two stages
    run.fetch_tile_routes(0);
    for (int i = 0; i < 4; ++i) run.fetch_stage_routes(i);
    wait_vmcnt<0>();
    __syncthreads();
    for (int i = 0; i < min(2, stages); ++i) {
        run.open();
        if constexpr (G::WEIGHTS) {
            run.place_row(run.read_route(i));
#pragma unroll
            for (int j = 0; j < 8; ++j) run.read_row(j);
        }
        hg_all(HgIssue<G>(p, run.c, l, true, i));
        hg_all(HgIssue<G>(p, run.c, l, false, i));
        run.close();
    }
    if (stages > 1) wait_vmcnt<16>();
    else wait_vmcnt<0>();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) run.read_first(0, i);
    for (int k = 0; k < n; ++k) {
        if (k > 0 && k % (kHgList / 2) == 0) {
            __syncthreads();  // nobody looks at the older half any more: tiles without stages have no barrier
            look_up(k + kHgList / 2);
            __syncthreads();
        }
        const HgTile t = run.tile(k);
        if constexpr (G::WEIGHTS) {
            if (t.red == 0 && p.accumulate) continue;
            if (t.rows > 128) run.template multiply_tile<8>(t, k);
            else run.template multiply_tile<4>(t, k);
        } else {
            if (t.rows > 192) run.template multiply_tile<8>(t, k);
            else if (t.rows > 128) run.template multiply_tile<6>(t, k);
            else if (t.rows > 64) run.template multiply_tile<4>(t, k);
            else run.template multiply_tile<2>(t, k);
        }
    }
}

// The tiles, at most.
template <typename G>
static long long hg_most_tiles(const HalfGmmParams &p) {
    const long long cols = (p.N + G::COLS - 1) / G::COLS;
    if (G::WEIGHTS) return (long long)p.E * ((p.M + kHgTile - 1) / kHgTile) * cols;
    return ((long long)p.R / kHgTile + (p.E < p.R ? p.E : p.R)) * cols;
}

template <typename G>
static void hg_launch(const HalfGmmParams &p, int cu_count, hipStream_t stream) {
    const long long n = hg_most_tiles<G>(p);  // one workgroup fits a CU
    hipLaunchKernelGGL(half_gmm_kernel<G>, dim3((unsigned)((n < cu_count ? n : cu_count) + 7) / 8 * 8), dim3(kHgThreads),
                       0, stream, p);
}

hipError_t launch_half_gmm(const HalfGmmParams &p, int kind, int type, int cu_count, hipStream_t stream) {
    const bool b = type == kBf16;
    if (half_small_ok(p, kind, cu_count)) return launch_half_small(p, kind, type, stream);
    if (kind == kHalfProduct && half_few_ok(p)) return launch_half_few(p, type, stream);
    if (kind == kHalfProduct && p.swiglu) {
        if (b) hg_launch<HgGeom<kHalfProduct, kBf16, true>>(p, cu_count, stream);
        else hg_launch<HgGeom<kHalfProduct, kFp16, true>>(p, cu_count, stream);
    } else if (kind == kHalfProduct) {
        if (b) hg_launch<HgGeom<kHalfProduct, kBf16, false>>(p, cu_count, stream);
        else hg_launch<HgGeom<kHalfProduct, kFp16, false>>(p, cu_count, stream);
    } else if (kind == kHalfRows) {
        if (b) hg_launch<HgGeom<kHalfRows, kBf16, false>>(p, cu_count, stream);
        else hg_launch<HgGeom<kHalfRows, kFp16, false>>(p, cu_count, stream);
    } else {
        if (p.gather == 1 && b) hg_launch<HgGeom<kHalfWeights, kBf16, false, 1>>(p, cu_count, stream);
        else if (p.gather == 1) hg_launch<HgGeom<kHalfWeights, kFp16, false, 1>>(p, cu_count, stream);
        else if (b) hg_launch<HgGeom<kHalfWeights, kBf16, false, 2>>(p, cu_count, stream);
        else hg_launch<HgGeom<kHalfWeights, kFp16, false, 2>>(p, cu_count, stream);
    }
    return hipGetLastError();
}

}  // namespace megamoe
