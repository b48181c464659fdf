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
//  * few_gmm1_kernel, one workgroup per chosen expert and 32 output columns:
//    quantises its expert's tokens into LDS, multiplies them by 16 silu and 16
//    gate columns at a time with the reduction split over its waves (an exact
//    integer sum), and writes y = silu * gate in fp32 with the largest |y| of
//    its columns.
//  * few_gmm2_kernel, one workgroup per 32 or 16 output columns: quantises every
//    pair's y into LDS (the row maximum is that of the 16-column maxima),
//    multiplies each expert's rows by its columns, and combines the slots of
//    every token in order, so no partial result leaves the workgroup.
// A wave reads weights straight from memory into fragments: 16 columns of one
// 64-byte K slice are 1 KB in a row in the packed layout.
#include <type_traits>

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
    int end[kFewE];        // one past the last pair of the a-th such expert
    int n_act, n_pair, valid;
};

template <int THREADS>
__device__ __forceinline__ void few_find_pairs(const int32_t *__restrict__ ids, int R, int E,
                                               int top_k, FewPairs &s) {
    const int tid = threadIdx.x;
    for (int e = tid; e < kFewE; e += THREADS) s.mask[e] = 0;
    if (tid == 0) s.valid = 0;
    const int id = tid < R ? ids[tid] : -1;  // R <= kFewThreads <= THREADS
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
            if (v[j]) {
                s.act[run >> 16] = tid * 4 + j;
                s.end[run >> 16] = (run + v[j]) & 0xffff;
            }
            run += v[j];
        }
        if (tid == kWave - 1) {
            s.n_pair = run & 0xffff;
            s.n_act = run >> 16;
        }
    }
    __syncthreads();
}

// Workgroup b of n -> its column group (a permutation where n is a multiple of 8).  Workgroups go round
// the 8 XCDs; the groups of one XCD are consecutive, so that the 1 KB pieces of
// a K slice that it reads lie together.  Reading weights alone in this way, the
// mapping took 5.8 to 6.2 TB/s with 8 experts and 6.3 to 6.7 with 32.
__device__ __forceinline__ int few_group(int b, int n) {
    return (n & 7) ? b : (b & 7) * (n >> 3) + (b >> 3);
}

// 16 bytes of a wave-uniform block at the lane's offset
__device__ __forceinline__ v4i few_load(const int8_t *block, uint32_t off) {
    typedef const __attribute__((address_space(1))) v4i *global_v4i;
    return __builtin_nontemporal_load((global_v4i)(uint64_t)(block + off));
}

// The largest v of the wave's lanes, in every lane: four shifted maxima inside the
// rows of 16 lanes, then across rows to lane 63.  (Lane exchanges through the
// LDS crossbar take several times as long each.)
template <int CTRL>
__device__ __forceinline__ uint32_t max_step(uint32_t v) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
    return o > v ? o : v;
}
__device__ __forceinline__ uint32_t wave_max_all(uint32_t v) {
    v = max_step<0x111>(v);  // row_shr 1, 2, 4, 8
    v = max_step<0x112>(v);
    v = max_step<0x114>(v);
    v = max_step<0x118>(v);
    v = max_step<0x142>(v);  // row_bcast 15, 31
    v = max_step<0x143>(v);
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ v4i few_mfma(v4i w, v4i a, v4i acc) {
    // weights first: lane l holds row l & 15 and the columns 4 (l >> 4) + 0..3
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, a, acc, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// K = 7168, I = 2048, E = 32, top_k = 8: 38 us at one token and 152 to 160 at 16, of 35 and 140 for
// the weights alone at 6.7 TB/s.  (With 1 group of columns 40 and 186, with 4 57 and 247.)
constexpr int kFew1Groups = 2;  // groups of 16 columns that share the quantised rows

template <int U>  // K slices a wave has in flight
__global__ __launch_bounds__(kFewThreads) __attribute__((amdgpu_waves_per_eu(4))) void
few_gmm1_kernel(FewParams p, int row_cap) {
    constexpr int NG = kFew1Groups;
    __shared__ FewPairs s_p;
    __shared__ int s_tok[16];
    __shared__ uint32_t s_red[16][kFewWaves];
    __shared__ float s_scale[16];
    __shared__ v4i s_part[kFewWaves][2][kWave];
    __shared__ v4i s_zero[4];
    extern __shared__ __align__(16) int8_t s_a[];  // [row_cap][K + 16]

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int K = p.K, I = p.I, stride = K + 16;
    few_find_pairs<kFewThreads>(p.expert_idx, p.M * p.top_k, p.E, p.top_k, s_p);
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) *p.err = p.M * p.top_k - s_p.valid;
    if ((int)blockIdx.y >= s_p.n_act) return;
    const int e = __builtin_amdgcn_readfirstlane(s_p.act[blockIdx.y]);
    const uint32_t mask = __builtin_amdgcn_readfirstlane(s_p.mask[e]);
    const int n = __popc(mask), pair0 = __builtin_amdgcn_readfirstlane(s_p.base[e]);
    if (tid < 4) s_zero[tid] = v4i{0, 0, 0, 0};
    if (tid < 16 && (mask >> tid & 1)) s_tok[__popc(mask & ((1u << tid) - 1))] = tid;
    __syncthreads();

    const int NB = (2 * I + kPackRowsF - 1) / kPackRowsF;
    const size_t slice = (size_t)p.E * NB * kPackBlockF;
    const int nu0 = few_group(blockIdx.x, gridDim.x) * 16 * NG, ns = K / 64;
    const int8_t *we = p.w1p + (size_t)e * NB * kPackBlockF;
    const uint32_t woff = (lane & 15) * 64 + (lane >> 4) * 16;
    const int s0 = wave * ns / kFewWaves, cnt = (wave + 1) * ns / kFewWaves - s0;
    const v4i zero = {0, 0, 0, 0};

    for (int r0 = 0; r0 < n; r0 += row_cap) {
        const int m = min(row_cap, n - r0);
        // A ring of U K slices in registers, each refilled as soon as it has been multiplied.  The
        // code is straight: past its share a wave loads the last slice again and multiplies
        // zero rows.  (Branches around single loads made the compiler wait for all of them.)
        v4i fu[U], fg[U];
        const int8_t *qu, *qg;  // the next slice to load, of the silu and of the gate columns
        int li;                 // its index in the share
        auto seek = [&](int nu) {
            const int ng = I + nu;
            const int8_t *first = we + (size_t)s0 * slice;
            qu = uniform_ptr(first + (size_t)(nu / kPackRowsF) * kPackBlockF + (nu % kPackRowsF) * 64);
            qg = uniform_ptr(first + (size_t)(ng / kPackRowsF) * kPackBlockF + (ng % kPackRowsF) * 64);
            li = 0;
        };
        auto load = [&](int u) {
            fu[u] = few_load(qu, woff);
            fg[u] = few_load(qg, woff);
            const size_t step = ++li < cnt ? slice : 0;
            qu = uniform_ptr(qu + step);
            qg = uniform_ptr(qg + step);
        };
        seek(nu0);
#pragma unroll
        for (int u = 0; u < U; ++u) load(u);  // on their way while the rows are quantised

        for (int i = 0; i < m; i += 2) {  // two rows at a time: their loads overlap
            const int j = i + 1 < m ? i + 1 : i;
            const uint4 *xi = reinterpret_cast<const uint4 *>(p.x + (size_t)s_tok[r0 + i] * K);
            const uint4 *xj = reinterpret_cast<const uint4 *>(p.x + (size_t)s_tok[r0 + j] * K);
            u16x2_t mi = {0, 0}, mj = {0, 0};
#pragma unroll 1
            for (int c = tid; c < K / 8; c += kFewThreads) {
                mi = absmax_step(mi, xi[c]);
                mj = absmax_step(mj, xj[c]);
            }
            const uint32_t bi = wave_max_all(mi[0] > mi[1] ? mi[0] : mi[1]);
            const uint32_t bj = wave_max_all(mj[0] > mj[1] ? mj[0] : mj[1]);
            if (lane == 0) {
                s_red[i][wave] = bi;
                s_red[j][wave] = bj;
            }
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
#pragma unroll 1
            for (int c = tid; c < K / 8; c += kFewThreads)
                *reinterpret_cast<uint2 *>(s_a + (size_t)i * stride + c * 8) =
                    quant_chunk8(xr[c], scale, inv);
            if (tid == 0) s_scale[i] = scale;
        }
        __syncthreads();

        // rows past the group read its first one; their results are not used
        const int8_t *arow = s_a + ((lane & 15) < m ? (lane & 15) : 0) * stride + (lane >> 4) * 16;
        const int8_t *zrow = reinterpret_cast<const int8_t *>(&s_zero[lane >> 4]);
#pragma unroll 1
        for (int g = 0; g < NG; ++g) {
            const int n_out = nu0 + 16 * g;
            v4i au = zero, ag = zero;
            auto batch = [&](auto refill, int i0) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const v4i a = *reinterpret_cast<const v4i *>(
                        i0 + u < cnt ? arow + (s0 + i0 + u) * 64 : zrow);
                    au = few_mfma(fu[u], a, au);
                    ag = few_mfma(fg[u], a, ag);
                    if constexpr (refill.value) load(u);
                }
            };
            int i0 = 0;
            for (; i0 + U < cnt; i0 += U) batch(std::true_type{}, i0);
            if (g + 1 < NG) {  // refill with the next columns' first slices
                seek(n_out + 16);
                batch(std::true_type{}, i0);
            } else {
                batch(std::false_type{}, i0);
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
                const float *sc = p.scale1 + (size_t)e * 2 * I + n_out + col;
                const uint16_t hu = f2h(keep_f32((float)su * sc[0]));
                const uint16_t hg = f2h(keep_f32((float)sg * sc[I]));
                const float p1 = s_scale[row < m ? row : 0];
                const float y = silu_times(__builtin_fmaf(h2f(hu), p1, 0.0f),
                                           __builtin_fmaf(h2f(hg), p1, 0.0f));
                // a NaN is passed over, as in the row's own maximum
                float big = fmaxf(0.0f, fabsf(y));
#pragma unroll
                for (int off = 1; off < 16; off <<= 1)
                    big = fmaxf(big, __shfl_xor(big, off, kWave));
                if (row < m) {
                    const size_t pair = pair0 + r0 + row;
                    p.y[pair * I + n_out + col] = y;
                    if (col == 0) p.ymax[pair * (I / 16) + n_out / 16] = big;
                }
            }
            __syncthreads();  // s_part is free, and s_a and s_scale after the last columns
        }
    }
}

// ---------------------------------------------------------------------------
// The second product.  A workgroup works through steps, each a run of experts
// whose rows fit an LDS buffer (and a chunk of I where I is long).  Twelve of its
// waves quantise the rows of the next step while four multiply the current one,
// so weights keep coming while y is read and rounded.  (K = 7168, I = 2048, E = 32,
// top_k = 8: 94 us at 16 tokens and 23.5 at one, of 71 and 18 for the weights
// alone; eight and eight waves took 100 and 23.4, all waves doing both in turn
// 125 and 26.6.)
constexpr int kFew2Threads = 1024;
constexpr int kFew2Mul = 4;                                 // waves that multiply
constexpr int kFew2Quant = kFew2Threads / kWave - kFew2Mul;  // and that quantise

// A barrier of all waves that each kind reaches at a place of its own.
__device__ __forceinline__ void few_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
}

struct FewStep {
    int a0, a1;  // experts of the step, as indices into the active list
    int p0, p1;  // their pairs
    int i0, ic;  // chunk of I
};
// the step that starts with active expert a0, whose first pair is p0
__device__ __forceinline__ FewStep few_step(const FewPairs &s, int n_act, int a0, int p0, int i0,
                                            int I, int row_cap, int i_cap) {
    FewStep t{a0, a0, p0, p0, i0, min(i_cap, I - i0)};
    while (t.a1 < n_act) {  // one expert always fits: it has at most M rows, and so has a buffer
        const int end = __builtin_amdgcn_readfirstlane(s.end[t.a1]);
        if (end - p0 > row_cap) break;
        t.p1 = end;
        ++t.a1;
    }
    return t;
}

template <int COLS>  // output columns of a workgroup, 16 or 32
__global__ __launch_bounds__(kFew2Threads) __attribute__((amdgpu_waves_per_eu(4))) void
few_gmm2_kernel(FewParams p, int row_cap, int i_cap) {
    constexpr int H = COLS / 16;  // weight fragments of a K slice
    constexpr int U = 16 / H;     // K slices a wave has in flight
    constexpr int NS = 8;         // channel scales a quantising thread fetches early
    __shared__ FewPairs s_p;
    __shared__ int s_id[kFewThreads];
    __shared__ v4i s_zero[4];
    __shared__ float s_prob[kFewThreads], s_pts2[kFewThreads];  // by route, by pair
    extern __shared__ __align__(16) int8_t s_dyn[];

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool multiplies = wave < kFew2Mul;
    const int hw = multiplies ? wave : wave - kFew2Mul;
    const int K = p.K, I = p.I, R = p.M * p.top_k, stride = i_cap + 16;
    int *s_acc = reinterpret_cast<int *>(s_dyn);               // [R][COLS], int32 then fp32
    int8_t *s_a = s_dyn + (size_t)R * COLS * 4;           // 2 x [row_cap][i_cap + 16]
    few_find_pairs<kFew2Threads>(p.expert_idx, R, p.E, p.top_k, s_p);
    const int n_act = __builtin_amdgcn_readfirstlane(s_p.n_act), n_pair = s_p.n_pair;

    const int NB = (K + kPackRowsF - 1) / kPackRowsF;
    const size_t block = (size_t)NB * kPackBlockF, slice = (size_t)p.E * block;
    const int n0 = few_group(blockIdx.x, gridDim.x) * COLS;
    const int8_t *w0 = p.w2p + (size_t)(n0 / kPackRowsF) * kPackBlockF + (n0 % kPackRowsF) * 64;
    const uint32_t woff = (lane & 15) * 64 + (lane >> 4) * 16;
    const v4i zero = {0, 0, 0, 0};

    FewStep cur = few_step(s_p, n_act, 0, 0, 0, I, row_cap, i_cap);
    // multiplying waves: a ring of U K slices in registers, as above, of the wave's shares of the
    // steps' (expert, K slice) lists
    v4i f[U][H];
    FewStep to = cur;        // the step whose slices are loaded now
    int ti = 0, te = 0;      // the next of the wave's share of it, and the share's end
    int la = 0, ls = 0;      // the same as expert and slice
    const int8_t *lq = w0;   // and its address
    auto share = [&](const FewStep &t, int &t0, int &t1) {
        const int T = (t.a1 - t.a0) * (t.ic / 64);
        t0 = hw * T / kFew2Mul;
        t1 = (hw + 1) * T / kFew2Mul;
    };
    auto expert = [&]() {
        lq = uniform_ptr(w0 + (size_t)(to.i0 / 64 + ls) * slice + s_p.act[la] * block);
    };
    auto seek = [&](const FewStep &t) {  // a step with experts
        to = t;
        share(t, ti, te);
        const int n = t.ic / 64, at = min(ti, (t.a1 - t.a0) * n - 1);
        la = __builtin_amdgcn_readfirstlane(t.a0 + at / n);
        ls = __builtin_amdgcn_readfirstlane(at % n);
        expert();
    };
    auto load = [&](int u) {
#pragma unroll
        for (int h = 0; h < H; ++h) f[u][h] = few_load(lq + 1024 * h, woff);
        if (ti + 1 < te) {
            ++ti;
            if (++ls == to.ic / 64) {
                ls = 0;
                ++la;
                expert();
            } else {
                lq = uniform_ptr(lq + slice);
            }
        }
    };
    // the channel scale of element i of the accumulators (pair i / 32, column i % 32)
    auto channel_scale = [&](int i) {
        const int pr = i / COLS;
        int lo = 0, hi = n_act - 1;  // the pair's expert: the first one that ends after it
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (s_p.end[mid] > pr) hi = mid;
            else lo = mid + 1;
        }
        return p.scale2[(size_t)s_p.act[lo] * K + n0 + i % COLS];
    };
    const int htid = hw * kWave + lane, n_out = n_pair * COLS;
    int8_t *buf = s_a, *other = s_a + (size_t)row_cap * stride;
    auto after = [&](const FewStep &t) {  // the same experts' next chunk, or the next experts
        const bool more = t.i0 + t.ic < I;
        return few_step(s_p, n_act, more ? t.a0 : t.a1, more ? t.p0 : t.p1, more ? t.i0 + t.ic : 0, I,
                        row_cap, i_cap);
    };
    auto swap = [&]() {
        int8_t *t = buf;
        buf = other;
        other = t;
    };
    // Both kinds of waves pass the same barriers: one before the first step and one after each.
    if (multiplies) {
        if (n_act > 0) {
            seek(cur);
#pragma unroll
            for (int u = 0; u < U; ++u) load(u);
        }
        if (tid < 4) s_zero[tid] = zero;
        for (int i = htid; i < n_out; i += kFew2Mul * kWave) s_acc[i] = 0;
        few_barrier();
        while (cur.a0 < n_act) {
            const FewStep nxt = after(cur);
            const int nsl = cur.ic / 64;
            int t0, t1;
            share(cur, t0, t1);
            int ca = __builtin_amdgcn_readfirstlane(cur.a0 + t0 / nsl);
            int cs = __builtin_amdgcn_readfirstlane(t0 % nsl);
            v4i acc[H] = {};
            int rows = 0, prow = 0;
            const int8_t *arow = buf, *zrow = reinterpret_cast<const int8_t *>(&s_zero[lane >> 4]);
            auto open = [&]() {
                prow = ca ? s_p.end[ca - 1] : 0;
                rows = s_p.end[ca] - prow;
                // rows past the group read its first one; their results are not used
                arow = buf + (prow - cur.p0 + ((lane & 15) < rows ? (lane & 15) : 0)) * stride +
                       (lane >> 4) * 16;
            };
            auto flush = [&]() {  // integer sums: the order of the waves does not matter
                if ((lane & 15) < rows) {
                    int *d = s_acc + (prow + (lane & 15)) * COLS + 4 * (lane >> 4);
#pragma unroll
                    for (int h = 0; h < H; ++h)
#pragma unroll
                        for (int v = 0; v < 4; ++v) atomicAdd(d + 16 * h + v, acc[h][v]);
                }
#pragma unroll
                for (int h = 0; h < H; ++h) acc[h] = zero;
            };
            auto batch = [&](auto refill, int t) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const v4i a =
                        *reinterpret_cast<const v4i *>(t + u < t1 ? arow + cs * 64 : zrow);
#pragma unroll
                    for (int h = 0; h < H; ++h) acc[h] = few_mfma(f[u][h], a, acc[h]);
                    if constexpr (refill.value) load(u);
                    if (t + u < t1 && ++cs == nsl) {
                        flush();
                        cs = 0;
                        if (++ca < cur.a1) open();
                    }
                }
            };
            if (t0 < t1) open();
            int t = t0;
            for (; t + U < t1; t += U) batch(std::true_type{}, t);
            if (nxt.a0 < n_act) {  // refill with the next step's first slices
                seek(nxt);
                batch(std::true_type{}, t);
            } else {
                batch(std::false_type{}, t);
            }
            if (t0 < t1 && cs != 0) flush();
            few_barrier();
            cur = nxt;
            swap();
        }
    } else {
        // A row at a time, the wave's next one (of this step or a later one) on its way meanwhile.
        // The row's maximum is that of its 16-column maxima; the rounding is swiglu_row_finish's:
        // the low bytes of y * mul + 1.5 * 2^23.
        FewStep fs = cur;  // the step of the row that is fetched next
        int fr = hw;       // and its place in it
        float4 next[8];    // i_cap <= 2048: all of the row's chunk
        float next_big;
        auto fetch = [&]() {
            while (fs.a0 < n_act && fr >= fs.p1 - fs.p0) {
                fs = after(fs);
                fr = hw;
            }
            if (fs.a0 >= n_act) return;
            const size_t pr = fs.p0 + fr;
            const float4 *y = reinterpret_cast<const float4 *>(p.y + pr * I + fs.i0);
            const float *ym = p.ymax + pr * (I / 16);
            fr += kFew2Quant;
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (c * kWave + lane < fs.ic / 4) next[c] = y[c * kWave + lane];
            next_big = lane < I / 16 ? ym[lane] : 0.0f;
            for (int c = lane + kWave; c < I / 16; c += kWave) next_big = fmaxf(next_big, ym[c]);
        };
        auto quantise = [&](const FewStep &t, int8_t *dst_rows) {
            for (int row = hw; row < t.p1 - t.p0; row += kFew2Quant) {
                float4 v[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) v[c] = next[c];
                // non-negative floats order like their bits
                const float big = __uint_as_float(wave_max_all(__float_as_uint(next_big)));
                fetch();
                const float mul = big != 0.0f ? 127.0f / big : 0.0f;
                if (lane == 0) s_pts2[t.p0 + row] = big / 127.0f;
                uint32_t *dst = reinterpret_cast<uint32_t *>(dst_rows + row * stride);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    if (c * kWave + lane >= t.ic / 4) break;
                    const uint32_t b0 = __float_as_uint(keep_f32(v[c].x * mul) + 12582912.0f);
                    const uint32_t b1 = __float_as_uint(keep_f32(v[c].y * mul) + 12582912.0f);
                    const uint32_t b2 = __float_as_uint(keep_f32(v[c].z * mul) + 12582912.0f);
                    const uint32_t b3 = __float_as_uint(keep_f32(v[c].w * mul) + 12582912.0f);
                    dst[c * kWave + lane] = __builtin_amdgcn_perm(
                        __builtin_amdgcn_perm(b3, b2, 0x0c0c0400u),
                        __builtin_amdgcn_perm(b1, b0, 0x0c0c0400u), 0x05040100u);
                }
            }
        };
        fetch();
        for (int i = htid; i < R; i += kFew2Quant * kWave) {
            s_id[i] = p.expert_idx[i];
            s_prob[i] = p.probs[i];
        }
        quantise(cur, buf);
        few_barrier();
        float sc[NS];
        while (cur.a0 < n_act) {
            const FewStep nxt = after(cur);
            if (nxt.a0 < n_act) {
                quantise(nxt, other);
            } else {  // the channel scales, while the last step is multiplied
#pragma unroll
                for (int k = 0; k < NS; ++k) {
                    const int i = htid + k * (kFew2Quant * kWave);
                    sc[k] = i < n_out ? channel_scale(i) : 0.0f;
                }
            }
            few_barrier();
            cur = nxt;
            swap();
        }
        // dequantise every pair's columns in place
        auto dequant = [&](int i, float scale) {
            const uint16_t h = f2h(keep_f32((float)s_acc[i] * scale));
            const float g = __builtin_fmaf(h2f(h), s_pts2[i / COLS], 0.0f);
            s_acc[i] = (int)__float_as_uint(bf2f_lo(f2bf_pk(g, 0.0f)));
        };
#pragma unroll
        for (int k = 0; k < NS; ++k) {
            const int i = htid + k * (kFew2Quant * kWave);
            if (i < n_out) dequant(i, sc[k]);
        }
        for (int i = htid + NS * (kFew2Quant * kWave); i < n_out; i += kFew2Quant * kWave)
            dequant(i, channel_scale(i));
    }
    __syncthreads();
    if (tid < p.M * COLS) {  // slots in order, multiply then add
        const int t = tid / COLS, col = tid % COLS;
        float acc = 0.0f;
        for (int s = 0; s < p.top_k; ++s) {
            const int e = s_id[t * p.top_k + s];
            if (e < 0 || e >= p.E) continue;
            const int pr = s_p.base[e] + __popc(s_p.mask[e] & ((1u << t) - 1));
            acc = acc + __uint_as_float((uint32_t)s_acc[pr * COLS + col]) *
                            s_prob[t * p.top_k + s];
        }
        p.out[(size_t)t * K + n0 + col] = (uint16_t)(f2bf_pk(acc, 0.0f) & 0xffffu);
    }
}

// ---------------------------------------------------------------------------
constexpr size_t kFewRowBytes = 56 << 10;  // quantised rows held in LDS: two workgroups fit a CU

constexpr size_t kFew2Bytes = 148 << 10;    // LDS of the second product beside its tables

bool few_ok(int M, int top_k) { return M <= kFewMaxM && M * top_k <= kFewThreads; }

hipError_t launch_few(const FewParams &p, hipStream_t stream) {
    const int R = p.M * p.top_k;
    const int most = p.E < R ? p.E : R;  // experts with a pair, at most
    // as many of the expert's rows as fit at once (one row of K <= 32768 always does)
    int cap1 = (int)(kFewRowBytes / (p.K + 16));
    cap1 = cap1 < 1 ? 1 : cap1 > p.M ? p.M : cap1;
    const size_t lds1 = (size_t)cap1 * (p.K + 16);
    const dim3 grid1(p.I / (16 * kFew1Groups), most), block1(kFewThreads);
    // the ring that loads fewer slices past a wave's share, the longer one where that is the same
    // (K = 7168, one token: 39.2 us with 7 and 40.5 with 4; K = 4096, 5 tokens: 51 and 39)
    const int share = (p.K / 64 + kFewWaves - 1) / kFewWaves;
    if ((share + 6) / 7 * 7 <= (share + 3) / 4 * 4)
        hipLaunchKernelGGL(few_gmm1_kernel<7>, grid1, block1, lds1, stream, p, cap1);
    else
        hipLaunchKernelGGL(few_gmm1_kernel<4>, grid1, block1, lds1, stream, p, cap1);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    // 32 columns to a workgroup (half as much quantising) where those fill most CUs
    const int cols = p.K / 32 >= 192 ? 32 : 16;
    // beside the accumulators (at most 64 KB) two buffers of rows of at most 2048 elements: at
    // least 16 rows fit each, and no expert has more than M
    const size_t acc = (size_t)R * cols * 4;
    const int i_cap = p.I < 2048 ? p.I : 2048;
    int cap2 = (int)((kFew2Bytes - acc) / 2 / (i_cap + 16));
    cap2 = cap2 > R ? R : cap2;
    const size_t lds2 = acc + (size_t)cap2 * 2 * (i_cap + 16);
    if (cols == 32)
        hipLaunchKernelGGL(few_gmm2_kernel<32>, dim3(p.K / 32), dim3(kFew2Threads), lds2, stream, p, cap2,
                           i_cap);
    else
        hipLaunchKernelGGL(few_gmm2_kernel<16>, dim3(p.K / 16), dim3(kFew2Threads), lds2, stream, p, cap2,
                           i_cap);
    return hipGetLastError();
}

}  // namespace megamoe
