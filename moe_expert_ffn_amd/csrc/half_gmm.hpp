// What the kernels of the 16-bit products share.
#pragma once

#include "common.hpp"
#include "element.hpp"
#include "half.hpp"

namespace megamoe {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
constexpr int kHgE = 256;

__device__ __forceinline__ int hg_row_end(const HalfGmmParams &p, int e) {
    const int v = e >= 0 ? p.cumsum[e] : 0;
    return v < 0 ? 0 : v > p.R ? p.R : v;
}

// A sorted route and its token: what lies past the valid rows stays in bounds.
__device__ __forceinline__ uint32_t hg_route(const HalfGmmParams &p, int v) { return min(max(v, 0), p.R - 1); }
__device__ __forceinline__ uint32_t hg_token(const HalfGmmParams &p, int v) {
    const uint32_t u = hg_route(p, v);
    return __umulhi(u, p.top_k_inv) + (u & p.one_k);
}

typedef float v4f __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));

// 16 x 16 x 32 with the columns' operand first: lane l holds output row l & 15 and the columns 4 (l >> 4) + 0..3.  Of
// either operand lane l has row l & 15 and 8 (l >> 4) + 0..7 of the reduction.  (From registers, on random operands,
// for which the card lowers its clock, it ran at 2030 TFLOP/s and the 32 x 32 x 16 form at 1730, as that one
// goes through its sums twice as often; on zeros 2420 and 2470.)
// A subnormal fp16 operand is taken as it is stored, 0.f 2^-14, and its product aligned to that: it counts, but no more exactly
// than if the operand were 2^-14 (five products of 2^-21 with values up to 2.3 were off by 2^-37 together, where a step
// of their sum in fp32 is 2^-43).
template <int T>
__device__ __forceinline__ v4f hg_mfma(v4i w, v4i a, v4f acc) {
    if constexpr (T == kBf16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, w), __builtin_bit_cast(v8bf, a), acc, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, w), __builtin_bit_cast(v8h, a), acc, 0, 0, 0);
}

// 16-byte piece c of a row that lies along the reduction: its place.  LDS has 64 banks, two rows; reads of one
// piece of 16 rows in the order of the lanes meet each bank once.
__device__ __forceinline__ int hg_swz(int row, int c) { return c ^ (row >> 1 & 7); }

// Fragments of an operand in LDS.
template <bool ACROSS>
struct HgRead {
    const uint8_t *at;
    int place[4];  // along: of the lane's piece of each step of 32, two; across: of the quarters of a panel
    __device__ __forceinline__ HgRead() {}
    __device__ __forceinline__ void lane_places() {
        const int lane = threadIdx.x & 63;
        if constexpr (ACROSS) {
            // row 8 (lane >> 4) + ((lane & 15) >> 2), and four on; columns 4 (lane & 3) + 0..3
            const int in = (lane >> 4) * 1024 + ((lane & 15) >> 2) * 128 + (lane & 3) * 8;
            const int swap = (lane >> 3 & 1) * 2 + (lane >> 4 & 1);  // bits 1 and 3 of the row
#pragma unroll
            for (int q = 0; q < 4; ++q) place[q] = in + (q ^ swap) * 32;
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) place[h] = (lane & 15) * 128 + hg_swz(lane & 15, 4 * h + (lane >> 4)) * 16;
        }
    }
    // fragment f of 16 rows or columns, step h
    __device__ __forceinline__ void read(int f, int h, v4i &v) const {
        if constexpr (ACROSS) {
            typedef __attribute__((address_space(3))) v4s *P;
            const uint8_t *q = at + place[f & 3] + (f >> 2) * 8192 + h * 4096;
            const uint2 lo = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)q));
            const uint2 hi = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(q + 512)));
            v = v4i{(int)lo.x, (int)lo.y, (int)hi.x, (int)hi.y};
        } else {
            v = *reinterpret_cast<const v4i *>(at + f * 2048 + place[h]);
        }
    }
};

struct FewTile {
    int e, row0, rows, nblk;
};
struct FewSchedule {
    int w[4], pre[kHgE + 1], first[kHgE], rows[kHgE];
};

// Tiles by expert, weight block and row block; -1 for e where there are not so many.
template <int RB>
__device__ __forceinline__ FewTile few_find_tile(const HalfGmmParams &p, int t, int cols, FewSchedule &s) {
    const int e = threadIdx.x, lane = e & (kWave - 1), wave = e >> 6;
    const int first = e < p.E ? hg_row_end(p, e - 1) : 0;
    const int rows = e < p.E ? max(0, hg_row_end(p, e) - first) : 0;
    const int nb = (p.N + cols - 1) / cols, tiles = (rows + RB - 1) / RB * nb;
    const int incl = wave_inclusive_scan(tiles);
    if (lane == kWave - 1) s.w[wave] = incl;
    s.first[e] = first;
    s.rows[e] = rows;
    __syncthreads();
    int pre = incl - tiles;
#pragma unroll
    for (int w = 0; w < 4; ++w) pre += w < wave ? s.w[w] : 0;
    s.pre[e] = pre;
    if (e == kHgE - 1) s.pre[kHgE] = pre + tiles;
    __syncthreads();
    const int total = __builtin_amdgcn_readfirstlane(s.pre[kHgE]);
    // workgroups go round the XCDs: each XCD takes a run of neighbouring tiles, which share weights or rows
    const int per = (total + 7) / 8;
    t = (t & 7) * per + (t >> 3);
    if ((int)(blockIdx.x >> 3) >= per || t >= total) return FewTile{-1, 0, 0, 0};
    int lo = 0, hi = kHgE - 1;  // the first expert that ends after t
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s.pre[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    const int n = s.rows[lo], local = t - s.pre[lo], mb = (n + RB - 1) / RB, m = local % mb;
    return FewTile{__builtin_amdgcn_readfirstlane(lo), __builtin_amdgcn_readfirstlane(s.first[lo] + m * RB),
                   __builtin_amdgcn_readfirstlane(min(RB, n - m * RB)), __builtin_amdgcn_readfirstlane(local / mb)};
}

// silu(u) * g for a result that is rounded to 16 bits: the reciprocal's last ulp is not corrected
__device__ __forceinline__ float hg_silu_times(float u, float g) {
    const float d = __builtin_amdgcn_exp2f(u * -1.4426950408889634f) + 1.0f;
    return u * __builtin_amdgcn_rcpf(d) * g;
}

}  // namespace megamoe
