// Eight consecutive elements of fp32, fp16 or bf16 as fp32, and back (rounded to nearest even).
#pragma once

#include "common.hpp"
#include "kernels.hpp"

namespace megamoe {

template <int T>
struct Element {  // fp16 and bf16: 16 bytes
    typedef uint16_t type;
    struct Raw {
        uint4 v;
    };
    __device__ __forceinline__ static float lo(uint32_t w) { return T == kBf16 ? bf2f_lo(w) : h2f((uint16_t)w); }
    __device__ __forceinline__ static float hi(uint32_t w) { return T == kBf16 ? bf2f_hi(w) : h2f((uint16_t)(w >> 16)); }
    __device__ __forceinline__ static uint32_t pack(float a, float b) {
        return T == kBf16 ? f2bf_pk(a, b) : f2h(a) | (uint32_t)f2h(b) << 16;
    }
    __device__ __forceinline__ static Raw load(const void *p, size_t i) {
        return Raw{*reinterpret_cast<const uint4 *>((const uint16_t *)p + i)};
    }
    __device__ __forceinline__ static Raw load_nt(const void *p, size_t i) { return Raw{load_nt16((const uint16_t *)p + i)}; }
    __device__ __forceinline__ static void values(const Raw &r, float (&v)[8]) {
        const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = lo(w[j]);
            v[2 * j + 1] = hi(w[j]);
        }
    }
    __device__ __forceinline__ static Raw round(const float (&v)[8]) {
        return Raw{make_uint4(pack(v[0], v[1]), pack(v[2], v[3]), pack(v[4], v[5]), pack(v[6], v[7]))};
    }
    __device__ __forceinline__ static void store(void *p, size_t i, const float (&v)[8]) {
        *reinterpret_cast<uint4 *>((uint16_t *)p + i) = round(v).v;
    }
    __device__ __forceinline__ static void store_nt(void *p, size_t i, const float (&v)[8]) {
        store_nt16((uint16_t *)p + i, round(v).v);
    }
    __device__ __forceinline__ static float load1(const void *p, size_t i) {
        const uint16_t b = ((const uint16_t *)p)[i];
        return T == kBf16 ? bf2f_lo(b) : h2f(b);
    }
    __device__ __forceinline__ static void store1(void *p, size_t i, float v) {
        ((uint16_t *)p)[i] = (uint16_t)pack(v, 0.0f);
    }
};

template <>
struct Element<kFp32> {  // 32 bytes
    typedef float type;
    struct Raw {
        uint4 a, b;
    };
    __device__ __forceinline__ static Raw load(const void *p, size_t i) {
        const uint4 *q = reinterpret_cast<const uint4 *>((const float *)p + i);
        return Raw{q[0], q[1]};
    }
    __device__ __forceinline__ static Raw load_nt(const void *p, size_t i) {
        return Raw{load_nt16((const float *)p + i), load_nt16((const float *)p + i + 4)};
    }
    __device__ __forceinline__ static void values(const Raw &r, float (&v)[8]) {
        const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
    }
    __device__ __forceinline__ static uint4 word4(const float *v) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
    __device__ __forceinline__ static void store(void *p, size_t i, const float (&v)[8]) {
        uint4 *q = reinterpret_cast<uint4 *>((float *)p + i);
        q[0] = word4(v);
        q[1] = word4(v + 4);
    }
    __device__ __forceinline__ static void store_nt(void *p, size_t i, const float (&v)[8]) {
        store_nt16((float *)p + i, word4(v));
        store_nt16((float *)p + i + 4, word4(v + 4));
    }
    __device__ __forceinline__ static float load1(const void *p, size_t i) { return ((const float *)p)[i]; }
    __device__ __forceinline__ static void store1(void *p, size_t i, float v) { ((float *)p)[i] = v; }
};

// The same with the type known at run time, where it is the same in every lane.
__device__ __forceinline__ void load_values(const void *p, int type, size_t i, float (&v)[8]) {
    if (type == kFp32) Element<kFp32>::values(Element<kFp32>::load(p, i), v);
    else if (type == kFp16) Element<kFp16>::values(Element<kFp16>::load(p, i), v);
    else Element<kBf16>::values(Element<kBf16>::load(p, i), v);
}
__device__ __forceinline__ void store_values(void *p, int type, size_t i, const float (&v)[8]) {
    if (type == kFp32) Element<kFp32>::store(p, i, v);
    else if (type == kFp16) Element<kFp16>::store(p, i, v);
    else Element<kBf16>::store(p, i, v);
}
__device__ __forceinline__ float load_value(const void *p, int type, size_t i) {
    return type == kFp32 ? Element<kFp32>::load1(p, i) : type == kFp16 ? Element<kFp16>::load1(p, i) : Element<kBf16>::load1(p, i);
}
__device__ __forceinline__ void store_value(void *p, int type, size_t i, float v) {
    if (type == kFp32) Element<kFp32>::store1(p, i, v);
    else if (type == kFp16) Element<kFp16>::store1(p, i, v);
    else Element<kBf16>::store1(p, i, v);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
    return v;
}

}  // namespace megamoe
