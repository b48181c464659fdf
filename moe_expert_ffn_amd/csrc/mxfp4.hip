// MXFP4: quantisation of rows to 4-bit elements with a scale for each 32, and back.
//
// The format is the OCP Microscaling MXFP4: an element is E2M1 (0, .5, 1, 1.5, 2,
// 3, 4, 6 and their negatives), and the 32 elements of a block along the row share
// a power of two, E8M0 (byte b stands for 2^(b - 127), 255 for NaN).  A block's
// scale is 2^(floor(log2 max|x|) - 2), so that its largest element lands in [4, 8);
// elements are x / scale to the nearest value, ties to the even code, and those
// above 6 become 6.  A block of zeros gets byte 0.  A block that holds a NaN or an
// infinity gets byte 255 and codes 0: every value of it is NaN.
//
// Both kernels are bound by HBM.  A lane owns 8 consecutive elements (one 16-byte
// load of a 16-bit type, one 4-byte store of codes), so a wave's accesses are
// contiguous, and a block is four lanes, whose maximum takes two lane exchanges.
// 128 rows of 7168 fp16 take 3.6 us and 3.9 back, 16211 of 2048 bf16 16.5 us and 13.9
// (84 MB each, 5.1 and 6.0 TB/s: a large copy reaches 5.2, and the codes are read back from a cache).
// The largest |x| is an integer maximum of the bits without the sign: NaN orders
// above infinity, which orders above every finite value.
#include "common.hpp"
#include "kernels.hpp"
#include "mxfp4_row.hpp"

namespace megamoe {

constexpr int kMxBlock = 256;   // threads
constexpr int kMxChunk = 8;     // elements of a lane
constexpr int kMxUnroll = 4;    // chunks a lane has in flight

// 8 elements as fp32
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    const uint4 a = load_nt16(p), b = load_nt16(p + 4);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
}
__device__ __forceinline__ void load8(const _Float16 *p, float (&v)[8]) {
    const uint4 a = load_nt16(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = h2f((uint16_t)(w[j >> 1] >> (16 * (j & 1))));
}
__device__ __forceinline__ void load8(const __bf16 *p, float (&v)[8]) {
    const uint4 a = load_nt16(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (j & 1) ? bf2f_hi(w[j >> 1]) : bf2f_lo(w[j >> 1]);
}

__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
    store_nt16(p, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                             __float_as_uint(v[3])));
    store_nt16(p + 4, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]),
                                 __float_as_uint(v[6]), __float_as_uint(v[7])));
}
__device__ __forceinline__ void store8(_Float16 *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = f2h(v[2 * j]) | (uint32_t)f2h(v[2 * j + 1]) << 16;
    store_nt16(p, make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ void store8(__bf16 *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = f2bf_pk(v[2 * j], v[2 * j + 1]);
    store_nt16(p, make_uint4(w[0], w[1], w[2], w[3]));
}

// chunks of 8 elements that hold data: of all rows, or of the first *valid_rows
__device__ __forceinline__ int64_t mx_chunks(int64_t rows, int64_t cols,
                                             const int32_t *__restrict__ valid_rows) {
    if (valid_rows) {
        const int64_t v = *valid_rows;
        rows = v < 0 ? 0 : v < rows ? v : rows;
    }
    return rows * cols / kMxChunk;  // cols is a multiple of 32
}

template <typename T>
__global__ __launch_bounds__(kMxBlock) void mxfp4_quant_kernel(
    const T *__restrict__ x, int64_t rows, int64_t cols, const int32_t *__restrict__ valid_rows,
    uint32_t *__restrict__ q, uint8_t *__restrict__ scale) {
    const int64_t n = mx_chunks(rows, cols, valid_rows);
    const int64_t c0 = (int64_t)blockIdx.x * (kMxBlock * kMxUnroll) + threadIdx.x;
    float v[kMxUnroll][kMxChunk];
#pragma unroll
    for (int u = 0; u < kMxUnroll; ++u) {
        const int64_t c = c0 + u * kMxBlock;
        if (c < n) load8(x + c * kMxChunk, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kMxUnroll; ++u) {
        const int64_t c = c0 + u * kMxBlock;
        if (c >= n) break;  // n is a multiple of 4: the lanes of a block agree
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < kMxChunk; ++j) {
            const uint32_t a = __float_as_uint(v[u][j]) & 0x7fffffffu;
            m = a > m ? a : m;
        }
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
            const uint32_t o = (uint32_t)__shfl_xor((int)m, off, kWave);
            m = o > m ? o : m;
        }
        const uint32_t b = mx_scale_byte(m);
        q[c] = mx_codes8(v[u], b);
        if ((c & 3) == 0) scale[c >> 2] = (uint8_t)b;
    }
}

// code -> value: E2M1 has the sign, two exponent bits (bias 1) and one mantissa bit
__device__ __forceinline__ float e2m1_f32(uint32_t c) {
    const uint32_t m = c & 7;
    // 1 and up: fp32 with exponent 126 + (m >> 1) and the mantissa bit on top; 1 is .5, 0 is 0
    const uint32_t f = m > 1 ? ((126 + (m >> 1)) << 23) | (m & 1) << 22 : m * 0x3f000000u;
    return __uint_as_float(f | (c & 8) << 28);
}

template <typename T>
__global__ __launch_bounds__(kMxBlock) void mxfp4_dequant_kernel(
    const uint32_t *__restrict__ q, const uint8_t *__restrict__ scale, int64_t rows, int64_t cols,
    const int32_t *__restrict__ valid_rows, T *__restrict__ x) {
    const int64_t n = mx_chunks(rows, cols, valid_rows);
    const int64_t c0 = (int64_t)blockIdx.x * (kMxBlock * kMxUnroll) + threadIdx.x;
    uint32_t w[kMxUnroll], b[kMxUnroll];
#pragma unroll
    for (int u = 0; u < kMxUnroll; ++u) {
        const int64_t c = c0 + u * kMxBlock;
        if (c < n) {
            w[u] = q[c];
            b[u] = scale[c >> 2];
        }
    }
#pragma unroll
    for (int u = 0; u < kMxUnroll; ++u) {
        const int64_t c = c0 + u * kMxBlock;
        if (c >= n) break;
        const float s = e8m0_f32(b[u]);
        float v[kMxChunk];
#pragma unroll
        for (int j = 0; j < kMxChunk; ++j) v[j] = e2m1_f32(w[u] >> (4 * j)) * s;
        store8(x + c * kMxChunk, v);
    }
}

static dim3 mx_grid(int64_t rows, int64_t cols) {
    const int64_t per = (int64_t)kMxBlock * kMxUnroll * kMxChunk;
    return dim3((unsigned)((rows * cols + per - 1) / per));
}

hipError_t launch_mxfp4_quant(const void *x, int type, int64_t rows, int64_t cols,
                              const int32_t *valid_rows, uint8_t *q, uint8_t *scale,
                              hipStream_t stream) {
#define MEGAMOE_MXQ(T)                                                                           \
    hipLaunchKernelGGL(mxfp4_quant_kernel<T>, mx_grid(rows, cols), dim3(kMxBlock), 0, stream,    \
                       static_cast<const T *>(x), rows, cols, valid_rows,                        \
                       reinterpret_cast<uint32_t *>(q), scale)
    if (type == kFp32) MEGAMOE_MXQ(float);
    else if (type == kFp16) MEGAMOE_MXQ(_Float16);
    else MEGAMOE_MXQ(__bf16);
#undef MEGAMOE_MXQ
    return hipGetLastError();
}

hipError_t launch_mxfp4_dequant(const uint8_t *q, const uint8_t *scale, int64_t rows, int64_t cols,
                                const int32_t *valid_rows, void *x, int type, hipStream_t stream) {
#define MEGAMOE_MXD(T)                                                                           \
    hipLaunchKernelGGL(mxfp4_dequant_kernel<T>, mx_grid(rows, cols), dim3(kMxBlock), 0, stream,  \
                       reinterpret_cast<const uint32_t *>(q), scale, rows, cols, valid_rows,     \
                       static_cast<T *>(x))
    if (type == kFp32) MEGAMOE_MXD(float);
    else if (type == kFp16) MEGAMOE_MXD(_Float16);
    else MEGAMOE_MXD(__bf16);
#undef MEGAMOE_MXD
    return hipGetLastError();
}

}  // namespace megamoe
