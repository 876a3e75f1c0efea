// int8_quantize_kernel.cuh -- BF16 rows -> signed 8-bit codes with one FP32 scale per
// row (token, or output channel of a weight matrix): the step ahead of the INT8 product.
//
//     s = amax / 127                          (1 for a row of zeros)
//     q = round-half-to-even( 127 x / amax )  of the real quotient, so |q| <= 127
//
// A row that holds an Inf or a NaN gets the scale NaN and zero codes: its products are
// NaN, and no other row is touched.
//
// The codes need no division.  With r = RN(127 / amax), raised by at most two steps, x * r
// lies within 2^-21 (relative) of the real quotient t = 127 x / amax.  x and amax are BF16
// (8 significant bits), so t is exactly a half-integer or at least 2^-16 * |t| away from
// every half-integer: the rounding of x * r is then that of t.  Exact half-integers are of
// two kinds.  When amax * r == 127 exactly (amax = 127 * 2^j or a power of two), x * r is
// exact too, and one FMA into 1.5 * 2^23 rounds it to even.  Otherwise the only one is
// x = +-amax / 2, t = +-63.5, which goes to +-64: raising the inexact r by two steps puts
// its product beyond 63.5.  So the code is the low byte of fma(x, r, 1.5 * 2^23).
//
// HBM-bound: 2 bytes read and 1 written per element.  A row stays in registers between
// the maximum and the codes, so X is read once: 4096 x 14336 in 27 to 29 us, 6.1 TB/s of a
// measured 6.47; 8192 x 4096 sent to two rows each in 21 to 23 us.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "ptx.cuh"

namespace nvfp4 {
namespace int8q {

constexpr int THREADS = 256;

// largest magnitude of eight BF16 values, as the 15 magnitude bits (which order like the
// values; Inf is 0x7F80 and NaN above it)
__device__ __forceinline__ unsigned amax8(const uint4& v) {
    const unsigned a = __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu);
    const unsigned b = __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu);
    const unsigned c = __vmaxu2(a, b);
    return max(c & 0xFFFFu, c >> 16);
}

struct RowScale {
    float s;    // the row's scale
    float r;    // codes = low byte of fma(x * pre, r, magic)
    float pre;  // 2^64 where 127 / amax would overflow, else 1 (exact either way)
};
__device__ __forceinline__ RowScale row_scale(unsigned bits) {
    RowScale o;
    o.pre = 1.0f;
    if (bits == 0) {
        o.s = 1.0f;
        o.r = 0.0f;
    } else if (bits >= 0x7F80u) {
        o.s = __uint_as_float(0x7FFFFFFFu);
        o.r = 0.0f;
    } else {
        float amax = __uint_as_float(bits << 16);
        o.s = __fdiv_rn(amax, 127.0f);
        if (amax < 0x1p-100f) {
            o.pre = 0x1p64f;
            amax *= o.pre;
        }
        o.r = __fdiv_rn(127.0f, amax);
        if (__fmaf_rn(o.r, amax, -127.0f) != 0.0f) o.r = __uint_as_float(__float_as_uint(o.r) + 2u);
    }
    return o;
}

__device__ __forceinline__ uint32_t codes4(uint32_t lo, uint32_t hi, const RowScale& q) {
    constexpr float magic = 12582912.0f;  // 1.5 * 2^23: the sum's low byte is the rounded product
    const uint32_t a = __float_as_uint(__fmaf_rn(__uint_as_float(lo << 16) * q.pre, q.r, magic));
    const uint32_t b = __float_as_uint(__fmaf_rn(__uint_as_float(lo & 0xFFFF0000u) * q.pre, q.r, magic));
    const uint32_t c = __float_as_uint(__fmaf_rn(__uint_as_float(hi << 16) * q.pre, q.r, magic));
    const uint32_t d = __float_as_uint(__fmaf_rn(__uint_as_float(hi & 0xFFFF0000u) * q.pre, q.r, magic));
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
__device__ __forceinline__ uint2 codes8(const uint4& v, const RowScale& q, bool finite) {
    // a non-finite row's products would be NaN, whose low byte is not zero
    if (!finite) return make_uint2(0u, 0u);
    return make_uint2(codes4(v.x, v.y, q), codes4(v.z, v.w, q));
}

// TPR threads hold a row of up to TPR * VPT * 8 elements in registers; VPT == 0: a row of
// any length, read twice.  dest == nullptr: row r goes to row r; else to rows
// dest[r*k .. r*k+k-1], those outside [0, rows*k) left out.  K % 16 == 0.
template <int TPR, int VPT>
__global__ void __launch_bounds__(THREADS)
int8_quantize_kernel(const uint4* __restrict__ X, int rows, int K, int8_t* __restrict__ codes,
                     float* __restrict__ scales, const int32_t* __restrict__ dest, int k) {
    static_assert(TPR % 32 == 0 && THREADS % TPR == 0, "whole warps per row");
    constexpr int RPB = THREADS / TPR;  // rows per block
    constexpr int WPR = TPR / 32;
    __shared__ unsigned wmax[THREADS / 32];
    const int sub = threadIdx.x / TPR, t = threadIdx.x % TPR;
    const int row = blockIdx.x * RPB + sub;
    const int nv = K / 8;
    grid_dependents_launch();  // the kernel behind may set itself up; it waits for this one's end
    grid_dependency_wait();
    const uint4* x = X + (size_t)row * nv;
    uint4 v[VPT ? VPT : 1];
    unsigned m = 0;
    if (row < rows) {
        if constexpr (VPT > 0) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                v[i] = t + i * TPR < nv ? __ldcs(x + t + i * TPR) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = 0; i < VPT; ++i) m = max(m, amax8(v[i]));
        } else {
            for (int i = t; i < nv; i += TPR) m = max(m, amax8(__ldg(x + i)));
        }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if constexpr (WPR > 1) {
        if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WPR; ++w) m = max(m, wmax[sub * WPR + w]);
    }
    if (row >= rows) return;
    const RowScale q = row_scale(m);
    const bool finite = m < 0x7F80u;
    const long long out_rows = (long long)rows * k;
    for (int j = 0; j < k; ++j) {
        const long long d = dest ? __ldg(dest + (size_t)row * k + j) : row;
        if (d < 0 || d >= out_rows) continue;
        uint2* c = reinterpret_cast<uint2*>(codes + (size_t)d * K);
        if (t == 0) scales[d] = q.s;
        if constexpr (VPT > 0) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (t + i * TPR < nv) c[t + i * TPR] = codes8(v[i], q, finite);
        } else {
            for (int i = t; i < nv; i += TPR) c[i] = codes8(__ldg(x + i), q, finite);
        }
    }
}

}  // namespace int8q
}  // namespace nvfp4
