// Shared by the operators over rows of logits: 16-byte vectors of rows of any
// alignment, and the exponentials and comparisons of their softmax.  Included
// from .cu files only.
#pragma once

#include "k3huf_ops.h"

namespace k3huf {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// max and min that keep a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// An exponent below which 2^x is 0 in fp32, and which times 0 is 0 (minus infinity is not).
constexpr float kFloor = -2000.f;

template <typename T> constexpr int kPer = 16 / int(sizeof(T));       // values per vector

template <typename T>
__device__ __forceinline__ void unpack(const uint4 v, float (&f)[kPer<T>]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            f[i] = __uint_as_float(w[i]);
        } else {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

template <typename T>
__device__ __forceinline__ float vec_max(const uint4 v) {
    if constexpr (sizeof(T) == 4) {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    } else {
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&v);
        const __nv_bfloat162 a = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(a), __high2float(a));
    }
}

// Vector v of a row whose first value sits `shift` values into its 16-byte
// block: values [v E - shift, v E - shift + E) of the row; those outside the
// row read as -infinity.
template <typename T>
__device__ __forceinline__ uint4 load_vec(const T *row, uint32_t shift, uint32_t n, uint32_t v) {
    constexpr int E = kPer<T>;
    const int64_t j = int64_t(v) * E - shift;
    if (j >= 0 && j + E <= int64_t(n)) return __ldcs(reinterpret_cast<const uint4 *>(row + j));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            w[i] = j + i >= 0 && j + i < int64_t(n) ? __float_as_uint(row[j + i]) : 0xFF800000u;
        } else {
            const uint16_t *p = reinterpret_cast<const uint16_t *>(row);
            const int64_t a = j + 2 * i, b = a + 1;
            w[i] = (a >= 0 && a < int64_t(n) ? p[a] : 0xFF80u) | (b >= 0 && b < int64_t(n) ? uint32_t(p[b]) << 16 : 0xFF800000u);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace k3huf
