// sfa_fp8.cuh -- 8-bit values (e4m3) as the kernels of libsfa write and read
// them.  Private to the CUDA library.
//
// An e4m3 value has a sign, four exponent bits and three of mantissa: 448 is the
// largest, 2^-6 the smallest normal one, 2^-9 the step below it; 0x7f is NaN and
// there is no infinity.  A value is kept as x = s c with a scale s for a row or
// a block of rows.
#pragma once

#include <cuda_fp8.h>
#include <cuda_fp16.h>

#include "sfa_ops.cuh"

namespace sfa {
namespace fp8 {

constexpr float kTop = 448.f;

// |x| where it is finite, else 0: what a scale is chosen from.
__device__ __forceinline__ float finite_size(float x) {
    const float a = fabsf(x);
    return a <= 3.402823466e38f ? a : 0.f;
}

// x and y in 8 bits, rounded to nearest even; what lies past the largest value
// becomes that value, what is not finite NaN (x * 0 is 0 or NaN).
__device__ __forceinline__ uint32_t code2(float x, float y) {
    const float2 v = make_float2(fmaf(x, 0.f, x), fmaf(y, 0.f, y));
    return __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d) {
    return code2(a, b) | code2(c, d) << 16;
}

// Two codes as halves: exact, NaN stays NaN.
__device__ __forceinline__ uint32_t halves(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    return (uint32_t)h.x | (uint32_t)h.y << 16;
}
__device__ __forceinline__ float2 values2(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    return __half22float2(__half2(h));
}

// Scale of a row: the largest size goes to the largest value.  It stays normal,
// so its reciprocal is finite; a row of zeros keeps zeros.
constexpr float kLeastRow = 1.17549435e-38f;  // 2^-126
__device__ __forceinline__ float row_scale(float amax) { return fmaxf(amax * (1.f / kTop), kLeastRow); }

// Scale of a block of cached rows: the smallest power of two s >= 2^-100 with
// amax <= 448 s (448 = 1.75 * 2^8).  A power of two, so that rows that are
// already there move to a larger one without a rounding, but for what then lies
// below 2^-6 s.
__device__ __forceinline__ float block_scale(float amax) {
    const int e = ((__float_as_int(amax) + 0x1fffff) >> 23) - 8;
    return __int_as_float(max(e, 127 - 100) << 23);
}

}  // namespace fp8
}  // namespace sfa
