// sfa_heads.cuh -- one head row (64 values) held by four lanes, and its RMS
// norm and rotation; shared by the norm kernels and the paged append.
// Private to the CUDA library.
//
// Lane c of the four holds the RoPE pairs m = 8c .. 8c + 7: dimensions
// 8c .. 8c + 7 (x) and their partners 32 + 8c .. (y).  Both members of a pair
// sit in one lane, so the rotation needs no exchange, the mean of squares two
// shuffles, and a bf16 row is two 16-byte loads a lane.
#pragma once

#include "sfa_internal.cuh"

namespace sfa {
namespace heads {

struct Row {
    float x[8], y[8];
};

// The raw words of a lane's part of a row, kept apart from their conversion so
// that the loads of several rows are in flight together.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
    uint4 x, y;
};
template <>
struct Raw<float> {
    float4 x0, x1, y0, y1;
};

__device__ __forceinline__ void fetch(const __nv_bfloat16* row, int c, Raw<__nv_bfloat16>& r) {
    const uint4* p = reinterpret_cast<const uint4*>(row);
    r.x = __ldg(p + c);
    r.y = __ldg(p + 4 + c);
}
__device__ __forceinline__ void fetch(const float* row, int c, Raw<float>& r) {
    const float4* p = reinterpret_cast<const float4*>(row);
    r.x0 = __ldg(p + 2 * c);
    r.x1 = __ldg(p + 2 * c + 1);
    r.y0 = __ldg(p + 8 + 2 * c);
    r.y1 = __ldg(p + 9 + 2 * c);
}

__device__ __forceinline__ void put(__nv_bfloat16* row, int c, const Raw<__nv_bfloat16>& r) {
    uint4* p = reinterpret_cast<uint4*>(row);
    p[c] = r.x;
    p[4 + c] = r.y;
}
__device__ __forceinline__ void put(float* row, int c, const Raw<float>& r) {
    float4* p = reinterpret_cast<float4*>(row);
    p[2 * c] = r.x0;
    p[2 * c + 1] = r.x1;
    p[8 + 2 * c] = r.y0;
    p[9 + 2 * c] = r.y1;
}

__device__ __forceinline__ void words(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ Row open(const Raw<__nv_bfloat16>& r) {
    Row a;
    words(r.x, a.x);
    words(r.y, a.y);
    return a;
}
__device__ __forceinline__ Row open(const Raw<float>& r) {
    Row a;
    const float4 v[4] = {r.x0, r.x1, r.y0, r.y1};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        a.x[4 * j] = v[j].x;
        a.x[4 * j + 1] = v[j].y;
        a.x[4 * j + 2] = v[j].z;
        a.x[4 * j + 3] = v[j].w;
        a.y[4 * j] = v[2 + j].x;
        a.y[4 * j + 1] = v[2 + j].y;
        a.y[4 * j + 2] = v[2 + j].z;
        a.y[4 * j + 3] = v[2 + j].w;
    }
    return a;
}

__device__ __forceinline__ void close(const Row& a, Raw<__nv_bfloat16>& r) {
    r.x = pack(a.x);
    r.y = pack(a.y);
}
__device__ __forceinline__ void close(const Row& a, Raw<float>& r) {
    r.x0 = make_float4(a.x[0], a.x[1], a.x[2], a.x[3]);
    r.x1 = make_float4(a.x[4], a.x[5], a.x[6], a.x[7]);
    r.y0 = make_float4(a.y[0], a.y[1], a.y[2], a.y[3]);
    r.y1 = make_float4(a.y[4], a.y[5], a.y[6], a.y[7]);
}

template <typename T>
__device__ __forceinline__ void store(T* row, int c, const Row& a) {
    Raw<T> r;
    close(a, r);
    put(row, c, r);
}

// A lane's part of D fp32 weights.
__device__ __forceinline__ Row weights(const float* w, int c) {
    Raw<float> r;
    fetch(w, c, r);
    return open(r);
}

// (cos, sin) of a lane's pairs at one position: 64 contiguous bytes of the
// table row.
struct Angles {
    float c[8], s[8];
};
__device__ __forceinline__ Angles angles(const float2* __restrict__ rope, int pos, int c) {
    const float4* p = reinterpret_cast<const float4*>(rope + (size_t)pos * kPairs + 8 * c);
    Angles a;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float4 v = __ldg(p + j);
        a.c[2 * j] = v.x;
        a.s[2 * j] = v.y;
        a.c[2 * j + 1] = v.z;
        a.s[2 * j + 1] = v.w;
    }
    return a;
}

__device__ __forceinline__ void rotate(Row& a, const Angles& r) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float x = a.x[j], y = a.y[j];
        a.x[j] = x * r.c[j] - y * r.s[j];
        a.y[j] = y * r.c[j] + x * r.s[j];
    }
}
// The transpose (inverse) of rotate.
__device__ __forceinline__ void rotate_back(Row& a, const Angles& r) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float x = a.x[j], y = a.y[j];
        a.x[j] = x * r.c[j] + y * r.s[j];
        a.y[j] = y * r.c[j] - x * r.s[j];
    }
}

// Sum over the four lanes of a row.
__device__ __forceinline__ float row_sum(float v) {
    v += __shfl_xor_sync(kFull, v, 1);
    return v + __shfl_xor_sync(kFull, v, 2);
}

__device__ __forceinline__ float dot(const Row& a, const Row& b) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s += a.x[j] * b.x[j] + a.y[j] * b.y[j];
    return row_sum(s);
}

// 1 / sqrt(mean(x^2) + eps) of a row.
__device__ __forceinline__ float inv_rms(const Row& a, float eps) {
    return 1.f / sqrtf(dot(a, a) * (1.f / kD) + eps);
}

}  // namespace heads
}  // namespace sfa
