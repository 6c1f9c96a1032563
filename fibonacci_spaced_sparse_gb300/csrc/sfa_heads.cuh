// sfa_heads.cuh -- one head row (64 values) held by four lanes, and its RMS
// norm and rotation; shared by the norm kernels and the paged append.
// Private to the CUDA library.
//
// Lane c of the four holds the RoPE pairs m = 8c .. 8c + 7: dimensions
// 8c .. 8c + 7 (x) and their partners 32 + 8c .. (y).  Both members of a pair
// sit in one lane, so the rotation needs no exchange, the mean of squares two
// shuffles, and a bf16 row is two 16-byte loads a lane.
#pragma once

#include "sfa_ops.cuh"

namespace sfa {
namespace heads {

// Values in pairs (j, j + 1) for the packed two-lane fp32 instructions.
constexpr int kP = 4;  // pairs of values of a half
struct Row {
    float2 x[kP], y[kP];
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 neg(float2 v) { return make_float2(-v.x, -v.y); }

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
    r.x = fresh(p + c);
    r.y = fresh(p + 4 + c);
}
__device__ __forceinline__ void fetch(const float* row, int c, Raw<float>& r) {
    const float4* p = reinterpret_cast<const float4*>(row);
    r.x0 = fresh(p + 2 * c);
    r.x1 = fresh(p + 2 * c + 1);
    r.y0 = fresh(p + 8 + 2 * c);
    r.y1 = fresh(p + 9 + 2 * c);
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

__device__ __forceinline__ void words(const uint4& u, float2 (&f)[kP]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < kP; ++j) f[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
}
__device__ __forceinline__ uint4 pack(const float2 (&f)[kP]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < kP; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[j].x, f[j].y);
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
        a.x[2 * j] = make_float2(v[j].x, v[j].y);
        a.x[2 * j + 1] = make_float2(v[j].z, v[j].w);
        a.y[2 * j] = make_float2(v[2 + j].x, v[2 + j].y);
        a.y[2 * j + 1] = make_float2(v[2 + j].z, v[2 + j].w);
    }
    return a;
}

__device__ __forceinline__ void close(const Row& a, Raw<__nv_bfloat16>& r) {
    r.x = pack(a.x);
    r.y = pack(a.y);
}
__device__ __forceinline__ void close(const Row& a, Raw<float>& r) {
    r.x0 = make_float4(a.x[0].x, a.x[0].y, a.x[1].x, a.x[1].y);
    r.x1 = make_float4(a.x[2].x, a.x[2].y, a.x[3].x, a.x[3].y);
    r.y0 = make_float4(a.y[0].x, a.y[0].y, a.y[1].x, a.y[1].y);
    r.y1 = make_float4(a.y[2].x, a.y[2].y, a.y[3].x, a.y[3].y);
}

// The same words of a bf16 row through shared memory: each lane copies its own
// 16-byte pieces there ahead of time and reads them back itself, so that loads in
// flight take no registers and no barrier.  Slot p of thread i is
// slot[p * blockDim.x + i].
constexpr int kPieces = sizeof(Raw<__nv_bfloat16>) / 16;

__device__ __forceinline__ void copy16(uint4* slot, const void* src, bool keep = false) {
    const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(slot));
    if (keep)  // worth a place in L1
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_row(uint4* slot, const __nv_bfloat16* row, int c) {
    const uint4* p = reinterpret_cast<const uint4*>(row);
    copy16(slot, p + c);
    copy16(slot + blockDim.x, p + 4 + c);
}
__device__ __forceinline__ Raw<__nv_bfloat16> take_row(const uint4* slot) { return {slot[0], slot[blockDim.x]}; }
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until all but the n latest groups of this thread's copies are there.
template <int n>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
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
    float2 c[kP], s[kP];
};
__device__ __forceinline__ Angles angles(const float2* rope, int pos, int c) {
    const float4* p = reinterpret_cast<const float4*>(rope + (size_t)pos * kPairs + 8 * c);
    Angles a;
#pragma unroll
    for (int j = 0; j < kP; ++j) {
        const float4 v = fresh(p + j);
        a.c[j] = make_float2(v.x, v.z);
        a.s[j] = make_float2(v.y, v.w);
    }
    return a;
}

// The same through shared memory (four pieces).
__device__ __forceinline__ void copy_angles(uint4* slot, const float2* rope, int pos, int c) {
    const uint4* p = reinterpret_cast<const uint4*>(rope + (size_t)pos * kPairs + 8 * c);
#pragma unroll
    for (int j = 0; j < kP; ++j) copy16(slot + j * blockDim.x, p + j, true);
}
__device__ __forceinline__ Angles take_angles(const uint4* slot) {
    Angles a;
#pragma unroll
    for (int j = 0; j < kP; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(slot + j * blockDim.x);
        a.c[j] = make_float2(v.x, v.z);
        a.s[j] = make_float2(v.y, v.w);
    }
    return a;
}

__device__ __forceinline__ void rotate(Row& a, const Angles& r) {
#pragma unroll
    for (int j = 0; j < kP; ++j) {
        const float2 x = a.x[j], y = a.y[j];
        a.x[j] = __ffma2_rn(x, r.c[j], __fmul2_rn(neg(y), r.s[j]));
        a.y[j] = __ffma2_rn(y, r.c[j], __fmul2_rn(x, r.s[j]));
    }
}
// The transpose (inverse) of rotate.
__device__ __forceinline__ void rotate_back(Row& a, const Angles& r) {
#pragma unroll
    for (int j = 0; j < kP; ++j) {
        const float2 x = a.x[j], y = a.y[j];
        a.x[j] = __ffma2_rn(x, r.c[j], __fmul2_rn(y, r.s[j]));
        a.y[j] = __ffma2_rn(y, r.c[j], __fmul2_rn(neg(x), r.s[j]));
    }
}

// a <- a f w
__device__ __forceinline__ void scale(Row& a, float f, const Row& w) {
#pragma unroll
    for (int j = 0; j < kP; ++j) {
        a.x[j] = __fmul2_rn(__fmul2_rn(a.x[j], both(f)), w.x[j]);
        a.y[j] = __fmul2_rn(__fmul2_rn(a.y[j], both(f)), w.y[j]);
    }
}

// Sum of the products of two rows, in every lane of the row; `mask`: lanes
// that are here together, whole rows.
__device__ __forceinline__ float dot(const Row& a, const Row& b, unsigned mask = kFull) {
    float2 s = __fmul2_rn(a.x[0], b.x[0]);
#pragma unroll
    for (int j = 1; j < kP; ++j) s = __ffma2_rn(a.x[j], b.x[j], s);
#pragma unroll
    for (int j = 0; j < kP; ++j) s = __ffma2_rn(a.y[j], b.y[j], s);
    float v = s.x + s.y;
    v += __shfl_xor_sync(mask, v, 1);
    return v + __shfl_xor_sync(mask, v, 2);
}

// 1 / sqrt(mean(x^2) + eps) of a row (the approximation's error, 2 units in
// the last place, is that of the products around it).
__device__ __forceinline__ float inv_rms(const Row& a, float eps, unsigned mask = kFull) {
    return rsqrtf(dot(a, a, mask) * (1.f / kD) + eps);
}

}  // namespace heads
}  // namespace sfa
