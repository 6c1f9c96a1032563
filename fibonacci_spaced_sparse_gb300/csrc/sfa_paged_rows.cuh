// sfa_paged_rows.cuh -- attention of a step's tokens over a paged cache in fp32
// arithmetic: the key list of sfa_forward ("Attended set", section 2 of
// "Depth-Staggered Fibonacci Spacing for Sparse Attention": window distances
// 0..W and one interpolated row per rung) read through each sequence's block
// table.  Private to the CUDA library.
//
// Rows kernel (fp32, wide windows, few tokens; pages of the tokens' type or of 8
// bits): kNW warps per (token, key/value head).  A warp takes four entries of
// the key list at a time, lane = (entry slot, 8-dimension chunk): a row of keys
// or values is eight 16-byte loads (bf16), the score of an entry for the four
// query heads is a reduction over its eight lanes that leaves head h in lanes
// 2h, 2h + 1 of the slot, and every slot keeps its own running maximum and sum
// (base 2), so that slots and warps meet only at the end.
//
// Rows of 8 bits are 8-byte loads with a scale each, looked up beside them; the
// scale joins the weight that a row has in its entry.
#pragma once

#include "sfa_fp8.cuh"
#include "sfa_mma.cuh"
#include "sfa_paged.cuh"

namespace sfa {
namespace paged {

using namespace mma;

template <typename T>
struct Chunk;  // 8 values of a row
template <>
struct Chunk<__nv_bfloat16> {
    uint4 u;
};
template <>
struct Chunk<float> {
    float4 u, v;
};
template <>
struct Chunk<__nv_fp8_e4m3> {
    uint2 u;
};
__device__ __forceinline__ void load(const __nv_fp8_e4m3* p, Chunk<__nv_fp8_e4m3>& x) {
    x.u = fresh(reinterpret_cast<const uint2*>(p));
}
__device__ __forceinline__ void load(const __nv_bfloat16* p, Chunk<__nv_bfloat16>& x) {
    x.u = fresh(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ void load(const float* p, Chunk<float>& x) {
    x.u = fresh(reinterpret_cast<const float4*>(p));
    x.v = fresh(reinterpret_cast<const float4*>(p) + 1);
}
// As pairs for the packed two-lane fp32 instructions.
__device__ __forceinline__ void open(const Chunk<__nv_bfloat16>& x, float2 (&f)[4]) {
    const uint32_t w[4] = {x.u.x, x.u.y, x.u.z, x.u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
}
__device__ __forceinline__ void open(const Chunk<__nv_fp8_e4m3>& x, float2 (&f)[4]) {
    f[0] = fp8::values2(x.u.x & 0xffffu), f[1] = fp8::values2(x.u.x >> 16);
    f[2] = fp8::values2(x.u.y & 0xffffu), f[3] = fp8::values2(x.u.y >> 16);
}
__device__ __forceinline__ void open(const Chunk<float>& x, float2 (&f)[4]) {
    f[0] = make_float2(x.u.x, x.u.y), f[1] = make_float2(x.u.z, x.u.w);
    f[2] = make_float2(x.v.x, x.v.y), f[3] = make_float2(x.v.z, x.v.w);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// A warp's part of one query over the entries first, first + step, ... (four
// consecutive ones at a time): each lane ends with its slots' merged sums.
// After merge(): lane (bits 4, 3) = head, chunk lane & 7: acc[0..7] unnormalised
// against the maximum m of that head, l the sum (the same in all eight lanes).
struct Partial {
    float acc[8];
    float m, l;
};

// kAhead: the rows of the next entries are loaded while the current ones are
// used.  T: the queries' type; C: the pages'.
template <typename T, typename C, bool kAhead>
__device__ Partial query_part(const PagedFwd& P, int s, int pos, int g, const Chunk<T> (&raw)[kG], int first, int step) {
    const int lane = threadIdx.x & 31, slot = lane >> 3, ch = lane & 7;
    const int nwin = min(P.a.W, pos) + 1;
    int nrung = 0;
    for (int r = 0; r < P.a.nr; ++r) nrung += P.a.r[r].c <= pos ? 1 : 0;  // sorted: a prefix
    const int n = nwin + nrung;
    constexpr bool kScaled = sizeof(C) == 1;
    const C* kb = static_cast<const C*>(P.c.k) + g * kD + 8 * ch;
    const C* vb = static_cast<const C*>(P.c.v) + g * kD + 8 * ch;
    float2 acc[kG][4];
#pragma unroll
    for (int h = 0; h < kG; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[h][j] = both(0.f);
    float m = kFloor, l = 0.f;  // of head (lane >> 1) & 3, this slot's entries
    bool bad = false;
    // row numbers of entry e of the key list; ra < 0: none
    int ra, rb;
    float wb;  // the second row's weight
    auto entry = [&](int e) {
        ra = rb = -1;
        wb = 0.f;
        if (e < nwin) {
            ra = paged::page_row(P.c, s, pos - e);
            bad |= ra < 0;
        } else if (e < n) {
            const Rung R = P.a.r[e - nwin];
            ra = paged::page_row(P.c, s, pos - R.n);
            bad |= ra < 0;
            if (R.t > 0.f) {
                rb = paged::page_row(P.c, s, pos - R.n - 1);
                bad |= rb < 0;
                if (rb < 0) ra = -1;  // an entry needs both of its rows
                wb = R.t;
            }
        }
    };
    // rows of four entries on their way (an entry without a second row: zeros)
    struct Rows {
        Chunk<C> ka, va, kc, vc;
        float t;  // weight of the second row; < 0: no entry
        float ska, sva, skc, svc;  // scales of 8-bit rows
    };
    auto rows = [&]() {
        Rows x{};
        x.t = ra < 0 ? -1.f : wb;
        if (ra >= 0) {
            load(kb + (size_t)ra * (kHkv * kD), x.ka);
            load(vb + (size_t)ra * (kHkv * kD), x.va);
            if (kScaled) {
                x.ska = fresh(paged::row_scales(P.c, ra) + g);
                x.sva = fresh(paged::row_scales(P.c, ra) + kHkv + g);
            }
            if (rb >= 0) {
                load(kb + (size_t)rb * (kHkv * kD), x.kc);
                load(vb + (size_t)rb * (kHkv * kD), x.vc);
                if (kScaled) {
                    x.skc = fresh(paged::row_scales(P.c, rb) + g);
                    x.svc = fresh(paged::row_scales(P.c, rb) + kHkv + g);
                }
            }
        }
        return x;
    };
    entry(first + slot);
    Rows next;
    if (kAhead) {
        next = rows();
        if (first + step < n) entry(first + step + slot);
    }
    float2 q[kG][4];
#pragma unroll
    for (int h = 0; h < kG; ++h) {
        open(raw[h], q[h]);
#pragma unroll
        for (int j = 0; j < 4; ++j) q[h][j] = __fmul2_rn(q[h][j], both(P.a.scale * kLog2e));
    }
    for (int e0 = first; e0 < n; e0 += step) {
        Rows now;
        if (kAhead) {
            now = next;
            if (e0 + step < n) {
                next = rows();
                if (e0 + 2 * step < n) entry(e0 + 2 * step + slot);
            }
        } else {
            now = rows();
        }
        float2 k[4], v[4];
        open(now.ka, k);
        open(now.va, v);
        if (kScaled) {
            const float near = now.t > 0.f ? 1.f - now.t : 1.f;
            const float2 nk = both(near * now.ska), nv = both(near * now.sva);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                k[j] = __fmul2_rn(nk, k[j]);
                v[j] = __fmul2_rn(nv, v[j]);
            }
        }
        if (now.t > 0.f) {
            float2 x[4], y[4];
            open(now.kc, x);
            open(now.vc, y);
            const float2 near = both(1.f - now.t);
            const float2 fk = both(kScaled ? now.t * now.skc : now.t), fv = both(kScaled ? now.t * now.svc : now.t);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                k[j] = __ffma2_rn(fk, x[j], kScaled ? k[j] : __fmul2_rn(near, k[j]));
                v[j] = __ffma2_rn(fv, y[j], kScaled ? v[j] : __fmul2_rn(near, v[j]));
            }
        }
        const bool there = now.t >= 0.f;
        if (!kAhead && e0 + step < n) entry(e0 + step + slot);  // the next entries' pages are looked up meanwhile
        float d[kG];
#pragma unroll
        for (int h = 0; h < kG; ++h) {
            float2 s = __fmul2_rn(q[h][0], k[0]);
#pragma unroll
            for (int j = 1; j < 4; ++j) s = __ffma2_rn(q[h][j], k[j], s);
            d[h] = s.x + s.y;
        }
        // sum over the slot's eight lanes; head h ends in lanes 2h, 2h + 1
        const bool up4 = lane & 4, up2 = lane & 2;
        float d0 = (up4 ? d[2] : d[0]) + __shfl_xor_sync(kFull, up4 ? d[0] : d[2], 4);
        float d1 = (up4 ? d[3] : d[1]) + __shfl_xor_sync(kFull, up4 ? d[1] : d[3], 4);
        float x = (up2 ? d1 : d0) + __shfl_xor_sync(kFull, up2 ? d0 : d1, 2);
        x += __shfl_xor_sync(kFull, x, 1);
        if (!there) x = -INFINITY;
        if (__any_sync(kFull, x > m + kLazy)) {
            const float up = fmaxf(m, x);
            const float f = exp2f(m - up);
            m = up;
            l *= f;
#pragma unroll
            for (int h = 0; h < kG; ++h) {
                const float fh = __shfl_sync(kFull, f, (lane & 24) + 2 * h);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[h][j] = __fmul2_rn(acc[h][j], both(fh));
            }
        }
        const float p = exp2f(x - m);
        l += p;
#pragma unroll
        for (int h = 0; h < kG; ++h) {
            const float ph = __shfl_sync(kFull, p, (lane & 24) + 2 * h);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[h][j] = __ffma2_rn(both(ph), v[j], acc[h][j]);
        }
    }
    if (__any_sync(kFull, bad) && lane == 0) paged::report(P.c.status);
    // the four slots: one maximum per head, then half the heads change sides twice
    float top = fmaxf(m, __shfl_xor_sync(kFull, m, 8));
    top = fmaxf(top, __shfl_xor_sync(kFull, top, 16));
    const float f = exp2f(m - top);
    l *= f;
    l += __shfl_xor_sync(kFull, l, 8);
    l += __shfl_xor_sync(kFull, l, 16);
#pragma unroll
    for (int h = 0; h < kG; ++h) {
        const float fh = __shfl_sync(kFull, f, (lane & 24) + 2 * h);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[h][j] = __fmul2_rn(acc[h][j], both(fh));
    }
    const bool up16 = lane & 16, up8 = lane & 8;
    Partial out;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        auto at = [&](int h) { return j & 1 ? acc[h][j / 2].y : acc[h][j / 2].x; };
        const float a0 = (up16 ? at(2) : at(0)) + __shfl_xor_sync(kFull, up16 ? at(0) : at(2), 16);
        const float a1 = (up16 ? at(3) : at(1)) + __shfl_xor_sync(kFull, up16 ? at(1) : at(3), 16);
        out.acc[j] = (up8 ? a1 : a0) + __shfl_xor_sync(kFull, up8 ? a0 : a1, 8);
    }
    out.m = __shfl_sync(kFull, top, 2 * slot);
    out.l = __shfl_sync(kFull, l, 2 * slot);
    return out;
}

// Token t of sequence s: its position; false when that is out of range (its
// outputs become zeros).
template <typename T>
__device__ __forceinline__ void zero_out(const PagedFwd& P, int t, int g, int i, int n) {
    T* o = static_cast<T*>(P.o) + ((size_t)t * kHq + g * kG) * kD;
    for (int j = i; j < kG * kD; j += n) o[j] = from_f32<T>(0.f);
    if (P.lse && i < kG) P.lse[(size_t)t * kHq + g * kG + i] = 0.f;
}

// A whole query's outputs from its merged state: lane (head h, chunk ch).
template <typename T>
__device__ __forceinline__ void write_part(const PagedFwd& P, int t, int g, int h, int ch, const Partial& x) {
    const size_t at = (size_t)t * kHq + g * kG + h;
    const float inv = x.l != 0.f ? 1.f / x.l : 0.f;  // no entry: zeros
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = x.acc[j] * inv;
    store8(static_cast<T*>(P.o) + at * kD + 8 * ch, f);
    if (P.lse && ch == 0) P.lse[at] = x.l == 0.f ? -INFINITY : (x.m + log2f(x.l)) * kLn2;
}

template <int kNW>
constexpr int kRowThreads = kNW > 1 ? 32 * kNW : 64;  // one unit a block, or two of one warp each (of eight: 2048 single tokens 15.9 and 15.5 us, 16 ragged fp32 prompts of up to 1024 50.1 and 45.8)

template <typename T, typename C, int kNW>
__global__ void __launch_bounds__(kRowThreads<kNW>, 512 / kRowThreads<kNW>) rows_kernel(const __grid_constant__ PagedFwd P) {
    constexpr int kThreads = kRowThreads<kNW>, kUnits = kNW > 1 ? 1 : 2;  // (token, head) of a block
    __shared__ __align__(16) float part[kNW > 1 ? kNW : 1][kNW > 1 ? kG * kD : 4];
    __shared__ float top[kNW][kG], sum[kNW][kG];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned unit = blockIdx.x * kUnits + (kNW > 1 ? 0 : warp);
    const int t = (int)(unit / kHkv), g = (int)(unit % kHkv);
    if (t >= P.c.N) return;  // with kNW > 1 the whole block, here and below
    // the query's loads go out before the lookups, and those of the metadata
    // together (sequence_of): three latencies in line, the lookups', the block
    // table's and the rows', where five took 0.2 to 0.3 us more (3 tokens 2.9 and
    // 3.3 us, 256 tokens 4.4 and 4.6)
    Chunk<T> raw[kG];
    const T* qrow = static_cast<const T*>(P.q) + (size_t)t * P.qs + g * kG * kD + 8 * (lane & 7);
#pragma unroll
    for (int h = 0; h < kG; ++h) load(qrow + h * kD, raw[h]);
    const paged::Where x = paged::sequence_of(P.c, t);
    if (x.s >= P.c.S) return;
    const int pos = x.len - (x.end - t);
    if (pos < 0 || pos >= P.c.cap) {
        const int i = kNW > 1 ? threadIdx.x : lane;
        if (i == 0 && g == 0) paged::report(P.c.status);
        zero_out<T>(P, t, g, i, kNW > 1 ? kThreads : 32);
        return;
    }
    // With several warps a token there are one or two rounds of loads; with one
    // there are six, and loads ahead pay (us, without and with, 1024 single
    // tokens 7.9 and 7.2, 2048 18.7 and 16.0).  fp32 rows do not fit the
    // registers twice (128 spill 90 bytes: 1024 single tokens 10.6 and 11.8).
    constexpr bool kAhead = kNW == 1 && sizeof(C) <= 2;
    const Partial y = query_part<T, C, kAhead>(P, x.s, pos, g, raw, kNW > 1 ? 4 * warp : 0, 4 * kNW);
    const int h = lane >> 3, ch = lane & 7;
    if (kNW == 1) {
        write_part<T>(P, t, g, h, ch, y);
        return;
    }
    if (ch == 0) {
        top[warp][h] = y.m;
        sum[warp][h] = y.l;
    }
    float* mine = part[kNW > 1 ? warp : 0] + (kNW > 1 ? h * kD + 8 * ch : 0);
    if (kNW > 1) {
        reinterpret_cast<float4*>(mine)[0] = make_float4(y.acc[0], y.acc[1], y.acc[2], y.acc[3]);
        reinterpret_cast<float4*>(mine)[1] = make_float4(y.acc[4], y.acc[5], y.acc[6], y.acc[7]);
    }
    __syncthreads();
    T* o = static_cast<T*>(P.o) + ((size_t)t * kHq + g * kG) * kD;
#pragma unroll
    for (int i = threadIdx.x; i < kG * kD; i += kThreads) {
        const int hh = i / kD;
        float m = top[0][hh];
#pragma unroll
        for (int w = 1; w < kNW; ++w) m = fmaxf(m, top[w][hh]);
        float l = 0.f, v = 0.f;
#pragma unroll
        for (int w = 0; w < kNW; ++w) {
            const float f = exp2f(top[w][hh] - m);
            l = fmaf(f, sum[w][hh], l);
            v = fmaf(f, part[kNW > 1 ? w : 0][kNW > 1 ? i : 0], v);
        }
        const float inv = l != 0.f ? 1.f / l : 0.f;
        o[i] = from_f32<T>(v * inv);
        if (P.lse && i % kD == 0)
            P.lse[(size_t)t * kHq + g * kG + hh] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
}

template <typename T, typename C, int kNW>
cudaError_t launch_rows_nw(const PagedFwd& P, cudaStream_t s) {
    constexpr int kUnits = kNW > 1 ? 1 : 2;
    const long long units = (long long)P.c.N * kHkv;
    return launch_early(rows_kernel<T, C, kNW>, (unsigned)((units + kUnits - 1) / kUnits), kRowThreads<kNW>, 0, s, P);
}

// As many warps a (token, head) as keep all of them resident at once (16 a SM
// at 128 registers, 152 SMs): a decode step is then one wave of one or two
// rounds of loads.  us for N single tokens over 3000 rows, bf16, with 8, 4, 2
// and 1 warps: N = 128 3.6, 4.2, 5.0, 4.8; 256 6.2, 4.3, 5.7, 5.5; 500 10.7, 7.5,
// 5.8, 6.5; 1024 19.8, 14.0, 10.7, 6.9.
template <typename T, typename C>
cudaError_t launch_rows(const PagedFwd& P, cudaStream_t s) {
    const long long most = kSms * 16 / ((long long)P.c.N * kHkv);
    return most >= 8   ? launch_rows_nw<T, C, 8>(P, s)
           : most >= 4 ? launch_rows_nw<T, C, 4>(P, s)
           : most >= 2 ? launch_rows_nw<T, C, 2>(P, s)
                       : launch_rows_nw<T, C, 1>(P, s);
}

}  // namespace paged
}  // namespace sfa
