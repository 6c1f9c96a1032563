// sfa_paged_fwd.cu -- attention of a step's tokens over a paged cache
// (sfa_paged_forward in include/sfa.h): the key list of sfa_forward ("Attended
// set", section 2 of "Depth-Staggered Fibonacci Spacing for Sparse
// Attention": window distances 0..W and one interpolated row per rung) read
// through each sequence's block table.
//
// Rows kernel (this file's general path: fp32, wide windows, few tokens): kNW
// warps per (token, key/value head).  A warp takes four entries of the key
// list at a time, lane = (entry slot, 8-dimension chunk): a row of keys or
// values is eight 16-byte loads (bf16), the score of an entry for the four
// query heads is a reduction over its eight lanes that leaves head h in lanes
// 2h, 2h + 1 of the slot, and every slot keeps its own running maximum and sum
// (base 2), so that slots and warps meet only at the end.
#include "sfa_mma.cuh"
#include "sfa_paged.cuh"
#include "sfa_paged_quad.cuh"

namespace sfa {

namespace {

using namespace mma;
using namespace paged;

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
// used.
template <typename T, bool kAhead>
__device__ Partial query_part(const PagedFwd& P, int s, int pos, int g, const Chunk<T> (&raw)[kG], int first, int step) {
    const int lane = threadIdx.x & 31, slot = lane >> 3, ch = lane & 7;
    const int nwin = min(P.a.W, pos) + 1;
    int nrung = 0;
    for (int r = 0; r < P.a.nr; ++r) nrung += P.a.r[r].c <= pos ? 1 : 0;  // sorted: a prefix
    const int n = nwin + nrung;
    const T* kb = static_cast<const T*>(P.c.k) + g * kD + 8 * ch;
    const T* vb = static_cast<const T*>(P.c.v) + g * kD + 8 * ch;
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
        Chunk<T> ka, va, kc, vc;
        float t;  // weight of the second row; < 0: no entry
    };
    auto rows = [&]() {
        Rows x{};
        x.t = ra < 0 ? -1.f : wb;
        if (ra >= 0) {
            load(kb + (size_t)ra * (kHkv * kD), x.ka);
            load(vb + (size_t)ra * (kHkv * kD), x.va);
            if (rb >= 0) {
                load(kb + (size_t)rb * (kHkv * kD), x.kc);
                load(vb + (size_t)rb * (kHkv * kD), x.vc);
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
        if (now.t > 0.f) {
            float2 x[4], y[4];
            open(now.kc, x);
            open(now.vc, y);
            const float2 near = both(1.f - now.t), far = both(now.t);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                k[j] = __ffma2_rn(far, x[j], __fmul2_rn(near, k[j]));
                v[j] = __ffma2_rn(far, y[j], __fmul2_rn(near, v[j]));
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

template <typename T, int kNW>
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
    constexpr bool kAhead = kNW == 1 && sizeof(T) == 2;
    const Partial y = query_part<T, kAhead>(P, x.s, pos, g, raw, kNW > 1 ? 4 * warp : 0, 4 * kNW);
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

template <typename T, int kNW>
cudaError_t launch_rows_nw(const PagedFwd& P, cudaStream_t s) {
    constexpr int kUnits = kNW > 1 ? 1 : 2;
    const long long units = (long long)P.c.N * kHkv;
    return launch_early(rows_kernel<T, kNW>, (unsigned)((units + kUnits - 1) / kUnits), kRowThreads<kNW>, 0, s, P);
}

// As many warps a (token, head) as keep all of them resident at once (16 a SM
// at 128 registers, 152 SMs): a decode step is then one wave of one or two
// rounds of loads.  us for N single tokens over 3000 rows, bf16, with 8, 4, 2
// and 1 warps: N = 128 3.6, 4.2, 5.0, 4.8; 256 6.2, 4.3, 5.7, 5.5; 500 10.7, 7.5,
// 5.8, 6.5; 1024 19.8, 14.0, 10.7, 6.9.
template <typename T>
cudaError_t launch_rows(const PagedFwd& P, cudaStream_t s) {
    const long long most = kSms * 16 / ((long long)P.c.N * kHkv);
    return most >= 8   ? launch_rows_nw<T, 8>(P, s)
           : most >= 4 ? launch_rows_nw<T, 4>(P, s)
           : most >= 2 ? launch_rows_nw<T, 2>(P, s)
                       : launch_rows_nw<T, 1>(P, s);
}

// ------------------------------------------------- many tokens: tensor cores

// Two tiles of rows on their way or in use, at 168 registers (12 warps a SM), or
// four (kDeep) at 242 (8 warps), where that keeps every warp resident (us, two and
// four: one chunk of 512 tokens 4.4 and 4.2, of 2048 7.0 and 5.6; of 3100 6.8 and
// 9.3, 512 chunks of 2 5.7 and 8.2, 1000 of 16 43 and 49).
constexpr int kQuadWarps = 4, kDeepSlots = kSms * 2 * kQuadWarps / kHkv;

// A call of its own, so that the rare pass takes no registers of the common one
// (and one for each kernel: they differ in their registers).
template <bool kDeep>
__device__ __noinline__ void one_alone(const PagedFwd& P, const Quad& Q, int only) {
    quad_pass<true, false>(P, Q, only);
}

template <bool kDeep>
__global__ void __launch_bounds__(kQuadWarps * 32, kDeep ? 2 : 3) quad_kernel(const __grid_constant__ PagedFwd P) {
    __shared__ int rn[SFA_MAX_RUNGS], rc[SFA_MAX_RUNGS];
    __shared__ float rt[SFA_MAX_RUNGS];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x < SFA_MAX_RUNGS) {
        const Rung r = P.a.r[threadIdx.x];
        rn[threadIdx.x] = r.n;
        rc[threadIdx.x] = threadIdx.x < P.a.nr ? r.c : 0x7fffffff;
        rt[threadIdx.x] = r.t;
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // slots of four queries: sequence s starts at slot cu[s] / 4 + s, which
    // leaves room for ceil(tokens / 4) before the next one's
    const int slot = (int)(blockIdx.x / kHkv) * kQuadWarps + warp;
    Quad Q;
    Q.g = blockIdx.x % kHkv;
    const paged::Where x = paged::last_at_most(P.c, slot, [](int start, int s) { return (start >> 2) + s; });
    const int end = x.end;
    Q.s = x.s;
    Q.t0 = x.start + 4 * (slot - (x.start >> 2) - x.s);
    if (Q.t0 < 0 || Q.t0 >= P.c.N || Q.t0 >= end) return;
    Q.cnt = min(4, min(end, P.c.N) - Q.t0);
    Q.i0 = x.len - (end - Q.t0);                       // position of the first query
    Q.last = min(Q.i0 + Q.cnt, P.c.cap) - 1;           // no row behind it is read
    Q.rn = rn;
    Q.rc = rc;
    Q.rt = rt;
    if (__any_sync(kFull, lane < Q.cnt && (Q.i0 + lane < 0 || Q.i0 + lane >= P.c.cap)) && lane == 0)
        paged::report(P.c.status);
    for (unsigned redo = quad_pass<false, false, kDeep>(P, Q, -1); redo; redo &= redo - 1)
        one_alone<kDeep>(P, Q, __ffs(redo) - 1);
}

// Slots of four queries at most (quad_kernel has their places).
long long quad_slots(const PagedArgs& c) { return (long long)c.N / 4 + c.S; }

cudaError_t launch_quads(const PagedFwd& P, cudaStream_t s) {
    const long long slots = quad_slots(P.c);
    void (*const kernel)(PagedFwd) = slots <= kDeepSlots ? quad_kernel<true> : quad_kernel<false>;
    return launch_early(kernel, (unsigned)((slots + kQuadWarps - 1) / kQuadWarps * kHkv), kQuadWarps * 32, 0, s, P);
}

// Token rows from which the quad kernel is taken, if there are two a sequence at
// least: where the rows kernel has less than four warps a token (us, rows and
// quads: 300 tokens in chunks of 2 4.6 and 4.7, in one 4.2 and 3.9; 320 5.8 and
// 4.7, 5.4 and 3.9; 8 chunks of 256 11.5 and 5.4).
// Single tokens stay with the rows kernel (2048 of them 15.4 and 24.1).
constexpr int kQuadsFrom = 305;

// The tile kernel is taken, in pages that hold 16 rows at least, where the quad
// kernel's slots are more than one wave of its blocks and chunks are long: tiles
// of 28 want 32 tokens a sequence (us, quads and tiles: one chunk of 2048 tokens
// 5.5 and 6.5, of 3500 6.7 and 7.0, of 4096 10.0 and 7.1, of 8192 16.2 and 10.6;
// after 1000 rows each, 128 chunks of 32 11.0 and 10.2, 1000 of 40 82 and 50, 200
// of 28 14.6 and 16.5, 256 of 16 12.2 and 13.1; 8 chunks of 512 beside 56 single
// tokens 8.7 and 8.9, beside 192 9.1 and 13.3).  A smaller call would wait for
// the host besides, which makes the tiles' maps in 3 us.
constexpr int kQuadsWave = kSms * 3 * kQuadWarps / kHkv, kTilesEach = 32;

}  // namespace

cudaError_t launch_paged_fwd(const LayerArgs& a, const PagedArgs& c, sfa_dtype dt, const void* q, long long qs, void* o,
                             float* lse, cudaStream_t s) {
    const PagedFwd P = {a, c, q, qs, o, lse};
    // the tensor-core kernels load 32 bytes of a row at a time
    const bool wide = ((reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v)) & 31u) == 0;
    if (dt == SFA_BF16 && a.W <= 28 && wide) {
        if (quad_slots(c) > kQuadsWave && c.N >= kTilesEach * (long long)c.S && c.shift >= 4)
            return launch_paged_tiles(P, s);
        if (c.N >= kQuadsFrom && c.N >= 2 * (long long)c.S) return launch_quads(P, s);
    }
    return dt == SFA_BF16 ? launch_rows<__nv_bfloat16>(P, s) : launch_rows<float>(P, s);
}

}  // namespace sfa
