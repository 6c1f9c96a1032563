// sfa_append_fp8.cu -- one step's keys and values into a paged cache of 8-bit
// rows, with the norm and rotation of the keys (and of the step's queries) on
// the way (sfa_paged_append_fp8 in include/sfa.h).
//
// A block of R = 2^block_shift positions has one scale for its keys and one for
// its values a head: the smallest power of two s with max |x| <= 448 s over what
// the block holds.  A step's new rows of a block are read, their largest size
// taken, and the rows written with the scale that this gives; where it is larger
// than the one that older rows of the block were written with, those are written
// again (c <- round(c s_old / s_new), exact but for what becomes subnormal).
//
// One warp has a block's keys or values of one head: nobody else touches its
// rows or its scale, so there are no atomics and no second launch.  Four lanes
// hold a head row (sfa_heads.cuh), eight rows a warp at a time.  Blocks are found
// in one of two ways: warps for N / R + 2 S places, where sequence s starts at
// place cu[s] / R + 2 s, which leaves room for all blocks that its tokens can
// touch; or, where sequences bring about one token each, a warp for every token,
// which has the token's block if the token is the first there.  Queries are rows
// as in sfa_append.cu, in thread blocks of their own in the same launch.
//
// Bound by memory when there are many tokens and by the latency of its lookups in
// a decode step (metadata -> block table -> scale -> rows).
#include "sfa_fp8.cuh"
#include "sfa_heads.cuh"
#include "sfa_paged.cuh"

namespace sfa {

namespace {

using namespace heads;

constexpr int kThreads = 128;
constexpr int kRoles = 2 * kHkv;          // warps of a block of rows: keys and values of each head
constexpr int kQuads = kHq / 2;           // quads of a token's queries
constexpr int kQueries = kThreads / 4 / kQuads;  // tokens of a thread block of queries
static_assert(kRoles * 32 == kThreads, "a thread block has one block of rows");

struct Fp8Append {
    AppendArgs a;
    int query_blocks;  // thread blocks of queries, in front
};

template <typename T>
__device__ __forceinline__ void queries(const AppendArgs& a, int block) {
    const int quad = block * (kThreads / 4) + (threadIdx.x >> 2), c = threadIdx.x & 3;
    const int t = quad / kQuads, role = quad % kQuads;
    const int warp_t = __shfl_sync(kFull, t, 0);
    if (warp_t >= a.c.N) return;
    const bool in_n = t < a.c.N;
    const int tt = in_n ? t : a.c.N - 1;
    const T* src = static_cast<const T*>(a.q) + (size_t)tt * a.qs + role * 2 * kD;
    Raw<T> raw[2];
    fetch(src, c, raw[0]);
    fetch(src + kD, c, raw[1]);
    Row w{};
    if (a.wq) w = weights(a.wq, c);
    bool live;
    const paged::Where x = paged::each_token(a.c, tt, in_n, warp_t, live);
    if (!live) return;
    const int pos = x.len - (x.end - tt);
    const bool good = pos >= 0 && pos < a.c.cap;
    Angles rot;
    if (a.rope && good) rot = angles(a.rope, pos, c);
    T* dst = static_cast<T*>(a.qhat) + (size_t)t * (kHq * kD) + role * 2 * kD;
    const unsigned mask = 0xfu << (threadIdx.x & 28);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        Row y = open(raw[h]);
        if (a.wq) scale(y, inv_rms(y, a.eps, mask), w);
        if (a.rope && good) rotate(y, rot);
        if (!good) y = Row{};
        store(dst + h * kD, c, y);
    }
}

__device__ __forceinline__ float top_of(const Row& y) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < kP; ++j) {
        m = fmaxf(m, fmaxf(fp8::finite_size(y.x[j].x), fp8::finite_size(y.x[j].y)));
        m = fmaxf(m, fmaxf(fp8::finite_size(y.y[j].x), fp8::finite_size(y.y[j].y)));
    }
    return m;
}

// f times a lane's part of a row, in 8 bits: dimensions 8c .. and 32 + 8c .. .
__device__ __forceinline__ uint2 codes_of(const float2 (&v)[kP], float f) {
    return make_uint2(fp8::code4(v[0].x * f, v[0].y * f, v[1].x * f, v[1].y * f),
                      fp8::code4(v[2].x * f, v[2].y * f, v[3].x * f, v[3].y * f));
}
__device__ __forceinline__ uint2 again(uint2 u, float f) {
    const float2 v[kP] = {fp8::values2(u.x & 0xffffu), fp8::values2(u.x >> 16), fp8::values2(u.y & 0xffffu),
                          fp8::values2(u.y >> 16)};
    return codes_of(v, f);
}

// kKept: rows of a block are at most 8 kKept and stay in registers between the
// two passes; 0: any number, read twice.
template <typename T, int kKept, bool kPerToken>
__global__ void __launch_bounds__(kThreads) append_fp8_kernel(const __grid_constant__ Fp8Append P) {
    const AppendArgs& a = P.a;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if ((int)blockIdx.x < P.query_blocks) {
        queries<T>(a, blockIdx.x);
        return;
    }
    const int unit = (int)blockIdx.x - P.query_blocks, role = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = lane >> 2, c = lane & 3, shift = a.c.block_shift;
    const bool key = role < kHkv;
    const int head = role & (kHkv - 1);
    // the block of rows: positions base .. base + R - 1 of sequence x.s, whose new
    // tokens start at position at
    paged::Where x;
    int at, base;
    if (kPerToken) {
        x = paged::sequence_of(a.c, unit);
        if (x.s >= a.c.S) return;
        at = x.len - (x.end - x.start);
        const int pos = at + (unit - x.start);
        if (pos < 0) {
            if (threadIdx.x == 0) paged::report(a.c.status);
            return;
        }
        base = pos >> shift << shift;
        if (unit != x.start && pos != base) return;  // not the first token of its block
    } else {
        x = paged::last_at_most(a.c, unit, [&](int start, int s) { return (start >> shift) + 2 * s; });
        if (x.start < 0 || x.start >= a.c.N || x.end <= x.start) return;
        at = x.len - (x.end - x.start);
        const int place = unit - (x.start >> shift) - 2 * x.s;
        if (place == 0 && at < 0 && threadIdx.x == 0) paged::report(a.c.status);
        const long long b = ((long long)(max(at, 0) >> shift) + place) << shift;
        if (place < 0 || b >= (long long)at + (x.end - x.start)) return;
        base = (int)b;
    }
    const int end = min(x.end, a.c.N) - x.start + at;   // behind the last new position
    if (end <= 0) return;  // no position exists
    const int first = max(max(at, 0), base) - base;     // new rows of the block: first .. last - 1
    const int last = min(min(end, a.c.cap) - base, 1 << shift);
    if (min(end - base, 1 << shift) > max(last, first) && threadIdx.x == 0) paged::report(a.c.status);
    if (first >= last) return;
    const int row0 = paged::page_row(a.c, x.s, base);
    if (row0 < 0) {
        if (threadIdx.x == 0) paged::report(a.c.status);
        return;
    }
    float* sp = paged::row_scales(a.c, row0) + (key ? 0 : kHkv) + head;
    const float old = first > 0 ? fresh(sp) : 0.f;
    const T* src = static_cast<const T*>(key ? a.kn : a.vn) + head * kD;
    const long long stride = key ? a.ks : a.vs;
    const int t0 = x.start + (base - at);  // the token row of the block's first position
    Row w{};
    if (key && a.wk) w = weights(a.wk, c);
    auto row_of = [&](int j) {  // new row j of the block (zeros where there is none)
        Raw<T> raw{};
        const bool in = j >= first && j < last;
        if (in) fetch(src + (long long)(t0 + j) * stride, c, raw);
        Row y = open(raw);
        if (key) {
            if (a.wk) scale(y, inv_rms(y, a.eps), w);
            if (a.rope && in) rotate(y, angles(a.rope, base + j, c));
            if (!in) y = Row{};  // (0 / 0 with eps = 0)
        }
        return y;
    };
    Row kept[kKept ? kKept : 1];
    float top = 0.f;
    if (kKept) {
#pragma unroll
        for (int i = 0; i < kKept; ++i) {
            kept[i] = row_of(8 * i + quad);
            top = fmaxf(top, top_of(kept[i]));
        }
    } else {
        for (int j = first & ~7; j < last; j += 8) top = fmaxf(top, top_of(row_of(j + quad)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    const float s = fmaxf(fp8::block_scale(top), old), inv = 1.f / s;
    unsigned char* dst = static_cast<unsigned char*>(key ? a.c.k : a.c.v) + (size_t)row0 * (kHkv * kD) + head * kD + 8 * c;
    auto put8 = [&](int j, const Row& y) {
        if (j < first || j >= last) return;
        unsigned char* p = dst + (size_t)j * (kHkv * kD);
        *reinterpret_cast<uint2*>(p) = codes_of(y.x, inv);
        *reinterpret_cast<uint2*>(p + kPairs) = codes_of(y.y, inv);
    };
    if (kKept) {
#pragma unroll
        for (int i = 0; i < kKept; ++i) put8(8 * i + quad, kept[i]);
    } else {
        for (int j = first & ~7; j < last; j += 8) put8(j + quad, row_of(j + quad));
    }
    if (first > 0 && s > old) {
        const float f = old / s;
        for (int j = quad; j < first; j += 8) {
            uint2* p = reinterpret_cast<uint2*>(dst + (size_t)j * (kHkv * kD));
            const uint2 u = fresh(p), v = fresh(p + kPairs / 8);
            p[0] = again(u, f);
            p[kPairs / 8] = again(v, f);
        }
    }
    if (lane == 0) *sp = s;
}

template <typename T, int kKept>
cudaError_t launch_blocks(const Fp8Append& P, cudaStream_t s) {
    const PagedArgs& c = P.a.c;
    const bool per_token = c.N <= 2LL * c.S;
    const long long units = per_token ? c.N : ((long long)c.N >> c.block_shift) + 2LL * c.S;
    return launch_early(per_token ? append_fp8_kernel<T, kKept, true> : append_fp8_kernel<T, kKept, false>,
                        (unsigned)(P.query_blocks + units), kThreads, 0, s, P);
}

template <typename T>
cudaError_t launch_append(const AppendArgs& a, cudaStream_t s) {
    const Fp8Append P = {a, a.q ? (a.c.N + kQueries - 1) / kQueries : 0};
    return a.c.block_shift == 3   ? launch_blocks<T, 1>(P, s)
           : a.c.block_shift == 4 ? launch_blocks<T, 2>(P, s)
                                  : launch_blocks<T, 0>(P, s);
}

}  // namespace

cudaError_t launch_paged_append_fp8(const AppendArgs& a, sfa_dtype dt, cudaStream_t s) {
    return dt == SFA_BF16 ? launch_append<__nv_bfloat16>(a, s) : launch_append<float>(a, s);
}

}  // namespace sfa
