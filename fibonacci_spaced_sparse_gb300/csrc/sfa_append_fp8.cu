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
// A thread block has a block of rows, kSplit warps its keys or values of one head:
// nobody else touches those rows or their scale, so there are no atomics and no second
// launch.  Four lanes hold a head row (sfa_heads.cuh), eight rows a warp at a time,
// sixteen in registers between the two passes, so a block of up to 64 rows is read
// once (64 rows read twice by one warp: 15.0 us for 16 prompts of up to 2048 tokens).
// Blocks of rows are found in one of two ways: a thread block for each of N / R + 2 S places,
// where sequence s starts at place cu[s] / R + 2 s, which leaves room for all blocks that its
// tokens can touch (the others return after the lookup); or, where sequences bring about one
// token each, a thread block for every token, which has the token's block of rows if the token
// is the first there.  Queries are rows
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

constexpr int kRoles = 2 * kHkv;  // of a block of rows: keys and values of each head
template <int kSplit>
constexpr int kThreads = 32 * kRoles * kSplit;

// Query rows of a quad: four share their token's angles where there are many bf16
// tokens, two otherwise (us, four and two: 16 prompts of up to 2048 tokens 8.0 and 8.3,
// fp32 15.4 and 12.9, 100 sequences of two tokens 3.8 and 3.25).
constexpr int kFourFrom = 4096;

struct Fp8Append {
    AppendArgs a;
    int query_blocks;  // thread blocks of queries, in front
    bool four;         // query rows of a quad, not two
};

template <typename T, int kEach>
__device__ __forceinline__ void queries(const AppendArgs& a, int block) {
    constexpr int kQuads = kHq / kEach;  // of a token
    const int quad = block * (int)(blockDim.x / 4) + (threadIdx.x >> 2), c = threadIdx.x & 3;
    const int t = quad / kQuads, role = quad % kQuads;
    const int warp_t = __shfl_sync(kFull, t, 0);
    if (warp_t >= a.c.N) return;
    const bool in_n = t < a.c.N;
    const int tt = in_n ? t : a.c.N - 1;
    const T* src = static_cast<const T*>(a.q) + (size_t)tt * a.qs + role * kEach * kD;
    Raw<T> raw[kEach];
#pragma unroll
    for (int h = 0; h < kEach; ++h) fetch(src + h * kD, c, raw[h]);
    Row w{};
    if (a.wq) w = weights(a.wq, c);
    bool live;
    const paged::Where x = paged::each_token(a.c, tt, in_n, warp_t, live);
    if (!live) return;
    const int pos = x.len - (x.end - tt);
    const bool good = pos >= 0 && pos < a.c.cap;
    Angles rot;
    if (a.rope && good) rot = angles(a.rope, pos, c);
    T* dst = static_cast<T*>(a.qhat) + (size_t)t * (kHq * kD) + role * kEach * kD;
    const unsigned mask = 0xfu << (threadIdx.x & 28);
#pragma unroll
    for (int h = 0; h < kEach; ++h) {
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

// kKept: rows of a block are at most 8 kKept kSplit and stay in registers between
// the two passes; 0: any number, read twice.  With many tokens 24 warps a SM, at 80
// registers, are faster than what fits without a limit, 16 (us for 16 prompts of up to
// 2048 tokens 8.3 and 8.9), with single tokens they are slower (256 of them 3.2 and
// 3.0).
template <typename T, int kKept, int kSplit, bool kPerToken>
__global__ void __launch_bounds__(kThreads<kSplit>, kPerToken ? 1 : 6 / kSplit)
    append_fp8_kernel(const __grid_constant__ Fp8Append P) {
    const AppendArgs& a = P.a;
    __shared__ float tops[kRoles][kSplit];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if ((int)blockIdx.x < P.query_blocks) {
        if (sizeof(T) == 2 && P.four)
            queries<T, 4>(a, blockIdx.x);
        else
            queries<T, 2>(a, blockIdx.x);
        return;
    }
    const int unit = (int)blockIdx.x - P.query_blocks, role = (threadIdx.x >> 5) % kRoles, lane = threadIdx.x & 31;
    const int part = threadIdx.x / (32 * kRoles), quad = 8 * part + (lane >> 2), c = lane & 3;
    const int shift = a.c.block_shift;
    constexpr int kStep = 8 * kSplit;  // rows of a role's warps together
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
    const T* src = static_cast<const T*>(key ? a.kn : a.vn) + head * kD;
    const long long stride = key ? a.ks : a.vs;
    const int t0 = x.start + (base - at);  // the token row of the block's first position
    Row w{};
    if (key && a.wk) w = weights(a.wk, c);
    auto is_new = [&](int j) { return j >= first && j < last; };
    auto row_of = [&](int j, const Raw<T>& raw, const Angles& rot) {  // new row j of the block (zeros where there is none)
        Row y = open(raw);
        if (key) {
            if (a.wk) scale(y, inv_rms(y, a.eps), w);
            if (a.rope) rotate(y, rot);
            if (!is_new(j)) y = Row{};  // (0 / 0 with eps = 0)
        }
        return y;
    };
    auto load = [&](int j, Raw<T>& raw, Angles& rot) {
        raw = Raw<T>{};
        rot = Angles{};
        if (!is_new(j)) return;
        fetch(src + (long long)(t0 + j) * stride, c, raw);
        if (key && a.rope) rot = angles(a.rope, base + j, c);
    };
    // the new rows are on their way while the page and the scale so far are looked up
    Raw<T> raw[kKept ? kKept : 1];
    Angles rot[kKept ? kKept : 1];
#pragma unroll
    for (int i = 0; i < kKept; ++i) load(kStep * i + quad, raw[i], rot[i]);
    const int row0 = paged::page_row(a.c, x.s, base);
    if (row0 < 0) {
        if (threadIdx.x == 0) paged::report(a.c.status);
        return;
    }
    float* sp = paged::row_scales(a.c, row0) + (key ? 0 : kHkv) + head;
    const float old = first > 0 ? fresh(sp) : 0.f;
    Row kept[kKept ? kKept : 1];
    float top = 0.f;
    auto again_row = [&](int j) {
        load(j, raw[0], rot[0]);
        return row_of(j, raw[0], rot[0]);
    };
    if (kKept) {
#pragma unroll
        for (int i = 0; i < kKept; ++i) {
            kept[i] = row_of(kStep * i + quad, raw[i], rot[i]);
            top = fmaxf(top, top_of(kept[i]));
        }
    } else {
        for (int j = first & -kStep; j < last; j += kStep) top = fmaxf(top, top_of(again_row(j + quad)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    if (kSplit > 1) {  // (what ends a warp above ends the others as well)
        if (lane == 0) tops[role][part] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSplit; ++i) top = fmaxf(top, tops[role][i]);
    }
    const float s = fmaxf(fp8::block_scale(top), old), inv = 1.f / s;
    unsigned char* dst = static_cast<unsigned char*>(key ? a.c.k : a.c.v) + (size_t)row0 * (kHkv * kD) + head * kD + 8 * c;
    auto put8 = [&](int j, const Row& y) {
        if (!is_new(j)) return;
        unsigned char* p = dst + (size_t)j * (kHkv * kD);
        *reinterpret_cast<uint2*>(p) = codes_of(y.x, inv);
        *reinterpret_cast<uint2*>(p + kPairs) = codes_of(y.y, inv);
    };
    if (kKept) {
#pragma unroll
        for (int i = 0; i < kKept; ++i) put8(kStep * i + quad, kept[i]);
    } else {
        for (int j = first & -kStep; j < last; j += kStep) put8(j + quad, again_row(j + quad));
    }
    if (first > 0 && s > old) {
        const float f = old / s;
        for (int j = quad; j < first; j += kStep) {
            uint2* p = reinterpret_cast<uint2*>(dst + (size_t)j * (kHkv * kD));
            const uint2 u = fresh(p), v = fresh(p + kPairs / 8);
            p[0] = again(u, f);
            p[kPairs / 8] = again(v, f);
        }
    }
    if (lane == 0 && part == 0) *sp = s;
}

template <typename T, int kKept, int kSplit, bool kPerToken>
cudaError_t launch_blocks(const AppendArgs& a, cudaStream_t s) {
    const bool four = sizeof(T) == 2 && a.c.N >= kFourFrom;
    const int tokens = kThreads<kSplit> / 4 / (kHq / (four ? 4 : 2));  // of a thread block of queries
    const Fp8Append P = {a, a.q ? (a.c.N + tokens - 1) / tokens : 0, four};
    const long long units = kPerToken ? a.c.N : ((long long)a.c.N >> a.c.block_shift) + 2LL * a.c.S;
    return launch_early(append_fp8_kernel<T, kKept, kSplit, kPerToken>, (unsigned)(P.query_blocks + units), kThreads<kSplit>, 0,
                        s, P);
}

// A thread block a token where sequences bring about one each: one row or two then have
// to be read, whatever the size of a block of rows (us, a token and a place: 256 single
// tokens 3.0 and 3.2, 1000 sequences of two 8.3 and 7.5).
template <typename T>
cudaError_t launch_append(const AppendArgs& a, cudaStream_t s) {
    const int shift = a.c.block_shift;
    if (2LL * a.c.N <= 3LL * a.c.S)
        return shift == 3   ? launch_blocks<T, 1, 1, true>(a, s)
               : shift == 4 ? launch_blocks<T, 2, 1, true>(a, s)
                            : launch_blocks<T, 0, 1, true>(a, s);
    switch (shift) {
        case 3: return launch_blocks<T, 1, 1, false>(a, s);
        case 4: return launch_blocks<T, 2, 1, false>(a, s);
        case 5: return launch_blocks<T, 2, 2, false>(a, s);
        case 6: return launch_blocks<T, 2, 4, false>(a, s);
        default: return launch_blocks<T, 0, 4, false>(a, s);
    }
}

}  // namespace

cudaError_t launch_paged_append_fp8(const AppendArgs& a, sfa_dtype dt, cudaStream_t s) {
    return dt == SFA_BF16 ? launch_append<__nv_bfloat16>(a, s) : launch_append<float>(a, s);
}

}  // namespace sfa
