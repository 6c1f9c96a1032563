// sfa_paged_quad.cuh -- the tensor-core arithmetic of the attention over a
// paged cache: four queries of one sequence and one key/value head by a warp.
// Private to the CUDA library.
//
// Quad kernel (bf16, W <= 28): a warp owns four consecutive queries of one
// sequence and one key/value head, as two pairs of 2 queries x 4 heads, and
// forms both products with mma.sync m16n8k16, keys on M:
//   S^T (16 key rows x 8 columns) = K_rows . Q^T,   O^T += V_rows^T . P^T.
// Window: rows i - W .. i + 3 of the quad's first position i are one tile that
// both pairs share, two from W = 13 on.  Rungs: one tile a pair holds four
// rungs, row r < 8 the far row i + e - n - 1 and row r + 8 the near row
// i + e - n of rung r % 4 for query e = r / 4 of the pair, so both rows of an
// interpolation sit in one thread: it mixes their scores (the interpolated
// key's score, by linearity), and splits the probability onto the rows.
// (Tiles of five rows a rung that both pairs share load a third less, but the
// two rows then sit in different threads and every thread computes four
// exponentials for three rungs instead of two for four: 1870 instructions a
// quad instead of 1520, 63 against 56 us for 32 x 1024 tokens.)
//
// Rows come through the block table, so no block of rows is contiguous and no
// tiled copy fits; the fragments are loaded straight into registers instead,
// with no shared memory, no transpose and no barrier.  The dimensions of the
// two products are taken in an order that keeps the loads wide:
//   scores: k-step s of thread (row g, lane t) takes words s and 4 + s of
//     bytes 32 t .. 32 t + 31 of the row, for keys and queries alike;
//   values: the same loads, turned by movmatrix: words 2j and 2j + 1 make
//     product j, whose output rows g and g + 8 are dimensions
//     16 (g / 2) + 4 j + g % 2 and that + 2.
// (Loading a row's chunk g for each of the four rows 2t, 2t + 1, 2t + 8,
// 2t + 9 of the value fragment saves the turn, but eight neighbouring lanes
// then hit two banks: 12 wavefronts a load instead of 4.)
// Neighbouring queries read neighbouring rows, so a row comes from L2 once a
// block and from L1 after that.
//
// Probabilities are rounded to bf16, the type of the value product's operands;
// the sum that divides the result keeps them in fp32, as lse needs it.  A rounding
// is off by 2^-8 of its probability at most, and the errors of some 25 entries
// add up to 1.2e-3 of O's norm, beside the 1.7e-3 of rounding O itself (2.1e-3
// together).  A second product with what the first rounding left would bring that
// back for 8 more MMAs and a second turned operand beside the 16 MMAs of a pair
// of tiles, in a kernel that its instructions bound.
//
// Masked entries get probability 0.  A row that some queries of the quad read
// is multiplied with the others' zeros, and a tile row that none reads is
// filled with the first query's own row; infinity or NaN there would reach
// queries that do not read it.  The epilogue looks for values that are not
// finite and redoes those queries one at a time (kAlone), with that query's
// rows and zeros.  Nothing of a column's arithmetic depends on another column,
// so this gives what the first pass would have given without the others' rows,
// bit for bit.
//
// Rows of 8 bits (RowsFp8) come as 16-byte loads, the same 16 dimensions a
// thread, and are turned into halves, which is exact: both products are f16
// ones.  A query is scaled by a power of two to a largest element in [1, 2), which
// its scores take back with the keys' scales, so its halves hold what its bf16
// values did (but for elements below 2^-14 of the largest, to 2^-25 of it).  A
// value row's scale joins its probability: p s is rounded to a half, 2^-11 where
// bf16 pages lose 2^-8, and the running maximum runs over score + log2(s), so that
// the largest p s lies between 2^kUp and 2^(kUp + kLazy), in a half's range.  The sum
// for lse takes p alone.  What is below 2^-14 is off by up to 2^-25, 2^-32 of the
// largest p s.  A scale says nothing about the row's codes, though: where the row of the
// largest p s holds zeros, the output can be made of such remainders.  With n rows each
// element of O is off by 448 n 2^-25 at most, so a query of which a head's largest
// element is less than 2^13 times that is redone in fp32 arithmetic (one_exact), and the
// others' loss is below 2^-10 of O's norm, whatever the scales are.  (Turning 8 bits into
// bf16 instead takes nine operations for four values where halves take two.)
//
// Long chunks of 8-bit rows are attended over exact bf16 copies (PairSplit).  There
// a probability is the sum of two bf16 parts, p = hi + lo with lo = p - hi rounded,
// which leaves 2^-16 of it, and the value product is made of both: 4 more MMAs a
// tile and pair, so that a long chunk is no less exact than a short one.  A copy holds
// the codes times the power of two in their scale; the factor that is left, in [1, 2),
// joins a key's score and a value's probability in fp32, as the scales of 8-bit rows do
// (kFactors).  With a factor of 1 that changes no bit, so tiles without another skip it.
#pragma once

#include <type_traits>

#include "sfa_fp8.cuh"
#include "sfa_mma.cuh"
#include "sfa_paged.cuh"
#include "sfa_paged_rows.cuh"

namespace sfa {
namespace paged {

using namespace mma;

struct Tile {
    uint32_t k[2][8], v[2][8];  // rows g, g + 8: bytes 32 t .. 32 t + 31
};

// One query pair: the B fragments of Q^T, O^T, and of this thread's two
// columns (query tig / 2 of the pair, heads 2 (tig & 1) and that + 1) minus
// the running maximum (log2 units), the score that raises it, and the sum over
// this thread's rows.
struct Pair {
    uint32_t qf[4][2];
    float o[4][4];
    float2 nm, th, l;
};

// The same with scaled halves; qn: what scales the scores of this thread's columns
// back.
struct PairFp8 : Pair {
    float2 qn;
};

// A pair whose probabilities go into the value product in two parts.
struct PairSplit : Pair {};
template <class P>
constexpr bool kSplit = false;
template <>
constexpr bool kSplit<PairSplit> = true;

// 8-bit rows g, g + 8 (bytes 16 t .. 16 t + 15) and their scales.
struct TileFp8 {
    uint32_t k[2][4], v[2][4];
    float ks[2], vs[2];
};

// Whether a tile's rows have scales.
template <class X>
constexpr bool kScaled = false;
template <>
constexpr bool kScaled<TileFp8> = true;

// Where the running maximum puts the largest probability (times its scale), log2.
template <class X>
constexpr float kUp = kScaled<X> ? 7.f : 0.f;
// log2 of a value row's scale, of a zero one (all of its codes are zero) that of the
// smallest there is.
constexpr float kLeastScale = 7.8886090522101181e-31f;  // 2^-100
__device__ __forceinline__ float log2_scale(float s) { return fast_log2(fmaxf(s, kLeastScale)); }

// The factors of copied rows g, g + 8, and whether a tile has some.
struct Factors {
    float ks[2], vs[2];
};
struct TileCopied : Tile, Factors {};
template <class X>
constexpr bool kFactors = std::is_base_of_v<Factors, X>;

// The factors of a copied row: row_scales holds them.  Where no row was copied it holds
// anything, which here becomes a factor like the others.
__device__ __forceinline__ float factor_of(float x) { return __uint_as_float(__float_as_uint(x) & 0x7fffffu | 0x3f800000u); }
__device__ __forceinline__ void put_factors(const PagedArgs& c, int g, int row, int h, Factors& x) {
    const float4 s = fresh(reinterpret_cast<const float4*>(row_scales(c, row)));
    static_assert(kHkv == 2, "a block's factors are one load");
    x.ks[h] = factor_of(g ? s.y : s.x);
    x.vs[h] = factor_of(g ? s.w : s.z);
}

__device__ __forceinline__ float2 f2(float x, float y) { return make_float2(x, y); }

__device__ __forceinline__ uint32_t word(const uint4& u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; }

__device__ __forceinline__ void load32(const char* p, uint32_t (&w)[8]) {
    asm("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
        : "l"(p));
}

// The same words of a row in the natural order of the dimensions: words s and
// 4 + s are word t of its 16-byte chunks 2s and 2s + 1.
__device__ __forceinline__ void load32_natural(const char* row, int tig, uint32_t (&w)[8]) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        w[s] = fresh(reinterpret_cast<const uint32_t*>(row + 32 * s) + tig);
        w[4 + s] = fresh(reinterpret_cast<const uint32_t*>(row + 32 * s + 16) + tig);
    }
}

// The tile whose 16 row numbers lanes base .. base + 15 hold in `row`; in a
// kAlone pass rows that are not there (-1) are zeros.
template <bool kAlone, bool kNatural>
__device__ __forceinline__ void load_tile(const char* k, const char* v, int row, int base,
                                          Tile& x) {
    constexpr int kStride = kHkv * kD * 2;  // bytes of a page row
    const int lane = threadIdx.x & 31, g8 = lane >> 2, tig = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = __shfl_sync(kFull, row, base + 8 * h + g8);
        if (kAlone) {
#pragma unroll
            for (int w = 0; w < 8; ++w) x.k[h][w] = x.v[h][w] = 0u;
            if (r < 0) continue;
        }
        const size_t at = (size_t)(unsigned)r * kStride;
        if (kNatural)
            load32_natural(k + at, tig, x.k[h]);
        else
            load32(k + at + 32 * tig, x.k[h]);
        load32(v + at + 32 * tig, x.v[h]);
    }
}

// S^T of a tile and kN pairs: c[0], c[1] row g, c[2], c[3] row g + 8.
template <int kN, class P>
__device__ __forceinline__ void scores(const Tile& x, const P* U, float (*c)[4]) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            if (s == 0)
                mma16816_z(c[k], x.k[0][0], x.k[1][0], x.k[0][4], x.k[1][4], U[k].qf[0][0], U[k].qf[0][1]);
            else
                mma16816(c[k], x.k[0][s], x.k[1][s], x.k[0][4 + s], x.k[1][4 + s], U[k].qf[s][0], U[k].qf[s][1]);
        }
}

// The A fragments of V_rows^T, product j: words 2j and 2j + 1 of the rows, each
// an 8 x 8 matrix turned in registers.
__device__ __forceinline__ void value_frag(const Tile& x, int j, uint32_t (&a)[4]) {
    a[0] = movm_t(x.v[0][2 * j]);
    a[1] = movm_t(x.v[0][2 * j + 1]);
    a[2] = movm_t(x.v[1][2 * j]);
    a[3] = movm_t(x.v[1][2 * j + 1]);
}

// The same of 8-bit rows; word r has dimensions 4 r .. 4 r + 3 of the thread's 16.
template <int kN, class P>
__device__ __forceinline__ void scores(const TileFp8& x, const P* U, float (*c)[4]) {
    uint32_t a[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            a[h][2 * r] = fp8::halves(x.k[h][r] & 0xffffu);
            a[h][2 * r + 1] = fp8::halves(x.k[h][r] >> 16);
        }
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            if (s == 0)
                mma16816_f16_z(c[k], a[0][0], a[1][0], a[0][4], a[1][4], U[k].qf[0][0], U[k].qf[0][1]);
            else
                mma16816_f16(c[k], a[0][s], a[1][s], a[0][4 + s], a[1][4 + s], U[k].qf[s][0], U[k].qf[s][1]);
        }
}
__device__ __forceinline__ void value_frag(const TileFp8& x, int j, uint32_t (&a)[4]) {
    a[0] = movm_t(fp8::halves(x.v[0][j] & 0xffffu));
    a[1] = movm_t(fp8::halves(x.v[0][j] >> 16));
    a[2] = movm_t(fp8::halves(x.v[1][j] & 0xffffu));
    a[3] = movm_t(fp8::halves(x.v[1][j] >> 16));
}

// The value product of a tile and one pair, with the operands' type.
template <class X>
__device__ __forceinline__ void value_mma(float (&o)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    if constexpr (kScaled<X>)
        mma16816_f16(o, a[0], a[1], a[2], a[3], b[0], b[1]);
    else
        mma16816(o, a[0], a[1], a[2], a[3], b[0], b[1]);
}
template <class X>
__device__ __forceinline__ void value_mma_z(float (&o)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    if constexpr (kScaled<X>)
        mma16816_f16_z(o, a[0], a[1], a[2], a[3], b[0], b[1]);
    else
        mma16816_z(o, a[0], a[1], a[2], a[3], b[0], b[1]);
}

// Largest of a column over the eight threads that hold it.
__device__ __forceinline__ float2 column_max(float2 x) {
#pragma unroll
    for (int w = 4; w <= 16; w <<= 1) {
        x.x = fmaxf(x.x, __shfl_xor_sync(kFull, x.x, w));
        x.y = fmaxf(x.y, __shfl_xor_sync(kFull, x.y, w));
    }
    return x;
}

// Raise the running maximum of each column whose largest x passes the margin,
// and rescale it.
template <class X>
__device__ __forceinline__ void raise(Pair& U, float2 x) {
    x = column_max(x);
    if constexpr (kScaled<X>) {
        x.x = x.x > U.th.x ? x.x - kUp<X> : -U.nm.x;
        x.y = x.y > U.th.y ? x.y - kUp<X> : -U.nm.y;
    }
    const float n0 = kScaled<X> || x.x > U.th.x ? -x.x : U.nm.x, n1 = kScaled<X> || x.y > U.th.y ? -x.y : U.nm.y;
    const float2 f = f2(fast_exp2(n0 - U.nm.x), fast_exp2(n1 - U.nm.y));
    U.nm = f2(n0, n1);
    U.th = f2(kLazy + kUp<X> - n0, kLazy + kUp<X> - n1);
    U.l = __fmul2_rn(U.l, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 a = __fmul2_rn(f2(U.o[j][0], U.o[j][1]), f), b = __fmul2_rn(f2(U.o[j][2], U.o[j][3]), f);
        U.o[j][0] = a.x;
        U.o[j][1] = a.y;
        U.o[j][2] = b.x;
        U.o[j][3] = b.y;
    }
}

// What rounding x and y to the two bf16 of w left.
__device__ __forceinline__ uint32_t rest_of(uint32_t w, float x, float y) {
    const float2 h = unpack_bf16(w);
    return pack_bf16(x - h.x, y - h.y);
}

// Window tile.  mask: bit 2k (2k + 1) says that row g (g + 8) is in the window
// of this thread's query of pair k.  kFirst: nothing is accumulated yet.
template <bool kFirst, class X, class P>
__device__ __forceinline__ void window_tile(const X& x, unsigned mask, float sl2, P (&U)[2]) {
    uint32_t b[2][2], rest[2][2];
    const float2 sl = f2(sl2, sl2);
    float c[2][4];
    scores<2>(x, U, c);
    float2 lo[2], hi[2], top[2];
    bool over = false;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if constexpr (kScaled<X>) {
            const float s0 = sl2 * x.ks[0], s1 = sl2 * x.ks[1];
            lo[k] = __fmul2_rn(f2(c[k][0], c[k][1]), __fmul2_rn(U[k].qn, f2(s0, s0)));
            hi[k] = __fmul2_rn(f2(c[k][2], c[k][3]), __fmul2_rn(U[k].qn, f2(s1, s1)));
        } else if constexpr (kFactors<X>) {
            const float s0 = sl2 * x.ks[0], s1 = sl2 * x.ks[1];
            lo[k] = __fmul2_rn(f2(c[k][0], c[k][1]), f2(s0, s0));
            hi[k] = __fmul2_rn(f2(c[k][2], c[k][3]), f2(s1, s1));
        } else {
            lo[k] = __fmul2_rn(f2(c[k][0], c[k][1]), sl);
            hi[k] = __fmul2_rn(f2(c[k][2], c[k][3]), sl);
        }
        if (!(mask >> (2 * k) & 1u)) lo[k] = f2(-INFINITY, -INFINITY);
        if (!(mask >> (2 * k + 1) & 1u)) hi[k] = f2(-INFINITY, -INFINITY);
        if constexpr (kScaled<X>) {
            const float l0 = log2_scale(x.vs[0]), l1 = log2_scale(x.vs[1]);
            top[k] = f2(fmaxf(lo[k].x + l0, hi[k].x + l1), fmaxf(lo[k].y + l0, hi[k].y + l1));
        } else {
            top[k] = f2(fmaxf(lo[k].x, hi[k].x), fmaxf(lo[k].y, hi[k].y));
        }
        if (kFirst) {
            const float2 m = column_max(top[k]);
            U[k].nm = f2(kUp<X> - fmaxf(m.x, kFloor), kUp<X> - fmaxf(m.y, kFloor));
            U[k].th = f2(kLazy + kUp<X> - U[k].nm.x, kLazy + kUp<X> - U[k].nm.y);
        } else {
            over = over || top[k].x > U[k].th.x || top[k].y > U[k].th.y;
        }
    }
    if (!kFirst && __any_sync(kFull, over)) {
#pragma unroll
        for (int k = 0; k < 2; ++k) raise<X>(U[k], top[k]);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        lo[k] = __fadd2_rn(lo[k], U[k].nm);
        hi[k] = __fadd2_rn(hi[k], U[k].nm);
        lo[k] = f2(fast_exp2(lo[k].x), fast_exp2(lo[k].y));
        hi[k] = f2(fast_exp2(hi[k].x), fast_exp2(hi[k].y));
        U[k].l = kFirst ? __fadd2_rn(lo[k], hi[k]) : __fadd2_rn(U[k].l, __fadd2_rn(lo[k], hi[k]));
        if constexpr (kScaled<X>) {
            b[k][0] = movm_t(pack_f16(lo[k].x * x.vs[0], lo[k].y * x.vs[0]));
            b[k][1] = movm_t(pack_f16(hi[k].x * x.vs[1], hi[k].y * x.vs[1]));
        } else {
            if constexpr (kFactors<X>) {
                lo[k] = __fmul2_rn(lo[k], f2(x.vs[0], x.vs[0]));
                hi[k] = __fmul2_rn(hi[k], f2(x.vs[1], x.vs[1]));
            }
            b[k][0] = pack_bf16(lo[k].x, lo[k].y);
            b[k][1] = pack_bf16(hi[k].x, hi[k].y);
            if constexpr (kSplit<P>) {
                rest[k][0] = movm_t(rest_of(b[k][0], lo[k].x, lo[k].y));
                rest[k][1] = movm_t(rest_of(b[k][1], hi[k].x, hi[k].y));
            }
            b[k][0] = movm_t(b[k][0]);
            b[k][1] = movm_t(b[k][1]);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t a[4];
        value_frag(x, j, a);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (kFirst)
                value_mma_z<X>(U[k].o[j], a, b[k]);
            else
                value_mma<X>(U[k].o[j], a, b[k]);
            if constexpr (kSplit<P>) value_mma<X>(U[k].o[j], a, rest[k]);
        }
    }
}

// Rung tiles of kN pairs.  ok: this thread's rung is an entry of its query; t:
// the rung's fraction.
template <int kN, class X, class P>
__device__ __forceinline__ void rung_tiles(const X* x, const bool* ok, float t, float sl2, P* U) {
    float c[kN][1][4];
#pragma unroll
    for (int k = 0; k < kN; ++k) scores<1>(x[k], U + k, c[k]);
    const float u = 1.f - t;
    const float2 tt = f2(t, t), uu = f2(u, u), ts = f2(t * sl2, t * sl2), us = f2(u * sl2, u * sl2);
    float2 s[kN], top[kN];
    bool over = false;
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        if constexpr (kScaled<X>) {
            const float fs = t * sl2 * x[k].ks[0], ns = u * sl2 * x[k].ks[1];
            s[k] = __fmul2_rn(__ffma2_rn(f2(fs, fs), f2(c[k][0][0], c[k][0][1]), __fmul2_rn(f2(ns, ns), f2(c[k][0][2], c[k][0][3]))),
                              U[k].qn);
        } else if constexpr (kFactors<X>) {
            const float fs = t * sl2 * x[k].ks[0], ns = u * sl2 * x[k].ks[1];
            s[k] = __ffma2_rn(f2(fs, fs), f2(c[k][0][0], c[k][0][1]), __fmul2_rn(f2(ns, ns), f2(c[k][0][2], c[k][0][3])));
        } else {
            s[k] = __ffma2_rn(ts, f2(c[k][0][0], c[k][0][1]), __fmul2_rn(us, f2(c[k][0][2], c[k][0][3])));
        }
        if (!ok[k]) s[k] = f2(-INFINITY, -INFINITY);
        top[k] = s[k];
        if constexpr (kScaled<X>) {
            const float l = log2_scale(fmaxf(t * x[k].vs[0], u * x[k].vs[1]));
            top[k] = f2(s[k].x + l, s[k].y + l);
        }
        over = over || top[k].x > U[k].th.x || top[k].y > U[k].th.y;
    }
    if (__any_sync(kFull, over)) {
#pragma unroll
        for (int k = 0; k < kN; ++k) raise<X>(U[k], top[k]);
    }
    uint32_t b[kN][2], rest[kN][2];
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        s[k] = __fadd2_rn(s[k], U[k].nm);
        const float2 p = f2(fast_exp2(s[k].x), fast_exp2(s[k].y));
        U[k].l = __fadd2_rn(U[k].l, p);
        if constexpr (kScaled<X>) {
            const float fv = t * x[k].vs[0], nv = u * x[k].vs[1];
            b[k][0] = movm_t(pack_f16(p.x * fv, p.y * fv));
            b[k][1] = movm_t(pack_f16(p.x * nv, p.y * nv));
        } else {
            float2 far_p, near_p;
            if constexpr (kFactors<X>) {
                const float fv = t * x[k].vs[0], nv = u * x[k].vs[1];
                far_p = __fmul2_rn(p, f2(fv, fv));
                near_p = __fmul2_rn(p, f2(nv, nv));
            } else {
                far_p = __fmul2_rn(p, tt);
                near_p = __fmul2_rn(p, uu);
            }
            b[k][0] = pack_bf16(far_p.x, far_p.y);
            b[k][1] = pack_bf16(near_p.x, near_p.y);
            if constexpr (kSplit<P>) {
                rest[k][0] = movm_t(rest_of(b[k][0], far_p.x, far_p.y));
                rest[k][1] = movm_t(rest_of(b[k][1], near_p.x, near_p.y));
            }
            b[k][0] = movm_t(b[k][0]);
            b[k][1] = movm_t(b[k][1]);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            uint32_t a[4];
            value_frag(x[k], j, a);
            value_mma<X>(U[k].o[j], a, b[k]);
            if constexpr (kSplit<P>) value_mma<X>(U[k].o[j], a, rest[k]);
        }
}

// The formats of the pages' rows: how a tile is loaded and what becomes of a query.
struct RowsBf16 {
    using Tile = paged::Tile;
    using Pair = paged::Pair;
    static constexpr int kBytes = 2;  // of an element
    static constexpr bool kCopied = false;
    template <bool kAlone, bool kNatural>
    static __device__ __forceinline__ void load(const PagedArgs&, int, const char* k, const char* v, int row, int base, Tile& x) {
        load_tile<kAlone, kNatural>(k, v, row, base, x);
    }
    static __device__ __forceinline__ void query(const uint32_t (&w)[8], Pair& U) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            U.qf[j][0] = w[j];
            U.qf[j][1] = w[4 + j];
        }
    }
};

// bf16 copies of 8-bit rows.
struct RowsCopied : RowsBf16 {
    using Tile = TileCopied;
    using Pair = PairSplit;
    static constexpr bool kCopied = true;
    template <bool kAlone, bool kNatural>
    static __device__ __forceinline__ void load(const PagedArgs& c, int g, const char* k, const char* v, int row, int base,
                                                Tile& x) {
        load_tile<kAlone, kNatural>(k, v, row, base, x);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = __shfl_sync(kFull, row, base + 8 * h + ((threadIdx.x & 31) >> 2));
            put_factors(c, g, max(r, 0), h, x);
        }
    }
};

struct RowsFp8 {
    using Tile = TileFp8;
    using Pair = PairFp8;
    static constexpr int kBytes = 1;
    template <bool kAlone, bool kNatural>
    static __device__ __forceinline__ void load(const PagedArgs& c, int g, const char* k, const char* v, int row, int base,
                                                Tile& x) {
        const int lane = threadIdx.x & 31, g8 = lane >> 2, tig = lane & 3;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = __shfl_sync(kFull, row, base + 8 * h + g8);
            if (kAlone) {
#pragma unroll
                for (int w = 0; w < 4; ++w) x.k[h][w] = x.v[h][w] = 0u;
                x.ks[h] = x.vs[h] = 0.f;
                if (r < 0) continue;
            }
            const size_t at = (size_t)(unsigned)r * (kHkv * kD) + 16 * tig;
            const uint4 a = fresh(reinterpret_cast<const uint4*>(k + at)), b = fresh(reinterpret_cast<const uint4*>(v + at));
            const float4 s = fresh(reinterpret_cast<const float4*>(row_scales(c, r)));
            static_assert(kHkv == 2, "a block's scales are one load");
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                x.k[h][w] = word(a, w);
                x.v[h][w] = word(b, w);
            }
            x.ks[h] = g ? s.y : s.x;
            x.vs[h] = g ? s.w : s.z;
        }
    }
    // The row's halves, its largest element in [1, 2) (an infinite one stays so).
    static __device__ __forceinline__ void query(const uint32_t (&w)[8], Pair& U) {
        const int tig = threadIdx.x & 3;
        float2 v[8];
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = unpack_bf16(w[j]);
            top = fmaxf(top, fmaxf(fabsf(v[j].x), fabsf(v[j].y)));
        }
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
        const int e = min(max(__float_as_int(top) >> 23, 1), 253);
        const float f = __int_as_float((254 - e) << 23), back = __int_as_float(e << 23);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            U.qf[j][0] = pack_f16(v[j].x * f, v[j].y * f);
            U.qf[j][1] = pack_f16(v[4 + j].x * f, v[4 + j].y * f);
        }
        // column n is lane 4 n's; this thread's scores are of columns 2 tig and 2 tig + 1
        U.qn = f2(__shfl_sync(kFull, back, 8 * tig), __shfl_sync(kFull, back, 8 * tig + 4));
    }
};

struct Quad {
    int s, t0, cnt, i0, last, g;
    const int *rn, *rc;
    const float* rt;
};

// A rung tile's entry as a thread sees it: the fraction, and for its query of
// each pair whether the rung is an entry of it.
struct Entry {
    float frac;
    bool ok[2];
};

// All queries of the quad, or the query `only` alone; returns the queries
// whose results are not finite (bits 0 .. 3; not when alone) or too small for halves (bits
// 4 .. 7); they are not written.  kNatural: the sums of
// the scores run over the dimensions in their natural order.  kDeep: four tiles
// of rows in registers instead of two.
template <bool kAlone, bool kNatural, bool kDeep = false, class F = RowsBf16>
__device__ __forceinline__ unsigned quad_pass(const PagedFwd& P, const Quad& Q, int only) {
    const int lane = threadIdx.x & 31, g8 = lane >> 2, tig = lane & 3;
    const int W = P.a.W, i0 = Q.i0, last = Q.last;
    const float sl2 = P.a.scale * kLog2e;
    const char* kb = static_cast<const char*>(P.c.k) + Q.g * (kD * F::kBytes);
    const char* vb = static_cast<const char*>(P.c.v) + Q.g * (kD * F::kBytes);
    // this lane's row of the window: position i0 - W + lane
    bool want = lane < W + 4 && i0 - W + lane >= 0 && i0 - W + lane <= last && (!kAlone || (lane >= only && lane <= only + W));
    const int wrow = paged::page_row_if(P.c, Q.s, i0 - W + lane, want);
    bool bad = want && wrow < 0;
    // rungs that the last query uses: a prefix, four to a tile
    const int nt = (__popc(__ballot_sync(kFull, Q.rc[lane] <= last)) + 3) >> 2;
    // this lane's row of a rung tile: lanes 0-15 the first pair's, 16-31 the second's
    const int my_q = 2 * (lane >> 4) + ((lane >> 2) & 1);
    const bool near_row = lane & 8;
    auto rung_rows = [&](int t) {
        const int r = 4 * t + (lane & 3), i = i0 + my_q;
        const bool w = i <= last && i >= Q.rc[r] && (near_row || Q.rt[r] > 0.f) && (!kAlone || my_q == only);
        const int row = paged::page_row_if(P.c, Q.s, i - Q.rn[r] - (near_row ? 0 : 1), w);
        bad |= w && row < 0;
        return row;
    };
    int row = nt > 0 ? rung_rows(0) : -1, next = kDeep && nt > 1 ? rung_rows(1) : -1;
    const int fill = kAlone ? -1 : max(__shfl_sync(kFull, wrow, W), 0);  // the first query's own row
    using Tile = typename F::Tile;
    typename F::Pair U[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int qt = Q.t0 + min(2 * k + (g8 >> 2), Q.cnt - 1);
        const char* qp = reinterpret_cast<const char*>(static_cast<const __nv_bfloat16*>(P.q) + (size_t)qt * P.qs +
                                                       (Q.g * kG + (g8 & 3)) * kD);
        uint32_t w[8];
        if (kNatural) {
            load32_natural(qp, tig, w);
        } else {
            const uint4 a = fresh(reinterpret_cast<const uint4*>(qp) + 2 * tig);
            const uint4 b = fresh(reinterpret_cast<const uint4*>(qp) + 2 * tig + 1);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[j] = word(a, j);
                w[4 + j] = word(b, j);
            }
        }
        F::query(w, U[k]);
    }
    // window rows of this thread's queries
    unsigned mask[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int R = 16 * (e >> 2) + 8 * (e & 1) + g8, d = R - 2 * ((e >> 1) & 1) - (tig >> 1);
        if (d >= 0 && d <= W && R >= W - i0) mask[e >> 2] |= 1u << (e & 3);
    }
    if (__any_sync(kFull, bad)) {
        const unsigned w = __ballot_sync(kFull, wrow >= 0);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (!(w >> (16 * (e >> 2) + 8 * (e & 1) + g8) & 1u)) mask[e >> 2] &= ~(1u << (e & 3));
    }
    const int my_i = (g8 >> 2) == (tig >> 1) ? i0 + (tig >> 1) : -(1 << 30);  // its own rung's query, or none
    auto load = [&](int r, int half, Tile& x) {
        F::template load<kAlone, kNatural>(P.c, Q.g, kb, vb, r >= 0 ? r : fill, 16 * half, x);
    };
    // of rung tile t with the rows r
    auto entry_of = [&](int t, int r) {
        Entry y;
        y.frac = Q.rt[4 * t + (g8 & 3)];
        const int c = Q.rc[4 * t + (g8 & 3)];
        y.ok[0] = my_i >= c;
        y.ok[1] = my_i + 2 >= c;
        if (__any_sync(kFull, bad)) {
            const unsigned there = __ballot_sync(kFull, r >= 0);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                y.ok[k] = y.ok[k] && (there >> (16 * k + 8 + g8) & 1u) && ((there >> (16 * k + g8) & 1u) || y.frac == 0.f);
        }
        return y;
    };
    if constexpr (kDeep) {
        // both pairs' tiles of four rungs are loaded while those before are used
        Tile A[2], B[2];
        auto use = [&](const Tile(&x)[2], int t, int r) {
            const Entry y = entry_of(t, r);
            rung_tiles<2>(x, y.ok, y.frac, sl2, U);
        };
        load(wrow, 0, B[0]);
        if (W > 12) load(wrow, 1, B[1]);
        if (nt > 0) load(row, 0, A[0]), load(row, 1, A[1]);
        window_tile<true>(B[0], mask[0], sl2, U);
        if (W > 12) window_tile<false>(B[1], mask[1], sl2, U);
        for (int t = 0; t < nt; t += 2) {
            if (t + 1 < nt) load(next, 0, B[0]), load(next, 1, B[1]);
            const int after = t + 2 < nt ? rung_rows(t + 2) : -1;
            use(A, t, row);
            if (t + 1 >= nt) break;
            if (t + 2 < nt) load(after, 0, A[0]), load(after, 1, A[1]);
            row = after;
            const int r = next;
            next = t + 3 < nt ? rung_rows(t + 3) : -1;
            use(B, t + 1, r);
        }
    } else {
        // two tiles in turn: one is loaded while the other is used
        Tile A, B;
        load(wrow, 0, A);
        if (W > 12) {
            load(wrow, 1, B);
            window_tile<true>(A, mask[0], sl2, U);
            if (nt > 0) load(row, 0, A);
            window_tile<false>(B, mask[1], sl2, U);
        } else {
            if (nt > 0) load(row, 0, B);
            window_tile<true>(A, mask[0], sl2, U);
            A = B;
        }
        for (int t = 0; t < nt; ++t) {
            load(row, 1, B);
            const Entry y = entry_of(t, row);
            row = t + 1 < nt ? rung_rows(t + 1) : -1;
            rung_tiles<1>(&A, y.ok, y.frac, sl2, U);
            if (t + 1 < nt) load(row, 0, A);
            rung_tiles<1>(&B, y.ok + 1, y.frac, sl2, U + 1);
        }
    }
    if (__any_sync(kFull, bad) && lane == 0) paged::report(P.c.status);
    unsigned redo = 0, small = 0;
    const float least = (float)(W + 1 + 2 * P.a.nr) * (448.f * 8192.f / 33554432.f);  // 2^13 448 n 2^-25
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float2 l = U[k].l;
#pragma unroll
        for (int w = 4; w <= 16; w <<= 1)
            l = __fadd2_rn(l, f2(__shfl_xor_sync(kFull, l.x, w), __shfl_xor_sync(kFull, l.y, w)));
        const int qq = 2 * k + (tig >> 1);
        const bool in = i0 + qq >= 0 && i0 + qq < P.c.cap;
        if (!kAlone) {
            float2 odd = f2(0.f, 0.f);  // stays 0 while every value is finite
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                odd = __ffma2_rn(f2(U[k].o[j][0], U[k].o[j][1]), f2(0.f, 0.f), odd);
                odd = __ffma2_rn(f2(U[k].o[j][2], U[k].o[j][3]), f2(0.f, 0.f), odd);
            }
            // lanes with tig < 2 hold the pair's first query
            const unsigned who = __ballot_sync(kFull, odd.x + odd.y != 0.f && qq < Q.cnt && in);
            redo |= ((who & 0x33333333u ? 1u : 0u) | (who & 0xccccccccu ? 2u : 0u)) << (2 * k);
        }
        if constexpr (kScaled<Tile>) {
            float2 top = f2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                top = f2(fmaxf(top.x, fmaxf(fabsf(U[k].o[j][0]), fabsf(U[k].o[j][2]))),
                         fmaxf(top.y, fmaxf(fabsf(U[k].o[j][1]), fabsf(U[k].o[j][3]))));
            // columns 2 tig and 2 tig + 1 are the eight lanes' with this tig
            unsigned a = __ballot_sync(kFull, top.x >= least), b = __ballot_sync(kFull, top.y >= least);
            a |= a >> 16, b |= b >> 16;
            a |= a >> 8, b |= b >> 8;
            a |= a >> 4, b |= b >> 4;
            a = ~(a & b);
            const unsigned who = __ballot_sync(kFull, (a >> tig & 1u) && qq < Q.cnt && in && (!kAlone || qq == only));
            small |= ((who & 0x33333333u ? 1u : 0u) | (who & 0xccccccccu ? 2u : 0u)) << (2 * k);
            small &= ~redo;
        }
        const bool stores = qq < Q.cnt && (kAlone ? qq == only : !(redo >> qq & 1u)) && !(small >> qq & 1u);
        const unsigned who_stores = __ballot_sync(kFull, stores);
        if (!stores) continue;
        // l >= 2^-8 (the entry at the maximum, at most the margin below it; with 8-bit rows that
        // over the largest scale), or 0 with no entry: zeros
        const float2 f = f2(in && l.x != 0.f ? fast_rcp(l.x) : 0.f, in && l.y != 0.f ? fast_rcp(l.y) : 0.f);
        const size_t at = (size_t)(Q.t0 + qq) * kHq + Q.g * kG + 2 * (tig & 1);
        // dimensions 16 (g8 / 2) + g8 % 2 + 2 d, d = 0 .. 7, of both columns; lane ^ 4 has
        // the others: the even one of the two takes the first eight, the odd one the last
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 a = __fmul2_rn(f2(U[k].o[j][0], U[k].o[j][1]), f), b = __fmul2_rn(f2(U[k].o[j][2], U[k].o[j][3]), f);
            w[2 * j] = in ? pack_bf16(a.x, a.y) : 0u;  // (a sum that is not finite would survive f = 0)
            w[2 * j + 1] = in ? pack_bf16(b.x, b.y) : 0u;
        }
        const bool odd_row = g8 & 1;
        uint32_t w0[4], w1[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const uint32_t mine = odd_row ? w[4 + d] : w[d];
            const uint32_t got = __shfl_xor_sync(who_stores, odd_row ? w[d] : w[4 + d], 4);
            const uint32_t even = odd_row ? got : mine, odd = odd_row ? mine : got;
            w0[d] = __byte_perm(even, odd, 0x5410);
            w1[d] = __byte_perm(even, odd, 0x7632);
        }
        uint4* o = static_cast<uint4*>(P.o) + at * (kD / 8) + g8;
        o[0] = make_uint4(w0[0], w0[1], w0[2], w0[3]);
        o[kD / 8] = make_uint4(w1[0], w1[1], w1[2], w1[3]);
        if (P.lse && g8 == 0) {
            const float y0 = l.x != 0.f ? (__log2f(l.x) - U[k].nm.x) * kLn2 : -INFINITY;
            const float y1 = l.y != 0.f ? (__log2f(l.y) - U[k].nm.y) * kLn2 : -INFINITY;
            *reinterpret_cast<float2*>(P.lse + at) = in ? f2(y0, y1) : f2(0.f, 0.f);
        }
    }
    return redo | small << 4;
}

// ----------------------------------------------------------------- the kernel

// kBlocks a SM: two tiles of rows on their way or in use, at 168 registers (3, 12
// warps a SM), or four at 242 (2, 8 warps), where that keeps every warp resident
// (us, two and four: one chunk of 512 tokens 4.4 and 4.2, of 2048 7.0 and 5.6; of
// 3100 6.8 and 9.3, 512 chunks of 2 5.7 and 8.2, 1000 of 16 43 and 49).  A tile of
// 8-bit rows has half the words, so that two fit 128 registers as well (4, 16
// warps), which pays where 12 warps a SM do not hold all (us, 3 and 4: 64 chunks of
// up to 100 tokens, one wave of 3, 8.2 and 9.9; 1000 of 4 behind up to 1000 rows 14.4
// and 14.6, 32 of 1024 58.8 and 55.0).
constexpr int kQuadWarps = 4;
constexpr long long quad_wave(int blocks) { return kSms * (long long)blocks * kQuadWarps / kHkv; }  // slots at once

// A call of its own, so that the rare pass takes no registers of the common one
// (and one for each kernel: they differ in their registers).
template <class F, int kBlocks>
__device__ __noinline__ unsigned one_alone(const PagedFwd& P, const Quad& Q, int only) {
    return quad_pass<true, false, false, F>(P, Q, only);
}

// The query `only` in fp32 arithmetic (sfa_paged_rows.cuh), by one warp.
template <int kBlocks>
__device__ __noinline__ void one_exact(const PagedFwd& P, const Quad& Q, int only) {
    const int lane = threadIdx.x & 31, t = Q.t0 + only;
    Chunk<__nv_bfloat16> raw[kG];
#pragma unroll
    for (int h = 0; h < kG; ++h)
        load(static_cast<const __nv_bfloat16*>(P.q) + (size_t)t * P.qs + (Q.g * kG + h) * kD + 8 * (lane & 7), raw[h]);
    const Partial y = query_part<__nv_bfloat16, __nv_fp8_e4m3, false>(P, Q.s, Q.i0 + only, Q.g, raw, 0, 4);
    write_part<__nv_bfloat16>(P, t, Q.g, lane >> 3, lane & 7, y);
}

template <class F, int kBlocks>
__global__ void __launch_bounds__(kQuadWarps * 32, kBlocks) quad_kernel(const __grid_constant__ PagedFwd P) {
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
    unsigned redo = quad_pass<false, false, kBlocks == 2, F>(P, Q, -1);
    if constexpr (kScaled<typename F::Tile>) {
        unsigned small = redo >> 4;
        for (redo &= 15u; redo; redo &= redo - 1) small |= one_alone<F, kBlocks>(P, Q, __ffs(redo) - 1) >> 4;
        for (; small; small &= small - 1) one_exact<kBlocks>(P, Q, __ffs(small) - 1);
    } else {
        for (; redo; redo &= redo - 1) one_alone<F, kBlocks>(P, Q, __ffs(redo) - 1);
    }
}

// Slots of four queries at most (quad_kernel has their places).
inline long long quad_slots(const PagedArgs& c) { return (long long)c.N / 4 + c.S; }

template <class F>
cudaError_t launch_quads(const PagedFwd& P, cudaStream_t s) {
    const long long slots = quad_slots(P.c);
    void (*kernel)(PagedFwd) = slots <= quad_wave(2) ? quad_kernel<F, 2> : quad_kernel<F, 3>;
    if constexpr (F::kBytes == 1) {
        if (slots > quad_wave(3)) kernel = quad_kernel<F, 4>;
    }
    return launch_early(kernel, (unsigned)((slots + kQuadWarps - 1) / kQuadWarps * kHkv), kQuadWarps * 32, 0, s, P);
}

}  // namespace paged
}  // namespace sfa
