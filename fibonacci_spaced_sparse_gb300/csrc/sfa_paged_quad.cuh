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
#pragma once

#include "sfa_mma.cuh"
#include "sfa_paged.cuh"

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
template <int kN>
__device__ __forceinline__ void scores(const Tile& x, const Pair* U, float (*c)[4]) {
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
__device__ __forceinline__ void raise(Pair& U, float2 x) {
    x = column_max(x);
    const float n0 = x.x > U.th.x ? -x.x : U.nm.x, n1 = x.y > U.th.y ? -x.y : U.nm.y;
    const float2 f = f2(fast_exp2(n0 - U.nm.x), fast_exp2(n1 - U.nm.y));
    U.nm = f2(n0, n1);
    U.th = f2(kLazy - n0, kLazy - n1);
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

// Window tile.  mask: bit 2k (2k + 1) says that row g (g + 8) is in the window
// of this thread's query of pair k.  kFirst: nothing is accumulated yet.
template <bool kFirst, class X>
__device__ __forceinline__ void window_tile(const X& x, unsigned mask, float sl2, Pair (&U)[2]) {
    uint32_t b[2][2];
    const float2 sl = f2(sl2, sl2);
    float c[2][4];
    scores<2>(x, U, c);
    float2 lo[2], hi[2], top[2];
    bool over = false;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        lo[k] = __fmul2_rn(f2(c[k][0], c[k][1]), sl);
        hi[k] = __fmul2_rn(f2(c[k][2], c[k][3]), sl);
        if (!(mask >> (2 * k) & 1u)) lo[k] = f2(-INFINITY, -INFINITY);
        if (!(mask >> (2 * k + 1) & 1u)) hi[k] = f2(-INFINITY, -INFINITY);
        top[k] = f2(fmaxf(lo[k].x, hi[k].x), fmaxf(lo[k].y, hi[k].y));
        if (kFirst) {
            const float2 m = column_max(top[k]);
            U[k].nm = f2(-fmaxf(m.x, kFloor), -fmaxf(m.y, kFloor));
            U[k].th = f2(kLazy - U[k].nm.x, kLazy - U[k].nm.y);
        } else {
            over = over || top[k].x > U[k].th.x || top[k].y > U[k].th.y;
        }
    }
    if (!kFirst && __any_sync(kFull, over)) {
#pragma unroll
        for (int k = 0; k < 2; ++k) raise(U[k], top[k]);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        lo[k] = __fadd2_rn(lo[k], U[k].nm);
        hi[k] = __fadd2_rn(hi[k], U[k].nm);
        lo[k] = f2(fast_exp2(lo[k].x), fast_exp2(lo[k].y));
        hi[k] = f2(fast_exp2(hi[k].x), fast_exp2(hi[k].y));
        U[k].l = kFirst ? __fadd2_rn(lo[k], hi[k]) : __fadd2_rn(U[k].l, __fadd2_rn(lo[k], hi[k]));
        b[k][0] = movm_t(pack_bf16(lo[k].x, lo[k].y));
        b[k][1] = movm_t(pack_bf16(hi[k].x, hi[k].y));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t a[4];
        value_frag(x, j, a);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (kFirst)
                mma16816_z(U[k].o[j], a[0], a[1], a[2], a[3], b[k][0], b[k][1]);
            else
                mma16816(U[k].o[j], a[0], a[1], a[2], a[3], b[k][0], b[k][1]);
        }
    }
}

// Rung tiles of kN pairs.  ok: this thread's rung is an entry of its query; t:
// the rung's fraction.
template <int kN, class X>
__device__ __forceinline__ void rung_tiles(const X* x, const bool* ok, float t, float sl2, Pair* U) {
    float c[kN][1][4];
#pragma unroll
    for (int k = 0; k < kN; ++k) scores<1>(x[k], U + k, c[k]);
    const float u = 1.f - t;
    const float2 tt = f2(t, t), uu = f2(u, u), ts = f2(t * sl2, t * sl2), us = f2(u * sl2, u * sl2);
    float2 s[kN];
    bool over = false;
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        s[k] = __ffma2_rn(ts, f2(c[k][0][0], c[k][0][1]), __fmul2_rn(us, f2(c[k][0][2], c[k][0][3])));
        if (!ok[k]) s[k] = f2(-INFINITY, -INFINITY);
        over = over || s[k].x > U[k].th.x || s[k].y > U[k].th.y;
    }
    if (__any_sync(kFull, over)) {
#pragma unroll
        for (int k = 0; k < kN; ++k) raise(U[k], s[k]);
    }
    uint32_t b[kN][2];
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        s[k] = __fadd2_rn(s[k], U[k].nm);
        const float2 p = f2(fast_exp2(s[k].x), fast_exp2(s[k].y));
        U[k].l = __fadd2_rn(U[k].l, p);
        const float2 far_p = __fmul2_rn(p, tt), near_p = __fmul2_rn(p, uu);
        b[k][0] = movm_t(pack_bf16(far_p.x, far_p.y));
        b[k][1] = movm_t(pack_bf16(near_p.x, near_p.y));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            uint32_t a[4];
            value_frag(x[k], j, a);
            mma16816(U[k].o[j], a[0], a[1], a[2], a[3], b[k][0], b[k][1]);
        }
}

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
// whose results are not finite (they are not written).  kNatural: the sums of
// the scores run over the dimensions in their natural order.  kDeep: four tiles
// of rows in registers instead of two.
template <bool kAlone, bool kNatural, bool kDeep = false>
__device__ __forceinline__ unsigned quad_pass(const PagedFwd& P, const Quad& Q, int only) {
    const int lane = threadIdx.x & 31, g8 = lane >> 2, tig = lane & 3;
    const int W = P.a.W, i0 = Q.i0, last = Q.last;
    const float sl2 = P.a.scale * kLog2e;
    const char* kb = static_cast<const char*>(P.c.k) + Q.g * (kD * 2);
    const char* vb = static_cast<const char*>(P.c.v) + Q.g * (kD * 2);
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
    Pair U[2];
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
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            U[k].qf[j][0] = w[j];
            U[k].qf[j][1] = w[4 + j];
        }
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
    auto load = [&](int r, int half, Tile& x) { load_tile<kAlone, kNatural>(kb, vb, r >= 0 ? r : fill, 16 * half, x); };
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
    unsigned redo = 0;
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
        const bool stores = qq < Q.cnt && (kAlone ? qq == only : !(redo >> qq & 1u));
        const unsigned who_stores = __ballot_sync(kFull, stores);
        if (!stores) continue;
        // l >= 2^-8 (the entry at the maximum, at most the margin below it), or 0 with no entry: zeros
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
    return redo;
}

}  // namespace paged
}  // namespace sfa
