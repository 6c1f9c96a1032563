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

namespace sfa {

namespace {

using namespace mma;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.0f;      // raise a running maximum past this margin
constexpr float kFloor = -1e30f;   // running maximum before the first entry

struct PagedFwd {
    LayerArgs a;
    PagedArgs c;
    const void* q;
    long long qs;
    void* o;
    float* lse;
};

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
    x.u = __ldg(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ void load(const float* p, Chunk<float>& x) {
    x.u = __ldg(reinterpret_cast<const float4*>(p));
    x.v = __ldg(reinterpret_cast<const float4*>(p) + 1);
}
__device__ __forceinline__ void open(const Chunk<__nv_bfloat16>& x, float (&f)[8]) {
    const uint32_t w[4] = {x.u.x, x.u.y, x.u.z, x.u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}
__device__ __forceinline__ void open(const Chunk<float>& x, float (&f)[8]) {
    f[0] = x.u.x, f[1] = x.u.y, f[2] = x.u.z, f[3] = x.u.w;
    f[4] = x.v.x, f[5] = x.v.y, f[6] = x.v.z, f[7] = x.v.w;
}
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

template <typename T>
__device__ Partial query_part(const PagedFwd& P, int s, int pos, int g, const T* qrow, int first, int step) {
    const int lane = threadIdx.x & 31, slot = lane >> 3, ch = lane & 7;
    float q[kG][8];
#pragma unroll
    for (int h = 0; h < kG; ++h) {
        Chunk<T> x;
        load(qrow + h * kD + 8 * ch, x);
        open(x, q[h]);
#pragma unroll
        for (int j = 0; j < 8; ++j) q[h][j] *= P.a.scale * kLog2e;
    }
    const int nwin = min(P.a.W, pos) + 1;
    int nrung = 0;
    for (int r = 0; r < P.a.nr; ++r) nrung += P.a.r[r].c <= pos ? 1 : 0;  // sorted: a prefix
    const int n = nwin + nrung;
    const T* kb = static_cast<const T*>(P.c.k) + g * kD + 8 * ch;
    const T* vb = static_cast<const T*>(P.c.v) + g * kD + 8 * ch;
    float acc[kG][8];
#pragma unroll
    for (int h = 0; h < kG; ++h)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[h][j] = 0.f;
    float m = kFloor, l = 0.f;  // of head (lane >> 1) & 3, this slot's entries
    bool bad = false;
    for (int e0 = first; e0 < n; e0 += step) {
        const int e = e0 + slot;
        int ra = -1, rb = -1;
        float wa = 1.f, wb = 0.f;
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
                wa = 1.f - R.t;
                wb = R.t;
            }
        }
        float k[8], v[8];
        {
            Chunk<T> ka{}, va{}, kc{}, vc{};
            if (ra >= 0) {
                load(kb + (size_t)ra * (kHkv * kD), ka);
                load(vb + (size_t)ra * (kHkv * kD), va);
                if (rb >= 0) {
                    load(kb + (size_t)rb * (kHkv * kD), kc);
                    load(vb + (size_t)rb * (kHkv * kD), vc);
                }
            }
            open(ka, k);
            open(va, v);
            if (rb >= 0 && ra >= 0) {
                float x[8], y[8];
                open(kc, x);
                open(vc, y);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    k[j] = wa * k[j] + wb * x[j];
                    v[j] = wa * v[j] + wb * y[j];
                }
            }
        }
        float d[kG];
#pragma unroll
        for (int h = 0; h < kG; ++h) {
            d[h] = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) d[h] = fmaf(q[h][j], k[j], d[h]);
        }
        // sum over the slot's eight lanes; head h ends in lanes 2h, 2h + 1
        const bool up4 = lane & 4, up2 = lane & 2;
        float d0 = (up4 ? d[2] : d[0]) + __shfl_xor_sync(kFull, up4 ? d[0] : d[2], 4);
        float d1 = (up4 ? d[3] : d[1]) + __shfl_xor_sync(kFull, up4 ? d[1] : d[3], 4);
        float x = (up2 ? d1 : d0) + __shfl_xor_sync(kFull, up2 ? d0 : d1, 2);
        x += __shfl_xor_sync(kFull, x, 1);
        if (ra < 0) x = -INFINITY;
        if (__any_sync(kFull, x > m + kLazy)) {
            const float up = fmaxf(m, x);
            const float f = exp2f(m - up);
            m = up;
            l *= f;
#pragma unroll
            for (int h = 0; h < kG; ++h) {
                const float fh = __shfl_sync(kFull, f, (lane & 24) + 2 * h);
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[h][j] *= fh;
            }
        }
        const float p = exp2f(x - m);
        l += p;
#pragma unroll
        for (int h = 0; h < kG; ++h) {
            const float ph = __shfl_sync(kFull, p, (lane & 24) + 2 * h);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[h][j] = fmaf(ph, v[j], acc[h][j]);
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
        for (int j = 0; j < 8; ++j) acc[h][j] *= fh;
    }
    const bool up16 = lane & 16, up8 = lane & 8;
    Partial out;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float a0 = (up16 ? acc[2][j] : acc[0][j]) + __shfl_xor_sync(kFull, up16 ? acc[0][j] : acc[2][j], 16);
        const float a1 = (up16 ? acc[3][j] : acc[1][j]) + __shfl_xor_sync(kFull, up16 ? acc[1][j] : acc[3][j], 16);
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

template <typename T, int kNW>
__global__ void __launch_bounds__(256) rows_kernel(const __grid_constant__ PagedFwd P) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int kUnits = 8 / kNW;  // (token, head) of a block
    __shared__ float part[kNW > 1 ? kNW : 1][kNW > 1 ? kG * kD : 1];
    __shared__ float top[kNW][kG], sum[kNW][kG];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned unit = blockIdx.x * kUnits + warp / kNW;
    const int t = (int)(unit / kHkv), g = (int)(unit % kHkv);
    if (t >= P.c.N) return;  // with kNW > 1 the whole block
    const int s = paged::sequence_of(P.c, t);
    if (s >= P.c.S) return;
    const int pos = __ldg(P.c.lens + s) - (__ldg(P.c.cu + s + 1) - t);
    if (pos < 0 || pos >= P.c.cap) {
        if (threadIdx.x % (32 * kNW) == 0 && g == 0) paged::report(P.c.status);
        zero_out<T>(P, t, g, threadIdx.x % (32 * kNW), 32 * kNW);
        return;
    }
    const T* qrow = static_cast<const T*>(P.q) + (size_t)t * P.qs + g * kG * kD;
    const Partial x = query_part<T>(P, s, pos, g, qrow, 4 * (warp % kNW), 4 * kNW);
    const int h = lane >> 3, ch = lane & 7;
    if (kNW == 1) {
        write_part<T>(P, t, g, h, ch, x);
        return;
    }
    T* o = static_cast<T*>(P.o) + ((size_t)t * kHq + g * kG) * kD;
    float* lse = P.lse ? P.lse + (size_t)t * kHq + g * kG : nullptr;
    if (ch == 0) {
        top[warp][h] = x.m;
        sum[warp][h] = x.l;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) part[kNW > 1 ? warp : 0][kNW > 1 ? h * kD + 8 * ch + j : 0] = x.acc[j];
    __syncthreads();
    {
        const int hh = threadIdx.x >> 6;  // 256 threads: one output each
        float m = top[0][hh];
#pragma unroll
        for (int w = 1; w < kNW; ++w) m = fmaxf(m, top[w][hh]);
        float l = 0.f, v = 0.f;
#pragma unroll
        for (int w = 0; w < kNW; ++w) {
            const float f = exp2f(top[w][hh] - m);
            l = fmaf(f, sum[w][hh], l);
            v = fmaf(f, part[kNW > 1 ? w : 0][kNW > 1 ? threadIdx.x : 0], v);
        }
        const float inv = l != 0.f ? 1.f / l : 0.f;
        o[threadIdx.x] = from_f32<T>(v * inv);
        if (lse && (threadIdx.x & 63) == 0) lse[hh] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
}

template <typename T, int kNW>
cudaError_t launch_rows(const PagedFwd& P, cudaStream_t s) {
    constexpr int kUnits = 8 / kNW;
    const long long units = (long long)P.c.N * kHkv;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((units + kUnits - 1) / kUnits));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, rows_kernel<T, kNW>, P);
    if (e == cudaSuccess) count_launch();
    return e;
}

// ------------------------------------------------- many tokens: tensor cores
//
// Quad kernel (bf16, W <= 28): a warp owns four consecutive queries of one
// sequence and one key/value head, as two pairs of 2 queries x 4 heads, and
// forms both products with mma.sync m16n8k16, keys on M:
//   S^T (16 key rows x 8 columns) = K_rows . Q^T,   O^T += V_rows^T . P^T.
// Window: rows i - W .. i + 3 of the quad are one M tile (two from W = 13 on)
// shared by both pairs.  Rungs: one M tile a pair holds four rungs, row r < 8
// the far row i + e - n - 1 and row r + 8 the near row i + e - n of rung r % 4
// for query e = r / 4 of the pair, so both rows of an interpolation sit in one
// thread: it mixes their scores, and splits the probability onto them.
//
// Rows come through the block table, so no block of rows is contiguous and no
// tiled copy fits; the fragments are loaded straight into registers instead,
// with no shared memory, no transpose and no barrier.  The dimensions of the
// two products are taken in an order that makes every load 16 bytes:
//   scores: k-step s of thread (row g, lane t) takes words s of the row's
//     16-byte chunks t and 4 + t, for keys and queries alike;
//   values: output row m of tile j is dimension 8 (m % 8) + 2 j + m / 8, so
//     thread (g, t) needs chunk g of its four rows 2t, 2t + 1, 2t + 8, 2t + 9,
//     and ends with dimensions 8g .. 8g + 7 of its columns: one 16-byte store.
// Neighbouring queries read neighbouring rows, so a row comes from L2 once a
// block and from L1 after that.
//
// Entries that are masked get probability 0, and rows that no query of the
// quad may read are not loaded (zeros), but a row that one query reads is
// multiplied with the others' zeros: infinity or NaN in it would reach them.
// The epilogue looks for values that are not finite and redoes those queries
// one at a time with the rows of that query alone.  Nothing of a column's
// arithmetic depends on another column, so the second pass gives what the
// first would have given without the others' rows, bit for bit.

constexpr int kQuadWarps = 4;

struct Tile {
    uint4 k[4];      // rows g, g + 8: chunks t, 4 + t of each
    uint4 v[4];      // rows 2t, 2t + 1, 2t + 8, 2t + 9: chunk g
    bool lo, hi;     // rows g and g + 8 are there
};

// One query pair: the B fragments of Q^T, O^T, and the running maximum (log2
// units) and sum of this thread's two columns (query tig / 2 of the pair,
// heads 2 (tig & 1) and that + 1); the sums are this thread's rows' alone.
struct Pair {
    uint32_t qf[4][2];
    float o[4][4];
    float m[2], l[2];
};

__device__ __forceinline__ uint32_t word(const uint4& u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; }

// The tile whose 16 row numbers lanes base .. base + 15 hold in `row`.
__device__ __forceinline__ void load_tile(const uint4* __restrict__ k, const uint4* __restrict__ v, int row, int base,
                                          Tile& x) {
    const int lane = threadIdx.x & 31, g8 = lane >> 2, tig = lane & 3;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const int ra = __shfl_sync(kFull, row, base + g8), rb = __shfl_sync(kFull, row, base + 8 + g8);
    x.lo = ra >= 0;
    x.hi = rb >= 0;
    const uint4* pa = k + (size_t)ra * (kHkv * kD / 8) + tig;
    const uint4* pb = k + (size_t)rb * (kHkv * kD / 8) + tig;
    x.k[0] = x.lo ? __ldg(pa) : zero;
    x.k[1] = x.lo ? __ldg(pa + 4) : zero;
    x.k[2] = x.hi ? __ldg(pb) : zero;
    x.k[3] = x.hi ? __ldg(pb + 4) : zero;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = __shfl_sync(kFull, row, base + 2 * tig + (j & 1) + 8 * (j >> 1));
        x.v[j] = r >= 0 ? __ldg(v + (size_t)r * (kHkv * kD / 8) + g8) : zero;
    }
}

// S^T of a tile and a pair: c[0], c[1] row g, c[2], c[3] row g + 8.
__device__ __forceinline__ void scores(const Tile& x, const Pair& U, float (&c)[4]) {
    mma16816_z(c, x.k[0].x, x.k[2].x, x.k[1].x, x.k[3].x, U.qf[0][0], U.qf[0][1]);
    mma16816(c, x.k[0].y, x.k[2].y, x.k[1].y, x.k[3].y, U.qf[1][0], U.qf[1][1]);
    mma16816(c, x.k[0].z, x.k[2].z, x.k[1].z, x.k[3].z, U.qf[2][0], U.qf[2][1]);
    mma16816(c, x.k[0].w, x.k[2].w, x.k[1].w, x.k[3].w, U.qf[3][0], U.qf[3][1]);
}

// O^T += V_rows^T . P^T
__device__ __forceinline__ void values(const Tile& x, Pair& U, uint32_t b0, uint32_t b1) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t v0 = word(x.v[0], j), v1 = word(x.v[1], j), v2 = word(x.v[2], j), v3 = word(x.v[3], j);
        mma16816(U.o[j], __byte_perm(v0, v1, 0x5410), __byte_perm(v0, v1, 0x7632), __byte_perm(v2, v3, 0x5410),
                 __byte_perm(v2, v3, 0x7632), b0, b1);
    }
}

// Raise the running maximum of each column whose largest of x0 (x1) over the
// eight threads that hold it passes the margin, and rescale it.
__device__ __forceinline__ void raise(Pair& U, float x0, float x1) {
#pragma unroll
    for (int w = 4; w <= 16; w <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(kFull, x0, w));
        x1 = fmaxf(x1, __shfl_xor_sync(kFull, x1, w));
    }
    const float n0 = x0 > U.m[0] + kLazy ? x0 : U.m[0], n1 = x1 > U.m[1] + kLazy ? x1 : U.m[1];
    const float f0 = fast_exp2(U.m[0] - n0), f1 = fast_exp2(U.m[1] - n1);
    U.m[0] = n0;
    U.m[1] = n1;
    U.l[0] *= f0;
    U.l[1] *= f1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        U.o[j][0] *= f0;
        U.o[j][1] *= f1;
        U.o[j][2] *= f0;
        U.o[j][3] *= f1;
    }
}

// Window tile: R is the tile's first row counted from i - W of the quad's
// first query; pair k holds queries 2k, 2k + 1.
__device__ __forceinline__ void window_tile(const Tile& x, int k, int R, int W, float sl2, Pair& U) {
    const int lane = threadIdx.x & 31, g8 = lane >> 2, tig = lane & 3;
    float c[4];
    scores(x, U, c);
    const int qq = 2 * k + (tig >> 1);
    const bool lo = x.lo && R + g8 >= qq && R + g8 <= W + qq;
    const bool hi = x.hi && R + g8 + 8 >= qq && R + g8 + 8 <= W + qq;
    c[0] = lo ? c[0] * sl2 : -INFINITY;
    c[1] = lo ? c[1] * sl2 : -INFINITY;
    c[2] = hi ? c[2] * sl2 : -INFINITY;
    c[3] = hi ? c[3] * sl2 : -INFINITY;
    const float x0 = fmaxf(c[0], c[2]), x1 = fmaxf(c[1], c[3]);
    if (__any_sync(kFull, x0 > U.m[0] + kLazy || x1 > U.m[1] + kLazy)) raise(U, x0, x1);
    c[0] = fast_exp2(c[0] - U.m[0]);
    c[1] = fast_exp2(c[1] - U.m[1]);
    c[2] = fast_exp2(c[2] - U.m[0]);
    c[3] = fast_exp2(c[3] - U.m[1]);
    U.l[0] += c[0] + c[2];
    U.l[1] += c[1] + c[3];
    values(x, U, movm_t(pack_bf16(c[0], c[1])), movm_t(pack_bf16(c[2], c[3])));
}

// Rung tile of one pair; t: the fraction of this thread's rung (row g % 4).
__device__ __forceinline__ void rung_tile(const Tile& x, float t, float sl2, Pair& U) {
    const int lane = threadIdx.x & 31, g8 = lane >> 2, tig = lane & 3;
    float c[4];
    scores(x, U, c);
    const bool ok = (g8 >> 2) == (tig >> 1) && x.hi && (x.lo || t == 0.f);
    const float u = 1.f - t;
    const float x0 = ok ? (u * c[2] + t * c[0]) * sl2 : -INFINITY;
    const float x1 = ok ? (u * c[3] + t * c[1]) * sl2 : -INFINITY;
    if (__any_sync(kFull, x0 > U.m[0] + kLazy || x1 > U.m[1] + kLazy)) raise(U, x0, x1);
    const float p0 = fast_exp2(x0 - U.m[0]), p1 = fast_exp2(x1 - U.m[1]);
    U.l[0] += p0;
    U.l[1] += p1;
    values(x, U, movm_t(pack_bf16(p0 * t, p1 * t)), movm_t(pack_bf16(p0 * u, p1 * u)));
}

__global__ void __launch_bounds__(kQuadWarps * 32, 3) quad_kernel(const __grid_constant__ PagedFwd P) {
    __shared__ int rn[SFA_MAX_RUNGS], rc[SFA_MAX_RUNGS];
    __shared__ float rt[SFA_MAX_RUNGS];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g8 = lane >> 2, tig = lane & 3;
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
    const int g = blockIdx.x % kHkv, slot = (int)(blockIdx.x / kHkv) * kQuadWarps + warp;
    const int s = paged::last_at_most(P.c.S, slot, [&](int i) { return (__ldg(P.c.cu + i) >> 2) + i; });
    const int start = __ldg(P.c.cu + s), end = __ldg(P.c.cu + s + 1);
    const int t0 = start + 4 * (slot - (start >> 2) - s);
    if (t0 < 0 || t0 >= P.c.N || t0 >= end) return;
    const int cnt = min(4, min(end, P.c.N) - t0);
    const int i0 = __ldg(P.c.lens + s) - (end - t0);     // position of the first query
    const int last = min(i0 + cnt, P.c.cap) - 1;         // no row behind it is read
    const float sl2 = P.a.scale * kLog2e;
    const int W = P.a.W;
    const uint4* kb = static_cast<const uint4*>(P.c.k) + g * (kD / 8);
    const uint4* vb = static_cast<const uint4*>(P.c.v) + g * (kD / 8);
    bool bad = false;
    auto look_up = [&](int pos, bool want) {
        if (!want) return -1;
        const int row = paged::page_row(P.c, s, pos);
        bad |= row < 0;
        return row;
    };
    // rungs that the last query uses: a prefix, four to a tile
    const int used = __popc(__ballot_sync(kFull, rc[lane] <= last));
    const int nt = (used + 3) >> 2;
    if (__any_sync(kFull, lane < cnt && (i0 + lane < 0 || i0 + lane >= P.c.cap)) && lane == 0) paged::report(P.c.status);
    unsigned redo = 0;       // queries to do alone
    for (int only = -1;;) {  // the query that is done alone, -1: all
        // this lane's row of the window: position i0 - W + lane
        const int wpos = i0 - W + lane;
        const int wrow = look_up(wpos, wpos >= 0 && wpos <= last && (only < 0 || (lane >= only && lane <= only + W)));
        // this lane's row of rung tile t: lanes 0-15 the first pair's, 16-31 the second's
        const int my_q = 2 * (lane >> 4) + ((lane >> 2) & 1);
        auto rung_row = [&](int t) {
            const int r = 4 * t + (lane & 3), i = i0 + my_q;
            const bool near_row = lane & 8;
            return look_up(i - rn[r] - (near_row ? 0 : 1), i <= last && i >= rc[r] && (near_row || rt[r] > 0.f) &&
                                                               (only < 0 || my_q == only));
        };
        Pair U[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int qt = t0 + min(2 * k + (g8 >> 2), cnt - 1);
            const uint4* qp = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(P.q) +
                                                             (size_t)qt * P.qs + (g * kG + (g8 & 3)) * kD) + tig;
            const uint4 a = __ldg(qp), b = __ldg(qp + 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                U[k].qf[j][0] = word(a, j);
                U[k].qf[j][1] = word(b, j);
#pragma unroll
                for (int e = 0; e < 4; ++e) U[k].o[j][e] = 0.f;
            }
            U[k].m[0] = U[k].m[1] = kFloor;
            U[k].l[0] = U[k].l[1] = 0.f;
        }
        // two tiles in turn: one is loaded while the other is used
        Tile A, B;
        load_tile(kb, vb, wrow, 0, A);
        int row = nt > 0 ? rung_row(0) : -1;
        if (W > 12) {
            load_tile(kb, vb, wrow, 16, B);
#pragma unroll
            for (int k = 0; k < 2; ++k) window_tile(A, k, 0, W, sl2, U[k]);
            load_tile(kb, vb, row, 0, A);
#pragma unroll
            for (int k = 0; k < 2; ++k) window_tile(B, k, 16, W, sl2, U[k]);
        } else {
            load_tile(kb, vb, row, 0, B);
#pragma unroll
            for (int k = 0; k < 2; ++k) window_tile(A, k, 0, W, sl2, U[k]);
            A = B;
        }
        for (int t = 0; t < nt; ++t) {
            load_tile(kb, vb, row, 16, B);
            const int next = t + 1 < nt ? rung_row(t + 1) : -1;
            const float frac = rt[4 * t + (g8 & 3)];
            rung_tile(A, frac, sl2, U[0]);
            if (t + 1 < nt) load_tile(kb, vb, next, 0, A);
            rung_tile(B, frac, sl2, U[1]);
            row = next;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int w = 4; w <= 16; w <<= 1) {
                U[k].l[0] += __shfl_xor_sync(kFull, U[k].l[0], w);
                U[k].l[1] += __shfl_xor_sync(kFull, U[k].l[1], w);
            }
            const int qq = 2 * k + (tig >> 1), pos = i0 + qq;
            const bool in = pos >= 0 && pos < P.c.cap;
            float odd = 0.f;  // stays 0 while every value is finite
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) odd = fmaf(U[k].o[j][e], 0.f, odd);
            if (only < 0) {
                // lanes with tig < 2 hold the pair's first query
                const unsigned who = __ballot_sync(kFull, odd != 0.f && qq < cnt && in);
                redo |= ((who & 0x33333333u ? 1u : 0u) | (who & 0xccccccccu ? 2u : 0u)) << (2 * k);
            }
            if (qq >= cnt || (only < 0 ? (redo >> qq) & 1u : qq != only)) continue;
            const float f0 = in && U[k].l[0] != 0.f ? 1.f / U[k].l[0] : 0.f;  // no entry: zeros
            const float f1 = in && U[k].l[1] != 0.f ? 1.f / U[k].l[1] : 0.f;
            const size_t at = (size_t)(t0 + qq) * kHq + g * kG + 2 * (tig & 1);
            uint32_t w0[4], w1[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w0[j] = pack_bf16(U[k].o[j][0] * f0, U[k].o[j][2] * f0);
                w1[j] = pack_bf16(U[k].o[j][1] * f1, U[k].o[j][3] * f1);
            }
            uint4* o = static_cast<uint4*>(P.o) + at * (kD / 8) + g8;
            o[0] = make_uint4(w0[0], w0[1], w0[2], w0[3]);
            o[kD / 8] = make_uint4(w1[0], w1[1], w1[2], w1[3]);
            if (P.lse && g8 == 0) {
                const float y0 = U[k].l[0] != 0.f ? (U[k].m[0] + __log2f(U[k].l[0])) * kLn2 : -INFINITY;
                const float y1 = U[k].l[1] != 0.f ? (U[k].m[1] + __log2f(U[k].l[1])) * kLn2 : -INFINITY;
                P.lse[at] = in ? y0 : 0.f;
                P.lse[at + 1] = in ? y1 : 0.f;
            }
        }
        if (redo == 0) break;
        only = __ffs(redo) - 1;
        redo &= redo - 1;
    }
    if (__any_sync(kFull, bad) && lane == 0) paged::report(P.c.status);
}

cudaError_t launch_quads(const PagedFwd& P, cudaStream_t s) {
    const long long slots = (long long)P.c.N / 4 + P.c.S;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((slots + kQuadWarps - 1) / kQuadWarps * kHkv));
    cfg.blockDim = dim3(kQuadWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, quad_kernel, P);
    if (e == cudaSuccess) count_launch();
    return e;
}

}  // namespace

cudaError_t launch_paged_fwd(const LayerArgs& a, const PagedArgs& c, sfa_dtype dt, const void* q, long long qs, void* o,
                             float* lse, cudaStream_t s) {
    const PagedFwd P = {a, c, q, qs, o, lse};
    const bool few = c.N <= 512;
    if (dt == SFA_BF16 && !few && a.W <= 28) return launch_quads(P, s);
    if (dt == SFA_BF16) return few ? launch_rows<__nv_bfloat16, 8>(P, s) : launch_rows<__nv_bfloat16, 1>(P, s);
    return few ? launch_rows<float, 8>(P, s) : launch_rows<float, 1>(P, s);
}

}  // namespace sfa
