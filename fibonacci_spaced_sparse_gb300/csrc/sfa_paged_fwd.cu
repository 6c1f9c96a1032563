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

template <int kNW>
constexpr int kRowThreads = kNW > 1 ? 32 * kNW : 256;  // one unit a block, or eight of one warp each

template <typename T, int kNW>
__global__ void __launch_bounds__(kRowThreads<kNW>, 512 / kRowThreads<kNW>) rows_kernel(const __grid_constant__ PagedFwd P) {
    constexpr int kThreads = kRowThreads<kNW>, kUnits = kNW > 1 ? 1 : 8;  // (token, head) of a block
    __shared__ __align__(16) float part[kNW > 1 ? kNW : 1][kNW > 1 ? kG * kD : 4];
    __shared__ float top[kNW][kG], sum[kNW][kG];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned unit = blockIdx.x * kUnits + (kNW > 1 ? 0 : warp);
    const int t = (int)(unit / kHkv), g = (int)(unit % kHkv);
    if (t >= P.c.N) return;  // with kNW > 1 the whole block, here and below
    const int s = paged::sequence_of(P.c, t);
    if (s >= P.c.S) return;
    const int pos = __ldg(P.c.lens + s) - (__ldg(P.c.cu + s + 1) - t);
    if (pos < 0 || pos >= P.c.cap) {
        const int i = kNW > 1 ? threadIdx.x : lane;
        if (i == 0 && g == 0) paged::report(P.c.status);
        zero_out<T>(P, t, g, i, kNW > 1 ? kThreads : 32);
        return;
    }
    const T* qrow = static_cast<const T*>(P.q) + (size_t)t * P.qs + g * kG * kD;
    const Partial x = query_part<T>(P, s, pos, g, qrow, kNW > 1 ? 4 * warp : 0, 4 * kNW);
    const int h = lane >> 3, ch = lane & 7;
    if (kNW == 1) {
        write_part<T>(P, t, g, h, ch, x);
        return;
    }
    if (ch == 0) {
        top[warp][h] = x.m;
        sum[warp][h] = x.l;
    }
    float* mine = part[kNW > 1 ? warp : 0] + (kNW > 1 ? h * kD + 8 * ch : 0);
    if (kNW > 1) {
        reinterpret_cast<float4*>(mine)[0] = make_float4(x.acc[0], x.acc[1], x.acc[2], x.acc[3]);
        reinterpret_cast<float4*>(mine)[1] = make_float4(x.acc[4], x.acc[5], x.acc[6], x.acc[7]);
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
    constexpr int kUnits = kNW > 1 ? 1 : 8;
    const long long units = (long long)P.c.N * kHkv;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((units + kUnits - 1) / kUnits));
    cfg.blockDim = dim3(kRowThreads<kNW>);
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

// As many warps a (token, head) as keep all of them resident at once (16 a SM
// at 128 registers, 152 SMs): a decode step is then one wave of one or two
// rounds of loads.  us for N single tokens over 3000 rows, bf16, with 8, 4, 2
// and 1 warps: N = 128 3.9, 4.6, 5.6, 6.6; 256 6.9, 4.8, 6.2, 6.9; 1024 22.7,
// 16.0, 12.0, 8.6.
template <typename T>
cudaError_t launch_rows(const PagedFwd& P, cudaStream_t s) {
    const long long most = 152 * 16 / ((long long)P.c.N * kHkv);
    return most >= 8   ? launch_rows_nw<T, 8>(P, s)
           : most >= 4 ? launch_rows_nw<T, 4>(P, s)
           : most >= 2 ? launch_rows_nw<T, 2>(P, s)
                       : launch_rows_nw<T, 1>(P, s);
}

// ------------------------------------------------- many tokens: tensor cores
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
// Masked entries get probability 0.  A row that some queries of the quad read
// is multiplied with the others' zeros, and a tile row that none reads is
// filled with the first query's own row; infinity or NaN there would reach
// queries that do not read it.  The epilogue looks for values that are not
// finite and redoes those queries one at a time (kAlone), with that query's
// rows and zeros.  Nothing of a column's arithmetic depends on another column,
// so this gives what the first pass would have given without the others' rows,
// bit for bit.

constexpr int kQuadWarps = 4;

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
    asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
        : "l"(p));
}

// The tile whose 16 row numbers lanes base .. base + 15 hold in `row`; in a
// kAlone pass rows that are not there (-1) are zeros.
template <bool kAlone>
__device__ __forceinline__ void load_tile(const char* __restrict__ k, const char* __restrict__ v, int row, int base,
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
        const size_t at = (size_t)(unsigned)r * kStride + 32 * tig;
        load32(k + at, x.k[h]);
        load32(v + at, x.v[h]);
    }
}

// S^T of a tile and a pair: c[0], c[1] row g, c[2], c[3] row g + 8.
__device__ __forceinline__ void scores(const Tile& x, const Pair& U, float (&c)[4]) {
    mma16816_z(c, x.k[0][0], x.k[1][0], x.k[0][4], x.k[1][4], U.qf[0][0], U.qf[0][1]);
#pragma unroll
    for (int s = 1; s < 4; ++s)
        mma16816(c, x.k[0][s], x.k[1][s], x.k[0][4 + s], x.k[1][4 + s], U.qf[s][0], U.qf[s][1]);
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
template <bool kFirst>
__device__ __forceinline__ void window_tile(const Tile& x, unsigned mask, float sl2, Pair (&U)[2]) {
    uint32_t b[2][2];
    const float2 sl = f2(sl2, sl2);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float c[4];
        scores(x, U[k], c);
        float2 lo = __fmul2_rn(f2(c[0], c[1]), sl), hi = __fmul2_rn(f2(c[2], c[3]), sl);
        if (!(mask >> (2 * k) & 1u)) lo = f2(-INFINITY, -INFINITY);
        if (!(mask >> (2 * k + 1) & 1u)) hi = f2(-INFINITY, -INFINITY);
        const float2 top = f2(fmaxf(lo.x, hi.x), fmaxf(lo.y, hi.y));
        if (kFirst) {
            const float2 m = column_max(top);
            U[k].nm = f2(-fmaxf(m.x, kFloor), -fmaxf(m.y, kFloor));
            U[k].th = f2(kLazy - U[k].nm.x, kLazy - U[k].nm.y);
        } else if (__any_sync(kFull, top.x > U[k].th.x || top.y > U[k].th.y)) {
            raise(U[k], top);
        }
        lo = __fadd2_rn(lo, U[k].nm);
        hi = __fadd2_rn(hi, U[k].nm);
        lo = f2(fast_exp2(lo.x), fast_exp2(lo.y));
        hi = f2(fast_exp2(hi.x), fast_exp2(hi.y));
        U[k].l = kFirst ? __fadd2_rn(lo, hi) : __fadd2_rn(U[k].l, __fadd2_rn(lo, hi));
        b[k][0] = movm_t(pack_bf16(lo.x, lo.y));
        b[k][1] = movm_t(pack_bf16(hi.x, hi.y));
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

// Rung tile of one pair.  ok: this thread's rung is an entry of its query;
// t: the rung's fraction.
__device__ __forceinline__ void rung_tile(const Tile& x, bool ok, float t, float sl2, Pair& U) {
    float c[4];
    scores(x, U, c);
    const float u = 1.f - t;
    const float2 tt = f2(t, t), uu = f2(u, u);
    float2 s = __ffma2_rn(f2(t * sl2, t * sl2), f2(c[0], c[1]), __fmul2_rn(f2(u * sl2, u * sl2), f2(c[2], c[3])));
    if (!ok) s = f2(-INFINITY, -INFINITY);
    if (__any_sync(kFull, s.x > U.th.x || s.y > U.th.y)) raise(U, s);
    s = __fadd2_rn(s, U.nm);
    const float2 p = f2(fast_exp2(s.x), fast_exp2(s.y));
    U.l = __fadd2_rn(U.l, p);
    const float2 far_p = __fmul2_rn(p, tt), near_p = __fmul2_rn(p, uu);
    const uint32_t b0 = movm_t(pack_bf16(far_p.x, far_p.y)), b1 = movm_t(pack_bf16(near_p.x, near_p.y));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t a[4];
        value_frag(x, j, a);
        mma16816(U.o[j], a[0], a[1], a[2], a[3], b0, b1);
    }
}

struct Quad {
    int s, t0, cnt, i0, last, g;
    const int *rn, *rc;
    const float* rt;
};

// All queries of the quad, or the query `only` alone; returns the queries
// whose results are not finite (they are not written).
template <bool kAlone>
__device__ __forceinline__ unsigned quad_pass(const PagedFwd& P, const Quad& Q, int only) {
    const int lane = threadIdx.x & 31, g8 = lane >> 2, tig = lane & 3;
    const int W = P.a.W, i0 = Q.i0, last = Q.last;
    const float sl2 = P.a.scale * kLog2e;
    const char* kb = static_cast<const char*>(P.c.k) + Q.g * (kD * 2);
    const char* vb = static_cast<const char*>(P.c.v) + Q.g * (kD * 2);
    // this lane's row of the window: position i0 - W + lane
    bool want = lane < W + 4 && i0 - W + lane >= 0 && i0 - W + lane <= last && (!kAlone || (lane >= only && lane <= only + W));
    int wrow = want ? paged::page_row(P.c, Q.s, i0 - W + lane) : -1;
    bool bad = want && wrow < 0;
    const int fill = kAlone ? -1 : max(__shfl_sync(kFull, wrow, W), 0);  // the first query's own row
    // rungs that the last query uses: a prefix, four to a tile
    const int nt = (__popc(__ballot_sync(kFull, Q.rc[lane] <= last)) + 3) >> 2;
    // this lane's row of a rung tile: lanes 0-15 the first pair's, 16-31 the second's
    const int my_q = 2 * (lane >> 4) + ((lane >> 2) & 1);
    const bool near_row = lane & 8;
    unsigned there = 0;  // rows of the tile that are there, where pages are bad
    auto rung_rows = [&](int t) {
        const int r = 4 * t + (lane & 3), i = i0 + my_q;
        const bool w = i <= last && i >= Q.rc[r] && (near_row || Q.rt[r] > 0.f) && (!kAlone || my_q == only);
        const int row = w ? paged::page_row(P.c, Q.s, i - Q.rn[r] - (near_row ? 0 : 1)) : -1;
        bad |= w && row < 0;
        return row;
    };
    Pair U[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int qt = Q.t0 + min(2 * k + (g8 >> 2), Q.cnt - 1);
        const uint4* qp = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(P.q) + (size_t)qt * P.qs +
                                                         (Q.g * kG + (g8 & 3)) * kD) + 2 * tig;
        const uint4 a = __ldg(qp), b = __ldg(qp + 1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            U[k].qf[j][0] = word(a, j);
            U[k].qf[j][1] = word(b, j);
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
    // two tiles in turn: one is loaded while the other is used
    Tile A, B;
    load_tile<kAlone>(kb, vb, wrow >= 0 ? wrow : fill, 0, A);
    int row = nt > 0 ? rung_rows(0) : -1;
    if (W > 12) {
        load_tile<kAlone>(kb, vb, wrow >= 0 ? wrow : fill, 16, B);
        window_tile<true>(A, mask[0], sl2, U);
        if (nt > 0) load_tile<kAlone>(kb, vb, row >= 0 ? row : fill, 0, A);
        window_tile<false>(B, mask[1], sl2, U);
    } else {
        if (nt > 0) load_tile<kAlone>(kb, vb, row >= 0 ? row : fill, 0, B);
        window_tile<true>(A, mask[0], sl2, U);
        A = B;
    }
    const int my_i = (g8 >> 2) == (tig >> 1) ? i0 + (tig >> 1) : -(1 << 30);  // its own rung's query, or none
    for (int t = 0; t < nt; ++t) {
        load_tile<kAlone>(kb, vb, row >= 0 ? row : fill, 16, B);
        const bool holes = __any_sync(kFull, bad);
        if (holes) there = __ballot_sync(kFull, row >= 0);
        const float frac = Q.rt[4 * t + (g8 & 3)];
        const int c = Q.rc[4 * t + (g8 & 3)];
        bool ok[2] = {my_i >= c, my_i + 2 >= c};
        if (holes) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
                ok[k] = ok[k] && (there >> (16 * k + 8 + g8) & 1u) && ((there >> (16 * k + g8) & 1u) || frac == 0.f);
        }
        row = t + 1 < nt ? rung_rows(t + 1) : -1;
        rung_tile(A, ok[0], frac, sl2, U[0]);
        if (t + 1 < nt) load_tile<kAlone>(kb, vb, row >= 0 ? row : fill, 0, A);
        rung_tile(B, ok[1], frac, sl2, U[1]);
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
            w[2 * j] = pack_bf16(a.x, a.y);
            w[2 * j + 1] = pack_bf16(b.x, b.y);
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

// A call of its own, so that the rare pass takes no registers of the common one.
__device__ __noinline__ void one_alone(const PagedFwd& P, const Quad& Q, int only) { quad_pass<true>(P, Q, only); }

__global__ void __launch_bounds__(kQuadWarps * 32, 3) quad_kernel(const __grid_constant__ PagedFwd P) {
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
    Q.s = paged::last_at_most(P.c.S, slot, [&](int i) { return (__ldg(P.c.cu + i) >> 2) + i; });
    const int start = __ldg(P.c.cu + Q.s), end = __ldg(P.c.cu + Q.s + 1);
    Q.t0 = start + 4 * (slot - (start >> 2) - Q.s);
    if (Q.t0 < 0 || Q.t0 >= P.c.N || Q.t0 >= end) return;
    Q.cnt = min(4, min(end, P.c.N) - Q.t0);
    Q.i0 = __ldg(P.c.lens + Q.s) - (end - Q.t0);       // position of the first query
    Q.last = min(Q.i0 + Q.cnt, P.c.cap) - 1;           // no row behind it is read
    Q.rn = rn;
    Q.rc = rc;
    Q.rt = rt;
    if (__any_sync(kFull, lane < Q.cnt && (Q.i0 + lane < 0 || Q.i0 + lane >= P.c.cap)) && lane == 0)
        paged::report(P.c.status);
    for (unsigned redo = quad_pass<false>(P, Q, -1); redo; redo &= redo - 1) one_alone(P, Q, __ffs(redo) - 1);
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

constexpr int kQuadsFrom = 512;

}  // namespace

cudaError_t launch_paged_fwd(const LayerArgs& a, const PagedArgs& c, sfa_dtype dt, const void* q, long long qs, void* o,
                             float* lse, cudaStream_t s) {
    const PagedFwd P = {a, c, q, qs, o, lse};
    const bool quads = dt == SFA_BF16 && a.W <= 28 && c.N >= kQuadsFrom && c.N >= 2 * c.S;
    if (quads) return launch_quads(P, s);
    return dt == SFA_BF16 ? launch_rows<__nv_bfloat16>(P, s) : launch_rows<float>(P, s);
}

}  // namespace sfa
