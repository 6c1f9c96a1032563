// sfa_add_norm.cu -- the residual's addition and the RMS norm of every row, to
// the rows' type or to 8 bits with a scale a row; its backward pass; and rows to
// 8 bits as they are (sfa_add_rms_norm in include/sfa.h).
//
// h = x + res, rounded to the type it is kept in; r = 1 / sqrt(mean(h^2) + eps),
// y = h r w.  In 8 bits y = s c with s = max |y| / 448.  Backward, with g = w dy:
// dx = dh + r g - h r^3 mean(g h), dw = sum over rows of dy h r.
//
// All of it is bound by memory: two rows in and two out (or one and a half), in
// the backward pass three in and one out, with some ten operations a value.  A
// row is held in registers by kW warps, kV pieces of eight values a lane, so it
// is read once whatever is computed from it; sums over it are a warp's shuffles,
// and one exchange through shared memory where several warps hold it.  32 x 1024 bf16
// tokens of 512: forward 21.3 us, backward 23.1 (93 and 86 % of the copy rate).
#include <type_traits>

#include "sfa_fp8.cuh"
#include "sfa_heads.cuh"
#include "sfa_ops.cuh"

namespace sfa {

namespace {

// Eight values of a row.
template <typename T>
struct Piece;
template <>
struct Piece<__nv_bfloat16> {
    uint4 u;
};
template <>
struct Piece<float> {
    float4 u, v;
};
__device__ __forceinline__ void fetch(const __nv_bfloat16* p, Piece<__nv_bfloat16>& x) {
    x.u = fresh(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ void fetch(const float* p, Piece<float>& x) {
    x.u = fresh(reinterpret_cast<const float4*>(p));
    x.v = fresh(reinterpret_cast<const float4*>(p) + 1);
}
__device__ __forceinline__ void put(__nv_bfloat16* p, const Piece<__nv_bfloat16>& x) { *reinterpret_cast<uint4*>(p) = x.u; }
__device__ __forceinline__ void put(float* p, const Piece<float>& x) {
    reinterpret_cast<float4*>(p)[0] = x.u;
    reinterpret_cast<float4*>(p)[1] = x.v;
}
// As pairs for the packed two-lane fp32 instructions.
struct Eight {
    float2 f[4];
};
__device__ __forceinline__ Eight open(const Piece<__nv_bfloat16>& x) {
    const uint32_t w[4] = {x.u.x, x.u.y, x.u.z, x.u.w};
    Eight e;
#pragma unroll
    for (int j = 0; j < 4; ++j) e.f[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
    return e;
}
__device__ __forceinline__ Eight open(const Piece<float>& x) {
    return {{make_float2(x.u.x, x.u.y), make_float2(x.u.z, x.u.w), make_float2(x.v.x, x.v.y), make_float2(x.v.z, x.v.w)}};
}
__device__ __forceinline__ void close(const Eight& e, Piece<__nv_bfloat16>& x) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(e.f[j].x, e.f[j].y);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    x.u = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void close(const Eight& e, Piece<float>& x) {
    x.u = make_float4(e.f[0].x, e.f[0].y, e.f[1].x, e.f[1].y);
    x.v = make_float4(e.f[2].x, e.f[2].y, e.f[3].x, e.f[3].y);
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float warp_top(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
    return x;
}

// Rows of a block: kW warps each, at least eight warps together.
template <int kW>
constexpr int kRows = kW < 8 ? 8 / kW : 1;
template <int kW>
constexpr int kRowThreads = 32 * kW * kRows<kW>;

// The sum (or the largest) of x over the kW warps of a row, in every thread; `slot`:
// kW floats of shared memory of this row's.  The caller lets no two exchanges through one
// slot follow without a barrier between them.
template <int kW, bool kTop>
__device__ __forceinline__ float over_row(float x, float* slot) {
    x = kTop ? warp_top(x) : warp_sum(x);
    if (kW == 1) return x;
    const int warp = (threadIdx.x >> 5) % kW;
    if ((threadIdx.x & 31) == 0) slot[warp] = x;
    __syncthreads();
    float y = slot[0];
#pragma unroll
    for (int w = 1; w < kW; ++w) y = kTop ? fmaxf(y, slot[w]) : y + slot[w];
    return y;
}

enum class To { kSame, kFp8, kFp8AsIs };  // the norm in the rows' type, in 8 bits; the rows themselves in 8 bits

template <typename T, int kV, int kW, To kTo>
__global__ void __launch_bounds__(kRowThreads<kW>) add_norm_kernel(const AddNormArgs a) {
    __shared__ float sums[kRows<kW>][kW], tops[kRows<kW>][kW];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int group = threadIdx.x / (32 * kW), i = threadIdx.x % (32 * kW);
    const long long row = (long long)blockIdx.x * kRows<kW> + group;
    const bool live = row < a.N;
    if (kW == 1 && !live) return;
    const long long at = live ? row : a.N - 1;  // a row that is not there repeats the last one and stores nothing
    const T* x = static_cast<const T*>(a.x) + at * a.xs;
    const T* res = static_cast<const T*>(a.r) + at * a.rs;
    Piece<T> px[kV], pr[kV];
    bool in[kV];
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        const int e = 8 * (j * 32 * kW + i);
        in[j] = e < a.dim;
        px[j] = pr[j] = Piece<T>{};
        if (in[j]) {
            fetch(x + e, px[j]);
            if (kTo != To::kFp8AsIs && a.r) fetch(res + e, pr[j]);
        }
    }
    Eight v[kV];
    float2 square = both(0.f);
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        v[j] = open(px[j]);
        if (kTo == To::kFp8AsIs) continue;
        if (a.r) {
            const Eight y = open(pr[j]);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[j].f[k] = __fadd2_rn(v[j].f[k], y.f[k]);
            close(v[j], px[j]);
            v[j] = open(px[j]);  // the norm reads the sum as it is kept
            if (a.h && live && in[j]) put(static_cast<T*>(a.h) + row * a.dim + 8 * (j * 32 * kW + i), px[j]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) square = __ffma2_rn(v[j].f[k], v[j].f[k], square);
    }
    if (kTo != To::kFp8AsIs) {
        const float r = rsqrtf(over_row<kW, false>(square.x + square.y, sums[group]) * a.inv_dim + a.eps);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            Piece<float> w{};
            if (in[j]) fetch(a.w + 8 * (j * 32 * kW + i), w);
            const Eight ww = open(w);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[j].f[k] = __fmul2_rn(__fmul2_rn(v[j].f[k], both(r)), ww.f[k]);
        }
    }
    if (kTo == To::kSame) {
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            Piece<T> p;
            close(v[j], p);
            if (live && in[j]) put(static_cast<T*>(a.y) + row * a.dim + 8 * (j * 32 * kW + i), p);
        }
        return;
    }
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < kV; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (in[j]) top = fmaxf(top, fmaxf(fp8::finite_size(v[j].f[k].x), fp8::finite_size(v[j].f[k].y)));
    const float s = fp8::row_scale(over_row<kW, true>(top, tops[group])), inv = 1.f / s;
    if (!live) return;
    if (i == 0) a.scale[row] = s;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        float2 c[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) c[k] = __fmul2_rn(v[j].f[k], both(inv));
        if (in[j])
            *reinterpret_cast<uint2*>(static_cast<unsigned char*>(a.y) + row * a.dim + 8 * (j * 32 * kW + i)) =
                make_uint2(fp8::code4(c[0].x, c[0].y, c[1].x, c[1].y), fp8::code4(c[2].x, c[2].y, c[3].x, c[3].y));
    }
}

// ------------------------------------------------------------------ backward

// Forms of the backward pass.
//   kHeld: the weights in registers;
//   kRead: the weights read again (from L1) twice in every row, which leaves registers
//          for more blocks or for a wider row;
//   kAhead: the weights in registers, and while a row is computed the next one is on its
//           way to shared memory, each lane's own pieces (no barrier, no registers).
enum class Form { kHeld, kRead, kAhead };

// The form of long calls, by the pieces of a row that a lane has (times in us).
//   One: kRead, which fits five blocks a SM (32 x 1024 bf16 tokens of 256: 14.1, ahead 17.3).
//   Two, bf16: kAhead (held, read and ahead: 32 x 1024 of 512 29.6, 24.6 and 23.1; read and
//     ahead: 5000 of 512 6.9 and 5.3, 4096 of 4096 26.8 and 24.4; a third and a fourth row on
//     their way, 32 x 1024 of 512: 23.9 and 24.4).  fp32: kHeld (4083 of 320 6.2, ahead 8.9).
//   Four: kRead, the only one without many spills (1024 bf16 of 16384 38.4, ahead 48.8).
template <typename T, int kV>
constexpr Form kLong = kV != 2 ? Form::kRead : sizeof(T) == 2 ? Form::kAhead : Form::kHeld;

// Blocks a SM in the split that by_width chooses, as many as are resident: each writes one
// partial sum of dw (us, with one less or more: 32 x 1024 bf16 tokens of 256 15.6 with four,
// 14.1 with five; 2048 of 8192 26.3 with one, 28.0 with two).
template <typename T>
int bwd_each(int dim) {
    return dim > 4096 ? 1 : dim > 256 ? 2 : sizeof(T) == 2 ? 5 : 4;
}
constexpr int kBwdBlocks = kSms * 5;  // at most

// One piece a lane: blocks up to which the weights are held, two a SM.
constexpr int kHeldBlocks = kSms * 2;

// Block b writes dx of its rows (b, b + gridDim, ... in groups of kRows) and its
// part of dw to partial[b]; the launch after it sums the parts in a fixed order.
template <typename T, int kV, int kW, Form kForm>
__global__ void __launch_bounds__(kRowThreads<kW>) add_norm_bwd_kernel(const AddNormBwdArgs a, float* partial) {
    constexpr int kGroups = kRows<kW>, kWide = 256 * kV * kW;  // columns held
    constexpr bool kHeld = kForm != Form::kRead, kAhead = kForm == Form::kAhead;
    extern __shared__ uint4 ahead[];  // kAhead: [2 rows][h, dy, dh][kV][threads]
    __shared__ float sums[2][2][kGroups][kW];
    __shared__ float part[kGroups > 1 ? kGroups : 1][kGroups > 1 ? kWide : 1];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int group = threadIdx.x / (32 * kW), i = threadIdx.x % (32 * kW);
    Eight dw[kV], wt[kV];
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        const int e = 8 * (j * 32 * kW + i);
        Piece<float> w{};
        if (kHeld && e < a.dim) fetch(a.w + e, w);
        wt[j] = open(w);
        dw[j] = Eight{};
    }
    auto weight = [&](int j) {
        if (kHeld) return wt[j];
        const int e = 8 * (j * 32 * kW + i);
        Piece<float> w{};
        if (e < a.dim) fetch(a.w + e, w);
        return open(w);
    };
    // the pieces of the warp's row of h, dy and dh: to shared memory, and back
    auto slot = [&](int t, int which, int j) { return ahead + ((t * 3 + which) * kV + j) * kRowThreads<kW> + threadIdx.x; };
    auto send = [&](long long row0, int t) {
        const long long at = (row0 + group < a.N ? row0 + group : a.N - 1) * a.dim;
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int e = 8 * (j * 32 * kW + i);
            if (row0 >= a.N || e >= a.dim) continue;
            heads::copy16(slot(t, 0, j), static_cast<const T*>(a.h) + at + e);
            heads::copy16(slot(t, 1, j), static_cast<const T*>(a.dy) + at + e);
            if (a.dh) heads::copy16(slot(t, 2, j), static_cast<const T*>(a.dh) + at + e);
        }
        heads::copies_end();
    };
    if constexpr (kAhead) send((long long)blockIdx.x * kGroups, 0);
    int turn = 0;
    for (long long row0 = (long long)blockIdx.x * kGroups; row0 < a.N; row0 += (long long)gridDim.x * kGroups, turn ^= 1) {
        const bool live = row0 + group < a.N;
        const long long at = (live ? row0 + group : a.N - 1) * a.dim;  // idle warps repeat the last row; it counts once
        Piece<T> ph[kV], pg[kV], pd[kV];
        if constexpr (kAhead) {
            send(row0 + (long long)gridDim.x * kGroups, turn ^ 1);
            heads::copies_wait<1>();
        }
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int e = 8 * (j * 32 * kW + i);
            ph[j] = pg[j] = pd[j] = Piece<T>{};
            if constexpr (kAhead) {
                if (e >= a.dim) continue;
                ph[j].u = *slot(turn, 0, j);
                pg[j].u = *slot(turn, 1, j);
                if (a.dh) pd[j].u = *slot(turn, 2, j);
            } else if (e < a.dim) {
                fetch(static_cast<const T*>(a.h) + at + e, ph[j]);
                fetch(static_cast<const T*>(a.dy) + at + e, pg[j]);
                if (a.dh) fetch(static_cast<const T*>(a.dh) + at + e, pd[j]);
            }
        }
        float2 square = both(0.f), cross = both(0.f);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const Eight h = open(ph[j]), g = open(pg[j]), ww = weight(j);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                square = __ffma2_rn(h.f[k], h.f[k], square);
                cross = __ffma2_rn(__fmul2_rn(g.f[k], ww.f[k]), h.f[k], cross);
            }
        }
        float s2 = warp_sum(square.x + square.y), sc = warp_sum(cross.x + cross.y);
        if (kW > 1) {
            // two sets of slots in turn: a warp that is a row ahead writes the other one
            const int warp = (threadIdx.x >> 5) % kW;
            if ((threadIdx.x & 31) == 0) {
                sums[turn][0][group][warp] = s2;
                sums[turn][1][group][warp] = sc;
            }
            __syncthreads();
            s2 = sc = 0.f;
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                s2 += sums[turn][0][group][w];
                sc += sums[turn][1][group][w];
            }
        }
        const float r = rsqrtf(s2 * a.inv_dim + a.eps);
        const float2 rr = both(r), m = both(-r * r * (sc * a.inv_dim));  // dx = dh + r (g + h m)
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int e = 8 * (j * 32 * kW + i);
            const Eight h = open(ph[j]), g = open(pg[j]), ww = weight(j);
            Eight d = open(pd[j]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (live) dw[j].f[k] = __ffma2_rn(__fmul2_rn(h.f[k], rr), g.f[k], dw[j].f[k]);
                d.f[k] = __ffma2_rn(rr, __ffma2_rn(h.f[k], m, __fmul2_rn(g.f[k], ww.f[k])), d.f[k]);
            }
            Piece<T> p;
            close(d, p);
            if (live && e < a.dim) put(static_cast<T*>(a.dx) + at + e, p);
        }
    }
    float* mine = partial + (size_t)blockIdx.x * a.dim;
    if (kGroups == 1) {
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int e = 8 * (j * 32 * kW + i);
            Piece<float> p;
            close(dw[j], p);
            if (e < a.dim) put(mine + e, p);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        Piece<float> p;
        close(dw[j], p);
        put(&part[group][8 * (j * 32 * kW + i)], p);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.dim; e += kRowThreads<kW>) {
        float s = part[0][e];
#pragma unroll
        for (int g = 1; g < kGroups; ++g) s += part[g][e];
        mine[e] = s;
    }
}

// dw: the sum of the blocks' parts.  A block sums kFinCols columns, kFinRows
// threads a column, each with all of its loads in flight at once.
constexpr int kFinCols = 8, kFinRows = 64, kFinEach = (kBwdBlocks + kFinRows - 1) / kFinRows;
__global__ void __launch_bounds__(kFinCols* kFinRows) add_norm_dw_kernel(const float* partial, int blocks, int dim, float* dw) {
    __shared__ float sums[kFinRows / 4][kFinCols + 1];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int col = threadIdx.x % kFinCols, row = threadIdx.x / kFinCols;
    const int d = blockIdx.x * kFinCols + col;  // dim is a multiple of kFinCols
    float part[kFinEach];
#pragma unroll
    for (int i = 0; i < kFinEach; ++i) {
        const int b = row + i * kFinRows;
        part[i] = b < blocks ? fresh(partial + (size_t)b * dim + d) : 0.f;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kFinEach; ++i) s += part[i];
    // a warp holds four rows of the same columns
    s += __shfl_xor_sync(kFull, s, 8);
    s += __shfl_xor_sync(kFull, s, 16);
    if ((threadIdx.x & 31) < kFinCols) sums[row / 4][col] = s;
    __syncthreads();
    if (threadIdx.x < kFinCols) {
        s = 0.f;
#pragma unroll
        for (int r = 0; r < kFinRows / 4; ++r) s += sums[r][col];
        dw[d] = s;
    }
}

// Calls f with the row's split over lanes: at most 16 values a lane, so that a
// row's words, weights and gradients stay in registers.
template <typename F>
cudaError_t by_width(int dim, F f) {
#define SFA_SPLIT(v, w) f(std::integral_constant<int, v>{}, std::integral_constant<int, w>{})
    return dim <= 256    ? SFA_SPLIT(1, 1)
           : dim <= 512  ? SFA_SPLIT(2, 1)
           : dim <= 1024 ? SFA_SPLIT(2, 2)
           : dim <= 2048 ? SFA_SPLIT(2, 4)
           : dim <= 4096 ? SFA_SPLIT(2, 8)
           : dim <= 8192 ? SFA_SPLIT(2, 16)
                         : SFA_SPLIT(4, 16);
#undef SFA_SPLIT
}

template <typename T, To kTo>
cudaError_t launch_rows(const AddNormArgs& a, cudaStream_t s) {
    return by_width(a.dim, [&](auto v, auto w) {
        constexpr int kR = kRows<w()>;
        return launch_early(add_norm_kernel<T, v(), w(), kTo>, (unsigned)((a.N + kR - 1) / kR), kRowThreads<w()>, 0, s, a);
    });
}

// Blocks of the backward pass, in the split that by_width chooses.
template <typename T>
int bwd_blocks(int N, int dim) {
    const int warps = dim <= 512 ? 1 : dim <= 1024 ? 2 : dim <= 2048 ? 4 : 8, rows = 8 / warps;
    const int steps = (N + rows - 1) / rows, most = kSms * bwd_each<T>(dim);
    return steps < most ? steps : most;
}

template <typename T>
cudaError_t launch_bwd(const AddNormBwdArgs& a, float* ws, cudaStream_t s) {
    const int blocks = bwd_blocks<T>(a.N, a.dim);
    float* partial = blocks > 1 ? ws : a.dw;
    const cudaError_t e = by_width(a.dim, [&](auto v, auto w) {
        constexpr int kR = kRows<w()>;
        constexpr Form kMany = kLong<T, v()>, kFew = v() == 4 ? kMany : Form::kHeld;
        const bool many = kMany == Form::kAhead ? (a.N + kR - 1) / kR > blocks : blocks > kHeldBlocks;
        auto* kernel = add_norm_bwd_kernel<T, v(), w(), kFew>;
        size_t smem = 0;
        if (many && kMany != kFew) {
            kernel = add_norm_bwd_kernel<T, v(), w(), kMany>;
            if (kMany == Form::kAhead) {
                smem = (size_t)2 * 3 * v() * kRowThreads<w()> * sizeof(uint4);
                int dev = 0;
                cudaError_t e = cudaGetDevice(&dev);
                if (e != cudaSuccess) return e;
                static CtxSetting configured[64];
                if (!ctx_setting_holds(configured[dev & 63], smem)) {
                    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
                    if (e != cudaSuccess) return e;
                    ctx_setting_done(configured[dev & 63], smem);
                }
            }
        }
        return launch_early(kernel, (unsigned)blocks, kRowThreads<w()>, smem, s, a, partial);
    });
    if (e != cudaSuccess || blocks == 1) return e;
    return launch_early(add_norm_dw_kernel, (unsigned)(a.dim / kFinCols), (unsigned)(kFinCols * kFinRows), 0, s,
                        (const float*)partial, blocks, a.dim, a.dw);
}

}  // namespace

cudaError_t launch_add_norm(const AddNormArgs& a, sfa_dtype dt, bool norm, bool fp8, cudaStream_t s) {
    if (dt == SFA_BF16)
        return !norm ? launch_rows<__nv_bfloat16, To::kFp8AsIs>(a, s)
               : fp8 ? launch_rows<__nv_bfloat16, To::kFp8>(a, s)
                     : launch_rows<__nv_bfloat16, To::kSame>(a, s);
    return !norm ? launch_rows<float, To::kFp8AsIs>(a, s)
           : fp8 ? launch_rows<float, To::kFp8>(a, s)
                 : launch_rows<float, To::kSame>(a, s);
}

size_t add_norm_bwd_workspace(sfa_dtype dt, int N, int dim) {
    const int blocks = dt == SFA_BF16 ? bwd_blocks<__nv_bfloat16>(N, dim) : bwd_blocks<float>(N, dim);
    return blocks > 1 ? (size_t)blocks * dim * sizeof(float) : 0;
}

cudaError_t launch_add_norm_bwd(const AddNormBwdArgs& a, sfa_dtype dt, void* ws, cudaStream_t s) {
    return dt == SFA_BF16 ? launch_bwd<__nv_bfloat16>(a, static_cast<float*>(ws), s)
                          : launch_bwd<float>(a, static_cast<float*>(ws), s);
}

}  // namespace sfa
