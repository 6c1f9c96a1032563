// sfa_norm.cu -- RMS norm of every query and key head with the rotation, and
// its backward pass (sfa_qk_norm_rope in include/sfa.h).
//
// A head row x of 64 values at position i: r = 1 / sqrt(mean(x^2) + eps),
// n = x r, xhat = R(i) (w n).  Backward, with g = R(i)^T dxhat:
// dw = sum g n over tokens and heads, dx = r (w g - n mean(w g n)).
//
// Both directions are bound by memory: 640 elements a token in and out
// (forward), 640 of x and of dxhat in and 640 of dx out (backward), a few
// operations each.  Four lanes hold a row (sfa_heads.cuh); a quad of lanes
// handles two heads of one token that share their weights (queries 0-1, 2-3,
// 4-5, 6-7, keys 0-1), so five quads cover a token and the (cos, sin) of its
// position are read once for two rows.
#include "sfa_heads.cuh"

namespace sfa {

namespace {

using namespace heads;

constexpr int kTok = 16;                        // tokens of a block
constexpr int kPairsOfHeads = (kHq + kHkv) / 2;  // quads of a token
constexpr int kThreads = kTok * kPairsOfHeads * 4;

// Position of token t; -1 when it lies outside the table.
__device__ __forceinline__ int position(const NormArgs& a, int t) {
    if (!a.rope) return 0;
    const int pos = a.positions ? __ldg(a.positions + t) : t % a.T;
    return pos >= 0 && pos < a.table_rows ? pos : -1;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_fwd_kernel(const NormArgs a, T* __restrict__ qhat,
                                                            T* __restrict__ khat) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int quad = threadIdx.x >> 2, c = threadIdx.x & 3;
    const int hp = quad % kPairsOfHeads;
    const bool is_q = hp < kHq / 2;
    const int t = blockIdx.x * kTok + quad / kPairsOfHeads;
    const bool live = t < a.N;
    const int tt = live ? t : a.N - 1;  // idle lanes repeat the last token and store nothing
    const T* src = is_q ? static_cast<const T*>(a.q) + (size_t)tt * a.qs + hp * 2 * kD
                        : static_cast<const T*>(a.k) + (size_t)tt * a.ks;
    T* dst = is_q ? qhat + (size_t)tt * (kHq * kD) + hp * 2 * kD : khat + (size_t)tt * (kHkv * kD);
    Raw<T> raw[2];
    fetch(src, c, raw[0]);
    fetch(src + kD, c, raw[1]);
    const Row w = weights(is_q ? a.wq : a.wk, c);
    const int pos = position(a, tt);
    Angles rot;
    if (a.rope) rot = angles(a.rope, max(pos, 0), c);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        Row x = open(raw[h]);
        const float r = inv_rms(x, a.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x.x[j] = x.x[j] * r * w.x[j];
            x.y[j] = x.y[j] * r * w.y[j];
        }
        if (a.rope) rotate(x, rot);
        if (pos < 0) x = Row{};
        if (live) store(dst + h * kD, c, x);
    }
    if (pos < 0 && live && c == 0 && hp == 0 && a.status) atomicOr(a.status, SFA_DEVSTAT_BAD_INDEX);
}

// -------------------------------------------------------------- backward

constexpr int kMaxBlocks = 608;          // partial sums of dw (4 a SM at 152 SMs)
constexpr int kPartial = 2 * kD;         // floats of one: dwq, dwk

// Block b writes dx of its tokens (b, b + gridDim, ... in groups of kTok) and
// its part of dwq, dwk to partial[b]; dw is summed by the launch after it, in
// a fixed order.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_bwd_kernel(const NormArgs a, const T* __restrict__ dqhat,
                                                            const T* __restrict__ dkhat, T* __restrict__ dq,
                                                            T* __restrict__ dk, float* __restrict__ partial) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float sums[kTok * kPairsOfHeads][kD + 1];
    const int quad = threadIdx.x >> 2, c = threadIdx.x & 3;
    const int hp = quad % kPairsOfHeads;
    const bool is_q = hp < kHq / 2;
    const Row w = weights(is_q ? a.wq : a.wk, c);
    Row dw{};
    for (int t0 = blockIdx.x * kTok; t0 < a.N; t0 += gridDim.x * kTok) {
        const int t = t0 + quad / kPairsOfHeads;
        const bool live = t < a.N;
        const int tt = live ? t : a.N - 1;
        const T* src = is_q ? static_cast<const T*>(a.q) + (size_t)tt * a.qs + hp * 2 * kD
                            : static_cast<const T*>(a.k) + (size_t)tt * a.ks;
        const size_t at = is_q ? (size_t)tt * (kHq * kD) + hp * 2 * kD : (size_t)tt * (kHkv * kD);
        const T* up = (is_q ? dqhat : dkhat) + at;
        T* dst = (is_q ? dq : dk) + at;
        Raw<T> rx[2], rg[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            fetch(src + h * kD, c, rx[h]);
            fetch(up + h * kD, c, rg[h]);
        }
        const int pos = position(a, tt);
        Angles rot;
        if (a.rope) rot = angles(a.rope, max(pos, 0), c);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            Row x = open(rx[h]), g = open(rg[h]);
            if (a.rope) rotate_back(g, rot);
            const float r = inv_rms(x, a.eps);
            const bool counts = live && pos >= 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x.x[j] *= r;
                x.y[j] *= r;
                dw.x[j] += counts ? g.x[j] * x.x[j] : 0.f;
                dw.y[j] += counts ? g.y[j] * x.y[j] : 0.f;
                g.x[j] *= w.x[j];
                g.y[j] *= w.y[j];
            }
            const float m = dot(g, x) * (1.f / kD);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                g.x[j] = r * (g.x[j] - x.x[j] * m);
                g.y[j] = r * (g.y[j] - x.y[j] * m);
            }
            if (pos < 0) g = Row{};
            if (live) store(dst + h * kD, c, g);
        }
        if (pos < 0 && live && c == 0 && hp == 0 && a.status) atomicOr(a.status, SFA_DEVSTAT_BAD_INDEX);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        sums[quad][8 * c + j] = dw.x[j];
        sums[quad][kPairs + 8 * c + j] = dw.y[j];
    }
    __syncthreads();
    if (threadIdx.x < kPartial) {
        const int d = threadIdx.x & (kD - 1);
        const bool of_q = threadIdx.x < kD;
        float s = 0.f;
        for (int tk = 0; tk < kTok; ++tk) {
            if (of_q) {
#pragma unroll
                for (int p = 0; p < kHq / 2; ++p) s += sums[tk * kPairsOfHeads + p][d];
            } else {
                s += sums[tk * kPairsOfHeads + kHq / 2][d];
            }
        }
        partial[(size_t)blockIdx.x * kPartial + threadIdx.x] = s;
    }
}

// dwq, dwk: the sum of the blocks' parts.  A block sums 16 columns, 32 threads
// a column.
constexpr int kFinCols = 16, kFinRows = 32;
__global__ void __launch_bounds__(kFinCols* kFinRows) norm_dw_kernel(const float* __restrict__ partial, int blocks,
                                                                     float* __restrict__ dwq, float* __restrict__ dwk) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float sums[kFinRows][kFinCols + 1];
    const int col = threadIdx.x % kFinCols, row = threadIdx.x / kFinCols;
    const int d = blockIdx.x * kFinCols + col;
    float s = 0.f;
    for (int b = row; b < blocks; b += kFinRows) s += partial[(size_t)b * kPartial + d];
    sums[row][col] = s;
    __syncthreads();
    if (row == 0) {
        s = 0.f;
        for (int r = 0; r < kFinRows; ++r) s += sums[r][col];
        (d < kD ? dwq : dwk)[d & (kD - 1)] = s;
    }
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), unsigned grid, unsigned threads, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e == cudaSuccess) count_launch();
    return e;
}

unsigned blocks_of(int N) { return (unsigned)((N + kTok - 1) / kTok); }

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a, sfa_dtype dt, void* qhat, void* khat, cudaStream_t s) {
    if (dt == SFA_BF16)
        return launch(norm_fwd_kernel<__nv_bfloat16>, blocks_of(a.N), kThreads, s, a, (__nv_bfloat16*)qhat,
                      (__nv_bfloat16*)khat);
    return launch(norm_fwd_kernel<float>, blocks_of(a.N), kThreads, s, a, (float*)qhat, (float*)khat);
}

size_t norm_bwd_workspace() { return (size_t)kMaxBlocks * kPartial * sizeof(float); }

cudaError_t launch_norm_bwd(const NormArgs& a, sfa_dtype dt, const void* dqhat, const void* dkhat, void* dq, void* dk,
                            float* dwq, float* dwk, void* ws, cudaStream_t s) {
    const unsigned blocks = blocks_of(a.N) < (unsigned)kMaxBlocks ? blocks_of(a.N) : (unsigned)kMaxBlocks;
    float* partial = static_cast<float*>(ws);
    cudaError_t e;
    if (dt == SFA_BF16)
        e = launch(norm_bwd_kernel<__nv_bfloat16>, blocks, kThreads, s, a, (const __nv_bfloat16*)dqhat,
                   (const __nv_bfloat16*)dkhat, (__nv_bfloat16*)dq, (__nv_bfloat16*)dk, partial);
    else
        e = launch(norm_bwd_kernel<float>, blocks, kThreads, s, a, (const float*)dqhat, (const float*)dkhat,
                   (float*)dq, (float*)dk, partial);
    if (e != cudaSuccess) return e;
    return launch(norm_dw_kernel, (unsigned)(kPartial / kFinCols), (unsigned)(kFinCols * kFinRows), s,
                  (const float*)partial, (int)blocks, dwq, dwk);
}

}  // namespace sfa
