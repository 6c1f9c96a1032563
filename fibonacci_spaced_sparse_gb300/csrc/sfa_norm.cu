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
// position are read once for two rows.  Packed fp32 arithmetic and one
// approximate root a row keep the instructions well below the memory time.
#include "sfa_heads.cuh"
#include "sfa_ops.cuh"

namespace sfa {

namespace {

using namespace heads;

constexpr int kTok = 8;                          // tokens of a block's step
constexpr int kPairsOfHeads = (kHq + kHkv) / 2;  // quads of a token
constexpr int kThreads = kTok * kPairsOfHeads * 4;

// Position of token t; -1 when it lies outside the table.
__device__ __forceinline__ int position(const NormArgs& a, int t) {
    if (!a.rope) return 0;
    const int pos = a.positions ? fresh(a.positions + t) : t % a.T;
    return pos >= 0 && pos < a.table_rows ? pos : -1;
}

// The two rows of a quad's heads in a [token][head][64] tensor.
template <typename T>
struct Rows {
    T* p;
    long long stride;  // of tokens
    __device__ T* of(int t) const { return p + (size_t)t * stride; }
};
template <typename T>
__device__ __forceinline__ Rows<const T> inputs(const NormArgs& a, int hp) {
    return hp < kHq / 2 ? Rows<const T>{static_cast<const T*>(a.q) + hp * 2 * kD, a.qs}
                        : Rows<const T>{static_cast<const T*>(a.k), a.ks};
}
template <typename T>
__device__ __forceinline__ Rows<T> dense(T* q, T* k, int hp) {
    return hp < kHq / 2 ? Rows<T>{q + hp * 2 * kD, kHq * kD} : Rows<T>{k, kHkv * kD};
}

// A bad position is reported once a token.
__device__ __forceinline__ void report(const NormArgs& a, int hp, int c) {
    if (hp == 0 && c == 0 && a.status) atomicOr(a.status, SFA_DEVSTAT_BAD_INDEX);
}

// Norm and rotation of a row at position pos (< 0: zeros).
__device__ __forceinline__ void norm_row(const NormArgs& a, Row& x, const Row& w, const Angles& rot, int pos,
                                         unsigned mask) {
    scale(x, inv_rms(x, a.eps, mask), w);
    if (a.rope) rotate(x, rot);
    if (pos < 0) x = Row{};
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) norm_fwd_kernel(const NormArgs a, T* qhat, T* khat) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int quad = threadIdx.x >> 2, c = threadIdx.x & 3, hp = quad % kPairsOfHeads;
    const int t = blockIdx.x * kTok + quad / kPairsOfHeads;
    const bool live = t < a.N;
    const int tt = live ? t : a.N - 1;  // idle lanes repeat the last token and store nothing
    const T* src = inputs<T>(a, hp).of(tt);
    T* dst = dense(qhat, khat, hp).of(tt);
    Raw<T> raw[2];
    fetch(src, c, raw[0]);
    fetch(src + kD, c, raw[1]);
    const Row w = weights(hp < kHq / 2 ? a.wq : a.wk, c);
    const int pos = position(a, tt);
    Angles rot;
    if (a.rope) rot = angles(a.rope, max(pos, 0), c);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        Row x = open(raw[h]);
        norm_row(a, x, w, rot, pos, kFull);
        if (live) store(dst + h * kD, c, x);
    }
    if (pos < 0 && live) report(a, hp, c);
}

// The same for many bf16 tokens: a bf16 lane's loads are too few bytes in
// flight for the memory's latency (45 KB a SM), so a block goes through tokens
// a grid apart and copies the next step's rows and angles to shared memory
// meanwhile, each lane its own pieces (sfa_heads.cuh): no registers, no
// barrier.
constexpr int kFwdPieces = 2 * kPieces, kSlots = kFwdPieces + 4;  // pieces of a step: rows, angles
constexpr int kAhead = 2;  // steps whose rows are on their way or in use
constexpr int kPipedBlocks = kSms * 3;
constexpr size_t kPipedSmem = (size_t)kAhead * kSlots * kThreads * sizeof(uint4);

__global__ void __launch_bounds__(kThreads, 3)
    norm_fwd_piped_kernel(const NormArgs a, __nv_bfloat16* qhat, __nv_bfloat16* khat) {
    using T = __nv_bfloat16;
    extern __shared__ uint4 slots[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int quad = threadIdx.x >> 2, c = threadIdx.x & 3, hp = quad % kPairsOfHeads;
    const unsigned mask = 0xfu << (threadIdx.x & 28);  // this quad's lanes
    const Rows<const T> in = inputs<T>(a, hp);
    const Rows<T> out = dense(qhat, khat, hp);
    const Row w = weights(hp < kHq / 2 ? a.wq : a.wk, c);
    const int step = gridDim.x * kTok;
    int next = blockIdx.x * kTok + quad / kPairsOfHeads;  // the token to copy next
    int t[kAhead], pos[kAhead];                           // of the steps on their way
    auto start = [&](int i) {
        t[i] = next;
        if (next < a.N) {
            uint4* slot = slots + i * kSlots * kThreads + threadIdx.x;
            pos[i] = position(a, next);
#pragma unroll
            for (int h = 0; h < 2; ++h) copy_row(slot + h * kPieces * kThreads, in.of(next) + h * kD, c);
            if (a.rope) copy_angles(slot + kFwdPieces * kThreads, a.rope, max(pos[i], 0), c);
            next += step;
        }
        copies_end();
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) start(i);
    for (;;) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (t[i] >= a.N) return;
            copies_wait<kAhead - 1>();
            const uint4* slot = slots + i * kSlots * kThreads + threadIdx.x;
            T* dst = out.of(t[i]);
            const int p = pos[i];
            Angles rot;
            if (a.rope) rot = take_angles(slot + kFwdPieces * kThreads);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                Row x = open(take_row(slot + h * kPieces * kThreads));
                if (h == 1) start(i);  // the slots have been read
                norm_row(a, x, w, rot, p, mask);
                store(dst + h * kD, c, x);
            }
            if (p < 0) report(a, hp, c);
        }
    }
}

// -------------------------------------------------------------- backward

// Resident blocks (of 8 tokens a step): 3 a SM at the 128 registers of bf16, 2
// at the 167 of fp32.
template <typename T>
constexpr int kBwdBlocks = kSms * (sizeof(T) == 2 ? 3 : 2);
constexpr int kMaxBlocks = kSms * 3;  // partial sums of dw
constexpr int kPartial = 2 * kD;     // floats of one: dwq, dwk

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The float at this address in the shared memory of block `rank` of the cluster.
__device__ __forceinline__ float cluster_load(const float* p, unsigned rank) {
    uint32_t at;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

// Block b writes dx of its tokens (b, b + gridDim, ... in groups of kTok) and
// its part of dwq, dwk to partial[b]; dw is summed by the launch after it, in
// a fixed order.  (Copies ahead through shared memory, as in the forward, are
// no faster here: 27.3 against 26.4 us for 32 x 1024 bf16 tokens, 75 against
// 48 us in fp32.)
// kCluster: the grid is one cluster of blocks, whose parts are summed through
// distributed shared memory by its first block, dw = partial: one launch.
template <typename T, bool kCluster>
__global__ void __launch_bounds__(kThreads, kBwdBlocks<T> / kSms)
    norm_bwd_kernel(const NormArgs a, const T* dqhat, const T* dkhat, T* dq, T* dk, float* partial, float* dwk) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float sums[kTok * kPairsOfHeads][kD + 1], part[kCluster ? kPartial : 1];
    const int quad = threadIdx.x >> 2, c = threadIdx.x & 3, hp = quad % kPairsOfHeads;
    const Rows<const T> in = inputs<T>(a, hp), up = dense(dqhat, dkhat, hp);
    const Rows<T> out = dense(dq, dk, hp);
    const Row w = weights(hp < kHq / 2 ? a.wq : a.wk, c);
    Row dw{};
    for (int t0 = blockIdx.x * kTok; t0 < a.N; t0 += gridDim.x * kTok) {
        const int t = t0 + quad / kPairsOfHeads;
        const bool live = t < a.N;
        const int tt = live ? t : a.N - 1;  // idle lanes repeat the last token; it counts once
        Raw<T> rx[2], rg[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            fetch(in.of(tt) + h * kD, c, rx[h]);
            fetch(up.of(tt) + h * kD, c, rg[h]);
        }
        const int pos = position(a, tt);
        Angles rot;
        if (a.rope) rot = angles(a.rope, max(pos, 0), c);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            Row x = open(rx[h]), g = open(rg[h]);
            if (a.rope) rotate_back(g, rot);
            const float2 r = both(inv_rms(x, a.eps));
#pragma unroll
            for (int j = 0; j < kP; ++j) {
                x.x[j] = __fmul2_rn(x.x[j], r);
                x.y[j] = __fmul2_rn(x.y[j], r);
                if (live && pos >= 0) {
                    dw.x[j] = __ffma2_rn(g.x[j], x.x[j], dw.x[j]);
                    dw.y[j] = __ffma2_rn(g.y[j], x.y[j], dw.y[j]);
                }
                g.x[j] = __fmul2_rn(g.x[j], w.x[j]);
                g.y[j] = __fmul2_rn(g.y[j], w.y[j]);
            }
            const float2 m = both(dot(g, x) * (-1.f / kD));
#pragma unroll
            for (int j = 0; j < kP; ++j) {
                g.x[j] = __fmul2_rn(__ffma2_rn(x.x[j], m, g.x[j]), r);
                g.y[j] = __fmul2_rn(__ffma2_rn(x.y[j], m, g.y[j]), r);
            }
            if (pos < 0) g = Row{};
            if (live) store(out.of(tt) + h * kD, c, g);
        }
        if (pos < 0 && live) report(a, hp, c);
    }
#pragma unroll
    for (int j = 0; j < kP; ++j) {
        sums[quad][8 * c + 2 * j] = dw.x[j].x;
        sums[quad][8 * c + 2 * j + 1] = dw.x[j].y;
        sums[quad][kPairs + 8 * c + 2 * j] = dw.y[j].x;
        sums[quad][kPairs + 8 * c + 2 * j + 1] = dw.y[j].y;
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
        if (kCluster)
            part[threadIdx.x] = s;
        else
            partial[(size_t)blockIdx.x * kPartial + threadIdx.x] = s;
    }
    if (kCluster) {
        cluster_sync();
        if (blockIdx.x == 0 && threadIdx.x < kPartial) {
            float s = 0.f;
            for (unsigned b = 0; b < gridDim.x; ++b) s += cluster_load(&part[threadIdx.x], b);
            (threadIdx.x < kD ? partial : dwk)[threadIdx.x & (kD - 1)] = s;
        }
        cluster_sync();  // no block's shared memory goes before it has been read
    }
}

// dwq, dwk: the sum of the blocks' parts.  A block sums kFinCols columns,
// kFinRows threads a column, each with all of its loads in flight at once.
constexpr int kFinCols = 8, kFinRows = 64, kFinEach = (kMaxBlocks + kFinRows - 1) / kFinRows;
__global__ void __launch_bounds__(kFinCols* kFinRows) norm_dw_kernel(const float* partial, int blocks, float* dwq,
                                                                     float* dwk) {
    __shared__ float sums[kFinRows / 4][kFinCols + 1];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int col = threadIdx.x % kFinCols, row = threadIdx.x / kFinCols;
    const int d = blockIdx.x * kFinCols + col;
    float part[kFinEach];
#pragma unroll
    for (int i = 0; i < kFinEach; ++i) {
        const int b = row + i * kFinRows;
        part[i] = b < blocks ? fresh(partial + (size_t)b * kPartial + d) : 0.f;
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
        (d < kD ? dwq : dwk)[d & (kD - 1)] = s;
    }
}

unsigned steps_of(int N) { return (unsigned)((N + kTok - 1) / kTok); }

cudaError_t launch_piped(const NormArgs& a, __nv_bfloat16* qhat, __nv_bfloat16* khat, cudaStream_t s) {
    static CtxSetting done[64];  // per device: dynamic shared memory allowed
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!ctx_setting_holds(done[dev & 63], kPipedSmem)) {
        e = cudaFuncSetAttribute(norm_fwd_piped_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPipedSmem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(norm_fwd_piped_kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
        if (e != cudaSuccess) return e;
        ctx_setting_done(done[dev & 63], kPipedSmem);
    }
    return launch_early(norm_fwd_piped_kernel, kPipedBlocks, kThreads, kPipedSmem, s, a, qhat, khat);
}

// bf16 tokens from which the piped kernel is the faster one (us, direct and
// piped): 8192 tokens 4.8 and 5.4, 12288 8.9 and 8.4, 32768 18.2 and 15.9,
// 131072 65.1 and 54.3 (92 % of the measured copy rate).
constexpr int kPipedFrom = 10240;

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a, sfa_dtype dt, void* qhat, void* khat, cudaStream_t s) {
    if (dt == SFA_F32)
        return launch_early(norm_fwd_kernel<float>, steps_of(a.N), kThreads, 0, s, a, (float*)qhat, (float*)khat);
    if (a.N >= kPipedFrom) return launch_piped(a, (__nv_bfloat16*)qhat, (__nv_bfloat16*)khat, s);
    return launch_early(norm_fwd_kernel<__nv_bfloat16>, steps_of(a.N), kThreads, 0, s, a, (__nv_bfloat16*)qhat,
                  (__nv_bfloat16*)khat);
}

// Tokens up to which one cluster of blocks does the backward pass in one launch:
// a step of eight blocks (us, two launches and one: 8 tokens 3.5 and 2.9, 64 3.5
// and 3.2, 128 3.6 and 4.4; the host's 3 us for the other launch and the
// workspace come to it).
constexpr int kClusterBlocks = 8, kClusterTo = kClusterBlocks * kTok;

size_t norm_bwd_workspace(long long N) {
    return N <= kClusterTo ? 0 : (size_t)kMaxBlocks * kPartial * sizeof(float);
}

namespace {

template <typename T>
cudaError_t launch_bwd(const NormArgs& a, const void* dqhat, const void* dkhat, void* dq, void* dk, float* dwq,
                       float* dwk, void* ws, cudaStream_t s) {
    const T *gq = static_cast<const T*>(dqhat), *gk = static_cast<const T*>(dkhat);
    T *oq = static_cast<T*>(dq), *ok = static_cast<T*>(dk);
    const unsigned steps = steps_of(a.N);
    if (a.N <= kClusterTo)
        return launch_early<true>(norm_bwd_kernel<T, true>, steps, kThreads, 0, s, a, gq, gk, oq, ok, dwq, dwk);
    const unsigned blocks = steps < (unsigned)kBwdBlocks<T> ? steps : (unsigned)kBwdBlocks<T>;
    float* partial = static_cast<float*>(ws);
    const cudaError_t e =
        launch_early(norm_bwd_kernel<T, false>, blocks, kThreads, 0, s, a, gq, gk, oq, ok, partial, (float*)nullptr);
    if (e != cudaSuccess) return e;
    return launch_early(norm_dw_kernel, (unsigned)(kPartial / kFinCols), (unsigned)(kFinCols * kFinRows), 0, s,
                  (const float*)partial, (int)blocks, dwq, dwk);
}

}  // namespace

cudaError_t launch_norm_bwd(const NormArgs& a, sfa_dtype dt, const void* dqhat, const void* dkhat, void* dq, void* dk,
                            float* dwq, float* dwk, void* ws, cudaStream_t s) {
    return dt == SFA_BF16 ? launch_bwd<__nv_bfloat16>(a, dqhat, dkhat, dq, dk, dwq, dwk, ws, s)
                          : launch_bwd<float>(a, dqhat, dkhat, dq, dk, dwq, dwk, ws, s);
}

}  // namespace sfa
