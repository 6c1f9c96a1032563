// sfa_paged_fwd.cu -- attention of a step's tokens over a paged cache of the
// tokens' type (sfa_paged_forward in include/sfa.h): the general kernel
// (sfa_paged_rows.cuh), the tensor-core kernel of short chunks
// (sfa_paged_quad.cuh) and the rules between them and the kernel of long chunks
// (sfa_paged_tile.cu).
#include "sfa_paged_quad.cuh"
#include "sfa_paged_rows.cuh"

namespace sfa {

namespace {

using namespace paged;

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
    return dt == SFA_BF16 ? launch_rows<__nv_bfloat16, __nv_bfloat16>(P, s) : launch_rows<float, float>(P, s);
}

}  // namespace sfa
