// sfa_append.cu -- one step's keys and values into a paged cache, with the
// norm and rotation of the keys (and of the step's queries) on the way
// (sfa_paged_append in include/sfa.h).
//
// A copy with arithmetic, bound by memory when there are many tokens and by
// the latency of its lookups (cu_q and seq_lens -> block_table and the rotation's
// angles) in a decode step: what does not depend on a lookup is loaded before it
// (256 tokens 2.4 us; with the weights and angles loaded last 2.6), and each lane
// looks its own token up first (2.2).  Blocks that
// go through consecutive tokens and copy the next step's rows ahead, as the norm
// does for many tokens, are slower here (14.9 against 13.0 us for 16 prompts of
// up to 2048 tokens, 26.5 against 22.5 us for 32768 tokens, before the order of
// the loads; 12.5 us now): the lookups of a step stand in line with its copies.
// Four lanes hold a head row (sfa_heads.cuh); a quad of lanes handles two rows
// of one token: queries 0-1, 2-3, 4-5, 6-7, keys 0-1, values 0-1.
#include "sfa_heads.cuh"
#include "sfa_paged.cuh"

namespace sfa {

namespace {

using namespace heads;

constexpr int kThreads = 96;  // 24 quads: 4 tokens with queries, 12 without

// kQ: the step's queries are transformed too.
template <typename T, bool kQ>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendArgs a) {
    constexpr int kRoles = kQ ? kHq / 2 + 2 : 2;  // quads of a token
    constexpr int kKey = kRoles - 2, kValue = kRoles - 1;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int quad = blockIdx.x * (kThreads / 4) + (threadIdx.x >> 2), c = threadIdx.x & 3;
    const int t = quad / kRoles, role = quad - t * kRoles;
    const int warp_t = __shfl_sync(kFull, t, 0);
    if (warp_t >= a.c.N) return;
    const bool in_n = t < a.c.N;
    const int tt = in_n ? t : a.c.N - 1;
    // what does not depend on the lookups is loaded before them
    const T* src;
    if (role == kValue)
        src = static_cast<const T*>(a.vn) + (size_t)tt * a.vs;
    else if (role == kKey)
        src = static_cast<const T*>(a.kn) + (size_t)tt * a.ks;
    else
        src = static_cast<const T*>(a.q) + (size_t)tt * a.qs + role * 2 * kD;
    Raw<T> raw[2];
    fetch(src, c, raw[0]);
    fetch(src + kD, c, raw[1]);
    const float* wp = role == kKey ? a.wk : a.wq;
    Row w{};
    if (wp && role != kValue) w = weights(wp, c);
    bool live;
    const paged::Where x = paged::each_token(a.c, tt, in_n, warp_t, live);
    if (!live) return;
    const int pos = x.len - (x.end - tt);
    const bool good = pos >= 0 && pos < a.c.cap;
    Angles rot;
    if (a.rope && good && role != kValue) rot = angles(a.rope, pos, c);
    if (!good && c == 0 && role == kKey) paged::report(a.c.status);
    T* dst;
    if (role >= kKey) {
        if (!good) return;
        const int row = paged::page_row(a.c, x.s, pos);
        if (row < 0) {
            if (c == 0 && role == kKey) paged::report(a.c.status);
            return;
        }
        dst = static_cast<T*>(role == kKey ? a.c.k : a.c.v) + (size_t)row * (kHkv * kD);
        if (role == kValue || (!a.wk && !a.rope)) {
            put(dst, c, raw[0]);
            put(dst + kD, c, raw[1]);
            return;
        }
    } else {
        dst = static_cast<T*>(a.qhat) + (size_t)t * (kHq * kD) + role * 2 * kD;
    }
    const unsigned mask = 0xfu << (threadIdx.x & 28);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        Row y = open(raw[h]);
        if (wp) scale(y, inv_rms(y, a.eps, mask), w);
        if (a.rope && good) rotate(y, rot);
        if (!good) y = Row{};
        store(dst + h * kD, c, y);
    }
}

template <typename T, bool kQ>
cudaError_t launch_append(const AppendArgs& a, cudaStream_t s) {
    const int roles = kQ ? kHq / 2 + 2 : 2, tokens = kThreads / 4 / roles;
    return launch_early(append_kernel<T, kQ>, (unsigned)((a.c.N + tokens - 1) / tokens), kThreads, 0, s, a);
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs& a, sfa_dtype dt, cudaStream_t s) {
    if (dt == SFA_BF16)
        return a.q ? launch_append<__nv_bfloat16, true>(a, s) : launch_append<__nv_bfloat16, false>(a, s);
    return a.q ? launch_append<float, true>(a, s) : launch_append<float, false>(a, s);
}

}  // namespace sfa
