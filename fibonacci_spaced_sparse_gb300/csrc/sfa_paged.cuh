// sfa_paged.cuh -- reading a paged cache's metadata (sfa_paged in sfa.h):
// which sequence a token row belongs to and which page row a position lives
// in.  Every lookup is checked here, so that metadata that is wrong leads to
// an error bit and never to an access out of range.  Private to the library.
#pragma once

#include "sfa_ops.cuh"

namespace sfa {
namespace paged {

// The last index s in [0, n) with first(s) <= x, where first() does not
// decrease and first(0) <= x is assumed (0 otherwise); the whole warp asks for
// the same x.  A 32-way search: two rounds of loads up to 1024 entries.
template <typename F>
__device__ __forceinline__ int last_at_most(int n, int x, F first) {
    const int lane = threadIdx.x & 31;
    int lo = 0, len = n;
    while (len > 1) {
        const int step = (len + 31) >> 5;
        const int at = lane * step;
        const bool le = at < len && first(lo + at) <= x;
        const int last = max(31 - __clz(__ballot_sync(kFull, le)), 0);  // -1 with no lane set
        lo += last * step;
        len = min(step, len - last * step);
    }
    return lo;
}

// The sequence that token row t belongs to, or S when it belongs to none (the
// whole warp asks for the same t).  A step in which every sequence brings one
// token is found at once.
__device__ __forceinline__ int sequence_of(const PagedArgs& c, int t) {
    if (t < c.S && fresh(c.cu + t) == t && fresh(c.cu + t + 1) == t + 1) return t;
    const int s = last_at_most(c.S, t, [&](int i) { return fresh(c.cu + i); });
    return fresh(c.cu + s) <= t && t < fresh(c.cu + s + 1) ? s : c.S;
}

// Row of the pages that holds position pos >= 0 of sequence s; -1 for a page
// number out of range.  pos < c.cap.
__device__ __forceinline__ int page_row(const PagedArgs& c, int s, int pos) {
    const int page = fresh(c.table + (size_t)s * c.max_pages + (pos >> c.shift));
    return (unsigned)page < (unsigned)c.num_pages ? (page << c.shift) + (pos & ((1 << c.shift) - 1)) : -1;
}

__device__ __forceinline__ void report(unsigned* status) {
    if (status) atomicOr(status, SFA_DEVSTAT_BAD_INDEX);
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.0f;     // raise a running maximum (log2 units) past this margin
constexpr float kFloor = -1e30f;  // running maximum before the first entry

// Arguments of the attention kernels.
struct PagedFwd {
    LayerArgs a;
    PagedArgs c;
    const void* q;
    long long qs;  // token stride of q
    void* o;
    float* lse;
};

}  // namespace paged

// The kernel for long chunks (sfa_paged_tile.cu).
cudaError_t launch_paged_tiles(const paged::PagedFwd& P, cudaStream_t s);

}  // namespace sfa
