// sfa_paged.cuh -- reading a paged cache's metadata (sfa_paged in sfa.h):
// which sequence a token row belongs to and which page row a position lives
// in.  Every lookup is checked here, so that metadata that is wrong leads to
// an error bit and never to an access out of range.  Private to the library.
#pragma once

#include "sfa_ops.cuh"

namespace sfa {
namespace paged {

// A sequence, its first and its last row's successor and its length.
struct Where {
    int s, start, end, len;
};

// Those of sequence s, loaded together, used or not: a chain of dependent
// lookups is what a short step's time consists of.  A length below 0 counts as
// 0 (no token's position is then in range, as with the length itself): len -
// (end - t) and the sums that the kernels form with it cannot pass the lowest
// int that way and come out as a position that exists.
__device__ __forceinline__ Where look(const PagedArgs& c, int s) {
    const Where x = {s, fresh(c.cu + s), fresh(c.cu + s + 1), max(fresh(c.lens + s), 0)};
    asm volatile("" ::"r"(x.start), "r"(x.end), "r"(x.len));  // none of the loads moves behind a branch
    return x;
}

// The last sequence s with first(cu[s], s) <= x, where first() does not
// decrease with s and is at most x for s = 0 (sequence 0 otherwise); the whole
// warp asks for the same x.  A 32-way search: one round of loads up to 32
// sequences, two up to 1024.
template <typename F>
__device__ __forceinline__ Where last_at_most(const PagedArgs& c, int x, F first) {
    const int lane = threadIdx.x & 31;
    auto last = [](bool le) { return max(31 - __clz(__ballot_sync(kFull, le)), 0); };  // -1 with no lane set
    int lo = 0, len = c.S;
    while (len > 32) {
        const int step = (len + 31) >> 5, at = lane * step;
        const int k = last(at < len && first(fresh(c.cu + lo + min(at, len - 1)), lo + at) <= x);
        lo += k * step;
        len = min(step, len - k * step);
    }
    const Where y = look(c, lo + min(lane, len - 1));
    const int k = last(lane < len && first(y.start, lo + lane) <= x);
    return Where{lo + k, __shfl_sync(kFull, y.start, k), __shfl_sync(kFull, y.end, k), __shfl_sync(kFull, y.len, k)};
}

// The sequence that token row t belongs to, or S when it belongs to none (the
// whole warp asks for the same t).
__device__ __forceinline__ Where search(const PagedArgs& c, int t) {
    Where x = last_at_most(c, t, [](int start, int) { return start; });
    if (t < x.start || t >= x.end) x.s = c.S;
    return x;
}

// The same; a step in which every sequence brings one token is found at once.
__device__ __forceinline__ Where sequence_of(const PagedArgs& c, int t) {
    if (t < c.S) {
        const Where x = look(c, t);
        if (x.start == t && x.end == t + 1) return x;
    }
    return search(c, t);
}

// The sequence of each lane's own token row tt (min(t, N - 1) of a row t that rises
// with the lane; in_n: t < N), warp_t the first lane's t; live: it belongs to one.  A step
// in which every sequence brings one token takes one round of loads.
__device__ __forceinline__ Where each_token(const PagedArgs& c, int tt, bool in_n, int warp_t, bool& live) {
    Where x{};
    bool found = false;
    live = in_n;
    if (warp_t < c.S) {
        x = look(c, min(tt, c.S - 1));
        found = x.start == tt && x.end == tt + 1;
    }
    if (__all_sync(kFull, found || !in_n)) return x;
    // the sequence of the warp's first token, then the next one, and a search for
    // tokens that lie further on (there may be any number of sequences without
    // a token between two of a warp's few tokens)
    live = live && tt < fresh(c.cu + c.S);
    x = search(c, warp_t);
    if (x.s >= c.S) {  // it lies behind the last sequence, and so do the others
        live = false;
        return x;
    }
    if (live && x.end <= tt && x.s + 1 < c.S) x = look(c, x.s + 1);
    for (unsigned behind; (behind = __ballot_sync(kFull, live && x.end <= tt)) != 0u;) {
        const Where y = search(c, __shfl_sync(kFull, tt, __ffs(behind) - 1));
        if (live && x.end <= tt) {
            x = y;
            live = y.s < c.S;  // with offsets that decrease a token may be in none
        }
    }
    return x;
}

// Row of the pages that holds position pos >= 0 of sequence s; -1 for a page
// number out of range.  pos < c.cap.
__device__ __forceinline__ int page_row(const PagedArgs& c, int s, int pos) {
    const int page = fresh(c.table + (size_t)s * c.max_pages + (pos >> c.shift));
    return (unsigned)page < (unsigned)c.num_pages ? (page << c.shift) + (pos & ((1 << c.shift) - 1)) : -1;
}

// The same where it is wanted, -1 elsewhere (pos may be anything there).  No
// branch, so that several lookups are on their way together; an unwanted one
// reads the sequence's first entry.
__device__ __forceinline__ int page_row_if(const PagedArgs& c, int s, int pos, bool want) {
    const int page = fresh(c.table + (size_t)s * c.max_pages + (want ? pos >> c.shift : 0));
    const bool in = want && (unsigned)page < (unsigned)c.num_pages;
    return in ? (page << c.shift) + (pos & ((1 << c.shift) - 1)) : -1;
}

// The scales of the block of 8-bit rows that holds a row of the pages: of its
// keys, a head each, then of its values.
__device__ __forceinline__ float* row_scales(const PagedArgs& c, int row) {
    return c.scales + (size_t)((unsigned)row >> c.block_shift) * (2 * kHkv);
}

__device__ __forceinline__ void report(unsigned* status) {
    if (status) atomicOr(status, SFA_DEVSTAT_BAD_INDEX);
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.0f;     // raise a running maximum (log2 units) past this margin
// Running maximum before the first entry: the lowest finite value, so that any
// score raises it or lies within the margin of it, and -infinity, which marks
// what is no entry, stays below it.
constexpr float kFloor = -3.402823466e38f;

// Arguments of the attention kernels.
struct PagedFwd {
    LayerArgs a;
    PagedArgs c;
    const void* q;
    long long qs;  // token stride of q
    void* o;
    float* lse;
};

// What goes with bf16 copies of 8-bit rows (sfa_paged_fp8.cu).
constexpr int kMark = 1 << 30;
struct Copies {
    const int* marked;      // the block table, with kMark more for a page with factors other than 1
    const int* first_rows;  // [S]: the row of the copies that is position 0; the others follow it
};

}  // namespace paged

// The kernel for long chunks (sfa_paged_tile.cu).  copies: of pages that are bf16 copies
// of 8-bit rows.
cudaError_t launch_paged_tiles(const paged::PagedFwd& P, const paged::Copies* copies, cudaStream_t s);

}  // namespace sfa
