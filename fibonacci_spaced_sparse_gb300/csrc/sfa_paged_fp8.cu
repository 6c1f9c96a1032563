// sfa_paged_fp8.cu -- attention of a step's tokens over a paged cache of 8-bit
// rows (sfa_paged_forward_fp8 in include/sfa.h): the kernels of
// sfa_paged_fwd.cu on such rows, and the rules between them.
//
// Long chunks: a row is an entry of some ten queries' key lists and stands in as many
// tiles, and turning it from 8 bits costs more than the bytes it saves once it is in
// L2.  So the rows that the chunks can reach are turned into bf16 once, into pages of
// their own in the caller's workspace, and the kernel for long chunks of bf16 pages
// runs on those (32 x 1024 tokens: 40.4 us, and 55.0 for quads on 8-bit rows), with its
// probabilities in two parts (PairSplit; rounded to bf16 once, as over bf16 pages, 37.1 us and
// an error of O of 2.0e-3 of its norm instead of 1.7e-3).
// Sequence s reaches from position c - back on, c its rows before the step and back the
// farthest row of a key list.  Its pages start at place (cu[s] >> shift) + s * extra of
// the workspace, and at position 64 h of the sequence: all positions move by that, which
// changes no mask, since every entry of a query exists from position back on.
// A code times a power of two is exact in bf16, so a copy holds the codes times the power
// of two in their scale, and the factor that is left stands in the workspace beside it, for
// 8 rows of a head each, with a mark for every page that has one that is not 1.
// Every word of the copies' table and lengths is written, page or no page, so what
// the workspace held before reaches nothing, whatever the offsets are.
#include "sfa_paged_quad.cuh"
#include "sfa_paged_rows.cuh"

namespace sfa {

using namespace paged;

namespace {

struct Expand {
    PagedArgs c;
    uint4 *k, *v;         // bf16 rows, [places][rows of a page][Hkv][D]
    float* factors;       // [places][rows of a page / 8][2][Hkv]: what the copies leave of their scales
    int *table, *lens;    // [S][cols], [S]: the pages and lengths that the attention sees
    int *marked, *first_rows;  // [S][cols], [S]: as Copies has them
    int back, extra;      // rows, pages before a sequence's chunk
    int shift, cols;      // log2 of the rows of such a page; entries of a sequence
    int cap, places;      // positions [0, cap) exist, as it sees them; pages
    int chunks, heads;    // 32 entries each of a sequence; thread blocks of entries, in front
};

constexpr int kExpandRows = 16, kRowChunks = kHkv * kD / 16;  // of a thread block; 16-byte pieces of a row
constexpr int kExpandThreads = 2 * kExpandRows * kRowChunks;  // a piece of keys or values each

// A scale as a power of two and a factor in [1, 2).  Zero, what is not finite, and what
// leaves no room for the codes (outside of what a scale may be) stay whole.
__device__ __forceinline__ float2 parts_of(float s) {
    const unsigned u = __float_as_uint(s), e = u >> 23 & 255u;
    if (e < 127u - 100u || e > 127u + 100u) return make_float2(s, 1.f);
    return make_float2(__uint_as_float(u & 0xff800000u), __uint_as_float(u & 0x7fffffu | 0x3f800000u));
}
constexpr int kFactorShift = 3;  // log2 of the rows that share a factor (a block of rows has 8 at least)

// Whether a page's first `rows` rows, from row row0 of the cache on, have factors other than 1.
__device__ __forceinline__ bool has_factors(const PagedArgs& c, int row0, int rows) {
    bool y = false;
    for (int j = 0; j < rows; j += 1 << c.block_shift) {
        const float4 s = fresh(reinterpret_cast<const float4*>(paged::row_scales(c, row0 + j)));
        static_assert(kHkv == 2, "a block's scales are one load");
        y = y || parts_of(s.x).y != 1.f || parts_of(s.y).y != 1.f || parts_of(s.z).y != 1.f || parts_of(s.w).y != 1.f;
    }
    return y;
}

// 16 codes and their scale as bf16.
__device__ __forceinline__ void expand16(uint4 u, float s, uint4* to) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float2 v = fp8::values2(j & 1 ? w[j / 2] >> 16 : w[j / 2] & 0xffffu);
        o[j] = pack_bf16(v.x * s, v.y * s);
    }
    to[0] = make_uint4(o[0], o[1], o[2], o[3]);
    to[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

// A sequence's pages: the first that is read, the one that becomes number 0 and the last.
// The first two are the same, but where the sequence's length passes the capacity, which
// then has to stay where it is.
struct Span {
    int first, zero, last;
};
__device__ __forceinline__ Span span_of(const Expand& E, const paged::Where& x) {
    const long long before = x.len - max((long long)x.end - x.start, 0LL);  // (offsets may be anything)
    const int first = (int)(max(before - E.back, 0LL) >> E.shift);
    return Span{first, x.len > E.c.cap ? (E.c.cap - E.cap) >> E.shift : first, (min(x.len, E.c.cap) - 1) >> E.shift};
}
__device__ __forceinline__ int place_of(const Expand& E, int start, int s) { return (start >> E.shift) + s * E.extra; }

// 32 entries of a sequence in the copies' table, a warp: the places of its pages, where
// the thread blocks of those places find the sequence as well (they do unless offsets
// make no sense; a search that ends at it for two places does so for all between them).
__device__ __forceinline__ void write_entries(const Expand& E, int s, int chunk) {
    const int lane = threadIdx.x & 31, at = 32 * chunk + lane;
    const paged::Where x = paged::look(E.c, s);
    const Span y = span_of(E, x);
    const int index = at + y.zero, place = place_of(E, x.start, s) + index - y.first;
    if (at == 0) {
        E.lens[s] = x.len - (y.zero << E.shift);
        E.first_rows[s] = place << E.shift;
    }
    const bool in = at < E.cols && index >= y.first && index <= y.last && place >= 0 && place < E.places;
    const unsigned who = __ballot_sync(kFull, in);
    bool found = who != 0u;
    if (found) {
        auto finder = [&](int of) {
            return paged::last_at_most(E.c, __shfl_sync(kFull, place, of), [&](int start, int i) { return place_of(E, start, i); }).s;
        };
        found = finder(__ffs(who) - 1) == s && finder(31 - __clz(who)) == s;
    }
    int entry = -1, marked = -1;
    if (in && found) {
        const int pos = index << E.shift, row0 = paged::page_row(E.c, s, pos);
        const int rows = min(min(x.len, E.c.cap) - pos, 1 << E.shift);  // that exist
        if (row0 >= 0) {
            entry = place;
            marked = has_factors(E.c, row0, rows) ? place + paged::kMark : place;
        }
    }
    if (at < E.cols) {
        E.table[(size_t)s * E.cols + at] = entry;
        E.marked[(size_t)s * E.cols + at] = marked;
    }
}

// A thread block for 16 rows of a page.
__global__ void __launch_bounds__(kExpandThreads) expand_kernel(const __grid_constant__ Expand E) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if ((int)blockIdx.x < E.heads) {
        const int w = blockIdx.x * (kExpandThreads / 32) + (threadIdx.x >> 5), s = w / E.chunks;
        if (s < E.c.S) write_entries(E, s, w % E.chunks);
        return;
    }
    const PagedArgs& c = E.c;
    const int parts = E.shift - 4, block = blockIdx.x - E.heads, place = block >> parts, part = block & ((1 << parts) - 1);
    static_assert(kExpandRows == 1 << 4, "parts of a page");
    const paged::Where x = paged::last_at_most(c, place, [&](int start, int s) { return place_of(E, start, s); });
    const Span y = span_of(E, x);
    const int n = place - place_of(E, x.start, x.s), index = y.first + n;  // of the sequence's pages
    if (n < 0 || index > y.last) return;
    const int row0 = paged::page_row(c, x.s, index << E.shift);
    if (row0 < 0) return;
    const bool value = threadIdx.x >= kExpandThreads / 2;
    const int piece = threadIdx.x % (kExpandThreads / 2), row = part * kExpandRows + piece / kRowChunks;
    const size_t i = (size_t)row0 * kRowChunks + part * kExpandRows * kRowChunks + piece;
    const uint4 u = fresh(static_cast<const uint4*>(value ? c.v : c.k) + i);
    const int head = piece % kRowChunks / (kRowChunks / kHkv);
    const float2 s = parts_of(fresh(paged::row_scales(c, row0 + row) + (value ? kHkv : 0) + head));
    // a lane of each head and 8 rows writes their factor
    if ((row & ((1 << kFactorShift) - 1)) == 0 && piece % (kRowChunks / kHkv) == 0)
        E.factors[(((size_t)place << E.shift) + row >> kFactorShift) * (2 * kHkv) + (value ? kHkv : 0) + head] = s.y;
    expand16(u, s.x, (value ? E.v : E.k) + 2 * ((((size_t)place << E.shift) + part * kExpandRows) * kRowChunks + piece));
}

constexpr int kQuadsFrom = 305, kTilesEach = 32;  // as in sfa_paged_fwd.cu
// Tokens from which rows are expanded (us, quads and expanded: one chunk of 8000 16.9 and
// 15.7, of 12000 24.7 and 25.1; 16 chunks of 512 behind 2000 rows 17.2 and 16.6; 32 x 1024
// in pages of 64 rows 55.0 and 40.4, of 16 55.7 and 44.1).
constexpr int kExpandFrom = 7000;

// Whether a call's rows are expanded, and how.
bool expands(const LayerArgs& a, const PagedArgs& c, sfa_dtype dt, Expand* E) {
    if (dt != SFA_BF16 || a.W > 28 || c.shift < 4 || c.N < kExpandFrom || c.N < kTilesEach * (long long)c.S) return false;
    E->c = c;
    E->shift = c.shift < 6 ? c.shift : 6;
    E->back = a.W;
    for (int i = 0; i < a.nr; ++i) E->back = E->back > a.r[i].n + 1 ? E->back : a.r[i].n + 1;
    // A sequence of n new tokens is back + n + rows - 1 rows long in the copy at most: (back >>
    // shift) + 3 pages more than n >> shift.  One more, since the capacity below, which moves by
    // whole pages, can lie up to rows - 1 before the end of the table.
    E->extra = (E->back >> E->shift) + 4;
    // (at most three rows expanded for one of the chunks, and a table of no more words)
    const long long own = c.N >> E->shift, reach = (long long)c.S * E->extra, cols = own + E->extra;
    if (reach > 2 * own || cols * c.S > 4LL * c.N) return false;
    E->cols = (int)cols;
    E->places = (int)(own + reach);
    E->chunks = (E->cols + 31) / 32;
    E->heads = (int)(((long long)E->chunks * c.S + kExpandThreads / 32 - 1) / (kExpandThreads / 32));
    const int rows = 1 << E->shift;
    const long long room = cols * rows - (rows - c.cap % rows) % rows;
    E->cap = c.cap <= room ? c.cap : (int)room;
    return true;
}

size_t page_bytes(const Expand& E) { return ((size_t)E.places << E.shift) * kHkv * kD * 2; }
size_t factor_bytes(const Expand& E) { return ((size_t)E.places << E.shift >> kFactorShift) * 2 * kHkv * sizeof(float); }

}  // namespace

size_t paged_fwd_fp8_workspace(const LayerArgs& a, const PagedArgs& c, sfa_dtype dt) {
    Expand E;
    return expands(a, c, dt, &E) ? 2 * page_bytes(E) + factor_bytes(E) + 2 * ((size_t)E.cols + 1) * c.S * sizeof(int) : 0;
}

cudaError_t launch_paged_fwd_fp8(const LayerArgs& a, const PagedArgs& c, sfa_dtype dt, const void* q, long long qs,
                                 void* o, float* lse, void* ws, cudaStream_t s) {
    const PagedFwd P = {a, c, q, qs, o, lse};
    Expand E;
    if (expands(a, c, dt, &E)) {
        char* at = static_cast<char*>(ws);
        E.k = reinterpret_cast<uint4*>(at);
        E.v = reinterpret_cast<uint4*>(at + page_bytes(E));
        E.factors = reinterpret_cast<float*>(at + 2 * page_bytes(E));
        E.table = reinterpret_cast<int*>(at + 2 * page_bytes(E) + factor_bytes(E));
        E.marked = E.table + (size_t)E.cols * c.S;
        E.lens = E.marked + (size_t)E.cols * c.S;
        E.first_rows = E.lens + c.S;
        const Copies copies = {E.marked, E.first_rows};
        const cudaError_t e = launch_early(expand_kernel, (unsigned)E.heads + ((unsigned)E.places << (E.shift - 4)), kExpandThreads, 0, s, E);
        if (e != cudaSuccess) return e;
        PagedFwd B = P;
        B.c.k = E.k;
        B.c.v = E.v;
        B.c.table = E.table;
        B.c.lens = E.lens;
        B.c.max_pages = E.cols;
        B.c.num_pages = E.places;
        B.c.shift = E.shift;
        B.c.cap = E.cap;
        B.c.scales = E.factors;
        B.c.block_shift = kFactorShift;
        return launch_paged_tiles(B, &copies, s);
    }
    if (dt == SFA_BF16 && a.W <= 28 && c.N >= kQuadsFrom && c.N >= 2 * (long long)c.S) return launch_quads<RowsFp8>(P, s);
    return dt == SFA_BF16 ? launch_rows<__nv_bfloat16, __nv_fp8_e4m3>(P, s) : launch_rows<float, __nv_fp8_e4m3>(P, s);
}

}  // namespace sfa
