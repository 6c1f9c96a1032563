// sfa_paged_tile.cu -- attention over a paged cache for long chunks (bf16,
// W <= 28; sfa_paged_forward in include/sfa.h): the arithmetic of
// sfa_paged_quad.cuh with its rows in shared memory.
//
// A block takes tiles of 28 consecutive queries of one sequence and one
// key/value head, a quad to each of seven warps, the heads one after the other
// (they read the same rows, so a slot of 28 queries is looked up once).  The
// rows that a tile reads are the window block, W + 28 rows, and 29 rows a rung,
// so a row is looked up and fetched once a tile, where the quad kernel's warps
// each fetch their own.
// An eighth warp does nothing else: it looks the blocks' pages up in the block
// table and fetches the part of a block that lies in a page (pages of 16 rows
// and more) with one TMA box, rows of one head under the 128-byte swizzle, into
// a ring of three stages, an item to a stage: a tile's window with its queries,
// or four of its rungs.  A full barrier a stage counts the bytes, an empty one
// the warps that are done with it; every wait is bounded, as in sfa_ring.cuh.
//
// Rung p of an item starts at row 30 p of its stage, so the eight rows of an
// ldmatrix phase (four rungs, two queries) lie in eight different phases of
// the swizzle.  Rows that no query reads keep what the stage held before.
//
// Other ways to fill the ring, us for 32 x 1024 tokens in pages of 64 rows:
// four-row gathers (tile::gather4) 59, a box of four rows in each one's place 55
// -- a TMA instruction costs some 45 cycles of its SM whatever it fetches, and
// a tile took 153 of them; boxes of 1, 2, 4, ... 32 rows, two that overlap for
// any other number, 37.8 (44.0 in pages of 16); a map for every height, as here,
// 35.2 (39.9), and 3 us of the host's time for the maps.  Looking a slot up for
// both heads at once 34.4 (36.9), and the epilogue below, with both pairs
// staged at once and fixed addresses, 31.9 (35.1; pages of 256 rows 31.2); a
// search that ends with a sequence's metadata in hand 31.0.
// 16-byte cp.async by all warps with a barrier an item took 58 (26 M
// instructions, a third of them copies and lookups).
//
// What bounds it: with the warps' arithmetic left out it takes 21 us (the ring's
// latency: three stages a block, two blocks a SM), and the arithmetic, 1000
// instructions a quad at 16 warps a SM, hides that only in part.
//
// Queries whose result is not finite are kept in a list and redone from global
// memory when the block's tiles are done (redo_query, with the score sums in
// this kernel's order of the dimensions; a call inside the loop costs it 1 KB
// of spills a thread).
#include <cstring>

#include "sfa_paged_quad.cuh"
#include "sfa_ring.cuh"

namespace sfa {

namespace {

using namespace mma;
using paged::Pair;
using paged::PagedFwd;
using paged::Quad;
using paged::kLn2;
using paged::kLog2e;
using ring::warp_wait;

constexpr int kWarps = 7, kTQ = 4 * kWarps, kThreads = 32 * (kWarps + 1);
constexpr int kRowB = kD * 2;                   // bytes of a row of one head
constexpr int kPitch = (kTQ + 2) * kRowB;       // from rung to rung of an item
constexpr int kValues = 4 * kPitch + 4 * kRowB; // the values' part of a rung stage
constexpr int kWinRows = 56;                    // rows of a window at most (W <= 28)
constexpr int kWinValues = kWinRows * kRowB;    // the values' part of a window stage
constexpr int kQueries = 2 * kWinValues;        // its queries: (query, head) rows
constexpr int kQueryB = kTQ * kG * kRowB;
constexpr int kStageB = 2 * kValues;
constexpr int kStages = 3;
constexpr int kTaken = 256; // slots that a block takes at most
constexpr int kRedo = 256;  // queries of a block that are not finite (at least a slot's); past that, all of its queries are redone
static_assert(kRedo >= kTQ, "a block with one tile never runs over");
static_assert(kQueries + kQueryB <= kStageB && kQueries % 1024 == 0 && kStageB % 1024 == 0, "stage layout");
static_assert((kPitch / kRowB) % 8 == 6, "rungs start in different swizzle phases");

// A tile; cnt = 0: there is none (the end of the block's work).
struct Work {
    int s, g, t0, cnt, i0, last;
    int used, groups;  // rungs that its last query uses, in groups of four
};

struct Shared {
    unsigned char stage[kStages][kStageB];
    unsigned char out[kWarps][16 * kRowB];  // a quad's outputs on their way
    unsigned long long full[kStages], empty[kStages], asked;
    uint4 answer;
    // The tile of a window item.  The producer is at most three items ahead of
    // a warp that is done with its tile's last item, so four places are enough.
    Work work[4];
    int holes[kStages];                    // an item has rows in bad pages
    int redo[kRedo], redos;                // token rows x heads to redo alone
    int taken[kTaken], ntaken;             // this block's slots
    int rn[SFA_MAX_RUNGS], rc[SFA_MAX_RUNGS];
    float rt[SFA_MAX_RUNGS];
    int abort_flag;
};

constexpr int kHeights = kTQ + 1;  // boxes of 1 to 29 rows

struct TileParams {
    CUtensorMap kv[2][kHeights], q;  // keys, values
    PagedFwd f;
    int slots;
    bool split;  // a block takes one head only
};

// K and V rows of a tile in shared memory: the row addresses that this lane
// gives to ldmatrix for keys and (transposed) values, swizzle folded in.
struct SharedTile {
    uint32_t k, v;
};

template <int kN>
__device__ __forceinline__ void scores(const SharedTile& x, const Pair* U, float (*c)[4]) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        uint32_t a0, a1, a2, a3;
        ldsm_x4(x.k ^ (uint32_t)(s << 5), a0, a1, a2, a3);
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            if (s == 0)
                mma16816_z(c[k], a0, a1, a2, a3, U[k].qf[0][0], U[k].qf[0][1]);
            else
                mma16816(c[k], a0, a1, a2, a3, U[k].qf[s][0], U[k].qf[s][1]);
        }
    }
}
__device__ __forceinline__ void value_frag(const SharedTile& x, int j, uint32_t (&a)[4]) {
    ldsm_x4_t(x.v ^ (uint32_t)(j << 5), a[0], a[1], a[2], a[3]);
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

// Asks for the index of a block of this grid that has not started, which then
// never does; the answer is 16 bytes that complete on the barrier.
__device__ __forceinline__ void ask_block(uint32_t answer, uint32_t bar) {
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer),
        "r"(bar)
        : "memory");
}
// That block's index; -1: all have started.
__device__ __forceinline__ int asked_block(uint32_t answer) {
    int x;
    asm volatile(
        "{\n .reg .b128 h;\n .reg .pred p;\n ld.shared.b128 h, [%1];\n mov.s32 %0, -1;\n"
        " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n"
        " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, h;\n}\n"
        : "=r"(x)
        : "r"(answer)
        : "memory");
    return x;
}

// Address of 16-byte chunk c of the row that starts at byte `row` of shared
// memory (a multiple of 128) under the 128-byte swizzle.
__device__ __forceinline__ uint32_t swizzled(uint32_t row, int c) { return row + ((((uint32_t)c ^ (row >> 7)) & 7u) << 4); }

// The first head's tile of a slot of 28 queries: sequence s starts at slot
// cu[s] / 28 + s, which leaves room for ceil(tokens / 28) before the next's.
__device__ __forceinline__ Work work_of(const PagedFwd& P, const int* rc, int slot) {
    const int lane = threadIdx.x & 31;
    Work x;
    x.g = 0;
    const paged::Where w = paged::last_at_most(P.c, slot, [](int start, int s) { return start / kTQ + s; });
    const int start = w.start, end = w.end;
    x.s = w.s;
    x.t0 = start + kTQ * (slot - start / kTQ - x.s);
    x.cnt = x.t0 < 0 || x.t0 >= P.c.N || x.t0 >= end ? 0 : min(kTQ, min(end, P.c.N) - x.t0);
    x.i0 = w.len - (end - x.t0);
    x.last = min(x.i0 + x.cnt, P.c.cap) - 1;
    x.used = __popc(__ballot_sync(kFull, rc[lane] <= x.last));
    x.groups = (x.used + 3) >> 2;
    return x;
}

// ------------------------------------------------------------- the producer

// The part of a block of rows that a lane fetches: `rows` positions (0:
// nothing) from row `row` of the pages on, to row `at` of the block.
struct Part {
    int row, rows, at;
    bool bad;  // its page is
};

// Part `n` of the block whose row 0 is position `base` and of which the
// positions lo .. hi are read: what lies in the n-th page from lo's.
__device__ __forceinline__ Part part_of(const PagedFwd& P, int s, int base, int lo, int hi, int n) {
    const int sh = P.c.shift, index = (max(lo, 0) >> sh) + n;
    const int from = max(lo, index << sh), to = min(hi, ((index + 1) << sh) - 1);
    if (from > to) return Part{0, 0, 0, false};
    const int page = fresh(P.c.table + (size_t)s * P.c.max_pages + index);
    if ((unsigned)page >= (unsigned)P.c.num_pages) return Part{0, 0, 0, true};
    return Part{(page << sh) + (from & ((1 << sh) - 1)), to - from + 1, from - base, false};
}

// Rung r's block: row j is position i0 - n - 1 + j, the far row of query j and
// the near row of query j - 1.
__device__ __forceinline__ Part rung_part(const PagedFwd& P, const Shared& S, const Work& x, int r, int n) {
    const int c = r < SFA_MAX_RUNGS ? S.rc[r] : 0x7fffffff;
    if (c > x.last) return Part{0, 0, 0, false};
    const int back = S.rn[r] + 1, from = max(c, x.i0) + (S.rt[r] > 0.f ? 0 : 1);
    return part_of(P, x.s, x.i0 - back, from - back, x.last + 1 - back, n);
}

// kAsk: the block's slots after its own are those of blocks that have not started,
// one asked for at a time; else those a grid apart.
template <bool kAsk>
__device__ void produce(const TileParams& T, Shared& S) {
    const PagedFwd& P = T.f;
    const int lane = threadIdx.x & 31, W = P.a.W;
    const uint32_t stage0 = smem_u32(S.stage[0]), full0 = smem_u32(S.full), empty0 = smem_u32(S.empty);
    int n = 0, tile = 0;  // items, tiles
    bool ok = true;
    auto wait = [&]() {
        ok = warp_wait(empty0 + 8 * (n % kStages), ((n / kStages) & 1) ^ 1, &S.abort_flag);
        return ok;
    };
    // The next item: every lane's part, to row 0 of its block at byte `block` of
    // the stage; `more` bytes that lane 0 fetches besides.  The item's bytes are
    // announced, and what goes with them published, before the first copy starts.
    const int tensor = lane & 1;
    auto fetch = [&](const Part& y, const Work& x, uint32_t block, uint32_t more) {
        const uint32_t dst = stage0 + (uint32_t)(n % kStages) * kStageB, full = full0 + 8 * (n % kStages);
        const int high = min(max(y.rows, 1), kHeights);  // 56 rows at most: two boxes, the second may overlap
        const int boxes = y.rows == 0 ? 0 : y.rows > high ? 2 : 1;
        const uint32_t bytes = __reduce_add_sync(kFull, (unsigned)(boxes * high * kRowB)) + more;
        const bool bad = __any_sync(kFull, y.bad);
        if (lane == 0) {
            S.holes[n % kStages] = bad;
            if (bad) paged::report(P.c.status);
            mbar_arrive_expect_tx(full, bytes);
        }
        __syncwarp();
        if (more && lane == 0) tma_load_3d(dst + kQueries, &T.q, 0, x.g * kG, x.t0, full);
        const CUtensorMap* map = &T.kv[tensor][high - 1];
        const uint32_t to = dst + block + (uint32_t)y.at * kRowB;
        if (boxes > 0) tma_load_2d(to, map, x.g * kD, y.row, full);
        if (boxes > 1) tma_load_2d(to + (uint32_t)(y.rows - high) * kRowB, map, x.g * kD, y.row + y.rows - high, full);
        ++n;
    };
    // What is fetched for a tile: lanes (part, tensor) of its window, 56 rows and
    // five pages at most; lanes (block p, part, tensor) of its groups, 29 rows
    // and three pages at most.  The first groups are looked up with the window.
    constexpr int kEarly = 4;
    const int p = lane >> 3, part = (lane >> 1) & 3;
    struct Plan {
        Work x;
        Part win, run[kEarly];
    };
    const int g0 = T.split ? blockIdx.x % kHkv : 0, g1 = T.split ? g0 + 1 : kHkv;
    const int step = T.split ? T.slots : gridDim.x;
    const uint32_t answer = smem_u32(&S.answer), asked = smem_u32(&S.asked);
    int slot = T.split ? blockIdx.x / kHkv : blockIdx.x, asks = 0, taken = 0;
    bool waiting = false;
    auto ask = [&]() {
        if (!kAsk || taken == kTaken) return;
        if (lane == 0) {
            fence_proxy_async();  // the answer before has been read
            mbar_arrive_expect_tx(asked, sizeof(uint4));
            ask_block(answer, asked);
        }
        waiting = true;
    };
    auto next_slot = [&]() {
        if (!kAsk) return slot + step < T.slots ? slot + step : -1;
        if (!waiting) return -1;
        if (!warp_wait(asked, asks & 1, &S.abort_flag)) {
            ok = false;
            return -1;
        }
        ++asks;
        waiting = false;
        const int x = asked_block(answer);
        __syncwarp();
        return x;
    };
    auto plan = [&]() {
        Plan y;
        y.x.cnt = 0;
        while (slot >= 0 && y.x.cnt == 0) {
            y.x = work_of(P, S.rc, slot);
            if (y.x.cnt == 0) {
                ask();
                slot = next_slot();
            }
        }
        if (y.x.cnt == 0) return y;
        if (kAsk) {
            if (lane == 0) {
                S.taken[taken] = slot;
                S.ntaken = taken + 1;
            }
            ++taken;
        }
        y.win = part_of(P, y.x.s, y.x.i0 - W, max(0, y.x.i0 - W), y.x.last, lane >> 1);
#pragma unroll
        for (int k = 0; k < kEarly; ++k) y.run[k] = rung_part(P, S, y.x, 4 * k + p, part);
        if (lane < y.x.cnt && (y.x.i0 + lane < 0 || y.x.i0 + lane >= P.c.cap)) paged::report(P.c.status);
        return y;
    };
    const uint32_t block = tensor * kValues + p * kPitch;
    Plan y = plan(), z;
    while (ok && y.x.cnt > 0) {
        // the heads' tiles read the same rows
        for (int g = g0; ok && g < g1; ++g) {
            Work x = y.x;
            x.g = g;
            if (g == g1 - 1) ask();
            if (!wait()) break;
            if (lane == 0) S.work[tile & 3] = x;
            fetch(y.win, x, tensor * kWinValues, kQueryB);
            ++tile;
            if (x.groups > 0 && wait()) fetch(y.run[0], x, block, 0u);
            // the next slot is looked up while the warps have these items to work on
            if (g == g1 - 1) {
                slot = next_slot();
                z = plan();
            }
#pragma unroll
            for (int k = 1; k < kEarly; ++k)
                if (ok && k < x.groups && wait()) fetch(y.run[k], x, block, 0u);
            for (int k = kEarly; k < x.groups; ++k) {
                const Part more = rung_part(P, S, x, 4 * k + p, part);
                if (ok && wait()) fetch(more, x, block, 0u);
            }
        }
        y = z;
    }
    if (ok && wait()) {  // the end
        if (lane == 0) {
            S.work[tile & 3].cnt = 0;
            mbar_arrive(full0 + 8 * (n % kStages));
        }
        return;
    }
    if (lane == 0) {
        S.abort_flag = 1;
        if (P.c.status) atomicOr(P.c.status, SFA_DEVSTAT_WAIT_TIMEOUT);
        // no copy of this block may land after it is gone
        for (int i = max(0, n - kStages); i < n; ++i)
            (void)mbar_wait(full0 + 8 * (i % kStages), (i / kStages) & 1, nullptr);
        if (kAsk && waiting) (void)mbar_wait(asked, asks & 1, nullptr);
    }
    __syncwarp();
}

// ------------------------------------------------------------ the consumers

// One tile after another, until the end; false when a wait gave up.
__device__ bool consume(const TileParams& T, Shared& S) {
    const PagedFwd& P = T.f;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g8 = lane >> 2, tig = lane & 3;
    const int W = P.a.W, u0 = 4 * warp;
    const float sl2 = P.a.scale * kLog2e;
    const uint32_t stage0 = smem_u32(S.stage[0]), full0 = smem_u32(S.full), empty0 = smem_u32(S.empty);
    // ldmatrix row of this lane: keys row (lane & 7) + 8 ((lane >> 3) & 1), half
    // lane >> 4 of a 32-byte step; values row (lane & 7) + 8 (lane >> 4), half
    // (lane >> 3) & 1.  Row m of a rung tile is rung m & 3, query (m >> 2) & 1,
    // far row for m < 8.  Stages start at multiples of 1024 bytes, so offsets in
    // a stage carry the swizzle.
    const int km = (lane & 7) + (((lane >> 3) & 1) << 3), vm = (lane & 7) + ((lane >> 4) << 3);
    const int kh = lane >> 4, vh = (lane >> 3) & 1;
    auto rung_at = [&](int k, int np) {
        const int p = (lane & 3) < np ? (lane & 3) : 0, e = (lane >> 2) & 1, u = u0 + 2 * k;
        auto row = [&](int j) { return (uint32_t)(p * kPitch + j * kRowB); };
        return SharedTile{swizzled(row(u + e + (km >> 3)), kh), swizzled(row(u + e + (vm >> 3)) + kValues, vh)};
    };
    auto window_at = [&](int wt) {
        const uint32_t kr = min(u0 + 16 * wt + km, W + kTQ - 1), vr = min(u0 + 16 * wt + vm, W + kTQ - 1);
        return SharedTile{swizzled(kr * kRowB, kh), swizzled(kWinValues + vr * kRowB, vh)};
    };
    // bit e: row 16 wt + 8 (e & 1) + g8 of the window is at a distance 0 .. W of
    // this thread's query of pair e / 2
    auto window_mask = [&](int wt, auto there) {
        unsigned m = 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int R = 16 * wt + 8 * (e & 1) + g8, d = R - 2 * (e >> 1) - (tig >> 1);
            if (d >= 0 && d <= W && there(R)) m |= 1u << e;
        }
        return m;
    };
    const SharedTile whole[2] = {rung_at(0, 4), rung_at(1, 4)}, first = window_at(0);
    const unsigned mask0 = window_mask(0, [](int) { return true; });
    // outputs: stmatrix rows of this lane in the staging buffer, its 16-byte piece
    // of query row 8 k + 4 e + lane / 8 there
    const uint32_t out = smem_u32(S.out[warp]);
    const int mi = lane >> 3;
    const uint32_t put = swizzled(out + (lane & 7) * kRowB, mi);           // chunks mi and 4 + mi
    const uint32_t get = swizzled(out + (lane >> 3) * kRowB, lane & 7);    // row lane / 8; row + 4: chunk ^ 4
    int st_index = 0, phase = 0, tile = 0;
    auto done_with_stage = [&]() {
        __syncwarp();
        mbar_arrive_if(empty0 + 8 * st_index, lane == 0);
        if (++st_index == kStages) {
            st_index = 0;
            phase ^= 1;
        }
    };
    for (;; ++tile) {
        if (!warp_wait(full0 + 8 * st_index, phase, &S.abort_flag)) return false;
        const Work& x = S.work[tile & 3];
        const int cnt = x.cnt, i0 = x.i0, groups = x.groups;
        if (cnt == 0) return true;
        const bool mine = u0 < cnt;
        Pair U[2];
        if (mine) {
            const uint32_t st = stage0 + (uint32_t)st_index * kStageB;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                // column g8 of a pair is row 4 u + g8 of the queries; matrix i of the loads is chunk i
                const uint32_t at = swizzled(st + kQueries + (uint32_t)((4 * (u0 + 2 * k) + (lane & 7)) * kRowB), mi);
                ldsm_x4(at, U[k].qf[0][0], U[k].qf[0][1], U[k].qf[1][0], U[k].qf[1][1]);
                ldsm_x4(at ^ 64u, U[k].qf[2][0], U[k].qf[2][1], U[k].qf[3][0], U[k].qf[3][1]);
            }
            const bool holes = S.holes[st_index];
            const int lo = W - i0 - u0;  // rows before it lie before the sequence
            auto there = [&](int R) {
                if (R < lo) return false;
                const int pos = R - lo;
                return !holes || (pos <= x.last && paged::page_row(P.c, x.s, pos) >= 0);
            };
            const unsigned m = lo > 0 || holes ? window_mask(0, there) : mask0;
            paged::window_tile<true>(SharedTile{first.k + st, first.v + st}, m, sl2, U);
            if (W > 12) {
                const SharedTile X = window_at(1);
                paged::window_tile<false>(SharedTile{X.k + st, X.v + st}, window_mask(1, there), sl2, U);
            }
        }
        done_with_stage();
        const int my_i = (g8 >> 2) == (tig >> 1) ? i0 + u0 + (tig >> 1) : -(1 << 30);
        for (int k = 0; k < groups; ++k) {
            if (!warp_wait(full0 + 8 * st_index, phase, &S.abort_flag)) return false;
            if (mine) {
                const uint32_t st = stage0 + (uint32_t)st_index * kStageB;
                const int r = 4 * k + (g8 & 3), np = x.used - 4 * k;
                const float frac = S.rt[r];
                const int c = S.rc[r];
                bool ok[2] = {my_i >= c, my_i + 2 >= c};
                if (S.holes[st_index]) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int pos = my_i + 2 * i - S.rn[r];
                        ok[i] = ok[i] && my_i + 2 * i <= x.last && paged::page_row(P.c, x.s, pos) >= 0 &&
                                (frac == 0.f || paged::page_row(P.c, x.s, pos - 1) >= 0);
                    }
                }
                SharedTile X[2] = {whole[0], whole[1]};
                if (np < 4) {  // absent rungs read the first one's rows, masked
                    X[0] = rung_at(0, np);
                    X[1] = rung_at(1, np);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    X[i].k += st;
                    X[i].v += st;
                }
                paged::rung_tiles<2>(X, ok, frac, sl2, U);
            }
            done_with_stage();
        }
        if (!mine) continue;
        // positions that are out of range
        const int live = min(4, cnt - u0), i1 = i0 + u0;
        unsigned out_of = 0u;
        if (i1 < 0 || i1 + live > P.c.cap)
            for (int e = 0; e < 4; ++e) out_of |= (i1 + e < 0 || i1 + e >= P.c.cap ? 1u : 0u) << e;
        unsigned redo = 0;
        float2 l[2] = {U[0].l, U[1].l}, f[2];
#pragma unroll
        for (int w = 4; w <= 16; w <<= 1)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                l[k] = __fadd2_rn(l[k], make_float2(__shfl_xor_sync(kFull, l[k].x, w), __shfl_xor_sync(kFull, l[k].y, w)));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float2 odd = make_float2(0.f, 0.f);  // stays 0 while every value is finite
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                odd = __ffma2_rn(make_float2(U[k].o[j][0], U[k].o[j][1]), make_float2(0.f, 0.f), odd);
                odd = __ffma2_rn(make_float2(U[k].o[j][2], U[k].o[j][3]), make_float2(0.f, 0.f), odd);
            }
            const unsigned who = __ballot_sync(kFull, odd.x + odd.y != 0.f);
            redo |= ((who & 0x33333333u ? 1u : 0u) | (who & 0xccccccccu ? 2u : 0u)) << (2 * k);
            // l >= 2^-8 (the entry at the maximum, at most the margin below it), or 0 with no entry: zeros
            f[k] = make_float2(l[k].x != 0.f ? fast_rcp(l[k].x) : 0.f, l[k].y != 0.f ? fast_rcp(l[k].y) : 0.f);
        }
        redo &= (1u << live) - 1u & ~out_of;
        // transposed into rows (query, head), then out in 16-byte pieces that cover a
        // query's four heads
        __syncwarp();  // the tile before has been read
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t r[4][2];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 a = __fmul2_rn(make_float2(U[k].o[j][0], U[k].o[j][1]), f[k]);
                const float2 c = __fmul2_rn(make_float2(U[k].o[j][2], U[k].o[j][3]), f[k]);
                r[j][0] = pack_bf16(a.x, a.y);
                r[j][1] = pack_bf16(c.x, c.y);
            }
            if (out_of >> (2 * k + (tig >> 1)) & 1u) {  // zeros (a sum that is not finite would survive f = 0)
#pragma unroll
                for (int j = 0; j < 4; ++j) r[j][0] = r[j][1] = 0u;
            }
            stsm_x4_t(put + k * 8 * kRowB, r[0][0], r[0][1], r[1][0], r[1][1]);
            stsm_x4_t((put ^ 64u) + k * 8 * kRowB, r[2][0], r[2][1], r[3][0], r[3][1]);
        }
        __syncwarp();
        const size_t at = (size_t)(x.t0 + u0) * kHq + x.g * kG;
        uint4* o = reinterpret_cast<uint4*>(P.o) + (at + (lane >> 3)) * (kD / 8) + (lane & 7);
        const unsigned write = (1u << live) - 1u & ~redo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint4 v = ring::lds_u4((get ^ (e & 1 ? 64u : 0u)) + e * 4 * kRowB);
            if (write >> e & 1u) o[e * (kHq * kD / 8)] = v;
        }
        if (P.lse && g8 < 2) {  // lanes g8 = k: queries of pair k
            const float2 s = g8 == 0 ? l[0] : l[1], nm = g8 == 0 ? U[0].nm : U[1].nm;
            const int e = 2 * g8 + (tig >> 1);
            float2 v = make_float2(s.x != 0.f ? (__log2f(s.x) - nm.x) * kLn2 : -INFINITY,
                                   s.y != 0.f ? (__log2f(s.y) - nm.y) * kLn2 : -INFINITY);
            if (out_of >> e & 1u) v = make_float2(0.f, 0.f);
            if (e < live) *reinterpret_cast<float2*>(P.lse + at + e * kHq + 2 * (tig & 1)) = v;
        }
        if (lane < 4 && (redo >> lane & 1u)) {
            const int i = atomicAdd(&S.redos, 1);
            if (i < kRedo) S.redo[i] = (x.t0 + u0 + lane) * kHkv + x.g;
        }
    }
}

// Token row t alone, as the quad that it stands in computes it.  (One for each
// kernel: ptxas ends in a fault over a function that both call.)
template <bool kAsk>
__device__ __noinline__ void redo_query(const PagedFwd& P, const Shared& S, int t, int g) {
    const paged::Where x = paged::sequence_of(P.c, t);
    if (x.s >= P.c.S) return;
    Quad Q;
    Q.s = x.s;
    const int only = (t - x.start) & 3;
    Q.t0 = t - only;
    Q.cnt = min(4, min(x.end, P.c.N) - Q.t0);
    Q.i0 = x.len - (x.end - Q.t0);
    Q.last = min(Q.i0 + Q.cnt, P.c.cap) - 1;
    Q.g = g;
    Q.rn = S.rn;
    Q.rc = S.rc;
    Q.rt = S.rt;
    paged::quad_pass<true, true>(P, Q, only);
}

template <bool kAsk>
__global__ void __launch_bounds__(kThreads, 2) tile_kernel(const __grid_constant__ TileParams T) {
    extern __shared__ unsigned char raw[];
    Shared& S = *reinterpret_cast<Shared*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5;
    if (tid < SFA_MAX_RUNGS) {
        const Rung r = T.f.a.r[tid];
        S.rn[tid] = r.n;
        S.rc[tid] = tid < T.f.a.nr ? r.c : 0x7fffffff;
        S.rt[tid] = r.t;
    }
    // (finite) values for rows that are never fetched
    for (uint32_t i = tid; i < sizeof(S.stage) / 16; i += kThreads)
        reinterpret_cast<uint4*>(S.stage)[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async();
    if (tid == 0) {
        S.redos = S.ntaken = 0;
        S.abort_flag = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&S.full[i]), 1);
            mbar_init(smem_u32(&S.empty[i]), kWarps);
        }
        mbar_init(smem_u32(&S.asked), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == kWarps) {
        produce<kAsk>(T, S);
    } else if (!consume(T, S) && (tid & 31) == 0) {
        S.abort_flag = 1;
        if (T.f.c.status) atomicOr(T.f.c.status, SFA_DEVSTAT_WAIT_TIMEOUT);
    }
    __syncthreads();
    const int redos = S.redos;
    if (redos == 0 || S.abort_flag) return;
    if (redos <= kRedo) {
        for (int i = warp; i < redos; i += kWarps + 1) redo_query<kAsk>(T.f, S, S.redo[i] / kHkv, S.redo[i] % kHkv);
        return;
    }
    // more than the list holds: only a block that goes through many slots, both heads of each
    for (int v = 0;; ++v) {
        const int slot = kAsk ? v : blockIdx.x + v * gridDim.x;
        if (slot >= (kAsk ? S.ntaken : T.slots)) break;
        const Work x = work_of(T.f, S.rc, kAsk ? S.taken[slot] : slot);
        for (int i = warp; i < x.cnt * kHkv; i += kWarps + 1) redo_query<kAsk>(T.f, S, x.t0 + i / kHkv, i % kHkv);
    }
}

// Map over the pages as rows of both heads (innermost first: dimension, row),
// box of `high` rows of one head.
bool encode_pages(CUtensorMap* m, const void* base, long long rows, int high) {
    auto fn = ring::encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)(kHkv * kD), (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(kHkv * kRowB)};
    const cuuint32_t box[2] = {(cuuint32_t)kD, (cuuint32_t)high};
    const cuuint32_t estr[2] = {1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Map over the queries (innermost first: dimension, head, token), box of 4
// heads x 28 tokens; tokens past the last are zeros.
bool encode_queries(CUtensorMap* m, const void* base, int N, long long stride) {
    auto fn = ring::encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)kHq, (cuuint64_t)N};
    const cuuint64_t strides[2] = {(cuuint64_t)kRowB, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {(cuuint32_t)kD, (cuuint32_t)kG, (cuuint32_t)kTQ};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Blocks ask for their slots where chunks are short and rounds few: slots differ
// in their work there (a chunk's first ones have few rungs, its last one few
// queries or none), and a round more or less counts.  (us, a grid apart and asked
// for: 80 chunks of up to 900 tokens after up to 900 40.9 and 36.0, 64 of 512 31.5
// and 30.2, 50 of 700 34.3 and 32.7; 30 of up to 2000 32.7 and 31.2, but 32 of 1024
// 30.8 and 31.5, 128 of 1024 102.5 and 105.3, 300 of up to 2000 253 and 255.)  What
// decides is how unequal the slots are, which the host does not know; it goes by the
// average length, and so leaves out the 30 ragged chunks for the 32 equal ones.
constexpr int kAskRounds = 6, kAskEach = 800;

}  // namespace

cudaError_t launch_paged_tiles(const PagedFwd& P, cudaStream_t s) {
    const long long slots = (long long)P.c.N / kTQ + P.c.S, most = kSms * 2;
    const bool ask = slots > most && slots <= kAskRounds * most && P.c.N <= kAskEach * (long long)P.c.S;
    void (*const kernel)(TileParams) = ask ? tile_kernel<true> : tile_kernel<false>;
    static CtxSetting done[2][64];  // per kernel and device: dynamic shared memory allowed
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    constexpr size_t smem = sizeof(Shared) + 1024;
    if (!ctx_setting_holds(done[ask][dev & 63], smem)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
        if (e != cudaSuccess) return e;
        ctx_setting_done(done[ask][dev & 63], smem);
    }
    TileParams T;
    std::memset(&T, 0, sizeof(T));
    T.f = P;
    T.slots = (int)slots;
    T.split = slots * kHkv <= most;  // fewer slots than blocks: the heads side by side
    const long long rows = (long long)P.c.num_pages << P.c.shift;
    for (int h = 0; h < kHeights; ++h)
        if (!encode_pages(&T.kv[0][h], P.c.k, rows, h + 1) || !encode_pages(&T.kv[1][h], P.c.v, rows, h + 1))
            return cudaErrorInvalidValue;
    if (!encode_queries(&T.q, P.q, P.c.N, P.qs)) return cudaErrorInvalidValue;
    return launch_early(kernel, (unsigned)(T.split ? slots * kHkv : ask || slots < most ? slots : most), kThreads, smem, s, T);
}

}  // namespace sfa
