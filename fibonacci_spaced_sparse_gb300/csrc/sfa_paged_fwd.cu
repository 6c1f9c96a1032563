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
constexpr int kTilesEach = 32;

}  // namespace

cudaError_t launch_paged_fwd(const LayerArgs& a, const PagedArgs& c, sfa_dtype dt, const void* q, long long qs, void* o,
                             float* lse, cudaStream_t s) {
    const PagedFwd P = {a, c, q, qs, o, lse};
    // the tensor-core kernels load 32 bytes of a row at a time
    const bool wide = ((reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v)) & 31u) == 0;
    if (dt == SFA_BF16 && a.W <= 28 && wide) {
        if (quad_slots(c) > quad_wave(3) && c.N >= kTilesEach * (long long)c.S && c.shift >= 4)
            return launch_paged_tiles(P, nullptr, s);
        if (c.N >= kQuadsFrom && c.N >= 2 * (long long)c.S) return launch_quads<RowsBf16>(P, s);
    }
    return dt == SFA_BF16 ? launch_rows<__nv_bfloat16, __nv_bfloat16>(P, s) : launch_rows<float, float>(P, s);
}

}  // namespace sfa
