// sfa_paged_fp8.cu -- attention of a step's tokens over a paged cache of 8-bit
// rows (sfa_paged_forward_fp8 in include/sfa.h): the kernels of
// sfa_paged_fwd.cu on such rows, and the rule between them.
#include "sfa_paged_quad.cuh"
#include "sfa_paged_rows.cuh"

namespace sfa {

using namespace paged;

namespace {
constexpr int kQuadsFrom = 305;
}

cudaError_t launch_paged_fwd_fp8(const LayerArgs& a, const PagedArgs& c, sfa_dtype dt, const void* q, long long qs,
                                 void* o, float* lse, cudaStream_t s) {
    const PagedFwd P = {a, c, q, qs, o, lse};
    if (dt == SFA_BF16 && a.W <= 28 && c.N >= kQuadsFrom && c.N >= 2 * (long long)c.S) return launch_quads<RowsFp8>(P, s);
    return dt == SFA_BF16 ? launch_rows<__nv_bfloat16, __nv_fp8_e4m3>(P, s) : launch_rows<float, __nv_fp8_e4m3>(P, s);
}

}  // namespace sfa
