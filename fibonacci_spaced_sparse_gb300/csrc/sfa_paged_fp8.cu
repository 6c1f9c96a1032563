// sfa_paged_fp8.cu -- attention of a step's tokens over a paged cache of 8-bit
// rows (sfa_paged_forward_fp8 in include/sfa.h).
#include "sfa_paged_rows.cuh"

namespace sfa {

using namespace paged;

cudaError_t launch_paged_fwd_fp8(const LayerArgs& a, const PagedArgs& c, sfa_dtype dt, const void* q, long long qs,
                                 void* o, float* lse, cudaStream_t s) {
    const PagedFwd P = {a, c, q, qs, o, lse};
    return dt == SFA_BF16 ? launch_rows<__nv_bfloat16, __nv_fp8_e4m3>(P, s) : launch_rows<float, __nv_fp8_e4m3>(P, s);
}

}  // namespace sfa
