// sfa_ops_api.cu -- the C ABI of the norm and paged-cache calls (declared in
// include/sfa.h): argument checks and dispatch.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "sfa.h"
#include "sfa_ops.cuh"

using sfa::LayerArgs;

namespace {

constexpr int kMaxT = 1 << 24;  // as sfa_forward's

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

const float2* rope_ptr(const sfa_params* p, const float* table) {
    return p->rope_theta > 0.f ? reinterpret_cast<const float2*>(table) : nullptr;
}

sfa_status launched(cudaError_t e) {
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return SFA_ERR_CUDA;
    }
    return SFA_OK;
}

// The checks of every entry point, which sfa_rung_plan makes, and the layer's
// kept rungs.
sfa_status validate(const sfa_params* p, LayerArgs* l = nullptr) {
    int n = 0, index[SFA_MAX_RUNGS], fl[SFA_MAX_RUNGS], ce[SFA_MAX_RUNGS];
    float t[SFA_MAX_RUNGS];
    const sfa_status st = sfa_rung_plan(p, &n, index, fl, t, ce);
    if (st != SFA_OK || !l) return st;
    std::memset(l, 0, sizeof(*l));
    l->B = p->B;
    l->T = p->T;
    l->W = p->W;
    l->scale = p->scale > 0.f ? p->scale : 1.0f / std::sqrt((float)p->D);
    l->alpha = p->alpha;
    l->nr = n;
    for (int i = 0; i < n; ++i) l->r[i] = sfa::Rung{fl[i], t[i], ce[i], p->rungs[index[i]], index[i]};
    return SFA_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A tensor of token rows: 16-byte aligned, its token stride (elements) at
// least the row and a multiple of 16 bytes, so that every row is loaded in
// 16-byte pieces.
bool rows_ok(const sfa_params* p, const void* x, long long stride, int heads) {
    const int es = p->dtype == SFA_BF16 ? 2 : 4;
    return x && aligned16(x) && stride >= (long long)heads * p->D && stride < (1LL << 40) && (stride * es) % 16 == 0;
}

// Checks shared by sfa_qk_norm_rope and its backward; fills the launch
// arguments.
sfa_status check_norm(const sfa_params* p, const void* Q, long long q_stride, const void* K, long long k_stride,
                      const float* wq, const float* wk, float eps, const int* positions, const float* rope_table,
                      int table_rows, unsigned* status, sfa::NormArgs* a) {
    if (!rows_ok(p, Q, q_stride, p->Hq) || !rows_ok(p, K, k_stride, p->Hkv)) return SFA_ERR_INVALID_ARG;
    if (!wq || !wk || !aligned16(wq) || !aligned16(wk) || !std::isfinite(eps) || eps < 0.f)
        return SFA_ERR_INVALID_ARG;
    if (!aligned4(positions) || !aligned4(status)) return SFA_ERR_INVALID_ARG;
    if (p->rope_theta > 0.f) {
        if (!rope_table || !aligned16(rope_table) || table_rows < 1 || table_rows > kMaxT) return SFA_ERR_INVALID_ARG;
        if (!positions && table_rows < p->T) return SFA_ERR_INVALID_ARG;
    }
    std::memset(a, 0, sizeof(*a));
    a->N = p->B * p->T;
    a->T = p->T;
    a->eps = eps;
    a->qs = q_stride;
    a->ks = k_stride;
    a->q = Q;
    a->k = K;
    a->wq = wq;
    a->wk = wk;
    a->status = status;
    if (p->rope_theta > 0.f) {
        a->positions = positions;
        a->rope = reinterpret_cast<const float2*>(rope_table);
        a->table_rows = table_rows;
    }
    return SFA_OK;
}

// The parameters of a paged call: p->B counts sequences there and p->T is a
// capacity, so their product is no token count and has no cap.
sfa_status validate_paged(const sfa_params* p, LayerArgs* l = nullptr) {
    if (!p) return SFA_ERR_INVALID_ARG;
    sfa_params one = *p;
    if (one.B > 1) one.B = 1;
    const sfa_status st = validate(&one, l);
    if (st != SFA_OK) return st;
    return p->B > kMaxT ? SFA_ERR_UNSUPPORTED : SFA_OK;
}

sfa_status check_paged(const sfa_params* p, const sfa_paged* c, unsigned* status, sfa::PagedArgs* a) {
    if (c->num_pages < 1 || c->max_pages < 1 || c->page_size < 1 || (c->page_size & (c->page_size - 1)) || p->T < 1)
        return SFA_ERR_INVALID_ARG;
    if ((long long)c->num_pages * c->page_size > 0x7fffffffLL) return SFA_ERR_UNSUPPORTED;
    if (!c->k_pages || !c->v_pages || !aligned16(c->k_pages) || !aligned16(c->v_pages)) return SFA_ERR_INVALID_ARG;
    if (!c->block_table || !c->cu_q || !c->seq_lens || !aligned4(c->block_table) || !aligned4(c->cu_q) ||
        !aligned4(c->seq_lens) || !aligned4(status))
        return SFA_ERR_INVALID_ARG;
    std::memset(a, 0, sizeof(*a));
    a->k = c->k_pages;
    a->v = c->v_pages;
    a->table = c->block_table;
    a->cu = c->cu_q;
    a->lens = c->seq_lens;
    a->status = status;
    a->S = p->B;
    a->N = c->N;
    a->max_pages = c->max_pages;
    a->num_pages = c->num_pages;
    while ((1 << a->shift) < c->page_size) ++a->shift;
    const long long cap = (long long)c->max_pages * c->page_size;
    a->cap = cap < p->T ? (int)cap : p->T;
    return SFA_OK;
}

constexpr long long kMaxRows = 1LL << 28;  // token rows of a paged call, as kMaxTokens

}  // namespace

extern "C" {

SFA_API sfa_status sfa_qk_norm_rope(const sfa_params* p, const void* Q, long long q_stride, const void* K,
                                    long long k_stride, const float* wq, const float* wk, float eps,
                                    const int* positions, const float* rope_table, int table_rows, void* Qhat,
                                    void* Khat, unsigned int* status, cudaStream_t stream) {
    sfa_status st = validate(p);
    if (st != SFA_OK) return st;
    if (p->B == 0 || p->T == 0) return SFA_OK;
    sfa::NormArgs a;
    if ((st = check_norm(p, Q, q_stride, K, k_stride, wq, wk, eps, positions, rope_table, table_rows, status, &a)) !=
        SFA_OK)
        return st;
    if (!Qhat || !Khat || !aligned16(Qhat) || !aligned16(Khat)) return SFA_ERR_INVALID_ARG;
    if (sfa::fault_injected()) return SFA_ERR_CUDA;
    return launched(sfa::launch_norm_fwd(a, p->dtype, Qhat, Khat, stream));
}

SFA_API size_t sfa_qk_norm_rope_backward_workspace_size(const sfa_params* p) {
    if (validate(p) != SFA_OK || p->B == 0 || p->T == 0) return 0;
    return sfa::norm_bwd_workspace((long long)p->B * p->T);
}

SFA_API sfa_status sfa_qk_norm_rope_backward(const sfa_params* p, const void* Q, long long q_stride, const void* K,
                                             long long k_stride, const float* wq, const float* wk, float eps,
                                             const int* positions, const float* rope_table, int table_rows,
                                             const void* dQhat, const void* dKhat, void* dQ, void* dK, float* dwq,
                                             float* dwk, void* workspace, size_t workspace_bytes, unsigned int* status,
                                             cudaStream_t stream) {
    sfa_status st = validate(p);
    if (st != SFA_OK) return st;
    if (!dwq || !dwk || !aligned4(dwq) || !aligned4(dwk)) return SFA_ERR_INVALID_ARG;
    if (p->B == 0 || p->T == 0) {
        if (sfa::fault_injected()) return SFA_ERR_CUDA;
        if (cudaMemsetAsync(dwq, 0, p->D * sizeof(float), stream) != cudaSuccess ||
            cudaMemsetAsync(dwk, 0, p->D * sizeof(float), stream) != cudaSuccess)
            return launched(cudaGetLastError());
        return SFA_OK;
    }
    sfa::NormArgs a;
    if ((st = check_norm(p, Q, q_stride, K, k_stride, wq, wk, eps, positions, rope_table, table_rows, status, &a)) !=
        SFA_OK)
        return st;
    const void* ptrs[] = {dQhat, dKhat, dQ, dK};
    for (const void* x : ptrs)
        if (!x || !aligned16(x)) return SFA_ERR_INVALID_ARG;
    const size_t need = sfa::norm_bwd_workspace(a.N);
    if (need && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < need))
        return SFA_ERR_INVALID_ARG;
    if (sfa::fault_injected()) return SFA_ERR_CUDA;
    return launched(sfa::launch_norm_bwd(a, p->dtype, dQhat, dKhat, dQ, dK, dwq, dwk, workspace, stream));
}

SFA_API sfa_status sfa_paged_append(const sfa_params* p, const sfa_paged* c, const void* Q, long long q_stride,
                                    const void* K, long long k_stride, const void* V, long long v_stride,
                                    const float* wq, const float* wk, float eps, const float* rope_table, void* Qhat,
                                    unsigned int* status, cudaStream_t stream) {
    sfa_status st = validate_paged(p);
    if (st != SFA_OK) return st;
    if (!c || c->N < 0) return SFA_ERR_INVALID_ARG;
    if (c->N > kMaxRows) return SFA_ERR_UNSUPPORTED;
    if (p->B == 0 || c->N == 0) return SFA_OK;
    sfa::AppendArgs a;
    std::memset(&a, 0, sizeof(a));
    if ((st = check_paged(p, c, status, &a.c)) != SFA_OK) return st;
    if (!rows_ok(p, K, k_stride, p->Hkv) || !rows_ok(p, V, v_stride, p->Hkv)) return SFA_ERR_INVALID_ARG;
    if ((Q != nullptr) != (Qhat != nullptr)) return SFA_ERR_INVALID_ARG;
    if (Q && (!rows_ok(p, Q, q_stride, p->Hq) || !aligned16(Qhat))) return SFA_ERR_INVALID_ARG;
    if (!aligned16(wq) || !aligned16(wk) || !std::isfinite(eps) || eps < 0.f) return SFA_ERR_INVALID_ARG;
    if (p->rope_theta > 0.f && (!rope_table || !aligned16(rope_table))) return SFA_ERR_INVALID_ARG;
    a.q = Q;
    a.kn = K;
    a.vn = V;
    a.qs = q_stride;
    a.ks = k_stride;
    a.vs = v_stride;
    a.wq = wq;
    a.wk = wk;
    a.rope = rope_ptr(p, rope_table);
    a.qhat = Qhat;
    a.eps = eps;
    if (sfa::fault_injected()) return SFA_ERR_CUDA;
    return launched(sfa::launch_paged_append(a, p->dtype, stream));
}

SFA_API sfa_status sfa_paged_forward(const sfa_params* p, const sfa_paged* c, const void* Q, long long q_stride,
                                     void* O, float* lse, unsigned int* status, cudaStream_t stream) {
    LayerArgs l;
    sfa_status st = validate_paged(p, &l);
    if (st != SFA_OK) return st;
    if (!c || c->N < 0 || p->rope_theta > 0.f) return SFA_ERR_INVALID_ARG;
    if (c->N > kMaxRows) return SFA_ERR_UNSUPPORTED;
    if (p->B == 0 || c->N == 0) return SFA_OK;
    sfa::PagedArgs a;
    if ((st = check_paged(p, c, status, &a)) != SFA_OK) return st;
    if (!rows_ok(p, Q, q_stride, p->Hq) || !O || !aligned16(O) || (reinterpret_cast<uintptr_t>(lse) & 7u))
        return SFA_ERR_INVALID_ARG;
    if (sfa::fault_injected()) return SFA_ERR_CUDA;
    return launched(sfa::launch_paged_fwd(l, a, p->dtype, Q, q_stride, O, lse, stream));
}

}  // extern "C"
