// sfa_ops_api.cu -- the C ABI of the norm, paged-cache and 8-bit calls (declared
// in include/sfa.h): argument checks and dispatch.
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

// The checks of sfa_paged_append and its 8-bit form; fills the launch arguments
// (*nothing: there is nothing to launch).
sfa_status check_append(const sfa_params* p, const sfa_paged* c, const void* Q, long long q_stride, const void* K,
                        long long k_stride, const void* V, long long v_stride, const float* wq, const float* wk, float eps,
                        const float* rope_table, void* Qhat, unsigned* status, sfa::AppendArgs* a, bool* nothing) {
    *nothing = false;
    sfa_status st = validate_paged(p);
    if (st != SFA_OK) return st;
    if (!c || c->N < 0) return SFA_ERR_INVALID_ARG;
    if (c->N > kMaxRows) return SFA_ERR_UNSUPPORTED;
    if (p->B == 0 || c->N == 0) {
        *nothing = true;
        return SFA_OK;
    }
    std::memset(a, 0, sizeof(*a));
    if ((st = check_paged(p, c, status, &a->c)) != SFA_OK) return st;
    if (!rows_ok(p, K, k_stride, p->Hkv) || !rows_ok(p, V, v_stride, p->Hkv)) return SFA_ERR_INVALID_ARG;
    if ((Q != nullptr) != (Qhat != nullptr)) return SFA_ERR_INVALID_ARG;
    if (Q && (!rows_ok(p, Q, q_stride, p->Hq) || !aligned16(Qhat))) return SFA_ERR_INVALID_ARG;
    if (!aligned16(wq) || !aligned16(wk) || !std::isfinite(eps) || eps < 0.f) return SFA_ERR_INVALID_ARG;
    if (p->rope_theta > 0.f && (!rope_table || !aligned16(rope_table))) return SFA_ERR_INVALID_ARG;
    a->q = Q;
    a->kn = K;
    a->vn = V;
    a->qs = q_stride;
    a->ks = k_stride;
    a->vs = v_stride;
    a->wq = wq;
    a->wk = wk;
    a->rope = rope_ptr(p, rope_table);
    a->qhat = Qhat;
    a->eps = eps;
    return SFA_OK;
}

// Those of sfa_paged_forward and its 8-bit form.
sfa_status check_forward(const sfa_params* p, const sfa_paged* c, const void* Q, long long q_stride, const void* O,
                         const float* lse, unsigned* status, LayerArgs* l, sfa::PagedArgs* a, bool* nothing) {
    *nothing = false;
    sfa_status st = validate_paged(p, l);
    if (st != SFA_OK) return st;
    if (!c || c->N < 0 || p->rope_theta > 0.f) return SFA_ERR_INVALID_ARG;
    if (c->N > kMaxRows) return SFA_ERR_UNSUPPORTED;
    if (p->B == 0 || c->N == 0) {
        *nothing = true;
        return SFA_OK;
    }
    if ((st = check_paged(p, c, status, a)) != SFA_OK) return st;
    if (!rows_ok(p, Q, q_stride, p->Hq) || !O || !aligned16(O) || (reinterpret_cast<uintptr_t>(lse) & 7u))
        return SFA_ERR_INVALID_ARG;
    return SFA_OK;
}

// What 8-bit pages add.
sfa_status check_blocks(const sfa_paged_fp8* c, sfa::PagedArgs* a) {
    const int b = c->block_size;
    if (b < 1 || (b & (b - 1)) || b > c->pages.page_size || !c->scales || !aligned16(c->scales)) return SFA_ERR_INVALID_ARG;
    if (b < 8) return SFA_ERR_UNSUPPORTED;
    a->scales = c->scales;
    while ((1 << a->block_shift) < b) ++a->block_shift;
    return SFA_OK;
}

constexpr int kMaxDim = 1 << 14;  // columns of a row

// N rows of dim values at a stride, each loaded in 16-byte pieces.
sfa_status check_rows(sfa_dtype dtype, int N, int dim) {
    if (dtype != SFA_BF16 && dtype != SFA_F32) return SFA_ERR_INVALID_ARG;
    if (N < 0 || dim < 1) return SFA_ERR_INVALID_ARG;
    return N > kMaxRows || dim % 8 || dim > kMaxDim ? SFA_ERR_UNSUPPORTED : SFA_OK;
}
bool strided_ok(sfa_dtype dtype, int dim, const void* x, long long stride) {
    const int es = dtype == SFA_BF16 ? 2 : 4;
    return x && aligned16(x) && stride >= dim && stride < (1LL << 40) && (stride * es) % 16 == 0;
}

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
    sfa::AppendArgs a;
    bool nothing;
    const sfa_status st = check_append(p, c, Q, q_stride, K, k_stride, V, v_stride, wq, wk, eps, rope_table, Qhat, status, &a,
                                       &nothing);
    if (st != SFA_OK || nothing) return st;
    if (sfa::fault_injected()) return SFA_ERR_CUDA;
    return launched(sfa::launch_paged_append(a, p->dtype, stream));
}

SFA_API sfa_status sfa_paged_forward(const sfa_params* p, const sfa_paged* c, const void* Q, long long q_stride,
                                     void* O, float* lse, unsigned int* status, cudaStream_t stream) {
    LayerArgs l;
    sfa::PagedArgs a;
    bool nothing;
    const sfa_status st = check_forward(p, c, Q, q_stride, O, lse, status, &l, &a, &nothing);
    if (st != SFA_OK || nothing) return st;
    if (sfa::fault_injected()) return SFA_ERR_CUDA;
    return launched(sfa::launch_paged_fwd(l, a, p->dtype, Q, q_stride, O, lse, stream));
}

SFA_API sfa_status sfa_paged_append_fp8(const sfa_params* p, const sfa_paged_fp8* c, const void* Q, long long q_stride,
                                        const void* K, long long k_stride, const void* V, long long v_stride,
                                        const float* wq, const float* wk, float eps, const float* rope_table, void* Qhat,
                                        unsigned int* status, cudaStream_t stream) {
    sfa::AppendArgs a;
    bool nothing;
    sfa_status st = check_append(p, c ? &c->pages : nullptr, Q, q_stride, K, k_stride, V, v_stride, wq, wk, eps, rope_table,
                                 Qhat, status, &a, &nothing);
    if (st != SFA_OK || nothing) return st;
    if ((st = check_blocks(c, &a.c)) != SFA_OK) return st;
    if (sfa::fault_injected()) return SFA_ERR_CUDA;
    return launched(sfa::launch_paged_append_fp8(a, p->dtype, stream));
}

SFA_API size_t sfa_paged_forward_fp8_workspace_size(const sfa_params* p, const sfa_paged_fp8* c) {
    LayerArgs l;
    sfa::PagedArgs a;
    if (!c || validate_paged(p, &l) != SFA_OK || c->pages.N < 1 || c->pages.N > kMaxRows || p->B == 0 ||
        check_paged(p, &c->pages, nullptr, &a) != SFA_OK)
        return 0;
    return sfa::paged_fwd_fp8_workspace(l, a, p->dtype);
}

SFA_API sfa_status sfa_paged_forward_fp8(const sfa_params* p, const sfa_paged_fp8* c, const void* Q, long long q_stride,
                                         void* O, float* lse, void* workspace, size_t workspace_bytes, unsigned int* status,
                                         cudaStream_t stream) {
    LayerArgs l;
    sfa::PagedArgs a;
    bool nothing;
    sfa_status st = check_forward(p, c ? &c->pages : nullptr, Q, q_stride, O, lse, status, &l, &a, &nothing);
    if (st != SFA_OK || nothing) return st;
    if ((st = check_blocks(c, &a)) != SFA_OK) return st;
    const size_t need = sfa::paged_fwd_fp8_workspace(l, a, p->dtype);
    if (need && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < need))
        return SFA_ERR_INVALID_ARG;
    if (sfa::fault_injected()) return SFA_ERR_CUDA;
    return launched(sfa::launch_paged_fwd_fp8(l, a, p->dtype, Q, q_stride, O, lse, workspace, stream));
}

SFA_API sfa_status sfa_add_rms_norm(sfa_dtype dtype, int N, int dim, const void* X, long long x_stride, const void* R,
                                    long long r_stride, const float* w, float eps, void* H, void* Y, void* Y8, float* scale,
                                    cudaStream_t stream) {
    const sfa_status st = check_rows(dtype, N, dim);
    if (st != SFA_OK || N == 0) return st;
    if (!strided_ok(dtype, dim, X, x_stride) || (R && !strided_ok(dtype, dim, R, r_stride)) || !w || !aligned16(w) ||
        !std::isfinite(eps) || eps < 0.f || !aligned16(H) || (H && !R))
        return SFA_ERR_INVALID_ARG;
    if ((Y != nullptr) == (Y8 != nullptr) || !aligned16(Y) || (reinterpret_cast<uintptr_t>(Y8) & 7u)) return SFA_ERR_INVALID_ARG;
    if ((Y8 != nullptr) != (scale != nullptr) || !aligned4(scale)) return SFA_ERR_INVALID_ARG;
    const sfa::AddNormArgs a = {N, dim, x_stride, r_stride, X, R, w, eps, 1.f / (float)dim, H, Y8 ? Y8 : Y, scale};
    if (sfa::fault_injected()) return SFA_ERR_CUDA;
    return launched(sfa::launch_add_norm(a, dtype, true, Y8 != nullptr, stream));
}

SFA_API sfa_status sfa_quantize_rows_fp8(sfa_dtype dtype, int N, int dim, const void* X, long long x_stride, void* X8,
                                         float* scale, cudaStream_t stream) {
    const sfa_status st = check_rows(dtype, N, dim);
    if (st != SFA_OK || N == 0) return st;
    if (!strided_ok(dtype, dim, X, x_stride) || !X8 || (reinterpret_cast<uintptr_t>(X8) & 7u) || !scale || !aligned4(scale))
        return SFA_ERR_INVALID_ARG;
    const sfa::AddNormArgs a = {N, dim, x_stride, 0, X, nullptr, nullptr, 0.f, 1.f / (float)dim, nullptr, X8, scale};
    if (sfa::fault_injected()) return SFA_ERR_CUDA;
    return launched(sfa::launch_add_norm(a, dtype, false, true, stream));
}

SFA_API size_t sfa_add_rms_norm_backward_workspace_size(sfa_dtype dtype, int N, int dim) {
    return check_rows(dtype, N, dim) != SFA_OK || N == 0 ? 0 : sfa::add_norm_bwd_workspace(dtype, N, dim);
}

SFA_API sfa_status sfa_add_rms_norm_backward(sfa_dtype dtype, int N, int dim, const void* H, const float* w, float eps,
                                             const void* dY, const void* dH, void* dX, float* dw, void* workspace,
                                             size_t workspace_bytes, cudaStream_t stream) {
    const sfa_status st = check_rows(dtype, N, dim);
    if (st != SFA_OK) return st;
    if (!dw || !aligned16(dw)) return SFA_ERR_INVALID_ARG;
    if (N == 0) {
        if (sfa::fault_injected()) return SFA_ERR_CUDA;
        return launched(cudaMemsetAsync(dw, 0, dim * sizeof(float), stream));
    }
    if (!H || !dY || !dX || !w || !aligned16(H) || !aligned16(dY) || !aligned16(dH) || !aligned16(dX) || !aligned16(w) ||
        !std::isfinite(eps) || eps < 0.f)
        return SFA_ERR_INVALID_ARG;
    const size_t need = sfa::add_norm_bwd_workspace(dtype, N, dim);
    if (need && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < need))
        return SFA_ERR_INVALID_ARG;
    const sfa::AddNormBwdArgs a = {N, dim, H, dY, dH, w, eps, 1.f / (float)dim, dX, dw};
    if (sfa::fault_injected()) return SFA_ERR_CUDA;
    return launched(sfa::launch_add_norm_bwd(a, dtype, workspace, stream));
}

SFA_API sfa_status sfa_qkv_rope_fp8(const sfa_params* p, int d_model, const void* X8, const float* x_scale, const void* Wqkv8,
                                    const float* w_scale, const float* rope_table, void* Qhat, void* Khat, void* V,
                                    unsigned int* status, cudaStream_t stream) {
    const sfa_status st = validate(p);
    if (st != SFA_OK) return st;
    if (p->dtype != SFA_BF16) return SFA_ERR_UNSUPPORTED;
    if (d_model < 64 || d_model > kMaxDim || d_model % 64) return SFA_ERR_INVALID_ARG;
    if (p->B == 0 || p->T == 0) return SFA_OK;
    const void* ptrs[] = {X8, Wqkv8, Qhat, Khat, V};
    for (const void* x : ptrs)
        if (!x || !aligned16(x)) return SFA_ERR_INVALID_ARG;
    if (!x_scale || !w_scale || !aligned4(x_scale) || !aligned4(w_scale) || !aligned4(status)) return SFA_ERR_INVALID_ARG;
    if (p->rope_theta > 0.f && (!rope_table || !aligned16(rope_table))) return SFA_ERR_INVALID_ARG;
    const sfa::QkvFp8Args a = {p->B * p->T, p->T, d_model, X8, Wqkv8, x_scale, w_scale, rope_ptr(p, rope_table), Qhat, Khat, V,
                               status};
    if (sfa::fault_injected()) return SFA_ERR_CUDA;
    return launched(sfa::launch_qkv_fp8(a, stream));
}

}  // extern "C"
