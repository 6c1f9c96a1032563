// sfa_ops.cuh -- launch arguments of the norm and paged-cache kernels, and what
// they and the decode share to start before the launch ahead of them has ended.
// Private to the CUDA library.
#pragma once

#include "sfa_internal.cuh"

namespace sfa {

// A load of memory that the launch before this one may have written.  It is
// plain on purpose: a read-only (non-coherent) load, and so __ldg or a const
// __restrict__ argument, promises that nothing writes the memory while this
// grid is in flight, and may be moved ahead of griddepcontrol.wait.
template <typename V>
__device__ __forceinline__ V fresh(const V* p) {
    return *p;
}

constexpr int kSms = 152;  // of a GB300; grids and the rules between kernels go by it

// Launches a kernel that waits for the launch before it by itself
// (griddepcontrol.wait), so its blocks may start while that one drains.  kCluster:
// the grid is one cluster.
template <bool kCluster = false, typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t s,
                         const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {grid, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = kCluster ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e == cudaSuccess) count_launch();
    return e;
}

// Norm with rotation (sfa_norm.cu).  Token strides in elements.
struct NormArgs {
    int N, T;              // tokens; tokens per sequence (position = index % T)
    int table_rows;
    float eps;
    long long qs, ks;      // token strides
    const void *q, *k;
    const float *wq, *wk;
    const int* positions;  // nullptr: the index in the sequence
    const float2* rope;    // nullptr: no rotation
    unsigned* status;
};
cudaError_t launch_norm_fwd(const NormArgs& a, sfa_dtype dt, void* qhat, void* khat, cudaStream_t s);
size_t norm_bwd_workspace(long long N);  // N tokens; 0: none
cudaError_t launch_norm_bwd(const NormArgs& a, sfa_dtype dt, const void* dqhat, const void* dkhat, void* dq, void* dk,
                            float* dwq, float* dwk, void* ws, cudaStream_t s);

// The residual's addition and the norm of rows (sfa_add_norm.cu).  Strides in
// elements; what a row is written to is dense.
struct AddNormArgs {
    int N, dim;
    long long xs, rs;      // row strides
    const void *x, *r;     // r: nullptr for no residual
    const float* w;
    float eps, inv_dim;
    void *h, *y;           // the sum (nullptr: not kept); the norm, or its 8-bit values
    float* scale;          // of 8-bit rows
};
// norm = false: the rows themselves in 8 bits.
cudaError_t launch_add_norm(const AddNormArgs& a, sfa_dtype dt, bool norm, bool fp8, cudaStream_t s);
struct AddNormBwdArgs {
    int N, dim;
    const void *h, *dy, *dh;  // dh: nullptr for none
    const float* w;
    float eps, inv_dim;
    void* dx;
    float* dw;
};
size_t add_norm_bwd_workspace(sfa_dtype dt, int N, int dim);  // 0: none
cudaError_t launch_add_norm_bwd(const AddNormBwdArgs& a, sfa_dtype dt, void* ws, cudaStream_t s);

// A paged cache and one step's tokens (sfa_paged in sfa.h).
struct PagedArgs {
    void *k, *v;
    const int *table, *cu, *lens;
    unsigned* status;
    int S, N;
    int max_pages, num_pages;
    int shift;             // log2 of the page size
    int cap;               // positions [0, cap) exist
    float* scales;         // of 8-bit pages: [block of rows][key or value][head]
    int block_shift;       // log2 of the rows of a block
};
struct AppendArgs {
    PagedArgs c;
    const void *q, *kn, *vn;  // new queries (nullptr: none), keys, values
    long long qs, ks, vs;     // token strides in elements
    const float *wq, *wk;     // nullptr: no norm
    const float2* rope;       // nullptr: no rotation
    void* qhat;
    float eps;
};
cudaError_t launch_paged_append(const AppendArgs& a, sfa_dtype dt, cudaStream_t s);
cudaError_t launch_paged_append_fp8(const AppendArgs& a, sfa_dtype dt, cudaStream_t s);
cudaError_t launch_paged_fwd(const LayerArgs& a, const PagedArgs& c, sfa_dtype dt, const void* q, long long qs, void* o,
                             float* lse, cudaStream_t s);
size_t paged_fwd_fp8_workspace(const LayerArgs& a, const PagedArgs& c, sfa_dtype dt);  // 0: none
cudaError_t launch_paged_fwd_fp8(const LayerArgs& a, const PagedArgs& c, sfa_dtype dt, const void* q, long long qs,
                                 void* o, float* lse, void* ws, cudaStream_t s);

// The projection of 8-bit rows (sfa_qkv_fp8.cu).
struct QkvFp8Args {
    int M, T, dm;           // tokens, positions of a sequence, columns
    const void *x, *w;
    const float *sx, *sw;   // scales of the rows of x and w
    const float2* rope;     // nullptr: no rotation
    void *q, *k, *v;
    unsigned* status;
};
cudaError_t launch_qkv_fp8(const QkvFp8Args& a, cudaStream_t s);

}  // namespace sfa
