// sfa_qkv_fp8.cu -- the query, key and value projection of 8-bit rows on the
// 5th-generation tensor cores (sfa_qkv_rope_fp8 in include/sfa.h):
//   [Q | K | V][t][r] = sx[t] sw[r] sum_c X8[t][c] W8[r][c],
// with the rotation of queries and keys in the epilogue, as sfa_qkv.cu does it
// for bf16 operands.  The products are exact in fp32 (e4m3 has four significant
// bits); the sum is the tensor core's fp32 one; scales and rotation are fp32 and
// the result is rounded once.
//
// A persistent CTA per SM walks tiles of 128 tokens x 64 kHeads output features
// over the whole d_model:
//   warp 0 (one lane): TMA loads of k-blocks (128 columns, one 128-byte swizzle
//                      row) into an mbarrier ring;
//   warp 1:            one lane issues tcgen05.mma (kind::f8f6f4, M = 128, K = 32)
//                      into one of two accumulators in tensor memory;
//   warps 2..9:        the epilogue, two warps a quarter of the lanes, which take
//                      the heads in turn: a thread has one token's 64 features of
//                      a head, scales and rotates them and stages them for a TMA
//                      store of the warp's 32 rows.
// What the SMs fetch from L2 is the limit before the tensor cores are: a tile of
// 128 x 192 takes 40 KB a k-block.  Where a CTA's 192 rows of W8 fit beside the
// ring (kResident: d_model <= 640) they are loaded once, every CTA keeps to
// its quarter of the features, and a k-block is the 16 KB of X8 alone.
//
// Every wait is bounded; a timeout sets SFA_DEVSTAT_WAIT_TIMEOUT and the CTA
// stops.
#include <cstring>

#include "sfa_internal.cuh"
#include "sfa_mma.cuh"
#include "sfa_ops.cuh"
#include "sfa_ring.cuh"
#include "sfa_tc.cuh"
#include "sfa_tma.cuh"

namespace sfa {

namespace {

using namespace mma;
using namespace tma;

constexpr int BM = 128;                    // tokens of a tile (TMEM lanes)
constexpr int BK = 128;                    // columns of a k-block: 128 bytes
constexpr int kSteps = BK / 32;            // MMAs of a k-block
constexpr uint32_t kXBytes = BM * BK;      // 16 KB
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr int kRows = (kHq + 2 * kHkv) * kD;         // 768 output features
constexpr uint32_t kStoreBytes = 32 * kD * 2;        // a warp's 32 rows of one head
constexpr int kMaxResident = 5;                      // k-blocks of W8 that stay in shared memory

template <int kHeads, bool kResident>
struct Shape {
    static constexpr int kBN = kHeads * kD, kTiles = kRows / kBN;
    static constexpr int kStages = kHeads == 1 ? 6 : 4;
    static constexpr uint32_t kWBytes = kBN * BK;    // of a k-block
    static constexpr uint32_t kStageBytes = kXBytes + (kResident ? 0 : kWBytes);
    static constexpr uint32_t kAccCols = kHeads == 1 ? 64 : 256, kTmemCols = 2 * kAccCols;
    // header: the barriers, the TMEM address, the abort flag; then sw
    static constexpr uint32_t kFull = 0, kEmpty = 8 * kStages, kTFull = 16 * kStages, kTEmpty = kTFull + 16,
                              kWFull = kTEmpty + 16, kSlot = kWFull + 8 * kMaxResident, kAbort = kSlot + 8;
    static constexpr uint32_t kScales = 1024, kData = kScales + 1024 * 3;  // 768 floats
    static constexpr uint32_t resident(int nkb) { return kResident ? (uint32_t)nkb * kWBytes : 0u; }
    static constexpr size_t smem(int nkb) {
        return 1024 + kData + resident(nkb) + kStages * (size_t)kStageBytes + kEpiWarps * (size_t)kStoreBytes;
    }
    static_assert(kRows % kBN == 0 && kAbort + 4 <= kScales && kRows * 4 <= kData - kScales, "layout");
    static_assert(kData % 1024 == 0 && kWBytes % 1024 == 0 && kStageBytes % 1024 == 0, "swizzle periods");
};
static_assert(Shape<3, true>::smem(kMaxResident) <= 232448 && Shape<3, false>::smem(0) <= 232448 &&
                  Shape<1, false>::smem(0) <= 232448,
              "shared memory of one CTA");

struct Params {
    CUtensorMap xmap, wmap;         // X8 [M][dm], box 128 x 128; W8 [768][dm], box 128 x kBN
    CUtensorMap qmap, kmap, vmap;   // outputs as [M][512], [M][128], [M][128], box 64 x 32 (stores)
    const float *sx, *sw;
    const float2* rope;
    unsigned* status;
    int M, T, nkb, tiles;           // tiles: of all features, features the faster index
};

template <int kHeads, bool kResident>
__global__ void __launch_bounds__(kThreads, 1) qkv_fp8_kernel(const __grid_constant__ Params P) {
    using S = Shape<kHeads, kResident>;
    constexpr uint32_t kIdesc = tc::idesc_e4m3(BM, S::kBN);
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    unsigned char* hdr = smem_raw + (base - raw);
    const uint32_t bar_full = base + S::kFull, bar_empty = base + S::kEmpty, bar_w = base + S::kWFull;
    const uint32_t bar_tfull = base + S::kTFull, bar_tempty = base + S::kTEmpty;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(hdr + S::kSlot);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(hdr + S::kAbort);
    float* sw = reinterpret_cast<float*>(hdr + S::kScales);
    const uint32_t wbase = base + S::kData, stages = wbase + S::resident(P.nkb);
    const uint32_t stores = stages + S::kStages * S::kStageBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_tfull + 8 * b, 1);
            mbar_init(bar_tempty + 8 * b, kEpiWarps);
        }
        for (int b = 0; b < kMaxResident; ++b) mbar_init(bar_w + 8 * b, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tc::alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), S::kTmemCols);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = threadIdx.x; i < kRows; i += kThreads) sw[i] = fresh(P.sw + i);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            int kbg = 0, loaded = 0;
            for (int t = blockIdx.x; t < P.tiles && *abort_flag == 0; t += gridDim.x) {
                const int m0 = (t / S::kTiles) * BM, n0 = (t % S::kTiles) * S::kBN;
                for (int kb = 0; kb < P.nkb; ++kb, ++kbg) {
                    if (kResident && loaded < P.nkb) {
                        mbar_arrive_expect_tx(bar_w + 8 * kb, S::kWBytes);
                        tma_load_2d(wbase + kb * S::kWBytes, &P.wmap, kb * BK, n0, bar_w + 8 * kb);
                        ++loaded;
                    }
                    const int s = kbg % S::kStages;
                    if (!mbar_wait(bar_empty + 8 * s, ((uint32_t)(kbg / S::kStages) & 1u) ^ 1u, abort_flag)) {
                        *abort_flag = 1;
                        break;
                    }
                    const uint32_t a = stages + (uint32_t)s * S::kStageBytes;
                    mbar_arrive_expect_tx(bar_full + 8 * s, S::kStageBytes);
                    tma_load_2d(a, &P.xmap, kb * BK, m0, bar_full + 8 * s);
                    if (!kResident) tma_load_2d(a + kXBytes, &P.wmap, kb * BK, n0, bar_full + 8 * s);
                }
            }
            // Nothing may land in this CTA's shared memory after it leaves: wait
            // for the MMA's release of the last use of every stage, or, once a
            // wait has failed, for the copies themselves.
            const bool clean = *abort_flag == 0;
            for (int n = max(0, kbg - S::kStages); n < kbg; ++n) {
                const uint32_t ph = (uint32_t)(n / S::kStages) & 1u;
                if (!clean || !mbar_wait(bar_empty + 8 * (n % S::kStages), ph, nullptr))
                    (void)mbar_wait(bar_full + 8 * (n % S::kStages), ph, nullptr);
            }
            for (int kb = 0; kb < loaded; ++kb) (void)mbar_wait(bar_w + 8 * kb, 0, nullptr);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int kbg = 0, j = 0;
            for (int t = blockIdx.x; t < P.tiles; t += gridDim.x, ++j) {
                const int buf = j & 1;
                // the epilogue has read this accumulator's previous tile
                if (!mbar_wait(bar_tempty + 8 * buf, ((uint32_t)(j >> 1) & 1u) ^ 1u, abort_flag)) {
                    *abort_flag = 1;
                    break;
                }
                tc::fence_after();
                const uint32_t acc = tmem + (uint32_t)buf * S::kAccCols;
                bool ok = true;
                for (int kb = 0; kb < P.nkb; ++kb, ++kbg) {
                    const int s = kbg % S::kStages;
                    if ((kResident && j == 0 && !mbar_wait(bar_w + 8 * kb, 0, abort_flag)) ||
                        !mbar_wait(bar_full + 8 * s, (uint32_t)(kbg / S::kStages) & 1u, abort_flag)) {
                        *abort_flag = 1;
                        ok = false;
                        break;
                    }
                    tc::fence_after();
                    const uint32_t a = stages + (uint32_t)s * S::kStageBytes;
                    const uint64_t ad = tc::desc_kmajor(a);
                    const uint64_t bd = tc::desc_kmajor(kResident ? wbase + kb * S::kWBytes : a + kXBytes);
#pragma unroll
                    for (int k = 0; k < kSteps; ++k)
                        tc::mma_ss_fp8(acc, ad + (uint64_t)(2 * k), bd + (uint64_t)(2 * k), kIdesc, (kb | k) != 0);
                    tc::commit(bar_empty + 8 * s);  // the stage is free once these have read it
                }
                // the accumulator is complete once every MMA above has
                tc::commit(bar_tfull + 8 * buf);
                if (!ok) break;
            }
        }
        __syncwarp();
    } else {
        // epilogue: warp w reads TMEM lanes 32 (w % 4) .. + 31 (its rows)
        const int lb = 32 * (warp & 3), half = (warp - 2) >> 2;
        const uint32_t sbuf = stores + (uint32_t)(warp - 2) * kStoreBytes;
        int j = 0;
        for (int t = blockIdx.x; t < P.tiles; t += gridDim.x, ++j) {
            const int buf = j & 1;
            const int m0 = (t / S::kTiles) * BM, n0 = (t % S::kTiles) * S::kBN;
            const int m = m0 + lb + lane;
            // this token's scale and the (cos, sin) row of its position, on their way
            // while the tile is computed
            const float sxm = m < P.M ? fresh(P.sx + m) : 0.f;
            float4 cs[kPairs / 2];
            if (P.rope && n0 < (kHq + kHkv) * kD) {
                const float4* tr = reinterpret_cast<const float4*>(P.rope + (size_t)(m < P.M ? m % P.T : 0) * kPairs);
#pragma unroll
                for (int i = 0; i < kPairs / 2; ++i) cs[i] = fresh(tr + i);
            }
            if (!mbar_wait(bar_tfull + 8 * buf, (uint32_t)(j >> 1) & 1u, abort_flag)) {
                if (lane == 0) *abort_flag = 1;
                break;
            }
            if (*abort_flag) break;
            tc::fence_after();
#pragma unroll 1
            for (int h = (j * kHeads + half) & 1; h < kHeads; h += 2) {
                uint32_t xu[32], yu[32];
                const uint32_t ta = tmem + ((uint32_t)lb << 16) + (uint32_t)buf * S::kAccCols + (uint32_t)(h * kD);
                tc::ld_x32(ta, xu);
                tc::ld_x32(ta + kPairs, yu);
                tc::wait_ld();
                tc::hold(xu);
                tc::hold(yu);
                const int hh = n0 / kD + h;  // Q heads 0..7, K heads 8..9, V heads 10..11
                const bool rot = P.rope != nullptr && hh < kHq + kHkv;
                const float4* wx = reinterpret_cast<const float4*>(sw + hh * kD);
                uint32_t xo[16], yo[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 a = wx[i], b = wx[8 + i];
                    const float wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
                    float x[4], y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[e] = __uint_as_float(xu[4 * i + e]) * (sxm * wa[e]);
                        y[e] = __uint_as_float(yu[4 * i + e]) * (sxm * wb[e]);
                    }
                    if (rot) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 q = cs[2 * i + e / 2];  // pairs 4 i + e and its neighbour
                            const float c = e & 1 ? q.z : q.x, s = e & 1 ? q.w : q.y;
                            const float u = x[e], v = y[e];
                            x[e] = __fmaf_rn(u, c, __fmul_rn(-v, s));
                            y[e] = __fmaf_rn(v, c, __fmul_rn(u, s));
                        }
                    }
                    xo[2 * i] = pack_bf16(x[0], x[1]);
                    xo[2 * i + 1] = pack_bf16(x[2], x[3]);
                    yo[2 * i] = pack_bf16(y[0], y[1]);
                    yo[2 * i + 1] = pack_bf16(y[2], y[3]);
                }
                // stage the warp's 32 rows (row = lane, 128 bytes, 16-byte chunk c
                // at c ^ (lane & 7): the 128-byte swizzle of the store map)
                if (lane == 0) bulk_wait_read();  // the store before has read the buffer
                __syncwarp();
                const uint32_t rb = sbuf + (uint32_t)lane * 128u;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    sts_u4(rb + (uint32_t)(((c ^ lane) & 7) << 4), xo[4 * c], xo[4 * c + 1], xo[4 * c + 2], xo[4 * c + 3]);
                    sts_u4(rb + (uint32_t)((((4 + c) ^ lane) & 7) << 4), yo[4 * c], yo[4 * c + 1], yo[4 * c + 2],
                           yo[4 * c + 3]);
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0 && m0 + lb < P.M) {
                    const CUtensorMap* map = hh < kHq ? &P.qmap : hh < kHq + kHkv ? &P.kmap : &P.vmap;
                    const int col = (hh < kHq ? hh : hh < kHq + kHkv ? hh - kHq : hh - kHq - kHkv) * kD;
                    tma_store_2d(map, sbuf, col, m0 + lb);  // rows past M are not written
                    bulk_commit();
                }
            }
            // this warp has read its part of the accumulator
            tc::fence_before();
            __syncwarp();
            mbar_arrive_if(bar_tempty + 8 * buf, lane == 0);
        }
        if (lane == 0) bulk_wait_all();
        if (*abort_flag && lane == 0 && warp == 2 && P.status) atomicOr(P.status, SFA_DEVSTAT_WAIT_TIMEOUT);
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after();
        tc::dealloc(tmem, S::kTmemCols);
    }
}

template <int kHeads, bool kResident>
cudaError_t launch(Params& P, const QkvFp8Args& a, int sms, int dev, cudaStream_t s) {
    using S = Shape<kHeads, kResident>;
    if (!encode_rows(&P.wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.w, kRows, a.dm, S::kBN)) return cudaErrorInvalidValue;
    P.tiles = (P.M + BM - 1) / BM * S::kTiles;
    const size_t smem = S::smem(P.nkb);
    static CtxSetting configured[64];
    if (!ctx_setting_holds(configured[dev & 63], smem)) {
        const cudaError_t e = cudaFuncSetAttribute(qkv_fp8_kernel<kHeads, kResident>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        ctx_setting_done(configured[dev & 63], smem);
    }
    // with W8 in place a CTA keeps its features: a grid of whole rows of tiles
    const int most = kResident ? sms / S::kTiles * S::kTiles : sms;
    return launch_early(qkv_fp8_kernel<kHeads, kResident>, (unsigned)(P.tiles < most ? P.tiles : most), kThreads, smem, s, P);
}

}  // namespace

cudaError_t launch_qkv_fp8(const QkvFp8Args& a, cudaStream_t s) {
    Params P;
    std::memset(&P, 0, sizeof(P));
    const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    if (!encode_rows(&P.xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.x, a.M, a.dm, BM) ||
        !encode_rows(&P.qmap, bf16, 2, a.q, a.M, kHq * kD, 32) || !encode_rows(&P.kmap, bf16, 2, a.k, a.M, kHkv * kD, 32) ||
        !encode_rows(&P.vmap, bf16, 2, a.v, a.M, kHkv * kD, 32))
        return cudaErrorInvalidValue;
    P.sx = a.sx;
    P.sw = a.sw;
    P.rope = a.rope;
    P.status = a.status;
    P.M = a.M;
    P.T = a.T;
    P.nkb = (a.dm + BK - 1) / BK;  // columns behind the last are filled with zeros
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int sms = ring::sm_count(dev, &e);
    if (e != cudaSuccess) return e;
    const int rows = (a.M + BM - 1) / BM;
    if (rows * Shape<1, false>::kTiles <= sms) return launch<1, false>(P, a, sms, dev, s);
    return P.nkb <= kMaxResident ? launch<3, true>(P, a, sms, dev, s) : launch<3, false>(P, a, sms, dev, s);
}

}  // namespace sfa
