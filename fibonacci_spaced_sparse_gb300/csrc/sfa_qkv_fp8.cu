// sfa_qkv_fp8.cu -- the query, key and value projection of 8-bit rows on the
// 5th-generation tensor cores (sfa_qkv_rope_fp8 in include/sfa.h):
//   [Q | K | V][t][r] = sx[t] sw[r] sum_c X8[t][c] W8[r][c],
// with the rotation of queries and keys in the epilogue, as sfa_qkv.cu does it
// for bf16 operands.  The products are exact in fp32 (e4m3 has four significant
// bits); the sum is the tensor core's fp32 one; scales and rotation are fp32 and
// the result is rounded once.
//
// A persistent CTA per SM walks tiles of 128 (256) tokens x 64 or 192 output features
// over the whole d_model:
//   warp 0 (one lane): TMA loads of k-blocks (128 columns, one 128-byte swizzle
//                      row) into an mbarrier ring;
//   warp 1:            one lane issues tcgen05.mma (kind::f8f6f4, M = 128, K = 32)
//                      into one of two accumulators in tensor memory;
//   the other warps:   the epilogue.  A warp takes 16 tokens, eight warps 128; but for
//                      kSmall there are two such sets, which take the tiles in turn
//                      (kTall: a half of the tile each), so that one has its tokens'
//                      (cos, sin) rows by the time its accumulator is done.  The
//                      accumulator is read as fragments (16 rows x 8 columns a quad of
//                      lanes at a time) rather than a row a lane: a warp then reads the
//                      rotation's table in 64-byte pieces of eight rows, where a row a
//                      lane costs a cache line a lane and load (32 x 1024 tokens at
//                      d_model 512: 32.7 us that way, 18.0 us as it is), and stmatrix
//                      puts the rounded rows where a TMA store takes them from.
// What an SM fetches is the limit before the tensor cores are: a tile of 128 x 192
// takes 40 KB a k-block, 100 bytes a clock at the rate of the products, and an SM was
// seen to take 58.  Where a CTA's 192 rows of W8 fit beside the ring (kResident:
// d_model <= 512) they are loaded once, every CTA keeps to its quarter of the
// features, and a k-block is the 16 KB of X8 alone; above that, tiles of 256 tokens
// (kTall) take 56 KB for twice the products.
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
constexpr int kRows = (kHq + 2 * kHkv) * kD;         // 768 output features
constexpr uint32_t kStoreBytes = 16 * kD * 2;        // a warp's 16 rows of a head on their way out
constexpr int kMaxResident = 4;                      // k-blocks of W8 that stay in shared memory

// The forms of the kernel.
//   kSmall: tiles of 128 tokens and one head, while all of them run at once;
//   kResident: 128 tokens x 3 heads, W8 in place;
//   kStreamed: the same, W8 through the ring;
//   kTall: 256 tokens x 3 heads, in both accumulators, W8 through the ring.
enum Form { kSmall, kResident, kStreamed, kTall };

template <Form kForm>
struct Shape {
    static constexpr int kHeads = kForm == kSmall ? 1 : 3, kHalves = kForm == kTall ? 2 : 1;  // of 128 tokens
    static constexpr bool kHeld = kForm == kResident;
    static constexpr int kBN = kHeads * kD, kTiles = kRows / kBN;
    static constexpr int kSets = kForm == kSmall ? 1 : 2;  // of epilogue warps
    static constexpr int kEpiWarps = 8 * kSets, kThreads = 32 * (2 + kEpiWarps);
    static constexpr int kStages = kForm == kSmall ? 6 : kForm == kResident ? 5 : kForm == kStreamed ? 4 : 3;
    static constexpr uint32_t kWBytes = kBN * BK;    // of a k-block
    static constexpr uint32_t kStageBytes = kHalves * kXBytes + (kHeld ? 0 : kWBytes);
    static constexpr uint32_t kAccCols = kHeads == 1 ? 64 : 256, kTmemCols = 2 * kAccCols;
    // header: the barriers, the TMEM address, the abort flag; then sw
    static constexpr uint32_t kFull = 0, kEmpty = 8 * kStages, kTFull = 16 * kStages, kTEmpty = kTFull + 16,
                              kWFull = kTEmpty + 16, kSlot = kWFull + 8 * kMaxResident, kAbort = kSlot + 8;
    static constexpr uint32_t kScales = 1024, kData = kScales + 1024 * 3;  // 768 floats
    static constexpr uint32_t resident(int nkb) { return kHeld ? (uint32_t)nkb * kWBytes : 0u; }
    static constexpr size_t smem(int nkb) {
        return 1024 + kData + resident(nkb) + kStages * (size_t)kStageBytes + kEpiWarps * (size_t)kStoreBytes;
    }
    static_assert(kRows % kBN == 0 && kAbort + 4 <= kScales && kRows * 4 <= kData - kScales, "layout");
    static_assert(kData % 1024 == 0 && kWBytes % 1024 == 0 && kStageBytes % 1024 == 0, "swizzle periods");
};
static_assert(Shape<kSmall>::smem(0) <= 232448 && Shape<kResident>::smem(kMaxResident) <= 232448 &&
                  Shape<kStreamed>::smem(0) <= 232448 && Shape<kTall>::smem(0) <= 232448,
              "shared memory of one CTA");

struct Params {
    CUtensorMap xmap, wmap;         // X8 [M][dm], box 128 x 128; W8 [768][dm], box 128 x kBN
    CUtensorMap qmap, kmap, vmap;   // outputs as [M][512], [M][128], [M][128], box 64 x 16 (stores)
    const float *sx, *sw;
    const float2* rope;
    unsigned* status;
    int M, T, nkb, tiles;           // tiles: of all features, features the faster index
};

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

template <Form kForm>
__global__ void __launch_bounds__(Shape<kForm>::kThreads, 1) qkv_fp8_kernel(const __grid_constant__ Params P) {
    using S = Shape<kForm>;
    constexpr int kHeads = S::kHeads, kRowsOf = BM * S::kHalves;  // tokens of a tile
    constexpr uint32_t kIdesc = tc::idesc_e4m3(BM, S::kBN);
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    unsigned char* hdr = smem_raw + (base - raw);
    const uint32_t bar_full = base + S::kFull, bar_empty = base + S::kEmpty, bar_w = base + S::kWFull;
    const uint32_t bar_tfull = base + S::kTFull, bar_tempty = base + S::kTEmpty;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(hdr + S::kSlot);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(hdr + S::kAbort);
    const uint32_t wbase = base + S::kData, stages = wbase + S::resident(P.nkb);
    const uint32_t stores = stages + S::kStages * S::kStageBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 32) {
        prefetch_map(&P.xmap);
        prefetch_map(&P.wmap);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_tfull + 8 * b, 1);
            mbar_init(bar_tempty + 8 * b, 8 * S::kHalves);
        }
        for (int b = 0; b < kMaxResident; ++b) mbar_init(bar_w + 8 * b, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tc::alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), S::kTmemCols);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;
    // Only now may the next launch start: one that allocated tensor memory first, and then
    // waited for this grid, would leave this CTA without.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == 0) {
        if (lane == 0) {
            int kbg = 0, loaded = 0;
            for (int t = blockIdx.x; t < P.tiles && *abort_flag == 0; t += gridDim.x) {
                const int m0 = (t / S::kTiles) * kRowsOf, n0 = (t % S::kTiles) * S::kBN;
                for (int kb = 0; kb < P.nkb; ++kb, ++kbg) {
                    if (S::kHeld && loaded < P.nkb) {
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
                    for (int i = 0; i < S::kHalves; ++i)  // (rows past M are filled with zeros)
                        tma_load_2d(a + i * kXBytes, &P.xmap, kb * BK, m0 + i * BM, bar_full + 8 * s);
                    if (!S::kHeld) tma_load_2d(a + S::kHalves * kXBytes, &P.wmap, kb * BK, n0, bar_full + 8 * s);
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
                // the accumulator (with kTall both are one tile's) and the parity of its uses
                const int buf = S::kHalves == 1 ? j & 1 : 0;
                const uint32_t use = (uint32_t)(S::kHalves == 1 ? j >> 1 : j) & 1u;
                // the epilogue has read this accumulator's previous tile
                if (!mbar_wait(bar_tempty + 8 * buf, use ^ 1u, abort_flag)) {
                    *abort_flag = 1;
                    break;
                }
                tc::fence_after();
                const uint32_t acc = tmem + (uint32_t)buf * S::kAccCols;
                bool ok = true;
                for (int kb = 0; kb < P.nkb; ++kb, ++kbg) {
                    const int s = kbg % S::kStages;
                    if ((S::kHeld && j == 0 && !mbar_wait(bar_w + 8 * kb, 0, abort_flag)) ||
                        !mbar_wait(bar_full + 8 * s, (uint32_t)(kbg / S::kStages) & 1u, abort_flag)) {
                        *abort_flag = 1;
                        ok = false;
                        break;
                    }
                    tc::fence_after();
                    const uint32_t a = stages + (uint32_t)s * S::kStageBytes;
                    const uint64_t bd = tc::desc_kmajor(S::kHeld ? wbase + kb * S::kWBytes : a + S::kHalves * kXBytes);
#pragma unroll
                    for (int k = 0; k < kSteps; ++k)
#pragma unroll
                        for (int i = 0; i < S::kHalves; ++i)
                            tc::mma_ss_fp8(acc + i * S::kAccCols, tc::desc_kmajor(a + i * kXBytes) + (uint64_t)(2 * k),
                                           bd + (uint64_t)(2 * k), kIdesc, (kb | k) != 0);
                    tc::commit(bar_empty + 8 * s);  // the stage is free once these have read it
                }
                // the accumulator is complete once every MMA above has
                tc::commit(bar_tfull + 8 * buf);
                if (!ok) break;
            }
        }
        __syncwarp();
    } else {
        // epilogue: warp w reads 16 of TMEM lanes 32 (w % 4) .. + 31 (its rows) of every
        // second tile, with kTall of its set's half of every tile; this thread's rows are
        // g8 and g8 + 8 of them
        const int ew = warp - 2, set = ew >> 3, g8 = lane >> 2, tig = lane & 3;
        const int lb = 32 * (warp & 3) + 16 * (ew >> 2 & 1);
        const uint32_t sbuf = stores + (uint32_t)ew * kStoreBytes;
        float* swm = reinterpret_cast<float*>(hdr + S::kScales);
        for (int i = threadIdx.x - 64; i < kRows; i += 32 * S::kEpiWarps) swm[i] = fresh(P.sw + i);
        asm volatile("bar.sync 1, %0;" ::"n"(32 * S::kEpiWarps) : "memory");  // of the epilogue's warps
        // of the 16 staged rows (128 bytes, 16-byte chunk c of row r at c ^ (r & 7), the
        // swizzle of the store map) this lane gives stmatrix row lane % 16, in the first
        // or the last four chunks
        const uint32_t srow = sbuf + (uint32_t)(lane & 15) * 128u, schunk = (uint32_t)(lane >> 4 << 2);
        for (int j = S::kHalves == 1 ? set : 0; blockIdx.x + j * gridDim.x < P.tiles; j += S::kHalves == 1 ? S::kSets : 1) {
            const int t = blockIdx.x + j * gridDim.x, h0 = t % S::kTiles * kHeads;
            const int m0 = t / S::kTiles * kRowsOf + (S::kHalves == 1 ? 0 : set * BM) + lb;
            const int buf = S::kHalves == 1 ? j & 1 : 0;
            const uint32_t use = (uint32_t)(S::kHalves == 1 ? j >> 1 : j) & 1u;
            // the tokens' scales and the (cos, sin) of their positions are on their way
            // while the tile is computed
            const bool rotates = P.rope != nullptr && h0 < kHq + kHkv;
            float2 sx[2], cs[2][4], sn[2][4];  // pairs 8 i + 2 tig and the next one
            const int p0 = rotates ? m0 % P.T + g8 : 0;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int m = m0 + 8 * r + g8;
                sx[r] = both(m < P.M ? fresh(P.sx + m) : 0.f);
                if (!rotates) continue;
                int pos = p0 + 8 * r;
                if (pos >= P.T) pos = P.T >= 16 ? pos - P.T : pos % P.T;
                const float4* row = reinterpret_cast<const float4*>(P.rope + (size_t)pos * kPairs) + tig;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 v = fresh(row + 4 * i);
                    cs[r][i] = make_float2(v.x, v.z);
                    sn[r][i] = make_float2(v.y, v.w);
                }
            }
            if (!ring::warp_wait(bar_tfull + 8 * buf, use, abort_flag)) {
                if (lane == 0) *abort_flag = 1;
                break;
            }
            if (__any_sync(kFull, *abort_flag != 0)) break;
            tc::fence_after();
            const uint32_t acc0 = tmem + ((uint32_t)lb << 16) + (uint32_t)(S::kHalves == 1 ? buf : set) * S::kAccCols;
#pragma unroll 1
            for (int h = 0; h < kHeads; ++h) {
                const int hh = h0 + h;  // Q heads 0..7, K heads 8..9, V heads 10..11
                const bool rot = rotates && hh < kHq + kHkv;
                uint32_t acc[32];
                tc::ld_frag_x8(acc0 + (uint32_t)(h * kD), acc);
                const float2* sw = reinterpret_cast<const float2*>(swm + hh * kD) + tig;
                if (lane == 0) bulk_wait_read();  // the store before has read its rows
                tc::wait_ld();
                tc::hold(acc);
                if (h == kHeads - 1) tc::fence_before();  // this warp has read its part of the accumulator
                __syncwarp();
                mbar_arrive_if(bar_tempty + 8 * buf, h == kHeads - 1 && lane == 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 wx = sw[4 * i], wy = sw[16 + 4 * i];
                    uint32_t out[4];  // columns of 8 i and their partners, rows g8 and g8 + 8
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t* a = acc + 4 * i + 2 * r;
                        // the sum first: the scales' product alone may be too small for a float, or too large
                        float2 x = __fmul2_rn(__fmul2_rn(make_float2(__uint_as_float(a[0]), __uint_as_float(a[1])), wx), sx[r]);
                        float2 y = __fmul2_rn(__fmul2_rn(make_float2(__uint_as_float(a[16]), __uint_as_float(a[17])), wy), sx[r]);
                        if (rot) {
                            const float2 u = x, c = cs[r][i], n = sn[r][i];
                            x = make_float2(fmaf(u.x, c.x, -(y.x * n.x)), fmaf(u.y, c.y, -(y.y * n.y)));
                            y = __ffma2_rn(y, c, __fmul2_rn(u, n));
                        }
                        out[r] = pack_bf16(x.x, x.y);
                        out[2 + r] = pack_bf16(y.x, y.y);
                    }
                    stsm_x4(srow + (((schunk + i) ^ (lane & 7u)) << 4), out[0], out[1], out[2], out[3]);
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0 && m0 < P.M) {
                    const CUtensorMap* map = hh < kHq ? &P.qmap : hh < kHq + kHkv ? &P.kmap : &P.vmap;
                    const int col = (hh < kHq ? hh : hh < kHq + kHkv ? hh - kHq : hh - kHq - kHkv) * kD;
                    tma_store_2d(map, sbuf, col, m0);  // rows past M are not written
                    bulk_commit();
                }
            }
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

template <Form kForm>
cudaError_t launch(Params& P, const QkvFp8Args& a, int sms, int dev, cudaStream_t s) {
    using S = Shape<kForm>;
    if (!encode_rows(&P.wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.w, kRows, a.dm, S::kBN)) return cudaErrorInvalidValue;
    P.tiles = (P.M + BM * S::kHalves - 1) / (BM * S::kHalves) * S::kTiles;
    const size_t smem = S::smem(P.nkb);
    static CtxSetting configured[64];
    const cudaError_t e = allow_smem(configured[dev & 63], qkv_fp8_kernel<kForm>, smem);
    if (e != cudaSuccess) return e;
    // with W8 in place a CTA keeps its features: a grid of whole rows of tiles
    const int most = S::kHeld ? sms / S::kTiles * S::kTiles : sms;
    return launch_early(qkv_fp8_kernel<kForm>, (unsigned)(P.tiles < most ? P.tiles : most), S::kThreads, smem, s, P);
}

// Clocks of a call in the two forms that stream W8: rounds of tiles times what a k-block
// takes, 40 KB (56) at some 58 bytes a clock and SM, and with kTall, whose epilogue
// does not overlap the next tile's products, the epilogue (us, streamed and tall: 8157
// tokens at d_model 4096 24.9 and 22.1, 16384 45.7 and 41.0, 2048 12.5 and 18.0;
// 32768 at 2048 44.1 and 46.4, 4096 9.0 and 11.9; 8192 at 1024, where the estimate is
// wrong, 10.2 and 9.6).
constexpr int kStreamedBlock = 700, kTallBlock = 960, kTallTile = 4500;
bool tall_is_faster(int M, int nkb, int sms) {
    auto rounds = [&](int rows) { return (long long)(((M + rows - 1) / rows) * Shape<kTall>::kTiles + sms - 1) / sms; };
    return rounds(2 * BM) * (nkb * kTallBlock + kTallTile) < rounds(BM) * nkb * kStreamedBlock;
}

}  // namespace

cudaError_t launch_qkv_fp8(const QkvFp8Args& a, cudaStream_t s) {
    Params P;
    std::memset(&P, 0, sizeof(P));
    const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    if (!encode_rows(&P.xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.x, a.M, a.dm, BM) ||
        !encode_rows(&P.qmap, bf16, 2, a.q, a.M, kHq * kD, 16) || !encode_rows(&P.kmap, bf16, 2, a.k, a.M, kHkv * kD, 16) ||
        !encode_rows(&P.vmap, bf16, 2, a.v, a.M, kHkv * kD, 16))
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
    if (rows * Shape<kSmall>::kTiles <= sms) return launch<kSmall>(P, a, sms, dev, s);
    if (P.nkb <= kMaxResident) return launch<kResident>(P, a, sms, dev, s);
    return tall_is_faster(a.M, P.nkb, sms) ? launch<kTall>(P, a, sms, dev, s) : launch<kStreamed>(P, a, sms, dev, s);
}

}  // namespace sfa
