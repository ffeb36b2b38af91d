// fp8_gemm.cu -- 8-bit activations times FP8 block-128 weights on the
// 5th-generation tensor cores:
//   y[t][m] = sum_kb xs[kb][t] ws[m/128][kb] sum_{k in block kb} x[t][k] w[m][k],
// and the gated pair h[t][i] = SiLU(g) u of two such products, g and u.
//
// The tensor cores add up the 128 k of a block (E4M3 products, fp32 sums); the
// blocks' sums meet their two scales in fp32 registers. A CTA computes 128 rows
// of the weights (the MMA's M, one tile of scales) times BN tokens (its N):
//  - warp 0 copies a block of 128 k at a time into a ring by 2-D tensor copies
//    (128-byte swizzle; rows, tokens and k past the ends read as zero);
//  - warp 1, one elected lane, issues the block's MMAs (K = 32 each) into one of
//    a few buffers of tensor memory;
//  - warps 2..5 read a buffer (a row of the weights per thread, BN columns),
//    scale it and add it to their registers.
// With few tiles the k blocks of one are shared by a cluster of CTAs, which add
// up their parts in the order of their ranks, in one shared memory after the
// other: the same bits every time. With many, a CTA takes tile after tile, and
// its ring runs on from one to the next.
// Every wait is bounded (kErrWaitTimeout in the kernel's error word).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "common.cuh"
#include "f32x2.cuh"
#include "fp8.cuh"
#include "fp8.h"
#include "host_util.h"
#include "stream.cuh"

namespace bqd {

__device__ unsigned int g_fp8_error = 0;

namespace {

constexpr int kRows = 128;               // weight rows of a tile (MMA M), and of a tile of scales
constexpr int kBlk = 128;                // k of a block of scales and of a ring stage
constexpr int kTileW = kRows * kBlk;     // bytes
constexpr int kThreads = 192;
constexpr int kSumWarps = 4;

template <int BN, bool DUAL>
struct Narrow {
    static constexpr int kMats = DUAL ? 2 : 1;
    static constexpr int kTileX = BN * kBlk;
    static constexpr int kStage = kMats * kTileW + kTileX;
    static constexpr int kCtas = DUAL && BN == 64 ? 1 : 2;  // per SM
    static constexpr int kRoom = kCtas == 2 ? 110 * 1024 : 220 * 1024;
    static constexpr int kStages = (kRoom - 1024) / kStage < 8 ? (kRoom - 1024) / kStage : 8;
    static constexpr int kSmem = kStages * kStage + 1024;  // + alignment slack
    static constexpr int kCols = kMats * BN;               // tensor-memory columns of a buffer
    static constexpr int kBufs = 256 / kCols < 4 ? 256 / kCols : 4;
    static constexpr int kTmem = kBufs * kCols;
    static constexpr int kAhead = BN == 128 ? 2 : 4;       // blocks whose scales are on their way
    static_assert(BN % 16 == 0 && BN >= 16 && BN <= 128, "the MMA's N, and the threads' registers");
    static_assert(kTmem >= 32 && kTmem <= 256 && (kTmem & (kTmem - 1)) == 0, "two CTAs share 512 columns");
    static_assert(kStages >= 2 && kBufs >= 2, "copies, products and sums overlap");
    static_assert(kTileX % 1024 == 0, "stages start on 1024-byte boundaries (swizzle atoms)");
    static_assert(kMats * BN * kRows * 4 <= kStages * kStage, "a cluster's parts lie over the ring");
};

struct GemmShape {
    int64_t M;
    int T, KB;          // tokens, blocks of k
    int tilesM, tilesT; // tile = row tile * tilesT + token tile
    int y_type;
};

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.f + expf(-g)) * u; }

__device__ __forceinline__ void store_y(void* y, int type, int64_t at, float v)
{
    if (type == BQD_F32)
        static_cast<float*>(y)[at] = v;
    else
        static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
}

template <int BN, bool DUAL>
__global__ void __launch_bounds__(kThreads, Narrow<BN, DUAL>::kCtas)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap map_w0, const __grid_constant__ CUtensorMap map_w1,
                    const __grid_constant__ CUtensorMap map_x, const float* __restrict__ ws0,
                    const float* __restrict__ ws1, const float* __restrict__ xs, void* __restrict__ y,
                    float* __restrict__ ys, const GemmShape g)
{
    using S = Narrow<BN, DUAL>;
    constexpr int NM = S::kMats, kAhead = S::kAhead;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[S::kStages], empty[S::kStages], dfull[S::kBufs], dempty[S::kBufs];
    __shared__ uint32_t s_tmem;
    __shared__ __align__(16) float s_scale[kSumWarps][2][BN * NM];
    __shared__ uint32_t s_max[kSumWarps][BN];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;

    // This cluster's tiles, and this CTA's blocks of each
    uint32_t cs;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(cs));
    const int rank = cs > 1 ? static_cast<int>(cta_rank()) : 0;
    const int tiles = g.tilesM * g.tilesT, step = static_cast<int>(gridDim.x / cs);
    const int tile0 = static_cast<int>(blockIdx.x / cs);
    const int kb0 = static_cast<int>(static_cast<int64_t>(g.KB) * rank / cs);
    const int nkb = static_cast<int>(static_cast<int64_t>(g.KB) * (rank + 1) / cs) - kb0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < S::kBufs; ++i) {
            mbar_init(&dfull[i], 1);
            mbar_init(&dempty[i], kSumWarps);
        }
        fence_barrier_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                     "r"(S::kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = s_tmem;
    fp8_pdl_trigger();

    bool ok = true;
    if (warp == 0) {
        // ------------------------------------------------ copies
        if (lane == 0) {
            auto copy_w = [&](int st, int tile, int kb) {
                const uint32_t at = smem_u32(ring + st * S::kStage);
                const int row = tile / g.tilesT * kRows;
                mbar_arrive_expect_tx(&full[st], S::kStage);
                tma_2d(at, &map_w0, kb * kBlk, row, &full[st]);
                if constexpr (DUAL) tma_2d(at + kTileW, &map_w1, kb * kBlk, row, &full[st]);
            };
            auto copy_x = [&](int st, int tile, int kb) {
                tma_2d(smem_u32(ring + st * S::kStage + NM * kTileW), &map_x, kb * kBlk, tile % g.tilesT * BN, &full[st]);
            };
            // the first stages' weights before the wait for the previous kernel, whose output x may be
            const int first = min(S::kStages, tile0 < tiles ? nkb : 0);
            for (int i = 0; i < first; ++i) copy_w(i, tile0, kb0 + i);
            fp8_pdl_wait();
            for (int i = 0; i < first; ++i) copy_x(i, tile0, kb0 + i);
            int it = first;
            for (int tile = tile0; tile < tiles && ok; tile += step) {
                for (int i = tile == tile0 ? first : 0; i < nkb && ok; ++i, ++it) {
                    const int st = it % S::kStages;
                    if (it >= S::kStages) ok = mbar_wait(&empty[st], ((it / S::kStages) & 1) ^ 1, &g_fp8_error);
                    if (!ok) break;
                    copy_w(st, tile, kb0 + i);
                    copy_x(st, tile, kb0 + i);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ products
        constexpr uint32_t idesc = fp8_idesc(kRows, BN);
        int it = 0;
        for (int tile = tile0; tile < tiles && ok; tile += step) {
            for (int i = 0; i < nkb; ++i, ++it) {
                const int st = it % S::kStages, b = it % S::kBufs;
                ok = mbar_wait_warp(&full[st], (it / S::kStages) & 1, &g_fp8_error);
                if (ok && it >= S::kBufs) ok = mbar_wait_warp(&dempty[b], ((it / S::kBufs) & 1) ^ 1, &g_fp8_error);
                if (!ok) break;
                tc_after();
                if (fp8_elect()) {
                    const uint32_t at = smem_u32(ring + st * S::kStage), xat = at + NM * kTileW;
#pragma unroll
                    for (int m = 0; m < NM; ++m)
#pragma unroll
                        for (int j = 0; j < kBlk / 32; ++j)
                            fp8_mma(tmem + b * S::kCols + m * BN, fp8_desc(at + m * kTileW + 32 * j),
                                    fp8_desc(xat + 32 * j), idesc, j != 0 ? 1u : 0u);
                    fp8_commit(&empty[st]);
                    fp8_commit(&dfull[b]);
                }
                __syncwarp();
            }
        }
    } else {
        // ------------------------------------------------ sums, a row of the weights per thread
        const int q = warp % 4, sw = warp - 2;  // tensor-memory lane quarter; this warp's scales
        const uint32_t base = tmem + (static_cast<uint32_t>(32 * q) << 16);
        const int r = 32 * q + lane;
        constexpr int L = (BN + kWarp - 1) / kWarp;  // tokens of a lane when it fetches scales
        int it = 0;
        fp8_pdl_wait();
        for (int tile = tile0; tile < tiles; tile += step) {
            const int mt = tile / g.tilesT, n0 = tile % g.tilesT * BN;
            uint64_t acc[NM][BN / 2];
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int c = 0; c < BN / 2; ++c) acc[m][c] = 0;
            float far_x[kAhead][L], far_w[kAhead][NM];
            auto fetch = [&](int slot, int i) {
#pragma unroll
                for (int l = 0; l < L; ++l) {
                    const int t = n0 + lane + l * kWarp;
                    far_x[slot][l] = i < nkb && t < g.T && lane + l * kWarp < BN
                                         ? __ldg(xs + static_cast<int64_t>(kb0 + i) * g.T + t)
                                         : 0.f;
                }
                const int64_t at = static_cast<int64_t>(mt) * g.KB + kb0 + i;
                far_w[slot][0] = i < nkb ? __ldg(ws0 + at) : 0.f;
                if constexpr (DUAL) far_w[slot][1] = i < nkb ? __ldg(ws1 + at) : 0.f;
            };
#pragma unroll
            for (int i = 0; i < kAhead; ++i) fetch(i, i);
            for (int i = 0; i < nkb; ++i, ++it) {
                // the block's scales, to where every lane reads them all
                float* sc = s_scale[sw][it & 1];
#pragma unroll
                for (int l = 0; l < L; ++l)
                    if (BN % kWarp == 0 || lane + l * kWarp < BN)
#pragma unroll
                        for (int m = 0; m < NM; ++m) sc[m * BN + lane + l * kWarp] = far_x[0][l] * far_w[0][m];
#pragma unroll
                for (int d = 0; d + 1 < kAhead; ++d) {
#pragma unroll
                    for (int l = 0; l < L; ++l) far_x[d][l] = far_x[d + 1][l];
#pragma unroll
                    for (int m = 0; m < NM; ++m) far_w[d][m] = far_w[d + 1][m];
                }
                fetch(kAhead - 1, i + kAhead);
                const int b = it % S::kBufs;
                // (also orders the scales). After a wait that ran out the loops go on without
                // waiting, so that the warps still meet at every barrier.
                if (ok) ok = mbar_wait_warp(&dfull[b], (it / S::kBufs) & 1, &g_fp8_error);
                __syncwarp();
                tc_after();
#pragma unroll
                for (int m = 0; m < NM; ++m)
#pragma unroll
                    for (int c = 0; c < BN; c += 16) {
                        uint32_t d[16];
                        tmem_ld16(base + b * S::kCols + m * BN + c, d);
                        tmem_wait_ld();
                        const float4* s4 = reinterpret_cast<const float4*>(sc + m * BN + c);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 f = s4[e];
                            uint64_t* o = &acc[m][(c + 4 * e) / 2];
                            o[0] = fma2(pack(__uint_as_float(d[4 * e]), __uint_as_float(d[4 * e + 1])), pack(f.x, f.y), o[0]);
                            o[1] = fma2(pack(__uint_as_float(d[4 * e + 2]), __uint_as_float(d[4 * e + 3])), pack(f.z, f.w), o[1]);
                        }
                    }
                tc_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&dempty[b]);
            }
            // ---- the tile's outputs
            const int64_t row = static_cast<int64_t>(mt) * kRows + r;
            const bool live = row < g.M;
            float* part = reinterpret_cast<float*>(ring);  // [matrix][token][row], with a cluster
            int c0 = 0, c1 = BN;                           // this CTA's tokens of the tile
            if (cs > 1) {
                // the ring is done with (all its products have been read); the other warps
                // meet this barrier and the last one after their loops
#pragma unroll
                for (int m = 0; m < NM; ++m)
#pragma unroll
                    for (int c = 0; c < BN; c += 2) {
                        float u, v;
                        unpack(acc[m][c / 2], u, v);
                        part[(m * BN + c) * kRows + r] = u;
                        part[(m * BN + c + 1) * kRows + r] = v;
                    }
                cluster_barrier();
                c0 = BN * rank / static_cast<int>(cs);
                c1 = BN * (rank + 1) / static_cast<int>(cs);
                for (int c = c0; c < c1; ++c) {
                    float sum[NM];
#pragma unroll
                    for (int m = 0; m < NM; ++m) {
                        const uint32_t at = smem_u32(part + (m * BN + c) * kRows + r);
                        float v[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] = k < static_cast<int>(cs) ? ld_cluster(cta_map(at, k)) : 0.f;
                        sum[m] = v[0];
#pragma unroll
                        for (int k = 1; k < 8; ++k) sum[m] += v[k];
                    }
                    if constexpr (DUAL) sum[0] = silu_mul(sum[0], sum[1]);
                    if (g.y_type == BQD_E4M3) {
                        part[c * kRows + r] = sum[0];
                        const uint32_t w = __reduce_max_sync(0xFFFFFFFFu, live ? abs_bits(sum[0]) : 0u);
                        if (lane == 0) s_max[sw][c] = w;
                    } else if (live && n0 + c < g.T) {
                        store_y(y, g.y_type, static_cast<int64_t>(n0 + c) * g.M + row, sum[0]);
                    }
                }
            } else {
#pragma unroll
                for (int c = 0; c < BN; c += 2) {
                    float v[2];
                    unpack(acc[0][c / 2], v[0], v[1]);
                    if constexpr (DUAL) {
                        float u[2];
                        unpack(acc[1][c / 2], u[0], u[1]);
                        v[0] = silu_mul(v[0], u[0]);
                        v[1] = silu_mul(v[1], u[1]);
                        acc[0][c / 2] = pack(v[0], v[1]);
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (DUAL && g.y_type == BQD_E4M3) {
                            const uint32_t w = __reduce_max_sync(0xFFFFFFFFu, live ? abs_bits(v[e]) : 0u);
                            if (lane == 0) s_max[sw][c + e] = w;
                        } else if (live && n0 + c + e < g.T) {
                            store_y(y, g.y_type, static_cast<int64_t>(n0 + c + e) * g.M + row, v[e]);
                        }
                    }
                }
            }
            if (DUAL && g.y_type == BQD_E4M3) {
                named_sync(1, kSumWarps * kWarp);
                auto code = [&](int c, float v) {
                    const float s = block_scale(max(max(s_max[0][c], s_max[1][c]), max(s_max[2][c], s_max[3][c])));
                    if (n0 + c < g.T) {
                        if (live)
                            static_cast<uint8_t*>(y)[static_cast<int64_t>(n0 + c) * g.M + row] =
                                static_cast<uint8_t>(BlockCoder(s).one(v));
                        if (r == 0) ys[static_cast<int64_t>(mt) * g.T + n0 + c] = s;
                    }
                };
                if (cs > 1) {
                    for (int c = c0; c < c1; ++c) code(c, part[c * kRows + r]);
                } else {
#pragma unroll
                    for (int c = 0; c < BN; c += 2) {
                        float u, v;
                        unpack(acc[0][c / 2], u, v);
                        code(c, u);
                        code(c + 1, v);
                    }
                }
                named_sync(1, kSumWarps * kWarp);  // before the next tile's maxima
            }
        }
        tc_before();
    }
    if (!ok) let_copies_land();
    if (cs > 1) {
        // a cluster takes one tile, so each warp meets two barriers: parts written, parts read
        __syncwarp();
        if (warp < 2) cluster_barrier();
        cluster_barrier();
    }
    __syncthreads();
    if (warp == 1) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kTmem) : "memory");
    }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
        cudaGetLastError();
    });
    return fn;
}

// Codes [rows][K] in boxes of 128 k x `box` rows; k and rows past the ends read as zero.
bool codes_map(CUtensorMap* map, const uint8_t* codes, int64_t rows, int64_t K, int box)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K)};
    const cuuint32_t boxes[2] = {kBlk, static_cast<cuuint32_t>(box)};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, boxes, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, bool DUAL>
cudaError_t launch_narrow(const Fp8GemmArgs& a, cudaStream_t s)
{
    using S = Narrow<BN, DUAL>;
    CUtensorMap w0, w1, x;
    if (!codes_map(&w0, a.w0, a.M, a.K, kRows) || !codes_map(&w1, DUAL ? a.w1 : a.w0, a.M, a.K, kRows) ||
        !codes_map(&x, a.x, a.T, a.K, BN))
        return cudaErrorInvalidValue;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    auto kern = fp8_gemm_kernel<BN, DUAL>;
    static OccCache occ;
    blocks_per_sm(occ, reinterpret_cast<const void*>(kern), dev, kThreads, S::kSmem);
    GemmShape g{};
    g.M = a.M;
    g.T = static_cast<int>(a.T);
    g.KB = static_cast<int>((a.K + kBlk - 1) / kBlk);
    g.tilesM = static_cast<int>((a.M + kRows - 1) / kRows);
    g.tilesT = static_cast<int>((a.T + BN - 1) / BN);
    g.y_type = a.y_type;
    const int64_t tiles = static_cast<int64_t>(g.tilesM) * g.tilesT, slots = static_cast<int64_t>(dev_info(dev).sms) * S::kCtas;
    int cs = 1;
    while (cs < 8 && tiles * cs * 2 <= slots && cs * 2 <= g.KB) cs *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cs > 1 ? tiles * cs : tiles < slots ? tiles : slots));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int na = 0;
    if (cs > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = static_cast<unsigned>(cs);
        attr[na].val.clusterDim.y = 1;
        attr[na].val.clusterDim.z = 1;
        ++na;
    }
    if (launch_flags() & kLaunchPdl) {
        attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[na].val.programmaticStreamSerializationAllowed = 1;
        ++na;
    }
    cfg.attrs = attr;
    cfg.numAttrs = static_cast<unsigned>(na);
    return cudaLaunchKernelEx(&cfg, kern, w0, w1, x, a.s0, a.s1, a.xs, a.y, a.ys, g);
}

}  // namespace

bool fp8_gemm_supported(int64_t M, int64_t K, int64_t T)
{
    return K >= 16 && K % 16 == 0 && K <= (int64_t(1) << 24) && M >= 1 && M <= (int64_t(1) << 30) && T >= 1 &&
           T <= (int64_t(1) << 30) && (M + 127) / 128 <= (int64_t(1) << 30) / ((T + 15) / 16);
}

cudaError_t launch_fp8_gemm(const Fp8GemmArgs& a, bool dual, cudaStream_t s)
{
    if (dual) {
        if (a.T <= 16) return launch_narrow<16, true>(a, s);
        if (a.T <= 32) return launch_narrow<32, true>(a, s);
        return launch_narrow<64, true>(a, s);
    }
    if (a.T <= 16) return launch_narrow<16, false>(a, s);
    if (a.T <= 32) return launch_narrow<32, false>(a, s);
    if (a.T <= 64) return launch_narrow<64, false>(a, s);
    return launch_narrow<128, false>(a, s);
}

cudaError_t read_and_clear_fp8_error(unsigned int* out)
{
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_fp8_error, sizeof(v));
    if (e != cudaSuccess) return e;
    *out = v;
    if (v) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_fp8_error, &zero, sizeof(zero));
    }
    return e;
}

}  // namespace bqd
