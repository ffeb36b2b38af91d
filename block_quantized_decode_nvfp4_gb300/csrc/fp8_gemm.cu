// fp8_gemm.cu -- 8-bit activations times FP8 block-128 weights on the
// 5th-generation tensor cores:
//   y[t][m] = sum_kb xs[kb][t] ws[m/128][kb] sum_{k in block kb} x[t][k] w[m][k],
// and the gated pair h[t][i] = SiLU(g) u of two such products, g and u. Here: up
// to 64 tokens, whose bound is the one read of the weights; fp8_gemm_tokens.cu
// and fp8_gemm_pairs.cu have the kernels for more.
//
// The tensor cores add up the 128 k of a block (E4M3 products, fp32 sums); the
// blocks' sums meet their two scales in fp32 registers. A CTA computes 128 rows
// of a weight (the MMA's M, one tile of scales) times BN tokens (its N: 16, 32 or
// 64, so that few tokens take little of the ring, the products and the sums), two
// CTAs to an SM:
//  - warps 0 and 1 copy a block of 128 k each in turn into a ring by 2-D tensor
//    copies (128-byte swizzle; rows, tokens and k past the ends read as zero);
//  - warps 2 and 3, one elected lane of each, issue the MMAs (K = 32 each) of
//    every other block into one of a few buffers of tensor memory. A thread takes
//    about 450 cycles for a block's waits and copies or products, and the blocks
//    do not depend on one another: hence two of each;
//  - the other warps read a buffer (a row of the weights per thread), scale it
//    and add it to their registers.
// With few tiles the k blocks of one are shared by a cluster of CTAs, and so are
// the two weights of a gated pair. Each CTA then has a share of the tile's
// tokens: the others write their parts into its shared memory, and it adds them
// up in the order of the k blocks: the same bits every time. With many tiles of
// one weight, a CTA takes tile after tile, and its ring runs on from one to the
// next.
//
// One token: 151936 x 4096 92 to 94 us (6.7 TB/s, the rate of a copy), 12288 x 4096 11.0
// us in calls that follow one another (10.7 with BQD_LAUNCH_PDL), of which the weights
// stream for 7.8 (6.4 TB/s); the rest is the wait for the call before, the first bytes
// and the last sums with the cluster's exchange, 1 to 1.5 us each. 16, 32, 64 tokens:
// 11.6, 12.9, 14.8 us. A gated pair of 12288 x 4096 by 64 tokens 25 us: its 192 CTAs lie
// unevenly on 152 SMs, and the exchange, whole fp32 parts of both weights, and outputs
// take 5 of them. Copies by cp.async from four warps instead of tensor copies: 14.4 us for
// one token, and twice as long as now where tokens are many. The first weights are called
// into the L2 ahead of the wait for the call before: without that one and 32 tokens take
// 11.6 and 13.5 us, 4096 x 12288 by 17 12.7 in place of 12.2.
// Every wait for an mbarrier is bounded (kErrWaitTimeout in the kernel's error word), and
// begins after the kernel before has completed. The others have no limit: all warps reach
// the barriers of the block and of the cluster, after a wait that ran out too, and tensor
// memory is there when it is asked for (see kSmem: who may lie beside one of these CTAs).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "common.cuh"
#include "f32x2.cuh"
#include "fp8.cuh"
#include "fp8_gemm.cuh"
#include "fp8.h"
#include "host_util.h"
#include "stream.cuh"

namespace bqd {

__device__ unsigned int g_fp8_error = 0;

namespace {

using namespace fp8;

template <int BN>
struct Narrow {
    static constexpr int kCtas = 2;  // per SM
    static constexpr int kSumWarps = BN > 32 ? 8 : 4;
    static constexpr int kGroups = kSumWarps / 4;  // of 128 threads, a row of the weights each
    static constexpr int kThreads = (4 + kSumWarps) * kWarp;
    static constexpr int kTileX = BN * kBlk;
    static constexpr int kStage = kTileBytes + kTileX;
    static constexpr int kParts = (BN + kMaxCluster - 1) * kRows * 4;  // a cluster's parts of this CTA's tokens
    static constexpr bool kOver = BN > 32;  // they lie over the ring: its room is worth more than a barrier
    static constexpr int kRoom = 109 * 1024 - (kOver ? 0 : kParts);
    static constexpr int kStages = kRoom / kStage / 2 < 4 ? kRoom / kStage / 2 * 2 : 8;  // even: each for one warp
    // (+ alignment slack.) No less than two CTAs leave each other: a kernel that takes all of an SM's
    // tensor memory, and more than half of its shared memory, then never comes to lie beside one of
    // these, and no CTA of a cluster waits for tensor memory whose holder waits for a peer of its own
    static constexpr int kNeed = kStages * kStage + (kOver ? 0 : kParts) + 1024, kSmem = kNeed > 109 * 1024 ? kNeed : 109 * 1024;
    static_assert(2 * (kSmem + 4096) <= 228 * 1024, "two CTAs on an SM, with their static shared memory");
    static constexpr int kBufs = 512 / kCtas / BN < 4 ? 512 / kCtas / BN : 4;
    static constexpr int kTmem = kBufs * BN;
    static constexpr int kCols = BN / kGroups;  // columns of a thread
    static constexpr int kAhead = BN == 64 ? 2 : 4;  // blocks whose scales are on their way
    // Registers of a thread at launch, of the first four warps and of those of the sums: with the same for
    // all, a few of them went to memory and back, block after block (12288 x 4096 by 64 tokens 17.7 us, the
    // pair 28.9, where these take 15.6 and 25.2; 32 tokens 14.1 and 13.8). 16 tokens fit.
    static constexpr bool kSplit = BN > 16;
    static constexpr int kRegs = BN == 64 ? 80 : 128, kFewRegs = BN == 64 ? 56 : 72, kSumRegs = BN == 64 ? 88 : 184;
    static_assert(!kSplit || 4 * kWarp * kFewRegs + kSumWarps * kWarp * kSumRegs <= kThreads * kRegs, "the split of the registers");
    static_assert(BN % 16 == 0 && BN >= 16 && BN <= 64, "the MMA's N, and the threads' registers");
    static_assert(kTmem >= 32 && kTmem <= 512 / kCtas && (kTmem & (kTmem - 1)) == 0, "an SM's CTAs share 512 columns");
    static_assert(kStages >= 2 && kStages % 2 == 0 && kBufs % 2 == 0, "a stage and a buffer for each of two warps");
    static_assert(!kOver || kParts <= kStages * kStage, "the parts fit the ring");
    static_assert(kTileX % 1024 == 0, "stages start on 1024-byte boundaries (swizzle atoms)");
};

template <int BN>
__global__ void __launch_bounds__(Narrow<BN>::kThreads, Narrow<BN>::kCtas)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap map_w0, const __grid_constant__ CUtensorMap map_w1,
                    const __grid_constant__ CUtensorMap map_x, const __grid_constant__ GemmShape g)
{
    using S = Narrow<BN>;
    constexpr int H = S::kCols, kAhead = S::kAhead;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[S::kStages], empty[S::kStages], dfull[S::kBufs], dempty[S::kBufs], got;
    __shared__ uint32_t s_tmem;
    __shared__ __align__(16) float s_scale[S::kSumWarps][2][H];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;

    // This cluster's tiles, and this CTA's weight and blocks of k of each
    uint32_t ranks_;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks_));
    const int ranks = static_cast<int>(ranks_), rank = ranks > 1 ? static_cast<int>(cta_rank()) : 0;
    const int mat = g.mats > 1 ? rank & 1 : 0, cs = ranks / g.mats, ks = rank / g.mats;
    const int tiles = g.tilesM, step = static_cast<int>(gridDim.x) / ranks;
    const int tile0 = static_cast<int>(blockIdx.x) / ranks;
    const int kb0 = static_cast<int>(static_cast<int64_t>(g.KB) * ks / cs);
    const int nkb = static_cast<int>(static_cast<int64_t>(g.KB) * (ks + 1) / cs) - kb0;
    const CUtensorMap* map_w = mat ? &map_w1 : &map_w0;

    if (threadIdx.x == 0) {
        prefetch_map(map_w);
        prefetch_map(&map_x);
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < S::kBufs; ++i) {
            mbar_init(&dfull[i], 1);
            mbar_init(&dempty[i], S::kSumWarps);
        }
        mbar_init(&got, 1);
        fence_barrier_init();
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                     "r"(S::kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = s_tmem;
    float* parts = reinterpret_cast<float*>(ring + (S::kOver ? 0 : S::kStages * S::kStage));  // [part][token][row]
    if (ranks > 1) {
        if (threadIdx.x == 0) {
            mbar_arrive_expect_tx(&got, ranks * ((g.T - rank + ranks - 1) / ranks) * (kRows * 4));
        }
        __syncwarp();
        cluster_arrive();  // its barrier may be counted at
    }

    bool ok = true;
    if constexpr (S::kSplit) {
        if (warp < 4)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kFewRegs));
        else
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kSumRegs));
    }
    if (warp < 2) {
        // ------------------------------------------------ copies, of every other block
        if (lane == 0) {
            auto copy_w = [&](int st, int tile, int kb) {
                mbar_arrive_expect_tx(&full[st], S::kStage);
                tma_2d(smem_u32(ring + st * S::kStage), map_w, kb * kBlk, tile * kRows, &full[st]);
            };
            auto copy_x = [&](int st, int kb) {
                tma_2d(smem_u32(ring + st * S::kStage + kTileBytes), &map_x, kb * kBlk, 0, &full[st]);
            };
            // the first stages' weights before the wait for the previous kernel, whose output x may be
            const int first = min(S::kStages, nkb);
            if (g.early)
                for (int i = warp; i < first; i += 2) copy_w(i, tile0, kb0 + i);
            fp8_pdl_wait();
            for (int i = warp; i < first; i += 2) {
                if (!g.early) copy_w(i, tile0, kb0 + i);
                copy_x(i, kb0 + i);
            }
            int it = first;
            for (int tile = tile0; tile < tiles && ok; tile += step) {
                for (int i = tile == tile0 ? first : 0; i < nkb; ++i, ++it) {
                    if ((it & 1) != warp) continue;
                    const int st = it % S::kStages;
                    if (it >= S::kStages) ok = mbar_wait(&empty[st], ((it / S::kStages) & 1) ^ 1, &g_fp8_error);
                    if (!ok) break;
                    copy_w(st, tile, kb0 + i);
                    copy_x(st, kb0 + i);
                }
            }
            // The next kernel's start may overlap this one's end. No earlier: CTAs of the calls behind
            // it would take the SMs' places and leave this one's unevenly spread.
            fp8_pdl_trigger();
        }
        __syncwarp();
    } else if (warp < 4) {
        // ------------------------------------------------ products, of every other block
        // (the tokens come after the kernel before this one has completed, however long it stays: no time of it counts
        // for the bounded waits)
        fp8_pdl_wait();
        constexpr uint32_t idesc = fp8_idesc(kRows, BN);
        int it = 0;
        for (int tile = tile0; tile < tiles && ok; tile += step) {
            for (int i = 0; i < nkb; ++i, ++it) {
                if ((it & 1) != warp - 2) continue;
                const int st = it % S::kStages, b = it % S::kBufs;
                ok = fp8_wait(&full[st], (it / S::kStages) & 1, &g_fp8_error);
                if (ok && it >= S::kBufs) ok = fp8_wait(&dempty[b], ((it / S::kBufs) & 1) ^ 1, &g_fp8_error);
                if (!ok) break;
                tc_after();
                if (fp8_elect()) {
                    const uint32_t at = smem_u32(ring + st * S::kStage);
#pragma unroll
                    for (int j = 0; j < kBlk / 32; ++j)
                        fp8_mma(tmem + b * BN, fp8_desc(at + 32 * j), fp8_desc(at + kTileBytes + 32 * j), idesc, j != 0 ? 1u : 0u);
                    fp8_commit(&empty[st]);
                    fp8_commit(&dfull[b]);
                }
                __syncwarp();
            }
        }
    } else {
        // ------------------------------------------------ sums: a row of the weights and kCols tokens per thread
        const int q = warp % 4, sw = warp - 4, c0 = sw / 4 * H;  // tensor-memory lane quarter; columns
        const uint32_t base = tmem + (static_cast<uint32_t>(32 * q) << 16) + c0;
        const int r = 32 * q + lane;
        constexpr int L = (H + kWarp - 1) / kWarp;  // tokens of a lane when it fetches scales
        int it = 0;
        if (sw < 4 && step >= tiles) call_weights(g, mat, static_cast<int64_t>(tile0) * kRows + r, kb0, nkb);
        fp8_pdl_wait();
        for (int tile = tile0; tile < tiles; tile += step) {
            uint64_t acc[H / 2];
#pragma unroll
            for (int c = 0; c < H / 2; ++c) acc[c] = 0;
            float far_x[kAhead][L], far_w[kAhead];
            const float* ws = g.s[mat] + static_cast<int64_t>(tile) * g.KB + kb0;
            const float* xs = g.xs + static_cast<int64_t>(kb0) * g.T + c0 + lane;
            auto fetch = [&](int slot, int i) {
#pragma unroll
                for (int l = 0; l < L; ++l)
                    far_x[slot][l] = i < nkb && c0 + lane + l * kWarp < g.T && (H % kWarp == 0 || lane + l * kWarp < H)
                                         ? __ldg(xs + static_cast<int64_t>(i) * g.T + l * kWarp)
                                         : 0.f;
                far_w[slot] = i < nkb ? __ldg(ws + i) : 0.f;
            };
#pragma unroll
            for (int i = 0; i < kAhead; ++i) fetch(i, i);
            for (int i0 = 0; i0 < nkb; i0 += kAhead) {
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {  // a register of scales on their way may not be moved
                    const int i = i0 + u;
                    if (i >= nkb) break;
                    // the block's scales, to where every lane reads them all
                    float* sc = s_scale[sw][it & 1];
#pragma unroll
                    for (int l = 0; l < L; ++l)
                        if (H % kWarp == 0 || lane + l * kWarp < H) sc[lane + l * kWarp] = far_x[u][l] * far_w[u];
                    fetch(u, i + kAhead);
                    const int b = it % S::kBufs;
                    // After a wait that ran out the loops go on without waiting, so that the warps
                    // still meet at every barrier.
                    if (ok) ok = fp8_wait(&dfull[b], (it / S::kBufs) & 1, &g_fp8_error);
                    __syncwarp();  // the scales are there
                    tc_after();
                    constexpr int D = 16;  // columns at a time
#pragma unroll
                    for (int c = 0; c < H; c += D) {
                        uint32_t d[D];
                        tmem_load<D>(base + b * BN + c, d);
                        tmem_wait_ld();
                        if (c + D == H) {  // the buffer has been read
                            tc_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&dempty[b]);
                        }
                        const float4* s4 = reinterpret_cast<const float4*>(sc + c);
#pragma unroll
                        for (int e = 0; e < D / 4; ++e) {
                            const float4 f = s4[e];
                            uint64_t* o = &acc[(c + 4 * e) / 2];
                            o[0] = fma2(pack(__uint_as_float(d[4 * e]), __uint_as_float(d[4 * e + 1])), pack(f.x, f.y), o[0]);
                            o[1] = fma2(pack(__uint_as_float(d[4 * e + 2]), __uint_as_float(d[4 * e + 3])), pack(f.z, f.w), o[1]);
                        }
                    }
                    ++it;
                }
            }
            if (ranks > 1) {
                // the parts to their tokens' CTAs
                __syncwarp();
                cluster_wait();
                if (S::kOver) {  // once every ring of the cluster is done with
                    cluster_arrive();
                    cluster_wait();
                }
                const int most = (g.T + ranks - 1) / ranks;
                const uint32_t mine = smem_u32(parts) + static_cast<uint32_t>(rank * most * kRows + r) * 4;
                int to = c0 % ranks, j = c0 / ranks;
#pragma unroll
                for (int c = 0; c < H; c += 2) {
                    float v[2];
                    unpack(acc[c / 2], v[0], v[1]);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (c0 + c + e < g.T)
                            st_async(cta_map(mine + j * (kRows * 4), to), v[e], cta_map(smem_u32(&got), to));
                        if (++to == ranks) {
                            to = 0;
                            ++j;
                        }
                    }
                }
            } else {
                const int64_t row = static_cast<int64_t>(tile) * kRows + r;
                if (row < g.M) {
#pragma unroll
                    for (int c = 0; c < H; c += 2) {
                        float u, v;
                        unpack(acc[c / 2], u, v);
                        const int64_t at = static_cast<int64_t>(c0 + c) * g.M + row;
                        if (c0 + c < g.T) store_y(g.y, g.y_type, at, u);
                        if (c0 + c + 1 < g.T) store_y(g.y, g.y_type, at + g.M, v);
                    }
                }
            }
        }
        tc_before();
    }
    if (!ok) let_copies_land();
    if (ranks > 1) {
        // ---- a cluster takes one tile: this CTA's tokens
        __syncwarp();
        if (warp < 4) {
            cluster_wait();
            if (S::kOver) {
                cluster_arrive();
                cluster_wait();
            }
        } else {
            // (four times the limit of the other waits: a CTA that gives up one of those still stores)
            if (!fp8_wait_cluster(&got, 0, &g_fp8_error, 4 * kWaitCycles)) ok = false;
            finish_tokens<false>(g, parts, (g.T + ranks - 1) / ranks, (g.T - rank + ranks - 1) / ranks, ranks, tile0, rank, ranks, 0,
                                 warp - 4, S::kSumWarps);
        }
    }
    __syncthreads();
    if (warp == 2) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kTmem) : "memory");
    }
}

template <int BN>
cudaError_t launch_narrow(const Fp8GemmArgs& a, bool dual, cudaStream_t s)
{
    using S = Narrow<BN>;
    CUtensorMap w0, w1, x;
    if (!fp8_codes_map(&w0, a.w0, a.M, a.K, kRows) || !fp8_codes_map(&x, a.x, a.T, a.K, BN)) return cudaErrorInvalidValue;
    if (!dual)
        w1 = w0;
    else if (!fp8_codes_map(&w1, a.w1, a.M, a.K, kRows))
        return cudaErrorInvalidValue;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    auto kern = fp8_gemm_kernel<BN>;
    static OccCache occ;
    blocks_per_sm(occ, reinterpret_cast<const void*>(kern), dev, S::kThreads, S::kSmem);
    // the split of the registers needs what the block is launched with
    if (S::kSplit && launch_regs(occ, reinterpret_cast<const void*>(kern), dev) < S::kRegs) return cudaErrorInvalidConfiguration;
    GemmShape g{};
    g.w[0] = a.w0;
    g.w[1] = a.w1;
    g.K = a.K;
    g.s[0] = a.s0;
    g.s[1] = a.s1;
    g.xs = a.xs;
    g.y = a.y;
    g.ys = a.ys;
    g.M = a.M;
    g.T = static_cast<int>(a.T);
    g.KB = static_cast<int>((a.K + kBlk - 1) / kBlk);
    g.tilesM = static_cast<int>((a.M + kRows - 1) / kRows);
    g.tilesT = 1;
    g.mats = dual ? 2 : 1;
    g.y_type = a.y_type;
    g.whole = a.M % 4 == 0;  // y starts on 16 bytes
    g.early = (launch_flags() & kLaunchPdl) != 0;
    // the k blocks of a tile over as many CTAs as may be (with one weight and many tiles: a CTA
    // for tile after tile)
    const int64_t tiles = g.tilesM, slots = static_cast<int64_t>(dev_info(dev).sms) * S::kCtas;
    static ClusterCache clusters;
    const int ranks =
        g.mats * share_k(clusters, reinterpret_cast<const void*>(kern), dev, S::kThreads, S::kSmem, S::kCtas, tiles, g.mats, g.KB);
    return launch_clusters(kern, static_cast<unsigned>(ranks > 1 ? tiles * ranks : tiles < slots ? tiles : slots), ranks,
                           S::kThreads, S::kSmem, s, w0, w1, x, g);
}

}  // namespace

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn encode_fn()
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

bool fp8_codes_map(CUtensorMap* map, const uint8_t* codes, int64_t rows, int64_t K, int box)
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

bool fp8_rows_map(CUtensorMap* map, void* y, int y_type, int64_t rows, int64_t M, int box, int line)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const int size = y_type == BQD_F32 ? 4 : 2;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(M), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(M) * size};
    const cuuint32_t boxes[2] = {static_cast<cuuint32_t>(line / size), static_cast<cuuint32_t>(box)};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, y_type == BQD_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, y, dims, strides,
              boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool fp8_gemm_supported(int64_t M, int64_t K, int64_t T)
{
    return K >= 16 && K % 16 == 0 && K <= (int64_t(1) << 24) && M >= 1 && M <= (int64_t(1) << 30) && T >= 1 &&
           T <= (int64_t(1) << 30) && (M + 127) / 128 <= (int64_t(1) << 30) / ((T + 15) / 16);
}

cudaError_t launch_fp8_gemm(const Fp8GemmArgs& a, bool dual, cudaStream_t s)
{
    if (fp8_gemm_wants_pairs(a, dual)) return launch_fp8_gemm_pairs(a, dual, s);
    if (a.T <= 16) return launch_narrow<16>(a, dual, s);
    if (a.T <= 32) return launch_narrow<32>(a, dual, s);
    if (a.T <= 64) return launch_narrow<64>(a, dual, s);
    return launch_fp8_gemm_tokens(a, dual, s);
}

cudaError_t read_and_clear_fp8_error(unsigned int* out)
{
    unsigned int v = 0, w = 0;
    unsigned int x = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_fp8_error, sizeof(v));
    if (e == cudaSuccess) e = read_and_clear_fp8_pairs_error(&w);
    if (e == cudaSuccess) e = read_and_clear_fp8_tokens_error(&x);
    if (e != cudaSuccess) return e;
    *out = v | w | x;
    if (v) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_fp8_error, &zero, sizeof(zero));
    }
    return e;
}

}  // namespace bqd
