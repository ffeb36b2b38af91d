// fp8_gemm_tokens.cu -- the products of fp8_gemm.cu for more than 64 tokens, where
// neither the one read of the weights bounds a call nor are there tiles enough
// for the pairs of fp8_gemm_pairs.cu: 128 tokens x 128 rows of a weight per CTA.
//
// Tokens lie on the tensor cores' rows, so a block's scales are one register for
// a thread's token times one value for all its columns. (With the tokens as
// columns every thread fetches all their scales from shared memory, 16 loads of 16
// bytes a block: 4096 x 12288 by 512 tokens took 48 us where this takes 40.) The
// bound is what an SM is given of the L2, 32 KiB a block of k at about 55 bytes a
// cycle, behind it the port of shared memory, 32 KiB in and 32 KiB out, 512 cycles,
// twice what the MMAs take: a block takes 0.33 us, without sums 0.31, without
// copies 0.24. 4870 x 4096 by 333 tokens: 15.8 us, 4096 x 4096 by 512 14.2.
//  - warps 0 and 1 copy every other block of k; warps 2 and 3 issue every other
//    block's MMAs (M = 128, N = 128, K = 32) into one of four buffers;
//  - warps 4..11 read a buffer, 64 columns of a token a thread, scale it and add
//    it to their registers.
// A tile's k blocks, and the two weights of a gated pair, are shared by a cluster
// as in fp8_gemm.cu; a CTA lays its part out in shared memory, and whole rows of it
// are copied to the CTAs that have their tokens. Without a cluster a CTA takes tile
// after tile.
// Every wait for an mbarrier is bounded (kErrWaitTimeout in the kernel's error word), and
// begins after the kernel before has completed. The others have no limit: all warps reach
// the barriers of the block and of the cluster, after a wait that ran out too, and no
// kernel with tensor memory fits beside a CTA's shared memory.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "f32x2.cuh"
#include "fp8.cuh"
#include "fp8_gemm.cuh"
#include "fp8.h"
#include "host_util.h"
#include "stream.cuh"

namespace bqd {

__device__ unsigned int g_fp8_tokens_error = 0;

namespace {

using namespace fp8;

constexpr int kTok = 128;                             // tokens of a tile (MMA M)
constexpr int kStage = 2 * kTileBytes;                // tokens, then weights
constexpr int kStages = 4;
constexpr int kBufs = 4;
constexpr int kSumWarps = 8;
constexpr int kThreads = (4 + kSumWarps) * kWarp;
constexpr int kLineBytes = 128;                       // of a token's outputs, staged by a warp at once
constexpr int kRowBytes = kRows * 4;                  // a token's part
constexpr int kParts = (kTok + kMaxCluster - 1) * kRowBytes;
constexpr int kSmem = kStages * kStage + kParts + 1024;  // + alignment slack
// 128 x 56 + 256 x 224 are the 384 x 168 registers that the block has
constexpr int kRegs = 168, kFewRegs = 56, kSumRegs = 224;
static_assert(4 * kWarp * kFewRegs + kSumWarps * kWarp * kSumRegs <= kThreads * kRegs, "the split of the registers");
static_assert(kSmem <= 227 * 1024 - 512, "shared memory of one CTA, static beside it");
static_assert(kSumWarps * kWarp * kLineBytes <= kParts, "without a cluster outputs are staged where parts would come");
static_assert(kTok * kRowBytes <= kStages * kStage, "a CTA's part is laid out over its ring");
static_assert(kStages % 2 == 0 && kBufs % 2 == 0, "a stage and a buffer for each of two warps");

__global__ void __launch_bounds__(kThreads, 1)
    fp8_tokens_kernel(const __grid_constant__ CUtensorMap map_w0, const __grid_constant__ CUtensorMap map_w1,
                      const __grid_constant__ CUtensorMap map_x, const __grid_constant__ GemmShape g)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[kStages], empty[kStages], dfull[kBufs], dempty[kBufs], got;
    __shared__ uint32_t s_tmem;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* parts = reinterpret_cast<float*>(ring + kStages * kStage);  // [part][token][row]
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;

    // This cluster's tiles, and this CTA's weight and blocks of k of each
    uint32_t ranks_;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks_));
    const int ranks = static_cast<int>(ranks_), rank = ranks > 1 ? static_cast<int>(cta_rank()) : 0;
    const int mat = g.mats > 1 ? rank & 1 : 0, cs = ranks / g.mats, ks = rank / g.mats;
    const int tiles = g.tilesM * g.tilesT, step = static_cast<int>(gridDim.x) / ranks;
    const int tile0 = static_cast<int>(blockIdx.x) / ranks;
    const int kb0 = static_cast<int>(static_cast<int64_t>(g.KB) * ks / cs);
    const int nkb = static_cast<int>(static_cast<int64_t>(g.KB) * (ks + 1) / cs) - kb0;
    const CUtensorMap* map_w = mat ? &map_w1 : &map_w0;
    // the first tile's tokens, and which of them are this CTA's, with a cluster
    const int n0 = tile0 % g.tilesT * kTok, here = min(kTok, g.T - n0), most = (here + ranks - 1) / ranks;
    const int own0 = here * rank / ranks, own = here * (rank + 1) / ranks - own0;

    if (threadIdx.x == 0) {
        prefetch_map(map_w);
        prefetch_map(&map_x);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(&dfull[i], 1);
            mbar_init(&dempty[i], kSumWarps);
        }
        mbar_init(&got, 1);
        fence_barrier_init();
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = s_tmem;
    if (ranks > 1) {
        if (threadIdx.x == 0) mbar_arrive_expect_tx(&got, static_cast<uint32_t>(ranks * own) * kRowBytes);
        __syncwarp();
        cluster_arrive();  // its barrier may be counted at
    }

    bool ok = true;
    if (warp < 4)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    else
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
    if (warp < 2) {
        // ------------------------------------------------ copies, of every other block
        if (lane == 0) {
            auto copy_w = [&](int st, int tile, int kb) {
                mbar_arrive_expect_tx(&full[st], kStage);
                tma_2d(smem_u32(ring + st * kStage + kTileBytes), map_w, kb * kBlk, tile / g.tilesT * kRows, &full[st]);
            };
            auto copy_x = [&](int st, int tile, int kb) {
                tma_2d(smem_u32(ring + st * kStage), &map_x, kb * kBlk, tile % g.tilesT * kTok, &full[st]);
            };
            // the first stages' weights before the wait for the previous kernel, whose output x may be
            const int first = min(kStages, nkb);
            if (g.early)
                for (int i = warp; i < first; i += 2) copy_w(i, tile0, kb0 + i);
            fp8_pdl_wait();
            for (int i = warp; i < first; i += 2) {
                if (!g.early) copy_w(i, tile0, kb0 + i);
                copy_x(i, tile0, kb0 + i);
            }
            int it = first;
            for (int tile = tile0; tile < tiles && ok; tile += step) {
                for (int i = tile == tile0 ? first : 0; i < nkb; ++i, ++it) {
                    if ((it & 1) != warp) continue;
                    const int st = it % kStages;
                    if (it >= kStages) ok = mbar_wait(&empty[st], ((it / kStages) & 1) ^ 1, &g_fp8_tokens_error);
                    if (!ok) break;
                    copy_w(st, tile, kb0 + i);
                    copy_x(st, tile, kb0 + i);
                }
            }
            fp8_pdl_trigger();
        }
        __syncwarp();
    } else if (warp < 4) {
        // ------------------------------------------------ products, of every other block
        // (the tokens come after the kernel before this one has completed, however long it stays: no time of it counts
        // for the bounded waits)
        fp8_pdl_wait();
        constexpr uint32_t idesc = fp8_idesc(kTok, kRows);
        int it = 0;
        for (int tile = tile0; tile < tiles && ok; tile += step) {
            for (int i = 0; i < nkb; ++i, ++it) {
                if ((it & 1) != warp - 2) continue;
                const int st = it % kStages, b = it % kBufs;
                ok = fp8_wait(&full[st], (it / kStages) & 1, &g_fp8_tokens_error);
                if (ok && it >= kBufs) ok = fp8_wait(&dempty[b], ((it / kBufs) & 1) ^ 1, &g_fp8_tokens_error);
                if (!ok) break;
                tc_after();
                if (fp8_elect()) {
                    const uint32_t at = smem_u32(ring + st * kStage);
#pragma unroll
                    for (int j = 0; j < kBlk / 32; ++j)
                        fp8_mma(tmem + b * kRows, fp8_desc(at + 32 * j), fp8_desc(at + kTileBytes + 32 * j), idesc, j != 0 ? 1u : 0u);
                    fp8_commit(&empty[st]);
                    fp8_commit(&dfull[b]);
                }
                __syncwarp();
            }
        }
    } else {
        // ------------------------------------------------ sums: a token and 64 columns per thread
        const int q = warp % 4, half = (warp - 4) / 4, r = 32 * q + lane;
        const uint32_t base = tmem + (static_cast<uint32_t>(32 * q) << 16) + 64 * half;
        int it = 0;
        if (half == 0) call_weights(g, mat, static_cast<int64_t>(tile0 / g.tilesT) * kRows + r, kb0, nkb);
        fp8_pdl_wait();
        for (int tile = tile0; tile < tiles; tile += step) {
            const int mt = tile / g.tilesT, t = tile % g.tilesT * kTok + r;
            const float* ws = g.s[mat] + static_cast<int64_t>(mt) * g.KB + kb0;
            const float* xs = g.xs + static_cast<int64_t>(kb0) * g.T + t;
            uint64_t sum[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) sum[c] = 0;
            // scales are on their way two blocks ahead, and a block's columns while the one before
            // it is added up (in registers of their own: none on its way may be moved)
            float far_x[2], far_w[2];
            auto fetch = [&](int u, int i) {
                far_x[u] = i < nkb && t < g.T ? __ldg(xs + static_cast<int64_t>(i) * g.T) : 0.f;
                far_w[u] = i < nkb ? __ldg(ws + i) : 0.f;
            };
            uint32_t d[2][64];
            // After a wait that ran out the loops go on without waiting, so that the warps still
            // meet at every barrier.
            auto begin = [&](int u, bool ready) {
                const int b = it % kBufs;
                if (!__all_sync(0xFFFFFFFFu, ready) && ok) ok = fp8_wait(&dfull[b], (it / kBufs) & 1, &g_fp8_tokens_error);
                tc_after();
                tmem_load<32>(base + b * kRows, d[u]);
                tmem_load<32>(base + b * kRows + 32, d[u] + 32);
            };
            fetch(0, 0);
            fetch(1, 1);
            begin(0, false);
            for (int i0 = 0; i0 < nkb; i0 += 2) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int i = i0 + u;
                    if (i >= nkb) break;
                    const float f = far_x[u] * far_w[u];
                    fetch(u, i + 2);
                    const int b = it % kBufs;
                    ++it;
                    const bool ready = fp8_look(&dfull[it % kBufs], (it / kBufs) & 1);  // of the next: a look
                    tmem_wait_ld();
                    tc_before();  // the buffer has been read
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&dempty[b]);
                    if (i + 1 < nkb) begin(u ^ 1, ready);
                    const uint64_t ff = pack(f, f);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        sum[e] = fma2(pack(__uint_as_float(d[u][2 * e]), __uint_as_float(d[u][2 * e + 1])), ff, sum[e]);
                }
            }
            float acc[64];
#pragma unroll
            for (int c = 0; c < 32; ++c) unpack(sum[c], acc[2 * c], acc[2 * c + 1]);
            if (ranks > 1) {
                // the CTA's part, a token's 128 rows in 512 bytes (16 bytes i at i ^ token % 32), over the ring, which
                // is done with (all its products have been read); then rows of it to their tokens' CTAs
                float4* mine = reinterpret_cast<float4*>(ring + r * kRowBytes);
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    mine[(16 * half + c) ^ (r & 31)] = make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]);
                fence_async_smem();  // read by the copies
                __syncwarp();
                named_sync(1, kSumWarps * kWarp);
                cluster_wait();
                if (warp == 4 && lane < ranks) {
                    const int a = here * lane / ranks, n = here * (lane + 1) / ranks - a;
                    if (n > 0)
                        bulk_s2s(cta_map(smem_u32(parts) + static_cast<uint32_t>(rank * most) * kRowBytes, lane),
                                 smem_u32(ring + a * kRowBytes), static_cast<uint32_t>(n) * kRowBytes,
                                 cta_map(smem_u32(&got), lane));
                }
                __syncwarp();
            } else {
                // outputs by whole lines, staged by each warp for itself
                uint8_t* stage = reinterpret_cast<uint8_t*>(parts) + (warp - 4) * (kWarp * kLineBytes);
                const int tok0 = t - lane, tokens = g.T - tok0;
                const int64_t m0 = static_cast<int64_t>(mt) * kRows + 64 * half, left = g.M - m0;
                if (g.y_type == BQD_BF16) {
                    uint4 v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float* x = acc + 8 * i;
                        v[i] = make_uint4(to_bf16x2(x[0], x[1]), to_bf16x2(x[2], x[3]), to_bf16x2(x[4], x[5]), to_bf16x2(x[6], x[7]));
                    }
                    store_lines<128>(stage, v, static_cast<uint8_t*>(g.y) + 2 * (static_cast<int64_t>(tok0) * g.M + m0), 2 * g.M,
                                     2 * left, tokens, g.align);
                } else {
#pragma unroll
                    for (int k = 0; k < 64; k += 32) {
                        uint4 v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float* x = acc + k + 4 * i;
                            v[i] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
                        }
                        store_lines<128>(stage, v, static_cast<uint8_t*>(g.y) + 4 * (static_cast<int64_t>(tok0) * g.M + m0 + k),
                                         4 * g.M, 4 * (left - k), tokens, g.align);
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
        } else {
            // (four times the limit of the other waits: a CTA that gives up one of those still copies)
            if (!fp8_wait_cluster(&got, 0, &g_fp8_tokens_error, 4 * kWaitCycles)) ok = false;
            finish_tokens<true>(g, parts, most, own, ranks, tile0 / g.tilesT, n0 + own0, 1, own0, warp - 4, kSumWarps);
        }
        __syncwarp();
        cluster_arrive();  // the copies from this shared memory have been counted where they went
        cluster_wait();
    }
    __syncthreads();
    if (warp == 2) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

}  // namespace

cudaError_t launch_fp8_gemm_tokens(const Fp8GemmArgs& a, bool dual, cudaStream_t s)
{
    CUtensorMap w0, w1, x;
    if (!fp8_codes_map(&w0, a.w0, a.M, a.K, kRows) || !fp8_codes_map(&x, a.x, a.T, a.K, kTok)) return cudaErrorInvalidValue;
    if (!dual)
        w1 = w0;
    else if (!fp8_codes_map(&w1, a.w1, a.M, a.K, kRows))
        return cudaErrorInvalidValue;
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static OccCache occ;
    const void* kern = reinterpret_cast<const void*>(fp8_tokens_kernel);
    blocks_per_sm(occ, kern, dev, kThreads, kSmem);
    // the split of the registers needs what the block is launched with
    if (launch_regs(occ, kern, dev) < kRegs) return cudaErrorInvalidConfiguration;
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
    g.tilesT = static_cast<int>((a.T + kTok - 1) / kTok);
    g.mats = dual ? 2 : 1;
    g.y_type = a.y_type;
    g.align = row_align(a.M, a.y_type);
    g.whole = a.M % 4 == 0;  // y starts on 16 bytes
    g.early = (launch_flags() & kLaunchPdl) != 0;
    const int64_t tiles = static_cast<int64_t>(g.tilesM) * g.tilesT, sms = dev_info(dev).sms;
    static ClusterCache clusters;
    const int ranks = g.mats * share_k(clusters, kern, dev, kThreads, kSmem, 1, tiles, g.mats, g.KB);
    return launch_clusters(fp8_tokens_kernel, static_cast<unsigned>(ranks > 1 ? tiles * ranks : tiles < sms ? tiles : sms), ranks,
                           kThreads, kSmem, s, w0, w1, x, g);
}

cudaError_t read_and_clear_fp8_tokens_error(unsigned int* out)
{
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_fp8_tokens_error, sizeof(v));
    if (e != cudaSuccess) return e;
    *out = v;
    if (v) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_fp8_tokens_error, &zero, sizeof(zero));
    }
    return e;
}

}  // namespace bqd
