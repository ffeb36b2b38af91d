// fp8_gemm_pairs.cu -- the products of fp8_gemm.cu for many tokens, where the
// tensor cores are the bound: pairs of CTAs (cta_group::2) on tiles of 256
// tokens x 256 rows of a weight, or x 128 rows of each of a gated pair.
//
// A CTA of a pair holds 128 tokens (the MMA's rows; its lanes of tensor memory)
// and half of the weight's rows in its ring, 32 KiB a block of 128 k, and the
// tensor cores of both read both halves: half the copies and reads of shared
// memory per product that a CTA alone needs, whose port would be the bound.
// Tokens lie on the lanes, so a block's scales are one register for a thread's
// token times one value for its columns. Per CTA:
//  - warp 0 copies the tokens of a block, warp 1 the weights (counted at the first CTA's
//    barriers);
//  - warps 2 and 3 of the first CTA issue every other block's MMAs (M = 256,
//    N = 256, K = 32) into one of two buffers of 256 columns;
//  - warps 4..11 read a buffer, 128 columns of a token a thread, scale it and
//    add it to 128 registers, while the next block's products run.
// Pairs are persistent, so the ring runs on over the outputs of a tile, which go
// through shared memory: rows of whole 16 bytes as boxes that the copy engine stores
// while the sums go on, others in whole lines.
//
// 12288 x 4096 by 8192 tokens: 284 to 297 us in a few calls (2.8 to 2.9 PFLOP/s), 316 to 328
// in many one after the other, under the power cap (2.5 to 2.6). A gated pair by 4099
// tokens, the same: 331 to 340 and 354 to 368 with 8-bit outputs, 312 to 319 with bf16 and
// 333 to 338 with fp32 ones in a few calls. A block takes about 750 cycles where the MMAs
// need 512: without the sums' multiply-adds 630, without their loads from tensor memory
// too 620, and without copies as well 560. A CTA's 32 KiB a block are 64 bytes a cycle at
// the MMAs' rate, and an SM is given about 55 by the L2: 600 cycles are the least for this
// tile, whatever the sums do. Those take 330 cycles by themselves (128 packed multiply-adds
// of an SM quarter and their loads); the rest are the block's scales and barriers, each
// access of which waits for the tensor cores' reads of shared memory. What did not shorten
// it, all with this tile (a wider one is not tried): rounds of 32 columns in place of 64, the next
// on its way or not (308 us where two of 64 took 308), 64 by one load (322), scalar
// multiply-adds (314), sixteen warps of 64 columns (378), buffers of 128 columns, one for
// each half of the warps (322), scales by warps of their own (380) or by asynchronous
// copies (362). Outputs cost about 30 us of the whole.
// Every wait for an mbarrier is bounded (kErrWaitTimeout in the kernel's error word). The
// others have no limit: all warps reach the barriers of the block and of the pair, after a
// wait that ran out too, the copies out end by themselves, and no kernel with tensor memory
// fits beside a CTA's shared memory.
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

__device__ unsigned int g_fp8_pairs_error = 0;

namespace {

using namespace fp8;
constexpr int kHalf = 128;                // tokens and weight rows of a CTA's half
constexpr int kTile = 2 * kHalf;          // tokens of a tile (MMA M), columns of a buffer (N)
constexpr int kHalfBytes = kHalf * kBlk;
constexpr int kStage = 2 * kHalfBytes;    // of one CTA
constexpr int kStages = 5;
constexpr int kBufs = 2;
constexpr int kSumWarps = 8;
constexpr int kThreads = (4 + kSumWarps) * kWarp;
constexpr int kLineBytes = 128;           // of a token's outputs, staged by a warp at once
constexpr int kBox = kWarp * kLineBytes;  // 32 tokens' outputs: what a warp copies out at once
constexpr int kBoxes = 2;                 // of a warp, on their way out one behind the other
constexpr int kOut = kBoxes * kBox;
constexpr int kSmem = kStages * kStage + kSumWarps * kOut + 1024;  // + alignment slack
constexpr int kGroup = 8;                 // token tiles that share a sweep over the weights
// 128 x 56 + 256 x 224 are the 384 x 168 registers that the block has
constexpr int kRegs = 168, kFewRegs = 56, kSumRegs = 224;
static_assert(4 * kWarp * kFewRegs + kSumWarps * kWarp * kSumRegs <= kThreads * kRegs, "the split of the registers");
static_assert(kSmem <= 227 * 1024 - 512, "shared memory of one CTA, static beside it");
static_assert(kBufs == 2 && kStages >= 5, "a buffer for each of two warps, and what their waits rest on");

struct PairShape {
    const float *s[2], *xs;
    void* y;
    float* ys;
    int64_t M;
    int T, KB;
    int tilesM, tilesT;
    int blocksM;  // of 128 rows
    int y_type;
    int align;    // of y's rows: see row_align
    int boxes;    // outputs leave as boxes of map_y
};

// Tile i: kGroup token tiles under each tile of the weights, group after group.
__device__ __forceinline__ void find_tile(const PairShape& g, int i, int& mt, int& tt)
{
    const int per = kGroup * g.tilesM, group = i / per, in = i - group * per;
    const int wide = min(kGroup, g.tilesT - group * kGroup);
    mt = in / wide;
    tt = group * kGroup + in - mt * wide;
}

// A warp's 32 tokens x 128 bytes of outputs, a lane's token in v: staged, and copied out.
__device__ __forceinline__ void store_box(uint8_t* stage, const uint4 (&v)[8], const CUtensorMap* map, int64_t m, int tok, bool any)
{
    const int lane = threadIdx.x % kWarp;
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(stage + lane * kLineBytes + ((i ^ (lane & 7)) << 4)) = v[i];
    fence_async_smem();
    __syncwarp();
    if (lane == 0) {
        if (any) tma_store_2d(map, smem_u32(stage), static_cast<int>(m), tok);
        bulk_commit();
    }
}

template <bool DUAL>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_pairs_kernel(const __grid_constant__ CUtensorMap map_w0, const __grid_constant__ CUtensorMap map_w1,
                     const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_y,
                     const __grid_constant__ PairShape g)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[kStages], empty[kStages], dfull[kBufs], dempty[kBufs];
    __shared__ uint32_t s_tmem;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
    const int rank = static_cast<int>(cta_rank());
    const int tiles = g.tilesM * g.tilesT, step = static_cast<int>(gridDim.x) / 2, tile0 = static_cast<int>(blockIdx.x) / 2;
    const CUtensorMap* map_w = DUAL && rank ? &map_w1 : &map_w0;

    if (threadIdx.x == 0) {
        prefetch_map(map_w);
        prefetch_map(&map_x);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 4);  // the first CTA's counts, for both and for both operands
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(&dfull[i], 1);
            mbar_init(&dempty[i], 2 * kSumWarps);  // the first CTA's counts, for both
        }
        fence_barrier_init();
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = s_tmem;
    cluster_arrive();  // the pair's barriers and tensor memory are there
    cluster_wait();
    fp8_pdl_wait();

    bool ok = true;
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
        if (warp < 2) {
            // -------------------------------------------- copies: an operand a warp
            if (lane == 0) {
                int it = 0;
                for (int tile = tile0; tile < tiles && ok; tile += step) {
                    int mt, tt;
                    find_tile(g, tile, mt, tt);
                    const int row = DUAL ? mt * kHalf : mt * kTile + rank * kHalf, tok = tt * kTile + rank * kHalf;
                    for (int i = 0; i < g.KB; ++i, ++it) {
                        const int st = it % kStages;
                        if (it >= kStages) ok = mbar_wait(&empty[st], ((it / kStages) & 1) ^ 1, &g_fp8_pairs_error);
                        if (!ok) break;
                        const uint32_t at = smem_u32(ring + st * kStage), bar = cta_map(smem_u32(&full[st]), 0);
                        arrive_expect_cluster(bar, kHalfBytes);
                        if (warp == 0)
                            tma_2d_pair(at, &map_x, i * kBlk, tok, bar);
                        else
                            tma_2d_pair(at + kHalfBytes, map_w, i * kBlk, row, bar);
                    }
                }
                fp8_pdl_trigger();
                // the first CTA's products arrive here: none may be on its way when this CTA ends
                for (int u = warp ? it : max(it - kStages, 0); u < it && ok; ++u)
                    ok = mbar_wait(&empty[u % kStages], (u / kStages) & 1, &g_fp8_pairs_error);
            }
            __syncwarp();
        } else if (rank == 0) {
            // -------------------------------------------- products, of every other block
            constexpr uint32_t idesc = fp8_idesc(kTile, kTile);
            int it = 0;
            for (int tile = tile0; tile < tiles && ok; tile += step) {
                for (int i = 0; i < g.KB; ++i, ++it) {
                    if ((it & 1) != warp - 2) continue;
                    const int st = it % kStages, b = it % kBufs;
                    // (never two rounds behind: the block two before this one waited for the sums of two
                    // more before it, and so for the copies of all up to it - kStages)
                    ok = fp8_wait(&full[st], (it / kStages) & 1, &g_fp8_pairs_error);
                    if (ok && it >= kBufs) ok = fp8_wait(&dempty[b], ((it / kBufs) & 1) ^ 1, &g_fp8_pairs_error);
                    if (!ok) break;
                    tc_after();
                    if (fp8_elect()) {
                        const uint32_t at = smem_u32(ring + st * kStage);
#pragma unroll
                        for (int j = 0; j < kBlk / 32; ++j)
                            fp8_mma_pair(tmem + b * kTile, fp8_desc(at + 32 * j), fp8_desc(at + kHalfBytes + 32 * j), idesc,
                                         j != 0 ? 1u : 0u);
                        fp8_commit_pair(&empty[st]);
                        fp8_commit_pair(&dfull[b]);
                    }
                    __syncwarp();
                }
            }
        }
    } else {
        // ------------------------------------------------ sums: a token and 128 columns per thread
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
        const int q = warp % 4, half = (warp - 4) / 4;
        const uint32_t base = tmem + (static_cast<uint32_t>(32 * q) << 16);
        // its columns, 32 at a time: 128 of one weight block, or 64 each of the two weights
        const int col0 = DUAL ? 64 * half : kHalf * half, col2 = DUAL ? kHalf + 64 * half : kHalf * half + 64;
        uint8_t* stage = ring + kStages * kStage + (warp - 4) * kOut;
        const uint32_t free0 = cta_map(smem_u32(&dempty[0]), 0);
        int it = 0, turn = 0;
        for (int tile = tile0; tile < tiles; tile += step, turn ^= 1) {
            int mt, tt;
            find_tile(g, tile, mt, tt);
            const int t = tt * kTile + rank * kHalf + 32 * q + lane;
            const int mb = DUAL ? mt : min(2 * mt + half, g.blocksM - 1);
            const float* ws0 = g.s[0] + static_cast<int64_t>(mb) * g.KB;
            const float* ws1 = DUAL ? g.s[1] + static_cast<int64_t>(mb) * g.KB : nullptr;
            const float* xs = g.xs + t;
            uint64_t sum[64];
#pragma unroll
            for (int c = 0; c < 64; ++c) sum[c] = 0;
            // A block's scales are on their way while the one before it is added up. Nothing may be moved
            // that is on its way, and waits for tensor memory wait for these loads too, so they come from
            // the L1, where they were called one block before.
            const bool live = t < g.T;
            const int64_t pitch = g.T;
            float far_x = live ? __ldg(xs) : 0.f, far_w = __ldg(ws0), far_u = DUAL ? __ldg(ws1) : 0.f;
            for (int i = 0; i < g.KB; ++i, ++it) {
                const int b = it % kBufs;
                // looked at ahead of the scales: beside the tensor cores' reads of shared memory that takes
                // a hundred cycles
                const bool ready = mbar_try_wait(&dfull[b], (it / kBufs) & 1);
                const float f[2] = {far_x * far_w, DUAL ? far_x * far_u : far_x * far_w};
                if (i + 1 < g.KB) {
                    xs += pitch;
                    if (live) far_x = __ldg(xs);
                    far_w = __ldg(++ws0);
                    if constexpr (DUAL) far_u = __ldg(++ws1);
                }
                if (i + 2 < g.KB && live) asm volatile("prefetch.global.L1 [%0];" ::"l"(xs + pitch));
                // After a wait that ran out the loops go on without waiting, so that the warps
                // still meet at every barrier.
                if (!__all_sync(0xFFFFFFFFu, ready) && ok) ok = fp8_wait(&dfull[b], (it / kBufs) & 1, &g_fp8_pairs_error);
                __syncwarp();
                tc_after();
                // 64 columns at a time: the fewer loads wait for one another, the sooner is the buffer free
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t d[64];
                    tmem_load<32>(base + b * kTile + (h ? col2 : col0), d);
                    tmem_load<32>(base + b * kTile + (h ? col2 : col0) + 32, d + 32);
                    tmem_wait_ld();
                    if (h) {  // the buffer has been read
                        tc_before();
                        __syncwarp();
                        if (lane == 0) arrive_cluster(free0 + b * 8);
                    }
                    const uint64_t ff = pack(f[h], f[h]);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        sum[32 * h + e] = fma2(pack(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1])), ff, sum[32 * h + e]);
                }
            }
            // ---- the tile's outputs
            float acc[128];
#pragma unroll
            for (int c = 0; c < 64; ++c) unpack(sum[c], acc[2 * c], acc[2 * c + 1]);
            const int tok0 = tt * kTile + rank * kHalf + 32 * q, tokens = g.T - tok0;
            const int64_t m0 = DUAL ? static_cast<int64_t>(mt) * kHalf + 64 * half : static_cast<int64_t>(mt) * kTile + kHalf * half;
            constexpr int N = DUAL ? 64 : 128;  // outputs of a thread
            if constexpr (DUAL) {
#pragma unroll
                for (int c = 0; c < 64; ++c) acc[c] = silu_mul(acc[c], acc[64 + c]);
            }
            const int64_t left = g.M - m0;  // elements of the row from this thread's first
            if (DUAL && g.y_type == BQD_E4M3) {
                float most = 0.f;
#pragma unroll
                for (int c = 0; c < N; c += 2) most = max_abs(most, c < left ? acc[c] : 0.f, c + 1 < left ? acc[c + 1] : 0.f);
                // with the warp that has the other half of these tokens: past the codes' lines in its
                // staging, at another place for the next tile
                const int seen = kOut / 2 + turn * (4 * kWarp) + 4 * lane;
                *reinterpret_cast<float*>(stage + seen) = most;
                __syncwarp();
                named_sync(1 + q, 2 * kWarp);
                const float sc = block_scale(max_abs(most, *reinterpret_cast<const float*>(stage + (half ? -4 : 4) * kOut + seen)));
                if (half == 0 && t < g.T) g.ys[static_cast<int64_t>(mt) * g.T + t] = sc;
                uint4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint64_t w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = pack(acc[16 * i + 2 * e], acc[16 * i + 2 * e + 1]);
                    const uint32_t x = scale_down(w, sc);
                    v[i] = make_uint4(e4m3x4(w[0], w[1], x), e4m3x4(w[2], w[3], x), e4m3x4(w[4], w[5], x), e4m3x4(w[6], w[7], x));
                }
                store_lines<64>(stage, v, static_cast<uint8_t*>(g.y) + static_cast<int64_t>(tok0) * g.M + m0, g.M, left, tokens,
                                g.align);
            } else if (g.y_type == BQD_BF16) {
#pragma unroll
                for (int k = 0; k < N / 64; ++k) {
                    uint4 v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[e] = to_bf16x2(acc[64 * k + 8 * i + 2 * e], acc[64 * k + 8 * i + 2 * e + 1]);
                        v[i] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    if (g.boxes) {
                        // the places follow one another over the tiles too: of a gated pair a tile has one box
                        const int place = N == 64 ? turn : k % kBoxes;
                        static_assert(kBoxes == 2, "turn counts tiles by two");
                        if (lane == 0) bulk_wait_read<kBoxes - 1>();  // its place has been left
                        __syncwarp();
                        store_box(stage + place * kBox, v, &map_y, m0 + 64 * k, tok0, left > 64 * k && tokens > 0);
                    } else {
                        store_lines<128>(stage, v, static_cast<uint8_t*>(g.y) + 2 * (static_cast<int64_t>(tok0) * g.M + m0 + 64 * k),
                                         2 * g.M, 2 * (left - 64 * k), tokens, g.align);
                    }
                }
            } else {
#pragma unroll
                for (int k = 0; k < N / 32; ++k) {
                    uint4 v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        v[i] = make_uint4(__float_as_uint(acc[32 * k + 4 * i]), __float_as_uint(acc[32 * k + 4 * i + 1]),
                                          __float_as_uint(acc[32 * k + 4 * i + 2]), __float_as_uint(acc[32 * k + 4 * i + 3]));
                    if (g.boxes) {
                        if (lane == 0) bulk_wait_read<kBoxes - 1>();  // its place has been left
                        __syncwarp();
                        store_box(stage + k % kBoxes * kBox, v, &map_y, m0 + 32 * k, tok0, left > 32 * k && tokens > 0);
                    } else {
                        store_lines<128>(stage, v, static_cast<uint8_t*>(g.y) + 4 * (static_cast<int64_t>(tok0) * g.M + m0 + 32 * k),
                                         4 * g.M, 4 * (left - 32 * k), tokens, g.align);
                    }
                }
            }
        }
        if (lane == 0) bulk_wait_all();
        tc_before();
    }
    if (!ok) let_copies_land();
    __syncwarp();
    cluster_arrive();  // the pair's products and arrivals are over
    cluster_wait();
    if (warp == 2) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

template <bool DUAL>
cudaError_t launch(const Fp8GemmArgs& a, cudaStream_t s)
{
    CUtensorMap w0, w1, x, y;
    if (!fp8_codes_map(&w0, a.w0, a.M, a.K, kHalf) || !fp8_codes_map(&x, a.x, a.T, a.K, kHalf)) return cudaErrorInvalidValue;
    if (!DUAL)
        w1 = w0;
    else if (!fp8_codes_map(&w1, a.w1, a.M, a.K, kHalf))
        return cudaErrorInvalidValue;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    auto kern = fp8_pairs_kernel<DUAL>;
    static OccCache occ;
    blocks_per_sm(occ, reinterpret_cast<const void*>(kern), dev, kThreads, kSmem);
    // the split of the registers needs what the block is launched with
    if (launch_regs(occ, reinterpret_cast<const void*>(kern), dev) < kRegs) return cudaErrorInvalidConfiguration;
    PairShape g{};
    g.s[0] = a.s0;
    g.s[1] = a.s1;
    g.xs = a.xs;
    g.y = a.y;
    g.ys = a.ys;
    g.M = a.M;
    g.T = static_cast<int>(a.T);
    g.KB = static_cast<int>((a.K + kBlk - 1) / kBlk);
    g.tilesM = static_cast<int>((a.M + (DUAL ? kHalf : kTile) - 1) / (DUAL ? kHalf : kTile));
    g.tilesT = static_cast<int>((a.T + kTile - 1) / kTile);
    g.blocksM = static_cast<int>((a.M + 127) / 128);
    g.y_type = a.y_type;
    g.align = row_align(a.M, a.y_type);
    // rows of whole 16 bytes leave as boxes of 128 bytes by 32 tokens
    g.boxes = a.y_type != BQD_E4M3 && g.align == 16;
    if (!g.boxes)
        y = x;
    else if (!fp8_rows_map(&y, a.y, a.y_type, a.T, a.M, kWarp, kLineBytes))
        return cudaErrorInvalidValue;
    const int64_t tiles = static_cast<int64_t>(g.tilesM) * g.tilesT, pairs = dev_info(dev).sms / 2;
    return launch_clusters(kern, static_cast<unsigned>(2 * (tiles < pairs ? tiles : pairs)), 2, kThreads, kSmem, s, w0, w1, x, y, g);
}

}  // namespace

// Up to 64 tokens the weights' one read is the bound, and fp8_gemm.cu takes tokens
// by 16. Beyond that a block of k takes a CTA of fp8_gemm_tokens.cu 0.35 us and a
// pair here, with four times the products, 0.45 us: the kernel that goes through
// fewer blocks one after the other is the sooner done. Measured, us there and here:
// 12288 x 4096 by 256 tokens (64 blocks there, 32 here) 31 and 21, 4096 x 4096 by 256
// (16, 32) 16 and 18, 4096 x 12288 by 512 (96, 96) 40 and 43, 4870 x 4096 by 1000
// (96, 64) 41 and 36; gated 6144 x 4096 by 100 (32, 32) 22 and 21.
bool fp8_gemm_wants_pairs(const Fp8GemmArgs& a, bool dual)
{
    if (a.T <= 64) return false;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const int64_t sms = dev_info(dev).sms > 1 ? dev_info(dev).sms : 2, KB = (a.K + kBlk - 1) / kBlk;
    const int64_t alone = (a.M + 127) / 128 * ((a.T + 127) / 128) * (dual ? 2 : 1);
    const int64_t share = alone < sms ? sms / alone : 1;  // CTAs that share a tile's k
    const int64_t rows = dual ? kHalf : kTile, tiles = (a.M + rows - 1) / rows * ((a.T + kTile - 1) / kTile);
    const int64_t there = (alone * share + sms - 1) / sms * ((KB + share - 1) / share);
    const int64_t here = (tiles + sms / 2 - 1) / (sms / 2) * KB;
    return dual ? here <= there : here < there;
}

cudaError_t launch_fp8_gemm_pairs(const Fp8GemmArgs& a, bool dual, cudaStream_t s)
{
    return dual ? launch<true>(a, s) : launch<false>(a, s);
}

cudaError_t read_and_clear_fp8_pairs_error(unsigned int* out)
{
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_fp8_pairs_error, sizeof(v));
    if (e != cudaSuccess) return e;
    *out = v;
    if (v) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_fp8_pairs_error, &zero, sizeof(zero));
    }
    return e;
}

}  // namespace bqd
