// fp8_gemm.cuh -- what the products with 8-bit activations share: a call's
// sizes, the gate, the end of a tile that a cluster of CTAs has computed, and
// stores of rows that start anywhere.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>
#include <mutex>

#include "bqd.h"
#include "common.cuh"
#include "fp8.cuh"
#include "fp8.h"
#include "host_util.h"

namespace bqd {

namespace fp8 {

constexpr int kRows = 128;            // weight rows of a tile of scales
constexpr int kBlk = 128;             // k of a block of scales and of a ring stage
constexpr int kTileBytes = kRows * kBlk;
constexpr int kMaxCluster = 8;

struct GemmShape {
    const uint8_t* w[2];
    const float *s[2], *xs;
    void* y;
    float* ys;
    int64_t M, K;
    int T, KB;           // tokens, blocks of k
    int tilesM, tilesT;  // tile = row tile * tilesT + token tile
    int mats;            // 2: a gated pair
    int y_type;
    int align;           // of y's rows: see row_align
    int whole;           // y's rows are so aligned that four elements of one may be stored at once
    int early;           // weights may be read before the previous kernel has completed
};

// A row's first blocks called into the L2, by a thread that waits for the previous kernel:
// the memory has less to do at a kernel's end. More than two of them, or by the copy engine
// (6 blocks: 0.6 us later for small calls), hold up a call that need not wait. The L2 keeps
// what that kernel may still write.
__device__ __forceinline__ void call_weights(const GemmShape& g, int mat, int64_t row, int kb, int blocks)
{
    constexpr int kMost = 2;
    if (g.early || row >= g.M) return;
    const uint8_t* at = g.w[mat] + row * g.K + static_cast<int64_t>(kb) * kBlk;
    for (int i = 0; i < kMost; ++i)
        if (i < blocks) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + i * kBlk) : "memory");
}

// SiLU(g) u = g / (1 + e^-g) u, with e = e^-|g|: 1 / (1 + e) for g from 0 on, e / (1 + e) below, so that the divisor
// stays between 1 and 2. By 1 + e^-g the fast division would give 0 from g = -87.3 on, where it passes 2^126, and an
// infinity from -88.7 on, while the product with a large u is still a normal number.
__device__ __forceinline__ float silu_mul(float g, float u)
{
    const float e = expf(-fabsf(g));
    return __fdividef(g >= 0.f ? g : g * e, 1.f + e) * u;
}

__device__ __forceinline__ void store_y(void* y, int type, int64_t at, float v)
{
    if (type == BQD_F32)
        static_cast<float*>(y)[at] = v;
    else
        static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
}

// Four consecutive elements of a row of y, the first `live` of which there are.
__device__ __forceinline__ void store_codes4(uint8_t* p, uint32_t codes, int live, bool whole)
{
    if (whole && live == 4) {
        *reinterpret_cast<uint32_t*>(p) = codes;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < live) p[e] = static_cast<uint8_t>(codes >> (8 * e));
    }
}
__device__ __forceinline__ void store_rows4(void* y, int type, int64_t at, const float (&v)[4], int live, bool whole)
{
    if (whole && live == 4) {
        if (type == BQD_F32)
            *reinterpret_cast<float4*>(static_cast<float*>(y) + at) = make_float4(v[0], v[1], v[2], v[3]);
        else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + at) = make_uint2(to_bf16x2(v[0], v[1]), to_bf16x2(v[2], v[3]));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < live) store_y(y, type, at + e, v[e]);
    }
}

// A warp's 32 tokens x BYTES of outputs, as lane l has token l's in v, to rows of
// y: through shared memory, so that a store has whole lines. at: bytes from y to
// token 0's; pitch: bytes of a row; left: bytes of the row from `at`; tokens: how
// many there are.
template <int BYTES>
__device__ __forceinline__ void store_lines(uint8_t* stage, const uint4 (&v)[BYTES / 16], uint8_t* at, int64_t pitch,
                                            int64_t left, int tokens, int align)
{
    constexpr int C = BYTES / 16;  // 16-byte pieces of a line
    const int lane = threadIdx.x % kWarp;
    __syncwarp();  // what was staged before has been read
#pragma unroll
    for (int i = 0; i < C; ++i) *reinterpret_cast<uint4*>(stage + lane * BYTES + ((i ^ (lane & (C - 1))) << 4)) = v[i];
    __syncwarp();
    if (align == 16) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int t = i * (kWarp / C) + lane / C, c = lane & (C - 1);
            const uint4 w = *reinterpret_cast<const uint4*>(stage + t * BYTES + ((c ^ (t & (C - 1))) << 4));
            if (t < tokens && 16 * c < left) *reinterpret_cast<uint4*>(at + t * pitch + 16 * c) = w;
        }
        return;
    }
    // rows that start anywhere: words, halves or bytes, neighbours by neighbouring lanes
    constexpr int W = BYTES / 4;  // words of a line
    const int c = lane & (W - 1);
    const int64_t n = left - 4 * c;  // bytes of the row from this lane's
#pragma unroll 4
    for (int i = 0; i < W; ++i) {
        const int t = i * (kWarp / W) + lane / W;
        const uint32_t w = *reinterpret_cast<const uint32_t*>(stage + t * BYTES + (((c / 4) ^ (t & (C - 1))) << 4) + c % 4 * 4);
        if (t >= tokens) continue;
        uint8_t* p = at + t * pitch + 4 * c;
        if (align >= 4) {
            if (n > 0) *reinterpret_cast<uint32_t*>(p) = w;
        } else if (align == 2) {
            if (n > 0) *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w);
            if (n > 2) *reinterpret_cast<uint16_t*>(p + 2) = static_cast<uint16_t>(w >> 16);
        } else {
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (n > b) p[b] = static_cast<uint8_t>(w >> (8 * b));
        }
    }
}

// The end of a tile of one row block whose CTAs (`ranks`, of g.mats weights) have
// left their parts here: parts [part][token][128 rows] fp32, `most` tokens a part,
// n of them this CTA's (token j is t0 + j t_step). A token per warp at a time, four
// rows a lane; the parts are added up in the order of the k blocks. SWIZZLED: 16
// bytes i of token j lie at i ^ (key + j) % 32.
template <bool SWIZZLED>
__device__ __forceinline__ void finish_tokens(const GemmShape& g, const float* parts, int most, int n, int ranks, int mt,
                                              int64_t t0, int t_step, int key, int first, int step)
{
    const int lane = threadIdx.x % kWarp;
    const int64_t row = static_cast<int64_t>(mt) * kRows + 4 * lane;
    const int live = static_cast<int>(min(static_cast<int64_t>(4), max(static_cast<int64_t>(0), g.M - row)));
    for (int j = first; j < n; j += step) {
        const float4* part = reinterpret_cast<const float4*>(parts + j * kRows) + (SWIZZLED ? lane ^ ((key + j) & 31) : lane);
        const int next = most * (kRows / 4);  // to the next part
        float v[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
        for (int k = 0; k < ranks; k += g.mats) {
            const float4 p = part[k * next];
            v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w;
            if (g.mats > 1) {
                const float4 w = part[(k + 1) * next];
                u[0] += w.x, u[1] += w.y, u[2] += w.z, u[3] += w.w;
            }
        }
        if (g.mats > 1) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = silu_mul(v[e], u[e]);
        }
        const int64_t t = t0 + static_cast<int64_t>(j) * t_step;
        if (g.y_type == BQD_E4M3) {
            float m = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) m = max_abs(m, e < live ? v[e] : 0.f);
            // (non-negative floats order as integers, NaN above all)
            const float sc = block_scale(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m))));
            uint64_t w[2] = {pack(v[0], v[1]), pack(v[2], v[3])};
            const uint32_t x = scale_down(w, sc);
            store_codes4(static_cast<uint8_t*>(g.y) + t * g.M + row, e4m3x4(w[0], w[1], x), live, g.whole);
            if (lane == 0) g.ys[static_cast<int64_t>(mt) * g.T + t] = sc;
        } else {
            store_rows4(g.y, g.y_type, t * g.M + row, v, live, g.whole);
        }
    }
}

// Clusters of `ranks` CTAs that run at once on the device: fewer than its slots
// hold, as a cluster stays within a group of SMs. The query counts a CTA per SM;
// `ctas` fit on one. Cached; 0 if it cannot be told.
struct ClusterCache {
    std::mutex mu;
    int known[64][kMaxCluster + 1] = {};
};
inline int clusters_at_once(ClusterCache& c, const void* kern, int dev, int threads, size_t smem, int ctas, int ranks)
{
    std::lock_guard<std::mutex> lock(c.mu);
    if (dev < 0 || dev >= 64) return 0;
    int& n = c.known[dev][ranks];
    if (n == 0) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
            cudaSuccess)
            cudaGetLastError();
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(ranks * ctas * dev_info(dev).sms));
        cfg.blockDim = dim3(static_cast<unsigned>(threads));
        cfg.dynamicSmemBytes = smem;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int found = 0;
        if (cudaOccupancyMaxActiveClusters(&found, kern, &cfg) != cudaSuccess) {
            cudaGetLastError();  // consumed: it must not surface as a launch error later
            return 0;
        }
        n = found > 0 ? found : -1;
    }
    return n > 0 ? n * ctas : 0;
}

// CTAs that share the k blocks of a tile: as many as may be with every cluster
// running at once.
inline int share_k(ClusterCache& c, const void* kern, int dev, int threads, size_t smem, int ctas, int64_t tiles, int mats, int KB)
{
    const int64_t slots = static_cast<int64_t>(dev_info(dev).sms) * ctas;
    int cs = kMaxCluster / mats < KB ? kMaxCluster / mats : KB;
    while (cs > 1 && (tiles * cs * mats > slots || tiles > clusters_at_once(c, kern, dev, threads, smem, ctas, cs * mats))) --cs;
    return cs;
}

// A launch in clusters that may begin while the kernel before it ends: the kernel
// itself waits for that one.
template <typename... A>
cudaError_t launch_clusters(void (*kern)(A...), unsigned grid, int ranks, int threads, size_t smem, cudaStream_t s, const A&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ranks);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ranks > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// The bytes to which every row of y [T][M] is aligned: 16, 4, or an element's.
inline int row_align(int64_t M, int y_type)
{
    const int64_t size = y_type == BQD_F32 ? 4 : y_type == BQD_BF16 ? 2 : 1, pitch = M * size;
    return static_cast<int>(pitch % 16 == 0 ? 16 : pitch % 4 == 0 ? 4 : size);
}

}  // namespace fp8

}  // namespace bqd
