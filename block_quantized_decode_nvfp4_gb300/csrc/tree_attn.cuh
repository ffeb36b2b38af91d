// tree_attn.cuh -- what the kernels of tree_attention share: the requests'
// lengths, the even split of ragged work over the CTAs, what a token sees,
// and the join of an item's parts.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn.h"
#include "common.cuh"

namespace bqd {

constexpr int kAttnMaxGrid = 3 * 152;
constexpr float kAttnLog2e = 1.4426950408889634f, kAttnLn2 = 0.6931471805599453f;
constexpr float kAttnPShift = 12.f;  // E4M3: log2 of the scale p carries

struct AttnMeta {  // of a CTA's unfinished last item: whose it is and the last CTA with a part of it
    int32_t r, h, tile, last;  // r = -1: none
};

__host__ __device__ constexpr size_t attn_meta_bytes() { return (kAttnMaxGrid * sizeof(AttnMeta) + 255) / 256 * 256; }
// A part: o [rows][D], m [rows], z [rows].
__host__ __device__ constexpr size_t attn_part_floats(int rows, int D) { return static_cast<size_t>(rows) * (D + 2); }

struct AttnReq {
    int o0, n;    // first token, new tokens
    int64_t ctx;  // cached tokens
    int64_t len;  // tokens to look at
    int tiles;    // of `rows` rows
    int64_t nb;   // units per item: `over` for its beginning and end, then one per `unit` tokens
};

__device__ __forceinline__ AttnReq attn_request(const AttnArgs& a, int64_t r, int rows, int unit, int over)
{
    AttnReq q;
    const int T = static_cast<int>(a.T);
    q.o0 = min(max(a.offsets[r], 0), T);
    q.n = min(max(a.offsets[r + 1], q.o0), T) - q.o0;
    q.ctx = max(a.context[r], 0);
    q.len = min(q.ctx + q.n, a.width * a.cache.page_size);
    q.tiles = static_cast<int>((static_cast<int64_t>(q.n) * a.group + rows - 1) / rows);
    q.nb = over + max(int64_t(1), (q.len + unit - 1) / unit);
    return q;
}

__device__ __forceinline__ int64_t attn_units(const AttnArgs& a, int64_t r, int rows, int unit, int over)
{
    const AttnReq q = attn_request(a, r, rows, unit, over);
    return q.nb * q.tiles * a.cache.heads;
}

// A CTA's share [start, end) of the line of all items' units, the request
// that holds its first unit and the units before that request.
struct AttnShare {
    int64_t start, end, total, ctas;  // ctas: those with a share, a unit at least
    int64_t r, base;
};

// Each thread sums a run of requests, one scan places them. sh: THREADS / 32
// + 2 entries of shared memory; called by the whole CTA.
template <int THREADS>
__device__ __forceinline__ AttnShare attn_find_share(const AttnArgs& a, int rows, int unit, int over, int64_t* sh)
{
    constexpr int W = THREADS / kWarp;
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    const int64_t per = (a.R + THREADS - 1) / THREADS;
    const int64_t r0 = min(threadIdx.x * per, a.R), r1 = min(r0 + per, a.R);
    int64_t mine = 0;
    for (int64_t i = r0; i < r1; ++i) mine += attn_units(a, i, rows, unit, over);
    int64_t incl = mine;
#pragma unroll
    for (int d = 1; d < kWarp; d <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += v;
    }
    if (lane == kWarp - 1) sh[warp] = incl;
    __syncthreads();
    AttnShare s{};
    int64_t before = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        if (w < warp) before += sh[w];
        s.total += sh[w];
    }
    s.ctas = min(static_cast<int64_t>(gridDim.x), s.total);
    if (blockIdx.x >= s.ctas) {
        s.start = s.end = s.total;
    } else if (s.total < (int64_t(1) << 22)) {  // 32-bit divisions (grids are below 2^10)
        s.start = static_cast<uint32_t>(s.total) * blockIdx.x / static_cast<uint32_t>(s.ctas);
        s.end = static_cast<uint32_t>(s.total) * (blockIdx.x + 1) / static_cast<uint32_t>(s.ctas);
    } else {
        s.start = s.total * blockIdx.x / s.ctas;
        s.end = s.total * (blockIdx.x + 1) / s.ctas;
    }
    const int64_t first = before + incl - mine;
    if (s.start < s.end && s.start >= first && s.start < first + mine) {
        int64_t b = first, i = r0;
        for (;; ++i) {
            const int64_t u = attn_units(a, i, rows, unit, over);
            if (s.start < b + u) break;
            b += u;
        }
        sh[W] = i;
        sh[W + 1] = b;
    }
    __syncthreads();
    s.r = sh[W];
    s.base = sh[W + 1];
    return s;
}

// Unit u of the line: item (kv head, tile) of request s.r and the unit in it.
__device__ __forceinline__ void attn_place(const AttnShare& s, const AttnReq& q, int64_t u, int& h, int& tile,
                                           int64_t& b0)
{
    const int64_t at = u - s.base;
    if (at < (int64_t(1) << 32) && q.nb < (int64_t(1) << 32)) {
        const uint32_t nb = static_cast<uint32_t>(q.nb), item = static_cast<uint32_t>(at) / nb;
        b0 = static_cast<uint32_t>(at) - item * nb;
        h = static_cast<int>(item / static_cast<uint32_t>(q.tiles));
        tile = static_cast<int>(item) - h * q.tiles;
    } else {
        const int64_t item = at / q.nb;
        b0 = at % q.nb;
        h = static_cast<int>(item / q.tiles);
        tile = static_cast<int>(item % q.tiles);
    }
}

// The meta entry of a CTA whose item (units up to `ends` of the line) goes on
// in other CTAs: the last CTA whose share begins before the item's end.
__device__ __forceinline__ AttnMeta attn_meta(const AttnShare& s, int h, int tile, int64_t ends)
{
    return {static_cast<int32_t>(s.r), h, tile, static_cast<int32_t>((ends * s.ctas + s.total - 1) / s.total - 1)};
}

// Whether query token i of the request (token t of the call) sees draft j
// (j < 0: a cached token).
__device__ __forceinline__ bool attn_sees(const AttnArgs& a, int64_t t, int i, int64_t j)
{
    if (j < 0) return true;
    if (!a.mask) return j <= i;
    return (j >> 6) < a.mask_words && ((a.mask[t * a.mask_words + (j >> 6)] >> (j & 63)) & 1);
}

__device__ __forceinline__ float attn_ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t attn_bf16x2(float lo, float hi)
{
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// Four elements of a finished row: o / z, zero where nothing was seen.
__device__ __forceinline__ uint2 attn_out4(float4 v, float z, float vscale)
{
    const float k = z == 0.f ? 0.f : vscale / z;
    if (z == 0.f) v = make_float4(0.f, 0.f, 0.f, 0.f);
    return make_uint2(attn_bf16x2(v.x * k, v.y * k), attn_bf16x2(v.z * k, v.w * k));
}
__device__ __forceinline__ float attn_lse(float m, float z, float shift)
{
    return z == 0.f ? -INFINITY : (m + log2f(z) - shift) * kAttnLn2;
}

// Weight of a part with maximum mw in a join with maximum m.
__device__ __forceinline__ float attn_weight(float mw, float m)
{
    return mw == -INFINITY ? (m == -INFINITY ? 1.f : 0.f) : attn_ex2(mw - m);
}

// Joins the parts of the item that CTA blockIdx.x of the first kernel began
// and did not finish: its own second part, then the first parts of the CTAs
// after it, in order. blockIdx.y: four rows each, D / 4 threads a row. Parts
// are row by row.
template <int D, int ROWS, bool F8>
__global__ void __launch_bounds__(D) tree_attn_join_kernel(AttnArgs a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const AttnMeta md = static_cast<const AttnMeta*>(a.ws)[blockIdx.x];
    if (md.r < 0) return;
    const float* parts = reinterpret_cast<const float*>(static_cast<const uint8_t*>(a.ws) + attn_meta_bytes());
    const int row = blockIdx.y * 4 + threadIdx.x / (D / 4), d = threadIdx.x % (D / 4) * 4;
    const AttnReq q = attn_request(a, md.r, ROWS, 1, 0);
    const int G = a.group;
    const int64_t grow = static_cast<int64_t>(md.tile) * ROWS + row;
    if (grow >= static_cast<int64_t>(q.n) * G) return;
    constexpr size_t P = attn_part_floats(ROWS, D);
    const int b = blockIdx.x;
    auto part = [&](int k) { return parts + (k == b ? 2 * k + 1 : 2 * k) * P; };
    float m = -INFINITY;
    for (int k = b; k <= md.last; ++k) m = fmaxf(m, part(k)[ROWS * D + row]);
    float z = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = b; k <= md.last; ++k) {
        const float* p = part(k);
        const float f = attn_weight(p[ROWS * D + row], m);
        const float4 y = *reinterpret_cast<const float4*>(p + row * D + d);
        z += p[ROWS * D + ROWS + row] * f;
        v.x += y.x * f;
        v.y += y.y * f;
        v.z += y.z * f;
        v.w += y.w * f;
    }
    const int64_t at = (q.o0 + grow / G) * static_cast<int64_t>(a.Hq) + md.h * G + grow % G;
    const float vscale = (F8 && a.cache.v_scale) ? a.cache.v_scale[md.h] : 1.f;
    *reinterpret_cast<uint2*>(a.out + at * D + d) = attn_out4(v, z, vscale);
    if (d == 0 && a.lse) a.lse[at] = attn_lse(m, z, F8 ? kAttnPShift : 0.f);
}

// The same for parts that lie column by column (o [D][rows]): blockIdx.y is
// eight rows, a thread one of their D columns.
template <int D, int ROWS>
__global__ void __launch_bounds__(D) tree_attn_join_columns_kernel(AttnArgs a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const AttnMeta md = static_cast<const AttnMeta*>(a.ws)[blockIdx.x];
    if (md.r < 0) return;
    const float* parts = reinterpret_cast<const float*>(static_cast<const uint8_t*>(a.ws) + attn_meta_bytes());
    const int row0 = blockIdx.y * 8, d = threadIdx.x, b = blockIdx.x;
    const AttnReq q = attn_request(a, md.r, ROWS, 1, 0);
    const int64_t grow0 = static_cast<int64_t>(md.tile) * ROWS + row0;
    const int live = static_cast<int>(min(static_cast<int64_t>(q.n) * a.group - grow0, int64_t(8)));
    if (live <= 0) return;
    constexpr size_t P = attn_part_floats(ROWS, D);
    auto part = [&](int k) { return parts + (k == b ? 2 * k + 1 : 2 * k) * P; };
    float m[8], z[8], v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        m[i] = -INFINITY;
        z[i] = v[i] = 0.f;
    }
    for (int k = b; k <= md.last; ++k) {
        const float* p = part(k) + ROWS * D + row0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < live) m[i] = fmaxf(m[i], p[i]);
    }
#pragma unroll 2
    for (int k = b; k <= md.last; ++k) {
        const float* p = part(k);
        const float4 lo = *reinterpret_cast<const float4*>(p + d * ROWS + row0);
        const float4 hi = *reinterpret_cast<const float4*>(p + d * ROWS + row0 + 4);
        const float y[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < live) {
                const float f = attn_weight(p[ROWS * D + row0 + i], m[i]);
                z[i] += p[ROWS * D + ROWS + row0 + i] * f;
                v[i] += y[i] * f;
            }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < live) {
            const uint32_t g = static_cast<uint32_t>(grow0 + i), tok = g / a.group;
            const int64_t at = (q.o0 + static_cast<int64_t>(tok)) * a.Hq + md.h * a.group + (g - tok * a.group);
            a.out[at * D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(z[i] == 0.f ? 0.f : v[i] / z[i]));
            if (d == 0 && a.lse) a.lse[at] = attn_lse(m[i], z[i], 0.f);
        }
}

// Launches a join after the first kernel in the same stream; it may be set up
// while that one still runs, and waits for its end.
inline cudaError_t launch_attn_join(void (*kernel)(AttnArgs), dim3 grid, int threads, const AttnArgs& a, cudaStream_t s)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// The kernel for many rows a kv head (tree_attn_wide.cu), bf16 caches.
bool tree_attention_wide_fits(const AttnArgs& a);
size_t tree_attention_wide_ws(int64_t R, int64_t T, int Hq, int Hkv, int D);
cudaError_t launch_tree_attention_wide(const AttnArgs& a, cudaStream_t s);

}  // namespace bqd
