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

// Of a CTA's unfinished last item: the last CTA with a part of it, its first
// row's token and head (of all query heads), live rows (0: there is none such).
struct alignas(16) AttnMeta {
    int32_t last, rows, o0, row0, h0;  // row0: of the request, in rows of the group; h0: the group's first head
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

__device__ __forceinline__ void attn_cut(AttnShare& s)  // the share from the total
{
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
}

// Up to 32 requests: every warp for itself, a request per lane. More: each
// thread sums a run of requests, one scan places them. sh: THREADS / 32 + 2
// entries of shared memory; called by the whole CTA.
template <int THREADS>
__device__ __forceinline__ AttnShare attn_find_share(const AttnArgs& a, int rows, int unit, int over, int64_t* sh)
{
    constexpr int W = THREADS / kWarp;
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    AttnShare s{};
    if (a.R <= kWarp) {
        const int64_t mine = lane < a.R ? attn_units(a, lane, rows, unit, over) : 0;
        int64_t incl = mine;
#pragma unroll
        for (int d = 1; d < kWarp; d <<= 1) {
            const int64_t v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
            if (lane >= d) incl += v;
        }
        s.total = __shfl_sync(0xFFFFFFFFu, incl, kWarp - 1);
        attn_cut(s);
        const uint32_t past = __ballot_sync(0xFFFFFFFFu, incl > s.start);
        const int at = past ? __ffs(past) - 1 : 0;  // none: the CTA has no share
        s.r = at;
        s.base = __shfl_sync(0xFFFFFFFFu, incl - mine, at);
        __syncthreads();  // as the other way does: what the CTA has set up is visible
        return s;
    }
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
    int64_t before = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        if (w < warp) before += sh[w];
        s.total += sh[w];
    }
    attn_cut(s);
    const int64_t first = before + incl - mine;
    if (s.start < s.end && s.start >= first && s.start < first + mine) {
        int64_t b = first, i = r0;
        for (; i + 1 < r1; ++i) {
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
__device__ __forceinline__ AttnMeta attn_meta(const AttnArgs& a, const AttnShare& s, const AttnReq& q, int h, int tile,
                                              int rows, int64_t ends)
{
    const int64_t left = static_cast<int64_t>(q.n) * a.group - static_cast<int64_t>(tile) * rows;
    return {static_cast<int32_t>((ends * s.ctas + s.total - 1) / s.total - 1),
            static_cast<int32_t>(left < rows ? left : rows), q.o0, tile * rows, h * a.group};
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

constexpr int kJoinThreads = 256;
constexpr int kJoinGrid = 6 * 152;
constexpr int kAttnDeep = 8;  // CTAs an item reaches on for: from here its parts are shared by more threads

// The items that the first kernel's CTAs left unfinished, as a list in shared
// memory (list: kAttnMaxGrid entries, counts: two per warp); returns their
// number, and whether one is deep. Every block of a
// join makes it for itself: one read of the metas, and no idle blocks.
__device__ __forceinline__ int attn_unfinished(const AttnArgs& a, int grid, int16_t* list, int* counts, bool& deep)
{
    const AttnMeta* meta = static_cast<const AttnMeta*>(a.ws);
    constexpr int kPer = (kAttnMaxGrid + kJoinThreads - 1) / kJoinThreads;
    const int lane = threadIdx.x % kWarp;
    static_assert(kPer <= 2, "counts");
    bool open[kPer], far = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int b = i * kJoinThreads + threadIdx.x;
        const int2 x = b < grid ? *reinterpret_cast<const int2*>(&meta[b]) : make_int2(0, 0);  // last, rows
        open[i] = x.y > 0;
        far |= open[i] && x.x - b >= kAttnDeep;
    }
    deep = __syncthreads_or(far);
    // the same order in every block: by CTA, a warp's ballot at a time
    constexpr int kWarps = kJoinThreads / kWarp;
    uint32_t m[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        m[i] = __ballot_sync(0xFFFFFFFFu, open[i]);
        if (lane == 0) counts[i * kWarps + threadIdx.x / kWarp] = __popc(m[i]);
    }
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int x = 0; x < kPer * kWarps; ++x) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (open[i] && x == i * kWarps + static_cast<int>(threadIdx.x / kWarp))
                list[total + __popc(m[i] & ((1u << lane) - 1))] = static_cast<int16_t>(i * kJoinThreads + threadIdx.x);
        total += counts[x];
    }
    __syncthreads();
    return total;
}

// (m, z, o) of N values with another such of maximum m2.
template <int N>
__device__ __forceinline__ void attn_join(float& m, float& z, float (&o)[N], float m2, float z2, const float (&o2)[N])
{
    const float mm = fmaxf(m, m2), f = attn_weight(m, mm), f2 = attn_weight(m2, mm);
    z = z * f + z2 * f2;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = o[i] * f + o2[i] * f2;
    m = mm;
}

// Joins the parts of every item that a CTA b of the first kernel began and did
// not finish: b's own second part, then the first parts of the CTAs after it,
// in order. Parts are row by row. D / 4 threads a row. Few parts: a row's
// threads take them all, four loads in flight. Many (a long context's item is
// shared by dozens of CTAs): they go round among GROUPS such sets of threads,
// whose results join in order (8 for D = 128: 57 parts in two rounds of loads).
template <int D, int ROWS, bool F8, int GROUPS>
__device__ __forceinline__ void attn_join_rows(const AttnArgs& a, const AttnMeta& md, int b, int row,
                                               float (*s_part)[6])
{
    constexpr int TPR = D / 4;
    constexpr size_t P = attn_part_floats(ROWS, D);
    const float* parts = reinterpret_cast<const float*>(static_cast<const uint8_t*>(a.ws) + attn_meta_bytes());
    const int d = threadIdx.x % TPR * 4, group = threadIdx.x / TPR % GROUPS;
    float m = -INFINITY, z = 0.f, o[4] = {};
    if (row < md.rows) {
        for (int k0 = b + group; k0 <= md.last; k0 += 4 * GROUPS) {
            float pm[4], pz[4];
            float4 po[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = k0 + i * GROUPS;
                pm[i] = -INFINITY, pz[i] = 0.f, po[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k <= md.last) {
                    const float* p = parts + (k == b ? 2 * k + 1 : 2 * k) * P;
                    pm[i] = p[ROWS * D + row];
                    pz[i] = p[ROWS * D + ROWS + row];
                    po[i] = *reinterpret_cast<const float4*>(p + row * D + d);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float v[4] = {po[i].x, po[i].y, po[i].z, po[i].w};
                attn_join(m, z, o, pm[i], pz[i], v);
            }
        }
    }
    if (GROUPS > 1) {
        float* mine = s_part[threadIdx.x];
        mine[0] = m, mine[1] = z, mine[2] = o[0], mine[3] = o[1], mine[4] = o[2], mine[5] = o[3];
        __syncthreads();
        if (group == 0)
#pragma unroll
            for (int x = 1; x < GROUPS; ++x) {
                const float* p = s_part[threadIdx.x + x * TPR];
                const float v[4] = {p[2], p[3], p[4], p[5]};
                attn_join(m, z, o, p[0], p[1], v);
            }
        __syncthreads();
    }
    if (group == 0 && row < md.rows) {
        const int g = md.row0 + row, tok = g / a.group;
        const int64_t at = (md.o0 + static_cast<int64_t>(tok)) * a.Hq + md.h0 + g - tok * a.group;
        const float vscale = (F8 && a.cache.v_scale) ? a.cache.v_scale[md.h0 / a.group] : 1.f;
        *reinterpret_cast<uint2*>(a.out + at * D + d) = attn_out4(make_float4(o[0], o[1], o[2], o[3]), z, vscale);
        if (d == 0 && a.lse) a.lse[at] = attn_lse(m, z, F8 ? kAttnPShift : 0.f);
    }
}

template <int D, int ROWS, bool F8>
__global__ void __launch_bounds__(kJoinThreads) tree_attn_join_kernel(AttnArgs a, int grid)
{
    constexpr int TPR = D / 4, kRowsAt = kJoinThreads / TPR;  // rows of a step
    constexpr int kSteps = (ROWS + kRowsAt - 1) / kRowsAt, kGroups = kRowsAt;  // deep: a row a step
    __shared__ int16_t list[kAttnMaxGrid];
    __shared__ int s_counts[kJoinThreads / kWarp * 2];
    __shared__ float s_part[kJoinThreads][6];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    bool deep;
    const int count = attn_unfinished(a, grid, list, s_counts, deep);
    const AttnMeta* meta = static_cast<const AttnMeta*>(a.ws);
    for (int w = blockIdx.x; w < count * kSteps; w += gridDim.x) {
        const int b = list[w / kSteps];
        const AttnMeta md = meta[b];
        if (md.last - b < kAttnDeep)
            attn_join_rows<D, ROWS, F8, 1>(a, md, b, w % kSteps * kRowsAt + threadIdx.x / TPR, s_part);
    }
    if (deep)
        for (int w = blockIdx.x; w < count * ROWS; w += gridDim.x) {
            const int b = list[w / ROWS];
            const AttnMeta md = meta[b];
            if (md.last - b >= kAttnDeep && w % ROWS < md.rows)
                attn_join_rows<D, ROWS, F8, kGroups>(a, md, b, w % ROWS, s_part);
        }
}

// The same for parts that lie column by column (o [D][rows]): a block takes 32
// rows, a warp D / 8 columns of them, and a load is four whole lines of 32 rows
// (eight lanes of four rows). The outputs turn into rows in shared memory.
// A column a thread instead, 32 lines a load, took 75.3 -> 84.5 us of four
// trees of 64 tokens over 8192 (64 query heads on 8).
template <int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) tree_attn_join_columns_kernel(AttnArgs a, int grid)
{
    constexpr int kRowsAt = 32, kSteps = ROWS / kRowsAt, kCols = D / (kJoinThreads / kWarp), kN = kCols / 4;
    constexpr int kStride = D + 8;  // of a row in s_out: 16-byte reads of it stay aligned
    static_assert(kN * 4 == kCols && ROWS % kRowsAt == 0, "split");
    __shared__ int16_t list[kAttnMaxGrid];
    __shared__ int s_counts[kJoinThreads / kWarp * 2];
    __shared__ __align__(16) uint16_t s_out[kRowsAt * kStride];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    bool deep;
    const int count = attn_unfinished(a, grid, list, s_counts, deep);
    const float* parts = reinterpret_cast<const float*>(static_cast<const uint8_t*>(a.ws) + attn_meta_bytes());
    constexpr size_t P = attn_part_floats(ROWS, D);
    const int lane = threadIdx.x % kWarp, r4 = lane % 8 * 4, d0 = threadIdx.x / kWarp * kCols + lane / 8;
    for (int w = blockIdx.x; w < count * kSteps; w += gridDim.x) {
        const int b = list[w / kSteps], row0 = w % kSteps * kRowsAt;
        const AttnMeta md = static_cast<const AttnMeta*>(a.ws)[b];
        if (row0 >= md.rows) continue;
        float m[4], z[4] = {}, o[kN][4] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = -INFINITY;
#pragma unroll 2
        for (int k = b; k <= md.last; ++k) {
            const float* p = parts + (k == b ? 2 * k + 1 : 2 * k) * P + row0 + r4;
            // rows past the live ones of the tile are written by nobody: their values are not used
            const float4 m4 = *reinterpret_cast<const float4*>(p + ROWS * D);
            const float4 z4 = *reinterpret_cast<const float4*>(p + ROWS * D + ROWS);
            float4 x[kN];
#pragma unroll
            for (int n = 0; n < kN; ++n) x[n] = *reinterpret_cast<const float4*>(p + (d0 + 4 * n) * ROWS);
            const float pm[4] = {m4.x, m4.y, m4.z, m4.w}, pz[4] = {z4.x, z4.y, z4.z, z4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float mm = fmaxf(m[i], pm[i]), f = attn_weight(m[i], mm), g = attn_weight(pm[i], mm);
                m[i] = mm;
                z[i] = z[i] * f + pz[i] * g;
#pragma unroll
                for (int n = 0; n < kN; ++n)
                    o[n][i] = o[n][i] * f + (i == 0 ? x[n].x : i == 1 ? x[n].y : i == 2 ? x[n].z : x[n].w) * g;
            }
        }
        auto at = [&](int row) {  // a row's place in out and lse
            const int g = md.row0 + row0 + row, tok = g / a.group;
            return (md.o0 + static_cast<int64_t>(tok)) * a.Hq + md.h0 + g - tok * a.group;
        };
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int n = 0; n < kN; ++n)
                s_out[(r4 + i) * kStride + d0 + 4 * n] =
                    __bfloat16_as_ushort(__float2bfloat16_rn(z[i] == 0.f ? 0.f : o[n][i] / z[i]));
        if (a.lse && d0 == 0)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (row0 + r4 + i < md.rows) a.lse[at(r4 + i)] = attn_lse(m[i], z[i], 0.f);
        __syncthreads();
        for (int x = threadIdx.x; x < kRowsAt * D / 8; x += kJoinThreads) {
            const int row = x / (D / 8), d = x % (D / 8) * 8;
            if (row0 + row < md.rows)
                *reinterpret_cast<uint4*>(a.out + at(row) * D + d) = *reinterpret_cast<const uint4*>(s_out + row * kStride + d);
        }
        __syncthreads();  // s_out is read
    }
}

// Launches a join after the first kernel in the same stream; it may be set up
// while that one still runs, and waits for its end.
inline cudaError_t launch_attn_join(void (*kernel)(AttnArgs, int), const AttnArgs& a, int grid, cudaStream_t s)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kJoinGrid);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, grid);
}

// The kernel for many rows a kv head (tree_attn_wide.cu), bf16 caches.
bool tree_attention_wide_fits(const AttnArgs& a);
size_t tree_attention_wide_ws(int64_t T, int Hq, int Hkv, int D);
cudaError_t launch_tree_attention_wide(const AttnArgs& a, cudaStream_t s);

}  // namespace bqd
