// tree_attn.cu -- attention of drafted tokens (a chain or a tree; one token:
// decode) over the paged cache.
//
// out = sum_l p_l v_l / sum_l p_l with p_l = exp(s_l - m), s_l = scale q . k_l
// over the visible l, m the running maximum: a partial result over some of
// the tokens is (m, z = sum p, o = sum p v), and two of them join as
// m = max(m1, m2), z = z1 e^(m1 - m) + z2 e^(m2 - m), o likewise. lse = m +
// log z. A partial that saw nothing has m = -inf, z = 0.
//
// Simple form: one CTA per (token, query head), its warps taking tokens in
// turn, a lane holding D / 32 elements; joined in shared memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn.h"
#include "common.cuh"

namespace bqd {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / kWarp;

__device__ __forceinline__ float cache_elem(const bqd_kv_cache& c, const void* base, int64_t i)
{
    return c.type == BQD_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i])
                              : e4m3_to_float(static_cast<const uint8_t*>(base)[i]);
}

__global__ void __launch_bounds__(kThreads) tree_attn_kernel(const AttnArgs a)
{
    __shared__ float s_m[kWarps], s_z[kWarps], s_o[kWarps][256];
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    const int64_t t = blockIdx.x;
    const int h = blockIdx.y, D = a.cache.head_dim, E = D / kWarp, kvh = h / (a.Hq / a.cache.heads);
    // the request of token t: the last r with offsets[r] <= t < offsets[r + 1]
    int64_t lo = 0, hi = a.R;
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (a.offsets[mid + 1] <= t)
            lo = mid + 1;
        else
            hi = mid;
    }
    if (lo >= a.R || t < a.offsets[lo]) return;
    const int64_t r = lo, o0 = max(0, a.offsets[r]), n = min(static_cast<int64_t>(a.offsets[r + 1]), a.T) - o0;
    const int64_t i = t - o0, ctx = max(0, a.context[r]);
    float q[8], o[8], m = -INFINITY, z = 0.f;
    const float ks = (a.cache.type == BQD_E4M3 && a.cache.k_scale) ? a.cache.k_scale[kvh] : 1.f;
    const float vs = (a.cache.type == BQD_E4M3 && a.cache.v_scale) ? a.cache.v_scale[kvh] : 1.f;
    for (int e = 0; e < 8; ++e) {
        o[e] = 0.f;
        q[e] = e < E ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.q)[t * a.q_pitch + h * D + lane * E + e])
                     : 0.f;
    }
    for (int64_t l = warp; l < ctx + n; l += kWarps) {
        if (l >= ctx) {
            const int64_t j = l - ctx;
            const bool see = a.mask ? (j / 64 < a.mask_words && ((a.mask[t * a.mask_words + j / 64] >> (j % 64)) & 1))
                                    : j <= i;
            if (!see) continue;
        }
        const int64_t b = l / a.cache.page_size;
        if (b >= a.width) break;
        const int32_t page = a.table[r * a.width + b];
        if (page < 0 || page >= a.cache.num_pages) continue;
        const int64_t at = page * a.cache.page_stride + l % a.cache.page_size * a.cache.token_stride +
                           kvh * a.cache.head_stride + lane * E;
        float s = 0.f;
        for (int e = 0; e < E; ++e) s += q[e] * cache_elem(a.cache, a.cache.k, at + e);
        s = warp_sum(s) * (a.scale * ks);
        const float mn = fmaxf(m, s);
        const float f = m == -INFINITY ? 0.f : expf(m - mn);  // a first token of score -inf: exp(nan) below
        const float p = s == -INFINITY ? 0.f : expf(s - mn);
        z = z * f + p;
        for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * cache_elem(a.cache, a.cache.v, at + e);
        m = mn;
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_z[warp] = z;
    }
    for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
    __syncthreads();
    float mm = -INFINITY;
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w]);
    float zz = 0.f, f[kWarps];
    for (int w = 0; w < kWarps; ++w) {
        f[w] = s_m[w] == -INFINITY ? 0.f : expf(s_m[w] - mm);
        zz += s_z[w] * f[w];
    }
    for (int d = threadIdx.x; d < D; d += kThreads) {
        float v = 0.f;
        for (int w = 0; w < kWarps; ++w) v += s_o[w][d] * f[w];
        a.out[(t * a.Hq + h) * D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(zz == 0.f ? 0.f : v * vs / zz));
    }
    if (a.lse && threadIdx.x == 0) a.lse[t * a.Hq + h] = zz == 0.f ? -INFINITY : mm + logf(zz);
}

}  // namespace

size_t tree_attention_ws(int64_t, int64_t, int, int, int) { return 16; }

cudaError_t launch_tree_attention(const AttnArgs& a, cudaStream_t s)
{
    tree_attn_kernel<<<dim3(static_cast<unsigned>(a.T), static_cast<unsigned>(a.Hq)), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace bqd
