// qk_rope.cu -- RMS norm of query and key heads, rotary positions, and the
// write of K and V into the paged cache, in one pass over the projections.
//
// Per head x of D elements: y = x * rsqrt(sum x^2 / D + eps) * w; the first
// rot elements turn by their position's angles, (a, b) -> (a cos - b sin,
// b cos + a sin). Each input element is read once and each output written
// once; the bound is memory.
//
// Simple form: one warp per (token, head), element by element, the normed
// head in shared memory between the norm and the rotation.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn.h"
#include "common.cuh"

namespace bqd {

namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float load_one(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float load_one(const __nv_bfloat16* p, int64_t i) { return __bfloat162float(p[i]); }

__device__ __forceinline__ uint8_t to_e4m3(float x)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
    return static_cast<uint8_t>(r);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) qk_rope_kernel(const QkRopeArgs a)
{
    __shared__ float buf[kThreads / kWarp][256];
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    const int Hkv = a.cache.heads, D = a.cache.head_dim, heads = a.Hq + 2 * Hkv;
    float* y = buf[warp];
    const int64_t items = a.T * heads, step = static_cast<int64_t>(gridDim.x) * (kThreads / kWarp);
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * (kThreads / kWarp) + warp; it < items; it += step) {
        const int64_t t = it / heads;
        const int h = static_cast<int>(it % heads);
        const int kind = h < a.Hq ? 0 : h < a.Hq + Hkv ? 1 : 2;  // q, k, v
        const int hh = kind == 0 ? h : kind == 1 ? h - a.Hq : h - a.Hq - Hkv;
        const T* src = kind == 0   ? static_cast<const T*>(a.q) + t * a.q_pitch
                       : kind == 1 ? static_cast<const T*>(a.k) + t * a.k_pitch
                                   : static_cast<const T*>(a.v) + t * a.v_pitch;
        src += static_cast<int64_t>(hh) * D;
        const int pos = a.rot ? a.positions[t] : 0;
        const bool pos_ok = a.rot == 0 || (pos >= 0 && pos < a.max_pos);
        float ss = 0.f;
        for (int i = lane; i < D; i += kWarp) {
            y[i] = load_one(src, i);
            ss += y[i] * y[i];
        }
        const float* w = kind == 0 ? a.q_weight : kind == 1 ? a.k_weight : nullptr;
        if (w) {
            const float r = rsqrtf(warp_sum(ss) / D + a.eps);
            for (int i = lane; i < D; i += kWarp) y[i] = y[i] * r * w[i];
        }
        __syncwarp();
        if (kind != 2 && pos_ok) {
            const float* cs = a.cos_sin + static_cast<int64_t>(pos) * a.rot;
            const int half = a.rot / 2;
            for (int i = lane; i < half; i += kWarp) {
                const int ia = a.pairs ? 2 * i : i, ib = a.pairs ? 2 * i + 1 : i + half;
                const float u = y[ia], v = y[ib], c = cs[i], s = cs[half + i];
                y[ia] = u * c - v * s;
                y[ib] = v * c + u * s;
            }
        }
        __syncwarp();
        if (kind == 0) {
            __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.q_out) + (t * a.Hq + hh) * D;
            for (int i = lane; i < D; i += kWarp) out[i] = __float2bfloat16_rn(pos_ok ? y[i] : 0.f);
        } else {
            const int64_t slot = a.slots[t];
            if (pos_ok && slot >= 0 && slot < a.cache.num_pages * a.cache.page_size) {
                const int64_t at = slot / a.cache.page_size * a.cache.page_stride +
                                   slot % a.cache.page_size * a.cache.token_stride +
                                   static_cast<int64_t>(hh) * a.cache.head_stride;
                void* base = kind == 1 ? a.cache.k : a.cache.v;
                const float* sc = kind == 1 ? a.cache.k_scale : a.cache.v_scale;
                if (a.cache.type == BQD_BF16) {
                    for (int i = lane; i < D; i += kWarp)
                        static_cast<__nv_bfloat16*>(base)[at + i] = __float2bfloat16_rn(y[i]);
                } else {
                    const float inv = sc ? 1.f / sc[hh] : 1.f;
                    for (int i = lane; i < D; i += kWarp) static_cast<uint8_t*>(base)[at + i] = to_e4m3(y[i] * inv);
                }
            }
        }
        __syncwarp();
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope_cache(const QkRopeArgs& a, int in_type, cudaStream_t s)
{
    const int64_t items = a.T * (a.Hq + 2 * a.cache.heads);
    const int64_t need = (items + kThreads / kWarp - 1) / (kThreads / kWarp);
    const unsigned grid = static_cast<unsigned>(need < 152 * 16 ? need : 152 * 16);
    if (in_type == BQD_F32)
        qk_rope_kernel<float><<<grid, kThreads, 0, s>>>(a);
    else
        qk_rope_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace bqd
