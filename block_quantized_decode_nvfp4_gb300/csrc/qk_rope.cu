// qk_rope.cu -- RMS norm of query and key heads, rotary positions, and the
// write of K and V into the paged cache, in one pass over the projections.
//
// Per head x of D elements: y = x * rsqrt(sum x^2 / D + eps) * w; the first
// rot elements turn by their position's angles, (a, b) -> (a cos - b sin,
// b cos + a sin). Each input element is read once and each output written
// once; the bound is memory (a launch's latency for the few tokens of a
// decode step).
//
// A warp takes kHeads consecutive heads of a token, all loaded before the
// first is used, with D / 32 consecutive elements of each head in a lane: the
// mean square is one warp sum, and the other element of a rotated pair is the
// lane's own (pairs) or sits rot / 2 elements away in one lane (halves:
// rot / 2 is a multiple of the lane's share). The token's cosines and sines
// are read once for all of its heads in the warp.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn.h"
#include "common.cuh"

namespace bqd {

namespace {

constexpr int kThreads = 128;
constexpr int kHeads = 4;

template <int N>
__device__ __forceinline__ void load_f32(const float* p, float (&x)[N])
{
    if constexpr (N == 1) {
        x[0] = __ldg(p);
    } else if constexpr (N == 2) {
        const float2 v = __ldg(reinterpret_cast<const float2*>(p));
        x[0] = v.x, x[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(p) + i);
            x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
        }
    }
}

// E elements of a row as they come: raw words, unpacked later so that a
// warp's loads are all in flight together.
template <typename T, int E>
struct Raw {
    static constexpr int kWords = E * static_cast<int>(sizeof(T)) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T* p)
    {
        if constexpr (kWords == 1) {
            w[0] = __ldcs(reinterpret_cast<const uint32_t*>(p));
        } else if constexpr (kWords == 2) {
            const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
            w[0] = v.x, w[1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p) + i);
                w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
            }
        }
    }
    __device__ __forceinline__ void get(float (&x)[E]) const
    {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if constexpr (sizeof(T) == 4)
                x[i] = __uint_as_float(w[i]);
            else
                x[i] = (i & 1) ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
        }
    }
};

template <int N>
__device__ __forceinline__ void store_words(void* p, const uint32_t (&w)[N])
{
    if constexpr (N == 1)
        *static_cast<uint32_t*>(p) = w[0];
    else if constexpr (N == 2)
        *static_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else
        *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <int E>
__device__ __forceinline__ void store_bf16(uint16_t* p, const float (&y)[E])
{
    uint32_t w[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    store_words(p, w);
}

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int E>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float (&y)[E], float inv)
{
    uint16_t h[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) h[i] = e4m3x2(y[2 * i] * inv, y[2 * i + 1] * inv);
    if constexpr (E == 2) {
        *reinterpret_cast<uint16_t*>(p) = h[0];
    } else {
        uint32_t w[E / 4];
#pragma unroll
        for (int i = 0; i < E / 4; ++i) w[i] = h[2 * i] | (static_cast<uint32_t>(h[2 * i + 1]) << 16);
        store_words(p, w);
    }
}

template <typename T, int D, bool F8>
__global__ void __launch_bounds__(kThreads) qk_rope_kernel(const QkRopeArgs a, uint32_t groups)
{
    constexpr int E = D / kWarp;
    const int lane = threadIdx.x % kWarp;
    const int Hkv = a.cache.heads, heads = a.Hq + 2 * Hkv;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / kWarp) + threadIdx.x / kWarp;
    int64_t t;
    int h0;
    if (a.T * groups < 0xFFFFFF00ll) {  // a 32-bit division where it will do
        const uint32_t tt = static_cast<uint32_t>(item) / groups;
        t = tt;
        h0 = static_cast<int>(static_cast<uint32_t>(item) - tt * groups) * kHeads;
    } else {
        t = item / groups;
        h0 = static_cast<int>(item % groups) * kHeads;
    }
    if (t >= a.T) return;
    const int e0 = lane * E;

    Raw<T, E> raw[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int h = h0 + i;
        if (h < heads) {
            const T* src = h < a.Hq         ? static_cast<const T*>(a.q) + t * a.q_pitch + static_cast<int64_t>(h) * D
                           : h < a.Hq + Hkv ? static_cast<const T*>(a.k) + t * a.k_pitch + static_cast<int64_t>(h - a.Hq) * D
                                            : static_cast<const T*>(a.v) + t * a.v_pitch +
                                                  static_cast<int64_t>(h - a.Hq - Hkv) * D;
            raw[i].load(src + e0);
        }
    }
    const int pos = a.rot ? a.positions[t] : 0;
    const bool pos_ok = a.rot == 0 || (pos >= 0 && pos < a.max_pos);
    const int64_t slot = h0 + kHeads > a.Hq ? a.slots[t] : -1;
    const bool stored = pos_ok && slot >= 0 && slot < a.cache.num_pages * a.cache.page_size;
    const int64_t at0 = stored ? (slot / a.cache.page_size) * a.cache.page_stride +
                                     (slot & (a.cache.page_size - 1)) * a.cache.token_stride
                               : 0;

    // this lane's cosines and sines, signed so that y' = y c + other s
    const int half = a.rot / 2;
    const bool turns = pos_ok && e0 < a.rot;
    const bool upper = e0 >= half;  // halves: which end of its pairs the lane holds
    const int other = turns && !a.pairs ? (upper ? lane - half / E : lane + half / E) : lane;
    float cs[E], sn[E];
    if (turns) {
        const float* p = a.cos_sin + static_cast<int64_t>(pos) * a.rot;
        if (a.pairs) {
            float c2[E / 2], s2[E / 2];
            load_f32(p + e0 / 2, c2);
            load_f32(p + half + e0 / 2, s2);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                cs[i] = c2[i / 2];
                sn[i] = (i & 1) ? s2[i / 2] : -s2[i / 2];
            }
        } else {
            const int i0 = upper ? e0 - half : e0;
            load_f32(p + i0, cs);
            load_f32(p + half + i0, sn);
            if (!upper)
#pragma unroll
                for (int i = 0; i < E; ++i) sn[i] = -sn[i];
        }
    }

#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int h = h0 + i;
        if (h >= heads) break;
        const int kind = h < a.Hq ? 0 : h < a.Hq + Hkv ? 1 : 2;  // q, k, v
        float y[E];
        raw[i].get(y);
        if (kind != 2) {
            const float* w = kind == 0 ? a.q_weight : a.k_weight;
            if (w) {
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < E; ++j) ss += y[j] * y[j];
                const float r = rsqrtf(warp_sum(ss) / D + a.eps);
                float g[E];
                load_f32(w + e0, g);
#pragma unroll
                for (int j = 0; j < E; ++j) y[j] *= r * g[j];
            }
            if (a.rot) {
                float z[E];
#pragma unroll
                for (int j = 0; j < E; ++j) z[j] = a.pairs ? y[j ^ 1] : __shfl_sync(0xFFFFFFFFu, y[j], other);
                if (turns)
#pragma unroll
                    for (int j = 0; j < E; ++j) y[j] = y[j] * cs[j] + z[j] * sn[j];
            }
        }
        if (kind == 0) {
            if (!pos_ok)
#pragma unroll
                for (int j = 0; j < E; ++j) y[j] = 0.f;
            store_bf16(a.q_out + (t * a.Hq + h) * D + e0, y);
        } else if (stored) {
            const int hh = kind == 1 ? h - a.Hq : h - a.Hq - Hkv;
            const int64_t at = at0 + static_cast<int64_t>(hh) * a.cache.head_stride + e0;
            void* base = kind == 1 ? a.cache.k : a.cache.v;
            if constexpr (F8) {
                const float* sc = kind == 1 ? a.cache.k_scale : a.cache.v_scale;
                store_e4m3(static_cast<uint8_t*>(base) + at, y, sc ? 1.f / sc[hh] : 1.f);
            } else {
                store_bf16(static_cast<uint16_t*>(base) + at, y);
            }
        }
    }
}

template <typename T, int D>
void launch(const QkRopeArgs& a, cudaStream_t s)
{
    const uint32_t groups = static_cast<uint32_t>((a.Hq + 2 * a.cache.heads + kHeads - 1) / kHeads);
    const int64_t blocks = (a.T * groups + kThreads / kWarp - 1) / (kThreads / kWarp);
    if (a.cache.type == BQD_E4M3)
        qk_rope_kernel<T, D, true><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a, groups);
    else
        qk_rope_kernel<T, D, false><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a, groups);
}

template <typename T>
void launch_d(const QkRopeArgs& a, cudaStream_t s)
{
    switch (a.cache.head_dim) {
        case 64: return launch<T, 64>(a, s);
        case 128: return launch<T, 128>(a, s);
        default: return launch<T, 256>(a, s);
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope_cache(const QkRopeArgs& a, int in_type, cudaStream_t s)
{
    if (in_type == BQD_F32)
        launch_d<float>(a, s);
    else
        launch_d<__nv_bfloat16>(a, s);
    return cudaGetLastError();
}

}  // namespace bqd
