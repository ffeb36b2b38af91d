// qk_rope.cu -- RMS norm of query and key heads, rotary positions, and the
// write of K and V into the paged cache, in one pass over the projections.
//
// Per head x of D elements: y = x * rsqrt(sum x^2 / D + eps) * w; the first
// rot elements turn by their position's angles, (a, b) -> (a cos - b sin,
// b cos + a sin). Each input element is read once and each output written
// once; the bound is memory (a launch's latency for the few tokens of a
// decode step), and next to it the instructions per element.
//
// A head takes D / 16 lanes of 16 elements, so a warp does 2, 4 or 8 heads of
// a token in a step, and the shuffles, addresses and the square root are
// shared by 16 elements a lane. The D / 2 pairs of a head (the rotated ones,
// then the rest two by two) go to its lanes in order, eight each: both ends
// of a pair are in one lane, the rotation needs no exchange, and a lane's
// elements are two runs of eight (rot / 2 is a multiple of 8). Arithmetic is
// two elements an instruction. Weights and angles come from L1 at every step,
// which leaves the registers to loads in flight: two steps of bf16 or one of
// fp32 ahead of the work, 2 KiB a warp and 64 KiB an SM. 8191 bf16 tokens of
// 16 + 2 x 2 heads of 256 take 33.8 us, 168 MB at 5.0 TB/s (54 % of the issue
// slots, 41 % of the warps: the loads' latency and the instructions share the
// rest); one token 2.4 us, 128 tokens over an E4M3 cache 4.1 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn.h"
#include "common.cuh"
#include "f32x2.cuh"

namespace bqd {

namespace {

constexpr int kThreads = 256;
constexpr int kRun = 8;  // elements of one of a lane's two runs

// Eight elements of a row as they come.
template <typename T>
struct Raw {
    static constexpr int kVec = kRun * static_cast<int>(sizeof(T)) / 16;
    uint4 v[kVec];
    __device__ __forceinline__ void load(const T* p)
    {
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void get(uint64_t (&x)[kRun / 2]) const
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                x[2 * i] = pack(__uint_as_float(v[i].x), __uint_as_float(v[i].y));
                x[2 * i + 1] = pack(__uint_as_float(v[i].z), __uint_as_float(v[i].w));
            }
        } else {
            x[0] = pack(bf16_lo(v[0].x), bf16_hi(v[0].x));
            x[1] = pack(bf16_lo(v[0].y), bf16_hi(v[0].y));
            x[2] = pack(bf16_lo(v[0].z), bf16_hi(v[0].z));
            x[3] = pack(bf16_lo(v[0].w), bf16_hi(v[0].w));
        }
    }
};

__device__ __forceinline__ void load8(const float* p, uint64_t (&x)[kRun / 2])
{
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = pack(a.x, a.y);
    x[1] = pack(a.z, a.w);
    x[2] = pack(b.x, b.y);
    x[3] = pack(b.z, b.w);
}

__device__ __forceinline__ uint32_t bf16x2(uint64_t v)
{
    float x, y;
    unpack(v, x, y);
    const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void store_bf16(uint16_t* p, const uint64_t (&y)[kRun / 2])
{
    *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2(y[0]), bf16x2(y[1]), bf16x2(y[2]), bf16x2(y[3]));
}

__device__ __forceinline__ uint32_t e4m3x2(float x, float y)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x4(uint64_t u, uint64_t v)
{
    float x0, x1, x2, x3;
    unpack(u, x0, x1);
    unpack(v, x2, x3);
    return e4m3x2(x0, x1) | (e4m3x2(x2, x3) << 16);
}
// A run's quotients by the head's scale, as codes. A product with the rounded
// reciprocal alone would now and then land on the other side of a boundary
// between codes: one step from its remainder (Markstein 1990) makes it the
// quotient, rounded once. Where that leaves fp32's range (infinities, products
// past it, scales beyond 2^+-60: inv is NaN) the codes are NaN, and are made
// again by division. 8191 bf16 tokens of 8 + 2 x 8 heads: 21.7 us, by division
// alone 23.8, by the product alone 20.7.
__device__ __forceinline__ void store_e4m3(uint8_t* p, const uint64_t (&y)[kRun / 2], float scale, float inv)
{
    const uint64_t i2 = pack(inv, inv), s2 = pack(-scale, -scale);
    auto quotient = [&](uint64_t v) {
        const uint64_t q = mul2(v, i2);
        return fma2(fma2(q, s2, v), i2, q);
    };
    uint2 c = make_uint2(e4m3x4(quotient(y[0]), quotient(y[1])), e4m3x4(quotient(y[2]), quotient(y[3])));
    auto nan_codes = [](uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; };
    if (nan_codes(c.x) | nan_codes(c.y)) {
#pragma unroll 1
        for (int i = 0; i < kRun / 2; ++i) {
            float a, b;
            unpack(i == 0 ? y[0] : i == 1 ? y[1] : i == 2 ? y[2] : y[3], a, b);
            const uint32_t k = e4m3x2(__fdiv_rn(a, scale), __fdiv_rn(b, scale)) << (i % 2 * 16);
            const uint32_t keep = i % 2 ? 0xFFFFu : 0u;
            if (i < 2)
                c.x = (c.x & keep) | k;
            else
                c.y = (c.y & keep) | k;
        }
    }
    *reinterpret_cast<uint2*>(p) = c;
}

template <typename T, int D, bool F8, bool PAIRS>
__global__ void __launch_bounds__(kThreads, 4) qk_rope_kernel(const QkRopeArgs a, uint32_t groups, int run)
{
    constexpr int L = D / 16, HW = kWarp / L;  // lanes of a head, heads of a step
    constexpr int N = kRun / 2;
    const int lane = threadIdx.x % kWarp, l = lane % L;
    const int Hkv = a.cache.heads, heads = a.Hq + 2 * Hkv;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / kWarp) + threadIdx.x / kWarp;
    int64_t t;
    int g;
    if (a.T * groups < 0xFFFFFF00ll) {  // a 32-bit division where it will do
        const uint32_t tt = static_cast<uint32_t>(item) / groups;
        t = tt;
        g = static_cast<int>(static_cast<uint32_t>(item) - tt * groups);
    } else {
        t = item / groups;
        g = static_cast<int>(item % groups);
    }
    if (t >= a.T) return;
    const int h0 = g * run + lane / L, h1 = min((g + 1) * run, heads);  // this lane's heads: h0, h0 + HW, ...
    const int s = l * kRun, half = a.rot / 2;                            // the lane's first pair
    const int e0 = PAIRS ? 2 * s : s < half ? s : half + s;
    const int e1 = PAIRS ? 2 * s + kRun : s < half ? s + half : e0 + (D - a.rot) / 2;

    // rows of q, k and v, each so that head h is h D further
    const T* qb = static_cast<const T*>(a.q) + t * a.q_pitch;
    const T* kb = static_cast<const T*>(a.k) + t * a.k_pitch - static_cast<int64_t>(a.Hq) * D;
    const T* vb = static_cast<const T*>(a.v) + t * a.v_pitch - static_cast<int64_t>(a.Hq + Hkv) * D;
    constexpr int kFar = sizeof(T) == 2 ? 2 : 1;  // steps in flight
    Raw<T> lo[kFar], hi[kFar];
    auto fetch = [&](int i, int h) {
        if (h < h1) {
            const T* src = (h < a.Hq ? qb : h < a.Hq + Hkv ? kb : vb) + static_cast<int64_t>(h) * D;
            lo[i].load(src + e0);
            hi[i].load(src + e1);
        }
    };
#pragma unroll
    for (int i = 0; i < kFar; ++i) fetch(i, h0 + i * HW);
    const int pos = a.rot ? a.positions[t] : 0;
    const bool pos_ok = a.rot == 0 || (pos >= 0 && pos < a.max_pos);
    const int64_t slot = h1 > a.Hq ? a.slots[t] : -1;
    const bool stored = pos_ok && slot >= 0 && slot < a.cache.num_pages * a.cache.page_size;
    const int shift = 31 - __clz(a.cache.page_size);
    const int64_t at0 = stored ? (slot >> shift) * a.cache.page_stride +
                                     (slot & (a.cache.page_size - 1)) * a.cache.token_stride
                               : 0;
    const bool turns = pos_ok && s < half;
    const float* angles = a.cos_sin + static_cast<int64_t>(turns ? pos : 0) * a.rot + s;  // one per pair

    for (int hb = h0; hb - lane / L < h1; hb += kFar * HW)  // as often for every lane of the warp
#pragma unroll
    for (int i = 0; i < kFar; ++i) {
        const int h = hb + i * HW;
        if (h - lane / L >= h1) break;
        uint64_t y0[N], y1[N];
        lo[i].get(y0);
        hi[i].get(y1);
        fetch(i, h + kFar * HW);
        const bool live = h < h1, is_q = live && h < a.Hq, is_k = live && !is_q && h < a.Hq + Hkv;
        const float* w = is_q ? a.q_weight : is_k ? a.k_weight : nullptr;
        uint64_t ss2 = 0;
#pragma unroll
        for (int x = 0; x < N; ++x) ss2 = fma2(y1[x], y1[x], fma2(y0[x], y0[x], ss2));
        float ss, st;
        unpack(ss2, ss, st);
        ss += st;
#pragma unroll
        for (int d = L / 2; d; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
        if (w) {
            const float r = rsqrtf(ss * (1.f / D) + a.eps);
            const uint64_t rr = pack(r, r);
            uint64_t g[N];
            load8(w + e0, g);
#pragma unroll
            for (int x = 0; x < N; ++x) y0[x] = mul2(mul2(y0[x], rr), g[x]);
            load8(w + e1, g);
#pragma unroll
            for (int x = 0; x < N; ++x) y1[x] = mul2(mul2(y1[x], rr), g[x]);
        }
        if (turns && (is_q || is_k)) {
            uint64_t cs[N], sn[N];
            load8(angles, cs);
            load8(angles + half, sn);
            if (PAIRS) {
                // pairs 0 .. 3 in y0, 4 .. 7 in y1, each one register pair
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    float p, q, c0, c1, s0, s1;
                    unpack(cs[i / 2], c0, c1);
                    unpack(sn[i / 2], s0, s1);
                    unpack(y0[i], p, q);
                    const float ca = i % 2 ? c1 : c0, sa = i % 2 ? s1 : s0;
                    y0[i] = pack(p * ca - q * sa, q * ca + p * sa);
                    unpack(cs[2 + i / 2], c0, c1);
                    unpack(sn[2 + i / 2], s0, s1);
                    unpack(y1[i], p, q);
                    const float cb = i % 2 ? c1 : c0, sb = i % 2 ? s1 : s0;
                    y1[i] = pack(p * cb - q * sb, q * cb + p * sb);
                }
            } else {
                const uint64_t minus = pack(-1.f, -1.f);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const uint64_t p = y0[i], q = y1[i];
                    y0[i] = fma2(p, cs[i], mul2(mul2(q, sn[i]), minus));
                    y1[i] = fma2(q, cs[i], mul2(p, sn[i]));
                }
            }
        }
        if (is_q) {
            if (!pos_ok)
#pragma unroll
                for (int i = 0; i < N; ++i) y0[i] = y1[i] = 0;
            uint16_t* out = a.q_out + (t * a.Hq + h) * D;
            store_bf16(out + e0, y0);
            store_bf16(out + e1, y1);
        } else if (live && stored) {
            const int hc = is_k ? h - a.Hq : h - a.Hq - Hkv;
            const int64_t at = at0 + static_cast<int64_t>(hc) * a.cache.head_stride;
            void* base = is_k ? a.cache.k : a.cache.v;
            if constexpr (F8) {
                const float* sc = is_k ? a.cache.k_scale : a.cache.v_scale;
                const float scale = sc ? sc[hc] : 1.f;
                const float inv = fabsf(scale) > 0x1p-60f && fabsf(scale) < 0x1p60f ? 1.f / scale : NAN;
                store_e4m3(static_cast<uint8_t*>(base) + at + e0, y0, scale, inv);
                store_e4m3(static_cast<uint8_t*>(base) + at + e1, y1, scale, inv);
            } else {
                store_bf16(static_cast<uint16_t*>(base) + at + e0, y0);
                store_bf16(static_cast<uint16_t*>(base) + at + e1, y1);
            }
        }
    }
}

template <typename T, int D, bool F8, bool PAIRS>
void launch(const QkRopeArgs& a, cudaStream_t s)
{
    // Heads per warp: one step's (512 / D), doubled while the warps still fill
    // the GPU once. Longer runs start fewer warps, each with the latency of its
    // first loads: 8191 tokens of 20 heads 33.8 us, against 36.0 where they fill
    // it four times and 44.1 at one step a warp.
    const int heads = a.Hq + 2 * a.cache.heads;
    int run = 512 / D;
    while (run < heads && a.T * ((heads + 2 * run - 1) / (2 * run)) >= 152 * 24) run *= 2;
    const uint32_t groups = static_cast<uint32_t>((heads + run - 1) / run);
    const int64_t blocks = (a.T * groups + kThreads / kWarp - 1) / (kThreads / kWarp);
    qk_rope_kernel<T, D, F8, PAIRS><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a, groups, run);
}

template <typename T, int D>
void launch_t(const QkRopeArgs& a, cudaStream_t s)
{
    if (a.cache.type == BQD_E4M3)
        a.pairs ? launch<T, D, true, true>(a, s) : launch<T, D, true, false>(a, s);
    else
        a.pairs ? launch<T, D, false, true>(a, s) : launch<T, D, false, false>(a, s);
}

template <typename T>
void launch_d(const QkRopeArgs& a, cudaStream_t s)
{
    switch (a.cache.head_dim) {
        case 64: return launch_t<T, 64>(a, s);
        case 128: return launch_t<T, 128>(a, s);
        default: return launch_t<T, 256>(a, s);
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
