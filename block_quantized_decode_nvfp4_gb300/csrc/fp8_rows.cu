// fp8_rows.cu -- 8-bit activations: rows to E4M3 codes with a scale for each
// token and 128 channels, and the residual add with its norms that writes them.
//
// A block of 128 channels of a token takes 16 lanes of 8 elements, so its
// largest magnitude is four shuffles away and a lane's codes are one 8-byte
// store. Scales lie block-major ([ceil(K/128)][T]): the products read the scale
// of a block for neighbouring tokens. Both kernels read each input once and
// write each output once; the bound is memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "f32x2.cuh"
#include "fp8.cuh"
#include "fp8.h"

namespace bqd {

namespace {

constexpr int kRun = 8;                // elements of a lane in a block
constexpr int kLanes = 128 / kRun;     // lanes of a block
constexpr int kEncThreads = 256;
constexpr int kEncTokens = 4;          // tokens of a 16-lane group

// Eight elements as fp32 pairs.
__device__ __forceinline__ void load8(const void* base, int64_t at, bool f32, uint64_t (&v)[4])
{
    if (f32) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + at);
        const uint4 a = __ldcs(p), b = __ldcs(p + 1);
        v[0] = pack(__uint_as_float(a.x), __uint_as_float(a.y));
        v[1] = pack(__uint_as_float(a.z), __uint_as_float(a.w));
        v[2] = pack(__uint_as_float(b.x), __uint_as_float(b.y));
        v[3] = pack(__uint_as_float(b.z), __uint_as_float(b.w));
    } else {
        const uint4 a = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at));
        v[0] = pack(bf16_lo(a.x), bf16_hi(a.x));
        v[1] = pack(bf16_lo(a.y), bf16_hi(a.y));
        v[2] = pack(bf16_lo(a.z), bf16_hi(a.z));
        v[3] = pack(bf16_lo(a.w), bf16_hi(a.w));
    }
}

__device__ __forceinline__ uint32_t bf16_pair(uint64_t v)
{
    float a, b;
    unpack(v, a, b);
    return to_bf16x2(a, b);
}

__device__ __forceinline__ void store8(void* base, int64_t at, bool f32, const uint64_t (&v)[4])
{
    if (f32) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) unpack(v[i], f[2 * i], f[2 * i + 1]);
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
        p[0] = make_float4(f[0], f[1], f[2], f[3]);
        p[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) =
            make_uint4(bf16_pair(v[0]), bf16_pair(v[1]), bf16_pair(v[2]), bf16_pair(v[3]));
    }
}

// The scale of a block from its 16 lanes' elements.
__device__ __forceinline__ float lanes_scale(const uint64_t (&v)[4])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        unpack(v[i], a, b);
        m = max(m, max(abs_bits(a), abs_bits(b)));
    }
#pragma unroll
    for (int d = kLanes / 2; d; d >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    return block_scale(m);
}

__device__ __forceinline__ void store_codes(uint8_t* p, const uint64_t (&v)[4], float scale)
{
    const BlockCoder c(scale);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(c.pair(v[0]) | (c.pair(v[1]) << 16), c.pair(v[2]) | (c.pair(v[3]) << 16));
}

template <bool F32>
__global__ void __launch_bounds__(kEncThreads) encode_x_kernel(const EncodeXArgs a, uint32_t blocks, uint64_t groups)
{
    const uint64_t g = (static_cast<uint64_t>(blockIdx.x) * kEncThreads + threadIdx.x) / kLanes;
    const int lane = threadIdx.x % kLanes;
    const uint64_t gc = g < groups ? g : groups - 1;  // lanes of a warp stay together
    const uint64_t tg = gc / blocks;
    const uint32_t kb = static_cast<uint32_t>(gc - tg * blocks);
    const int64_t k = static_cast<int64_t>(kb) * 128 + lane * kRun;
    const int64_t t0 = static_cast<int64_t>(tg) * kEncTokens;
    const bool live = g < groups && k < a.K;  // K is a multiple of 16
    uint64_t v[kEncTokens][4];
#pragma unroll
    for (int i = 0; i < kEncTokens; ++i) {
        if (live && t0 + i < a.T)
            load8(a.x, (t0 + i) * a.pitch + k, F32, v[i]);
        else
            v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0;
    }
#pragma unroll
    for (int i = 0; i < kEncTokens; ++i) {
        const float s = lanes_scale(v[i]);
        if (t0 + i < a.T && g < groups) {
            if (live) store_codes(a.codes + (t0 + i) * a.K + k, v[i], s);
            if (lane == 0) a.scales[static_cast<int64_t>(kb) * a.T + t0 + i] = s;
        }
    }
}

// A row takes TPR threads, VPT chunks of 8 elements each (chunk v of thread i
// is chunk v TPR + i of the row); a CTA takes max(1, 256 / TPR) rows.
constexpr int norm_rows(int tpr) { return tpr >= 256 ? 1 : 256 / tpr; }

// Sum over a row's threads, the same in all of them.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* buf)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    if constexpr (TPR > kWarp) {
        constexpr int W = TPR / kWarp;
        const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
        if (lane == 0) buf[warp] = v;
        __syncthreads();
        v = buf[warp / W * W + lane % W];
#pragma unroll
        for (int d = W / 2; d; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    }
    return v;
}

template <int TPR, int VPT>
__global__ void __launch_bounds__(TPR* norm_rows(TPR)) residual_norm_kernel(const NormArgs a)
{
    constexpr int R = norm_rows(TPR);
    __shared__ float buf[2][TPR * R / kWarp];
    const int i = threadIdx.x % TPR;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * R + threadIdx.x / TPR;
    const bool row = t < a.T;
    const int64_t at0 = t * a.H;
    fp8_pdl_trigger();
    fp8_pdl_wait();
    uint64_t z[VPT][4], r[VPT][4];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int e = (v * TPR + i) * kRun;
        const bool live = row && e < a.H;
        z[v][0] = z[v][1] = z[v][2] = z[v][3] = 0;
        r[v][0] = r[v][1] = r[v][2] = r[v][3] = 0;
        if (live && a.x) load8(a.x, t * a.x_pitch + e, a.x_f32, z[v]);
        if (live && a.residual) load8(a.residual, at0 + e, a.res_f32, r[v]);
    }
    if (a.x) {
        float rs = 1.f;
        if (a.post_weight) {
            uint64_t ss = 0;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int j = 0; j < 4; ++j) ss = fma2(z[v][j], z[v][j], ss);
            float s0, s1;
            unpack(ss, s0, s1);
            rs = rsqrtf(row_sum<TPR>(s0 + s1, buf[0]) / static_cast<float>(a.H) + a.eps);
        }
        const uint64_t rs2 = pack(rs, rs), sc = pack(a.scale, a.scale);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int e = (v * TPR + i) * kRun;
            if (!row || e >= a.H) continue;
            if (a.post_weight) {
                const float4 w0 = __ldg(reinterpret_cast<const float4*>(a.post_weight + e));
                const float4 w1 = __ldg(reinterpret_cast<const float4*>(a.post_weight + e) + 1);
                const uint64_t w[4] = {pack(w0.x, w0.y), pack(w0.z, w0.w), pack(w1.x, w1.y), pack(w1.z, w1.w)};
#pragma unroll
                for (int j = 0; j < 4; ++j) z[v][j] = mul2(mul2(z[v][j], rs2), w[j]);
            }
            if (a.gate) {
                uint64_t g[4];
                load8(a.gate, t * a.gate_pitch + e, a.gate_f32, g);
#pragma unroll
                for (int j = 0; j < 4; ++j) z[v][j] = mul2(z[v][j], g[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) r[v][j] = fma2(z[v][j], sc, r[v][j]);
        }
    }
    if (a.residual_out) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int e = (v * TPR + i) * kRun;
            if (row && e < a.H) store8(a.residual_out, at0 + e, a.res_f32, r[v]);
        }
    }
    if (!a.y) return;
    uint64_t ss = 0;
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int j = 0; j < 4; ++j) ss = fma2(r[v][j], r[v][j], ss);
    float s0, s1;
    unpack(ss, s0, s1);
    const float rs = rsqrtf(row_sum<TPR>(s0 + s1, buf[1]) / static_cast<float>(a.H) + a.eps);
    const uint64_t rs2 = pack(rs, rs);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int e = (v * TPR + i) * kRun;
        const bool live = row && e < a.H;
        if (live) {
            const float4 w0 = __ldg(reinterpret_cast<const float4*>(a.pre_weight + e));
            const float4 w1 = __ldg(reinterpret_cast<const float4*>(a.pre_weight + e) + 1);
            const uint64_t w[4] = {pack(w0.x, w0.y), pack(w0.z, w0.w), pack(w1.x, w1.y), pack(w1.z, w1.w)};
#pragma unroll
            for (int j = 0; j < 4; ++j) r[v][j] = mul2(mul2(r[v][j], rs2), w[j]);
        }
        if (a.y_e4m3) {
            const float s = lanes_scale(r[v]);  // every lane takes part; those past H hold zeros
            if (live) store_codes(static_cast<uint8_t*>(a.y) + at0 + e, r[v], s);
            if (live && e % 128 == 0) a.y_scales[static_cast<int64_t>(e / 128) * a.T + t] = s;
        } else if (live) {
            store8(a.y, at0 + e, false, r[v]);
        }
    }
}

template <int TPR, int VPT>
cudaError_t launch_norm(const NormArgs& a, cudaStream_t s)
{
    constexpr int R = norm_rows(TPR);
    residual_norm_kernel<TPR, VPT><<<static_cast<unsigned>((a.T + R - 1) / R), TPR * R, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp8_x_encode(const EncodeXArgs& a, int x_type, cudaStream_t s)
{
    const uint64_t blocks = static_cast<uint64_t>((a.K + 127) / 128);
    const uint64_t groups = blocks * static_cast<uint64_t>((a.T + kEncTokens - 1) / kEncTokens);
    const uint64_t per = kEncThreads / kLanes, ctas = (groups + per - 1) / per;
    if (ctas > 0x7FFFFFFFull) return cudaErrorInvalidValue;
    if (x_type == BQD_F32)
        encode_x_kernel<true><<<static_cast<unsigned>(ctas), kEncThreads, 0, s>>>(a, static_cast<uint32_t>(blocks), groups);
    else
        encode_x_kernel<false><<<static_cast<unsigned>(ctas), kEncThreads, 0, s>>>(a, static_cast<uint32_t>(blocks), groups);
    return cudaGetLastError();
}

cudaError_t launch_residual_norm(const NormArgs& a, cudaStream_t s)
{
    if (a.H <= 256) return launch_norm<32, 1>(a, s);
    if (a.H <= 512) return launch_norm<64, 1>(a, s);
    if (a.H <= 1024) return launch_norm<128, 1>(a, s);
    if (a.H <= 2048) return launch_norm<256, 1>(a, s);
    if (a.H <= 4096) return launch_norm<512, 1>(a, s);
    if (a.H <= 8192) return launch_norm<512, 2>(a, s);
    return launch_norm<1024, 2>(a, s);  // to kNormMaxH
}

}  // namespace bqd
