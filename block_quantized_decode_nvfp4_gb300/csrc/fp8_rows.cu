// fp8_rows.cu -- 8-bit activations: rows to E4M3 codes with a scale for each
// token and 128 channels, and the residual add with its norms that writes them.
//
// A block of 128 channels of a token takes 8 lanes of 16 elements (8 in each half
// of the block: loads and stores of 8 lanes are whole sectors), so its largest
// magnitude is three shuffles away. Scales lie block-major ([ceil(K/128)][T]): the
// products read the scale of a block for neighbouring tokens. Both kernels read
// each input once and write each output once; the bound is memory, and behind it
// the instructions (19 of them for 8 elements of fp32 in the encoder, twice that
// with two norms).
//   fp8_x_encode: 4099 x 12288 fp32 38 us (6.6 TB/s), bf16 27 us (5.6 TB/s);
//   residual_norm: 8191 x 4096, all fp32 to bf16, 71 us (6.6 TB/s); all bf16 with both
//   norms, gates of each token and 8-bit outputs 52 us (5.8 TB/s; reductions one behind
//   the other, 46 % of the warps); one token 2.0 us. The same of 65536 x 512, a warp a
//   row, 48 us (6.3 TB/s). Rows of more than 8192 channels fill an SM with one CTA:
//   2048 x 12288, the same, 56 us (4.0 TB/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "f32x2.cuh"
#include "fp8.cuh"
#include "fp8.h"
#include "stream.cuh"

namespace bqd {

namespace {

constexpr int kRun = 8;                   // consecutive elements of a lane
constexpr int kRuns = 2;                  // of them in a block, half a block apart
constexpr int kLanes = 128 / kRun / kRuns;
constexpr int kEncThreads = 256;

// Eight elements as they come, and as fp32 pairs.
template <bool F32>
struct Raw8 {
    uint4 v[F32 ? 2 : 1];
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (uint4& p : v) p = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void load(const void* p)
    {
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i) v[i] = __ldcs(static_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void get(uint64_t (&x)[4]) const
    {
        if constexpr (F32) {
            x[0] = pack(__uint_as_float(v[0].x), __uint_as_float(v[0].y));
            x[1] = pack(__uint_as_float(v[0].z), __uint_as_float(v[0].w));
            x[2] = pack(__uint_as_float(v[1].x), __uint_as_float(v[1].y));
            x[3] = pack(__uint_as_float(v[1].z), __uint_as_float(v[1].w));
        } else {
            x[0] = pack(bf16_lo(v[0].x), bf16_hi(v[0].x));
            x[1] = pack(bf16_lo(v[0].y), bf16_hi(v[0].y));
            x[2] = pack(bf16_lo(v[0].z), bf16_hi(v[0].z));
            x[3] = pack(bf16_lo(v[0].w), bf16_hi(v[0].w));
        }
    }
};

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
        float* p = static_cast<float*>(base) + at;
        if ((reinterpret_cast<uintptr_t>(base) & 31u) == 0) {  // rows are whole multiples of 64 bytes: a sector at once
            asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0]), "f"(f[1]), "f"(f[2]),
                         "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                         : "memory");
        } else {
            reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
            reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
        }
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) =
            make_uint4(bf16_pair(v[0]), bf16_pair(v[1]), bf16_pair(v[2]), bf16_pair(v[3]));
    }
}

// The scale of a block from its lanes' elements.
__device__ __forceinline__ float lanes_scale(const uint64_t (&v)[kRuns][4])
{
    float m = 0.f;
#pragma unroll
    for (int r = 0; r < kRuns; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            unpack(v[r][i], a, b);
            m = max_abs(m, a, b);
        }
#pragma unroll
    for (int d = kLanes / 2; d; d >>= 1) m = max_abs(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    return block_scale(m);
}

// A lane's codes of a block: p at the first of its channels in the first half.
__device__ __forceinline__ void store_codes(uint8_t* p, uint64_t (&v)[kRuns][4], float scale, bool lo, bool hi)
{
    uint64_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = v[i / 4][i % 4];
    const uint32_t x = scale_down(w, scale);
    if (lo) *reinterpret_cast<uint2*>(p) = make_uint2(e4m3x4(w[0], w[1], x), e4m3x4(w[2], w[3], x));
    if (hi) *reinterpret_cast<uint2*>(p + 64) = make_uint2(e4m3x4(w[4], w[5], x), e4m3x4(w[6], w[7], x));
}

template <bool F32>
__global__ void __launch_bounds__(kEncThreads) encode_x_kernel(const EncodeXArgs a, uint32_t blocks, uint64_t groups)
{
    constexpr int N = F32 ? 2 : 4;  // tokens of a group of lanes: 128 bytes of a thread's loads on their way
    const uint64_t g = (static_cast<uint64_t>(blockIdx.x) * kEncThreads + threadIdx.x) / kLanes;
    const int lane = threadIdx.x % kLanes;
    const uint64_t gc = g < groups ? g : groups - 1;  // lanes of a warp stay together
    const uint64_t tg = groups < 0xFFFFFFFFull ? static_cast<uint32_t>(gc) / blocks : gc / blocks;
    const uint32_t kb = static_cast<uint32_t>(gc - tg * blocks);
    const int64_t k = static_cast<int64_t>(kb) * 128 + lane * kRun, t0 = static_cast<int64_t>(tg) * N;
    const bool lo = g < groups && k < a.K, hi = g < groups && k + 64 < a.K;  // K is a multiple of 16
    fp8_pdl_wait();
    Raw8<F32> v[N][kRuns];
    constexpr int kSize = F32 ? 4 : 2;
    const uint8_t* x = static_cast<const uint8_t*>(a.x) + (t0 * a.pitch + k) * kSize;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i][0].zero();
        v[i][1].zero();
        if (t0 + i < a.T) {
            if (lo) v[i][0].load(x);
            if (hi) v[i][1].load(x + 64 * kSize);
        }
        x += a.pitch * kSize;
    }
    fp8_pdl_trigger();
    uint8_t* codes = a.codes + t0 * a.K + k;
    float* scales = a.scales + static_cast<int64_t>(kb) * a.T + t0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        uint64_t e[kRuns][4];
        v[i][0].get(e[0]);
        v[i][1].get(e[1]);
        const float s = lanes_scale(e);
        if (t0 + i < a.T) {
            store_codes(codes, e, s, lo, hi);
            if (lane == 0 && lo) scales[i] = s;
        }
        codes += a.K;
    }
}

// A row's blocks of 128 channels take eight lanes each, VPT blocks a lane: a warp
// (rows of at most 512 channels, eight to a CTA), or a CTA of as many warps as
// the row needs. All of a row's loads are on their way together, and the rows of
// an SM's other CTAs stand for those to come. Reads are marked as used once, so
// that the L2 keeps what was written: with reads by cp.async, which cannot say so,
// rows of fp32 took 110 us where these take 71 (8191 x 4096).
constexpr int kWarpRows = 8;
constexpr int kMostThreads = 512;

// Sum over a row's threads, the same in all of them; buf: a place for each of the
// CTA's warps.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* buf)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    if constexpr (!WARP) {
        if (threadIdx.x % kWarp == 0) buf[threadIdx.x / kWarp] = v;
        __syncthreads();
        v = 0.f;
        const int warps = static_cast<int>(blockDim.x) / kWarp;
#pragma unroll
        for (int i = 0; i < kMostThreads / kWarp; ++i)
            if (i < warps) v += buf[i];
    }
    return v;
}

// A thread's runs of eight elements as they come.
template <bool F32, int N>
struct Runs {
    Raw8<F32> v[N];
    __device__ __forceinline__ void load(const void* base, int64_t row, const uint32_t (&e)[N], const bool (&in)[N])
    {
        using T = typename std::conditional<F32, float, uint16_t>::type;
        const T* p = static_cast<const T*>(base) + row;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            v[n].zero();
            if (in[n]) v[n].load(p + e[n]);
        }
    }
    __device__ __forceinline__ void get(uint64_t (&x)[N][4]) const
    {
#pragma unroll
        for (int n = 0; n < N; ++n) v[n].get(x[n]);
    }
};
// Eight weights; of a run past the row's end zeros, with which its zeros stay zeros: another channel's weight may be
// no number, and would spoil the row's sum and its last block.
__device__ __forceinline__ void weight8(const float* p, bool in, uint64_t (&v)[4])
{
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    if (in) {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    v[0] = pack(a.x, a.y);
    v[1] = pack(a.z, a.w);
    v[2] = pack(b.x, b.y);
    v[3] = pack(b.z, b.w);
}
template <int N>
__device__ __forceinline__ float squares(const uint64_t (&v)[N][4])
{
    uint64_t ss[2] = {0, 0};
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) ss[j & 1] = fma2(v[n][j], v[n][j], ss[j & 1]);
    float a, b;
    unpack(add2(ss[0], ss[1]), a, b);
    return a + b;
}

template <bool WARP, int VPT, int MOST, int CTAS, bool XF, bool RF>
__global__ void __launch_bounds__(MOST, CTAS) residual_norm_kernel(const NormArgs a)
{
    constexpr int R = WARP ? kWarpRows : 1, N = VPT * kRuns;
    __shared__ float buf[2][kMostThreads / kWarp];  // a norm's each
    const int i = WARP ? threadIdx.x % kWarp : threadIdx.x, tpr = WARP ? kWarp : static_cast<int>(blockDim.x);
    const int64_t t = static_cast<int64_t>(blockIdx.x) * R + (WARP ? threadIdx.x / kWarp : 0), at0 = t * a.H;
    // first channel of each run, and whether there is one
    uint32_t e[N];
    bool in[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        e[n] = static_cast<uint32_t>((n / kRuns * (tpr / kLanes) + i / kLanes) * 128 + n % kRuns * 64 + i % kLanes * kRun);
        in[n] = t < a.T && e[n] < static_cast<uint32_t>(a.H);
    }
    fp8_pdl_wait();
    Runs<XF, N> xv;
    Runs<RF, N> rv;
    Runs<false, N> gv;
    if (a.x) xv.load(a.x, t * a.x_pitch, e, in);
    if (a.residual) rv.load(a.residual, at0, e, in);
    if (a.gate && !a.gate_f32) gv.load(a.gate, t * a.gate_pitch, e, in);
    fp8_pdl_trigger();
    const float inv_h = 1.f / static_cast<float>(a.H);
    uint64_t r[N][4];
    if (a.residual) {
        rv.get(r);
    } else {
#pragma unroll
        for (int n = 0; n < N; ++n) r[n][0] = r[n][1] = r[n][2] = r[n][3] = 0;
    }
    if (a.x) {
        uint64_t z[N][4];
        xv.get(z);
        if (a.post_weight) {
            const float rs = rsqrtf(__fmaf_rn(row_sum<WARP>(squares(z), buf[0]), inv_h, a.eps));
            const uint64_t rs2 = pack(rs, rs);
#pragma unroll
            for (int n = 0; n < N; ++n) {
                uint64_t w[4];
                weight8(a.post_weight + e[n], in[n], w);
#pragma unroll
                for (int j = 0; j < 4; ++j) z[n][j] = mul2(mul2(z[n][j], rs2), w[j]);
            }
        }
        if (a.gate) {
            uint64_t w[N][4];
            if (a.gate_f32) {  // the rarer type is loaded where it is used
                Runs<true, N> gf;
                gf.load(a.gate, t * a.gate_pitch, e, in);
                gf.get(w);
            } else {
                gv.get(w);
            }
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) z[n][j] = mul2(z[n][j], w[n][j]);
        }
        const uint64_t sc = pack(a.scale, a.scale);
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) r[n][j] = fma2(z[n][j], sc, r[n][j]);
    }
    if (a.residual_out) {
#pragma unroll
        for (int n = 0; n < N; ++n)
            if (in[n]) store8(a.residual_out, at0 + e[n], RF, r[n]);
    }
    if (!a.y) return;
    const float rs = rsqrtf(__fmaf_rn(row_sum<WARP>(squares(r), buf[1]), inv_h, a.eps));
    const uint64_t rs2 = pack(rs, rs);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        uint64_t w[4];
        weight8(a.pre_weight + e[n], in[n], w);
#pragma unroll
        for (int j = 0; j < 4; ++j) r[n][j] = mul2(mul2(r[n][j], rs2), w[j]);
    }
    if (a.y_e4m3) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int n = v * kRuns;
            uint64_t(&b)[kRuns][4] = *reinterpret_cast<uint64_t(*)[kRuns][4]>(&r[n]);
            const float s = lanes_scale(b);  // every lane takes part; those past H hold zeros
            store_codes(static_cast<uint8_t*>(a.y) + at0 + e[n], b, s, in[n], in[n + 1]);
            if (in[n] && i % kLanes == 0) a.y_scales[static_cast<int64_t>(e[n] / 128) * a.T + t] = s;
        }
    } else {
#pragma unroll
        for (int n = 0; n < N; ++n)
            if (in[n]) store8(a.y, at0 + e[n], false, r[n]);
    }
}

// Launches that may begin while the kernel before them ends: each waits for it
// ahead of its first access to memory.
template <typename... A>
cudaError_t launch_after(void (*kern)(A...), unsigned grid, int threads, size_t smem, cudaStream_t s, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <bool WARP, int VPT, int MOST, int CTAS, bool XF, bool RF>
cudaError_t launch_norm_of(const NormArgs& a, cudaStream_t s)
{
    constexpr int R = WARP ? kWarpRows : 1;
    const int lanes = ((a.H + 127) / 128 + VPT - 1) / VPT * kLanes;
    const int threads = WARP ? MOST : (lanes + kWarp - 1) / kWarp * kWarp;
    return launch_after(residual_norm_kernel<WARP, VPT, MOST, CTAS, XF, RF>, static_cast<unsigned>((a.T + R - 1) / R), threads, 0, s, a);
}

template <bool WARP, int VPT, int MOST, int CTAS>
cudaError_t launch_norm(const NormArgs& a, cudaStream_t s)
{
    if (a.x_f32)
        return a.res_f32 ? launch_norm_of<WARP, VPT, MOST, CTAS, true, true>(a, s)
                         : launch_norm_of<WARP, VPT, MOST, CTAS, true, false>(a, s);
    return a.res_f32 ? launch_norm_of<WARP, VPT, MOST, CTAS, false, true>(a, s)
                     : launch_norm_of<WARP, VPT, MOST, CTAS, false, false>(a, s);
}

}  // namespace

cudaError_t launch_fp8_x_encode(const EncodeXArgs& a, int x_type, cudaStream_t s)
{
    const uint64_t blocks = static_cast<uint64_t>((a.K + 127) / 128), tokens = x_type == BQD_F32 ? 2 : 4;
    const uint64_t groups = blocks * ((static_cast<uint64_t>(a.T) + tokens - 1) / tokens);
    const uint64_t per = kEncThreads / kLanes, ctas = (groups + per - 1) / per;
    if (ctas > 0x7FFFFFFFull) return cudaErrorInvalidValue;
    return launch_after(x_type == BQD_F32 ? encode_x_kernel<true> : encode_x_kernel<false>, static_cast<unsigned>(ctas),
                        kEncThreads, 0, s, a, static_cast<uint32_t>(blocks), groups);
}

cudaError_t launch_residual_norm(const NormArgs& a, cudaStream_t s)
{
    if (a.H <= 512) return launch_norm<true, 1, 256, 4>(a, s);
    if (a.H <= 4096) return launch_norm<false, 1, 256, 4>(a, s);
    if (a.H <= 8192) return launch_norm<false, 1, 512, 2>(a, s);
    return launch_norm<false, 2, 512, 1>(a, s);  // to kNormMaxH
}

}  // namespace bqd
