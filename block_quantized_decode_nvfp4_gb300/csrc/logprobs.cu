// logprobs.cu -- log probability of given tokens, entropy and the top
// alternatives of logits rows.
//
// With m = max x, z = sum e^(x - m), u = sum e^(x - m) (x - m):
//   lse = m + log z, logprob = x_tok - lse, entropy = log z - u / z.
// Alternatives are ordered by one 64-bit key per logit: the value's bits made
// monotonic (NaN lowest, -0 as +0) above the complemented index, so equal
// values go to the lower index.
//
// Simple form: one CTA per row; one pass for m, one for z and u, and one per
// alternative for the largest key below the last.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn.h"
#include "common.cuh"

namespace bqd {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / kWarp;

__device__ __forceinline__ float logit(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float logit(const __nv_bfloat16* p, int64_t i) { return __bfloat162float(p[i]); }

__device__ __forceinline__ uint64_t order_key(float x, uint32_t i)
{
    uint32_t b = __float_as_uint(x + 0.f);
    b = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    if (x != x) b = 0;
    return (static_cast<uint64_t>(b) << 32) | (0xFFFFFFFFu - i);
}

__device__ __forceinline__ uint64_t umax64(uint64_t a, uint64_t b) { return a > b ? a : b; }

template <typename T>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LogprobArgs a)
{
    __shared__ float s_f[kWarps], s_g[kWarps];
    __shared__ uint64_t s_k[kWarps];
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    const int64_t t = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + t * a.pitch;
    float m = -INFINITY;
    for (int i = threadIdx.x; i < a.V; i += kThreads) m = fmaxf(m, logit(x, i));
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    if (lane == 0) s_f[warp] = m;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_f[w]);
    __syncthreads();
    float z = 0.f, u = 0.f;
    if (m != -INFINITY) {
        for (int i = threadIdx.x; i < a.V; i += kThreads) {
            const float d = logit(x, i) - m, e = expf(d);
            z += e;
            if (e != 0.f) u += e * d;
        }
    } else {  // -inf throughout, or NaN among it
        for (int i = threadIdx.x; i < a.V; i += kThreads) {
            const float v = logit(x, i);
            if (v != v) z = v;
        }
    }
    z = warp_sum(z);
    u = warp_sum(u);
    if (lane == 0) {
        s_f[warp] = z;
        s_g[warp] = u;
    }
    __syncthreads();
    z = u = 0.f;
    for (int w = 0; w < kWarps; ++w) {
        z += s_f[w];
        u += s_g[w];
    }
    const float lse = z == 0.f ? INFINITY : m + logf(z);  // an empty row: every log probability is -inf
    if (threadIdx.x == 0) {
        if (a.logprob) {
            const int tok = a.tokens[t];
            a.logprob[t] = tok >= 0 && tok < a.V ? logit(x, tok) - lse : -INFINITY;
        }
        if (a.entropy) a.entropy[t] = z == 0.f ? 0.f : logf(z) - u / z;
    }
    uint64_t last = ~uint64_t(0);
    for (int k = 0; k < a.topk; ++k) {
        uint64_t best = 0;
        for (int i = threadIdx.x; i < a.V; i += kThreads) {
            const uint64_t key = order_key(logit(x, i), i);
            if (key < last) best = umax64(best, key);
        }
        for (int d = 16; d; d >>= 1) best = umax64(best, __shfl_xor_sync(0xFFFFFFFFu, best, d));
        __syncthreads();
        if (lane == 0) s_k[warp] = best;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) best = umax64(best, s_k[w]);
        last = best;
        if (threadIdx.x == 0) {
            const int i = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(best));
            a.top_ids[t * a.topk + k] = i;
            a.top_logprobs[t * a.topk + k] = logit(x, i) - lse;
        }
    }
}

}  // namespace

size_t token_logprobs_ws(int64_t, int64_t, int) { return 16; }

cudaError_t launch_token_logprobs(const LogprobArgs& a, int in_type, cudaStream_t s)
{
    if (in_type == BQD_F32)
        logprobs_kernel<float><<<static_cast<unsigned>(a.T), kThreads, 0, s>>>(a);
    else
        logprobs_kernel<__nv_bfloat16><<<static_cast<unsigned>(a.T), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace bqd
