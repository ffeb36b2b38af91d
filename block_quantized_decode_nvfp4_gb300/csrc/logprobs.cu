// logprobs.cu -- log probability of given tokens, entropy and the top
// alternatives of logits rows, in one pass over the logits.
//
// With m = max x, z = sum e^(x - m), u = sum e^(x - m) (x - m):
//   lse = m + log z, logprob = x_tok - lse, entropy = log z - u / z,
// and two partial results join as m = max(m1, m2), f = e^(m1 - m), z1' = f z1,
// u1' = f (u1 + z1 (m1 - m)), likewise the other, and sums. The alternatives
// are ordered by one 64-bit key per logit: the value's bits made monotonic
// (NaN lowest, -0 as +0) above the complemented index, so equal values go to
// the lower index; the k largest keys of a row are the k largest of the k
// largest of its parts.
//
// A row is shared by a cluster of C CTAs (1 to 16: one for many rows, 16 for
// a decode step's few), which join through distributed shared memory, so the
// call is one launch and needs no workspace. A CTA runs over its part in
// tiles held in registers, the next tile's loads in flight meanwhile: the
// tile's maximum, the sums, and a compare with the k-th best value so far,
// tau; what passes goes to a list in shared memory, which is cut back to the
// k best (each entry counts the larger ones) when it has grown. The first
// tile's tau is a bound: with q = ceil(k / warps), the smallest over the
// warps of the q-th largest of a warp's 32 lane maxima has k elements at or
// above it. Where the list overflows (a tile of equal or of NaN logits) the
// k best are taken by k rounds of a block maximum instead. After a cut, later
// logits equal to tau have higher indices and lose, so the compare is strict.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn.h"
#include "common.cuh"
#include "stream.cuh"

namespace bqd {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / kWarp;
constexpr int kElems = 16;            // logits per thread and tile
constexpr int kTile = kThreads * kElems;
constexpr int kCap = 1024;            // entries of the candidate list
constexpr int kCut = 96;              // it is cut back when it has more than topk + kCut
constexpr int kMaxK = 32;
constexpr int kMaxCluster = 16;
static_assert(kMaxCluster * kMaxK <= kThreads, "the leader gathers one key per thread");
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ uint64_t order_key(float x, uint32_t i)
{
    uint32_t b = __float_as_uint(x + 0.f);
    b = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    if (x != x) b = 0;
    return (static_cast<uint64_t>(b) << 32) | (0xFFFFFFFFu - i);
}
__device__ __forceinline__ float key_value(uint64_t key)
{
    const uint32_t b = static_cast<uint32_t>(key >> 32);
    return b == 0 ? __int_as_float(0x7FFFFFFF) : __uint_as_float((b & 0x80000000u) ? (b & 0x7FFFFFFFu) : ~b);
}
__device__ __forceinline__ uint64_t umax64(uint64_t a, uint64_t b) { return a > b ? a : b; }

// Maximum that is NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

struct Sums {
    float m, z, u;
};

__device__ __forceinline__ void raise(Sums& s, float m)  // s relative to m >= s.m
{
    if (s.m != -INFINITY) {
        const float d = s.m - m, f = ex2(d * kLog2e);
        s.u = d < -150.f ? 0.f : (s.u + s.z * d) * f;
        s.z *= f;
    }
    s.m = m;
}
__device__ __forceinline__ Sums join(Sums a, Sums b)
{
    const float m = max_nan(a.m, b.m);
    raise(a, m);
    raise(b, m);
    return {m, a.z + b.z, a.u + b.u};
}

// A 16-byte window of the row: elements first .. first + N - 1, those outside
// [0, V) as -inf. Windows lie on 16-byte boundaries; only the row's first and
// last may be partial, and those are read element by element.
template <typename T>
struct Window {
    static constexpr int kN = 16 / static_cast<int>(sizeof(T));
    static __device__ __forceinline__ uint4 load(const T* x, int64_t first, int V)
    {
        if (first >= 0 && first + kN <= V) return __ldcs(reinterpret_cast<const uint4*>(x + first));
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;
        if (first < V && first + kN > 0) {
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                const int64_t i = first + e;
                if (i < 0 || i >= V) continue;
                if constexpr (sizeof(T) == 4) {
                    w[e] = reinterpret_cast<const uint32_t*>(x)[i];
                } else {
                    const uint32_t b = reinterpret_cast<const uint16_t*>(x)[i];
                    w[e / 2] = (e & 1) ? (w[e / 2] & 0xFFFFu) | (b << 16) : (w[e / 2] & 0xFFFF0000u) | b;
                }
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ float get(const uint4& v, int e)
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
        return (e & 1) ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
    }
};

struct Shared {
    uint64_t cand[kCap + 2];  // candidates; +2: a list is padded to whole 16-byte reads
    uint64_t top[kMaxK];      // this CTA's best, descending
    uint64_t best[kWarps];
    Sums sums[kWarps];
    Sums total;
    uint32_t bound[kWarps];
    int count[2];             // candidates added in even and odd tiles
    int ntop;
};

// The k best of cand[0, c) in descending order to top[]; c <= kCap. Barriers
// before (the list is complete) and after (top is) are inside.
__device__ __forceinline__ void cut(Shared& s, int c, int k)
{
    __syncthreads();
    if (threadIdx.x < 2) s.cand[c + threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < c; i += kThreads) {
        const uint64_t mine = s.cand[i];
        int r = 0;
        for (int j = 0; j < c; j += 2) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&s.cand[j]);
            r += (v.x > mine) + (v.y > mine);
        }
        if (r < k && mine != 0) s.top[r] = mine;
    }
    __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) logprobs_kernel(const LogprobArgs a, int C)
{
    using W = Window<T>;
    constexpr int NW = kElems / W::kN;  // windows per thread and tile
    __shared__ __align__(16) Shared s;
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    const int64_t t = blockIdx.x / C;
    const int rank = static_cast<int>(blockIdx.x % C), k = a.topk, V = a.V;
    const T* x = static_cast<const T*>(a.x) + t * a.pitch;
    // windows of the row: `pre` elements of the first lie before the row
    const int pre = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
    const int64_t windows = (static_cast<int64_t>(pre) + V + W::kN - 1) / W::kN, share = (windows + C - 1) / C;
    const int64_t w0 = share * rank, w1 = min(w0 + share, windows);

    if (threadIdx.x < 2) s.count[threadIdx.x] = 0;
    if (threadIdx.x == 0) s.ntop = 0;
    Sums sum{-INFINITY, 0.f, 0.f};
    float tau = -INFINITY;
    bool strict = false;
    int have = 0, par = 0;  // entries of the list (known to all threads), tile parity

    auto first_of = [&](int64_t w) { return w * W::kN - pre; };
    uint4 next[NW];
    auto fetch = [&](int64_t w) {
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            const int64_t i = w + j * kThreads + threadIdx.x;
            next[j] = W::load(x, i < w1 ? first_of(i) : V, V);
        }
    };
    if (w0 < w1) fetch(w0);
    __syncthreads();
    for (int64_t w = w0; w < w1; w += kThreads * NW, par ^= 1) {
        uint4 cur[NW];
#pragma unroll
        for (int j = 0; j < NW; ++j) cur[j] = next[j];
        if (w + kThreads * NW < w1) fetch(w + kThreads * NW);

        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < NW; ++j)
#pragma unroll
            for (int e = 0; e < W::kN; ++e) top = max_nan(top, W::get(cur[j], e));
        if (!(top <= sum.m)) raise(sum, top);
        const float m = sum.m == -INFINITY ? 0.f : sum.m;
#pragma unroll
        for (int j = 0; j < NW; ++j)
#pragma unroll
            for (int e = 0; e < W::kN; ++e) {
                // -150: e^-150 is 0 in fp32, and 0 * -inf is not
                const float d = fmaxf(W::get(cur[j], e) - m, -150.f), p = ex2(d * kLog2e);
                sum.z += p;
                sum.u += p * d;
            }
        if (k == 0) continue;

        if (w == w0) {
            uint32_t b = static_cast<uint32_t>(order_key(top, 0) >> 32);
            uint32_t best = __reduce_max_sync(0xFFFFFFFFu, b);
            if (k > kWarps) {  // the second largest lane maximum
                const int at = __ffs(__ballot_sync(0xFFFFFFFFu, b == best)) - 1;
                best = __reduce_max_sync(0xFFFFFFFFu, lane == at ? 0u : b);
            }
            if (lane == 0) s.bound[warp] = best;
            __syncthreads();
            uint32_t least = s.bound[lane % kWarps];
            least = __reduce_min_sync(0xFFFFFFFFu, least);
            tau = least == 0 ? -INFINITY : key_value(static_cast<uint64_t>(least) << 32);
        }
        if (strict ? !(top <= tau) : !(top < tau)) {
#pragma unroll
            for (int j = 0; j < NW; ++j) {
                const int64_t i0 = first_of(w + j * kThreads + threadIdx.x);
#pragma unroll
                for (int e = 0; e < W::kN; ++e) {
                    const float v = W::get(cur[j], e);
                    const int64_t i = i0 + e;
                    if ((strict ? !(v <= tau) : !(v < tau)) && i >= 0 && i < V && w + j * kThreads + threadIdx.x < w1) {
                        const int p = have + atomicAdd(&s.count[par], 1);
                        if (p < kCap) s.cand[p] = order_key(v, static_cast<uint32_t>(i));
                    }
                }
            }
        }
        __syncthreads();
        const int c = have + s.count[par];
        if (threadIdx.x == 0) s.count[par ^ 1] = 0;  // read by all before this tile's barrier
        if (c > kCap) {
            // the list and this tile by rounds of a block maximum
            uint64_t last = ~uint64_t(0);
            int n = 0;
            for (; n < k; ++n) {
                uint64_t b = 0;
#pragma unroll
                for (int j = 0; j < NW; ++j) {
                    const int64_t i0 = first_of(w + j * kThreads + threadIdx.x);
#pragma unroll
                    for (int e = 0; e < W::kN; ++e) {
                        const int64_t i = i0 + e;
                        const uint64_t key = order_key(W::get(cur[j], e), static_cast<uint32_t>(i));
                        if (i >= 0 && i < V && w + j * kThreads + threadIdx.x < w1 && key < last) b = umax64(b, key);
                    }
                }
                for (int i = threadIdx.x; i < have; i += kThreads)
                    if (s.cand[i] < last) b = umax64(b, s.cand[i]);
#pragma unroll
                for (int d = 16; d; d >>= 1) b = umax64(b, __shfl_xor_sync(0xFFFFFFFFu, b, d));
                if (lane == 0) s.best[warp] = b;
                __syncthreads();
                for (int i = 0; i < kWarps; ++i) b = umax64(b, s.best[i]);
                __syncthreads();
                if (b == 0) break;
                last = b;
                if (threadIdx.x == 0) s.top[n] = b;
            }
            __syncthreads();
            if (threadIdx.x < n) s.cand[threadIdx.x] = s.top[threadIdx.x];
            have = n;
        } else if (c > k + kCut) {
            cut(s, c, k);
            if (threadIdx.x < k) s.cand[threadIdx.x] = s.top[threadIdx.x];
            have = k;
        } else {
            have = c;
            continue;
        }
        if (have == k) {
            tau = key_value(s.top[k - 1]);
            strict = true;
            if (tau != tau) {  // NaN among the best: everything else passes
                tau = -INFINITY;
                strict = false;
            }
        }
        __syncthreads();  // cand and tau are in place before the next tile adds to the list
    }
    if (k > 0) {
        cut(s, have, k);
        if (threadIdx.x == 0) s.ntop = min(have, k);
    }
    // the block's sums
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const Sums o{__shfl_xor_sync(0xFFFFFFFFu, sum.m, d), __shfl_xor_sync(0xFFFFFFFFu, sum.z, d),
                     __shfl_xor_sync(0xFFFFFFFFu, sum.u, d)};
        sum = (lane & d) ? join(o, sum) : join(sum, o);
    }
    if (lane == 0) s.sums[warp] = sum;
    __syncthreads();
    if (warp == 0) {
        sum = s.sums[lane % kWarps];
#pragma unroll
        for (int d = kWarps / 2; d; d >>= 1) {
            const Sums o{__shfl_xor_sync(0xFFFFFFFFu, sum.m, d), __shfl_xor_sync(0xFFFFFFFFu, sum.z, d),
                         __shfl_xor_sync(0xFFFFFFFFu, sum.u, d)};
            sum = (lane & d) ? join(o, sum) : join(sum, o);
        }
        if (lane == 0) s.total = sum;
    }
    // the cluster's: its first CTA gathers every CTA's sums and best
    int n = 0;
    if (C > 1) {
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        uint64_t key = 0;
        if (rank == 0) {
            auto remote = [&](const void* p, int r) {
                uint32_t at;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(r));
                return at;
            };
            const int r = threadIdx.x / kMaxK, l = threadIdx.x % kMaxK;
            if (r < C && k > 0) {
                int nt;
                asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(nt) : "r"(remote(&s.ntop, r)) : "memory");
                if (l < nt)
                    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(key) : "r"(remote(&s.top[l], r)) : "memory");
            }
            if (warp == 0) {
                Sums o{-INFINITY, 0.f, 0.f};
                if (lane < C) {
                    const uint32_t at = remote(&s.total, lane);
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o.m) : "r"(at) : "memory");
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o.z) : "r"(at + 4) : "memory");
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o.u) : "r"(at + 8) : "memory");
                }
#pragma unroll
                for (int d = kMaxCluster / 2; d; d >>= 1) {
                    const Sums p{__shfl_xor_sync(0xFFFFFFFFu, o.m, d), __shfl_xor_sync(0xFFFFFFFFu, o.z, d),
                                 __shfl_xor_sync(0xFFFFFFFFu, o.u, d)};
                    o = (lane & d) ? join(p, o) : join(o, p);
                }
                sum = o;
            }
        }
        // the others' shared memory is read no more
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (rank != 0) return;
        if (warp == 0 && lane == 0) s.total = sum;
        if (k > 0) {
            s.cand[threadIdx.x] = key;
            cut(s, C * kMaxK, k);
        }
    }
    __syncthreads();
    (void)n;
    sum = s.total;
    if (sum.m == INFINITY) sum.z = sum.m - sum.m;  // +inf among the logits: NaN
    const float lse = sum.z == 0.f ? INFINITY : sum.m + logf(sum.z);  // an empty row: every log probability is -inf
    if (threadIdx.x == 0) {
        if (a.logprob) {
            const int tok = a.tokens[t];
            float v = -INFINITY;
            if (tok >= 0 && tok < V) {
                if constexpr (sizeof(T) == 4)
                    v = x[tok] - lse;
                else
                    v = __bfloat162float(x[tok]) - lse;
            }
            a.logprob[t] = v;
        }
        if (a.entropy) a.entropy[t] = sum.z == 0.f ? 0.f : logf(sum.z) - sum.u / sum.z;
    }
    if (threadIdx.x < k) {
        const uint64_t key = s.top[threadIdx.x];
        a.top_ids[t * k + threadIdx.x] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(key));
        a.top_logprobs[t * k + threadIdx.x] = key_value(key) - lse;
    }
}

template <typename T>
cudaError_t launch(const LogprobArgs& a, cudaStream_t s)
{
    static const cudaError_t wide =
        cudaFuncSetAttribute(logprobs_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (wide != cudaSuccess) return wide;
    // CTAs per row: as many as fill the GPU once (two CTAs per SM), while
    // each still has a tile's worth of the row.
    int C = 1;
    while (C < kMaxCluster && a.T * C * 2 <= 2 * 152 && a.V / (C * 2) >= kTile) C *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.T * C));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = static_cast<unsigned>(C);
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<T>, a, C);
}

}  // namespace

size_t token_logprobs_ws(int64_t, int64_t, int) { return 16; }

cudaError_t launch_token_logprobs(const LogprobArgs& a, int in_type, cudaStream_t s)
{
    return in_type == BQD_F32 ? launch<float>(a, s) : launch<__nv_bfloat16>(a, s);
}

}  // namespace bqd
