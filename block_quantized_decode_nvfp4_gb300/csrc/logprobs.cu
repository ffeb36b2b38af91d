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
// call is one launch and needs no workspace. The row's whole 16-byte windows
// come through a ring of 32 KiB bulk copies (three stages, two CTAs per SM:
// 128 KiB and more in flight per SM); its ragged ends, at most 14 logits, are
// read one by one. The warps run through the ring without a barrier of the
// CTA. A tile costs its maximum, the sums (two logits an instruction where
// there is a packed form) and a compare of the thread's maximum with tau.
//
// Alternatives. The k-th largest of the maxima that the CTA's 32 half-warps
// have seen has k logits at or above it: that is tau, published in shared
// memory after the first tile and again by every warp that meets a logit at
// or above it (the maxima only grow, so an older one is a bound too). What
// passes goes to the warp's own list of up to 64 keys; one that has grown past
// 32 is cut back to its k best (each entry counts the larger ones), and as a
// warp's logits come in ascending tiles, those of later tiles have to exceed
// its k-th from then on. About k (1 + log(tiles)) logits pass in a row of
// distinct logits; rows of equal ones cost a few cuts in their first tile. At
// the end the lists are joined, first the CTA's, then the cluster's, by the
// same count.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "attn.h"
#include "common.cuh"
#include "f32x2.cuh"
#include "host_util.h"
#include "stream.cuh"

namespace bqd {

// Device error word (kErrWaitTimeout); read and cleared by
// read_and_clear_logprobs_error().
__device__ unsigned int g_logprobs_error = 0;

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / kWarp;
constexpr int kPer = 4;                             // windows per thread and tile
constexpr int kTileWindows = kThreads * kPer;
constexpr int kTileBytes = kTileWindows * 16;
constexpr int kStages = 3;
constexpr int kList = 64;                           // entries of a warp's list
constexpr int kMaxK = 32;
constexpr int kMaxCluster = 16;
static_assert(kMaxCluster * kMaxK <= kThreads, "the leader takes one key per thread");
static_assert(2 * kWarps == kWarp, "a warp ranks the half-warps' maxima, one per lane");
static_assert(kList == 2 * kWarp && kMaxK <= kWarp, "a cut handles two keys per lane, and leaves room for a ballot");
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ uint64_t order_key(float x, uint32_t i)
{
    uint32_t b = __float_as_uint(x + 0.f);
    b = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    if (x != x) b = 0;
    return (static_cast<uint64_t>(b) << 32) | (0xFFFFFFFFu - i);
}
// The value of a key's upper half; NaN for that of NaN.
__device__ __forceinline__ float ordered_value(uint32_t b)
{
    return b == 0 ? __int_as_float(0x7FFFFFFF) : __uint_as_float((b & 0x80000000u) ? (b & 0x7FFFFFFFu) : ~b);
}

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

// A thread's kPer 16-byte windows of a tile.
template <typename T>
struct Chunk {
    static constexpr int kN = 16 / static_cast<int>(sizeof(T));  // logits per window
    uint32_t w[kPer][4];

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int j = 0; j < kPer; ++j) clear(j);
    }
    __device__ __forceinline__ void clear(int j)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[j][i] = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;  // -inf
    }
    __device__ __forceinline__ void load(int j, uint32_t at)
    {
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[j][0]), "=r"(w[j][1]), "=r"(w[j][2]), "=r"(w[j][3])
                     : "r"(at)
                     : "memory");
    }
    __device__ __forceinline__ float get(int j, int e) const
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[j][e]);
        return (e & 1) ? bf16_hi(w[j][e / 2]) : bf16_lo(w[j][e / 2]);
    }
    __device__ __forceinline__ float top() const  // NaN if there is one
    {
        if constexpr (sizeof(T) == 4) {
            float m = -INFINITY;
#pragma unroll
            for (int j = 0; j < kPer; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) m = max_nan(m, __uint_as_float(w[j][e]));
            return m;
        } else {
            __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&w[0][0]);
#pragma unroll
            for (int j = 0; j < kPer; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) m = __hmax2_nan(m, *reinterpret_cast<const __nv_bfloat162*>(&w[j][e]));
            return max_nan(__low2float(m), __high2float(m));
        }
    }
    // z += sum e^(x - m), u += sum e^(x - m) (x - m). Between -1e29 and 1e29
    // of m, logits below -1e30 (-inf, and masks by the type's lowest value)
    // count as -1e30: their e^(x - m) is 0 either way, and x - m stays finite.
    __device__ __forceinline__ void add(float m, float& z, float& u) const
    {
        if (fabsf(m) < 1e29f) {
            const uint64_t mm = pack(-m, -m), l2 = pack(kLog2e, kLog2e);
            uint64_t zz = 0, uu = 0;
            const __nv_bfloat162 low = __float2bfloat162_rn(-1e30f);
#pragma unroll
            for (int j = 0; j < kPer; ++j)
#pragma unroll
                for (int e = 0; e < kN; e += 2) {
                    uint64_t x;
                    if constexpr (sizeof(T) == 4) {
                        x = pack(fmaxf(__uint_as_float(w[j][e]), -1e30f), fmaxf(__uint_as_float(w[j][e + 1]), -1e30f));
                    } else {
                        const __nv_bfloat162 b = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&w[j][e / 2]), low);
                        const uint32_t v = *reinterpret_cast<const uint32_t*>(&b);
                        x = pack(bf16_lo(v), bf16_hi(v));
                    }
                    const uint64_t d = add2(x, mm);
                    float a, b;
                    unpack(mul2(d, l2), a, b);
                    const uint64_t p = pack(ex2(a), ex2(b));
                    zz = add2(zz, p);
                    uu = fma2(p, d, uu);
                }
            float a, b;
            unpack(zz, a, b);
            z += a + b;
            unpack(uu, a, b);
            u += a + b;
        } else {
            const float mm = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int j = 0; j < kPer; ++j)
#pragma unroll
                for (int e = 0; e < kN; ++e) {
                    // -150: e^-150 is 0 in fp32, and 0 * -inf is not
                    const float d = fmaxf(get(j, e) - mm, -150.f), p = ex2(d * kLog2e);
                    z += p;
                    u += p * d;
                }
        }
    }
};

struct Shared {
    uint64_t full[kStages], empty[kStages];
    alignas(16) uint64_t list[kWarps][kList];  // a warp's candidates, read 16 bytes at a time
    uint64_t top[kMaxK];                       // this CTA's best, descending
    Sums sums[kWarps];
    uint32_t bound[kWarp];                     // the half-warps' maxima, as ordered bits; 0: none above -inf
    uint32_t tau;                              // the k-th largest of them; 0: fewer than k
    int count;
    int all_n[kMaxCluster];                    // of the leader: every CTA's number of best, sums and best
    Sums all_sums[kMaxCluster];
    uint64_t all_top[kMaxCluster][kMaxK];
    uint64_t all_tau;
};
static_assert(offsetof(Shared, list) % 16 == 0 && kList % 2 == 0, "16-byte reads of the lists");

// A bound's value: everything for none.
__device__ __forceinline__ float bits_value(uint32_t b) { return b == 0 ? -INFINITY : ordered_value(b); }

// The ordered bits of a value: the upper half of its key.
__device__ __forceinline__ uint32_t order_bits(float x) { return static_cast<uint32_t>(order_key(x, 0) >> 32); }

// The k-th largest of the 32 lanes' values.
__device__ __forceinline__ uint32_t kth_of_lanes(uint32_t v, int k)
{
    const int lane = threadIdx.x % kWarp;
    int r = 0;  // how many are ahead of this lane's
#pragma unroll
    for (int l = 0; l < kWarp; ++l) {
        const uint32_t o = __shfl_sync(0xFFFFFFFFu, v, l);
        r += o > v || (o == v && l < lane);
    }
    return __shfl_sync(0xFFFFFFFFu, v, __ffs(__ballot_sync(0xFFFFFFFFu, r == k - 1)) - 1);
}

// Cuts a warp's list of n <= kList keys back to its k best, descending.
__device__ __noinline__ void cut_list(uint64_t* list, int n, int k)
{
    const int lane = threadIdx.x % kWarp;
    __syncwarp();
    const uint64_t a = lane < n ? list[lane] : 0, b = lane + kWarp < n ? list[lane + kWarp] : 0;
    int ra = 0, rb = 0;
    for (int j = 0; j < n; j += 2) {
        const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&list[j]);
        ra += (v.x > a) + (j + 1 < n && v.y > a);
        rb += (v.x > b) + (j + 1 < n && v.y > b);
    }
    __syncwarp();
    if (a && ra < k) list[ra] = a;
    if (b && rb < k) list[rb] = b;
    __syncwarp();
}

// The k best of c keys at cand (16-byte aligned, room for c + 1) in
// descending order to top. Called by the whole CTA, with a barrier before.
__device__ __forceinline__ void cut_all(uint64_t* cand, int c, uint64_t* top, int k)
{
    if (threadIdx.x == 0) cand[c] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < c; i += kThreads) {
        const uint64_t mine = cand[i];
        int r = 0;
        for (int j = 0; j < c; j += 2) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&cand[j]);
            r += (v.x > mine) + (v.y > mine);
        }
        if (r < k) top[r] = mine;
    }
    __syncthreads();
}

__device__ __forceinline__ uint32_t in_cta(const void* p, int rank)  // its counterpart in another CTA of the cluster
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) logprobs_kernel(const LogprobArgs a, int C)
{
    using K = Chunk<T>;
    constexpr int N = K::kN;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(16) Shared s;
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    const int64_t t = blockIdx.x / C;
    const int rank = static_cast<int>(blockIdx.x % C), k = a.topk, V = a.V;
    const T* x = static_cast<const T*>(a.x) + t * a.pitch;
    // 16-byte windows, counted from the one that holds the row's first logit:
    // `pre` elements of it lie before the row. Whole ones: [whole0, whole1).
    const int pre = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
    const int64_t whole0 = pre ? 1 : 0, whole1 = (static_cast<int64_t>(pre) + V) / N;
    const int64_t whole = whole1 > whole0 ? whole1 - whole0 : 0, share = (whole + C - 1) / C;
    const int64_t w0 = whole0 + min(share * rank, whole), w1 = whole0 + min(share * (rank + 1), whole);
    const int tiles = static_cast<int>((w1 - w0 + kTileWindows - 1) / kTileWindows);

    if (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    auto copy = [&](int i) {  // tile i into its stage
        const int64_t w = w0 + static_cast<int64_t>(i) * kTileWindows;
        const uint32_t bytes = static_cast<uint32_t>(min(w1 - w, static_cast<int64_t>(kTileWindows))) * 16;
        mbar_arrive_expect_tx(&s.full[i % kStages], bytes);
        bulk_g2s(ring + (i % kStages) * kTileBytes, x + (w * N - pre), bytes, &s.full[i % kStages]);
    };
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], kWarps);
        }
        fence_barrier_init();
        for (int i = 0; i < min(kStages, tiles); ++i) copy(i);
        s.count = 0;
        s.tau = 0;
        s.all_tau = 0;
    }
    Sums sum{-INFINITY, 0.f, 0.f};
    uint64_t* list = s.list[warp];
    uint32_t kth = 0;        // of the own list, as ordered bits; 0: not cut yet, or NaN
    float seen = -INFINITY;  // largest so far, of the tiles that mattered
    bool ok = true;
    int have = 0;  // entries of the own list
    if (lane % 16 == 0) s.bound[2 * warp + lane / 16] = 0;

    // the row's ends, by the first CTA's first warp, a logit per lane
    if (rank == 0 && warp == 0) {
        const int head = whole ? static_cast<int>(whole0 * N - pre) : 0;
        const int64_t tail0 = whole ? whole1 * N - pre : 0;
        const int64_t i = lane < head ? lane : tail0 + (lane - head);
        have = head + static_cast<int>(V - tail0);
        if (i < V) {
            float v;
            if constexpr (sizeof(T) == 4)
                v = x[i];
            else
                v = __bfloat162float(x[i]);
            raise(sum, v);
            sum.z = v == -INFINITY ? 0.f : v - v + 1.f;  // NaN for NaN (and for +inf)
            seen = v;
            list[lane] = order_key(v, static_cast<uint32_t>(i));
        }
    }
    __syncthreads();
    for (int i = 0; i < tiles; ++i) {
        const int64_t w = w0 + static_cast<int64_t>(i) * kTileWindows + threadIdx.x;
        if (warp == 0 && i > 0 && i - 1 + kStages < tiles) {  // tile i - 1 has been read by all: its stage again
            ok = ok && mbar_wait_warp(&s.empty[(i - 1) % kStages], static_cast<uint32_t>(((i - 1) / kStages) & 1),
                                      &g_logprobs_error);
            if (ok && lane == 0) copy(i - 1 + kStages);
        }
        ok = ok && mbar_wait_warp(&s.full[i % kStages], static_cast<uint32_t>((i / kStages) & 1), &g_logprobs_error);
        K c;
        const uint32_t at = smem_u32(ring) + (i % kStages) * kTileBytes + threadIdx.x * 16;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (w + j * kThreads < w1)
                c.load(j, at + j * kThreads * 16);
            else
                c.clear(j);
        }
        const float top = c.top();
        if (!(top <= sum.m)) raise(sum, top);
        c.add(sum.m, sum.z, sum.u);

        bool hit = k > 0;
        uint32_t tau = 0;
        volatile uint32_t* bound = s.bound;
        // the half-warps' maxima so far, and the CTA's k-th of them
        auto publish = [&] {
            seen = fmaxf(seen, top);
            const uint32_t bits = seen == -INFINITY ? 0u : order_bits(seen);  // -inf may be padding, or NaN passed over
            const uint32_t best = lane < 16 ? __reduce_max_sync(0x0000FFFFu, bits) : __reduce_max_sync(0xFFFF0000u, bits);
            if (lane % 16 == 0) bound[2 * warp + lane / 16] = best;
        };
        if (k > 0) {
            if (i == 0) {
                publish();
                __syncthreads();
                if (warp == 0) {
                    tau = kth_of_lanes(bound[lane], k);
                    if (lane == 0) s.tau = tau;
                }
                __syncthreads();
            }
            tau = *static_cast<volatile uint32_t*>(&s.tau);
            hit = __any_sync(0xFFFFFFFFu, !(top < bits_value(tau)));
        }
        if (hit) {
            // at or above tau, above the own k-th
            const float low = kth >= tau && kth ? bits_value(kth + 1) : bits_value(tau);
            uint32_t mask = 0;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                uint32_t m = 0;
#pragma unroll
                for (int e = 0; e < N; ++e) m |= (c.get(j, e) >= low ? 1u : 0u) << e;
                if (tau == 0 && kth == 0)  // fewer than k numbers so far: NaN too
#pragma unroll
                    for (int e = 0; e < N; ++e) m |= (c.get(j, e) != c.get(j, e) ? 1u : 0u) << e;
                if (w + j * kThreads < w1) mask |= m << (j * N);
            }
            bool cut = false;
            while (const uint32_t b = __ballot_sync(0xFFFFFFFFu, mask != 0)) {
                if (mask) {
                    const int q = __ffs(mask) - 1, j = q / N, e = q % N;
                    mask &= mask - 1;
                    const uint8_t* src = ring + (i % kStages) * kTileBytes + (j * kThreads + threadIdx.x) * 16;
                    const float v = sizeof(T) == 4 ? reinterpret_cast<const float*>(src)[e]
                                                   : __uint_as_float(static_cast<uint32_t>(
                                                         reinterpret_cast<const uint16_t*>(src)[e]) << 16);
                    list[have + __popc(b & ((1u << lane) - 1))] =
                        order_key(v, static_cast<uint32_t>((w + j * kThreads) * N - pre) + e);
                }
                have += __popc(b);
                if (have > kList - kWarp) {
                    cut_list(list, have, k);
                    have = min(have, k);
                    cut = true;
                }
            }
            if (cut && have >= k) kth = static_cast<uint32_t>(list[k - 1] >> 32);
            if (i > 0) {
                publish();
                __syncwarp();
                tau = kth_of_lanes(bound[lane], k);
                if (lane == 0) atomicMax(&s.tau, tau);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.empty[i % kStages]);
    }
    int n = 0;
    if (k > 0) {
        // the CTA's lists into one (the ring is free), less what the last tau rules out
        __syncthreads();
        const uint32_t tau = s.tau;
        uint64_t* cand = reinterpret_cast<uint64_t*>(ring);
        for (int q = lane; q < have; q += kWarp) {
            const uint64_t key = list[q];
            if (static_cast<uint32_t>(key >> 32) >= tau) cand[atomicAdd(&s.count, 1)] = key;
        }
        __syncthreads();
        n = s.count;
        cut_all(cand, n, s.top, k);
        n = min(n, k);
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
    }
    // the cluster's: every CTA hands its sums and its best to the first
    if (C > 1) {
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // all of them have started
        if (static_cast<int>(threadIdx.x) < n)
            asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(in_cta(&s.all_top[rank][threadIdx.x], 0)),
                         "l"(s.top[threadIdx.x])
                         : "memory");
        if (threadIdx.x == 0) {
            asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(in_cta(&s.all_n[rank], 0)), "r"(n) : "memory");
            const uint32_t at = in_cta(&s.all_sums[rank], 0);
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(sum.m) : "memory");
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + 4), "f"(sum.z) : "memory");
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + 8), "f"(sum.u) : "memory");
            s.count = 0;
        }
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (rank != 0) return;
        if (k > 0) {
            // no key below any CTA's k-th can be among the k best
            const int r = threadIdx.x / kMaxK, l = threadIdx.x % kMaxK;
            const uint64_t key = r < C && l < s.all_n[r] ? s.all_top[r][l] : 0;
            if (l == k - 1 && key) atomicMax(reinterpret_cast<unsigned long long*>(&s.all_tau), key);
            uint64_t* cand = reinterpret_cast<uint64_t*>(ring);
            __syncthreads();
            if (key && key >= s.all_tau) cand[atomicAdd(&s.count, 1)] = key;
            __syncthreads();
            cut_all(cand, s.count, s.top, k);
        }
        if (warp == 0) {
            sum = lane < C ? s.all_sums[lane] : Sums{-INFINITY, 0.f, 0.f};
#pragma unroll
            for (int d = kMaxCluster / 2; d; d >>= 1) {
                const Sums o{__shfl_xor_sync(0xFFFFFFFFu, sum.m, d), __shfl_xor_sync(0xFFFFFFFFu, sum.z, d),
                             __shfl_xor_sync(0xFFFFFFFFu, sum.u, d)};
                sum = (lane & d) ? join(o, sum) : join(sum, o);
            }
        }
    }
    if (warp != 0) return;
    sum.m = __shfl_sync(0xFFFFFFFFu, sum.m, 0);
    sum.z = __shfl_sync(0xFFFFFFFFu, sum.z, 0);
    sum.u = __shfl_sync(0xFFFFFFFFu, sum.u, 0);
    if (sum.m == INFINITY) sum.z = sum.m - sum.m;  // +inf among the logits: NaN
    const float lse = sum.z == 0.f ? INFINITY : sum.m + logf(sum.z);  // an empty row: every log probability is -inf
    if (lane == 0) {
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
    if (lane < k) {
        const uint64_t key = s.top[lane];
        a.top_ids[t * k + lane] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(key));
        a.top_logprobs[t * k + lane] = ordered_value(static_cast<uint32_t>(key >> 32)) - lse;
    }
}

template <typename T>
cudaError_t launch(const LogprobArgs& a, cudaStream_t s)
{
    constexpr size_t kSmem = kStages * kTileBytes;
    static OccCache occ;
    static const cudaError_t wide =
        cudaFuncSetAttribute(logprobs_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (wide != cudaSuccess) return wide;
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    blocks_per_sm(occ, reinterpret_cast<const void*>(&logprobs_kernel<T>), dev, kThreads, kSmem);  // opts in to kSmem
    // CTAs per row: as many as fill the GPU once (two CTAs per SM), while
    // each still has 16 logits a thread.
    int C = 1;
    while (C < kMaxCluster && a.T * C * 2 <= 2 * 152 && a.V / (C * 2) >= kThreads * 16) C *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.T * C));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
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

cudaError_t read_and_clear_logprobs_error(unsigned int* out)
{
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_logprobs_error, sizeof(v));
    if (e != cudaSuccess) return e;
    *out = v;
    if (v) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_logprobs_error, &zero, sizeof(zero));
    }
    return e;
}

cudaError_t launch_token_logprobs(const LogprobArgs& a, int in_type, cudaStream_t s)
{
    return in_type == BQD_F32 ? launch<float>(a, s) : launch<__nv_bfloat16>(a, s);
}

}  // namespace bqd
