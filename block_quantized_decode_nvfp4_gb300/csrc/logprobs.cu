// logprobs.cu -- log probability of given tokens, entropy and the top
// alternatives of logits rows, in one pass over the logits.
//
// With m = max x, t = (x - m) log2(e), z = sum 2^t and u = sum 2^t t:
//   lse = m + log2(z) ln 2, logprob = x_tok - lse, entropy = (log2 z - u / z)
//   ln 2,
// and two partial results join as m = max(m1, m2), f = e^(m1 - m), z1' = f z1,
// u1' = f (u1 + z1 log2 f), likewise the other, and sums. t is one multiply-add,
// x log2(e) - r with r = m log2(e) rounded (what the rounding moved goes back
// into lse; the fp32 log2(e) is 1.3e-8 off, which moves lse by as much of
// itself). The alternatives are ordered by one
// 64-bit key per logit: the value's bits made monotonic (NaN lowest, -0 as
// +0) above the complemented index, so equal values go to
// the lower index; the k largest keys of a row are the k largest of the k
// largest of its parts.
//
// Few rows: a row is shared by a cluster of C CTAs (16 for a decode step's one
// row), which join through distributed shared memory; of many rows each has a
// CTA. Either way the call is one launch, and nothing passes through memory.
// A row's whole 16-byte windows come through a ring of 32 KiB bulk copies
// (two stages, three CTAs per SM: 96 KiB and more in flight per SM); its
// ragged ends, at most 14 logits, are read one by one. The warps run through
// the ring without a barrier of the CTA. A tile costs its maximum, the sums
// (two logits an instruction where there is a packed form) and a compare of
// the thread's maximum with tau; what a tile costs beside its logits (waits,
// addresses) made 32 KiB better than 16 or 8 KiB (the sums of 2047 bf16 rows of
// 151936: 128, 147 and 215 us).
//
// Alternatives. The k-th largest of the maxima that the CTA's 32 groups of
// lanes (8 or 16) have seen has k logits at or above it: that is tau, published in shared
// memory after the first tile and again by every warp that meets a logit at
// or above it (the maxima only grow, so an older one is a bound too). What
// passes goes to the warp's own list of up to 64 keys; one that has grown past
// 32 is cut back to its k best (each entry counts the larger ones), and as a
// warp's logits come in ascending tiles, those of later tiles have to exceed
// its k-th from then on: of equal logits the list has those of lower indices.
// (So the logits after the row's last whole window, its highest indices, join
// their warp's list after its last tile.) About k (1 + log(tiles)) logits pass
// in a row of distinct logits; rows of equal ones cost a few cuts in their
// first tile. At the end the lists are joined, first the CTA's, then the
// cluster's, by the same count.
//
// Measured over 151936 logits: one fp32 row with 20 alternatives 10.0 us, 128
// with 8 26 us (18.7 without alternatives), 2047 bf16 rows with 5 131 us or 4.7
// TB/s (107 without). What bounds it: the instructions per logit (64 % of the
// issue slots), a quarter of them the alternatives' bookkeeping. Chunks with a
// logit of -inf or of the type's lowest value are summed one by one: where
// those are nine of ten, 128 rows take 30 us and 2047 bf16 rows 255.
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

constexpr int kPer = 4;                             // windows per thread and pass over a tile
constexpr int kTileWindows = 2048;
constexpr int kTileBytes = kTileWindows * 16;
constexpr int kList = 64;                           // entries of a warp's list
constexpr int kMaxK = 32;
constexpr int kTail = 14;                           // logits outside a row's whole windows at most (bf16: 7 and 7)
constexpr int kMaxCluster = 16;
static_assert(kList == 2 * kWarp && kMaxK <= kWarp && kTail <= kWarp,
              "a cut handles two keys per lane, and leaves room for a ballot");
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

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

// From this size of a maximum on, differences are taken before the product with
// log2(e): the product's rounding, which t and with it z carry as a shift, would
// exceed 2^6 and leave the range of 2^t (logits masked throughout by a large
// negative value), and further on the product itself would overflow.
constexpr float kHuge = 1073741824.f;

// The shift of t and log2(z) for a maximum m: what m log2(e) lost when rounded.
__device__ __forceinline__ float shift_of(float m)
{
    return fabsf(m) < kHuge ? fmaf(m, kLog2e, -__fmul_rn(m, kLog2e)) : 0.f;
}

__device__ __forceinline__ void raise(Sums& s, float m)  // s relative to m >= s.m
{
    if (s.m != -INFINITY) {
        const bool plain = fabsf(s.m) < kHuge && fabsf(m) < kHuge;
        // rounded products, as add() takes them: equal maxima must give 0
        const float d = plain ? __fmul_rn(s.m, kLog2e) - __fmul_rn(m, kLog2e) : (s.m - m) * kLog2e, f = ex2(d);
        s.u = d < -150.f ? 0.f : (s.u + s.z * d) * f;
        s.z *= f;
    }
    s.m = m;
}
// The join of a warp's 32, the same in every lane.
__device__ __forceinline__ Sums join_warp(Sums s)
{
    float m = s.m;
#pragma unroll
    for (int d = 16; d; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    raise(s, m);
    s.z = warp_sum(s.z);
    s.u = warp_sum(s.u);
    return s;
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
    // Windows of it that are padding, when there are numbers above -1e29 in it:
    // a value that adds nothing and keeps t finite.
    __device__ __forceinline__ void pad(int j)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[j][i] = sizeof(T) == 4 ? 0xF149F2CAu : 0xF14AF14Au;  // -1e30
    }
    // z += sum 2^t, u += sum 2^t t; false, and nothing added, where a t is -inf
    // (a logit of -inf or of the type's lowest value: 0 * -inf), or m is huge.
    __device__ __forceinline__ bool add(float m, float& z, float& u) const
    {
        const float r = -__fmul_rn(m, kLog2e);
        const uint64_t r2 = pack(r, r), l2 = pack(kLog2e, kLog2e);
        uint64_t zz = 0, uu = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
#pragma unroll
            for (int e = 0; e < kN; e += 2) {
                const uint64_t t = fma2(pack(get(j, e), get(j, e + 1)), l2, r2);
                float v, w;
                unpack(t, v, w);
                const uint64_t p = pack(ex2(v), ex2(w));
                zz = add2(zz, p);
                uu = fma2(p, t, uu);
            }
        float a, b, c, d;
        unpack(zz, a, b);
        unpack(uu, c, d);
        if (c + d != c + d || !(fabsf(m) < kHuge)) return false;
        z += a + b;
        u += c + d;
        return true;
    }
};

// The same for any logits, from the tile in shared memory: t kept above -150
// (2^-150 is 0 in fp32), and differences first where m is huge.
template <typename T>
__device__ __noinline__ float2 add_slowly(const uint8_t* at, int stride, int windows, float m)
{
    constexpr int N = 16 / static_cast<int>(sizeof(T));
    const bool plain = fabsf(m) < kHuge;
    const float mm = m == -INFINITY ? 0.f : m, r = -__fmul_rn(m, kLog2e);
    float2 s = make_float2(0.f, 0.f);
    for (int j = 0; j < windows; ++j, at += stride)
        for (int e = 0; e < N; ++e) {
            float x;
            if constexpr (sizeof(T) == 4)
                x = reinterpret_cast<const float*>(at)[e];
            else
                x = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(at)[e]) << 16);
            const float t = fmaxf(plain ? fmaf(x, kLog2e, r) : (x - mm) * kLog2e, -150.f), p = ex2(t);
            s.x += p;
            s.y += p * t;
        }
    return s;
}

template <int WARPS, int STAGES>
struct Shared {
    uint64_t full[STAGES], empty[STAGES];
    union {
        alignas(16) uint64_t list[WARPS][kList];  // a warp's candidates, read 16 bytes at a time
        uint64_t all_top[kMaxCluster][kMaxK];     // of a cluster's leader: every CTA's best, once its lists are cut
    };
    // keys to be cut to the k best: at most kMaxK of each warp, or of each CTA; +16: padding
    alignas(16) uint64_t cand[kMaxCluster * kMaxK + 16];
    uint64_t top[kMaxK];                      // this CTA's best, descending
    uint64_t tail[kTail];                     // keys of the logits after the row's whole windows
    int tails;                                // their number
    Sums sums[WARPS];
    alignas(16) uint32_t bound[kWarp];        // the lane groups' maxima, as ordered bits; 0: none above -inf
    uint32_t tau;                             // the k-th largest of them; 0: fewer than k
    int count;
    int all_n[kMaxCluster];                   // of the leader: every CTA's number of best, and sums
    Sums all_sums[kMaxCluster];
};
using Shared8 = Shared<8, 2>;
static_assert(offsetof(Shared8, list) % 16 == 0 && offsetof(Shared8, cand) % 16 == 0 && kList % 2 == 0,
              "16-byte reads of the lists");

// A bound's value: everything for none.
__device__ __forceinline__ float bits_value(uint32_t b) { return b == 0 ? -INFINITY : ordered_value(b); }

// The ordered bits of a value: the upper half of its key.
__device__ __forceinline__ uint32_t order_bits(float x) { return static_cast<uint32_t>(order_key(x, 0) >> 32); }

// The k-th largest of 32 values, at least: the values are cut to their upper
// 27 bits and the lane's number, which makes them distinct. The same for every
// lane.
__device__ __forceinline__ uint32_t kth_of_32(const volatile uint32_t* v, int k)
{
    const int lane = threadIdx.x % kWarp;
    const uint32_t mine = (v[lane] & ~31u) | lane;
    int r = 0;  // how many are ahead
#pragma unroll 8
    for (int l = 0; l < kWarp; ++l) r += __shfl_sync(0xFFFFFFFFu, mine, l) > mine;
    return __shfl_sync(0xFFFFFFFFu, mine, __ffs(__ballot_sync(0xFFFFFFFFu, r == k - 1)) - 1) & ~31u;
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

// Adds the warp's keys that are `in` to a list of the CTA's.
__device__ __forceinline__ void collect(uint64_t* cand, int* count, uint64_t key, bool in)
{
    const int lane = threadIdx.x % kWarp;
    const uint32_t b = __ballot_sync(0xFFFFFFFFu, in);
    int at = 0;
    if (lane == 0 && b) at = atomicAdd(count, __popc(b));
    at = __shfl_sync(0xFFFFFFFFu, at, 0);
    if (in) cand[at + __popc(b & ((1u << lane) - 1))] = key;
}

// The k best of c keys at cand (room for 16 more) in descending order to top:
// eight lanes count a key's larger ones. Called by the whole CTA, with a
// barrier before.
template <int WARPS>
__device__ __forceinline__ void cut_all(uint64_t* cand, int c, uint64_t* top, int k)
{
    if (threadIdx.x < 16) cand[c + threadIdx.x] = 0;
    __syncthreads();
    const int sub = threadIdx.x % 8, group = threadIdx.x / 8;
#pragma unroll 1
    for (int i = group; i - group < c; i += WARPS * 4) {  // whole warps
        const uint64_t mine = i < c ? cand[i] : 0;
        int r = 0;
#pragma unroll 2
        for (int j = 2 * sub; j < c; j += 16) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&cand[j]);
            r += (v.x > mine) + (v.y > mine);
        }
        r += __shfl_xor_sync(0xFFFFFFFFu, r, 1);
        r += __shfl_xor_sync(0xFFFFFFFFu, r, 2);
        r += __shfl_xor_sync(0xFFFFFFFFu, r, 4);
        if (sub == 0 && mine && r < k) top[r] = mine;
    }
    __syncthreads();
}

__device__ __forceinline__ uint32_t in_cta(const void* p, int rank)  // its counterpart in another CTA of the cluster
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}

// A CTA's part of a row. 16-byte windows are counted from the one that holds
// the row's first logit; `pre` elements of it lie before the row. The CTA has
// the whole windows [w0, w1).
template <typename T>
struct Part {
    const T* x;
    int pre, tiles;
    int whole0, whole1, w0, w1;  // below 2^30: V is below 2^31
    __device__ __forceinline__ Part(const LogprobArgs& a, int64_t t, int rank, int C)
    {
        constexpr int N = 16 / static_cast<int>(sizeof(T));
        x = static_cast<const T*>(a.x) + t * a.pitch;
        pre = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
        whole0 = pre ? 1 : 0;
        whole1 = max(whole0, static_cast<int>((static_cast<uint32_t>(pre) + static_cast<uint32_t>(a.V)) / N));
        const uint32_t whole = whole1 - whole0, share = (whole + C - 1) / static_cast<uint32_t>(C);
        w0 = whole0 + static_cast<int>(min(share * rank, whole));
        w1 = whole0 + static_cast<int>(min(share * (rank + 1), whole));
        tiles = (w1 - w0 + kTileWindows - 1) / kTileWindows;
    }
};

// CLUSTER: C CTAs a row; else one.
template <typename T, int WARPS, int STAGES, int CTAS, bool CLUSTER>
__global__ void __launch_bounds__((WARPS + 1) * kWarp, CTAS) logprobs_kernel(const LogprobArgs a, int C)
{
    using K = Chunk<T>;
    constexpr int kStages = STAGES, N = K::kN, kThreads = WARPS * kWarp, kGroup = WARPS;  // lanes per group: 32 groups
    constexpr int kPasses = kTileWindows / (kThreads * kPer);
    static_assert(kPasses * kThreads * kPer == kTileWindows && (WARPS == 8 || WARPS == 16), "tile shape");
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(16) Shared<WARPS, STAGES> s;
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    const int rank = CLUSTER ? static_cast<int>(blockIdx.x % C) : 0, k = a.topk, V = a.V;
    const int64_t t = CLUSTER ? blockIdx.x / C : blockIdx.x;
    uint64_t* list = s.list[warp % WARPS];
    volatile uint32_t* bound = s.bound;
    const Part<T> p(a, t, rank, C);
    auto copy = [&](int i) {  // tile i into its stage
        const int w = p.w0 + i * kTileWindows;
        const uint32_t bytes = static_cast<uint32_t>(min(p.w1 - w, kTileWindows)) * 16;
        mbar_arrive_expect_tx(&s.full[i % kStages], bytes);
        bulk_g2s(ring + (i % kStages) * kTileBytes, p.x + (static_cast<int64_t>(w) * N - p.pre), bytes,
                 &s.full[i % kStages]);
    };
    if (threadIdx.x == kThreads) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], WARPS);
        }
        fence_barrier_init();
#pragma unroll 1
        for (int i = 0; i < min(kStages, p.tiles); ++i) copy(i);
    }
    bool ok = true;
    Sums sum{-INFINITY, 0.f, 0.f};
    uint32_t kth = 0;        // of the own list, as ordered bits; 0: not cut yet, or NaN
    float seen = -INFINITY;  // largest so far, of the tiles that mattered
    int have = 0;            // entries of the own list
    if (threadIdx.x < kWarp) s.bound[threadIdx.x] = 0;
    if (threadIdx.x == 0) {
        s.count = 0;
        s.tau = 0;
        s.tails = 0;
    }
    // the row's ends, by the first CTA's first warp, a logit per lane
    if (rank == 0 && warp == 0) {
        const bool whole = p.whole1 > p.whole0;
        const int head = whole ? p.whole0 * N - p.pre : 0;
        const int64_t tail0 = whole ? static_cast<int64_t>(p.whole1) * N - p.pre : 0;
        const int64_t i = lane < head ? lane : tail0 + (lane - head);
        have = head;
        if (lane == 0) s.tails = static_cast<int>(V - tail0);
        if (i < V) {
            float v;
            if constexpr (sizeof(T) == 4)
                v = p.x[i];
            else
                v = __bfloat162float(p.x[i]);
            raise(sum, v);
            const float shift = shift_of(v);
            sum.z = v == -INFINITY ? 0.f : v - v + ex2(shift);  // NaN for NaN (and for +inf)
            sum.u = sum.z * shift;
            seen = v;
            (lane < head ? list[lane] : s.tail[lane - head]) = order_key(v, static_cast<uint32_t>(i));
        }
    }
    __syncthreads();
    if (warp == WARPS) {
        // the rest of the copies; and tau, after the first pass and whenever there is a copy to issue
        auto update = [&] {
            const uint32_t tau = kth_of_32(bound, k);
            if (lane == 0) *static_cast<volatile uint32_t*>(&s.tau) = tau;  // the maxima only grow, and so does it
        };
        if (k > 0 && p.tiles > 0) {
            __syncthreads();
            update();
            __syncthreads();
        }
#pragma unroll 1
        for (int i = kStages; i < p.tiles; ++i) {
            if (k > 0) update();
            ok = ok && mbar_wait_warp(&s.empty[i % kStages], (i / kStages - 1) & 1, &g_logprobs_error);
            if (ok && lane == 0) copy(i);
        }
    }
    for (int i = 0; i < p.tiles && warp < WARPS; ++i) {
        const int st = i % kStages;
        ok = ok && mbar_wait_warp(&s.full[st], (i / kStages) & 1, &g_logprobs_error);
        const int wt = p.w0 + i * kTileWindows, left = min(p.w1 - wt, kTileWindows);  // the tile's first window, windows
#pragma unroll
        for (int pass = 0; pass < kPasses; ++pass) {
            const int w = pass * (kThreads * kPer) + threadIdx.x;  // of the tile
            K c;
            const uint32_t at = smem_u32(ring) + st * kTileBytes + w * 16;
            if (left == kTileWindows) {
#pragma unroll
                for (int j = 0; j < kPer; ++j) c.load(j, at + j * kThreads * 16);
            } else {
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    if (w + j * kThreads < left)
                        c.load(j, at + j * kThreads * 16);
                    else
                        c.clear(j);
                }
            }
            const float top = c.top();
            if (!(top <= sum.m)) raise(sum, top);
            if (left != kTileWindows && top > -1e29f)
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (w + j * kThreads >= left) c.pad(j);
            if (!c.add(sum.m, sum.z, sum.u)) {
                const int mine = min(kPer, (left - w + kThreads - 1) / kThreads);
                const float2 o = add_slowly<T>(ring + st * kTileBytes + w * 16, kThreads * 16, mine, sum.m);
                sum.z += o.x;
                sum.u += o.y;
            }
            if (k == 0) continue;

            // the lane groups' maxima so far
            auto publish = [&] {
                seen = fmaxf(seen, top);
                uint32_t best = seen == -INFINITY ? 0u : order_bits(seen);  // -inf may be padding, or NaN passed over
#pragma unroll
                for (int d = kGroup / 2; d; d >>= 1) best = max(best, __shfl_xor_sync(0xFFFFFFFFu, best, d));
                if (lane % kGroup == 0) bound[threadIdx.x / kGroup] = best;
            };
            if (i == 0 && pass == 0) {  // the CTA's k-th of them, for the first time
                publish();
                __syncthreads();
                __syncthreads();
            }
            const uint32_t tau = *static_cast<volatile uint32_t*>(&s.tau);
            if (!__any_sync(0xFFFFFFFFu, !(top < bits_value(tau)))) continue;

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
                if (w + j * kThreads < left) mask |= m << (j * N);
            }
            bool cut = false;
            while (const uint32_t b = __ballot_sync(0xFFFFFFFFu, mask != 0)) {
                if (mask) {
                    const int q = __ffs(mask) - 1, j = q / N, e = q % N;
                    mask &= mask - 1;
                    const uint8_t* src = ring + st * kTileBytes + (w + j * kThreads) * 16;
                    const float v = sizeof(T) == 4 ? reinterpret_cast<const float*>(src)[e]
                                                   : __uint_as_float(static_cast<uint32_t>(
                                                         reinterpret_cast<const uint16_t*>(src)[e]) << 16);
                    list[have + __popc(b & ((1u << lane) - 1))] =
                        order_key(v, static_cast<uint32_t>(wt + w + j * kThreads) * N - p.pre + e);
                }
                have += __popc(b);
                if (have > kList - kWarp) {
                    cut_list(list, have, k);
                    have = min(have, k);
                    cut = true;
                }
            }
            if (cut && have >= k) kth = static_cast<uint32_t>(list[k - 1] >> 32);
            if (i + pass > 0) publish();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.empty[st]);
    }
    if (!ok) let_copies_land();
    if (warp == 0) {  // the list holds 32 at most
        const int tails = s.tails;
        if (lane < tails) list[have + lane] = s.tail[lane];
        have += tails;
    }
    // the block's sums
    sum = join_warp(sum);
    if (lane == 0 && warp < WARPS) s.sums[warp] = sum;
    int n = 0;
    if (k > 0) {
        // the CTA's lists into one, less what the last tau rules out
        if (have > k) {
            cut_list(list, have, k);
            have = k;
        }
        __syncthreads();
        const uint32_t tau = kth_of_32(bound, k);
        const uint64_t key = lane < have ? list[lane] : 0;
        collect(s.cand, &s.count, key, key && static_cast<uint32_t>(key >> 32) >= tau);
        __syncthreads();  // the lists are read
        if (CLUSTER) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        n = s.count;
        cut_all<WARPS + 1>(s.cand, n, s.top, k);
        n = min(n, k);
    } else {
        __syncthreads();
        if (CLUSTER) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    if (warp == 0) {
        sum = Sums{-INFINITY, 0.f, 0.f};
        if (lane < WARPS) sum = s.sums[lane];
        __syncwarp();
        sum = join_warp(sum);
    }
    // the cluster's: every CTA hands its sums and its best to the first
    if (CLUSTER) {
        // all of them have read their lists: the leader's may be written over
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
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
            // the k-th largest of some 32 of the CTAs' first ones has k keys at or above it
            const int each = kWarp / C, r0 = lane / each, l0 = lane % each;
            const uint64_t some = r0 < C && l0 < s.all_n[r0] ? s.all_top[r0][l0] : 0;
            int ahead = 0;
#pragma unroll 8
            for (int l = 0; l < kWarp; ++l) ahead += __shfl_sync(0xFFFFFFFFu, some, l) > some;
            const uint32_t at = __ballot_sync(0xFFFFFFFFu, some != 0 && ahead == k - 1);
            const uint64_t least = at ? __shfl_sync(0xFFFFFFFFu, some, __ffs(at) - 1) : 0;
            for (int r = warp; r < C; r += WARPS + 1) {
                const uint64_t key = lane < s.all_n[r] ? s.all_top[r][lane] : 0;
                collect(s.cand, &s.count, key, key && key >= least);
            }
            __syncthreads();
            cut_all<WARPS + 1>(s.cand, s.count, s.top, k);
        }
        if (warp == 0) {
            sum = Sums{-INFINITY, 0.f, 0.f};
            if (lane < C) sum = s.all_sums[lane];
            __syncwarp();
            sum = join_warp(sum);
        }
    }
    if (warp == 0) {
        if (sum.m == INFINITY) sum.z = sum.m - sum.m;  // +inf among the logits: NaN
        // an empty row: every log probability is -inf
        const float lse = sum.z == 0.f ? INFINITY : sum.m + (log2f(sum.z) - shift_of(sum.m)) * kLn2;
        if (lane == 0) {
            if (a.logprob) {
                const int tok = a.tokens[t];
                float v = -INFINITY;
                if (tok >= 0 && tok < V) {
                    if constexpr (sizeof(T) == 4)
                        v = p.x[tok] - lse;
                    else
                        v = __bfloat162float(p.x[tok]) - lse;
                }
                a.logprob[t] = v;
            }
            if (a.entropy) a.entropy[t] = sum.z == 0.f ? 0.f : (log2f(sum.z) - sum.u / sum.z) * kLn2;
        }
        if (lane < k) {
            const uint64_t key = s.top[lane];
            a.top_ids[t * k + lane] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(key));
            a.top_logprobs[t * k + lane] = ordered_value(static_cast<uint32_t>(key >> 32)) - lse;
        }
    }
}

template <typename T, int WARPS, int STAGES, int CTAS, bool CLUSTER>
cudaError_t launch_as(const LogprobArgs& a, int C, cudaStream_t s)
{
    constexpr size_t kSmem = STAGES * kTileBytes;
    static_assert(CTAS * (kSmem + sizeof(Shared<WARPS, STAGES>) + 1024) <= 228 * 1024, "shared memory of an SM");
    auto kern = logprobs_kernel<T, WARPS, STAGES, CTAS, CLUSTER>;
    const unsigned grid = static_cast<unsigned>(a.T * C);
    static OccCache occ;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    blocks_per_sm(occ, reinterpret_cast<const void*>(kern), dev, (WARPS + 1) * kWarp, kSmem);  // opts in to kSmem
    if (!CLUSTER) {
        kern<<<grid, (WARPS + 1) * kWarp, kSmem, s>>>(a, 1);
        return cudaGetLastError();
    }
    e = allow_wide_clusters(occ, reinterpret_cast<const void*>(kern), dev);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((WARPS + 1) * kWarp);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = static_cast<unsigned>(C);
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a, C);
}

template <typename T>
cudaError_t launch(const LogprobArgs& a, cudaStream_t s)
{
    // CTAs per row: as many as the GPU holds at once (three per SM, less what
    // clusters leave free where they do not fit a GPC: 456 CTAs in clusters of
    // three took 35 us, 384 of them 24), while each has 32 logits a thread.
    const int64_t room = 384 / a.T, most = a.V / (256 * 32);
    int64_t C = room < most ? room : most;
    C = C < 1 ? 1 : C > kMaxCluster ? kMaxCluster : C;
    if (C > 1) return launch_as<T, 8, 2, 3, true>(a, static_cast<int>(C), s);
    return launch_as<T, 8, 2, 3, false>(a, 1, s);
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
