// tree_attn_wide.cu -- attention over the paged cache where many query rows
// share a kv head (drafted trees, several drafted tokens times the group's
// query heads), on the 5th-generation tensor cores; bf16 caches.
//
// The mathematics, the rows and the even split are those of tree_attn.cu.
// With hundreds of rows a key is worth 4 D rows flops for its 4 D bytes, so
// the bound is the tensor cores (and beside them the exponentials: one per
// 2 D of the products' multiply-adds); with tens of rows it is the one read
// of keys and values, and the padding to 128 rows costs nothing yet.
//
// A CTA (one per SM, an even share of units of 128 tokens) runs two softmax
// slots in turn, so that one slot's products run under the other's softmax:
//  - TWO: an item is 256 rows, a slot each 128 of them, over the same tokens;
//  - else: an item is 128 rows; the slots take every other block of 128
//    tokens, each with its own (m, z, o), and join at the item's end.
// Warps 0 and 3 load K and V blocks by 4-D tensor copies, one box per page
// and 64 elements of D (128-byte swizzle; pages outside the cache read as
// zero). Warps 1 and 2, a thread each, issue one slot's products: per block s
// = q k^T (both from shared memory, K-major) and o += p v with p from tensor
// memory and v MN-major, a block's o before the next block's s. The slots take
// turns block by block (left to themselves they fall into step, and both
// softmaxes run while the tensor cores wait); an issuing thread keeps pace with
// the tensor cores, so it does its waiting while the other issues. Warps 4..7
// and 8..11 are the slots' softmax, a row per thread (tensor-memory lane): they
// read s, write p in bf16 over the columns of s that they have read, and rescale
// o in tensor memory only when a row's maximum has grown by more than 2^8 (p
// then stays below 2^8, and nothing is lost: fp32 sums, bf16's range).
//
// Four trees of 64 tokens over 32768 (64 query heads on 8, D = 128): 191 us,
// 1.12 PFLOP/s of products. A block of both slots takes about 3000 cycles, 2670
// of them the tensor cores' (83 per M128 N128 K16: the score product reads 8 KB
// of shared memory for each); beside them the launch, the starts of two items
// per CTA, their parts and the join, 27 us together. Each of the two tiles of
// 256 rows reads the keys and values for itself (906 MB).
// Tensor memory: s0 | s1 (128 columns each) | o0 | o1 (D each).
//
// Blocks that reach past the cached tokens (drafts, the end), and all blocks
// of a share with a bad page id, take a slower way: visibility as 128 bits
// per row, and their V rows cleared in shared memory where they are not
// tokens or where a draft's value is infinite or NaN; what was cleared of
// drafts is added at the end to the rows that see it, so that 0 * v of a
// hidden draft counts nothing.
// Every wait is bounded (kErrWaitTimeout in the kernel's error word).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "attn.h"
#include "common.cuh"
#include "f32x2.cuh"
#include "host_util.h"
#include "stream.cuh"
#include "tree_attn.cuh"

namespace bqd {

__device__ unsigned int g_attn_error = 0;

namespace {

constexpr int kThreads = 384;
constexpr int kTok = 128;  // tokens per block (and unit of the split)
constexpr int kGrid = 152;
constexpr int kOver = 4;  // units that an item's beginning and end cost
constexpr float kGrow = 8.f;
constexpr float kHuge = 67108864.f;  // of a maximum in log2 units: below it, its rounding moves p by 2^4 at most

template <int D, bool TWO>
struct Wide {
    static constexpr int kRows = TWO ? 256 : 128;
    static constexpr int kQTile = 128 * D * 2;
    static constexpr int kBlk = kTok * D * 2;  // bytes of a K or V block
    static constexpr int kKS = D == 64 ? 4 : 3;
    static constexpr int kVS = D == 64 ? 4 : 2;
    static constexpr int kQBytes = (TWO ? 2 : 1) * kQTile;
    static constexpr int kSmem = kQBytes + (kKS + kVS) * kBlk + 1024;  // + alignment slack
    static constexpr int kPitch = D + 4;  // floats of a row in the slots' join
    static_assert(kSmem <= 227 * 1024 - (TWO ? 1024 : 2048), "shared memory of one CTA, static beside it");
    static_assert(128 * kPitch * 4 <= (kKS + kVS) * kBlk, "the join lies over the ring");
};

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
        : "memory");
}

// Shared-memory matrix descriptors, 128-byte swizzle (layout type 2, version
// 1): rows of 128 bytes in atoms of 8 rows, 1024 bytes apart. K-major: the
// leading offset is unused. MN-major (the 128 bytes run along n): `lead` is
// the distance of the next 64 elements of n.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr, uint32_t lead)
{
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((lead >> 4) & 0x3FFFu) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// 32 columns of this warp's 32 lanes; the loads of one wait may be several.
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t* r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st(uint32_t at, const uint32_t* r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// o of a slot's 32 rows of the warp times each row's f. Rare, so a call.
template <int D>
__device__ __noinline__ void rescale(uint32_t o_at, float f)
{
    const uint64_t ff = pack(f, f);
    for (int k = 0; k < D / 32; ++k) {
        uint32_t o[32];
        tmem_ld(o_at + 32 * k, o);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
            float x, y;
            unpack(mul2(pack(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), ff), x, y);
            o[e] = __float_as_uint(x);
            o[e + 1] = __float_as_uint(y);
        }
        tmem_st(o_at + 32 * k, o);
    }
    tmem_st_wait();
}

// The softmax of a block in which a row's scores are huge: s c - m in one
// rounding would leave of the row's largest what m was rounded by, which p
// cannot hold, so differences are taken of the rounded products. Writes p and
// hands it on as the loop does; the row's sum of p.
__device__ __noinline__ float far_block(uint32_t s_at, uint4 see, float c, float m, uint64_t* ready)
{
    const float sub = m == -INFINITY ? 0.f : m;
    float z = 0.f;
#pragma unroll 1
    for (int k = 1; k >= 0; --k) {
        uint32_t s[64], p[32];
        tmem_ld(s_at + 64 * k, s);
        tmem_ld(s_at + 64 * k + 32, s + 32);
        tmem_ld_wait();
        const uint32_t lo = k ? see.z : see.x, hi = k ? see.w : see.y;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            float x[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = 2 * e + i;
                const bool seen = ((t < 32 ? lo : hi) >> (t & 31)) & 1;
                x[i] = seen ? attn_ex2(__fmul_rn(__uint_as_float(s[t]), c) - sub) : 0.f;
            }
            z += x[0] + x[1];
            p[e] = attn_bf16x2(x[0], x[1]);
        }
        tmem_st(s_at + 64 * k, p);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (threadIdx.x % kWarp == 0) mbar_arrive(&ready[k]);
    }
    return z;
}

// Bits 0 .. 127: whether token i of the request (t of the call) sees draft j0 +
// e (negative: a cached token).
__device__ __forceinline__ uint4 sees128(const AttnArgs& a, int64_t t, int i, int64_t j0)
{
    uint32_t see[4];
    if (!a.mask) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t last = i - (j0 + 32 * k);  // bits 0 .. last
            see[k] = last < 0 ? 0u : last >= 31 ? 0xFFFFFFFFu : (2u << last) - 1u;
        }
        return make_uint4(see[0], see[1], see[2], see[3]);
    }
    const int64_t w = j0 > 0 ? j0 >> 6 : 0;
    const uint64_t* m = a.mask + t * a.mask_words + w;
    uint64_t x[3];  // 128 bits from any bit of the first
#pragma unroll
    for (int k = 0; k < 3; ++k) x[k] = j0 > -128 && w + k < a.mask_words ? m[k] : 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t j = j0 + 32 * k;
        if (j <= -32) {
            see[k] = 0xFFFFFFFFu;
        } else if (j < 0) {
            const int c = static_cast<int>(-j);  // bits 0 .. c - 1 are cached tokens
            see[k] = ((1u << c) - 1u) | static_cast<uint32_t>(x[0] << c);
        } else {
            const int at = static_cast<int>(j - 64 * w), b = at & 63;  // at: 0 .. 159
            uint64_t v = (at < 64 ? x[0] : at < 128 ? x[1] : x[2]) >> b;
            if (b > 32) v |= (at < 64 ? x[1] : x[2]) << (64 - b);  // at 128 .. 159: b <= 31
            see[k] = static_cast<uint32_t>(v);
        }
    }
    return make_uint4(see[0], see[1], see[2], see[3]);
}

// The item (or part of one) that the CTA works on: written by one thread, read
// by all, so that the softmax's registers hold scores and not bookkeeping.
struct Seg {
    int h, tile, n;         // kv head, tile of rows; blocks
    int rows, o0, group;    // live rows of the tile, first token of the request, rows per token
    int steps[2];           // softmax steps of the slots
    int plain, ctx, len;    // tokens every row sees, cached tokens, tokens: from l0, kept within +-2^30
    int64_t l0, table;      // first token; the request's row of the table
    int64_t parts;          // where its part goes; -1: it is the whole item
    int skip;               // there is none
    int odd, bad;           // drafts with values that are not finite, pages outside the cache: found while at it
};

struct Bars {
    uint64_t kfull[4], kempty[4], vfull[4], vempty[4], sfull[2], pready[2][2], odone[2], turn[2];
};

// A block that is not all tokens seen by every row: makes its V block fit for
// the products (the warp's 32 rows, from row0: cleared where they are no
// tokens, or not finite; both slots of a TWO item do so, each before its own
// products, and write the same) and returns the thread's row of visibility,
// 128 bits. v: the V block in shared memory, after it has landed.
template <int D>
__device__ __noinline__ uint4 special_block(const AttnArgs& a, const Seg& g, int j, int row0, int64_t qt, int qi,
                                            uint8_t* v, int* odd_flag)
{
    const int lane = threadIdx.x % kWarp;
    const int sh = min(a.page_shift, 7), nbox = kTok >> sh;  // log2 of a box's tokens; kTok is 2^7
    const int rel = j * kTok;  // of the block's first token, from l0
    const int lb = rel + (lane << sh);
    const int e = lane < nbox && lb < g.len ? a.table[g.table + ((g.l0 + lb) >> a.page_shift)] : -1;
    const uint4 sees = sees128(a, qt, qi, rel - g.ctx);
    const uint32_t pages = __ballot_sync(0xFFFFFFFFu, e >= 0 && e < a.cache.num_pages);  // boxes that are tokens
    const int at = rel + row0 + lane;
    const bool is_token = at < g.len && ((pages >> ((row0 + lane) >> sh)) & 1);
    const uint32_t tokens = __ballot_sync(0xFFFFFFFFu, is_token);
    const uint32_t drafts = __ballot_sync(0xFFFFFFFFu, is_token && at >= g.ctx);
    if (tokens != 0xFFFFFFFFu || drafts) {
        // a lane has 16 bytes of every fourth row, so that eight lanes read a whole line
        uint8_t* mine = v + (row0 + lane / 8) * 128 + lane % 8 * 16;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
            uint4 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = (drafts >> (4 * i + lane / 8)) & 1
                           ? *reinterpret_cast<const uint4*>(mine + h * (kTok * 128) + i * 512)
                           : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                bool odd = false;
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const bool lo = (w[y] & 0x7F80u) == 0x7F80u, hi = (w[y] & 0x7F800000u) == 0x7F800000u;
                    odd |= lo || hi;
                    if (lo) w[y] &= 0xFFFF0000u;
                    if (hi) w[y] &= 0xFFFFu;
                }
                if (odd) {
                    *static_cast<volatile int*>(odd_flag) = 1;  // known before the element is gone
                    __threadfence_block();
                }
                if (odd || !((tokens >> (4 * i + lane / 8)) & 1))
                    *reinterpret_cast<uint4*>(mine + h * (kTok * 128) + i * 512) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        fence_async();
    }
    uint32_t see[4] = {sees.x, sees.y, sees.z, sees.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int left = g.len - (rel + 32 * k);
        if (left < 32) see[k] &= left <= 0 ? 0u : (1u << left) - 1u;
        uint32_t real = 0;
        if (sh >= 5)
            real = ((pages >> (32 * k >> sh)) & 1) ? 0xFFFFFFFFu : 0u;
        else
            for (int x = 0; x < 32; x += 1 << sh)
                if ((pages >> ((32 * k + x) >> sh)) & 1) real |= ((1u << (1 << sh)) - 1u) << x;
        see[k] &= real;
    }
    return make_uint4(see[0], see[1], see[2], see[3]);
}

// The next item, or part of one, with tokens in the CTA's share (or a whole one
// that has none); g.skip: there is none such. One thread's work.
template <int D, bool TWO>
__device__ __noinline__ void next_seg(const AttnArgs& a, AttnShare& share, int64_t& from, Seg& g)
{
    using S = Wide<D, TWO>;
    AttnShare sh = share;
    int64_t u = from, b0;
    g.skip = 1;
    while (g.skip && u < sh.end) {
        const AttnReq q = attn_request(a, sh.r, S::kRows, kTok, kOver);
        attn_place(sh, q, u, g.h, g.tile, b0);
        int64_t cnt = min(q.nb - b0, sh.end - u);
        const int64_t item_end = u + q.nb - b0;
        u += cnt;
        // the item's first kOver units stand for what it costs beside its tokens
        cnt = max(b0 + cnt - kOver, int64_t(0));
        b0 = max(b0 - kOver, int64_t(0));
        cnt -= b0;
        g.skip = cnt <= 0;
        const int64_t l0 = b0 * kTok, l1 = min((b0 + max(cnt, int64_t(0))) * kTok, q.len);
        auto from_l0 = [&](int64_t l) {
            return static_cast<int>(min(max(l - l0, -(int64_t(1) << 30)), int64_t(1) << 30));
        };
        g.n = l1 > l0 ? static_cast<int>((l1 - l0 + kTok - 1) / kTok) : 0;
        g.group = a.group;
        g.rows = static_cast<int>(min(static_cast<int64_t>(q.n) * a.group - static_cast<int64_t>(g.tile) * S::kRows,
                                      static_cast<int64_t>(S::kRows)));
        g.o0 = q.o0;
        g.steps[0] = TWO ? g.n : (g.n + 1) / 2;
        g.steps[1] = TWO ? (g.rows > 128 ? g.n : 0) : g.n / 2;
        g.ctx = from_l0(q.ctx);
        g.len = min(from_l0(q.len), static_cast<int>(l1 - l0));
        g.plain = max(0, min(g.ctx, from_l0(q.len)));
        g.l0 = l0;
        g.table = sh.r * a.width;
        g.odd = g.bad = 0;
        const bool whole = b0 == 0 && cnt == q.nb - kOver;
        g.parts = whole ? -1 : (2 * blockIdx.x + (b0 == 0 ? 1 : 0)) * static_cast<int64_t>(attn_part_floats(S::kRows, D));
        if (b0 == 0 && !whole && !g.skip)
            static_cast<AttnMeta*>(a.ws)[blockIdx.x] = attn_meta(a, sh, q, g.h, g.tile, S::kRows, item_end);
        if (u < sh.end) {
            int64_t next = sh.base + q.nb * q.tiles * a.cache.heads;
            while (u == next) {  // the next request with rows
                ++sh.r;
                sh.base = next;
                next += attn_units(a, sh.r, S::kRows, kTok, kOver);
            }
        }
    }
    share.r = sh.r;
    share.base = sh.base;
    from = u;
}

template <int D, bool TWO>
__global__ void __launch_bounds__(kThreads, 1)
    tree_attn_wide_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_v)
{
    using S = Wide<D, TWO>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) Bars bar;
    __shared__ int64_t s_find[kThreads / kWarp + 2];
    __shared__ AttnShare s_share;
    __shared__ int64_t s_u;
    __shared__ Seg s_seg[2];
    __shared__ uint32_t s_tmem;
    __shared__ float s_mz[TWO ? 1 : 128][2];  // slot 1's m and z, for the join
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* const sm = smem_raw + (base - smem_u32(smem_raw));
    const uint32_t q_at = base, k_at = base + S::kQBytes, v_at = k_at + S::kKS * S::kBlk;
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join waits for this grid's end
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bar.kfull[i], 1);
            mbar_init(&bar.kempty[i], TWO ? 2 : 1);  // slots that read a block
            mbar_init(&bar.vfull[i], 1);
            mbar_init(&bar.vempty[i], TWO ? 2 : 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.sfull[i], 1);
            mbar_init(&bar.pready[i][0], 4);
            mbar_init(&bar.pready[i][1], 4);
            mbar_init(&bar.odone[i], 1);
            mbar_init(&bar.turn[i], 1);
        }
        fence_barrier_init();
        static_cast<AttnMeta*>(a.ws)[blockIdx.x].rows = 0;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    {
        const AttnShare sh = attn_find_share<kThreads>(a, S::kRows, kTok, kOver, s_find);  // barriers inside
        if (threadIdx.x == 0) {
            s_share = sh;
            s_u = sh.start;
            next_seg<D, TWO>(a, s_share, s_u, s_seg[0]);
        }
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    // q takes the scale's sign; a scale of 0 stays one that keeps -inf apart
    const bool minus = a.scale < 0.f;
    const float c = fmaxf(fabsf(a.scale), 1e-30f) * kAttnLog2e;

    bool ok = true;
    uint32_t blocks = 0;              // K (and V) blocks before this item
    uint32_t steps_done[2] = {0, 0};  // softmax steps of the slots before this item
    uint32_t items_done[2] = {0, 0};  // items with a step, per slot
    uint32_t turns[2] = {0, 0};       // turns that the slots have handed on
    auto advance = [&](int n, int steps0, int steps1) {
        blocks += n;
        steps_done[0] += steps0;
        steps_done[1] += steps1;
        items_done[0] += steps0 > 0;
        items_done[1] += steps1 > 0;
        turns[0] += steps0 > 0 ? steps0 + 1 : 0;
        turns[1] += steps1 > 0 ? steps1 + 1 : 0;
    };
    // The softmax holds a block's scores and more; the other warps need few registers. 128 x 128 + 256 x 184 of the
    // 384 x 168 that the block has.
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 128;");
        for (int cur = 0; !s_seg[cur].skip; cur ^= 1) {
            Seg& g = s_seg[cur];
            const int n = g.n, steps0 = g.steps[0], steps1 = g.steps[1];
            if (warp != 0 && warp != 3) named_sync(2, kThreads - 64);  // the loads need not wait for q
            if (warp == 0 || warp == 3) {
                // ------------------------------------------------ loads of K (warp 0) or V (warp 3)
                const bool is_v = warp == 3;
                const uint32_t stages = is_v ? S::kVS : S::kKS, ring = is_v ? v_at : k_at;
                const CUtensorMap* map = is_v ? &map_v : &map_k;
                const int br = min(a.cache.page_size, kTok), nbox = kTok / br;  // tokens per box, boxes per block
                const int32_t* table = a.table + g.table;
                auto entry = [&](int rel) -> int {
                    return lane < nbox && rel < g.len ? table[(g.l0 + rel) >> a.page_shift] : -1;
                };
                int rel = lane * br, next = entry(rel);
                for (int j = 0; j < n; ++j, rel += kTok) {
                    const int page = next >= 0 && next < a.cache.num_pages ? next : -1;
                    const int at = static_cast<int>((g.l0 + rel) & (a.cache.page_size - 1));
                    next = entry(rel + kTok);
                    const uint32_t b = blocks + j, st = b % stages;
                    uint64_t* full = is_v ? &bar.vfull[st] : &bar.kfull[st];
                    uint64_t* empty = is_v ? &bar.vempty[st] : &bar.kempty[st];
                    if (b >= stages) ok = ok && mbar_wait_warp(empty, (b / stages - 1) & 1, &g_attn_error);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(full, S::kBlk);
                    __syncwarp();
                    if (lane < nbox) {
                        const uint32_t dst = ring + st * S::kBlk + lane * br * 128;
#pragma unroll
                        for (int d = 0; d < D / 64; ++d) tma_load_4d(dst + d * (kTok * 128), map, 64 * d, at, g.h, page, full);
                    }
                    __syncwarp();
                }
                if (threadIdx.x == 0) next_seg<D, TWO>(a, s_share, s_u, s_seg[cur ^ 1]);  // beside the item's products
            } else if (warp < 3) {
                // ------------------------------------------------ products of slot warp - 1, by one thread
                const int t = warp - 1, steps = t ? steps1 : steps0;
                if (lane == 0 && steps > 0) {
                    const uint32_t id = (1u << 4) | (1u << 7) | (1u << 10) | (8u << 24);  // f32 D, bf16 A and B, M = 128
                    const uint32_t id_s = id | (static_cast<uint32_t>(kTok >> 3) << 17);
                    const uint32_t id_o = id | (1u << 16) | (static_cast<uint32_t>(D >> 3) << 17);  // B MN-major
                    // descriptors advance by addresses / 16, all below 2^14
                    const uint64_t q_desc = desc_sw128(q_at + (TWO ? t : 0) * S::kQTile, 16), k_desc = desc_sw128(k_at, 16);
                    const uint64_t v_desc = desc_sw128(v_at, kTok * 128);
                    const uint32_t s_col = tmem + 128 * t, o_col = tmem + 256 + t * D;
                    const bool alone = TWO && steps1 == 0;  // the other slot's arrivals are this one's
                    // turn u of slot 0 follows turn u - 1 of slot 1, which follows turn u - 1 of slot 0
                    auto my_turn = [&](int u) {
                        if (steps1 > 0 && (t == 1 || u > 0))
                            ok = ok && mbar_wait(&bar.turn[t], (turns[1 - t] + (t ? u : u - 1)) & 1, &g_attn_error);
                    };
                    auto values = [&](int i) {  // o += p v of step i
                        const uint32_t b = blocks + (TWO ? i : 2 * i + t), st = b % S::kVS, ph = (steps_done[t] + i) & 1;
                        const uint64_t vd = v_desc + st * (S::kBlk >> 4);
                        ok = ok && mbar_wait(&bar.vfull[st], (b / S::kVS) & 1, &g_attn_error);
#pragma unroll
                        for (int f = 1; f >= 0; --f) {  // p's second half comes first
                            ok = ok && mbar_wait(&bar.pready[t][f], ph, &g_attn_error);
                            if (f == 1) my_turn(i + 1);
                            if (!ok) return;
                            tc_fence_after();
#pragma unroll
                            for (int k = 4 * f; k < 4 * f + 4; ++k)
                                mma_ts(o_col, s_col + 64 * f + 8 * (k & 3), vd + (k * 2048 >> 4), id_o,
                                       i == 0 && k == 4 ? 0u : 1u);
                        }
                        mma_commit(&bar.vempty[st]);
                        if (alone) mma_commit(&bar.vempty[st]);
                    };
                    for (int i = 0; i < steps; ++i) {
                        const uint32_t b = blocks + (TWO ? i : 2 * i + t), st = b % S::kKS;
                        ok = ok && mbar_wait(&bar.kfull[st], (b / S::kKS) & 1, &g_attn_error);
                        if (i > 0)
                            values(i - 1);
                        else
                            my_turn(0);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t kd = k_desc + st * (S::kBlk >> 4);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const uint32_t off = ((k / 4) * (128 * 128) + (k % 4) * 32) >> 4;
                            mma_ss(s_col, q_desc + off, kd + off, id_s, k ? 1u : 0u);
                        }
                        mma_commit(&bar.sfull[t]);
                        mbar_arrive(&bar.turn[1 - t]);
                        mma_commit(&bar.kempty[st]);
                        if (alone) mma_commit(&bar.kempty[st]);
                    }
                    if (ok) values(steps - 1);
                    if (ok) {
                        mma_commit(&bar.odone[t]);
                        mbar_arrive(&bar.turn[1 - t]);
                    }
                }
                __syncwarp();
                ok = __shfl_sync(0xFFFFFFFFu, ok ? 1 : 0, 0) != 0;
            }
            advance(n, steps0, steps1);
            __syncthreads();  // all have read g and their own of the item
        }
        if (!ok) let_copies_land();
        __syncthreads();
        if (warp == 1) {
            tc_fence_after();
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        for (int cur = 0; !s_seg[cur].skip; cur ^= 1) {
            Seg& g = s_seg[cur];
            const int n = g.n, steps0 = g.steps[0], steps1 = g.steps[1];
            const int slot = warp >= 8 ? 1 : 0, quarter = warp % 4;  // of the softmax warps
            const int row = 32 * quarter + lane;                     // tensor-memory lane of the thread
            const int rows_s = TWO ? min(max(g.rows - 128 * slot, 0), 128) : g.rows;
            const bool live = row < rows_s;
            const uint32_t grow = live ? static_cast<uint32_t>(g.tile) * S::kRows + (TWO ? 128 * slot : 0) + row : 0u;
            const int qi = static_cast<int>(grow / static_cast<uint32_t>(g.group));
            const int head = g.h * g.group + static_cast<int>(grow) - qi * g.group;
            // q into shared memory; pages all right? (the first read of them ahead of q)
            const int64_t p0 = (g.l0 >> a.page_shift) + (threadIdx.x - 128), p1 = (g.l0 + g.len - 1) >> a.page_shift;
            const int32_t e0 = n > 0 && p0 <= p1 ? a.table[g.table + p0] : 0;
            if (TWO || slot == 0) {
                // a row's 16 bytes a lane, all loads ahead of the writes
                constexpr int kCh = D / 8, kAt = kWarp / kCh, kBatch = kWarp / kAt;
                const int ch = lane % kCh;
                uint8_t* dst = sm + (TWO ? slot : 0) * S::kQTile + (ch / 8) * (128 * 128);
                uint4 x[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int r = i * kAt + lane / kCh;
                    const int tok = __shfl_sync(0xFFFFFFFFu, qi, r), hd = __shfl_sync(0xFFFFFFFFu, head, r);
                    x[i] = make_uint4(0, 0, 0, 0);
                    if (32 * quarter + r < rows_s)
                        x[i] = *reinterpret_cast<const uint4*>(a.q + (g.o0 + static_cast<int64_t>(tok)) * a.q_pitch +
                                                               static_cast<int64_t>(hd) * D + 8 * ch);
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int r = 32 * quarter + i * kAt + lane / kCh;
                    if (minus) x[i].x ^= 0x80008000u, x[i].y ^= 0x80008000u, x[i].z ^= 0x80008000u, x[i].w ^= 0x80008000u;
                    *reinterpret_cast<uint4*>(dst + r * 128 + (((ch % 8) ^ (r & 7)) << 4)) = x[i];
                }
                fence_async();
            }
            bool bad = e0 < 0 || e0 >= a.cache.num_pages;
            for (int64_t p = p0 + 256; n > 0 && p <= p1; p += 256) {
                const int32_t e = a.table[g.table + p];
                bad |= e < 0 || e >= a.cache.num_pages;
            }
            if (bad) g.bad = 1;
            named_sync(2, kThreads - 64);
            // ------------------------------------------------ softmax
            const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
            const uint32_t s_at = tmem + lanes + 128 * slot, o_at = tmem + lanes + 256 + slot * D;
            const bool busy = 32 * quarter < rows_s;  // the warp has a live row
            float m = -INFINITY, z = 0.f;
            {
                const int steps = slot ? steps1 : steps0;
                const int all_seen = *static_cast<volatile int*>(&g.bad) ? 0 : g.plain / kTok;  // blocks that every row sees whole
                const uint32_t phase0 = steps_done[slot];
                for (int i = 0; i < steps; ++i) {
                    const int j = TWO ? i : 2 * i + slot;
                    ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(&bar.sfull[slot], (phase0 + i) & 1, &g_attn_error));
                    if (!ok) break;
                    tc_fence_after();
                    uint4 see = make_uint4(~0u, ~0u, ~0u, ~0u);
                    const bool special = j >= all_seen;
                    if (special) {
                        const uint32_t b = blocks + j, st = b % S::kVS;
                        ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(&bar.vfull[st], (b / S::kVS) & 1, &g_attn_error));
                        if (!ok) break;
                        see = special_block<D>(a, g, j, 32 * quarter, g.o0 + static_cast<int64_t>(qi), qi,
                                               sm + (v_at - base) + st * S::kBlk, &g.odd);
                    }
                    if (busy) {
                        // 64 scores at a time: all 128 would not fit beside the rest. The second half is still held
                        // when the maximum is known, so its p comes first; p of a half lies over its own scores.
                        uint32_t s[64];
                        auto scores = [&](int half) {
                            tmem_ld(s_at + 64 * half, s);
                            tmem_ld(s_at + 64 * half + 32, s + 32);
                            tmem_ld_wait();
                            if (special) {
                                const uint32_t lo = half ? see.z : see.x, hi = half ? see.w : see.y;
#pragma unroll
                                for (int e = 0; e < 32; ++e) {
                                    if (!((lo >> e) & 1)) s[e] = 0xFF800000u;
                                    if (!((hi >> e) & 1)) s[32 + e] = 0xFF800000u;
                                }
                            }
                        };
                        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            scores(k);
#pragma unroll
                            for (int e = 0; e < 64; ++e) top[e & 3] = fmaxf(top[e & 3], __uint_as_float(s[e]));
                        }
                        const float mn = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c;
                        const bool grown = m != -INFINITY && mn > m + kGrow;
                        const bool far = fabsf(mn) >= kHuge && mn != -INFINITY;
                        bool plain = true;
                        if (__any_sync(0xFFFFFFFFu, grown || far)) {
                            const float f = grown ? attn_ex2(m - mn) : 1.f;
                            z *= f;
                            rescale<D>(o_at, f);
                            plain = !__any_sync(0xFFFFFFFFu, far);
                        }
                        if (grown || m == -INFINITY) m = mn;
                        if (!plain) {
                            z += far_block(s_at, see, c, m, bar.pready[slot]);
                            continue;
                        }
                        const float sub = m == -INFINITY ? 0.f : -m;
                        const uint64_t cc = pack(c, c), ss = pack(sub, sub);
                        uint64_t z0 = 0, z1 = 0;
#pragma unroll
                        for (int k = 1; k >= 0; --k) {
                            uint32_t p[32];
                            if (k == 0) scores(0);
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                float x, y;
                                unpack(fma2(pack(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), cc, ss), x, y);
                                x = attn_ex2(x);
                                y = attn_ex2(y);
                                if (e & 1)
                                    z1 = add2(z1, pack(x, y));
                                else
                                    z0 = add2(z0, pack(x, y));
                                p[e] = attn_bf16x2(x, y);
                            }
                            tmem_st(s_at + 64 * k, p);
                            tmem_st_wait();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bar.pready[slot][k]);
                        }
                        float x, y;
                        unpack(add2(z0, z1), x, y);
                        z += x + y;
                    } else {
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&bar.pready[slot][1]);
                            mbar_arrive(&bar.pready[slot][0]);
                        }
                    }
                }
            }

            // ---- the item's end
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if ((TWO ? t == slot : true) && (t ? steps1 : steps0) > 0)
                    ok = ok && mbar_wait_warp(&bar.odone[t], items_done[t] & 1, &g_attn_error);
            tc_fence_after();
            float* join = reinterpret_cast<float*>(sm + (k_at - base));  // over the ring, which nothing reads or fills now
            if (!TWO) {
                if (slot == 1 && busy && steps1 > 0) {
                    for (int k = 0; k < D / 32; ++k) {
                        uint32_t o[32];
                        tmem_ld(o_at + 32 * k, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<uint4*>(join + row * S::kPitch + 32 * k + e) =
                                make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                }
                if (slot == 1) {
                    s_mz[TWO ? 0 : row][0] = m;
                    s_mz[TWO ? 0 : row][1] = z;
                }
                named_sync(1, 256);
            }
            if (busy && (TWO || slot == 0)) {
                const bool other = !TWO && steps1 > 0;
                float f0 = 1.f, f1 = 0.f;
                if (other) {
                    const float m1 = s_mz[TWO ? 0 : row][0], mm = fmaxf(m, m1);
                    f0 = attn_weight(m, mm);
                    f1 = attn_weight(m1, mm);
                    z = z * f0 + s_mz[TWO ? 0 : row][1] * f1;
                    m = mm;
                }
                const bool whole = g.parts < 0;
                const int64_t qt = g.o0 + static_cast<int64_t>(qi), at = qt * a.Hq + head;
                const int prow = (TWO ? 128 * slot : 0) + row;
                float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + attn_meta_bytes()) + g.parts;
                const bool odd = *static_cast<volatile int*>(&g.odd) != 0;
                for (int k = 0; k < D / 32; ++k) {
                    uint32_t o[32];
                    if (steps0 > 0) {  // a slot that is busy has steps if the other has
                        tmem_ld(o_at + 32 * k, o);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0;
                    }
                    if (other) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 y = *reinterpret_cast<const float4*>(join + row * S::kPitch + 32 * k + e);
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * f0 + y.x * f1);
                            o[e + 1] = __float_as_uint(__uint_as_float(o[e + 1]) * f0 + y.y * f1);
                            o[e + 2] = __float_as_uint(__uint_as_float(o[e + 2]) * f0 + y.z * f1);
                            o[e + 3] = __float_as_uint(__uint_as_float(o[e + 3]) * f0 + y.w * f1);
                        }
                    }
                    if (!live) continue;
                    if (odd) {  // the drafts' elements that are not finite, for the rows that see them
                        for (int rel = max(0, g.ctx); rel < g.len; ++rel) {
                            const int64_t l = g.l0 + rel;
                            const int32_t e = a.table[g.table + (l >> a.page_shift)];
                            if (e < 0 || e >= a.cache.num_pages || !attn_sees(a, qt, qi, rel - g.ctx)) continue;
                            const uint16_t* v = static_cast<const uint16_t*>(a.cache.v) + e * a.cache.page_stride +
                                                (l & (a.cache.page_size - 1)) * a.cache.token_stride +
                                                g.h * a.cache.head_stride + 32 * k;
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                if ((v[x] & 0x7F80u) == 0x7F80u)
                                    o[x] = __float_as_uint(__uint_as_float(o[x]) +
                                                           __uint_as_float(static_cast<uint32_t>(v[x]) << 16));
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        if (whole) {
                            const uint2 lo = attn_out4(make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                                                   __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3])),
                                                       z, 1.f);
                            const uint2 hi = attn_out4(make_float4(__uint_as_float(o[e + 4]), __uint_as_float(o[e + 5]),
                                                                   __uint_as_float(o[e + 6]), __uint_as_float(o[e + 7])),
                                                       z, 1.f);
                            *reinterpret_cast<uint4*>(a.out + at * D + 32 * k + e) = make_uint4(lo.x, lo.y, hi.x, hi.y);
                        } else {
                            // column by column: the rows of a warp are adjacent
#pragma unroll
                            for (int i = 0; i < 8; ++i) part[(32 * k + e + i) * S::kRows + prow] = __uint_as_float(o[e + i]);
                        }
                    }
                }
                if (live && whole && a.lse) a.lse[at] = attn_lse(m, z, 0.f);
                if (live && !whole) {
                    part[S::kRows * D + prow] = m;
                    part[S::kRows * D + S::kRows + prow] = z;
                }
            }
            tc_fence_before();
            fence_async();  // the join's memory goes back to the copies
            advance(n, steps0, steps1);
            __syncthreads();
        }
        if (!ok) let_copies_land();
        __syncthreads();
    }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
        cudaGetLastError();
    });
    return fn;
}

// K or V as (d, token of the page, head, page), boxes of 64 d x min(page,
// 128) tokens. A dimension of one element may have any stride.
bool make_map(CUtensorMap* map, const bqd_kv_cache& c, void* base)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.head_dim), static_cast<cuuint64_t>(c.page_size),
                                static_cast<cuuint64_t>(c.heads), static_cast<cuuint64_t>(c.num_pages)};
    const cuuint64_t row = static_cast<cuuint64_t>(c.head_dim) * 2;
    const cuuint64_t strides[3] = {c.page_size > 1 ? static_cast<cuuint64_t>(c.token_stride) * 2 : row,
                                   c.heads > 1 ? static_cast<cuuint64_t>(c.head_stride) * 2 : row,
                                   c.num_pages > 1 ? static_cast<cuuint64_t>(c.page_stride) * 2 : row};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(c.page_size < kTok ? c.page_size : kTok), 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Mean rows per kv head of a request.
bool wide_two(int64_t R, int64_t T, int Hq, int Hkv) { return T * (Hq / Hkv) > 128 * R; }

template <int D, bool TWO>
cudaError_t launch(const AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s)
{
    using S = Wide<D, TWO>;
    static OccCache occ;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    blocks_per_sm(occ, reinterpret_cast<const void*>(&tree_attn_wide_kernel<D, TWO>), dev, kThreads, S::kSmem);
    tree_attn_wide_kernel<D, TWO><<<kGrid, kThreads, S::kSmem, s>>>(a, mk, mv);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_attn_join(tree_attn_join_columns_kernel<D, S::kRows>, a, kGrid, s);
}

}  // namespace

// From a mean of 33 rows per kv head. Up to 32 rows, one tile of the narrow
// kernel holds a request, and its shorter pipeline reads faster: 16 requests of
// 24 rows over 8192 tokens take it 77 us, this kernel 87 (1000 tokens: 25 and
// 32). Above, the narrow one reads keys and values once per tile: with 48 rows
// 126 us against 95 here, with 512 rows (four contexts of 32768 tokens) 934
// against 191.
bool tree_attention_wide_fits(const AttnArgs& a)
{
    const bqd_kv_cache& c = a.cache;
    // tensor copies take strides of 16 bytes and more, below 2^40
    auto stride_ok = [](int64_t count, int64_t s) { return count <= 1 || (s > 0 && s < (int64_t(1) << 39)); };
    if (!stride_ok(c.page_size, c.token_stride) || !stride_ok(c.heads, c.head_stride) ||
        !stride_ok(c.num_pages, c.page_stride))
        return false;
    return c.type == BQD_BF16 && (c.head_dim == 64 || c.head_dim == 128) && c.page_size >= 8 && c.num_pages >= 1 &&
           c.num_pages < (int64_t(1) << 31) && a.T * a.group > 32 * a.R;
}

size_t tree_attention_wide_ws(int64_t T, int Hq, int Hkv, int D)
{
    if (D > 128) return 0;
    return attn_meta_bytes() + 2 * kGrid * attn_part_floats(wide_two(1, T, Hq, Hkv) ? 256 : 128, D) * sizeof(float);
}

cudaError_t launch_tree_attention_wide(const AttnArgs& a, cudaStream_t s)
{
    CUtensorMap mk, mv;
    if (!make_map(&mk, a.cache, a.cache.k) || !make_map(&mv, a.cache, a.cache.v)) return cudaErrorInvalidValue;
    const bool two = wide_two(a.R, a.T, a.Hq, a.cache.heads);
    if (a.cache.head_dim == 64) return two ? launch<64, true>(a, mk, mv, s) : launch<64, false>(a, mk, mv, s);
    return two ? launch<128, true>(a, mk, mv, s) : launch<128, false>(a, mk, mv, s);
}

cudaError_t read_and_clear_attn_error(unsigned int* out)
{
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_attn_error, sizeof(v));
    if (e != cudaSuccess) return e;
    *out = v;
    if (v) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_attn_error, &zero, sizeof(zero));
    }
    return e;
}

}  // namespace bqd
