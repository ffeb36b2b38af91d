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
// Warp 0 loads K and V blocks by 4-D tensor copies, one box per page and 64
// elements of D (128-byte swizzle; pages outside the cache read as zero);
// warp 1 issues, per block and slot, s = q k^T (both from shared memory,
// K-major) and o += p v with p from tensor memory and v MN-major, the
// previous block's o of a slot before its next s. Warps 4..7 and 8..11 are
// the slots' softmax, a row per thread (tensor-memory lane): they read s,
// write p in bf16 over the columns of s that they have read, and rescale o in
// tensor memory only when a row's maximum has grown by more than 2^8 (p then
// stays below 2^8, and nothing is lost: fp32 sums, bf16's range).
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
constexpr float kGrow = 8.f;

template <int D, bool TWO>
struct Wide {
    static constexpr int kRows = TWO ? 256 : 128;
    static constexpr int kQTile = 128 * D * 2;
    static constexpr int kBlk = kTok * D * 2;  // bytes of a K or V block
    static constexpr int kKS = D == 64 ? 4 : TWO ? 2 : 3;
    static constexpr int kVS = D == 64 ? 4 : 2;
    static constexpr int kQBytes = (TWO ? 2 : 1) * kQTile;
    static constexpr int kSmem = kQBytes + (kKS + kVS) * kBlk + 1024;  // + alignment slack
    static constexpr int kPitch = D + 4;  // floats of a row in the slots' join
    static_assert(kSmem <= 227 * 1024 - 1024, "shared memory of one CTA");
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

#define BQD_R32(v)                                                                                                  \
    v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], v[8], v[9], v[10], v[11], v[12], v[13], v[14], v[15], v[16],    \
        v[17], v[18], v[19], v[20], v[21], v[22], v[23], v[24], v[25], v[26], v[27], v[28], v[29], v[30], v[31]

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
#undef BQD_R32

__device__ __forceinline__ bool elect_one()
{
    uint32_t pred = 0;
    asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(pred));
    return pred != 0;
}

// Bits e = 0 .. 31: whether token i of the request (t of the call) sees draft
// j0 + e (negative: cached).
__device__ __forceinline__ uint32_t sees32(const AttnArgs& a, int64_t t, int i, int64_t j0)
{
    if (j0 <= -32) return 0xFFFFFFFFu;
    if (!a.mask) {
        const int64_t last = i - j0;  // bits 0 .. last
        return last < 0 ? 0u : last >= 31 ? 0xFFFFFFFFu : (2u << last) - 1u;
    }
    const uint64_t* m = a.mask + t * a.mask_words;
    if (j0 < 0) {
        const int k = static_cast<int>(-j0);  // bits 0 .. k - 1 are cached tokens
        return ((1u << k) - 1u) | static_cast<uint32_t>(m[0] << k);
    }
    const int64_t w = j0 >> 6;
    const int b = static_cast<int>(j0 & 63);
    uint64_t v = w < a.mask_words ? m[w] >> b : 0;
    if (b > 32 && w + 1 < a.mask_words) v |= m[w + 1] << (64 - b);
    return static_cast<uint32_t>(v);
}

struct Bars {
    uint64_t kfull[4], kempty[4], vfull[4], vempty[4], sfull[2], pready[2], odone[2];
};

template <int D, bool TWO>
__global__ void __launch_bounds__(kThreads, 1)
    tree_attn_wide_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_v)
{
    using S = Wide<D, TWO>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) Bars bar;
    __shared__ int64_t s_find[kThreads / kWarp + 2];
    __shared__ uint32_t s_tmem;
    __shared__ int s_odd;
    __shared__ float s_mz[128][2];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* const sm = smem_raw + (base - smem_u32(smem_raw));
    const uint32_t q_at = base, k_at = base + S::kQBytes, v_at = k_at + S::kKS * S::kBlk;
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
    const int G = a.Hq / a.cache.heads;
    const int shift = 31 - __clz(a.cache.page_size);
    const int br = min(a.cache.page_size, kTok), nbox = kTok / br;  // tokens per box, boxes per block

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join waits for this grid's end
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bar.kfull[i], 1);
            mbar_init(&bar.kempty[i], 1);
            mbar_init(&bar.vfull[i], 1);
            mbar_init(&bar.vempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.sfull[i], 1);
            mbar_init(&bar.pready[i], 4);
            mbar_init(&bar.odone[i], 1);
        }
        fence_barrier_init();
        static_cast<AttnMeta*>(a.ws)[blockIdx.x].r = -1;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    AttnShare sh = attn_find_share<kThreads>(a, S::kRows, kTok, s_find);  // barriers inside
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + attn_meta_bytes());
    // q takes the scale's sign; a scale of 0 stays one that keeps -inf apart
    const bool minus = a.scale < 0.f;
    const float c = fmaxf(fabsf(a.scale), 1e-30f) * kAttnLog2e;

    bool ok = true;
    uint32_t blocks = 0;            // K (and V) blocks before this item
    uint32_t steps_done[2] = {0, 0};  // softmax steps of the slots before this item
    uint32_t items_done[2] = {0, 0};  // items with a step, per slot
    int64_t u = sh.start;
    while (u < sh.end) {
        const AttnReq q = attn_request(a, sh.r, S::kRows, kTok);
        const int64_t item = (u - sh.base) / q.nb, b0 = (u - sh.base) % q.nb, cnt = min(q.nb - b0, sh.end - u);
        const int h = static_cast<int>(item / q.tiles), tile = static_cast<int>(item % q.tiles);
        const int64_t l0 = b0 * kTok, l1 = min((b0 + cnt) * kTok, q.len);
        const int n = l1 > l0 ? static_cast<int>((l1 - l0 + kTok - 1) / kTok) : 0;
        const int32_t* table = a.table + sh.r * a.width;
        const int rows = static_cast<int>(min(static_cast<int64_t>(q.n) * G - static_cast<int64_t>(tile) * S::kRows,
                                              static_cast<int64_t>(S::kRows)));
        const bool live1 = !TWO || rows > 128;
        const int steps0 = TWO ? n : (n + 1) / 2, steps1 = TWO ? (live1 ? n : 0) : n / 2;
        const int slot = warp >= 8 ? 1 : 0, quarter = warp % 4;  // of the softmax warps
        const int row = 32 * quarter + lane;                     // tensor-memory lane of the thread
        const int rows_s = TWO ? min(max(rows - 128 * slot, 0), 128) : rows;
        const int64_t grow = static_cast<int64_t>(tile) * S::kRows + (TWO ? 128 * slot : 0) + row;
        const bool live = row < rows_s;
        const int qi = live ? static_cast<int>(grow / G) : 0;
        const int64_t qt = q.o0 + qi;
        const int head = h * G + (live ? static_cast<int>(grow % G) : 0);

        // pages all right? q into shared memory
        bool bad = false;
        if (n > 0)
            for (int64_t p = (l0 >> shift) + threadIdx.x; p <= (l1 - 1) >> shift; p += kThreads)
                bad |= table[p] < 0 || table[p] >= a.cache.num_pages;
        if (warp >= 4 && (TWO || slot == 0)) {
            const uint16_t* src = a.q + qt * a.q_pitch + static_cast<int64_t>(head) * D;
            uint8_t* dst = sm + (TWO ? slot : 0) * S::kQTile + row * 128;
#pragma unroll
            for (int ch = 0; ch < D / 8; ++ch) {
                uint4 x = live ? *reinterpret_cast<const uint4*>(src + 8 * ch) : make_uint4(0, 0, 0, 0);
                if (minus) x.x ^= 0x80008000u, x.y ^= 0x80008000u, x.z ^= 0x80008000u, x.w ^= 0x80008000u;
                *reinterpret_cast<uint4*>(dst + (ch / 8) * (128 * 128) + (((ch % 8) ^ (row & 7)) << 4)) = x;
            }
            fence_async();
        }
        if (threadIdx.x == 0) s_odd = 0;
        bad = __syncthreads_or(bad);

        if (warp == 0) {
            // ------------------------------------------------ loads
            auto entry = [&](int64_t l) -> int { return lane < nbox && l < l1 ? table[l >> shift] : -1; };
            int64_t l = l0 + lane * br;
            int next = entry(l);
            for (int j = 0; j < n && ok; ++j, l += kTok) {
                const int e = next;
                next = entry(l + kTok);
                const int page = e >= 0 && e < a.cache.num_pages ? e : -1;
                const int at = static_cast<int>(l & (a.cache.page_size - 1));
                const uint32_t b = blocks + j;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const uint32_t stages = kv ? S::kVS : S::kKS, st = b % stages;
                    uint64_t* full = kv ? &bar.vfull[st] : &bar.kfull[st];
                    uint64_t* empty = kv ? &bar.vempty[st] : &bar.kempty[st];
                    if (b >= stages) ok = ok && mbar_wait_warp(empty, (b / stages - 1) & 1, &g_attn_error);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(full, S::kBlk);
                    __syncwarp();
                    if (lane < nbox) {
                        const uint32_t dst = (kv ? v_at : k_at) + st * S::kBlk + lane * br * 128;
#pragma unroll
                        for (int d = 0; d < D / 64; ++d)
                            tma_load_4d(dst + d * (kTok * 128), kv ? &map_v : &map_k, 64 * d, at, h, page, full);
                    }
                    __syncwarp();
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------ products
            const uint32_t id = (1u << 4) | (1u << 7) | (1u << 10) | (8u << 24);  // f32 D, bf16 A and B, M = 128
            const uint32_t id_s = id | (static_cast<uint32_t>(kTok >> 3) << 17);
            const uint32_t id_o = id | (1u << 16) | (static_cast<uint32_t>(D >> 3) << 17);  // B MN-major
            int pend[2] = {-1, -1};
            uint32_t used[2] = {steps_done[0], steps_done[1]};  // p blocks taken
            auto values = [&](int t) {  // o of slot t += p v of its pending block
                const uint32_t b = blocks + pend[t], st = b % S::kVS;
                ok = ok && mbar_wait_warp(&bar.pready[t], used[t] & 1, &g_attn_error) &&
                     mbar_wait_warp(&bar.vfull[st], (b / S::kVS) & 1, &g_attn_error);
                ++used[t];
                if (!ok) return;
                tc_fence_after();
                if (elect_one()) {
                    const bool first = TWO ? pend[t] == 0 : pend[t] == t;
#pragma unroll
                    for (int k = 0; k < kTok / 16; ++k)
                        mma_ts(tmem + 256 + t * D, tmem + 128 * t + 8 * k,
                               desc_sw128(v_at + st * S::kBlk + k * 2048, kTok * 128), id_o, first && k == 0 ? 0u : 1u);
                    if (!TWO || t == (live1 ? 1 : 0)) mma_commit(&bar.vempty[st]);
                }
                __syncwarp();
            };
            for (int j = 0; j < n && ok; ++j) {
                const uint32_t b = blocks + j, st = b % S::kKS;
                ok = ok && mbar_wait_warp(&bar.kfull[st], (b / S::kKS) & 1, &g_attn_error);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (TWO ? (t == 1 && !live1) : (j & 1) != t) continue;
                    if (pend[t] >= 0) values(t);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const uint32_t off = (k / 4) * (128 * 128) + (k % 4) * 32;
                            mma_ss(tmem + 128 * t, desc_sw128(q_at + (TWO ? t : 0) * S::kQTile + off, 16),
                                   desc_sw128(k_at + st * S::kBlk + off, 16), id_s, k ? 1u : 0u);
                        }
                        mma_commit(&bar.sfull[t]);
                    }
                    __syncwarp();
                    pend[t] = j;
                }
                if (ok && elect_one()) mma_commit(&bar.kempty[st]);
                __syncwarp();
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = TWO ? i : (n & 1) ^ i;  // the older block first
                if (pend[t] < 0) continue;
                if (ok) {
                    if (t == 0)
                        values(0);
                    else
                        values(1);
                }
                if (ok && elect_one()) mma_commit(&bar.odone[t]);
                __syncwarp();
            }
        } else if (warp >= 4) {
            // ------------------------------------------------ softmax
            const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
            const uint32_t s_at = tmem + lanes + 128 * slot, o_at = tmem + lanes + 256 + slot * D;
            const int steps = slot ? steps1 : steps0;
            const bool busy = 32 * quarter < rows_s;  // the warp has a live row
            const int64_t plain = min(q.ctx, q.len);  // tokens that every row sees
            float m = -INFINITY, z = 0.f;
            for (int i = 0; i < steps; ++i) {
                const int j = TWO ? i : 2 * i + slot;
                const int64_t l = l0 + static_cast<int64_t>(j) * kTok;
                ok = ok && mbar_wait_warp(&bar.sfull[slot], (steps_done[slot] + i) & 1, &g_attn_error);
                if (!ok) break;
                tc_fence_after();
                const bool special = bad || l + kTok > plain;
                uint32_t pages = 0;  // which boxes are tokens
                if (special) {
                    const int64_t lb = l + lane * br;
                    const int e = lane < nbox && lb < l1 ? table[lb >> shift] : -1;
                    pages = __ballot_sync(0xFFFFFFFFu, e >= 0 && e < a.cache.num_pages);
                    if (!TWO || slot == 0) {
                        // V row `row` of the block: cleared where it is no token, or not finite
                        const uint32_t b = blocks + j, st = b % S::kVS;
                        ok = ok && mbar_wait_warp(&bar.vfull[st], (b / S::kVS) & 1, &g_attn_error);
                        uint8_t* v = sm + (v_at - base) + st * S::kBlk + row * 128;
                        const bool token = l + row < q.len && ((pages >> (row / br)) & 1);
                        if (!token || l + row >= q.ctx) {
                            for (int ch = 0; ch < D / 8; ++ch) {
                                uint4* p = reinterpret_cast<uint4*>(v + (ch / 8) * (kTok * 128) + (ch % 8) * 16);
                                uint4 x = *p;
                                uint32_t w[4] = {x.x, x.y, x.z, x.w};
                                bool change = !token;
#pragma unroll
                                for (int y = 0; y < 4; ++y) {
                                    const bool lo = (w[y] & 0x7F80u) == 0x7F80u, hi = (w[y] & 0x7F800000u) == 0x7F800000u;
                                    change |= lo || hi;
                                    if (!token) w[y] = 0;
                                    if (lo) w[y] &= 0xFFFF0000u;
                                    if (hi) w[y] &= 0xFFFFu;
                                }
                                if (change) {
                                    *p = make_uint4(w[0], w[1], w[2], w[3]);
                                    if (token) s_odd = 1;
                                }
                            }
                        }
                        fence_async();
                    }
                }
                if (busy) {
                    uint32_t see[4];  // a special block's visible tokens
                    if (special) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            see[k] = sees32(a, qt, qi, l + 32 * k - q.ctx);
                            const int64_t left = q.len - (l + 32 * k);
                            if (left < 32) see[k] &= left <= 0 ? 0u : (1u << left) - 1u;
                            uint32_t real = 0;
                            if (br >= 32)
                                real = ((pages >> (32 * k / br)) & 1) ? 0xFFFFFFFFu : 0u;
                            else
                                for (int e = 0; e < 32; ++e) real |= ((pages >> ((32 * k + e) / br)) & 1) << e;
                            see[k] &= real;
                        }
                    }
                    // the scores are read twice, 64 at a time: all 128 would not fit beside the rest
                    auto scores = [&](int half, uint32_t (&s)[64]) {
                        tmem_ld(s_at + 64 * half, s);
                        tmem_ld(s_at + 64 * half + 32, s + 32);
                        tmem_ld_wait();
                        if (special)
#pragma unroll
                            for (int k = 0; k < 2; ++k)
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (!((see[2 * half + k] >> e) & 1)) s[32 * k + e] = 0xFF800000u;
                    };
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t s[64];
                        scores(k, s);
#pragma unroll
                        for (int e = 0; e < 64; ++e) top[e & 3] = fmaxf(top[e & 3], __uint_as_float(s[e]));
                    }
                    const float mn = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c;
                    const bool grown = m != -INFINITY && mn > m + kGrow;
                    if (__any_sync(0xFFFFFFFFu, grown)) {
                        const float f = grown ? attn_ex2(m - mn) : 1.f;
                        z *= f;
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
                    if (grown || m == -INFINITY) m = mn;
                    const float sub = m == -INFINITY ? 0.f : -m;
                    const uint64_t cc = pack(c, c), ss = pack(sub, sub);
                    uint64_t z0 = 0, z1 = 0;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t s[64], p[32];
                        scores(k, s);
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            float x, y;
                            unpack(fma2(pack(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), cc, ss),
                                   x, y);
                            x = attn_ex2(x);
                            y = attn_ex2(y);
                            if (e & 1)
                                z1 = add2(z1, pack(x, y));
                            else
                                z0 = add2(z0, pack(x, y));
                            p[e] = attn_bf16x2(x, y);
                        }
                        tmem_st(s_at + 32 * k, p);
                    }
                    float x, y;
                    unpack(add2(z0, z1), x, y);
                    z += x + y;
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.pready[slot]);
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
                    s_mz[row][0] = m;
                    s_mz[row][1] = z;
                }
                named_sync(1, 256);
            }
            if (busy && (TWO || slot == 0)) {
                const bool other = !TWO && steps1 > 0;
                float f0 = 1.f, f1 = 0.f;
                if (other) {
                    const float m1 = s_mz[row][0], mm = fmaxf(m, m1);
                    f0 = attn_weight(m, mm);
                    f1 = attn_weight(m1, mm);
                    z = z * f0 + s_mz[row][1] * f1;
                    m = mm;
                }
                const bool whole = b0 == 0 && cnt == q.nb;
                const int64_t at = qt * a.Hq + head;
                const int prow = (TWO ? 128 * slot : 0) + row;
                float* part = parts + (2 * blockIdx.x + (b0 == 0 ? 1 : 0)) * attn_part_floats(S::kRows, D);
                const bool odd = s_odd != 0;
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
                        for (int64_t l = max(l0, q.ctx); l < l1; ++l) {
                            const int32_t e = table[l >> shift];
                            if (e < 0 || e >= a.cache.num_pages || !attn_sees(a, qt, qi, l - q.ctx)) continue;
                            const uint16_t* v = static_cast<const uint16_t*>(a.cache.v) + e * a.cache.page_stride +
                                                (l & (a.cache.page_size - 1)) * a.cache.token_stride +
                                                h * a.cache.head_stride + 32 * k;
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                if ((v[x] & 0x7F80u) == 0x7F80u)
                                    o[x] = __float_as_uint(__uint_as_float(o[x]) +
                                                           __uint_as_float(static_cast<uint32_t>(v[x]) << 16));
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        const float4 x = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                                     __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
                        const float4 y = make_float4(__uint_as_float(o[e + 4]), __uint_as_float(o[e + 5]),
                                                     __uint_as_float(o[e + 6]), __uint_as_float(o[e + 7]));
                        if (whole) {
                            const uint2 lo = attn_out4(x, z, 1.f), hi = attn_out4(y, z, 1.f);
                            *reinterpret_cast<uint4*>(a.out + at * D + 32 * k + e) = make_uint4(lo.x, lo.y, hi.x, hi.y);
                        } else {
                            *reinterpret_cast<float4*>(part + prow * D + 32 * k + e) = x;
                            *reinterpret_cast<float4*>(part + prow * D + 32 * k + e + 4) = y;
                        }
                    }
                }
                if (live && whole && a.lse) a.lse[at] = attn_lse(m, z, 0.f);
                if (live && !whole) {
                    part[S::kRows * D + prow] = m;
                    part[S::kRows * D + S::kRows + prow] = z;
                }
                if (b0 == 0 && !whole && row == 0 && slot == 0)
                    static_cast<AttnMeta*>(a.ws)[blockIdx.x] = attn_meta(sh, h, tile, u + q.nb);
            }
            tc_fence_before();
            fence_async();  // the join's memory goes back to the copies
        }
        __syncthreads();
        blocks += n;
        steps_done[0] += steps0;
        steps_done[1] += steps1;
        items_done[0] += steps0 > 0;
        items_done[1] += steps1 > 0;
        u += cnt;
        if (u < sh.end) {
            int64_t next = sh.base + q.nb * q.tiles * a.cache.heads;
            while (u == next) {  // the next request with rows
                ++sh.r;
                sh.base = next;
                next += attn_units(a, sh.r, S::kRows, kTok);
            }
        }
    }
    if (warp == 0 && !ok) {  // a wait ran out: time for the copies in flight to land before the block ends
        const long long t0 = clock64();
        while (clock64() - t0 < (1ll << 27)) {
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
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
    return launch_attn_join<D, S::kRows, kTok, false>(a, kGrid, s);
}

}  // namespace

bool tree_attention_wide_fits(const AttnArgs& a)
{
    const bqd_kv_cache& c = a.cache;
    // tensor copies take strides of 16 bytes and more, below 2^40
    auto stride_ok = [](int64_t count, int64_t s) { return count <= 1 || (s > 0 && s < (int64_t(1) << 39)); };
    if (!stride_ok(c.page_size, c.token_stride) || !stride_ok(c.heads, c.head_stride) ||
        !stride_ok(c.num_pages, c.page_stride))
        return false;
    return c.type == BQD_BF16 && (c.head_dim == 64 || c.head_dim == 128) && c.page_size >= 8 && c.num_pages >= 1 &&
           c.num_pages < (int64_t(1) << 31) && a.T * (a.Hq / c.heads) > 64 * a.R;
}

size_t tree_attention_wide_ws(int64_t R, int64_t T, int Hq, int Hkv, int D)
{
    if (D > 128) return 0;
    return attn_meta_bytes() + 2 * kGrid * attn_part_floats(wide_two(R, T, Hq, Hkv) ? 256 : 128, D) * sizeof(float);
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
