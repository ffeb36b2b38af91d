// tree_attn.cu -- attention of drafted tokens (a chain or a tree; one token:
// decode) over the paged cache.
//
// out = sum_l p_l v_l / sum_l p_l with p_l = 2^(s_l - m), s_l = log2(e) scale
// q . k_l over the visible l, m the running maximum: a partial result over
// some of the tokens is (m, z = sum p, o = sum p v), and two of them join as
// m = max(m1, m2), z = z1 2^(m1 - m) + z2 2^(m2 - m), o likewise. lse =
// (m + log2 z) ln 2. A partial that saw nothing has m = -inf, z = 0.
//
// Rows. The new tokens of a request times the G = Hq / Hkv query heads of a
// kv head are the rows that share its keys and values: row = token * G + head
// within the group. An item is (request, kv head, tile of 16 RG rows); the
// bound is the one read of its keys and values (4 D rows flops a token
// against 4 D bytes: below the tensor cores' rate for tens of rows).
//
// Split. Lengths are known to the device only, and a batch is ragged, so the
// work of all items is laid out in units of kUnit tokens, and each of the
// grid's CTAs (three per SM; two for D = 256) takes an equal share of the line:
// at most two of its items are partial, the first and the last. A CTA writes the
// items that lie within its share; of an item that crosses a boundary each CTA
// writes its part to the workspace, and a second kernel joins them in ascending
// order (results do not depend on timing). A CTA finds its place by one scan of
// the requests' unit counts, within a warp for up to 32 requests.
//
// A CTA's four warps are 4 / RG token groups of RG warps, a warp per 16 rows.
// A token group streams blocks of 32 tokens (16 where two stages of 32 do not
// fit) through a shared-memory ring of its own (cp.async, 16 bytes a lane,
// waited for by the group alone: no barrier of the whole CTA in the loop) and
// holds its own (m, z, o) in registers; the groups join at the end of an item.
// Products run on mma.sync m16n8k16: scores from q (A, as fragments in shared
// memory, a 16-byte read each: in registers they left too few for three CTAs)
// and keys (B), then the probabilities, rounded, are the A operand as they lie
// in the score accumulators, and the values B.
//  - bf16 cache: B operands by ldmatrix (transposed for the values); p is
//    rounded to bf16, by up to 2^-8 of itself, which averages over the tokens.
//  - E4M3 cache: codes become f16 (exact) after the shared-memory read, which
//    takes 16 bytes of a token at a time: the order of the d along k, and of
//    the output columns along n, is permuted to fit. q enters as f16 times a
//    power of two per row that brings the row's largest element to 2^14
//    (what that drops is below 2^-38 of it); p is scaled by 2^12 before its
//    rounding to f16, so that p down to 2^-26 keeps 11 bits (what is smaller
//    keeps steps of 2^-36).
//
// Measured (8 kv heads, D = 128; 32 query heads over bf16, 64 over E4M3):
//  - 16 requests of 8 drafts over 8192 tokens, bf16: 77 us for 395 MB, 5.1
//    TB/s; the slope over longer contexts is 6.9 TB/s, the rest is start, the
//    spread of the CTAs' ends (56 to 71 us) and the join; over E4M3 73.5 us, half
//    the bytes: both row groups convert every code for themselves;
//  - 64 decodes over 8192 tokens, E4M3: 138 to 151 us from process to process,
//    5.3 to 5.8 TB/s, and in between the conversions' latency (16 tokens a step: 156 us);
//  - one decode over 1024 tokens: 8.9 us, two launches and one chain of loads.
//  - Many rows over E4M3, or at D = 256, come here too, in tiles of 32 that
//    each read and convert the cache: four trees of 64 drafts (64 query heads)
//    over 8192 tokens, E4M3, take 198 us where bf16 in tensor memory takes 66;
//    with 32 query heads on 4 of D = 256, bf16, 209 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn.h"
#include "common.cuh"
#include "host_util.h"
#include "stream.cuh"
#include "tree_attn.cuh"

namespace bqd {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / kWarp;
constexpr int kUnit = 64;          // tokens per unit of the split
constexpr int kOver = 2;           // units that an item's beginning and end cost
constexpr int kRows16 = 16;

template <int D, int RG, bool F8>
struct Shape {
    static constexpr int kRows = kRows16 * RG;
    static constexpr int kGroups = kWarps / RG;            // token groups
    static constexpr int kRowBytes = D * (F8 ? 1 : 2);
    // Tokens a token group takes at a time: 32 where two stages of them fit, so
    // that what a block costs beside its products (maximum, addresses, waits)
    // is shared by twice the tokens.
    static constexpr int kNB = D <= 128 && kGroups * 128 * kRowBytes <= 64 * 1024 ? 2 : 1, kBlock = 16 * kNB;
    static constexpr int kStage = 2 * kBlock * kRowBytes;  // K and V of one block
    static constexpr int kCtas = D <= 128 ? 3 : 2;         // per SM: 64 of o and 40 more registers, or 128 of o
    static constexpr int kGrid = kCtas * 152;
    static constexpr int kMost = (D <= 128 ? 64 : 96) * 1024 / (kGroups * kStage);
    static constexpr int kStages = kMost < 2 ? 2 : kMost > 8 ? 8 : kMost;
    static constexpr int kRing = kGroups * kStages * kStage;
    static constexpr int kJoin = kWarps * kRows16 * D * 4;
    static constexpr int kMain = kRing > kJoin ? kRing : kJoin;
    static constexpr int kQBytes = RG * (D / 16) * 512;    // q as mma fragments
    static constexpr int kSmem = kMain + kQBytes;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}

template <bool F8>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if (F8)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
            "%2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, "
            "%1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool F8>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if (F8) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// What is taken from a row's scores: its maximum, for E4M3 less p's shift. Where
// that difference rounds to 2 less or more (maxima from 2^25 on, whose scores
// are further apart than it rounds), the maximum alone: p must stay within f16.
template <bool F8>
__device__ __forceinline__ float shifted(float m)
{
    if (m == -INFINITY) m = 0.f;
    const float x = m - (F8 ? kAttnPShift : 0.f);
    return F8 && m - x > kAttnPShift + 1.f ? m : x;
}

// Byte offset of 16-byte chunk `ch` of token row `row` in a block. The chunk
// index is permuted by the row so that the reads of a phase fall into
// different banks: ldmatrix takes one chunk of 8 rows; the E4M3 reads take
// chunks c .. c + 3 of two adjacent rows (keys) or two chunks of every other
// row (values); 64-byte rows share a 128-byte line in pairs.
template <int RB, bool F8>
__device__ __forceinline__ uint32_t chunk_at(int row, int ch)
{
    if (!F8) return static_cast<uint32_t>(row * RB + ((ch ^ (row & 7)) << 4));
    const int f = ((row >> 1) & 3) << 1;
    if (RB == 64) return static_cast<uint32_t>((row >> 1) * 128 + (((((row & 1) << 2) | ch) ^ f) << 4));
    return static_cast<uint32_t>(row * RB + ((ch ^ f ^ ((row & 1) << 2)) << 4));
}

template <int D, int RG, bool F8>
__global__ void __launch_bounds__(kThreads, Shape<D, RG, F8>::kCtas) tree_attn_kernel(const AttnArgs a)
{
    using S = Shape<D, RG, F8>;
    constexpr int NT = D / 8;     // n tiles of the output; d of column n of tile j:
    constexpr int KS = D / 16;    // k steps of the scores
    constexpr int kBlock = S::kBlock, NB = S::kNB;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_find[kWarps + 2];
    __shared__ uint32_t s_vis[kWarps][8];
    __shared__ float s_m[kWarps][kRows16], s_z[kWarps][kRows16];
    constexpr uint32_t kAll = kBlock == 32 ? 0xFFFFFFFFu : 0xFFFFu;
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    const int rg = warp % RG, tg = warp / RG;  // row group, token group
    const int g = lane >> 2, c = lane & 3;     // row (and column) and k positions in mma fragments
    const int G = a.group;
    const uint32_t ring = smem_u32(smem) + tg * (S::kStages * S::kStage);

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join waits for this grid's end
    AttnShare sh = attn_find_share<kThreads>(a, S::kRows, kUnit, kOver, s_find);
    int64_t u = sh.start;
    AttnMeta* meta = static_cast<AttnMeta*>(a.ws);
    float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + attn_meta_bytes());
    if (threadIdx.x == 0) meta[blockIdx.x].rows = 0;
    const int page_shift = a.page_shift;

    while (u < sh.end) {
        const AttnReq q = attn_request(a, sh.r, S::kRows, kUnit, kOver);
        int h, tile;
        int64_t b0;
        attn_place(sh, q, u, h, tile, b0);
        int64_t cnt = min(q.nb - b0, sh.end - u);
        const int64_t u_next = u + cnt, item_end = u + q.nb - b0;
        // the item's first kOver units stand for what it costs beside its tokens
        cnt = max(b0 + cnt - kOver, int64_t(0));
        b0 = max(b0 - kOver, int64_t(0));
        cnt -= b0;
        if (cnt <= 0) {
            u = u_next;
            continue;
        }
        const int64_t l0 = b0 * kUnit, l1 = min((b0 + cnt) * kUnit, q.len);
        const int32_t* table = a.table + sh.r * a.width;
        const int rows = static_cast<int>(min(static_cast<int64_t>(q.n) * G - static_cast<int64_t>(tile) * S::kRows,
                                              static_cast<int64_t>(S::kRows)));
        // this thread's two rows
        const int row0 = tile * S::kRows + rg * kRows16 + g, row1 = row0 + 8;
        const int i0 = row0 / G, i1 = row1 / G;
        const bool live0 = i0 < q.n, live1 = i1 < q.n;
        const int64_t t0 = q.o0 + (live0 ? i0 : 0), t1 = q.o0 + (live1 ? i1 : 0);
        const uint16_t* q0 = a.q + t0 * a.q_pitch + static_cast<int64_t>(h * G + row0 % G) * D;
        const uint16_t* q1 = a.q + t1 * a.q_pitch + static_cast<int64_t>(h * G + row1 % G) * D;
        float c0 = a.scale * kAttnLog2e, c1 = c0;  // score to log2 units, per row

        // ---- the token group's stream
        const int64_t first = l0 + tg * kBlock;
        const int nblk = first < l1 ? static_cast<int>((l1 - first + S::kGroups * kBlock - 1) / (S::kGroups * kBlock)) : 0;
        auto entry = [&](int64_t l) -> int32_t { return l < l1 ? table[l >> page_shift] : -1; };
        int32_t ent = entry(first + (lane & (kBlock - 1)));  // table entry of the next block to fetch, a token per lane
        auto fetch = [&](int i) {  // block i into its stage
            if (i < nblk) {
                const int64_t l = first + static_cast<int64_t>(i) * (S::kGroups * kBlock) + (lane & (kBlock - 1));
                const bool ok = ent >= 0 && ent < a.cache.num_pages;
                const int64_t off = ok ? (ent * a.cache.page_stride + (l & (a.cache.page_size - 1)) * a.cache.token_stride +
                                          h * a.cache.head_stride) * (F8 ? 1 : 2)
                                       : 0;
                const uint32_t vis = __ballot_sync(0xFFFFFFFFu, ok) & kAll;
                ent = entry(l + S::kGroups * kBlock);
                if (rg == 0 && lane == 0) s_vis[tg][i % S::kStages] = vis;
                const uint32_t st = ring + (i % S::kStages) * S::kStage;
                constexpr int CPR = S::kRowBytes / 16;  // chunks per row
#pragma unroll
                for (int it = 0; it < kBlock * CPR / (kWarp * RG); ++it) {
                    const int ch = (it * RG + rg) * kWarp + lane, row = ch / CPR, cc = ch % CPR;
                    const int64_t o = __shfl_sync(0xFFFFFFFFu, off, row) + cc * 16;
                    const bool real = (vis >> row) & 1;
                    const uint32_t at = st + chunk_at<S::kRowBytes, F8>(row, cc);
                    cp_async16(at, static_cast<const uint8_t*>(a.cache.k) + o, real);
                    cp_async16(at + S::kStage / 2, static_cast<const uint8_t*>(a.cache.v) + o, real);
                }
            }
            cp_commit();
        };
#pragma unroll
        for (int i = 0; i < S::kStages - 1; ++i) fetch(i);

        // ---- q fragments, while the first blocks are on their way
        const uint32_t qsm = smem_u32(smem) + S::kMain + (rg * KS * 32 + lane) * 16;
        {
            uint32_t f[KS][4];
            if (F8) {
                float mx0 = 0.f, mx1 = 0.f;
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const int d = 64 * (s / 4) + 16 * c + 4 * (s % 4);
                    const uint2 x = live0 ? *reinterpret_cast<const uint2*>(q0 + d) : make_uint2(0, 0);
                    const uint2 y = live1 ? *reinterpret_cast<const uint2*>(q1 + d) : make_uint2(0, 0);
                    f[s][0] = x.x, f[s][2] = x.y, f[s][1] = y.x, f[s][3] = y.y;
                    mx0 = fmaxf(mx0, fmaxf(fmaxf(fabsf(bf16_lo(x.x)), fabsf(bf16_hi(x.x))),
                                           fmaxf(fabsf(bf16_lo(x.y)), fabsf(bf16_hi(x.y)))));
                    mx1 = fmaxf(mx1, fmaxf(fmaxf(fabsf(bf16_lo(y.x)), fabsf(bf16_hi(y.x))),
                                           fmaxf(fabsf(bf16_lo(y.y)), fabsf(bf16_hi(y.y)))));
                }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    mx0 = fmaxf(mx0, __shfl_xor_sync(0xFFFFFFFFu, mx0, o));
                    mx1 = fmaxf(mx1, __shfl_xor_sync(0xFFFFFFFFu, mx1, o));
                }
                // 2^(14 - e) for a largest element of [2^e, 2^(e + 1)); e kept within [-100, 100]
                const int e0 = min(max(static_cast<int>(__float_as_uint(mx0) >> 23), 27), 227);
                const int e1 = min(max(static_cast<int>(__float_as_uint(mx1) >> 23), 27), 227);
                const float up0 = __uint_as_float((127 + 14 + 127 - e0) << 23), up1 = __uint_as_float((127 + 14 + 127 - e1) << 23);
                c0 *= __uint_as_float((e0 - 14) << 23);
                c1 *= __uint_as_float((e1 - 14) << 23);
                if (a.cache.k_scale) {
                    c0 *= a.cache.k_scale[h];
                    c1 *= a.cache.k_scale[h];
                }
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float up = (e & 1) ? up1 : up0;
                        f[s][e] = pack2<true>(bf16_lo(f[s][e]) * up, bf16_hi(f[s][e]) * up);
                    }
            } else {
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const int d = 16 * s + 2 * c;
                    f[s][0] = live0 ? *reinterpret_cast<const uint32_t*>(q0 + d) : 0u;
                    f[s][1] = live1 ? *reinterpret_cast<const uint32_t*>(q1 + d) : 0u;
                    f[s][2] = live0 ? *reinterpret_cast<const uint32_t*>(q0 + d + 8) : 0u;
                    f[s][3] = live1 ? *reinterpret_cast<const uint32_t*>(q1 + d + 8) : 0u;
                }
            }
            if (tg == 0) {
#pragma unroll
                for (int s = 0; s < KS; ++s)
                    *reinterpret_cast<uint4*>(smem + S::kMain + ((rg * KS + s) * 32 + lane) * 16) =
                        make_uint4(f[s][0], f[s][1], f[s][2], f[s][3]);
            }
        }
        __syncthreads();

        float o[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, z0 = 0.f, z1 = 0.f;  // z: this lane's columns only

        for (int i = 0; i < nblk; ++i) {
            cp_wait<S::kStages - 2>();
            if (RG == 1)
                __syncwarp();
            else
                named_sync(1 + tg, RG * kWarp);
            fetch(i + S::kStages - 1);
            const uint32_t ks = ring + (i % S::kStages) * S::kStage, vs = ks + S::kStage / 2;
            const uint32_t vis = s_vis[tg][i % S::kStages];
            const int64_t l = first + static_cast<int64_t>(i) * (S::kGroups * kBlock);
            float s[2 * NB][4];
#pragma unroll
            for (int nt = 0; nt < 2 * NB; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
            // scores
            if (!F8) {
                const int mrow = (lane & 7) + ((lane >> 4) << 3), mch = (lane >> 3) & 1;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const uint4 x = lds128(qsm + k * 512);
                    const uint32_t qa[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        uint32_t b[4];
                        ldsm4(ks + chunk_at<S::kRowBytes, F8>(16 * nb + mrow, 2 * k + mch), b);
                        mma16816<F8>(s[2 * nb], qa, b[0], b[1]);
                        mma16816<F8>(s[2 * nb + 1], qa, b[2], b[3]);
                    }
                }
            } else {
#pragma unroll
                for (int k4 = 0; k4 < KS / 4; ++k4) {
                    uint32_t x[2 * NB][4];  // 16 d of token 8 nt + g
#pragma unroll
                    for (int nt = 0; nt < 2 * NB; ++nt) {
                        const uint4 v = lds128(ks + chunk_at<S::kRowBytes, F8>(8 * nt + g, 4 * k4 + c));
                        x[nt][0] = v.x, x[nt][1] = v.y, x[nt][2] = v.z, x[nt][3] = v.w;
                    }
#pragma unroll
                    for (int e4 = 0; e4 < 4; ++e4) {
                        const int k = 4 * k4 + e4;
                        const uint4 w = lds128(qsm + k * 512);
                        const uint32_t qa[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int nt = 0; nt < 2 * NB; ++nt)
                            mma16816<F8>(s[nt], qa, e4m3x2_to_f16x2(x[nt][e4] & 0xFFFFu), e4m3x2_to_f16x2(x[nt][e4] >> 16));
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < 2 * NB; ++nt) {
                s[nt][0] *= c0;
                s[nt][1] *= c0;
                s[nt][2] *= c1;
                s[nt][3] *= c1;
            }
            // what is hidden
            const bool drafts = l + kBlock > q.ctx;
            if (vis != kAll || drafts) {
#pragma unroll
                for (int nt = 0; nt < 2 * NB; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int tok = 8 * nt + 2 * c + e;
                        const bool v = (vis >> tok) & 1;
                        const int64_t j = l + tok - q.ctx;
                        if (!v || !attn_sees(a, t0, i0, j)) s[nt][e] = -INFINITY;
                        if (!v || !attn_sees(a, t1, i1, j)) s[nt][2 + e] = -INFINITY;
                    }
            }
            // running maximum
            float n0 = -INFINITY, n1 = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < 2 * NB; ++nt) {
                n0 = fmaxf(n0, fmaxf(s[nt][0], s[nt][1]));
                n1 = fmaxf(n1, fmaxf(s[nt][2], s[nt][3]));
            }
#pragma unroll
            for (int x = 1; x < 4; x <<= 1) {
                n0 = fmaxf(n0, __shfl_xor_sync(0xFFFFFFFFu, n0, x));
                n1 = fmaxf(n1, __shfl_xor_sync(0xFFFFFFFFu, n1, x));
            }
            n0 = fmaxf(n0, m0);
            n1 = fmaxf(n1, m1);
            if (__any_sync(0xFFFFFFFFu, n0 != m0 || n1 != m1)) {
                const float f0 = m0 == -INFINITY ? 0.f : attn_ex2(m0 - n0), f1 = m1 == -INFINITY ? 0.f : attn_ex2(m1 - n1);
                z0 *= f0;
                z1 *= f1;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    o[j][0] *= f0;
                    o[j][1] *= f0;
                    o[j][2] *= f1;
                    o[j][3] *= f1;
                }
                m0 = n0;
                m1 = n1;
            }
            const float sub0 = shifted<F8>(m0), sub1 = shifted<F8>(m1);
            uint32_t pa[NB][4];
#pragma unroll
            for (int nt = 0; nt < 2 * NB; ++nt) {
                const float p0 = attn_ex2(s[nt][0] - sub0), p1 = attn_ex2(s[nt][1] - sub0);
                const float p2 = attn_ex2(s[nt][2] - sub1), p3 = attn_ex2(s[nt][3] - sub1);
                z0 += p0 + p1;
                z1 += p2 + p3;
                pa[nt / 2][2 * (nt % 2)] = pack2<F8>(p0, p1);
                pa[nt / 2][2 * (nt % 2) + 1] = pack2<F8>(p2, p3);
            }
            // A draft's value may be infinite or NaN and hidden from some of
            // the rows, where 0 * v must count nothing: such elements leave
            // the product (zeros in the stage) and are added to the rows that
            // see them. Looked for in blocks with drafts only; every token
            // before them is seen by all rows.
            if (drafts) {
                bool odd = false;
                constexpr int CPR = S::kRowBytes / 16;
                for (int ch = lane; ch < kBlock * CPR; ch += kWarp) {
                    const uint4 x = lds128(vs + chunk_at<S::kRowBytes, F8>(ch / CPR, ch % CPR));
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int b = 0; b < (F8 ? 4 : 2); ++b)
                            odd |= F8 ? ((w[e] >> (8 * b)) & 0x7Fu) == 0x7Fu : ((w[e] >> (16 * b)) & 0x7F80u) == 0x7F80u;
                }
                if (__any_sync(0xFFFFFFFFu, odd)) {
                    for (int tok = 0; tok < kBlock; ++tok) {
                        if (!((vis >> tok) & 1)) continue;
                        const bool see0 = attn_sees(a, t0, i0, l + tok - q.ctx), see1 = attn_sees(a, t1, i1, l + tok - q.ctx);
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int d = F8 ? NT * (2 * c + e) + j : 8 * j + 2 * c + e;
                                float v;
                                const uint32_t at = vs + (F8 ? chunk_at<S::kRowBytes, F8>(tok, d / 16) + d % 16
                                                             : chunk_at<S::kRowBytes, F8>(tok, d / 8) + d % 8 * 2);
                                if (F8) {
                                    uint32_t b;
                                    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(b) : "r"(at) : "memory");
                                    v = e4m3_to_float(b);
                                } else {
                                    uint16_t b;
                                    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(b) : "r"(at) : "memory");
                                    v = __uint_as_float(static_cast<uint32_t>(b) << 16);
                                }
                                if (!isfinite(v)) {
                                    if (see0) o[j][e] += v;
                                    if (see1) o[j][2 + e] += v;
                                }
                            }
                    }
                    // all reads above come before the zeros below
                    if (RG == 1)
                        __syncwarp();
                    else
                        named_sync(1 + tg, RG * kWarp);
                    if (rg == 0)
                        for (int x = lane; x < S::kStage / 2 / 4; x += kWarp) {
                            uint32_t w;
                            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(vs + 4 * x) : "memory");
#pragma unroll
                            for (int b = 0; b < (F8 ? 4 : 2); ++b)
                                if (F8 ? ((w >> (8 * b)) & 0x7Fu) == 0x7Fu : ((w >> (16 * b)) & 0x7F80u) == 0x7F80u)
                                    w &= ~((F8 ? 0xFFu : 0xFFFFu) << (F8 ? 8 * b : 16 * b));
                            asm volatile("st.shared.u32 [%0], %1;" ::"r"(vs + 4 * x), "r"(w) : "memory");
                        }
                    if (RG == 1)
                        __syncwarp();
                    else
                        named_sync(1 + tg, RG * kWarp);
                }
            }
            // o += p v
            if (!F8) {
                const int mrow = (lane & 7) + (((lane >> 3) & 1) << 3), mch = lane >> 4;
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        uint32_t b[4];
                        ldsm4t(vs + chunk_at<S::kRowBytes, F8>(16 * nb + mrow, 2 * k + mch), b);
                        mma16816<F8>(o[2 * k], pa[nb], b[0], b[1]);
                        mma16816<F8>(o[2 * k + 1], pa[nb], b[2], b[3]);
                    }
            } else {
                // tokens 2c, 2c + 1, 2c + 8, 2c + 9; the NT d from NT g
                constexpr int W = NT / 4;       // words per token
                constexpr int WL = W < 4 ? W : 4;  // words per load
#pragma unroll
                for (int ww = 0; ww < W * NB; ww += WL) {
                    const int w0 = ww % W, nb = ww / W;  // words, 16 tokens
                    uint32_t x[4][4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int tok = 16 * nb + 2 * c + (e & 1) + 8 * (e >> 1), byte = NT * g + 4 * w0;
                        const uint32_t at = vs + chunk_at<S::kRowBytes, F8>(tok, byte / 16) + byte % 16;
                        if (WL == 4) {
                            const uint4 y = lds128(at);
                            x[e][0] = y.x, x[e][1] = y.y, x[e][2] = y.z, x[e][3] = y.w;
                        } else {
                            const uint2 y = lds64(at);
                            x[e][0] = y.x, x[e][1] = y.y;
                        }
                    }
#pragma unroll
                    for (int w = 0; w < WL; ++w) {
                        const uint32_t lo0 = __byte_perm(x[0][w], x[1][w], 0x5140), hi0 = __byte_perm(x[0][w], x[1][w], 0x7362);
                        const uint32_t lo1 = __byte_perm(x[2][w], x[3][w], 0x5140), hi1 = __byte_perm(x[2][w], x[3][w], 0x7362);
                        const int j = 4 * (w0 + w);
                        mma16816<F8>(o[j], pa[nb], e4m3x2_to_f16x2(lo0 & 0xFFFFu), e4m3x2_to_f16x2(lo1 & 0xFFFFu));
                        mma16816<F8>(o[j + 1], pa[nb], e4m3x2_to_f16x2(lo0 >> 16), e4m3x2_to_f16x2(lo1 >> 16));
                        mma16816<F8>(o[j + 2], pa[nb], e4m3x2_to_f16x2(hi0 & 0xFFFFu), e4m3x2_to_f16x2(hi1 & 0xFFFFu));
                        mma16816<F8>(o[j + 3], pa[nb], e4m3x2_to_f16x2(hi0 >> 16), e4m3x2_to_f16x2(hi1 >> 16));
                    }
                }
            }
        }

        // ---- join the token groups: everything of a warp to shared memory
        cp_wait<0>();
#pragma unroll
        for (int x = 1; x < 4; x <<= 1) {
            z0 += __shfl_xor_sync(0xFFFFFFFFu, z0, x);
            z1 += __shfl_xor_sync(0xFFFFFFFFu, z1, x);
        }
        __syncthreads();  // the rings are read no more
        if (c == 0) {
            s_m[warp][g] = m0;
            s_m[warp][g + 8] = m1;
            s_z[warp][g] = z0;
            s_z[warp][g + 8] = z1;
        }
        float* join = reinterpret_cast<float*>(smem) + warp * (kRows16 * D);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int d = F8 ? NT * (2 * c + e) + j : 8 * j + 2 * c + e;
                join[g * D + d] = o[j][e];
                join[(g + 8) * D + d] = o[j][2 + e];
            }
        __syncthreads();
        const bool whole = b0 == 0 && cnt == q.nb - kOver;
        float* part = parts + (2 * blockIdx.x + (b0 == 0 ? 1 : 0)) * attn_part_floats(S::kRows, D);
        const float vscale = (F8 && a.cache.v_scale) ? a.cache.v_scale[h] : 1.f;
        for (int x = threadIdx.x; x < rows * (D / 4); x += kThreads) {
            const int row = x / (D / 4), d = x % (D / 4) * 4, rw = row / kRows16, rr = row % kRows16;
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < S::kGroups; ++w) m = fmaxf(m, s_m[w * RG + rw][rr]);
            float z = 0.f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < S::kGroups; ++w) {
                const float mw = s_m[w * RG + rw][rr];
                const float f = attn_weight(mw, m);
                const float4 y = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem) +
                                                                  ((w * RG + rw) * kRows16 + rr) * D + d);
                z += s_z[w * RG + rw][rr] * f;
                v.x += y.x * f;
                v.y += y.y * f;
                v.z += y.z * f;
                v.w += y.w * f;
            }
            if (whole) {
                const int grow = tile * S::kRows + row;
                const int64_t at = (q.o0 + grow / G) * static_cast<int64_t>(a.Hq) + h * G + grow % G;
                *reinterpret_cast<uint2*>(a.out + at * D + d) = attn_out4(v, z, vscale);
                if (d == 0 && a.lse) a.lse[at] = attn_lse(m, z, F8 ? kAttnPShift : 0.f);
            } else {
                *reinterpret_cast<float4*>(part + row * D + d) = v;
                if (d == 0) {
                    part[S::kRows * D + row] = m;
                    part[S::kRows * D + S::kRows + row] = z;
                }
            }
        }
        if (b0 == 0 && !whole && threadIdx.x == 0) meta[blockIdx.x] = attn_meta(a, sh, q, h, tile, S::kRows, item_end);
        __syncthreads();
        u = u_next;
        if (u < sh.end) {
            int64_t next = sh.base + q.nb * q.tiles * a.cache.heads;
            while (u == next) {  // the next request with rows
                ++sh.r;
                sh.base = next;
                next += attn_units(a, sh.r, S::kRows, kUnit, kOver);
            }
        }
    }
}

// Row groups: 16 rows unless the requests have more on average (two halve the
// reads of the keys and values for wide drafts).
int row_groups(int64_t R, int64_t T, int Hq, int Hkv) { return T * (Hq / Hkv) > 16 * R ? 2 : 1; }

template <int D, int RG, bool F8>
cudaError_t launch(const AttnArgs& a, cudaStream_t s)
{
    using S = Shape<D, RG, F8>;
    static OccCache occ;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    blocks_per_sm(occ, reinterpret_cast<const void*>(&tree_attn_kernel<D, RG, F8>), dev, kThreads, S::kSmem);
    tree_attn_kernel<D, RG, F8><<<S::kGrid, kThreads, S::kSmem, s>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_attn_join(tree_attn_join_kernel<D, S::kRows, F8>, a, S::kGrid, s);
}

template <int D>
cudaError_t launch_d(const AttnArgs& a, cudaStream_t s)
{
    const bool f8 = a.cache.type == BQD_E4M3;
    if (row_groups(a.R, a.T, a.Hq, a.cache.heads) == 1) return f8 ? launch<D, 1, true>(a, s) : launch<D, 1, false>(a, s);
    return f8 ? launch<D, 2, true>(a, s) : launch<D, 2, false>(a, s);
}

}  // namespace

// Parts are as tall as a call's tiles, which grow with the mean rows per
// request: the size is that for one request with all T tokens, the tallest, so
// that it holds for any number of requests and grows with T alone.
size_t tree_attention_ws(int64_t T, int Hq, int Hkv, int D)
{
    const int rows = kRows16 * row_groups(1, T, Hq, Hkv);
    const size_t narrow = attn_meta_bytes() + 2 * kAttnMaxGrid * attn_part_floats(rows, D) * sizeof(float);
    const size_t wide = tree_attention_wide_ws(T, Hq, Hkv, D);
    return narrow > wide ? narrow : wide;
}

cudaError_t launch_tree_attention(const AttnArgs& a, cudaStream_t s)
{
    if (tree_attention_wide_fits(a)) return launch_tree_attention_wide(a, s);
    switch (a.cache.head_dim) {
        case 64: return launch_d<64>(a, s);
        case 128: return launch_d<128>(a, s);
        default: return launch_d<256>(a, s);
    }
}

}  // namespace bqd
