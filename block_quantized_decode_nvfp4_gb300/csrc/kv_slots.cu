// kv_slots.cu -- block table, slots and positions of a step's new tokens.
//
// Request r: have = ceil(c / p) pages, lacks need = ceil((c + n) / p) - have,
// takes free pages first .. first + need - 1 (first: sum of the needs before
// it). Token (r, j) sits at logical position c + j, block b = (c + j) / p:
// its page is the table's for b < have, else free page first + b - have.
//
// Integer work on a few hundred KB at most: what bounds it is latency, so it
// is one launch without a pass between the prefix sums and their use. Every
// CTA scans all requests, kChunk at a time in shared memory (a second read of
// the lengths costs less than a second launch), and meanwhile writes its own
// share of the tokens, found by a search of the chunk's sums, and its own
// share of the requests' new pages. Pages of new blocks are taken from the
// list and not from the table, which another CTA may be writing. 8 requests of
// one token take 3.4 us, 1024 requests with 49 thousand new tokens 5.1 us (an
// empty launch in the same graph: 2 us).
#include <cuda_runtime.h>

#include <cstdint>

#include "attn.h"
#include "common.cuh"

namespace bqd {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 4;  // requests per thread and chunk
constexpr int kChunk = kThreads * kPer;
constexpr int kTokens = kThreads;  // tokens per CTA at least (one per thread)
constexpr int kMaxCtas = 2 * 152;

struct Need {
    int64_t c, n;        // cached and new tokens
    int64_t have, want;  // pages, within the table
};

__device__ __forceinline__ Need need_of(const SlotsArgs& a, int64_t r)
{
    Need x;
    x.c = max(0, a.context[r]);
    x.n = max(0, a.fresh[r]);
    const int64_t p1 = (int64_t(1) << a.page_shift) - 1;
    x.have = min((x.c + p1) >> a.page_shift, a.width);
    x.want = max(x.have, min((x.c + x.n + p1) >> a.page_shift, a.width));
    return x;
}

__global__ void __launch_bounds__(kThreads) paged_slots_kernel(const SlotsArgs a)
{
    __shared__ int64_t s_tok[kChunk + 1], s_page[kChunk + 1];  // exclusive sums of the chunk's requests
    __shared__ int32_t s_ctx[kChunk];
    __shared__ int64_t s_warp[kThreads / kWarp][2];
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    const int64_t share = (a.capacity + gridDim.x - 1) / gridDim.x;
    const int64_t t0 = min(share * blockIdx.x, a.capacity), t1 = min(t0 + share, a.capacity);
    int64_t tokens = 0, pages = 0;  // before the chunk
    bool full = false;
    for (int64_t r0 = 0; r0 < a.R; r0 += kChunk) {
        const int count = static_cast<int>(min(static_cast<int64_t>(kChunk), a.R - r0));
        int64_t tk[kPer], pg[kPer], st = 0, sp = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int k = threadIdx.x * kPer + i;
            tk[i] = pg[i] = 0;
            if (k < count) {
                const Need x = need_of(a, r0 + k);
                s_ctx[k] = static_cast<int32_t>(x.c);
                tk[i] = x.n;
                pg[i] = x.want - x.have;
                full |= x.n > 0 && ((x.c + x.n - 1) >> a.page_shift) >= a.width;
            }
            st += tk[i];
            sp += pg[i];
        }
        int64_t it = st, ip = sp;
#pragma unroll
        for (int d = 1; d < kWarp; d <<= 1) {
            const int64_t u = __shfl_up_sync(0xFFFFFFFFu, it, d), v = __shfl_up_sync(0xFFFFFFFFu, ip, d);
            if (lane >= d) {
                it += u;
                ip += v;
            }
        }
        if (lane == kWarp - 1) {
            s_warp[warp][0] = it;
            s_warp[warp][1] = ip;
        }
        __syncthreads();
        int64_t bt = tokens, bp = pages;
        for (int w = 0; w < kThreads / kWarp; ++w) {
            if (w < warp) {
                bt += s_warp[w][0];
                bp += s_warp[w][1];
            }
            tokens += s_warp[w][0];
            pages += s_warp[w][1];
        }
        bt += it - st;
        bp += ip - sp;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int k = threadIdx.x * kPer + i;
            s_tok[k] = bt;
            s_page[k] = bp;
            bt += tk[i];
            bp += pg[i];
        }
        if (threadIdx.x == kThreads - 1) {
            s_tok[kChunk] = bt;
            s_page[kChunk] = bp;
        }
        __syncthreads();
        if (blockIdx.x == 0)
            for (int k = threadIdx.x; k < count; k += kThreads)
                a.offsets[r0 + k] = static_cast<int32_t>(min(s_tok[k], int64_t(0x7FFFFFFF)));
        // new pages of requests blockIdx.x, blockIdx.x + gridDim.x, ...
        for (int64_t k = blockIdx.x + static_cast<int64_t>(warp) * gridDim.x; k < count;
             k += static_cast<int64_t>(gridDim.x) * (kThreads / kWarp)) {
            const int64_t f0 = s_page[k], need = s_page[k + 1] - f0;
            if (need == 0) continue;
            const Need x = need_of(a, r0 + k);
            int32_t* row = a.table + (r0 + k) * a.width + x.have;
            for (int64_t b = lane; b < need; b += kWarp) row[b] = f0 + b < a.num_free ? a.free_pages[f0 + b] : -1;
        }
        // this CTA's tokens of the chunk's requests
        for (int64_t t = max(t0, s_tok[0]) + threadIdx.x; t < min(t1, s_tok[kChunk]); t += kThreads) {
            int lo = 0, hi = count;  // the last k with s_tok[k] <= t: requests without tokens come before it
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (s_tok[mid] <= t)
                    lo = mid;
                else
                    hi = mid;
            }
            const int64_t ctx = s_ctx[lo], j = t - s_tok[lo], b = (ctx + j) >> a.page_shift;
            const int64_t have = min((ctx + (int64_t(1) << a.page_shift) - 1) >> a.page_shift, a.width);
            int64_t slot = -1;
            if (b < a.width) {
                const int64_t f = s_page[lo] + b - have;
                const int32_t page = b < have ? a.table[(r0 + lo) * a.width + b] : f < a.num_free ? a.free_pages[f] : -1;
                if (page >= 0)
                    slot = (static_cast<int64_t>(page) << a.page_shift) + ((ctx + j) & ((1 << a.page_shift) - 1));
            }
            a.slots[t] = slot;
            a.positions[t] = static_cast<int32_t>(ctx + (a.depths ? a.depths[t] : j));
        }
        __syncthreads();  // the next chunk overwrites the sums
    }
    for (int64_t t = max(t0, tokens) + threadIdx.x; t < t1; t += kThreads) {
        a.slots[t] = -1;
        a.positions[t] = -1;
    }
    if (blockIdx.x == 0) {
        full = __syncthreads_or(full);
        if (threadIdx.x == 0) {
            const int64_t top = 0x7FFFFFFF;
            a.offsets[a.R] = static_cast<int32_t>(min(tokens, top));
            a.counts[0] = static_cast<int32_t>(min(tokens, top));
            a.counts[1] = static_cast<int32_t>(min(pages, a.num_free));
            a.counts[2] = static_cast<int32_t>(min(max(pages - a.num_free, int64_t(0)), top));
            a.counts[3] = (full ? BQD_SLOTS_TABLE_FULL : 0) | (tokens > a.capacity ? BQD_SLOTS_TOKENS_CUT : 0);
        }
    }
}

}  // namespace

cudaError_t launch_paged_slots(const SlotsArgs& a, cudaStream_t s)
{
    const int64_t by_tokens = (a.capacity + kTokens - 1) / kTokens, by_requests = (a.R + 63) / 64;
    const int64_t want = by_tokens > by_requests ? by_tokens : by_requests;
    const unsigned grid = static_cast<unsigned>(want < 1 ? 1 : want > kMaxCtas ? kMaxCtas : want);
    paged_slots_kernel<<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace bqd
