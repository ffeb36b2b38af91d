// kv_slots.cu -- block table, slots and positions of a step's new tokens.
//
// Request r: have = ceil(c / p) pages, lacks need = ceil((c + n) / p) - have,
// takes free pages first .. first + need - 1 (first: sum of the needs before
// it). Token (r, j) sits at logical position c + j: slot = table[r][(c + j)
// / p] * p + (c + j) % p. Integer work on a few hundred KB at most: what
// bounds it is latency.
//
// Simple form: one CTA scans the requests a block at a time, then a warp per
// request writes its pages and tokens.
#include <cuda_runtime.h>

#include <cstdint>

#include "attn.h"
#include "common.cuh"

namespace bqd {

namespace {

constexpr int kThreads = 1024;

struct Need {
    int64_t c, n;  // cached and new tokens
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

// Inclusive scan of (tokens, pages) over the block; totals in the last thread.
__device__ __forceinline__ void block_scan(int64_t& t, int64_t& p, int64_t (*sh)[2])
{
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
#pragma unroll
    for (int d = 1; d < kWarp; d <<= 1) {
        const int64_t a = __shfl_up_sync(0xFFFFFFFFu, t, d), b = __shfl_up_sync(0xFFFFFFFFu, p, d);
        if (lane >= d) {
            t += a;
            p += b;
        }
    }
    if (lane == kWarp - 1) {
        sh[warp][0] = t;
        sh[warp][1] = p;
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
        t += sh[w][0];
        p += sh[w][1];
    }
    __syncthreads();
}

__global__ void __launch_bounds__(kThreads) paged_slots_kernel(const SlotsArgs a)
{
    __shared__ int64_t sh[kThreads / kWarp][2], s_tok[kThreads], s_page[kThreads], s_base[2];
    __shared__ int s_flags;
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    if (threadIdx.x == 0) {
        s_base[0] = s_base[1] = 0;
        s_flags = 0;
    }
    __syncthreads();
    for (int64_t r0 = 0; r0 < a.R; r0 += kThreads) {
        const int64_t r = r0 + threadIdx.x;
        int64_t t = 0, p = 0;
        if (r < a.R) {
            const Need x = need_of(a, r);
            t = x.n;
            p = x.want - x.have;
            if (((x.c + x.n + (int64_t(1) << a.page_shift) - 1) >> a.page_shift) > a.width && x.n > 0)
                atomicOr(&s_flags, BQD_SLOTS_TABLE_FULL);
        }
        const int64_t t0 = t, p0 = p;
        block_scan(t, p, sh);
        const int64_t bt = s_base[0], bp = s_base[1];
        s_tok[threadIdx.x] = bt + t - t0;
        s_page[threadIdx.x] = bp + p - p0;
        if (r < a.R) a.offsets[r] = static_cast<int32_t>(min(bt + t - t0, int64_t(0x7FFFFFFF)));
        __syncthreads();
        if (threadIdx.x == kThreads - 1) {
            s_base[0] = bt + t;
            s_base[1] = bp + p;
        }
        for (int i = warp; i < kThreads && r0 + i < a.R; i += kThreads / kWarp) {
            const int64_t rr = r0 + i;
            const Need x = need_of(a, rr);
            int32_t* row = a.table + rr * a.width;
            for (int64_t b = x.have + lane; b < x.want; b += kWarp) {
                const int64_t f = s_page[i] + b - x.have;
                row[b] = f < a.num_free ? a.free_pages[f] : -1;
            }
            __syncwarp();
            for (int64_t j = lane; j < x.n; j += kWarp) {
                const int64_t tk = s_tok[i] + j;
                if (tk >= a.capacity) break;
                const int64_t pos = x.c + j, b = pos >> a.page_shift;
                int64_t slot = -1;
                if (b < a.width) {
                    const int32_t page = row[b];
                    if (page >= 0)
                        slot = (static_cast<int64_t>(page) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
                }
                a.slots[tk] = slot;
                a.positions[tk] = static_cast<int32_t>(x.c + (a.depths ? a.depths[tk] : j));
            }
        }
        __syncthreads();
    }
    const int64_t total = s_base[0], pages = s_base[1];
    for (int64_t t = total + threadIdx.x; t < a.capacity; t += kThreads) {
        a.slots[t] = -1;
        a.positions[t] = -1;
    }
    if (threadIdx.x == 0) {
        a.offsets[a.R] = static_cast<int32_t>(min(total, int64_t(0x7FFFFFFF)));
        a.counts[0] = static_cast<int32_t>(min(total, int64_t(0x7FFFFFFF)));
        a.counts[1] = static_cast<int32_t>(min(pages, a.num_free));
        a.counts[2] = static_cast<int32_t>(min(max(pages - a.num_free, int64_t(0)), int64_t(0x7FFFFFFF)));
        a.counts[3] = s_flags | (total > a.capacity ? BQD_SLOTS_TOKENS_CUT : 0);
    }
}

}  // namespace

cudaError_t launch_paged_slots(const SlotsArgs& a, cudaStream_t s)
{
    paged_slots_kernel<<<1, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace bqd
