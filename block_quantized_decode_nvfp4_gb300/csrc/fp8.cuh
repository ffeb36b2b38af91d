// fp8.cuh -- device helpers of the calls on 8-bit activations: E4M3 codes with
// a scale for each block of 128, and the PTX of the products (tensor copies,
// tcgen05 kind::f8f6f4, tensor memory, clusters).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include <cstdint>

#include "f32x2.cuh"
#include "stream.cuh"

namespace bqd {

// ---------------------------------------------------------------- E4M3 blocks
// The largest magnitude of three, NaN if there is one (an infinity is larger
// than any number), so that a block's largest tells what the block holds.
__device__ __forceinline__ float max_abs(float a, float b, float c)
{
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max_abs(float a, float b) { return max_abs(a, b, b); }

// The scale of a block of largest magnitude amax: amax / 448, rounded once and
// at least the smallest normal fp32, so that no quotient passes 448 by more than
// its rounding; NaN where the block has a NaN or an infinity. The quotient is a
// product with 1 / 448 and one step from its remainder (Markstein 1990), which
// is exact down to that smallest scale.
__device__ __forceinline__ float block_scale(float amax)
{
    constexpr float kInv = 1.f / 448.f;
    const float q = amax * kInv, s = __fmaf_rn(__fmaf_rn(q, -448.f, amax), kInv, q);
    return amax < INFINITY ? fmaxf(s, 1.17549435e-38f) : __uint_as_float(0x7FC00000u);
}

// Codes of quotients by one scale, each the fp32 quotient rounded to E4M3. A
// product with the rounded reciprocal alone would now and then land on the
// other side of a boundary between codes: one step from its remainder makes it
// the quotient, rounded once, as long as the remainder keeps its bits (scales
// from 2^-60); smaller scales divide, and so does NaN, but for the smallest.
__device__ __forceinline__ uint32_t e4m3x2(uint64_t v)  // code of the first in the low byte
{
    float a, b;
    unpack(v, a, b);
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
// The quotients of v by s through its reciprocal, negated (the last step then keeps the
// sign of zeros); by division.
template <int N>
__device__ __forceinline__ void quotients(uint64_t (&v)[N], float s)
{
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    inv = __fmaf_rn(__fmaf_rn(-s, inv, 1.f), inv, inv);
    const uint64_t i2 = pack(-inv, -inv), s2 = pack(s, s);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint64_t q = mul2(v[i], i2);
        v[i] = fma2(fma2(q, s2, v[i]), i2, q);
    }
}
template <int N>
__device__ __forceinline__ void divide(uint64_t (&v)[N], float s)
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float a, b;
        unpack(v[i], a, b);
        v[i] = pack(__fdiv_rn(a, s), __fdiv_rn(b, s));
    }
}
// v to quotients by s; returns what four of their codes are to be XORed with.
template <int N>
__device__ __forceinline__ uint32_t scale_down(uint64_t (&v)[N], float s)
{
    if (s >= 8.6736174e-19f) {  // 2^-60; false for NaN
        quotients(v, s);
        return 0x80808080u;
    }
    if (s == 1.17549435e-38f) {  // a block of zeros, such as a row past the last token: 2^126 is exact
        const uint64_t inv = pack(8.5070592e37f, 8.5070592e37f);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = mul2(v[i], inv);
    } else {
        divide(v, s);
    }
    return 0;
}
// Codes of four quotients, x (above) included.
__device__ __forceinline__ uint32_t e4m3x4(uint64_t a, uint64_t b, uint32_t x) { return (e4m3x2(a) | (e4m3x2(b) << 16)) ^ x; }

__device__ __forceinline__ uint32_t to_bf16x2(float x, float y)
{
    const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// ---------------------------------------------------------------- tensor cores
__device__ __forceinline__ void fp8_pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void fp8_pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
        : "memory");
}

// A box from shared memory to global memory, in groups of this thread: rows and
// columns past the tensor's end are left out.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int c0, int c1)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Until all groups but the last N have been read from shared memory; until all have been written.
template <int N>
__device__ __forceinline__ void bulk_wait_read()
{
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Shared-memory descriptor of a K-major operand with the 128-byte swizzle: rows
// of 128 bytes (128 k) in atoms of 8 rows, 1024 bytes apart; an MMA's 32 k are
// 32 bytes further into the row.
__device__ __forceinline__ uint64_t fp8_desc(uint32_t addr)
{
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(1) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
// Instruction descriptor: fp32 D (bit 4), A and B E4M3 (0), both K-major.
constexpr uint32_t fp8_idesc(int M, int N)
{
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void fp8_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void fp8_commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ bool fp8_elect()
{
    uint32_t pred = 0;
    asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(pred));
    return pred != 0;
}
// 16 or 32 columns of this warp's 32 lanes; several loads may share one wait.
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t* r)
{
    static_assert(N == 16 || N == 32, "columns of one load");
    if constexpr (N == 16)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
            "%15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
              "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(at)
            : "memory");
    else
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
            "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
              "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
              "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
              "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
            : "r"(at)
            : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// A look at a phase that does not wait for it (try_wait may, for microseconds).
__device__ __forceinline__ bool fp8_look(uint64_t* bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// A warp's wait: every lane looks, so that one that finds the phase complete
// costs no exchange; lane 0's word counts.
__device__ __forceinline__ bool fp8_wait(uint64_t* bar, uint32_t parity, unsigned int* err)
{
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
    return mbar_wait_warp(bar, parity, err);
}

// ---------------------------------------------------------------- pairs of CTAs
// A copy into this CTA's shared memory that is counted at a barrier of either
// CTA of its pair (bar: an address in the cluster).
__device__ __forceinline__ void tma_2d_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
        "{%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
// A product of the pair, issued by its first CTA: rows and columns of both.
__device__ __forceinline__ void fp8_mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// An arrival at the barrier of this address in both CTAs, after the products issued so far.
__device__ __forceinline__ void fp8_commit_pair(uint64_t* bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}
// Arrivals at a barrier of the cluster. They hand on what the tensor cores and
// copies use, and no thread's stores: a wider release than the default one would
// wait for every load in flight.
__device__ __forceinline__ void arrive_expect_cluster(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ uint32_t cta_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cta_map(uint32_t local, uint32_t rank)
{
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    return remote;
}
// A store to another CTA's shared memory that counts its bytes at a barrier there.
__device__ __forceinline__ void st_async(uint32_t addr, float v, uint32_t bar)
{
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr),
                 "r"(__float_as_uint(v)), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// A copy from this CTA's shared memory to another's, counted at a barrier there.
__device__ __forceinline__ void bulk_s2s(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "r"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// A warp's bounded wait for other CTAs' stores or arrivals, every lane by itself.
__device__ __forceinline__ bool fp8_wait_cluster(uint64_t* bar, uint32_t parity, unsigned int* err,
                                                 long long limit = kWaitCycles)
{
    bool done = try_wait_cluster(bar, parity);
    if (!done) {
        const long long t0 = clock64();
        do {
            done = try_wait_cluster(bar, parity);
        } while (!done && clock64() - t0 < limit);
        if (!done) atomicOr(err, kErrWaitTimeout);
    }
    return __all_sync(0xFFFFFFFFu, done);
}

}  // namespace bqd
