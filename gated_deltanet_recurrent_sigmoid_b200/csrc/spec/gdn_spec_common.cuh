// gdn_spec_common.cuh -- device helpers of the speculative-step kernels:
// thread-block clusters, distributed shared memory, element conversions.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "gdn_spec.h"
#include "mbarrier_sm100.cuh"

namespace gdn {
namespace spec {

// Every kernel here is launched with programmatic stream serialization: it may
// be scheduled while the kernel before it on the stream is ending, and waits
// (pdl_wait), before it touches global memory, until that one has completed.
// Back to back this saves 1 to 2.5 us a call (1 x 32768 probabilities 6.1 -> 3.7
// us, verification 8.2 -> 5.5).  No kernel calls for its successor early: its
// CTAs then wait where this one's still work (512 x 131072 probabilities 70.2 us
// against 68.8, 205,000 rows of maps 4.7 against 3.9).
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void report(uint32_t *status, uint32_t bits)
{
    if (status)
        atomicOr(status, bits);
}

// This thread's warp, the same register for the whole warp.  A shuffle: every
// lane has to call it.  Branches on it are
// then known to be uniform: shuffles behind a branch or loop that might be
// divergent are compiled to a path of about 230 clocks each instead of 24
// (measured), which __syncwarp() behind a loop avoids as well.
__device__ __forceinline__ int warp_index() { return __shfl_sync(~0u, static_cast<int>(threadIdx.x >> 5), 0); }

// ---- clusters.  A CTA learns of its peers' values by mbarriers in its own
// shared memory, which the peers' stores complete (st_peer): a cluster-wide
// barrier per exchange was measured to cost more than the stores, most of it
// in the fence of its release.  The barrier below runs once, behind the
// initialisation of those mbarriers.
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// Every thread of every CTA arrives and waits, its warp as one.  Warps that
// have nothing to publish arrive relaxed.
__device__ __forceinline__ void cluster_arrive(bool publishes)
{
    __syncwarp();
    if (publishes)
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    else
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait()
{
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A CTA that has given up a wait ends here: its peers may still store into its
// shared memory, so it stays until each of them has exited or is here too.
__device__ __forceinline__ void cluster_leave()
{
    __syncthreads();
    asm volatile("barrier.cluster.arrive.relaxed;\n\tbarrier.cluster.wait;" ::: "memory");
}

// Bounded wait, as sync::mbar_wait, that makes the peers' stores visible.
__device__ __forceinline__ bool mbar_try_peers(unsigned long long *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(sync::smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_peers(unsigned long long *bar, uint32_t parity)
{
    if (mbar_try_peers(bar, parity))
        return true;
    const uint64_t t0 = sync::global_ns();
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_peers(bar, parity))
            return true;
        if ((n & 63u) == 0u && sync::global_ns() - t0 > sync::WAIT_LIMIT_NS)
            return false;
    }
}

// This CTA's own arrival for the next phase of an exchange's mbarrier, which
// `bytes` of stores from the cluster's CTAs complete.  Copies of the library
// built for the timeout tests withhold it in the CTAs of one rank, or (-1) in
// all; product builds define neither switch.
__device__ __forceinline__ void expect_peers(unsigned long long *bar, uint32_t bytes)
{
#ifdef GDN_TEST_WITHHOLD_EXCHANGE
    if (GDN_TEST_WITHHOLD_EXCHANGE < 0 || cluster_rank() == static_cast<uint32_t>(GDN_TEST_WITHHOLD_EXCHANGE))
        return;
#endif
    sync::mbar_arrive_expect_tx(bar, bytes);
}
// The same for a bulk copy into this CTA's shared memory.
__device__ __forceinline__ void expect_copy(unsigned long long *bar, uint32_t bytes)
{
#ifdef GDN_TEST_WITHHOLD_COPY_RANK
    if (cluster_rank() == GDN_TEST_WITHHOLD_COPY_RANK)
        return;
#endif
    sync::mbar_arrive_expect_state_tx(bar, bytes);
}

// Address of this CTA's shared variable `p` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_addr(const void *p, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(sync::smem_addr(p)), "r"(rank));
    return r;
}
// Store to a peer's shared memory; completes 4 or 8 bytes on its mbarrier.
__device__ __forceinline__ void st_peer(uint32_t addr, float x, uint32_t bar)
{
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr),
                 "r"(__float_as_uint(x)), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void st_peer(uint32_t addr, double x, uint32_t bar)
{
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(addr),
                 "l"(__double_as_longlong(x)), "r"(bar)
                 : "memory");
}

// ---- elements
template <typename T> struct Elem;
template <> struct Elem<float> {
    static constexpr int PER16 = 4;
    __device__ static float get(float x) { return x; }
    __device__ static float put(float x) { return x; }
};
template <> struct Elem<__nv_bfloat16> {
    static constexpr int PER16 = 8;
    __device__ static float get(__nv_bfloat16 x) { return __bfloat162float(x); }
    __device__ static __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};

// The values of a 16-byte word.
__device__ __forceinline__ void unpack16(const uint4 &w, float (&x)[4], const float *)
{
    x[0] = __uint_as_float(w.x);
    x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z);
    x[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void unpack16(const uint4 &w, float (&x)[8], const __nv_bfloat16 *)
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

// The largest value of a 16-byte word; NaN is passed over (all NaN: NaN).
__device__ __forceinline__ float max16(const uint4 &w, const float *)
{
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
}
__device__ __forceinline__ float max16(const uint4 &w, const __nv_bfloat16 *)
{
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&w);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
}

// The largest of `most` and the word's elements as unsigned bit patterns (both
// halves of `most` for 16-bit elements), and whether one of them was not a
// finite number >= 0.
__device__ __forceinline__ uint32_t most_bits(const uint4 &w, uint32_t most, const float *)
{
    return max(max(max(w.x, w.y), max(w.z, w.w)), most);
}
__device__ __forceinline__ uint32_t most_bits(const uint4 &w, uint32_t most, const __nv_bfloat16 *)
{
    return __vmaxu2(__vmaxu2(__vmaxu2(w.x, w.y), __vmaxu2(w.z, w.w)), most);
}
__device__ __forceinline__ bool beyond_finite(uint32_t most, const float *) { return most >= 0x7f800000u; }
__device__ __forceinline__ bool beyond_finite(uint32_t most, const __nv_bfloat16 *)
{
    return (most & 0xffffu) >= 0x7f80u || most >= 0x7f800000u;
}

// N consecutive elements of shared memory at an address aligned to
// min(16, their size) bytes.
__device__ __forceinline__ void load_group(const float *p, float (&x)[4])
{
    unpack16(*reinterpret_cast<const uint4 *>(p), x, static_cast<const float *>(nullptr));
}
__device__ __forceinline__ void load_group(const float *p, float (&x)[8])
{
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load_group(const __nv_bfloat16 *p, float (&x)[8])
{
    unpack16(*reinterpret_cast<const uint4 *>(p), x, static_cast<const __nv_bfloat16 *>(nullptr));
}
__device__ __forceinline__ void load_group(const __nv_bfloat16 *p, float (&x)[4])
{
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    x[0] = __uint_as_float(w.x << 16);
    x[1] = __uint_as_float(w.x & 0xffff0000u);
    x[2] = __uint_as_float(w.y << 16);
    x[3] = __uint_as_float(w.y & 0xffff0000u);
}

// 2^x, relative error about 2^-22; -inf gives 0.
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The packed rows of sequence i: false (and a status bit) when cu_seqlens are
// not usable for it.
__device__ __forceinline__ bool rows_of(const int32_t *cu, int32_t T_fixed, int32_t T_tot, int32_t i, int32_t *start,
                                        int32_t *len)
{
    if (!cu) {
        *start = i * T_fixed;
        *len = T_fixed;
        return true;
    }
    const int32_t a = cu[i], b = cu[i + 1];
    *start = a;
    *len = b - a;
    return a >= 0 && b >= a && b <= T_tot;
}

}  // namespace spec
}  // namespace gdn
