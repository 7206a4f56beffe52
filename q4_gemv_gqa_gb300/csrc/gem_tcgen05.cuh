// gem_tcgen05.cuh — fifth-generation tensor core building blocks (sm_103a): tensor memory, tcgen05.mma on
// e4m3 operands in shared memory, completion through mbarriers, and the cluster forms of both.
#pragma once

#include "gem_device.cuh"

namespace gem {

// ---- descriptors -----------------------------------------------------------------------
// Operand in shared memory, K-major, rows of 128 bytes with the 128-byte swizzle (what a tensor map of that
// swizzle writes): 8 rows are 1024 bytes.  Steps along K inside the 128 bytes add to the start address.
__device__ __forceinline__ uint64_t umma_desc(uint32_t smem_addr) {
    constexpr uint64_t base = (uint64_t(2) << 61)           // 128-byte swizzle
                              | (uint64_t(1) << 46)         // descriptor version
                              | (uint64_t(1024 >> 4) << 32)  // bytes from 8 rows to the next 8
                              | (uint64_t(1) << 16);
    return base | ((smem_addr >> 4) & 0x3fff);
}
// e4m3 x e4m3 -> fp32, both operands K-major, m rows of D and n columns
__host__ __device__ constexpr uint32_t umma_idesc_e4m3(int m, int n) {
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// ---- tensor memory ---------------------------------------------------------------------
template <int G>   // CTAs that work on one tile
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, int cols) {   // one warp; G 2: one warp of each CTA
    if constexpr (G == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
}
template <int G>
__device__ __forceinline__ void tmem_free(uint32_t addr, int cols) {
    if constexpr (G == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// N columns of the warp's 32 lanes (its quarter of the lanes, warp index mod 4, is in the address)
template <int N>
__device__ __forceinline__ void tmem_ld(float (&v)[N], uint32_t addr) {
    static_assert(N == 8 || N == 16 || N == 32);
    uint32_t r[N];
    if constexpr (N == 8)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(addr));
    else if constexpr (N == 16)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                     : "r"(addr));
    else
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                     : "r"(addr));
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ---- products ----------------------------------------------------------------------------
// The calls below are made by a whole warp, whose elected lane acts: addresses and descriptors then stay in
// uniform registers (from one lane of a diverged warp a product took 70 cycles to issue and a copy 107).
// d = a x b over 128 bytes of K (four products of 32, the first of which overwrites d)
template <int G>
__device__ __forceinline__ void umma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
    if constexpr (G == 1)
        asm volatile(
            "{\n .reg .pred e;\n .reg .b64 x, y;\n elect.sync _|e, 0xffffffff;\n"
            " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, 0;\n"
            " add.s64 x, %1, 2;\n add.s64 y, %2, 2;\n @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, 1;\n"
            " add.s64 x, %1, 4;\n add.s64 y, %2, 4;\n @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, 1;\n"
            " add.s64 x, %1, 6;\n add.s64 y, %2, 6;\n @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, 1;\n}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred e;\n .reg .b64 x, y;\n elect.sync _|e, 0xffffffff;\n"
            " @e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, 0;\n"
            " add.s64 x, %1, 2;\n add.s64 y, %2, 2;\n @e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], x, y, %3, 1;\n"
            " add.s64 x, %1, 4;\n add.s64 y, %2, 4;\n @e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], x, y, %3, 1;\n"
            " add.s64 x, %1, 6;\n add.s64 y, %2, 6;\n @e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], x, y, %3, 1;\n}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc)
            : "memory");
}
// One arrival on `bar` (G 2: on the barrier at that place of the CTAs in `mask`) when the products issued so far are done.
template <int G>
__device__ __forceinline__ void umma_commit(uint64_t* bar, uint32_t mask = 1) {
    if constexpr (G == 1)
        asm volatile(
            "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
            " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar))
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
            " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}\n" ::"r"(
                smem_u32(bar)),
            "h"(static_cast<uint16_t>(mask))
            : "memory");
}
__device__ __forceinline__ void warp_expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n @e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}\n" ::"r"(
            smem_u32(bar)),
        "r"(bytes)
        : "memory");
}
__device__ __forceinline__ void warp_tma_2d(uint32_t dst, const CUtensorMap* tm, int32_t c0, int32_t c1, uint64_t* bar, uint64_t policy) {
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
        " @e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;\n}\n" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void warp_tma_3d(uint32_t dst, const CUtensorMap* tm, int32_t c0, int32_t c1, int32_t c2, uint64_t* bar,
                                            uint64_t policy) {
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
        " @e cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;\n}\n" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}
// Registers of the executing warpgroup (all of its warps): of the block's own at launch.
template <int N>
__device__ __forceinline__ void regs_take() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_give() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
// Shared memory to global memory; the source may be written again when at most `left` later groups are being read.
__device__ __forceinline__ void warp_tma_store_2d(const CUtensorMap* tm, int32_t c0, int32_t c1, uint32_t src) {
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
        " @e cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n @e cp.async.bulk.commit_group;\n}\n" ::"l"(
            reinterpret_cast<uint64_t>(tm)),
        "r"(c0), "r"(c1), "r"(src)
        : "memory");
}
template <int LEFT>
__device__ __forceinline__ void tma_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(LEFT) : "memory"); }
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }
// mbar_wait of a whole warp, which stays converged: false where the wait ran out, or where another warp's did
// (looked at only while this one has to wait: a phase that is done costs one test).
__device__ __forceinline__ bool warp_wait_slow(uint64_t* bar, uint32_t parity, int* status, volatile int* dead) {
    bool ok = false;
    const uint64_t t0 = globaltimer_ns(), limit = wait_limit_ns();
    while (true) {
        for (int i = 0; i < 64 && !ok; ++i) ok = mbar_try_wait(bar, parity);
        if (ok || *dead) break;
        if (globaltimer_ns() - t0 > limit) {
            if (status) atomicOr(status, GEM_DEVFLAG_TIMEOUT);
            break;
        }
    }
    return __all_sync(~0u, ok);
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* status, volatile int* dead) {
    if (__all_sync(~0u, mbar_try_wait(bar, parity))) return true;
    return warp_wait_slow(bar, parity, status, dead);
}

// Two sums in one register pair: (lo, hi) += (a, b) * (s, s), s given twice by pair_of.  Volatile, so that the adds
// stay between the reads of tensor memory that they stand between.
__device__ __forceinline__ uint64_t pair_of(float v) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ void pair_fma(uint64_t& acc, float a, float b, uint64_t s) {
    asm volatile("{\n .reg .b64 t;\n mov.b64 t, {%1, %2};\n fma.rn.f32x2 %0, t, %3, %0;\n}\n" : "+l"(acc) : "f"(a), "f"(b), "l"(s));
}
__device__ __forceinline__ float2 pair_get(uint64_t acc) {
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(acc));
    return v;
}

// ---- clusters ------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the address of this CTA's shared-memory location in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ float ld_peer(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_peer4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mbar_arrive_peer(uint32_t addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// Into this CTA's shared memory, its bytes counted on a barrier of either CTA of the pair.
__device__ __forceinline__ void warp_tma_2d_pair(uint32_t dst, const CUtensorMap* tm, int32_t c0, int32_t c1, uint32_t bar, uint64_t policy) {
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
        " @e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;\n}\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(bar), "l"(policy)
        : "memory");
}
__device__ __forceinline__ uint64_t l2_policy_evict_last() {
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}

}  // namespace gem
