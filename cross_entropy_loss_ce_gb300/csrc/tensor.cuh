// PTX wrappers for the 5th-generation tensor cores: tensor-map (TMA) loads into
// swizzled shared memory, tcgen05 matrix instructions on one CTA or on a pair
// of CTAs, their accumulators in tensor memory, and the mbarriers between them.
#pragma once

#include <cuda.h>

#include "device.cuh"

namespace gbce {

// One look at phase `parity` of an mbarrier that sleeps in hardware until the
// phase ends, 10 ms at most: waits that look again and again take issue slots
// and power from the matrix instructions (8192 x 128256, K 4096 forward: 5.06 ms
// so, 5.18 with the default sleep, 5.5 with tight loops).  CLUSTER: the other CTA
// of a pair arrives on it too.
template <bool CLUSTER>
__device__ __forceinline__ bool bar_try_wait(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    if constexpr (CLUSTER)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity), "r"(10000000u)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity), "r"(10000000u)
            : "memory");
    return done != 0;
}

// A wait that runs out sets *dead (shared memory); every later wait of the CTA
// then returns soon, so a failed copy ends the kernel instead of hanging it.
template <bool CLUSTER>
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int *dead)
{
    if (bar_try_wait<CLUSTER>(bar, parity))
        return true;
    const uint64_t t0 = globaltimer_ns();
    while (!bar_try_wait<CLUSTER>(bar, parity)) {
        if (*dead)
            return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            *dead = 1;
            return false;
        }
    }
    return true;
}

// One arrival on an mbarrier of this CTA / of any CTA of the cluster.
__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void bar_arrive_cluster(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
                 : "memory");
}

// After a failed wait: long enough for any copy or matrix instruction of the
// CTA that is still in flight to land before its memory is given up.
__device__ __forceinline__ void settle_after_failure()
{
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 50000000ull)
        __nanosleep(1000);
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// One box of a 2-D tensor map at (x, y) into this CTA's shared memory; its
// bytes count on `bar`, a shared::cluster address (pair form: either CTA's).
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap *map, int x, int y,
                                              uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int x, int y,
                                         uint32_t bar, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y), "l"(policy)
        : "memory");
}

// Tensor memory of this CTA (GROUP 2: of both CTAs of the pair, each running
// this): `cols` columns, whose address goes to the shared word `slot`.
template <int GROUP>
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols)
{
    if constexpr (GROUP == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
                     "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
                     "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}

template <int GROUP>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols)
{
    if constexpr (GROUP == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}

__device__ __forceinline__ void tc_fence_before()
{
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_after()
{
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// D (tensor memory) = A B^T (+ D when `add`): 16-bit operands in shared memory,
// fp32 sums.
template <int GROUP>
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add)
{
    if constexpr (GROUP == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(add)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(add)
            : "memory");
}

// One arrival on `bar` once every matrix instruction issued so far by this
// thread is done.  Pair form: on the barrier at that offset in both CTAs.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
}

// 32 columns of this warp's 32 tensor-memory lanes, lane i of the warp reading
// lane i (issue only; tmem_wait_ld before the values are used).
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}

// 16 columns.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}

// The loaded registers pass through the wait, so no use of them can be moved
// ahead of it.
template <int N>
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[N])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i)
        asm volatile("" : "+r"(r[i]));
}

// 32 columns straight into x[OFF ..] (issue only).
template <int OFF, int N>
__device__ __forceinline__ void tmem_ld32_into(uint32_t addr, float (&x)[N])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(x[OFF + 0]), "=f"(x[OFF + 1]), "=f"(x[OFF + 2]), "=f"(x[OFF + 3]),
          "=f"(x[OFF + 4]), "=f"(x[OFF + 5]), "=f"(x[OFF + 6]), "=f"(x[OFF + 7]),
          "=f"(x[OFF + 8]), "=f"(x[OFF + 9]), "=f"(x[OFF + 10]), "=f"(x[OFF + 11]),
          "=f"(x[OFF + 12]), "=f"(x[OFF + 13]), "=f"(x[OFF + 14]), "=f"(x[OFF + 15]),
          "=f"(x[OFF + 16]), "=f"(x[OFF + 17]), "=f"(x[OFF + 18]), "=f"(x[OFF + 19]),
          "=f"(x[OFF + 20]), "=f"(x[OFF + 21]), "=f"(x[OFF + 22]), "=f"(x[OFF + 23]),
          "=f"(x[OFF + 24]), "=f"(x[OFF + 25]), "=f"(x[OFF + 26]), "=f"(x[OFF + 27]),
          "=f"(x[OFF + 28]), "=f"(x[OFF + 29]), "=f"(x[OFF + 30]), "=f"(x[OFF + 31])
        : "r"(addr));
}

template <int N>
__device__ __forceinline__ void tmem_wait_into(float (&x)[N])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i)
        asm volatile("" : "+f"(x[i]));
}

// Shared-memory descriptor of a 16-bit operand tile in 128-byte-swizzled atoms
// of 8 rows x 128 bytes.  K-major (rows run along K): `sbo` = bytes from one
// group of 8 rows to the next.  MN-major (rows run along M or N, 64 values
// each): `sbo` = bytes from 8 K rows to the next 8, `lbo` = bytes from 64
// values of M or N to the next 64.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo)
{
    return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
           (static_cast<uint64_t>(sbo >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction descriptor of kind::f16 with fp32 sums: bf16 or fp16 operands,
// either of them MN-major, an M x N tile.
__host__ __device__ constexpr uint32_t mma_idesc(bool bf16, bool a_mn, bool b_mn, int m, int n)
{
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (a_mn ? 1u << 15 : 0u) |
           (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

}  // namespace gbce
