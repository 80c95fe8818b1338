// Steps that the kernels on tensor memory share: barriers with a limit, TMA copies,
// products and accumulator reads (kernels grouped.cuh and route.cuh).
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "common.cuh"

namespace fgm {
namespace tc {

__device__ __forceinline__ uint32_t saddr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ long long now_ns()
{
    long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ void bar_init(unsigned long long *bar, int arrivals)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(bar)), "r"(arrivals) : "memory");
}

__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Waits up to a tenth of a second for what is in flight after an abort. (The timer is
// read when there is something to wait for: it takes a fifth of a microsecond.)
__device__ __forceinline__ void bar_drain(uint32_t bar, uint32_t parity)
{
    if (bar_try(bar, parity))
        return;
    const long long end = now_ns() + 100000000LL;
    while (!bar_try(bar, parity) && now_ns() < end)
        ;
}

// A wait on a barrier of this CTA that gives up after timeout_ns or when another
// wait of the CTA has: false, with FGM_STATUS_WAIT_TIMEOUT and a report behind
// the status word.
struct Waiter {
    int *abort;              // shared
    int32_t *status;
    long long timeout_ns;

    // Whether a wait is to give up; asked now and then.
    __device__ __forceinline__ bool over(long long &since, int site, int index) const
    {
        if (*reinterpret_cast<volatile int *>(abort))
            return true;
        if (since == 0)
            since = now_ns();
        if (now_ns() - since <= timeout_ns)
            return false;
        *reinterpret_cast<volatile int *>(abort) = 1;
        if ((atomicOr(status, FGM_STATUS_WAIT_TIMEOUT) & FGM_STATUS_WAIT_TIMEOUT) == 0) {
            status[1] = site;
            status[2] = blockIdx.x;
            status[3] = threadIdx.x >> 5;
            status[4] = index;
        }
        return true;
    }

    __device__ __forceinline__ bool operator()(unsigned long long *bar, uint32_t phase, int site, int index) const
    {
        const uint32_t a = saddr(bar);
        long long since = 0;
        for (int it = 0;; ++it) {
            if (bar_try(a, phase & 1))
                return true;
            if ((it & 255) == 255 && over(since, site, index))
                return false;
        }
    }

    // The same for a count in shared memory to pass n. (Seldom; out of line it costs its caller no registers.)
    __device__ __noinline__ bool passed(const uint32_t *count, uint32_t n, int site, int index) const
    {
        const uint32_t a = saddr(count);
        long long since = 0;
        for (int it = 0;; ++it) {
            uint32_t v;
            asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
            if (v > n)
                return true;
            if ((it & 255) == 255 && over(since, site, index))
                return false;
        }
    }
};

// A shared-memory address of this CTA in the pair's first CTA.
__device__ __forceinline__ uint32_t in_first(uint32_t a)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(a));
    return r;
}

// The word at this shared-memory address in the pair's second CTA.
__device__ __forceinline__ uint32_t of_second(uint32_t a)
{
    uint32_t r;
    asm volatile("{\n\t.reg .b32 p;\n\tmapa.shared::cluster.u32 p, %1, 1;\n\tld.shared::cluster.u32 %0, [p];\n\t}" : "=r"(r) : "r"(a) : "memory");
    return r;
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() { asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory"); }

__device__ __forceinline__ bool elect()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// All of an SM's tensor memory, for this CTA alone (G = 1) or its pair (G = 2); by
// one warp (of each CTA), behind the wait for the kernel before.
template <int G>
__device__ __forceinline__ void memory_take(uint32_t *at)
{
    asm volatile("tcgen05.alloc.cta_group::%1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(saddr(at)), "n"(G) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::%0.sync.aligned;" ::"n"(G) : "memory");
}

template <int G>
__device__ __forceinline__ void memory_free(uint32_t at)
{
    asm volatile("tcgen05.dealloc.cta_group::%1.sync.aligned.b32 %0, 512;" ::"r"(at), "n"(G) : "memory");
}

// K-major operand in the 128-byte swizzle: atoms of 8 rows x 128 bytes, 1024 bytes apart.
__device__ __forceinline__ uint64_t operand(uint32_t addr)
{
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// d (+)= a b of 32 bytes of K: E4M3 (8-bit operands) or bf16, fp32 accumulators.
template <int G, bool kBytes>
__device__ __forceinline__ void product(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    if constexpr (kBytes)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::%5.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add)), "n"(G)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::%5.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add)), "n"(G)
            : "memory");
}

// d (+)= a b0 + a b1 in 8 bits: a is read from shared memory once and kept for the second product.
template <int G>
__device__ __forceinline__ void product_twice(uint32_t d, uint64_t a, uint64_t b0, uint64_t b1, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %5, 0;\n\tsetp.eq.u32 q, 0, 0;\n\t"
        "tcgen05.mma.cta_group::%6.kind::f8f6f4.collector::a::fill [%0], %1, %2, %4, p;\n\t"
        "tcgen05.mma.cta_group::%6.kind::f8f6f4.collector::a::lastuse [%0], %1, %3, %4, q;\n\t}" ::"r"(d),
        "l"(a), "l"(b0), "l"(b1), "r"(idesc), "r"(static_cast<uint32_t>(add)), "n"(G)
        : "memory");
}

// M x N accumulators; both operands E4M3 or both bf16.
__device__ __forceinline__ constexpr uint32_t product_desc(int M, int N, bool bytes)
{
    return (1u << 4) | (bytes ? 0u : (1u << 7) | (1u << 10)) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

// This thread's products so far arrive on the barrier when they are done: of both CTAs of a pair,
__device__ __forceinline__ void commit_both(unsigned long long *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(saddr(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// or of this CTA.
template <int G>
__device__ __forceinline__ void commit(unsigned long long *bar)
{
    asm volatile("tcgen05.commit.cta_group::%1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(saddr(bar)), "n"(G) : "memory");
}

// Eight columns of this warp's 32 lanes: a lane's own,
__device__ __forceinline__ void read(uint32_t at, uint32_t (&u)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                 : "r"(at)
                 : "memory");
}

// or as products hold them: of lanes l / 4, l / 4 + 8, + 16 and + 24 the columns 2 (l % 4) and the next.
__device__ __forceinline__ void read_pairs(uint32_t at, uint32_t (&u)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                 : "r"(at)
                 : "memory");
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                 : "r"(at + (16u << 16))
                 : "memory");
}

__device__ __forceinline__ void read_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// The kernel before this one in the stream may still run when this one starts (host.h).
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;"); }

}  // namespace tc
}  // namespace fgm
