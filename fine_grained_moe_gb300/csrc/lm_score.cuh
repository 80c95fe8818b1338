// Log probabilities from hidden rows (fgm_lm_head_logprobs): the tied lm_head
//   z[n][v] = sum_j h[n][j] emb[v][j]
// with the sums of logprobs.cuh in its epilogue, so that logits are never stored.
//
// 2 * 2816 operations a logit: bound by the tensor pipe from about 300 rows on,
// by the embedding's 1.48 GB below. 1,021 rows of 262,144 words take 0.84 ms, 1.80
// PFLOP/s, in short runs (0.95 ms, 1.59, where the part settles at its sustained
// rate): the products 0.81 with the tensor pipe 92 % busy, the join 0.02, the rest
// starts and the last epilogue. 16 rows take 264 us, 5.6 TB/s, and 256 rows 288 us.
// (Up to 8 rows are the persistent lm_head kernel's.) Rows are taken 256 at a time:
// 300 cost what 512 do, 0.45 ms. Built for the tensor pipe: a pair of CTAs
// (cta_group::2) holds 256 rows x 256 words in tensor memory, each CTA loading
// its 128 rows and half of the words, 64 bytes per cycle and SM at the full rate
// where one CTA on 128 x 256 would need 96.
//  * TMA copies boxes of two slices of 128 rows x 128 bytes (64 elements of K) in
//    the 128-byte swizzle into a ring (3 stages; 6 for a few rows, whose copies are
//    no larger than the rows), the second CTA's bytes counted on the first's
//    barriers; rows past N and words past V arrive as zeros. (A CTA that arrives
//    for its own bytes, the second across the pair: 30 % slower.)
//  * The first CTA's issuing warp runs M = 256, N = 256, K = 16 products into one
//    of two accumulators (2 x 256 columns), so that the next tile's products run
//    under this tile's epilogue.
//  * Eight epilogue warps per CTA own a row and half of a tile's columns a
//    thread: 16 at a time the logits go into the running (m, l, w), but those that
//    beat the row's L-th best (L = 12, or 20 for more than 8 alternatives) into
//    its list, sorted in registers, and what they push out of it into the sums (14
//    us of 16 rows' 264). A row meets about L (1 + ln(n / L)) such logits among n,
//    and a warp waits for each of its 32 rows' in turn, so an insertion decides
//    every place of the list at once (five instructions a place and none that waits
//    for another: with a bubble pass through the list the epilogue was longer than
//    the products, 333 us on 16 rows, 0.91 ms on 1,021).
//  * An item is 256 rows x a range of words; a pair takes items in turn, a row's
//    state stays in registers over the range, and k_lm_join merges the ranges.
//
// Precision. The tensor pipe adds 16 products at a time to an fp32 accumulator
// and truncates: 176 additions take up to 176 ulps off a logit, in one
// direction, measured 2e-5 at logits near 10. That is too much for the few large
// logits, which are what the outputs are made of, so the join computes them
// again: the row's L best and the given token with fp32 multiply-adds (88 a lane
// and a tree), orders the alternatives by these and adds them to the sums of all
// others. (Listed logits are never in those sums: taken out of a sum by their first
// values they would leave its rounding, and at a low temperature the first value of
// the largest is far from the second: T = 1e-6 gave infinities.) The others' share
// of the sums is small, or their logits are, with their ulps over T.
// Pairs whose items are the same words and other rows run at the same time, so
// the embedding comes from HBM once and from L2 for the others.
#pragma once

#include <cuda.h>

#include "logprobs.cuh"
#include "pair_copies.h"

namespace fgm {
namespace score {

constexpr int kLmThreads = 384;                  // copies, products, -, -, eight epilogue warps
constexpr int kLmStages = 12;                    // at most
constexpr int kLmBox = 128 * 128;                // 128 words x 128 bytes
constexpr int kLmBoxes = 2;                      // boxes of 64 elements of K in a stage
constexpr int kLmWords = 256;                    // words of a tile
constexpr int kLmRows = 256;                     // rows of a pair
constexpr int kLmK = kH / (64 * kLmBoxes);       // stages of a tile
constexpr int kLmSmem = 226 * 1024;
static_assert(kH % (64 * kLmBoxes) == 0, "K must split into whole stages");

struct LmArgs {
    int64_t N;
    int V;
    float T;
    int h_rows;              // rows of a copy of hidden rows: 128, or all there are rounded up to 8
    int stages;              // of the ring: h_rows hidden rows, then 128 words
    int splits;              // word ranges
    int64_t items;           // row tiles * splits
    Part *part;              // [N][splits][2 halves of the columns]
    int32_t *status;
    long long timeout_ns;
};

struct LmShared {
    unsigned long long full[kLmStages], empty[kLmStages], tfull[2], tempty[2], drained;
    uint32_t tmem;
    int abort;
    uint32_t issued;         // copies that this CTA issued, and the last ring's bytes,
    uint32_t bytes[kLmStages], others[kLmStages];       // its own and the other's
};

__device__ __forceinline__ uint32_t saddr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ long long now_ns()
{
    long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

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

__device__ __forceinline__ bool lm_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Waits up to a tenth of a second for what is in flight after an abort.
__device__ __forceinline__ void lm_drain(uint32_t bar, uint32_t parity)
{
    const long long end = now_ns() + 100000000LL;
    while (!lm_try(bar, parity) && now_ns() < end)
        ;
}

__device__ __forceinline__ bool lm_elect()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

// K-major operand in the 128-byte swizzle: atoms of 8 rows x 128 bytes, 1024 bytes apart.
__device__ __forceinline__ uint64_t lm_desc(uint32_t addr)
{
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// Commits this thread's products to a barrier of both CTAs.
__device__ __forceinline__ void lm_commit(unsigned long long *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(saddr(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

__device__ __forceinline__ void lm_copy(uint32_t dst, const CUtensorMap *map, int y, int z, uint32_t bar, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(z), "r"(bar), "l"(policy)
        : "memory");
}

// L: entries of a row's list.
template <int L>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kLmThreads, 1)
    k_lm_score(const __grid_constant__ CUtensorMap hmap, const __grid_constant__ CUtensorMap emap, const LmArgs p)
{
    // fp32 += bf16 x bf16, M = 256, N = 256
    constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(kLmWords >> 3) << 17) |
                                (static_cast<uint32_t>(kLmRows >> 4) << 24);
    extern __shared__ uint8_t dsm_raw[];
    __shared__ LmShared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t rank;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    uint8_t *dsm = dsm_raw + ((1024u - (saddr(dsm_raw) & 1023u)) & 1023u);
    // (With few hidden rows the first operand's 128 run on into the stage's words:
    // rows of the accumulator that nobody reads.)
    const uint32_t ring = saddr(dsm), h_box = p.h_rows * 128, words_at = kLmBoxes * h_box,
                   stage = words_at + kLmBoxes * kLmBox, stages = p.stages;
    const int pairs = gridDim.x / 2, pair = blockIdx.x / 2;
    const int tiles = (p.V + kLmWords - 1) / kLmWords;

    if (tid == 0) {
        auto init = [](unsigned long long *b, int n) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(b)), "r"(n) : "memory");
        };
        for (int i = 0; i < kLmStages; ++i) {
            init(&sh.full[i], 1);
            init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            init(&sh.tfull[i], 1);
            init(&sh.tempty[i], 16);             // the epilogue warps of both CTAs
        }
        init(&sh.drained, 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // (behind the wait: a kernel before this one that lets it start early may not have taken its own tensor memory yet)
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(saddr(&sh.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const uint32_t tmem = sh.tmem;

    // bounded wait on a barrier of this CTA; false on timeout or abort
    auto wait = [&](unsigned long long *bar, uint32_t phase, int site, int index) -> bool {
        const uint32_t a = saddr(bar);
        long long since = 0;
        for (int it = 0;; ++it) {
            if (lm_try(a, phase & 1))
                return true;
            if ((it & 255) == 255) {
                if (*reinterpret_cast<volatile int *>(&sh.abort))
                    return false;
                if (since == 0)
                    since = now_ns();
                if (now_ns() - since > p.timeout_ns) {
                    *reinterpret_cast<volatile int *>(&sh.abort) = 1;
                    if ((atomicOr(p.status, FGM_STATUS_WAIT_TIMEOUT) & FGM_STATUS_WAIT_TIMEOUT) == 0) {
                        p.status[1] = site;
                        p.status[2] = blockIdx.x;
                        p.status[3] = threadIdx.x >> 5;
                        p.status[4] = index;
                    }
                    return false;
                }
            }
        }
    };
    auto range = [&](int64_t item, int &t0, int &t1) {
        const int s = static_cast<int>(item % p.splits);
        t0 = static_cast<int>(static_cast<int64_t>(tiles) * s / p.splits);
        t1 = static_cast<int>(static_cast<int64_t>(tiles) * (s + 1) / p.splits);
    };

    if (warp == 0) {
        // ------------------------------------------------------------ copies (each CTA its own rows and words)
        if (lane == 0) {
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&hmap)) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&emap)) : "memory");
            uint64_t words, rows;
            asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(rows));
            if (p.items == p.splits)
                asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(words));
            else
                asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(words));
            bool ok = true;
            uint32_t n = 0;
            for (int64_t item = pair; item < p.items && ok; item += pairs) {
                int t0, t1;
                range(item, t0, t1);
                // (a CTA without rows copies none; its half of the accumulator is never read)
                const int y0 = static_cast<int>(item / p.splits) * kLmRows, y = y0 + rank * 128;
                auto bytes = [&](int y) { return kLmBoxes * (kLmBox + (y < p.N ? h_box : 0)); };
                const uint32_t mine = bytes(y), others = bytes(y0 + (1 - rank) * 128);
                for (int t = t0; t < t1 && ok; ++t)
                    for (int ks = 0; ks < kLmK; ++ks, ++n) {
                        const uint32_t slot = n % stages;
                        if (n >= stages && !(ok = wait(&sh.empty[slot], n / stages - 1, 30, ks)))
                            break;
                        const uint32_t bar = in_first(saddr(&sh.full[slot])), dst = ring + slot * stage;
                        if (rank == 0)
                            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(&sh.full[slot])),
                                         "r"(mine + others)
                                         : "memory");
                        sh.bytes[slot] = mine;
                        sh.others[slot] = others;
                        lm_copy(dst + words_at, &emap, t * kLmWords + rank * 128, ks * kLmBoxes, bar, words);
                        if (y < p.N)
                            lm_copy(dst, &hmap, y, ks * kLmBoxes, bar, rows);
                    }
            }
            sh.issued = n;
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ products (the first CTA's warp for both)
        if (rank == 0) {
            const bool lead = lm_elect();
            bool ok = true;
            uint32_t n = 0, tile = 0;
            for (int64_t item = pair; item < p.items && ok; item += pairs) {
                int t0, t1;
                range(item, t0, t1);
                for (int t = t0; t < t1 && ok; ++t, ++tile) {
                    const uint32_t buf = tile & 1;
                    if (tile >= 2)
                        ok = wait(&sh.tempty[buf], (tile >> 1) - 1, 31, t);
                    for (int ks = 0; ks < kLmK; ++ks, ++n) {
                        const uint32_t slot = n % stages;
                        ok = ok && wait(&sh.full[slot], n / stages, 32, ks);
                        ok = __all_sync(0xFFFFFFFFu, ok);
                        if (!ok)
                            break;
                        if (lead) {
                            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                            const uint64_t a = lm_desc(ring + slot * stage), b = lm_desc(ring + slot * stage + words_at);
#pragma unroll
                            for (int kk = 0; kk < 4 * kLmBoxes; ++kk)
                                asm volatile(
                                    "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                                    "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem + buf * kLmWords),
                                    "l"(a + (kk >> 2) * (h_box >> 4) + (kk & 3) * 2), "l"(b + (kk >> 2) * (kLmBox >> 4) + (kk & 3) * 2), "r"(kIdesc), "r"(static_cast<uint32_t>((ks | kk) != 0))
                                    : "memory");
                            lm_commit(&sh.empty[slot]);
                            if (ks == kLmK - 1)
                                lm_commit(&sh.tfull[buf]);
                        }
                        __syncwarp();
                    }
                }
            }
            // every issued product completes before the tensor memory is released
            if (lead) {
                asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(saddr(&sh.drained))
                             : "memory");
                lm_drain(saddr(&sh.drained), 0);
            }
            __syncwarp();
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------ epilogue: a thread is a row, of half the columns
        const int quarter = warp & 3, r = quarter * 32 + lane, half = (warp - 4) >> 2;
        const float c = per_nat(p.T);
        bool alive = true;
        uint32_t tile = 0;
        for (int64_t item = pair; item < p.items; item += pairs) {
            int t0, t1;
            range(item, t0, t1);
            const int64_t row = item / p.splits * kLmRows + rank * 128 + r;
            const int split = static_cast<int>(item % p.splits);
            const bool live = row - lane < p.N;  // (of the warp: some row is one)
            Sums s;
            s.clear();
            int nan = 0;
            float lv[L];                         // best first
            int32_t li[L];
#pragma unroll
            for (int j = 0; j < L; ++j) {
                lv[j] = __int_as_float(0x7FC00000);
                li[j] = kNone;
            }
            for (int t = t0; t < t1; ++t, ++tile) {
                const uint32_t buf = tile & 1;
                if (alive)
                    alive = wait(&sh.tfull[buf], tile >> 1, 33, t);
                alive = __all_sync(0xFFFFFFFFu, alive);
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                // 16 columns at a time, the next on their way meanwhile
                uint32_t u[2][16];
                const int c_end = live ? (half + 1) * (kLmWords / 2) : 0;
                auto load = [&](int c0, uint32_t (&u)[16]) {
                    asm volatile(
                        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                        "%14, %15}, [%16];"
                        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
                          "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
                        : "r"(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + buf * kLmWords + c0)
                        : "memory");
                };
                auto columns = [&](int c0, uint32_t (&u)[16], uint32_t (&ahead)[16]) {
                    __syncwarp();
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                    float v[kVals];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        asm volatile("" : "+r"(u[j]));
                        v[j] = __uint_as_float(u[j]);
                    }
                    if (c0 + 16 < c_end)
                        load(c0 + 16, ahead);
                    const int v0 = t * kLmWords + c0;
                    if (v0 + 16 > p.V)
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            v[j] = v0 + j < p.V ? v[j] : -INFINITY;
                    float mx = largest(v, nan);
                    if (!(mx <= lv[L - 1])) {
                        // (words come in order: an equal logit later does not replace an earlier one; an empty place's NaN
                        // is below everything)
                        unsigned in = 0;
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            in |= !(v[j] <= lv[L - 1]) ? 1u << j : 0u;
                        if (v0 + 16 > p.V)
                            in &= v0 < p.V ? (1u << (p.V - v0)) - 1 : 0u;
                        for (; in; in &= in - 1) {
                            const int j = __ffs(in) - 1;
                            float x[8];
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                x[q] = j & 8 ? v[q + 8] : v[q];
#pragma unroll
                            for (int o = 4; o > 0; o >>= 1)
#pragma unroll
                                for (int q = 0; q < o; ++q)
                                    x[q] = j & o ? x[q + o] : x[q];
                            // the list's last leaves it for the sums, in the new one's place among the 16
                            const float last = lv[L - 1] == lv[L - 1] ? lv[L - 1] : -INFINITY, left = !(x[0] <= lv[L - 1]) ? last : x[0];
#pragma unroll
                            for (int q = 0; q < 16; ++q)
                                v[q] = q == j ? left : v[q];
                            // every place at once: the one above's entry where that is beaten, else the new one or its own
#pragma unroll
                            for (int q = L - 1; q >= 0; --q) {
                                const bool here = !(x[0] <= lv[q]), above = q > 0 && !(x[0] <= lv[q > 0 ? q - 1 : 0]);
                                lv[q] = above ? lv[q > 0 ? q - 1 : 0] : here ? x[0] : lv[q];
                                li[q] = above ? li[q > 0 ? q - 1 : 0] : here ? v0 + j : li[q];
                            }
                        }
                        mx = max16(v);
                    }
                    fold(s, v, mx, c);
                };
                if (live) {
                    load(half * (kLmWords / 2), u[0]);
                    for (int c0 = half * (kLmWords / 2); c0 < c_end; c0 += 32) {
                        columns(c0, u[0], u[1]);
                        columns(c0 + 16, u[1], u[0]);
                    }
                }
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0)
                    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(in_first(saddr(&sh.tempty[buf])))
                                 : "memory");
            }
            if (row < p.N) {
                Part *o = p.part + (row * p.splits + split) * 2 + half;
                o->m = s.m;
                o->l = s.l;
                o->w = s.w;
                o->nan = nan;
#pragma unroll
                for (int j = 0; j < L; ++j) {
                    o->v[j] = lv[j] == lv[j] ? lv[j] : -INFINITY;
                    o->i[j] = li[j];
                }
            }
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    // neither CTA leaves while the other's products or arrivals may reach it,
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    // nor before every copy that either issued has landed (the first sees both CTAs' bytes)
    if (rank == 0 && tid == 0) {
        const uint32_t here = sh.issued;
        const PairEnd e = pair_end(here, of_second(saddr(&sh.issued)), stages);
        for (uint32_t i = e.only_from; i < e.to; ++i) {
            const uint32_t slot = i % stages, bar = saddr(&sh.full[slot]);
            if (i < here)
                asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(sh.others[slot]) : "memory");
            else
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
                             "r"(of_second(saddr(&sh.bytes[slot])))
                             : "memory");
        }
        for (uint32_t i = e.first; i < e.to; ++i)
            lm_drain(saddr(&sh.full[i % stages]), (i / stages) & 1);
    }
    __syncthreads();
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    if (warp == 1) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

constexpr int kJoinWarps = 4;

// A CTA per row: merges its ranges, computes the largest logits and the given
// token's again in fp32, adds them to the others' sums and writes the row. All of
// it is latency (a few KB a row), so the warps share the parts, and a warp's words
// are read side by side.
template <int L>
__global__ void __launch_bounds__(32 * kJoinWarps) k_lm_join(const uint16_t *emb, const uint16_t *h, const LmArgs p, const Outs o)
{
    constexpr int kMine = (L + 1 + kJoinWarps - 1) / kJoinWarps;      // words of a warp at most
    __shared__ float s_v[kJoinWarps][L], s_z[L + 1], s_last;
    __shared__ int32_t s_i[kJoinWarps][L], s_w[L + 1];
    __shared__ Sums s_sum[kJoinWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x;
    const float c = per_nat(o.T);
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int32_t tok = o.logp ? __ldcg(o.tokens + row) : -1;
    // a warp's share of the parts, in order
    const int parts = p.splits * 2, p0 = parts * warp / kJoinWarps, p1 = parts * (warp + 1) / kJoinWarps;
    const Part *part = p.part + row * parts;
    Sums s;
    int nan = 0;
    TopList top;
    join_parts(part + p0, p1 - p0, L, c, lane, s, nan, top);
    if (lane < L) {
        s_v[warp][lane] = top.v;
        s_i[warp][lane] = top.i;
    }
    nan = __syncthreads_or(nan);
    if (warp == 0) {
        merge_lists(s_v[lane & (kJoinWarps - 1)], s_i[lane & (kJoinWarps - 1)], lane < kJoinWarps ? L : 0, L, lane, top.v, top.i);
        if (lane < L)
            s_w[lane] = top.i;
        if (lane == L - 1)
            s_last = top.v;
        if (lane == 0)
            s_w[L] = tok >= 0 && tok < p.V ? tok : kNone;
    }
    __syncthreads();
    // listed logits that are not among the row's L best go to the others' sums
    Sums more;
    more.clear();
    const float last = s_last;
    const int32_t last_i = s_w[L - 1];
    constexpr int kAtOnce = 8;                 // loads on their way
    for (int e0 = threadIdx.x; e0 < parts * L; e0 += 32 * kJoinWarps * kAtOnce) {
        float v[kAtOnce];
        int32_t i[kAtOnce];
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) {
            const int e = e0 + q * 32 * kJoinWarps;
            const bool in = e < parts * L;
            v[q] = in ? __ldcg(part[e / L].v + e % L) : -INFINITY;
            i[q] = in ? __ldcg(part[e / L].i + e % L) : kNone;
        }
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q)
            if (v[q] > -INFINITY && better(last, last_i, v[q], i[q]))
                more.add(v[q], c);
    }
    s.add(warp_sums(more, c), c);
    if (lane == 0)
        s_sum[warp] = s;
    const uint4 *hr = reinterpret_cast<const uint4 *>(h + row * kH) + lane, *er[kMine];
    float acc[kMine][2];
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
        const int32_t w = warp + j * kJoinWarps <= L ? s_w[warp + j * kJoinWarps] : kNone;
        er[j] = reinterpret_cast<const uint4 *>(emb + static_cast<int64_t>(w == kNone ? 0 : w) * kH) + lane;
        acc[j][0] = acc[j][1] = 0.0f;
    }
#pragma unroll 3
    for (int i = 0; i < kH / 256; ++i) {
        const uint4 x = __ldcg(hr + i * 32);
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            const uint4 y = __ldg(er[j] + i * 32);
            const uint32_t ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 u = bf16x2_to_f32(xs[q]), v = bf16x2_to_f32(ys[q]);
                acc[j][0] = fmaf(u.x, v.x, acc[j][0]);
                acc[j][1] = fmaf(u.y, v.y, acc[j][1]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
        const float z = warp_sum(acc[j][0] + acc[j][1]);
        const int at = warp + j * kJoinWarps;
        if (lane == 0 && at <= L)
            s_z[at] = s_w[at] != kNone && z == z ? z : -INFINITY;
    }
    __syncthreads();
    if (warp)
        return;
    if (lane < kJoinWarps)
        s = s_sum[lane];
    else
        s.clear();
    s = warp_sums(s, c);
    // the L best enter the sums, which refer to the largest of all
    const float z1 = lane < L ? s_z[lane] : -INFINITY;
    s.rise(fmaxf(s.m, unordered(__reduce_max_sync(0xFFFFFFFFu, ordered(z1)))), c);
    const float d = fmaxf((z1 - s.m) * c, kClamp), e = ex2(d);
    s.l += warp_sum(e);
    s.w += warp_sum(e * d);
    TopList best;
    best.clear();
    best.offer(lane < L ? z1 : -INFINITY, lane < L ? top.i : kNone, L, lane);
    write_row(o, row, s, best, nan, s_z[L], lane);
}

}  // namespace score
}  // namespace fgm
