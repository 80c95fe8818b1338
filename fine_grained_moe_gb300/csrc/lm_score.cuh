// Log probabilities from hidden rows (fgm_lm_head_logprobs): the tied lm_head
//   z[n][v] = sum_j h[n][j] emb[v][j]
// with the sums of logprobs.cuh in its epilogue, so that logits are never stored.
//
// 2 * 2816 operations a logit: bound by the tensor pipe from about 300 rows on,
// by the embedding's 1.48 GB below. Built for the first: a pair of CTAs
// (cta_group::2) holds 256 rows x 256 words in tensor memory, each CTA loading
// its 128 rows and half of the words, 64 bytes per cycle and SM at the full rate
// where one CTA on 128 x 256 would need 96.
//  * TMA copies boxes of 128 rows x 128 bytes (64 elements of K) in the 128-byte
//    swizzle into a 6-stage ring, the second CTA's bytes counted on the first's
//    barriers; rows past N and words past V arrive as zeros.
//  * The first CTA's issuing warp runs M = 256, N = 256, K = 16 products into one
//    of two accumulators (2 x 256 columns), so that the next tile's products run
//    under this tile's epilogue.
//  * Four epilogue warps per CTA own a row a thread: 32 columns at a time they
//    go into the running (m, l, w), and those that beat the row's k-th best into
//    its list in shared memory (unsorted; the worst entry is replaced). A row
//    meets about k (1 + ln(n / k)) such logits among n.
//  * An item is 256 rows x a range of words; a pair takes items in turn, a row's
//    state stays in registers over the range, and k_logprob_join merges the
//    ranges.
// Pairs whose items are the same words and other rows run at the same time, so
// the embedding comes from HBM once and from L2 for the others.
#pragma once

#include <cuda.h>

#include "logprobs.cuh"

namespace fgm {
namespace score {

constexpr int kLmThreads = 256;                  // copies, products, -, -, four epilogue warps
constexpr int kLmStages = 6;
constexpr int kLmBox = 128 * 128;                // 128 rows x 128 bytes
constexpr int kLmStage = 2 * kLmBox;             // rows and words
constexpr int kLmWords = 256;                    // words of a tile
constexpr int kLmRows = 256;                     // rows of a pair
constexpr int kLmK = kH / 64;                    // stages of a tile
constexpr int kLmListBytes = kMaxTop * 128 * 8;  // [k][128 rows] values, then indices
constexpr int kLmSmem = kLmStages * kLmStage + kLmListBytes + 1024;
static_assert(kH % 64 == 0, "K must split into whole stages");

struct LmArgs {
    int64_t N;
    int V;
    const int32_t *tokens;   // or NULL
    float T;
    int k;
    int splits;              // word ranges
    int64_t items;           // row tiles * splits
    Part *part;              // [N][splits]
    float *ztok;             // [N] the given token's logit
    int32_t *status;
    long long timeout_ns;
};

struct LmShared {
    unsigned long long full[kLmStages], empty[kLmStages], tfull[2], tempty[2], drained;
    uint32_t tmem;
    int abort;
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

__device__ __forceinline__ void lm_copy(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

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
    const uint32_t ring = saddr(dsm);
    float *lv = reinterpret_cast<float *>(dsm + kLmStages * kLmStage);
    int32_t *li = reinterpret_cast<int32_t *>(lv + kMaxTop * 128);
    const long long deadline = now_ns() + p.timeout_ns;
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
            init(&sh.tempty[i], 8);              // the epilogue warps of both CTAs
        }
        init(&sh.drained, 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
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
        for (int it = 0;; ++it) {
            if (lm_try(a, phase & 1))
                return true;
            if ((it & 255) == 255) {
                if (*reinterpret_cast<volatile int *>(&sh.abort))
                    return false;
                if (now_ns() > deadline) {
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
            bool ok = true;
            uint32_t n = 0;
            for (int64_t item = pair; item < p.items && ok; item += pairs) {
                int t0, t1;
                range(item, t0, t1);
                const int y = static_cast<int>(item / p.splits) * kLmRows + rank * 128;
                for (int t = t0; t < t1 && ok; ++t)
                    for (int ks = 0; ks < kLmK; ++ks, ++n) {
                        const int slot = n % kLmStages;
                        if (n >= kLmStages && !(ok = wait(&sh.empty[slot], n / kLmStages - 1, 30, ks)))
                            break;
                        const uint32_t bar = in_first(saddr(&sh.full[slot])), dst = ring + slot * kLmStage;
                        if (rank == 0)
                            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(&sh.full[slot])),
                                         "r"(2 * kLmStage)
                                         : "memory");
                        lm_copy(dst, &hmap, ks * 64, y, bar);
                        lm_copy(dst + kLmBox, &emap, ks * 64, t * kLmWords + rank * 128, bar);
                    }
            }
            // every issued copy lands before the pair may exit (the first CTA sees both CTAs' bytes)
            if (rank == 0)
                for (uint32_t i = n > kLmStages ? n - kLmStages : 0; i < n; ++i)
                    lm_drain(saddr(&sh.full[i % kLmStages]), (i / kLmStages) & 1);
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
                        const int slot = n % kLmStages;
                        ok = ok && wait(&sh.full[slot], n / kLmStages, 32, ks);
                        ok = __all_sync(0xFFFFFFFFu, ok);
                        if (!ok)
                            break;
                        if (lead) {
                            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                            const uint64_t a = lm_desc(ring + slot * kLmStage), b = lm_desc(ring + slot * kLmStage + kLmBox);
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                asm volatile(
                                    "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                                    "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem + buf * kLmWords),
                                    "l"(a + kk * 2), "l"(b + kk * 2), "r"(kIdesc), "r"(static_cast<uint32_t>((ks | kk) != 0))
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
        // ------------------------------------------------------------ epilogue: a thread is a row
        const int quarter = warp & 3, r = quarter * 32 + lane, k = p.k;
        const float c = kLog2e / p.T;
        bool alive = true;
        uint32_t tile = 0;
        for (int64_t item = pair; item < p.items; item += pairs) {
            int t0, t1;
            range(item, t0, t1);
            const int64_t row = item / p.splits * kLmRows + rank * 128 + r;
            const int split = static_cast<int>(item % p.splits);
            const int tok = p.tokens && row < p.N ? __ldg(p.tokens + row) : -1;
            Sums s;
            s.clear();
            int nan = 0, worst = 0;              // the list's worst entry: its place, value and index
            float wv = -INFINITY;
            int32_t wi = kNone;
            for (int j = 0; j < k; ++j) {
                lv[j * 128 + r] = -INFINITY;
                li[j * 128 + r] = kNone;
            }
            float zt = -INFINITY;
            for (int t = t0; t < t1; ++t, ++tile) {
                const uint32_t buf = tile & 1;
                if (alive)
                    alive = wait(&sh.tfull[buf], tile >> 1, 33, t);
                alive = __all_sync(0xFFFFFFFFu, alive);
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                for (int c0 = 0; c0 < kLmWords; c0 += 16) {
                    uint32_t u[16];
                    asm volatile(
                        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                        "%14, %15}, [%16];"
                        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
                          "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
                        : "r"(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + buf * kLmWords + c0)
                        : "memory");
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                    float v[kVals];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        asm volatile("" : "+r"(u[j]));
                        v[j] = __uint_as_float(u[j]);
                    }
                    const int v0 = t * kLmWords + c0;
                    if (v0 + 16 > p.V)
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            v[j] = v0 + j < p.V ? v[j] : -INFINITY;
                    if (tok >= v0 && tok < v0 + 16)
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            zt = tok == v0 + j ? v[j] : zt;
                    fold(s, v, c, nan);
                    if (k == 0)
                        continue;
                    float mx = v[0];
#pragma unroll
                    for (int j = 1; j < 16; ++j)
                        mx = fmaxf(mx, v[j]);
                    if (mx > wv || wi == kNone) {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (better(v[j], v0 + j, wv, wi) && v0 + j < p.V) {
                                lv[worst * 128 + r] = v[j];
                                li[worst * 128 + r] = v0 + j;
                                wv = INFINITY;
                                wi = -1;
                                for (int q = 0; q < k; ++q) {
                                    const float qv = lv[q * 128 + r];
                                    const int32_t qi = li[q * 128 + r];
                                    if (better(wv, wi, qv, qi)) {
                                        wv = qv;
                                        wi = qi;
                                        worst = q;
                                    }
                                }
                            }
                    }
                }
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0)
                    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(in_first(saddr(&sh.tempty[buf])))
                                 : "memory");
            }
            if (row < p.N) {
                Part *o = p.part + row * p.splits + split;
                o->m = s.m;
                o->l = s.l;
                o->w = s.w;
                o->nan = nan;
                for (int j = 0; j < k; ++j) {    // the list in order
                    float bv = -INFINITY;
                    int32_t bi = kNone;
                    int at = 0;
                    for (int q = 0; q < k; ++q) {
                        const float qv = lv[q * 128 + r];
                        const int32_t qi = li[q * 128 + r];
                        if (qi >= 0 && better(qv, qi, bv, bi)) {
                            bv = qv;
                            bi = qi;
                            at = q;
                        }
                    }
                    o->v[j] = bv;
                    o->i[j] = bi;
                    li[at * 128 + r] = -1;       // taken
                }
                if (tok >= 0 && tok < p.V ? tok / kLmWords >= t0 && tok / kLmWords < t1 : split == 0)
                    p.ztok[row] = zt;
            }
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    // neither CTA leaves while the other's copies, products or arrivals may reach it
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    if (warp == 1) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

}  // namespace score
}  // namespace fgm
