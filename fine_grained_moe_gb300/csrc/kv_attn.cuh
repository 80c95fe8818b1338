// Attention of M <= 8 new tokens per sequence over the 8-bit cache
// (fgm_attn_fwd).
//
//   s_t = scale k_s <q, kq_t>,  P = softmax(s),  out = sum_t P_t v_s vq_t
//
// Bytes bound it: a cached token costs 2 D bytes per kv head and feeds 4 R D
// operations for the R = M n_q_heads / n_kv_heads <= 64 rows that share the
// head, at most 128 per byte. So the kernel is built around the copies, and the
// cache's codes go to the tensor cores as they lie in shared memory:
//
//  * Work is a list of units, two 64-token blocks of one (sequence, kv head),
//    in that order. CTA c of G (one per SM) takes units [U c / G, U (c + 1) / G),
//    whatever sequences they belong to: ragged batches, one long sequence and
//    windows are balanced to a unit. (Each (sequence, head) counts 512 / D units
//    more, what starting and finishing it costs.) Lengths are read on the device,
//    so the launch does not depend on them and can be captured.
//  * Two warps stream K and V with TMA tensor copies (rows of 64 bytes in the
//    64-byte swizzle) into a ring each, which fill the shared memory. (One warp
//    for both let the next keys wait for a value stage: 67 us a pass at 256K
//    tokens and 40 rows, where the rings are 2 and 3 deep.)
//  * Two issuing warps run tcgen05.mma kind::f8f6f4 with the cache as the first
//    operand: S^T = K Q^T (128 tokens x rows, K = D) and O^T += V^T P^T (D x rows,
//    K = tokens; V lies token-contiguous in the cache for this). The rows are
//    the narrow side, so 128 lanes are full whatever R is, both accumulators
//    stay in tensor memory, and no cache byte passes through a register. (On
//    sm_103 an E4M3 mma.sync is carried out as conversions and f16 products,
//    about 15 instructions each: a kernel built on it, with the codes read from
//    the same rings, ran the 32K verify step in 75 us, issue-bound.)
//  * Sixteen softmax warps read S^T (a thread is a token and a fourth of the rows),
//    exponentiate and write P^T back to shared memory as the next operand. S
//    and P have two buffers: the products of the next unit run under the
//    softmax of this one, and its scores are read while this one's
//    probabilities are rounded.
//  * The values' warp also prepares the query terms of the next (sequence, head).
//
// Precision. The second operands are split into 8-bit terms in columns of their
// own, each the rounding of what the ones before left, and added in fp32.
// Queries: two E4M3 terms, hi + lo / 16, of the row scaled by a power of two to a
// largest element in (224, 448]; a bf16 has 8 significant bits and a term carries
// 4, so the split is exact down to half a subnormal step of lo, 2^-14 / 224 of the
// row's largest. Probabilities: three E5M2 terms, t0 + t1 / 8 + t2 / 64, of 2^12
// exp2(s + log2 v_s - m), at most 2^15. A term carries 3 bits, so they are within
// 2^-9 of themselves or, where the last is subnormal, 2^-17 / 64 / 2^12 = 2^-35 of
// exp2(m); the f16 on the way adds 2^-12 and 2^-37. The wide range is what E5M2 is
// taken for: the row sums use the unrounded exponentials, so a body of many small
// probabilities under one large one must not be dropped from the product (two E4M3
// terms held 2^-20 of exp2(m): a first token 15 nats above 32,768 others, its value
// zero, left nothing of the output). V's block scale rides in the exponent, so that
// blocks of any scale add into one accumulator. The row sums are fp32.
//
// The reference m is not the running maximum but within 3 of it from below: a
// unit whose scores stay under m + 3 (most after the first few) needs no
// maximum over its tokens, which are spread over the lanes, only a vote; one
// that exceeds it computes the maxima and rescales the accumulator.
//
// What bounds it, a pass being both kernels: HBM in the steady state up to R = 16,
// where a unit takes 0.35 us a CTA at D = 128 and twice that at D = 256 (5 tokens
// at 32K, 8 heads of 256: 134 MB in 32 us); the softmax warps' chain above (R = 48,
// 2 heads at 256K tokens: 268 MB in 65 us). That chain does not shrink with D as the
// copies do: 2 heads at 128K tokens take 20, 22, 28, 32 and 58 us at D = 64 with 8,
// 16, 32, 48 and 64 rows, 33, 34, 38, 40 and 69 at D = 256 (copies: 5 and 20 us).
// Around that 5 to 6 us to the first product (cold code, then lens, block table and
// the first copies one after the other) and 3 to 4 us of k_attn_join: the ragged
// batch of 9 (147 MB in 37 us) has several starts a CTA, 1,000 tokens are little
// else (10 us in a captured graph). The third probability term costs 40 rows at 256K
// 6 %, 64 rows 11 % (D = 256) to 30 % (D = 64) over two E4M3 terms, 16 rows 0 to 6.
//
// A segment (the part of one (sequence, kv head) in one CTA) that is a whole
// (sequence, head) is written out; one that spans CTAs leaves partial sums that
// k_attn_join adds up in CTA order. No atomics: the same call gives the same
// bits.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "kv_append.cuh"

namespace fgm {
namespace kv {

constexpr int kSoftWarps = 16;                         // four per lane quarter, a fourth of the rows each
constexpr int kAttnThreads = 32 * (4 + kSoftWarps);    // keys, scores, outputs, values and queries, softmax
constexpr int kTile = 2 * kBlock;                      // tokens of a unit
constexpr int kMaxRing = 8;                            // stages of the K and of the V ring at most
constexpr int kMetas = 64;                             // units' scales kept, in two halves
constexpr int kMaxGrid = 160;                          // CTAs at most: the SMs of a full sm_103 part
constexpr float kLowest = -3.0e38f;                    // stands for the maximum of nothing, below every finite score that counts
constexpr float kLift = 12.0f;                         // probabilities enter the product times 2^12
constexpr float kSlack = 3.0f;                         // scores may exceed the reference by this much
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr size_t kSmemMax = 227 * 1024;

struct AttnArgs {
    Cache c;
    const uint16_t *q;
    int64_t stride;          // elements between tokens of q
    int B, M, G, Hq;
    const int32_t *lens;
    const int32_t *table;
    int max_blocks;
    float scale;
    int window;
    uint16_t *out;
    float *lse;
    int32_t *status;
    float *part;             // [G][2] partial segments: O [rows][D], m [rows], l [rows]
    int4 *rec;               // {b, h, first CTA, last CTA} of each (sequence, head) that spans CTAs, b = -1: none; by
                             // (sequence, head) or, where those are more than the CTAs, by the CTA it starts in
    int n_rec;
    int rows;                // rows of the products: M * G rounded up to an instantiation
    int k_ring, v_ring;      // stages
    int q_ring;              // query buffers: 2, or 1 where they are large
    long long timeout_ns;
};

// Floats of one partial segment.
__host__ __device__ inline int64_t partial_floats(int rows, int D) { return static_cast<int64_t>(rows) * (D + 2); }

// Columns of the probabilities' product: three terms a row, a multiple of 16.
__host__ __device__ constexpr int prob_cols(int rows) { return (3 * rows + 15) / 16 * 16; }

// Shared memory of the operands that the kernel writes: query terms and two
// buffers of probability terms; and 64 D bytes a block of K or V.
__host__ __device__ inline int query_bytes(int rows, int D) { return 2 * rows * D; }
__host__ __device__ inline int prob_bytes(int rows) { return prob_cols(rows) * kTile; }

struct Meta {                // a unit: K's block scales, log2 and inverse of V's, first token, its blocks
    float ks[2], lv[2], iv[2];
    int tok0;
    int row[2];              // first 64-byte row of a block's K and V, -1: there is no such block
};

struct AttnShared {
    unsigned long long kfull[kMaxRing], kempty[kMaxRing], vfull[kMaxRing], vempty[kMaxRing];
    unsigned long long mfull[2];
    unsigned long long sfull[2], sfree[2], pfull[2], pdone[2], qfull[2], qempty[2], drained[2];
    Meta meta[kMetas];
    alignas(16) float qf[2][FGM_ATTN_MAX_ROWS];                    // score of a unit product: 2^e scale log2(e)
    float mx[4][FGM_ATTN_MAX_ROWS];                    // per lane quarter: a unit's maxima
    float4 ls[2][FGM_ATTN_MAX_ROWS];                   // the sums of a segment's rows per lane quarter
    float m[2][FGM_ATTN_MAX_ROWS];                     // and their references
    int2 lim[2][FGM_ATTN_MAX_ROWS];                       // tokens [x, y) that a row sees
    int orow[FGM_ATTN_MAX_ROWS];                       // a row's place among the (token, q head) of its sequence
    int units[2];                                      // the CTA's units: [first, last + 1)
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

__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// The same without the pause that try_wait may take: for a look at one of several things to do.
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Waits up to a tenth of a second for what is in flight after an abort.
__device__ __forceinline__ void bar_drain(uint32_t bar, uint32_t parity)
{
    const long long end = now_ns() + 100000000LL;
    while (!bar_try(bar, parity) && now_ns() < end)
        ;
}

__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Whether the CTA has given up, or this wait's limit is over (since: 0 before the
// first look, then when that was): then it gives up here, and the first to do so
// says where.
__device__ __forceinline__ bool gave_up(int *abort, long long &since, long long limit, int32_t *status, int site, int index)
{
    if (*reinterpret_cast<volatile int *>(abort))
        return true;
    if (since == 0)
        since = now_ns();
    if (now_ns() - since <= limit)
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

// Bounded wait on a barrier phase; false on timeout or abort.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, int *abort, long long limit, int32_t *status,
                                         int site, int index)
{
    long long since = 0;
    for (int it = 0;; ++it) {
        if (bar_try(bar, parity))
            return true;
        if ((it & 255) == 255 && gave_up(abort, since, limit, status, site, index))
            return false;
    }
}

__device__ __forceinline__ void bar_init(unsigned long long *b, int count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(b)), "r"(count) : "memory");
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The tokens that row i of a sequence of length len sees: [lo, hi).
__device__ __forceinline__ void row_range(int len, int M, int window, int i, int &lo, int &hi)
{
    const int pos = len - M + i;
    hi = max(pos + 1, 0);
    lo = window > 0 ? max(pos - window + 1, 0) : 0;
}

// Blocks [first, first + count) of a sequence that any row sees.
__device__ __forceinline__ int seq_blocks(int len, int M, int window, int &first)
{
    int lo, hi;
    row_range(len, M, window, 0, lo, hi);
    first = lo / kBlock;
    return (len + kBlock - 1) / kBlock - first;
}


// Descriptor of a K-major operand in the 64-byte swizzle: atoms of 8 rows x 64
// bytes, 512 bytes apart; descriptor version 1, layout type 4.
__device__ __forceinline__ uint64_t desc64(uint32_t addr)
{
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (1ull << 16) | (32ull << 32) | (1ull << 46) | (4ull << 61);
}

// Byte of element k (0..63) of row n in such a slice: 16-byte unit k / 16 of row
// n lies at unit (k / 16) ^ (n / 2 % 4).
__device__ __forceinline__ uint32_t at64(int n, int k)
{
    return static_cast<uint32_t>(n * 64 + ((((k >> 4) ^ (n >> 1)) & 3) << 4) + (k & 15));
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
        : "memory");
}

__device__ __forceinline__ void commit(unsigned long long *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(saddr(bar)) : "memory");
}

__device__ __forceinline__ void after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// N (2 or 4) accumulator columns of a thread's lane.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t a, float *v)
{
    uint32_t r[4];
    if constexpr (N == 2)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a) : "memory");
    else
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(a)
                     : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = __uint_as_float(r[i]);
}

template <int N>
__device__ __forceinline__ void tmem_st(uint32_t a, const float *v)
{
    if constexpr (N == 2)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(a), "r"(__float_as_uint(v[0])),
                     "r"(__float_as_uint(v[1]))
                     : "memory");
    else
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(__float_as_uint(v[0])),
                     "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3]))
                     : "memory");
}

// (the loaded registers pass through, so that no use of them moves ahead of the wait)
template <int N>
__device__ __forceinline__ void tmem_wait_ld(float (&v)[N])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i)
        asm volatile("" : "+f"(v[i]));
}

// (Evict-first in L2: a cache is read once a step, and what every launch needs
// again, its code above all, stays.)
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap *map, int row, uint32_t bar, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3}], [%4], "
        "%5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(bar), "l"(policy)
        : "memory");
}

// The E5M2 roundings of two f16, and 8 times what they leave: an E5M2 is the upper
// half of an f16, and the difference and its multiple have no more bits than x, so
// both are exact (below 2^15 the difference is at most 2^12).
__device__ __forceinline__ uint32_t e5m2_term(__half2 &x)
{
    const uint32_t t = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x), __NV_SATFINITE, __NV_E5M2);
    const uint32_t w = __byte_perm(t, 0u, 0x1404);
    x = __hmul2(__hsub2(x, *reinterpret_cast<const __half2 *>(&w)), __float2half2_rn(8.0f));
    return t;
}

__device__ __forceinline__ void sts32(uint32_t a, uint32_t v)
{
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

__device__ __forceinline__ void sts8(uint32_t a, uint32_t v)
{
    asm volatile("st.shared.u8 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// A place in the list of units.
struct Cursor {
    int b, h, u, n, first, blocks;    // sequence, kv head, unit of the segment, its units, first block and blocks
};

// Query terms of one (sequence, head), whose first row is at `q`, by `warps`
// warps, of which this is number w: rows w, w + warps, ...; `batch` rows' loads at
// a time. qs, qf, lims are shared-memory addresses.
template <int D, int R, int kBatch>
__device__ __forceinline__ void build_queries(const uint16_t *q, int64_t stride, int M, int G, int window, int len, float scale,
                                              int w, int warps, int lane, uint32_t qs, uint32_t qf, uint32_t lims)
{
    constexpr int kN = 2 * R, kE = (D + 127) / 128;
    const int rows = M * G;
#pragma unroll 1
    for (int r0 = w; r0 < R; r0 += warps * kBatch) {
        uint2 x[kBatch][kE];
        int at[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = r0 + i * warps;
            at[i] = r / G;
            const uint16_t *src = q + at[i] * stride + (r - at[i] * G) * D;
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                const int d = (e * 32 + lane) * 4;
                x[i][e] = make_uint2(0, 0);
                if (r < rows && d < D)
                    x[i][e] = __ldcg(reinterpret_cast<const uint2 *>(src + d));
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = r0 + i * warps;
            if (r >= R)
                break;
            unsigned amax = 0;
#pragma unroll
            for (int e = 0; e < kE; ++e)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const unsigned a = ((k < 2 ? x[i][e].x : x[i][e].y) >> (16 * (k & 1))) & 0x7FFFu;
                    amax = max(amax, a < 0x7F80u ? a : 0u);
                }
            amax = __reduce_max_sync(0xFFFFFFFFu, amax);
            // 2^ex with the largest element in (224, 448] 2^ex; no lower than 2^-120
            const unsigned u = amax << 16;
            const int ex = max(static_cast<int>(u >> 23) + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0) - 8, 7);
            const float up = __uint_as_float(static_cast<unsigned>(254 - ex) << 23);
            if (lane == 0) {
                int lo = 0, hi = 0;
                if (r < rows)
                    row_range(len, M, window, at[i], lo, hi);
                sts32(lims + r * 8, lo);
                sts32(lims + r * 8 + 4, hi);
                sts32(qf + r * 4, __float_as_uint(__uint_as_float(static_cast<unsigned>(ex) << 23) * (scale * kLog2e)));
            }
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                const int d = (e * 32 + lane) * 4;
                if (d >= D)
                    break;
                const float2 v0 = bf16x2_to_f32(x[i][e].x), v1 = bf16x2_to_f32(x[i][e].y);
                auto fin = [&](float v) { return fabsf(v) < INFINITY ? v * up : __int_as_float(0x7FC00000); };
                const float y[4] = {fin(v0.x), fin(v0.y), fin(v1.x), fin(v1.y)};
                const uint32_t hi = to_e4m3x4(y[0], y[1], y[2], y[3]);
                float z[4];
                e4m3x4_to_f32(hi, z);
                const uint32_t lo = to_e4m3x4(16.0f * (y[0] - z[0]), 16.0f * (y[1] - z[1]), 16.0f * (y[2] - z[2]),
                                              16.0f * (y[3] - z[3]));
                sts32(qs + (d >> 6) * (kN * 64) + at64(r, d & 63), hi);
                sts32(qs + (d >> 6) * (kN * 64) + at64(R + r, d & 63), lo);
            }
        }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// D: head dim; R: rows of the products (8, 16, 32, 48 or 64).
template <int D, int R>
__global__ void __launch_bounds__(kAttnThreads, 1)
    k_attn(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
           const __grid_constant__ AttnArgs p)
{
    constexpr int kSlices = D / 64, kN = 2 * R, kNP = prob_cols(R);
    constexpr int kSide = kTile * D;                             // bytes of a unit's K or V
    constexpr int kMTiles = D == 256 ? 2 : 1;                    // 128-lane tiles of O^T
    constexpr int kNR = R / 4;                                   // rows of a softmax thread
    constexpr bool kAhead = R <= 32;                             // the next unit's scores fit the registers beside this one's
    constexpr int kCh = kNR < 4 ? kNR : 4;                       // accumulator columns read at a time
    constexpr int kG = kNR == 8 ? 8 : kCh;                       // rows rescaled at a time
    constexpr uint32_t kIdesc = (1u << 4) | (8u << 24);          // fp32 += E4M3 x ..., M = 128
    constexpr uint32_t kIdescS = kIdesc | (static_cast<uint32_t>(kN >> 3) << 17);                  // ... E4M3
    constexpr uint32_t kIdescO = kIdesc | (1u << 10) | (static_cast<uint32_t>(kNP >> 3) << 17);    // ... E5M2
    // Buffers of S: two, but one where O leaves no room (64 rows at D = 256). The
    // softmax then still reads a unit's scores before it works on them, so the
    // next unit's product runs meanwhile.
    constexpr int kSBuf = 2 * kN + kMTiles * kNP <= 512 ? 2 : 1;
    constexpr uint32_t kOCol = kSBuf * kN;                       // S buffers first, then O tiles
    constexpr uint32_t kUsed = kOCol + kMTiles * kNP;
    static_assert(kUsed <= 512, "tensor memory has 512 columns");
    static_assert(kSBuf == 2 || !kAhead, "scores are read ahead from a second buffer");
    constexpr uint32_t kCols = kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
    extern __shared__ uint8_t dsm_raw[];
    __shared__ AttnShared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int heads = p.c.heads;
    uint8_t *dsm = dsm_raw + ((1024u - (saddr(dsm_raw) & 1023u)) & 1023u);
    uint8_t *qs = dsm, *ps = qs + p.q_ring * query_bytes(R, D), *kring = ps + 2 * prob_bytes(R);
    uint8_t *vring = kring + p.k_ring * kSide;
    // (for D = 64 the 128-row first operand of O^T runs 4 KB past a block's V: one more block's room behind the ring)
    int *cum = reinterpret_cast<int *>(vring + p.v_ring * kSide + (D == 64 ? kBlock * D : 0));   // [B + 1] units before each sequence
    int *lens = cum + p.B + 1;                                   // [B] clamped lengths
    int *used = lens + p.B;                                      // [B + 1] (sequence, head)s with units before each sequence
    constexpr int kCost = 512 / D;                               // a (sequence, head)'s start and end, in units

    if (tid == 0) {
        for (int i = 0; i < kMaxRing; ++i) {
            bar_init(&sh.kfull[i], 1);
            bar_init(&sh.kempty[i], 1);
            bar_init(&sh.vfull[i], 1);
            bar_init(&sh.vempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&sh.mfull[i], 1);
            bar_init(&sh.sfull[i], 1);
            bar_init(&sh.sfree[i], kSoftWarps);
            bar_init(&sh.pfull[i], kSoftWarps);
            bar_init(&sh.pdone[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&sh.qfull[i], 1);
            bar_init(&sh.qempty[i], 1 + kSoftWarps);
        }
        bar_init(&sh.drained[0], 1);
        bar_init(&sh.drained[1], 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // (behind the wait: a kernel before this one that lets it start early may not have taken its own tensor memory yet)
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&sh.tmem)), "r"(kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == 2)
        for (int r = lane; r < R; r += 32)
            sh.orow[r] = r / p.G * p.Hq + r % p.G;
    if (warp == 0) {
        int base = 0, ubase = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const int b = b0 + lane;
            int n = 0, first;
            if (b < p.B) {
                const int len = clamp_len(__ldcg(p.lens + b), p.max_blocks, p.status, blockIdx.x == 0);
                lens[b] = len;
                n = (seq_blocks(len, p.M, p.window, first) + 1) / 2 * heads;
            }
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                if (lane >= o)
                    inc += v;
            }
            const unsigned some = __ballot_sync(0xFFFFFFFFu, n > 0);
            if (b < p.B) {
                cum[b] = base + inc - n;
                used[b] = ubase + __popc(some & ((1u << lane) - 1)) * heads;
            }
            base += __shfl_sync(0xFFFFFFFFu, inc, 31);
            ubase += __popc(some) * heads;
        }
        if (lane == 0) {
            cum[p.B] = base;
            used[p.B] = ubase;
        }
        __syncwarp();
        // Places: units, and kCost places before those of each (sequence, head).
        // CTA c of G takes the units at places [P c / G, P (c + 1) / G): lanes 0 and
        // 1 count the units below either end.
        const int P = base + ubase * kCost, G = min(static_cast<int>(gridDim.x), max(P, 1)), c = blockIdx.x + lane;
        if (lane < 2) {
            const int place = P / G * c + P % G * c / G;      // floor(P c / G) in 32 bits
            int units = base;
            if (place < P && blockIdx.x < G) {
                int a = 0, z = p.B;
                while (z - a > 1) {
                    const int mid = (a + z) >> 1;
                    if (cum[mid] + used[mid] * kCost <= place)
                        a = mid;
                    else
                        z = mid;
                }
                const int n = (cum[a + 1] - cum[a]) / heads;
                const int r = place - cum[a] - used[a] * kCost, h = r / (n + kCost);
                units = cum[a] + h * n + max(r - h * (n + kCost) - kCost, 0);
            }
            sh.units[lane] = units;
        }
    }
    before_sync();
    __syncthreads();
    after_sync();
    asm volatile("griddepcontrol.launch_dependents;");
    const uint32_t tmem = sh.tmem;

    const int n_places = cum[p.B] + used[p.B] * kCost, G = min(static_cast<int>(gridDim.x), max(n_places, 1));
    const int u0 = sh.units[0], u1 = sh.units[1], n_units = u1 - u0;

    auto locate = [&](int u) -> Cursor {
        int a = 0, z = p.B;                        // cum[a] <= u < cum[z]: ends on a sequence that has units
        while (z - a > 1) {
            const int mid = (a + z) >> 1;
            if (cum[mid] <= u)
                a = mid;
            else
                z = mid;
        }
        Cursor at;
        at.b = a;
        at.blocks = seq_blocks(lens[a], p.M, p.window, at.first);
        at.n = (at.blocks + 1) / 2;
        const int r = u - cum[a];
        at.h = r / at.n;
        at.u = r % at.n;
        return at;
    };
    // The segment after this one.
    auto next = [&](Cursor c) -> Cursor {
        c.u = 0;
        if (++c.h < heads)
            return c;
        c.h = 0;
        do
            ++c.b;
        while (c.b < p.B - 1 && cum[c.b + 1] == cum[c.b]);
        if (c.b < p.B) {
            c.blocks = seq_blocks(lens[c.b], p.M, p.window, c.first);
            c.n = (c.blocks + 1) / 2;
        }
        return c;
    };
    Cursor cu = {};                                // where a warp is
    if (n_units > 0 && warp > 0)
        cu = locate(u0);
    auto sbuf = [](int u) { return kSBuf == 2 ? u & 1 : 0; };       // a unit's buffer of S, and its turn of it
    auto sturn = [](int u) { return kSBuf == 2 ? u >> 1 : u; };
    auto wait = [&](unsigned long long *bar, int phase, int site, int index) -> bool {
        return bar_wait(saddr(bar), phase & 1, &sh.abort, p.timeout_ns, p.status, site, index);
    };

    auto queries = [&](auto batch, const Cursor &cu, int w, int warps, int slot) {
        build_queries<D, R, decltype(batch)::value>(p.q + static_cast<int64_t>(cu.b) * p.M * p.stride + cu.h * p.G * D, p.stride,
                                                    p.M, p.G, p.window, lens[cu.b], p.scale, w, warps, lane,
                                                    saddr(qs + slot * query_bytes(R, D)), saddr(sh.qf[slot]),
                                                    saddr(sh.lim[slot]));
    };

    if (warp == 0) {
        // ------------------------------------------------------------ keys
        // Lane i looks up unit 32 k + i (block table and scales) a round ahead; the
        // round's scales are published together once its first copies are out.
        int row_n[2], tok_n = 0;                   // first 64-byte row of a block's K and V, -1: none
        float ks_n[2], vs_n[2];
        auto look = [&](int i) {
            row_n[0] = row_n[1] = -1;
            ks_n[0] = ks_n[1] = vs_n[0] = vs_n[1] = 1.0f;
            if (i >= n_units)
                return;
            const Cursor cu = locate(u0 + i);
            const int j = cu.first + 2 * cu.u;
            tok_n = j * kBlock;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (j + k >= cu.first + cu.blocks)
                    break;
                const int64_t ph = phys_block(p.table, cu.b, j + k, p.max_blocks, p.c.n_blocks);
                if (ph >= 0) {
                    const int at = static_cast<int>(ph) * heads + cu.h;
                    row_n[k] = at * D;
                    ks_n[k] = __ldcg(p.c.k_s + at);
                    vs_n[k] = __ldcg(p.c.v_s + at);
                } else {
                    atomicOr(p.status, FGM_STATUS_BAD_BLOCK);
                }
            }
        };
        if (lane == 0) {
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
        }
        uint64_t policy;
        asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
        bool ok = true;
        int issued = 0, slot = 0, turn = 0;
        look(lane);
        for (int r = 0; r < n_units && ok; r += 32) {
            const int r0 = row_n[0], r1 = row_n[1], m = min(32, n_units - r), tok0 = tok_n;
            const float ks0 = ks_n[0], ks1 = ks_n[1], vs0 = vs_n[0], vs1 = vs_n[1];
            if (r + 32 < n_units)
                look(r + 32 + lane);
            for (int i = 0; i < m && ok; ++i) {
                const int u = r + i;
                const int row[2] = {__shfl_sync(0xFFFFFFFFu, r0, i), __shfl_sync(0xFFFFFFFFu, r1, i)};
                if (lane == 0) {
                    const uint32_t bytes = ((row[0] >= 0) + (row[1] >= 0)) * (kBlock * D);
                    if (turn > 0)
                        ok = wait(&sh.kempty[slot], turn - 1, 13, u);
                    if (ok) {
                        const uint32_t bar = saddr(&sh.kfull[slot]), dst = saddr(kring) + slot * kSide;
                        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            if (row[k] >= 0)
#pragma unroll
                                for (int c = 0; c < kSlices; ++c)
                                    tma_rows(dst + c * (kTile * 64) + k * (kBlock * 64), &kmap, row[k] + c * kBlock, bar, policy);
                        issued = u + 1;
                    }
                }
                if (++slot == p.k_ring) {
                    slot = 0;
                    ++turn;
                }
                if (i == 0) {
                    // (The half's last round was read long ago: its units are 33 and more behind this one, the
                    // rings at most 8 deep and the softmax 3 units behind the scores.)
                    if (lane < m)
                        sh.meta[(r + lane) & (kMetas - 1)] =
                            Meta{{ks0, ks1}, {log2f(vs0), log2f(vs1)}, {1.0f / vs0, 1.0f / vs1}, tok0, {r0, r1}};
                    __syncwarp();
                    if (lane == 0)
                        bar_arrive(saddr(&sh.mfull[(r >> 5) & 1]));
                }
                ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            }
        }
        // every issued copy lands before the CTA may exit
        if (lane == 0)
            for (int u = max(0, issued - p.k_ring); u < issued; ++u)
                bar_drain(saddr(&sh.kfull[u % p.k_ring]), (u / p.k_ring) & 1);
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ scores
        // (The whole warp waits and one lane issues. Scores and outputs have an
        // issuing warp each: one thread gets a product of this size out every 50
        // to 120 cycles, two threads two.)
        const bool lead = elect_one();
        bool ok = true;
        int seg = 0, slot = 0, turn = 0;
        for (int done = 0; done < n_units && ok; ++seg) {
            const int qslot = seg % p.q_ring;
            const uint64_t b0 = desc64(saddr(qs + qslot * query_bytes(R, D)));
            const int n = min(cu.n - cu.u, n_units - done);
            ok = wait(&sh.qfull[qslot], seg / p.q_ring, 17, seg);
            for (int u = done; u < done + n && ok; ++u) {
                if (u >= kSBuf)
                    ok = wait(&sh.sfree[sbuf(u)], sturn(u) - 1, 15, u);
                ok = ok && wait(&sh.kfull[slot], turn, 16, u);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (ok && lead) {
                    after_sync();
                    const uint64_t a0 = desc64(saddr(kring + slot * kSide));
                    const uint32_t d = tmem + sbuf(u) * kN;
#pragma unroll
                    for (int k = 0; k < D / 32; ++k)
                        mma_f8(d, a0 + (((k >> 1) * (kTile * 64) + (k & 1) * 32) >> 4),
                               b0 + (((k >> 1) * (kN * 64) + (k & 1) * 32) >> 4), kIdescS, k != 0);
                    commit(&sh.kempty[slot]);
                    commit(&sh.sfull[sbuf(u)]);
                    if (u == done + n - 1)
                        commit(&sh.qempty[qslot]);
                }
                __syncwarp();
                if (++slot == p.k_ring) {
                    slot = 0;
                    ++turn;
                }
            }
            done += n;
            cu = next(cu);
        }
        // every issued product completes before the tensor memory is released
        if (lead) {
            commit(&sh.drained[0]);
            bar_drain(saddr(&sh.drained[0]), 0);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------------------ outputs
        const bool lead = elect_one();
        bool ok = true;
        int slot = 0, turn = 0;
        for (int done = 0; done < n_units && ok;) {
            const int n = min(cu.n - cu.u, n_units - done);
            bool add = false;
            for (int u = done; u < done + n && ok; ++u) {
                ok = wait(&sh.vfull[slot], turn, 18, u) && wait(&sh.pfull[u & 1], u >> 1, 19, u);
                ok = __all_sync(0xFFFFFFFFu, ok);
                const int *row = sh.meta[u & (kMetas - 1)].row;
                const int have = (row[0] >= 0) | (row[1] >= 0) << 1;
                if (ok && lead) {
                    after_sync();
                    const uint64_t a0 = desc64(saddr(vring + slot * kSide)), b0 = desc64(saddr(ps + (u & 1) * prob_bytes(R)));
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (have >> (k >> 1) & 1) {
#pragma unroll
                            for (int t = 0; t < kMTiles; ++t)
                                mma_f8(tmem + kOCol + t * kNP, a0 + (((k >> 1) * (kBlock * D) + t * (128 * 64) + (k & 1) * 32) >> 4),
                                       b0 + (((k >> 1) * (kNP * 64) + (k & 1) * 32) >> 4), kIdescO, add);
                            add = true;
                        }
                    commit(&sh.vempty[slot]);
                    commit(&sh.pdone[u & 1]);
                }
                __syncwarp();
                if (++slot == p.v_ring) {
                    slot = 0;
                    ++turn;
                }
            }
            done += n;
            cu = next(cu);
        }
        if (lead) {
            commit(&sh.drained[1]);
            bar_drain(saddr(&sh.drained[1]), 0);
        }
        __syncwarp();
    } else if (warp == 3) {
        // ------------------------------------------------------------ values, and queries of the second segment and on
        if (lane == 0)
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&vmap)) : "memory");
        uint64_t policy;
        asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
        int slot = 0, turn = 0, issued = 0;        // values: ring place and units out
        int seg = 0, done = 0;                     // queries: segments prepared and the units before the next one
        int spin = 0;
        long long since = 0;
        while (issued < n_units || done < n_units) {
            // whichever can be done now: the queries of a segment whose buffer is free, a unit's values whose stage is
            int can = 0;
            if (lane == 0) {
                if (done < n_units &&
                    (seg < p.q_ring || bar_test(saddr(&sh.qempty[seg % p.q_ring]), (seg / p.q_ring - 1) & 1)))
                    can = 1;
                if (issued < n_units && (issued % 32 != 0 || bar_test(saddr(&sh.mfull[(issued >> 5) & 1]), (issued >> 6) & 1)) &&
                    (turn == 0 || bar_test(saddr(&sh.vempty[slot]), (turn - 1) & 1)))
                    can |= 2;
                if (can != 0)
                    since = 0;
                else if ((++spin & 255) == 0 && gave_up(&sh.abort, since, p.timeout_ns, p.status, 14, issued))
                    can = 4;
            }
            can = __shfl_sync(0xFFFFFFFFu, can, 0);
            if (can & 4)
                break;
            if (can & 2) {
                if (lane == 0) {
                    const int *row = sh.meta[issued & (kMetas - 1)].row;
                    const int row0 = row[0], row1 = row[1];
                    const uint32_t bar = saddr(&sh.vfull[slot]), dst = saddr(vring) + slot * kSide;
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
                                 "r"(((row0 >= 0) + (row1 >= 0)) * (kBlock * D))
                                 : "memory");
                    if (row0 >= 0)
                        tma_rows(dst, &vmap, row0, bar, policy);
                    if (row1 >= 0)
                        tma_rows(dst + kBlock * D, &vmap, row1, bar, policy);
                }
                ++issued;
                if (++slot == p.v_ring) {
                    slot = 0;
                    ++turn;
                }
            }
            if (can & 1) {
                if (seg > 0) {                     // (the first segment's are the softmax warps' work)
                    queries(std::integral_constant<int, 8>{}, cu, 0, 1, seg % p.q_ring);      // (eight rows of loads in flight)
                    __syncwarp();
                    if (lane == 0)
                        bar_arrive(saddr(&sh.qfull[seg % p.q_ring]));
                }
                done += min(cu.n - cu.u, n_units - done);
                cu = next(cu);
                ++seg;
            }
        }
        if (lane == 0)
            for (int u = max(0, issued - p.v_ring); u < issued; ++u)
                bar_drain(saddr(&sh.vfull[u % p.v_ring]), (u / p.v_ring) & 1);
        __syncwarp();
    } else if (warp >= 4) {
        // ------------------------------------------------------------ softmax
        const int w = warp - 4, quarter = warp & 3, part4 = w >> 2, stid = tid - 128;
        const int tl = quarter * 32 + lane;        // token of a unit, lane of an accumulator
        const int blk = quarter >> 1;
        const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
        const int rows = p.M * p.G;
        const int n0 = part4 * kNR;                // the thread's rows: n0 .. n0 + kNR - 1
        // where the thread's token goes in P^T, and the swizzle of its rows 2 j, 2 j + 1
        const uint32_t probs = saddr(ps) + blk * (kNP * 64) + n0 * 64 + (tl & 15);
        uint32_t phase[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            phase[j] = ((((tl & 63) >> 4) ^ ((n0 >> 1) + j)) & 3) << 4;
        bool alive = true;
        int scales = -1;                           // the round whose scales are known to be there
        const bool by_head = p.B * heads <= p.n_rec;
        int4 rec = make_int4(-1, 0, 0, 0);

        // sequences without a token: zero rows
        for (int b = blockIdx.x; b < p.B; b += gridDim.x)
            if (cum[b + 1] == cum[b]) {
                const int64_t row0 = static_cast<int64_t>(b) * p.M * p.Hq;
                for (int i = stid; i < p.M * p.Hq * (D / 8); i += kSoftWarps * 32)
                    reinterpret_cast<uint4 *>(p.out + row0 * D)[i] = make_uint4(0, 0, 0, 0);
                if (p.lse)
                    for (int i = stid; i < p.M * p.Hq; i += kSoftWarps * 32)
                        p.lse[row0 + i] = -INFINITY;
                if (by_head)
                    for (int i = stid; i < heads; i += kSoftWarps * 32)
                        p.rec[b * heads + i] = rec;
            }

        int seg = 0;
        for (int done = 0; done < n_units; ++seg) {
            const int n = min(cu.n - cu.u, n_units - done);
            const int len = lens[cu.b], qslot = seg % p.q_ring;
            const float *qf = sh.qf[qslot] + n0;
            if (seg == 0) {
                queries(std::integral_constant<int, (R + kSoftWarps - 1) / kSoftWarps>{}, cu, w, kSoftWarps, 0);
                asm volatile("bar.sync 1, 512;" ::: "memory");
                if (stid == 0)
                    bar_arrive(saddr(&sh.qfull[0]));
            } else if (alive) {
                alive = wait(&sh.qfull[qslot], seg / p.q_ring, 27, seg);
            }

            float m[kNR], l[kNR];
#pragma unroll
            for (int r = 0; r < kNR; ++r) {
                m[r] = kLowest;
                l[r] = 0.0f;
            }
            int lo_min, hi_min, lo_max, hi_max;
            row_range(len, p.M, p.window, 0, lo_min, hi_min);
            row_range(len, p.M, p.window, p.M - 1, lo_max, hi_max);
            bool any_pv = false;                   // a product went into the accumulator

            float s[2 * kNR];                      // a unit's scores: hi, then lo
            auto arrived = [&](int u) {            // its scores and scales are there
                if (alive && (u >> 5) != scales) {
                    alive = wait(&sh.mfull[(u >> 5) & 1], u >> 6, 20, u);
                    scales = u >> 5;
                }
                if (alive)
                    alive = wait(&sh.sfull[sbuf(u)], sturn(u), 21, u);
                alive = __all_sync(0xFFFFFFFFu, alive);
                after_sync();
            };
            auto read = [&](int u, float *v) {
#pragma unroll
                for (int r = 0; r < kNR; r += kCh) {
                    tmem_ld<kCh>(tmem + lanes + sbuf(u) * kN + n0 + r, v + r);
                    tmem_ld<kCh>(tmem + lanes + sbuf(u) * kN + R + n0 + r, v + kNR + r);
                }
            };
            auto taken = [&](int u) {              // read: the buffer is free
                before_sync();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(saddr(&sh.sfree[sbuf(u)]));
            };
            arrived(done);
            read(done, s);
            tmem_wait_ld(s);
            taken(done);
            for (int i = 0; i < n; ++i) {
                const int u = done + i;
                const Meta me = sh.meta[u & (kMetas - 1)];
                const float ks = blk ? me.ks[1] : me.ks[0], lv = blk ? me.lv[1] : me.lv[0], ivs = blk ? me.iv[1] : me.iv[0];
                const int tok = me.tok0 + tl;
                const bool here = (blk ? me.row[1] : me.row[0]) >= 0, whole_unit = me.row[0] >= 0 && me.row[1] >= 0;
                const bool edge = me.tok0 + kTile > hi_min || me.tok0 < lo_max || !whole_unit;

                // scores in powers of two, with V's scale on top
                bool over = false;
                float f[kNR];
                if constexpr (kNR % 4 == 0) {
#pragma unroll
                    for (int r = 0; r < kNR; r += 4) {
                        const float4 x = *reinterpret_cast<const float4 *>(qf + r);
                        f[r] = x.x;
                        f[r + 1] = x.y;
                        f[r + 2] = x.z;
                        f[r + 3] = x.w;
                    }
                } else {
                    f[0] = qf[0];
                    f[1] = qf[1];
                }
#pragma unroll
                for (int r = 0; r < kNR; ++r)
                    s[r] = fmaf(fmaf(s[kNR + r], 0.0625f, s[r]), f[r] * ks, lv);
                if (edge) {
#pragma unroll
                    for (int r = 0; r < kNR; ++r) {
                        const int2 lim = sh.lim[qslot][n0 + r];
                        s[r] = here && tok >= lim.x && tok < lim.y ? s[r] : -INFINITY;
                    }
                }
#pragma unroll
                for (int r = 0; r < kNR; ++r)
                    over |= s[r] > m[r] + kSlack;
                int any;
                asm volatile(
                    "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 128, p;\n\t"
                    "selp.s32 %0, 1, 0, q;\n\t}"
                    : "=r"(any)
                    : "r"(static_cast<int>(over)), "r"(2 + part4)
                    : "memory");
                if (any) {
                    // the unit's maxima over its 128 tokens; new references; the accumulator follows
#pragma unroll
                    for (int r = 0; r < kNR; ++r) {
                        float x = s[r];
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1)
                            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
                        if (lane == 0)
                            sh.mx[quarter][n0 + r] = x;
                    }
                    asm volatile("barrier.cta.sync %0, 128;" ::"r"(2 + part4) : "memory");
                    float c[kNR];
#pragma unroll
                    for (int r = 0; r < kNR; ++r) {
                        float x = m[r];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            x = fmaxf(x, sh.mx[k][n0 + r]);
                        c[r] = ex2(m[r] - x);
                        l[r] *= c[r];
                        m[r] = x;
                    }
                    if (any_pv) {
                        if (alive)
                            alive = wait(&sh.pdone[(u - 1) & 1], (u - 1) >> 1, 22, u);
                        alive = __all_sync(0xFFFFFFFFu, alive);
                        after_sync();
#pragma unroll
                        for (int t = 0; t < kMTiles; ++t)
#pragma unroll
                            for (int r0 = 0; r0 < kNR; r0 += kG) {
                                const uint32_t a = tmem + lanes + kOCol + t * kNP + n0 + r0;
                                float o[3 * kG];
#pragma unroll
                                for (int r = 0; r < kG; r += kCh)
#pragma unroll
                                    for (int k = 0; k < 3; ++k)
                                        tmem_ld<kCh>(a + k * R + r, o + k * kG + r);
                                tmem_wait_ld(o);
#pragma unroll
                                for (int r = 0; r < kG; ++r)
#pragma unroll
                                    for (int k = 0; k < 3; ++k)
                                        o[k * kG + r] *= c[r0 + r];
#pragma unroll
                                for (int r = 0; r < kG; r += kCh)
#pragma unroll
                                    for (int k = 0; k < 3; ++k)
                                        tmem_st<kCh>(a + k * R + r, o + k * kG + r);
                            }
                        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                    }
                    // (sh.mx is written again only after every reader has passed the next vote)
                }
                any_pv |= me.row[0] >= 0 || me.row[1] >= 0;
                // the next unit's scores, if they are there, are read while this one's probabilities are made
                float next[kAhead ? 2 * kNR : 1];
                const bool more = i + 1 < n;
                const bool early = kAhead && more && (u + 1) >> 5 == scales &&
                                   __all_sync(0xFFFFFFFFu, bar_test(saddr(&sh.sfull[sbuf(u + 1)]), sturn(u + 1) & 1));
                // the buffer's last product is done
                if (alive && u >= 2)
                    alive = wait(&sh.pdone[u & 1], (u >> 1) - 1, 23, u);
                alive = __all_sync(0xFFFFFFFFu, alive);
                if constexpr (kAhead)
                    if (early) {
                        after_sync();
                        read(u + 1, next);
                    }
                const uint32_t pt = probs + (u & 1) * prob_bytes(R);
#pragma unroll
                for (int r = 0; r < kNR; r += 2) {
                    const float p0 = ex2(s[r] - (m[r] - kLift)), p1 = ex2(s[r + 1] - (m[r + 1] - kLift));
                    l[r] = fmaf(p0, ivs, l[r]);
                    l[r + 1] = fmaf(p1, ivs, l[r + 1]);
                    __half2 x = __floats2half2_rn(p0, p1);
                    // rows r, r + 1 (r even) lie in one swizzle phase; the next term R rows on
                    const uint32_t at = pt + phase[(r >> 1) & 3] + r * 64;
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        const uint32_t t = e5m2_term(x);
                        sts8(at + k * R * 64, t);
                        sts8(at + k * R * 64 + 64, t >> 8);
                    }
                }
                if (edge) {
                    // V codes of tokens that no row sees may be anything, NaN included: zeros
                    const int slot = u % p.v_ring;
                    if (alive)
                        alive = wait(&sh.vfull[slot], u / p.v_ring, 24, u);
                    alive = __all_sync(0xFFFFFFFFu, alive);
                    if (alive && here && (tok < lo_min || tok >= len)) {
                        uint8_t *vt = vring + slot * kSide + blk * (kBlock * D);
                        for (int d = part4 * (D / 4); d < (part4 + 1) * (D / 4); ++d)
                            vt[at64(d, tl & 63)] = 0;
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                if constexpr (kAhead)
                    if (early) {
                        tmem_wait_ld(next);
#pragma unroll
                        for (int r = 0; r < 2 * kNR; ++r)
                            s[r] = next[r];
                    }
                before_sync();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(saddr(&sh.pfull[u & 1]));
                    if (early)
                        bar_arrive(saddr(&sh.sfree[sbuf(u + 1)]));
                }
                if (more && !early) {
                    arrived(u + 1);
                    read(u + 1, s);
                    tmem_wait_ld(s);
                    taken(u + 1);
                }
            }

            // -------------------------------------------------------- end of the segment
            // (a second copy of the sums by segment parity, so that a warp may go on to the next segment's end
            // while another still reads these)
            float *ms = sh.m[seg & 1];
            float4 *ls = sh.ls[seg & 1];
#pragma unroll
            for (int r = 0; r < kNR; ++r) {
                const float x = warp_sum(l[r]);
                if (lane == 0)
                    reinterpret_cast<float *>(ls + n0 + r)[quarter] = x;
                if (quarter == 0 && lane == 0)
                    ms[n0 + r] = m[r];
            }
            asm volatile("bar.sync 1, 512;" ::: "memory");
            auto sum_of = [&](int r) -> float {
                const float4 x = ls[r];
                return (x.x + x.y) + (x.z + x.w);
            };
            const int last_u = done + n - 1;
            if (alive)
                alive = wait(&sh.pdone[last_u & 1], last_u >> 1, 25, last_u);
            alive = __all_sync(0xFFFFFFFFu, alive);
            after_sync();
            const bool starts = cu.u == 0, ends = cu.u + n == cu.n, whole = starts && ends;
            float *part = p.part + (blockIdx.x * 2 + (starts ? 1 : 0)) * partial_floats(R, D);
            // a thread is a dim and a share of the rows; D = 256: half of the warps per lane tile
            const int mt = D == 256 ? part4 >> 1 : 0, d = mt * 128 + tl;
            constexpr int kShare = D == 256 ? R / 2 : R / 4;
            const int ra = (D == 256 ? part4 & 1 : part4) * kShare;
            const uint32_t oa = tmem + lanes + kOCol + mt * kNP;
            const int64_t row0 = static_cast<int64_t>(cu.b) * p.M * p.Hq + cu.h * p.G;
            if (D != 64 || quarter < 2) {
#pragma unroll 2
                for (int r = ra; r < ra + kShare; r += kCh) {
                    float o[3 * kCh];
#pragma unroll
                    for (int k = 0; k < 3; ++k)
                        tmem_ld<kCh>(oa + k * R + r, o + k * kCh);
                    tmem_wait_ld(o);
#pragma unroll
                    for (int k = 0; k < kCh; ++k) {
                        const float sum = sum_of(r + k);
                        const float v = sum == 0.0f ? 0.0f : fmaf(fmaf(o[2 * kCh + k], 0.125f, o[kCh + k]), 0.125f, o[k]);
                        if (!whole)
                            part[(r + k) * D + d] = v;
                        else if (r + k < rows)
                            p.out[(row0 + sh.orow[r + k]) * D + d] = f32_to_bf16(sum == 0.0f ? 0.0f : __fdividef(v, sum));
                    }
                }
            }
            if (stid < R) {
                const float sum = sum_of(stid), mm = ms[stid];
                if (!whole) {
                    part[R * D + stid] = mm;
                    part[R * (D + 1) + stid] = sum;
                } else if (p.lse && stid < rows) {
                    p.lse[row0 + sh.orow[stid]] = sum == 0.0f ? -INFINITY : (mm - kLift + log2f(sum)) * kLn2;
                }
            }
            if (starts) {
                int4 mine = make_int4(-1, 0, 0, 0);
                if (!ends) {
                    // the CTA that holds the segment's last unit, at this place: the largest c with floor(P c / G) <= place
                    const int place = u0 + done - cu.u + cu.n - 1 + (used[cu.b] + cu.h + 1) * kCost;
                    mine = make_int4(cu.b, cu.h, blockIdx.x, static_cast<int>((static_cast<int64_t>(place + 1) * G - 1) / n_places));
                    rec = mine;
                }
                if (by_head && stid == 0)
                    p.rec[cu.b * heads + cu.h] = mine;
            }
            if (lane == 0)
                bar_arrive(saddr(&sh.qempty[qslot]));
            done += n;
            cu = next(cu);
        }
        if (stid == 0 && !by_head)
            p.rec[blockIdx.x] = rec;
    }
    before_sync();
    __syncthreads();
    if (warp == 1) {
        after_sync();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
    }
}

// Adds up the partial segments of one (sequence, kv head) that spans CTAs of the
// first kernel, in CTA order; CTA (record, row). A thread owns four output elements of every
// kLanes-th partial, and the lanes meet in shared memory, also in order.
template <int D>
__global__ void __launch_bounds__(256) k_attn_join(const AttnArgs p)
{
    constexpr int kCols = D / 4, kLanes = 256 / kCols;
    __shared__ float4 acc[kLanes][kCols];
    __shared__ float w[kMaxGrid], sm[8], sl[8];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 rec = __ldcg(p.rec + blockIdx.x);
    if (rec.x < 0)
        return;
    const int R = p.M * p.G, rows = p.rows, c0 = rec.z, n = rec.w - c0 + 1;
    const int64_t pf = partial_floats(p.rows, D);
    // partial i: the first CTA's second slot, then the others' first slots
    auto part = [&](int i) { return p.part + ((c0 + i) * 2 + (i == 0 ? 1 : 0)) * pf; };
    for (int r = blockIdx.y; r < R; r += gridDim.y) {
        float m = kLowest, l = 0.0f;
        if (tid < n) {
            m = __ldcg(part(tid) + rows * D + r);
            l = __ldcg(part(tid) + rows * (D + 1) + r);
        }
        float mx = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
        if (lane == 0)
            sm[warp] = mx;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i)
            mx = fmaxf(mx, sm[i]);
        const float wt = ex2(m - mx);
        if (tid < n)
            w[tid] = wt;
        l = warp_sum(tid < n ? l * wt : 0.0f);
        if (lane == 0)
            sl[warp] = l;
        __syncthreads();
        const int col = tid % kCols, k = tid / kCols;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
        for (int i = k; i < n; i += kLanes) {
            const float4 o = __ldcg(reinterpret_cast<const float4 *>(part(i) + r * D + col * 4));
            const float wi = w[i];
            v.x += wi * o.x;
            v.y += wi * o.y;
            v.z += wi * o.z;
            v.w += wi * o.w;
        }
        acc[k][col] = v;
        __syncthreads();
        if (k == 0) {
            l = 0.0f;
            v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                l += sl[i];
#pragma unroll
            for (int i = 0; i < kLanes; ++i) {
                const float4 o = acc[i][col];
                v.x += o.x;
                v.y += o.y;
                v.z += o.z;
                v.w += o.w;
            }
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const int64_t row = (static_cast<int64_t>(rec.x) * p.M + r / p.G) * p.Hq + rec.y * p.G + r % p.G;
            uint2 o;
            o.x = f32_to_bf16(v.x * inv) | (static_cast<uint32_t>(f32_to_bf16(v.y * inv)) << 16);
            o.y = f32_to_bf16(v.z * inv) | (static_cast<uint32_t>(f32_to_bf16(v.w * inv)) << 16);
            *reinterpret_cast<uint2 *>(p.out + row * D + col * 4) = o;
            if (col == 0 && p.lse)
                p.lse[row] = l == 0.0f ? -INFINITY : (mx - kLift + log2f(l)) * kLn2;
        }
        __syncthreads();
    }
}

}  // namespace kv
}  // namespace fgm
