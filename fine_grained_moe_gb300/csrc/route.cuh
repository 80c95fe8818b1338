// Routing of any number of tokens (fgm_moe_route): logits l = W x + b of 128 experts,
// the 8 largest (ties to the lower index) and their softmax.
//
// 2 * 128 * 2816 operations and 5.6 KB a token: bound by HBM at long prompts, by
// latency at a few tokens, so K is split over CTAs while there are fewer tiles of
// 128 tokens than SMs. k_router_logits_tc runs M = 128 tokens x N = 128 experts on
// tcgen05 and takes the accumulator out every 256 elements of K, to add it in fp32
// registers: the tensor pipe truncates each addition, to 2^-22 of what it has added, and 16
// of them a chunk are within 2^-18 |x| |w| in all. The 11 chunks' additions in fp32 (and
// splits') are within 2^-24 of their sum each, 0.18 of 2^-18: kLogitError covers both, and what
// |x| itself is off by. 16,381 tokens: 26 us, 3.6 TB/s of x, and 16 for k_route_top; 5 tokens 3
// and 4 in a captured graph.
//
// Precision. Which experts a token takes is a whole number that hangs on logits that
// may lie next to each other, so it goes by the exact ones. k_route_top knows a bound
// d on the error of its logits (from |x| and the largest |w|, which the products'
// helper warps sum up from the tiles in shared memory). Chosen experts further than
// 2 d from every other candidate are in order; the others' logits are summed again
// without rounding error to speak of (each addition's error is kept, 2^-40 of the sum
// remains), and the 8 chosen by these. About one token in twenty has such a pair.
//
// The bound holds over bf16's range, whose squares fp32 does not hold: a row whose sum of
// squares is outside [kLow, kHigh] is read again and its norm taken under a power of two, which
// enters the exact sums, too. Experts' rows that are not finite have no finite logits and stay
// out of |w|; with one as large as 2^60 every two finite logits are near.
#pragma once

#include "tensor.cuh"

namespace fgm {
namespace route {

constexpr int kThreads = 576;                    // copies, products, eight epilogue warps; four for the tokens' norms, and
                                                 // four for the experts' in the first tile's CTAs
constexpr int kStages = 6;
constexpr int kBox = 128 * 128;                  // 128 rows x 64 elements
constexpr int kChunkBoxes = 4;                   // 256 elements of K between readings of the accumulator
constexpr int kChunks = kH / 256;
constexpr int kSmem = kStages * 2 * kBox + 1024;
constexpr float kLogitError = 0x1.4p-18f;        // of |x| |w|
// Sums of squares that are taken as they are: between rows of such norms no sum of products overflows, and what products
// below fp32's normal numbers lose is less than 2^-48 of |x| |w|.
constexpr float kLow = 0x1p-90f, kHigh = 0x1p100f;
constexpr float kHuge = 0x1p120f;                // stands for squares above it
static_assert(kH % 256 == 0 && kE == 128 && kK == 8, "the tiles are cut for these");

struct LogitArgs {
    int64_t T;
    int splits;              // of K
    float *part;             // [splits][T][128]
    float *xn2;              // [splits][T] sums of squares
    float *wn2;              // [splits][4] the largest of each 32 experts whose rows are finite
    const uint16_t *w;       // [128][2816]
    int32_t *count;          // the grouping's counts, made 0 for k_route_top
    int counts;
    int32_t *status;
    long long timeout_ns;
};

struct Shared {
    unsigned long long full[kStages], empty[kStages], tfull[2], tempty[2], drained;
    uint32_t tmem;
    int abort;
    uint32_t issued;
};

__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap *map, int k, int row, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(k), "r"(row), "r"(bar)
        : "memory");
}

// Sum of squares of a row of 64 bf16 at `at`, whatever their order.
__device__ __forceinline__ float squares(uint32_t at, int first, float s)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t w[4];
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(at + ((first + i) & 7) * 16)
                     : "memory");
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 f = bf16x2_to_f32(w[q]);
            s = fmaf(f.x, f.x, s);
            s = fmaf(f.y, f.y, s);
        }
    }
    return s;
}

// The largest of eight bf16's bits without their signs.
__device__ __forceinline__ uint32_t largest(const uint4 &v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        m = max(m, max(w[q] & 0x7FFFu, w[q] >> 16 & 0x7FFFu));
    return m;
}

__global__ void __launch_bounds__(kThreads, 1)
    k_router_logits_tc(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap, const LogitArgs p)
{
    extern __shared__ uint8_t dsm_raw[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t ring = (tc::saddr(dsm_raw) + 1023u) & ~1023u;
    const int64_t tile = blockIdx.x;
    const int split = blockIdx.y, b0 = kChunks * split / p.splits * kChunkBoxes, b1 = kChunks * (split + 1) / p.splits * kChunkBoxes;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            tc::bar_init(&sh.full[i], 1);
            tc::bar_init(&sh.empty[i], tile == 0 ? 9 : 5);   // the products and the norm warps
        }
        for (int i = 0; i < 2; ++i) {
            tc::bar_init(&sh.tfull[i], 1);
            tc::bar_init(&sh.tempty[i], 8);
        }
        tc::bar_init(&sh.drained, 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc::after_previous();
    if (warp == 1)
        tc::memory_take<1>(&sh.tmem);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    tc::let_next_start();
    for (int i = (blockIdx.y * gridDim.x + blockIdx.x) * kThreads + tid; i < p.counts; i += gridDim.x * gridDim.y * kThreads)
        p.count[i] = 0;
    const uint32_t tmem = sh.tmem;
    const tc::Waiter wait{&sh.abort, p.status, p.timeout_ns};

    if (warp == 0) {
        if (lane == 0) {
            uint32_t n = 0;
            for (int b = b0; b < b1; ++b, ++n) {
                const uint32_t slot = n % kStages, bar = tc::saddr(&sh.full[slot]), dst = ring + slot * 2 * kBox;
                if (n >= kStages && !wait(&sh.empty[slot], n / kStages - 1, 38, b))
                    break;
                tc::bar_expect(bar, 2 * kBox);
                copy_box(dst, &xmap, b * 64, static_cast<int>(tile * 128), bar);
                copy_box(dst + kBox, &wmap, b * 64, 0, bar);
            }
            sh.issued = n;
        }
        __syncwarp();
    } else if (warp == 1) {
        const bool lead = tc::elect();
        bool ok = true;
        uint32_t n = 0;
        for (int b = b0; b < b1 && ok; ++b, ++n) {
            const uint32_t slot = n % kStages, chunk = n / kChunkBoxes, buf = chunk & 1;
            if (chunk >= 2 && n % kChunkBoxes == 0)
                ok = wait(&sh.tempty[buf], (chunk >> 1) - 1, 39, b);
            ok = ok && wait(&sh.full[slot], n / kStages, 40, b);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (ok && lead) {
                tc::fence_after();
                const uint64_t x = tc::operand(ring + slot * 2 * kBox), w = tc::operand(ring + slot * 2 * kBox + kBox);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    tc::product<1, false>(tmem + buf * 128, x + j * 2, w + j * 2, tc::product_desc(128, 128, false),
                                          n % kChunkBoxes != 0 || j != 0);
                tc::commit<1>(&sh.empty[slot]);
                if (n % kChunkBoxes == kChunkBoxes - 1)
                    tc::commit<1>(&sh.tfull[buf]);
            }
            __syncwarp();
        }
        if (lead) {
            tc::commit<1>(&sh.drained);
            tc::bar_drain(tc::saddr(&sh.drained), 0);
        }
        __syncwarp();
    } else if (warp < 4 || warp >= 12) {
        // norms: a thread a row
        const int norm = warp < 4 ? warp - 2 : warp - 10, r = (norm & 3) * 32 + lane;
        const bool experts = norm >= 4;
        float sum = 0.0f;
        bool ok = !experts || tile == 0;
        uint32_t n = 0;
        for (int b = b0; b < b1 && ok; ++b, ++n) {
            const uint32_t slot = n % kStages;
            ok = wait(&sh.full[slot], n / kStages, 41, b);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok)
                break;
            sum = squares(ring + slot * 2 * kBox + (experts ? kBox : 0) + r * 128, r, sum);
            __syncwarp();
            if (lane == 0)
                tc::bar_arrive(tc::saddr(&sh.empty[slot]));
        }
        if (experts && ok) {
            // Rows whose squares fp32 does not hold, by the warp: zeros, not finite themselves, or beyond its range at either end.
            for (uint32_t odd = __ballot_sync(0xFFFFFFFFu, !(sum > 0.0f && sum < INFINITY)); odd; odd &= odd - 1) {
                const int row = __ffs(odd) - 1;
                const uint16_t *w = p.w + static_cast<int64_t>((norm & 3) * 32 + row) * kH;
                uint32_t m = 0;
                for (int k = b0 * 64 + lane * 8; k < b1 * 64; k += 256)
                    m = max(m, largest(__ldcg(reinterpret_cast<const uint4 *>(w + k))));
                m = __reduce_max_sync(0xFFFFFFFFu, m);
                if (lane == row)
                    sum = m == 0 || m >= 0x7F80u ? 0.0f : sum == 0.0f ? 0x1p-149f : kHuge;
            }
        }
        if (experts) {
            const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(sum));
            if (tile == 0 && lane == 0)
                p.wn2[split * 4 + (norm & 3)] = __uint_as_float(most);
        } else if (tile * 128 + r < p.T) {
            p.xn2[split * p.T + tile * 128 + r] = sum;
        }
    } else {
        const int quarter = warp & 3, side = (warp - 4) >> 2;
        float acc[64];
#pragma unroll
        for (int j = 0; j < 64; ++j)
            acc[j] = 0.0f;
        bool ok = true;
        for (int chunk = 0; chunk < (b1 - b0) / kChunkBoxes; ++chunk) {
            const uint32_t buf = chunk & 1;
            if (ok)
                ok = wait(&sh.tfull[buf], chunk >> 1, 42, chunk);
            ok = __all_sync(0xFFFFFFFFu, ok);
            tc::fence_after();
            if (ok)
#pragma unroll
                for (int j = 0; j < 64; j += 8) {
                    uint32_t u[8];
                    tc::read(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + buf * 128 + side * 64 + j, u);
                    tc::read_wait();
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        asm volatile("" : "+r"(u[q]));
                        acc[j + q] += __uint_as_float(u[q]);
                    }
                }
            tc::fence_before();
            __syncwarp();
            if (lane == 0)
                tc::bar_arrive(tc::saddr(&sh.tempty[buf]));
        }
        const int64_t t = tile * 128 + quarter * 32 + lane;
        if (t < p.T) {
            float4 *to = reinterpret_cast<float4 *>(p.part + (split * p.T + t) * kE + side * 64);
#pragma unroll
            for (int j = 0; j < 16; ++j)
                to[j] = make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
        }
    }
    tc::fence_before();
    __syncthreads();
    if (tid == 0) {                              // every issued copy lands before the CTA ends
        const uint32_t n = sh.issued;
        for (uint32_t i = n > kStages ? n - kStages : 0; i < n; ++i)
            tc::bar_drain(tc::saddr(&sh.full[i % kStages]), (i / kStages) & 1);
    }
    __syncthreads();
    if (warp == 1) {
        tc::fence_after();
        tc::memory_free<1>(tmem);
    }
}

struct TopArgs {
    const float *part, *xn2, *wn2;
    const float *b;          // [128] or NULL
    const uint16_t *x;
    int64_t stride;
    const uint16_t *w;       // [128][2816]
    int64_t T;
    int splits;
    int32_t *ids;            // [T][8]
    float *wts;              // [T][8]
    int32_t *count;          // [chunks][128] choices of each expert by a chunk's tokens, or NULL
    unsigned chunk;          // tokens of a chunk
    int32_t *status;
};

constexpr int kTopWarps = 4;                    // tokens of a CTA, and the parts of K that its warps take of a near expert's logit
constexpr int kUnits = kH / 256;                 // of 256 elements, eight a lane
static_assert(kH % 256 == 0, "whole units");

// (s, c) += v, s the rounded sum and c the sum of the roundings' errors.
__device__ __forceinline__ void sum_exactly(float &s, float &c, float v)
{
    const float t = __fadd_rn(s, v), z = __fsub_rn(t, s);
    c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(v, z)));
    s = t;
}

// A power of two s that brings a row of x's largest element (its bits) to 1, and its inverse.
__device__ __forceinline__ float row_power(uint32_t m, float &inverse)
{
    const int e = static_cast<int>(m >> 7), up = e > 253 ? 1 : e < 1 ? 253 : 254 - e;
    inverse = __int_as_float((254 - up) << 23);
    return __int_as_float(up << 23);
}

// |x| by a warp: the square root of a sum of squares under the row's power of two. 0: x is 0 or not finite.
__device__ __noinline__ float row_norm(const uint16_t *x, int lane, float &power, float &inverse)
{
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
        m = max(m, largest(__ldcg(reinterpret_cast<const uint4 *>(x) + u * 32 + lane)));
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    power = inverse = 1.0f;
    if (m == 0 || m >= 0x7F80u)
        return 0.0f;
    power = row_power(m, inverse);
    float s = 0.0f;
#pragma unroll 1
    for (int u = 0; u < kUnits; ++u) {
        const uint4 v = __ldcg(reinterpret_cast<const uint4 *>(x) + u * 32 + lane);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 f = bf16x2_to_f32(w[q]);
            s = fmaf(f.x * power, f.x * power, s);
            s = fmaf(f.y * power, f.y * power, s);
        }
    }
    return sqrtf(warp_sum(s));
}

// A warp's part of x . w of two experts, x times a power of two: two sums a lane of each. (Three units' loads on their way at
// once, and a loop: its instructions are seldom in a cache.)
template <bool SCALED>
__device__ __forceinline__ void exact_parts(const uint16_t *x, const uint16_t *w0, const uint16_t *w1, float power, int part, int lane, double &d0,
                                            double &d1)
{
    float s[2][2], c[2][2];
#pragma unroll
    for (int q = 0; q < 2; ++q)
        s[0][q] = s[1][q] = c[0][q] = c[1][q] = 0.0f;
    constexpr int kMine = 3;
#pragma unroll 1
    for (int first = part; first < kUnits; first += kMine * kTopWarps) {
        uint4 a[kMine], b[2][kMine];
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int u = first + i * kTopWarps;
            a[i] = u < kUnits ? __ldcg(reinterpret_cast<const uint4 *>(x) + u * 32 + lane) : make_uint4(0, 0, 0, 0);
            b[0][i] = u < kUnits ? __ldcg(reinterpret_cast<const uint4 *>(w0) + u * 32 + lane) : make_uint4(0, 0, 0, 0);
            b[1][i] = u < kUnits ? __ldcg(reinterpret_cast<const uint4 *>(w1) + u * 32 + lane) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const uint32_t as[4] = {a[i].x, a[i].y, a[i].z, a[i].w},
                           bs[2][4] = {{b[0][i].x, b[0][i].y, b[0][i].z, b[0][i].w}, {b[1][i].x, b[1][i].y, b[1][i].z, b[1][i].w}};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float2 u = bf16x2_to_f32(as[q]);
                if (SCALED) {
                    u.x *= power;
                    u.y *= power;
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float2 v = bf16x2_to_f32(bs[k][q]);
                    sum_exactly(s[k][0], c[k][0], __fmul_rn(u.x, v.x));    // (16 bits: exact products)
                    sum_exactly(s[k][1], c[k][1], __fmul_rn(u.y, v.y));
                }
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        c[k][0] = __fadd_rn(c[k][0], c[k][1]);
        sum_exactly(s[k][0], c[k][0], s[k][1]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float s1 = __shfl_xor_sync(0xFFFFFFFFu, s[k][0], o), c1 = __shfl_xor_sync(0xFFFFFFFFu, c[k][0], o);
            c[k][0] = __fadd_rn(c[k][0], c1);
            sum_exactly(s[k][0], c[k][0], s1);
        }
    d0 = static_cast<double>(s[0][0]) + static_cast<double>(c[0][0]);
    d1 = static_cast<double>(s[1][0]) + static_cast<double>(c[1][0]);
}

// Order-preserving whole numbers of floats (-0 as +0; NaNs do not occur here).
__device__ __forceinline__ uint32_t order_key(float v)
{
    const int b = __float_as_int(v + 0.0f);
    return static_cast<uint32_t>(b ^ ((b >> 31) | 0x80000000));
}

__device__ __forceinline__ float key_value(uint32_t k) { return __int_as_float(static_cast<int>(k & 0x80000000u ? k ^ 0x80000000u : ~k)); }

// The same of doubles. (A comparison of doubles takes this GPU 16 cycles.)
__device__ __forceinline__ uint64_t order_key(double v)
{
    const long long b = __double_as_longlong(v + 0.0);
    return static_cast<uint64_t>(b ^ ((b >> 63) | (1LL << 63)));
}

__device__ __forceinline__ double key_value(uint64_t k) { return __longlong_as_double(static_cast<long long>(k >> 63 ? k ^ (1ULL << 63) : ~k)); }

// A token's candidates, in the order of their experts.
struct Candidates {
    uint64_t key[kE];
    float v[kE];
    uint8_t e[kE], near[kE];                     // near: those with another candidate within the gap
    float pick_v[kK];
    int pick_i[kK];
};

// The near experts' logits of one token, x times a power of two, by its warp alone. (Seldom, and out of
// line: in the choice's own code this took a microsecond of 16,381 tokens' 48.)
__device__ __noinline__ void scaled_logits(Candidates &cand, int nears, const uint16_t *x, const uint16_t *w, const float *b, float power, int lane)
{
    for (int r = 0; r < nears; r += 2) {
        const int at = cand.near[r + (lane == 1 && r + 1 < nears)], e = cand.e[at], e0 = __shfl_sync(0xFFFFFFFFu, e, 0),
                  e1 = __shfl_sync(0xFFFFFFFFu, e, 1);
        double d = 0.0;
        for (int part = 0; part < kTopWarps; ++part) {
            double d0, d1;
            exact_parts<true>(x, w + static_cast<int64_t>(e0) * kH, w + static_cast<int64_t>(e1) * kH, power, part, lane, d0, d1);
            d += lane ? d1 : d0;
        }
        if (lane < 2)
            cand.key[at] = order_key(d / static_cast<double>(power) + static_cast<double>(b ? __ldcg(b + e) : 0.0f));
    }
}

// A warp per token; lane l has experts l, l + 32, l + 64, l + 96. MOST: splits at most. The
// CTA's warps share out the near experts' logits of all its tokens: one token in twenty has
// some (a token a warp for itself: 100 tokens 17.7 us in all, now 14.6; 16,381 tokens 53 and 48).
template <int MOST>
__global__ void __launch_bounds__(32 * kTopWarps, MOST == 1 ? 8 : 7) k_route_top(const TopArgs p)
{
    __shared__ int ask[kTopWarps];               // two experts of each warp's token, or -1
    __shared__ double answer[kTopWarps][kTopWarps][2];
    __shared__ Candidates cands[kTopWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTopWarps, t = t0 + warp;
    const bool has = t < p.T;
    tc::after_previous();
    tc::let_next_start();
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f}, b[4], part[MOST][4];
    // (all of a token's parts on their way at once)
    const float x2_part = has && lane < p.splits ? __ldcg(p.xn2 + lane * p.T + t) : 0.0f;
    float w2_part = 0.0f;
    if (lane < 4)
#pragma unroll
        for (int s = 0; s < MOST; ++s)
            w2_part += s < p.splits ? __ldcg(p.wn2 + s * 4 + lane) : 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        b[q] = p.b ? __ldcg(p.b + lane + 32 * q) : 0.0f;
#pragma unroll
    for (int s = 0; s < MOST; ++s)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            part[s][q] = has && s < p.splits ? __ldcg(p.part + (s * p.T + t) * kE + lane + 32 * q) : 0.0f;
#pragma unroll
    for (int s = 0; s < MOST; ++s)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            v[q] += part[s][q];
    const float x2 = warp_sum(x2_part), w2 = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(w2_part)));
    bool bad = false;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v[q] += b[q];
        if (isnan(v[q])) {
            v[q] = -INFINITY;
            bad = true;
        }
    }
    if (__any_sync(0xFFFFFFFFu, bad) && lane == 0)
        atomicOr(p.status, FGM_STATUS_NONFINITE_LOGITS);

    // The 9 largest: a lane's keys in falling order, equal ones by expert, and the largest head of all in
    // turn, of the lowest expert that has it. Lane r keeps the r-th.
    uint32_t key[4];
    int who[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        key[q] = order_key(v[q]);
        who[q] = q * 32 + lane;
    }
#pragma unroll
    for (int r = 0; r < 3; ++r)
#pragma unroll
        for (int q = 0; q < 3 - r; ++q) {
            const bool swap = key[q + 1] > key[q];
            const uint32_t k = key[q];
            const int w = who[q];
            key[q] = swap ? key[q + 1] : k;
            who[q] = swap ? who[q + 1] : w;
            key[q + 1] = swap ? k : key[q + 1];
            who[q + 1] = swap ? w : who[q + 1];
        }
    uint32_t top_k = 0;
    int top_i = 0;
#pragma unroll
    for (int r = 0; r <= kK; ++r) {
        const uint32_t best = __reduce_max_sync(0xFFFFFFFFu, key[0]);
        const int e = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, key[0] == best ? static_cast<unsigned>(who[0]) : ~0u));
        const bool mine = who[0] == e;
        top_k = lane == r ? best : top_k;
        top_i = lane == r ? e : top_i;
#pragma unroll
        for (int q = 0; q < 3; ++q) {
            key[q] = mine ? key[q + 1] : key[q];
            who[q] = mine ? who[q + 1] : who[q];
        }
        key[3] = mine ? 0u : key[3];             // (below every number's)
    }
    float top_v = key_value(top_k);
    // Twice the bound of a candidate's error: kLogitError |x| |w| of its products, 2^-23 of the sum with the bias
    // (without an x the logits are the biases; experts masked by a bias of -inf have no near one).
    const float most = __uint_as_float(
        __reduce_max_sync(0xFFFFFFFFu, lane < kK && fabsf(top_v) < INFINITY ? __float_as_uint(fabsf(top_v)) : 0u));
    float gap = 0.0f, power = 1.0f;
    if (x2 >= kLow && x2 <= kHigh && w2 >= kLow && w2 <= kHigh) {
        gap = 2.0f * (kLogitError * (x2 * rsqrtf(x2)) * (w2 * rsqrtf(w2)) + 0x1p-23f * most);
    } else if (has && w2 != 0.0f) {
        float inverse;
        const float x1 = row_norm(p.x + t * p.stride, lane, power, inverse), w1 = w2 < kHuge ? sqrtf(fmaxf(w2, kLow)) : INFINITY;
        // (2^-112: what products that fall below fp32's normal numbers may lose; elements of rows above kHigh and below kLow
        // meet x at a size that keeps products and sums within fp32's range)
        gap = x1 > 0.0f ? fmaxf(2.0f * (kLogitError * x1 * w1 * inverse + 0x1p-23f * most), 0x1p-112f) : 0.0f;
        power = fminf(power * (w2 > kHigh ? 0x1p-20f : w2 < kLow ? 0x1p60f : 1.0f), 0x1p126f);
    }
    // (in order, only neighbours can be the nearest)
    const float next = __shfl_down_sync(0xFFFFFFFFu, top_v, 1);
    const bool close = lane < kK && next > -INFINITY && (top_v - next <= gap || next >= top_v - gap);
    Candidates &cand = cands[warp];
    int n = 0, nears = 0;
    if (gap > 0.0f && __any_sync(0xFFFFFFFFu, close)) {
        const float low = __shfl_sync(0xFFFFFFFFu, top_v, kK - 1) - gap;
        const unsigned before = (1u << lane) - 1;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const unsigned m = __ballot_sync(0xFFFFFFFFu, v[q] >= low);
            if (v[q] >= low) {
                const int at = n + __popc(m & before);
                cand.e[at] = static_cast<uint8_t>(q * 32 + lane);
                cand.v[at] = v[q];
                cand.key[at] = order_key(static_cast<double>(v[q]));
            }
            n += __popc(m);
        }
        __syncwarp();
        for (int j = lane; j - lane < n; j += 32) {
            const float mine = cand.v[j < n ? j : 0];
            bool near = false;
            for (int i = 0; i < n; ++i) {
                const float d = fabsf(mine - cand.v[i]);
                near |= i != j && d <= gap && d < INFINITY;
            }
            near &= j < n;
            const unsigned m = __ballot_sync(0xFFFFFFFFu, near);
            if (near)
                cand.near[nears + __popc(m & before)] = static_cast<uint8_t>(j);
            nears += __popc(m);
        }
        __syncwarp();
    }
    int asks = nears;
    if (power != 1.0f) {
        scaled_logits(cand, nears, p.x + t * p.stride, p.w, p.b, power, lane);
        asks = 0;
    }
    if (__syncthreads_or(asks)) {
        // (two at a time: near ones come in pairs)
        for (int r = 0;; r += 2) {
            const bool more = r < asks;
            const int at = more ? cand.near[r + (lane == 1 && r + 1 < asks)] : 0, e = more ? cand.e[at] : 0,
                      e1 = __shfl_sync(0xFFFFFFFFu, e, 1);
            if (lane == 0)
                ask[warp] = more ? e | e1 << 8 : -1;
            if (!__syncthreads_or(more))
                break;
            const float bias = more && lane < 2 && p.b ? __ldcg(p.b + e) : 0.0f;
            for (int k = 0; k < kTopWarps; ++k) {
                const int pair = ask[k];
                if (pair < 0)
                    continue;
                double d0, d1;
                exact_parts<false>(p.x + (t0 + k) * p.stride, p.w + static_cast<int64_t>(pair & 255) * kH, p.w + static_cast<int64_t>(pair >> 8) * kH,
                                   1.0f, warp, lane, d0, d1);
                if (lane < 2)
                    answer[k][warp][lane] = lane ? d1 : d0;
            }
            __syncthreads();
            if (more && lane < 2) {
                double d = 0.0;
#pragma unroll
                for (int k = 0; k < kTopWarps; ++k)
                    d += answer[warp][k][lane];
                cand.key[at] = order_key(d + static_cast<double>(bias));
            }
        }
    }
    if (nears) {
        // each candidate's place: as many as are before it
        __syncwarp();
        for (int j = lane; j < n; j += 32) {
            const uint64_t mine = cand.key[j];
            int place = 0;
            for (int i = 0; i < n; ++i) {
                const uint64_t other = cand.key[i];
                place += other > mine || (other == mine && i < j);
            }
            if (place < kK) {
                cand.pick_i[place] = cand.e[j];
                cand.pick_v[place] = static_cast<float>(key_value(mine));
            }
        }
        __syncwarp();
        if (lane < kK) {
            top_i = cand.pick_i[lane];
            top_v = cand.pick_v[lane];
        }
    }
    const float largest = __shfl_sync(0xFFFFFFFFu, top_v, 0), ex = largest == -INFINITY ? 1.0f : expf(top_v - largest);
    float sum = 0.0f;
#pragma unroll
    for (int r = 0; r < kK; ++r)
        sum += __shfl_sync(0xFFFFFFFFu, ex, r);
    if (has && lane < kK) {
        p.ids[t * kK + lane] = top_i;
        p.wts[t * kK + lane] = ex / sum;
        if (p.count)                             // (whole numbers: their order does not matter)
            atomicAdd(p.count + static_cast<unsigned>(t) / p.chunk * kE + top_i, 1);
    }
}

}  // namespace route
}  // namespace fgm
