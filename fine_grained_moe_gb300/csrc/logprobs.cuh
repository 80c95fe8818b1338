// Log probabilities of given tokens, entropy and top alternatives of rows of
// logits (fgm_logprobs, and the second step of fgm_lm_head_logprobs).
//
//   l = sum_v exp((z_v - m) / T),  logp(t) = (z_t - m) / T - ln l,
//   H = ln l - (1 / l) sum_v exp((z_v - m) / T) (z_v - m) / T,  m = max z
//
// One pass over the logits, which bounds it: a lane keeps a running maximum m,
// l and w = sum e d (d = (z - m) log2(e) / T, e = 2^d) over 16 logits at a time
// and rescales when its maximum grows. Differences are clamped at -200, where e
// is 0 already, so that -inf (or a type's lowest value) adds 0 and not 0 * inf.
// About 7 instructions and one exponential a logit. 600 rows of 262,144 fp32
// logits: 96 us, 6.5 TB/s. 1,013 rows of 50,021 bf16 logits: 28 us, 3.6 TB/s,
// where 1,013 CTAs are 1.7 rounds of the 608 that run at a time, each with a start
// and an end. (Fewer instructions, six a logit, left both as they are; CTAs of
// four warps, eight an SM, too, and took 19 to 38 us on 5 rows.)
//
// The k best cost nothing in that pass: the k-th largest of 32 maxima, each of 8
// threads, bounds the k-th best logit from below, so only the threads that reach
// it (little more than k of 256 unless logits tie) can hold one of the k best, and
// the warps, which share them out, read those threads' logits a second time, from
// the caches; the few at or above the bound are ranked by counting. (Lists kept during the
// pass, with the same bound as a threshold, took 134 us on 1,013 x 50,021 bf16
// logits, against 15 us of HBM time: the insertions were most of it.)
//
// Short rows in large numbers have a warp each (k_logprob_rows). Long rows are cut
// into splits until the grid has several CTAs per SM; k_logprob_join merges a row's
// splits in order (no atomics on results: the same call gives the same bits).
#pragma once

#include "common.cuh"

namespace fgm {
namespace score {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxTop = FGM_MAX_TOP;
constexpr int kMaxList = kMaxTop + 4;         // entries of a partial list (lm_score.cuh keeps a few more than asked for)
constexpr int kVals = 16;                     // logits of a lane and chunk
constexpr int kCands = 64;                    // logits at or above the bound that are ranked as they are
constexpr float kClamp = -200.0f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kNone = 0x7FFFFFFF;

// A split's (or a row's) result.
struct Part {
    float m, l, w;
    int nan;
    float v[kMaxList];
    int32_t i[kMaxList];
};

struct Outs {
    const int32_t *tokens;   // [N] or NULL
    float *logp;             // [N] or NULL
    float *entropy;          // [N] or NULL
    int32_t *top_ids;        // [N][k]
    float *top_logp;         // [N][k]
    int k;
    float T;
    int64_t V;
    int32_t *status;
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max_nan(float a, float b, float c)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// Two fp32 in a register pair, for the packed multiply-add.
__device__ __forceinline__ uint64_t pack2(float a, float b)
{
    uint64_t y;
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(a), "f"(b));
    return y;
}

__device__ __forceinline__ float2 unpack2(uint64_t x)
{
    float2 y;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(y.x), "=f"(y.y) : "l"(x));
    return y;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t y;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(a), "l"(b), "l"(c));
    return y;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t y;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
    return y;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t y;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
    return y;
}

// log2(e) / T, held to a finite number (T down to the smallest with 1 / T finite).
__device__ __forceinline__ float per_nat(float T) { return fminf(kLog2e / T, 3.4028235e38f); }

// An order of floats as unsigned integers (NaN does not occur; -0 is 0).
__device__ __forceinline__ unsigned ordered(float x)
{
    const unsigned u = __float_as_uint(x + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float unordered(unsigned u)
{
    return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}

// Running sums of a lane, a warp or a row.
struct Sums {
    float m, l, w;

    __device__ void clear()
    {
        m = -INFINITY;
        l = w = 0.0f;
    }

    // Moves the reference up to nm >= m.
    __device__ void rise(float nm, float c)
    {
        const float d = fmaxf((m - nm) * c, kClamp), f = ex2(d);
        w = f * fmaf(d, l, w);
        l *= f;
        m = nm;
    }

    __device__ void add(Sums o, float c)
    {
        const float nm = fmaxf(m, o.m);
        rise(nm, c);
        o.rise(nm, c);
        l += o.l;
        w += o.w;
    }

    // One logit.
    __device__ void add(float z, float c)
    {
        if (z > m)
            rise(z, c);
        const float d = fmaxf((z - m) * c, kClamp), e = ex2(d);
        l += e;
        w = fmaf(e, d, w);
    }
};

// The largest of 16 logits, in three levels; NaN if one is.
__device__ __forceinline__ float max16(const float (&v)[kVals])
{
    const float a = max_nan(v[0], v[1], v[2]), b = max_nan(v[3], v[4], v[5]), d = max_nan(v[6], v[7], v[8]);
    const float e = max_nan(v[9], v[10], v[11]), f = max_nan(v[12], v[13], v[14]);
    return max_nan(max_nan(a, b, d), max_nan(e, f, v[15]), v[15]);
}

// The largest of 16 logits; NaN becomes -inf, in v too.
__device__ __forceinline__ float largest(float (&v)[kVals], int &nan)
{
    float mx = max16(v);
    if (mx != mx) {
        nan = 1;
        mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < kVals; ++j) {
            v[j] = v[j] == v[j] ? v[j] : -INFINITY;
            mx = fmaxf(mx, v[j]);
        }
    }
    return mx;
}

// 16 logits, the largest of them mx, into the running sums of a lane.
__device__ __forceinline__ void fold(Sums &s, const float (&v)[kVals], float mx, float c)
{
    if (mx > s.m)
        s.rise(mx, c);
    // (z - m) c, the difference first: it is exact near the maximum, where z c - m c would be off by m c's rounding, all
    // of a term at a low temperature. (What is not a number, -inf from -inf, the clamp takes too.)
    const uint64_t cc = pack2(c, c), nm = pack2(-s.m, -s.m);
    uint64_t l2[2] = {0, 0}, w2[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < kVals; j += 2) {
        const float2 d = unpack2(mul2(add2(pack2(v[j], v[j + 1]), nm), cc));
        const float d0 = fmaxf(d.x, kClamp), d1 = fmaxf(d.y, kClamp);
        const uint64_t e = pack2(ex2(d0), ex2(d1));
        l2[j >> 1 & 1] = add2(l2[j >> 1 & 1], e);
        w2[j >> 1 & 1] = fma2(e, pack2(d0, d1), w2[j >> 1 & 1]);
    }
    const float2 l = unpack2(add2(l2[0], l2[1])), w = unpack2(add2(w2[0], w2[1]));
    s.l += l.x + l.y;
    s.w += w.x + w.y;
}

// The sums of 32 lanes: one reference for all, then plain sums in a fixed order.
__device__ __forceinline__ Sums warp_sums(Sums s, float c)
{
    s.rise(unordered(__reduce_max_sync(0xFFFFFFFFu, ordered(s.m))), c);
    s.l = warp_sum(s.l);
    s.w = warp_sum(s.w);
    return s;
}

// The k best of a warp: lane i holds the i-th (value, index).
struct TopList {
    float v;
    int32_t i;

    __device__ void clear()
    {
        v = -INFINITY;
        i = kNone;
    }

    __device__ void insert(float nv, int32_t ni, int lane)
    {
        const int at = __popc(__ballot_sync(0xFFFFFFFFu, better(v, i, nv, ni)));
        const float pv = __shfl_up_sync(0xFFFFFFFFu, v, 1);
        const int32_t pi = __shfl_up_sync(0xFFFFFFFFu, i, 1);
        if (lane == at) {
            v = nv;
            i = ni;
        } else if (lane > at) {
            v = pv;
            i = pi;
        }
    }

    // Inserts every lane's candidate that is better than the k-th.
    __device__ void offer(float cv, int32_t ci, int k, int lane)
    {
        for (;;) {
            const float tv = __shfl_sync(0xFFFFFFFFu, v, k - 1);
            const int32_t ti = __shfl_sync(0xFFFFFFFFu, i, k - 1);
            const unsigned b = __ballot_sync(0xFFFFFFFFu, better(cv, ci, tv, ti));
            if (!b)
                return;
            const int src = __ffs(b) - 1;
            insert(__shfl_sync(0xFFFFFFFFu, cv, src), __shfl_sync(0xFFFFFFFFu, ci, src), lane);
            if (lane == src) {
                cv = -INFINITY;
                ci = kNone;
            }
        }
    }
};

// k-way merge of up to 32 sorted lists, one a lane (n entries, kNone past the
// end): lane j gets the j-th best of all.
__device__ __forceinline__ void merge_lists(const float *v, const int32_t *i, int n, int k, int lane, float &gv, int32_t &gi)
{
    float hv = n > 0 ? v[0] : -INFINITY, nv = n > 1 ? v[1] : -INFINITY;      // the head and the entry behind it
    int32_t hi = n > 0 ? i[0] : kNone, ni = n > 1 ? i[1] : kNone;
    int at = 2;
    gv = -INFINITY;
    gi = kNone;
    for (int j = 0; j < k; ++j) {
        const unsigned o = ordered(hv), bv = __reduce_max_sync(0xFFFFFFFFu, o);
        const unsigned bi = __reduce_min_sync(0xFFFFFFFFu, o == bv ? static_cast<unsigned>(hi) : 0xFFFFFFFFu);
        if (lane == j) {
            gv = unordered(bv);
            gi = static_cast<int32_t>(bi);
        }
        if (o == bv && static_cast<unsigned>(hi) == bi && hi != kNone) {
            hv = nv;
            hi = ni;
            nv = at < n ? v[at] : -INFINITY;
            ni = at < n ? i[at] : kNone;
            ++at;
        }
        __syncwarp();
    }
}

// A row's outputs from its sums and list (one warp). ztok: the given token's
// logit (-inf outside the vocabulary).
__device__ __forceinline__ void write_row(const Outs &o, int64_t row, const Sums &s, const TopList &t, int nan, float ztok, int lane)
{
    // a row without a finite maximum has no distribution
    const bool ok = fabsf(s.m) < INFINITY;
    const float lnl = logf(s.l), none = __int_as_float(0x7FC00000);
    if (lane == 0) {
        if (nan || !ok)
            atomicOr(o.status, FGM_STATUS_NONFINITE_LOGITS);
        if (o.logp)
            o.logp[row] = ok ? (ztok - s.m) / o.T - lnl : none;
        if (o.entropy)
            o.entropy[row] = ok ? lnl - s.w * kLn2 / s.l : none;
    }
    if (lane < o.k) {
        o.top_ids[row * o.k + lane] = t.i;
        o.top_logp[row * o.k + lane] = ok ? (t.v - s.m) / o.T - lnl : none;
    }
}

template <typename E>
struct Load;
template <>
struct Load<float> {
    static constexpr int kVec = 4;
    static __device__ float one(const float *p) { return *p; }
    static __device__ void unpack(const uint4 &r, float *v)
    {
        v[0] = __uint_as_float(r.x);
        v[1] = __uint_as_float(r.y);
        v[2] = __uint_as_float(r.z);
        v[3] = __uint_as_float(r.w);
    }
};
template <>
struct Load<__nv_bfloat16> {
    static constexpr int kVec = 8;
    static __device__ float one(const __nv_bfloat16 *p)
    {
        return bf16_to_f32(*reinterpret_cast<const uint16_t *>(p));
    }
    static __device__ void unpack(const uint4 &r, float *v)
    {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = bf16x2_to_f32(w[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
};
template <>
struct Load<__half> {
    static constexpr int kVec = 8;
    static __device__ float one(const __half *p)
    {
        __half_raw r;
        r.x = *reinterpret_cast<const uint16_t *>(p);
        return __half2float(__half(r));
    }
    static __device__ void unpack(const uint4 &r, float *v)
    {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __half2_raw h;
            h.x = static_cast<uint16_t>(w[i]);
            h.y = static_cast<uint16_t>(w[i] >> 16);
            const float2 f = __half22float2(__half2(h));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
};

// CTA (row, split): one pass over the split's logits.
template <typename E>
__global__ void __launch_bounds__(kThreads, 4)
    k_logprobs(const E *z, int64_t stride, int splits, Part *part, const Outs o)
{
    using L = Load<E>;
    constexpr int kVec = L::kVec, kLoads = kVals / kVec, kChunk = 32 * kLoads;      // vectors of a warp's chunk
    constexpr int kDepth = 4 / kLoads;         // chunks on their way: four vectors a lane, 64 KB an SM
    __shared__ unsigned s_max[kThreads], s_bound;
    __shared__ int s_who[kThreads], s_many, s_n;
    __shared__ float s_cv[kCands];
    __shared__ int32_t s_ci[kCands];
    __shared__ Sums s_sum[kWarps];
    __shared__ float s_v[kWarps][kMaxTop];
    __shared__ int32_t s_i[kWarps][kMaxTop];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, k = o.k;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t row = blockIdx.x / splits;
    const int split = static_cast<int>(blockIdx.x - row * splits);
    const E *zr = z + row * stride;
    const int V = static_cast<int>(o.V);
    // logits before the first 16-byte boundary, whole vectors, the rest
    const int off = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(zr) & 15u)) & 15u) / static_cast<int>(sizeof(E));
    const int head = min(V, off), nvec = (V - head) / kVec, tail = V - head - nvec * kVec;
    const uint4 *zv = reinterpret_cast<const uint4 *>(zr + head);
    const int v0 = static_cast<int>(static_cast<int64_t>(nvec) * split / splits);
    const int v1 = static_cast<int>(static_cast<int64_t>(nvec) * (split + 1) / splits);
    const float c = per_nat(o.T);

    float zt = -INFINITY;                      // the given token's logit
    if (splits == 1 && o.logp && tid == 0) {
        const int32_t t = __ldcg(o.tokens + row);
        if (t >= 0 && t < V)
            zt = L::one(zr + t);
        if (zt != zt)
            zt = -INFINITY;
    }
    Sums s;
    s.clear();
    int nan = 0;
    uint4 raw[kDepth][kLoads];
    auto fetch = [&](int at, uint4 (&r)[kLoads]) {      // one chunk's vectors of this lane
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if (at + i * 32 < v1)
                r[i] = zv[at + i * 32];
    };

    int at = v0 + warp * kChunk + lane;
    const int step = kWarps * kChunk;
#pragma unroll
    for (int q = 0; q < kDepth; ++q)
        fetch(at + q * step, raw[q]);
    const bool edges = split == 0 && warp == 0 && head + tail > 0;      // this warp takes the logits around the vectors
    if (edges) {
        float v[kVals];
#pragma unroll
        for (int j = 0; j < kVals; ++j)
            v[j] = -INFINITY;
        if (lane < head)
            v[0] = L::one(zr + lane);
        if (lane < tail)
            v[1] = L::one(zr + V - tail + lane);
        fold(s, v, largest(v, nan), c);
    }
    while (at - lane < v1) {
#pragma unroll
        for (int q = 0; q < kDepth; ++q) {
            if (at - lane < v1) {
                float v[kVals];
#pragma unroll
                for (int i = 0; i < kLoads; ++i)
                    L::unpack(raw[q][i], v + i * kVec);
                if (at - lane + kChunk > v1) { // past the end: -inf
#pragma unroll
                    for (int i = 0; i < kLoads; ++i)
                        if (at + i * 32 >= v1)
#pragma unroll
                            for (int j = 0; j < kVec; ++j)
                                v[i * kVec + j] = -INFINITY;
                }
                fetch(at + kDepth * step, raw[q]);
                fold(s, v, largest(v, nan), c);
            }
            at += step;
        }
    }

    // ------------------------------------------------------------ the k best
    TopList top;
    top.clear();
    if (k) {
        s_max[tid] = ordered(s.m);
        __syncthreads();
        if (warp == 0) {
            // the k-th largest of 32 maxima, of 8 threads each, by counting the larger ones
            unsigned best = 0;
#pragma unroll
            for (int i = 0; i < kWarps; ++i)
                best = max(best, s_max[i * 32 + lane]);
            int above = 0;
#pragma unroll
            for (int q = 0; q < 32; ++q) {
                const unsigned x = __shfl_sync(0xFFFFFFFFu, best, q);
                above += x > best || (x == best && q < lane);
            }
            if (above == k - 1)
                s_bound = best;
            if (lane == 0)
                s_many = s_n = 0;
        }
        __syncthreads();
        const float bound = unordered(s_bound);
        // the threads that reach the bound, in any order (the lists do not depend on it), dealt to the warps
        if (s.m >= bound)
            s_who[atomicAdd(&s_many, 1)] = tid;
        __syncthreads();
        // every logit of theirs that reaches the bound goes to `take`, which the whole warp calls
        auto look_again = [&](auto &&take) {
            for (int w = warp; w < s_many; w += kWarps) {
                const int who = s_who[w], src = who & 31, start = v0 + (who >> 5) * kChunk + src;
                if (who < 32 && split == 0 && head + tail > 0) {
                    float v = -INFINITY;
                    const int i = lane == 0 ? src : V - tail + src;
                    const bool in = lane == 0 ? src < head : lane == 1 && src < tail;
                    if (in) {
                        v = L::one(zr + i);
                        v = v == v ? v : -INFINITY;
                    }
                    take(in && v >= bound, v, i);
                }
                // its logits, a vector a lane
                for (int n0 = 0;; n0 += 32) {
                    const int n = n0 + lane;   // the thread's n-th vector
                    const int vec = start + n / kLoads * step + n % kLoads * 32;
                    const bool in = vec < v1;
                    if (!__any_sync(0xFFFFFFFFu, in))
                        break;
                    float v[kVec];
                    if (in)
                        L::unpack(zv[vec], v);
#pragma unroll
                    for (int j = 0; j < kVec; ++j) {
                        const float x = in && v[j] == v[j] ? v[j] : -INFINITY;
                        take(in && x >= bound, x, head + vec * kVec + j);
                    }
                }
            }
        };
        look_again([&](bool in, float x, int i) {
            if (in) {
                const int at = atomicAdd(&s_n, 1);
                if (at < kCands) {
                    s_cv[at] = x;
                    s_ci[at] = i;
                }
            }
        });
        __syncthreads();
        const int n = s_n;
        if (n <= kCands) {
            // few: the first warp ranks them (their order in the list does not matter)
            if (warp == 0) {
                float v[2];
                int32_t i[2];
                int above[2] = {0, 0};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool in = lane + 32 * h < n;
                    v[h] = in ? s_cv[lane + 32 * h] : -INFINITY;
                    i[h] = in ? s_ci[lane + 32 * h] : kNone;
                }
                for (int q = 0; q < n; ++q)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        above[h] += better(s_cv[q], s_ci[q], v[h], i[h]);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (lane + 32 * h < n && above[h] < k) {
                        s_v[0][above[h]] = v[h];
                        s_i[0][above[h]] = i[h];
                    }
                __syncwarp();
                if (lane < min(n, k)) {
                    top.v = s_v[0][lane];
                    top.i = s_i[0][lane];
                }
            }
        } else {
            // many that tie: lists of the warps' own, merged
            look_again([&](bool in, float x, int i) {
                if (__any_sync(0xFFFFFFFFu, in))
                    top.offer(in ? x : -INFINITY, in ? i : kNone, k, lane);
            });
            if (lane < k) {
                s_v[warp][lane] = top.v;
                s_i[warp][lane] = top.i;
            }
            __syncthreads();
            if (warp == 0)
                merge_lists(s_v[lane & (kWarps - 1)], s_i[lane & (kWarps - 1)], lane < kWarps ? k : 0, k, lane, top.v, top.i);
        }
    }

    // ------------------------------------------------------------ the CTA's split
    s = warp_sums(s, c);
    if (lane == 0)
        s_sum[warp] = s;
    nan = __syncthreads_or(nan);
    if (warp)
        return;
    if (lane < kWarps)
        s = s_sum[lane];
    else
        s.clear();
    s = warp_sums(s, c);
    if (splits == 1) {
        write_row(o, row, s, top, nan, zt, lane);
        return;
    }
    Part *p = part + static_cast<int64_t>(blockIdx.x);
    if (lane == 0) {
        p->m = s.m;
        p->l = s.l;
        p->w = s.w;
        p->nan = nan;
    }
    if (lane < k) {
        p->v[lane] = top.v;
        p->i[lane] = top.i;
    }
}

// The same with a warp per row and no split, for rows too short to be worth a
// CTA's barriers: 20,000 rows of 3 KB take 39 us at k = 8 where a CTA each takes
// 136 (17 and 81 at k = 0), 4,864 rows of 16 KB 21 us where it takes 39 (fp32) and 26
// where it takes 46 (bf16). 57,788 rows of 715 fp32 logits: 91 us, 1.8 TB/s, bound by
// a row's end (count, second look, ranking), under which a warp loads nothing.
template <typename E>
__global__ void __launch_bounds__(kThreads, 4) k_logprob_rows(const E *z, int64_t stride, int64_t N, const Outs o)
{
    using L = Load<E>;
    constexpr int kVec = L::kVec, kLoads = kVals / kVec, kChunk = 32 * kLoads;      // vectors of a chunk
    constexpr int kDepth = 4 / kLoads;         // chunks on their way
    __shared__ float s_cands[kWarps][kCands], s_tops[kWarps][kMaxTop];
    __shared__ int32_t s_candi[kWarps][kCands], s_topi[kWarps][kMaxTop];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = o.k;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (row >= N)
        return;
    const E *zr = z + row * stride;
    const int V = static_cast<int>(o.V);
    // logits before the first 16-byte boundary, whole vectors, the rest
    const int off = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(zr) & 15u)) & 15u) / static_cast<int>(sizeof(E));
    const int head = min(V, off), nvec = (V - head) / kVec, tail = V - head - nvec * kVec;
    const uint4 *zv = reinterpret_cast<const uint4 *>(zr + head);
    const float c = per_nat(o.T);

    uint4 raw[kDepth][kLoads];
    auto fetch = [&](int at, uint4 (&r)[kLoads]) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if (at + i * 32 < nvec)
                r[i] = zv[at + i * 32];
    };
    int at = lane;
#pragma unroll
    for (int q = 0; q < kDepth; ++q)
        fetch(at + q * kChunk, raw[q]);
    float zt = -INFINITY;                      // the given token's logit
    if (o.logp && lane == 0) {
        const int32_t t = __ldcg(o.tokens + row);
        if (t >= 0 && t < V)
            zt = L::one(zr + t);
        if (zt != zt)
            zt = -INFINITY;
    }
    Sums s;
    s.clear();
    int nan = 0;
    if (head + tail > 0) {
        float v[kVals];
#pragma unroll
        for (int j = 0; j < kVals; ++j)
            v[j] = -INFINITY;
        if (lane < head)
            v[0] = L::one(zr + lane);
        if (lane < tail)
            v[1] = L::one(zr + V - tail + lane);
        fold(s, v, largest(v, nan), c);
    }
    while (at - lane < nvec) {
#pragma unroll
        for (int q = 0; q < kDepth; ++q) {
            if (at - lane < nvec) {
                float v[kVals];
#pragma unroll
                for (int i = 0; i < kLoads; ++i)
                    L::unpack(raw[q][i], v + i * kVec);
                if (at - lane + kChunk > nvec) {
#pragma unroll
                    for (int i = 0; i < kLoads; ++i)
                        if (at + i * 32 >= nvec)
#pragma unroll
                            for (int j = 0; j < kVec; ++j)
                                v[i * kVec + j] = -INFINITY;
                }
                fetch(at + kDepth * kChunk, raw[q]);
                fold(s, v, largest(v, nan), c);
            }
            at += kChunk;
        }
    }

    TopList top;
    top.clear();
    if (k) {
        // the k-th largest of the lanes' maxima bounds the k-th best logit
        const unsigned best = ordered(s.m);
        int above = 0;
#pragma unroll
        for (int q = 0; q < 32; ++q) {
            const unsigned x = __shfl_sync(0xFFFFFFFFu, best, q);
            above += x > best || (x == best && q < lane);
        }
        const float bound = __shfl_sync(0xFFFFFFFFu, s.m, __ffs(__ballot_sync(0xFFFFFFFFu, above == k - 1)) - 1);
        const unsigned who_mask = __ballot_sync(0xFFFFFFFFu, s.m >= bound);
        // every logit of the lanes that reach it, read again
        auto look_again = [&](auto &&take) {
            for (unsigned left = who_mask; left; left &= left - 1) {
                const int who = __ffs(left) - 1;
                if (head + tail > 0) {
                    float v = -INFINITY;
                    const int i = lane == 0 ? who : V - tail + who;
                    const bool in = lane == 0 ? who < head : lane == 1 && who < tail;
                    if (in) {
                        v = L::one(zr + i);
                        v = v == v ? v : -INFINITY;
                    }
                    take(in && v >= bound, v, i);
                }
                for (int n0 = 0;; n0 += 32) {
                    const int n = n0 + lane;   // its n-th vector
                    const int vec = who + n / kLoads * kChunk + n % kLoads * 32;
                    const bool in = vec < nvec;
                    if (!__any_sync(0xFFFFFFFFu, in))
                        break;
                    float v[kVec];
                    if (in)
                        L::unpack(zv[vec], v);
#pragma unroll
                    for (int j = 0; j < kVec; ++j) {
                        const float x = in && v[j] == v[j] ? v[j] : -INFINITY;
                        take(in && x >= bound, x, head + vec * kVec + j);
                    }
                }
            }
        };
        float *const cv = s_cands[warp];
        int32_t *const ci = s_candi[warp];
        int n = 0;
        look_again([&](bool in, float x, int i) {
            const unsigned b = __ballot_sync(0xFFFFFFFFu, in);
            const int to = n + __popc(b & ((1u << lane) - 1));
            n += __popc(b);
            if (in && to < kCands) {
                cv[to] = x;
                ci[to] = i;
            }
        });
        __syncwarp();
        if (n <= kCands) {
            for (int h = lane; h < n; h += 32) {
                const float v = cv[h];
                const int32_t i = ci[h];
                int ahead = 0;
                for (int q = 0; q < n; ++q)
                    ahead += better(cv[q], ci[q], v, i);
                if (ahead < k) {
                    s_tops[warp][ahead] = v;
                    s_topi[warp][ahead] = i;
                }
            }
            __syncwarp();
            if (lane < min(n, k)) {
                top.v = s_tops[warp][lane];
                top.i = s_topi[warp][lane];
            }
        } else {
            look_again([&](bool in, float x, int i) {
                if (__any_sync(0xFFFFFFFFu, in))
                    top.offer(in ? x : -INFINITY, in ? i : kNone, k, lane);
            });
        }
    }
    s = warp_sums(s, c);
    write_row(o, row, s, top, __any_sync(0xFFFFFFFFu, nan), zt, lane);
}

// One warp: the sums and the k best (at most 32) of a row's parts.
__device__ __forceinline__ void join_parts(const Part *p, int n, int k, float c, int lane, Sums &s, int &nan, TopList &top)
{
    s.clear();
    top.clear();
    for (int s0 = 0; s0 < n; s0 += 32) {
        const Part *mine = p + s0 + lane;
        const bool in = s0 + lane < n;
        if (in) {
            s.add(Sums{__ldcg(&mine->m), __ldcg(&mine->l), __ldcg(&mine->w)}, c);
            nan |= __ldcg(&mine->nan);
        }
        if (!k)
            continue;
        float gv;
        int32_t gi;
        merge_lists(mine->v, mine->i, in ? k : 0, k, lane, gv, gi);
        if (s0 == 0) {
            top.v = gv;
            top.i = gi;
        } else {
            top.offer(lane < k ? gv : -INFINITY, lane < k ? gi : kNone, k, lane);
        }
    }
    s = warp_sums(s, c);
    nan = __any_sync(0xFFFFFFFFu, nan);
}

// A warp per row merges its splits in order: the sums lane by lane and then
// across the lanes, the lists as a k-way merge of 32 sorted lists at a time.
template <typename E>
__global__ void __launch_bounds__(kThreads)
    k_logprob_join(const E *z, int64_t stride, int64_t N, int splits, const Part *part, const Outs o)
{
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = o.k;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (row >= N)
        return;
    const float c = per_nat(o.T);
    float zt = -INFINITY;
    if (o.logp) {
        const int32_t t = __ldcg(o.tokens + row);
        if (t >= 0 && t < o.V)
            zt = Load<E>::one(z + row * stride + t);
        if (zt != zt)
            zt = -INFINITY;
    }
    Sums s;
    int nan = 0;
    TopList top;
    join_parts(part + row * splits, splits, k, c, lane, s, nan, top);
    write_row(o, row, s, top, nan, zt, lane);
}

}  // namespace score
}  // namespace fgm
