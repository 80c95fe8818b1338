// Log probabilities of given tokens, entropy and top alternatives of rows of
// logits (fgm_logprobs, and the second step of fgm_lm_head_logprobs).
//
//   l = sum_v exp((z_v - m) / T),  logp(t) = (z_t - m) / T - ln l,
//   H = ln l - (1 / l) sum_v exp((z_v - m) / T) (z_v - m) / T,  m = max z
//
// One pass over the logits, which bounds it: a lane keeps a running maximum m,
// l and w = sum e d (d = (z - m) log2(e) / T, e = 2^d) over 32 logits at a time
// and rescales when its maximum grows. Differences are clamped at -200, where e
// is 0 already, so that -inf (or a type's lowest value) adds 0 and not 0 * inf.
// About 7 instructions and one exponential a logit, half of what HBM leaves
// time for at 2 bytes.
//
// The k best are a list spread over a warp's lanes (lane i holds the i-th), and
// a threshold: the best k-th value that any warp of the CTA holds. It starts as
// the largest, over the warps, of the k-th largest of the 32 lane maxima of the
// first chunk (k lanes reach it, so k logits do), so that hardly more than k
// logits of the row are ever inserted. A chunk whose maximum is below it costs
// one comparison a lane.
//
// Rows are cut into splits until the grid has several CTAs per SM; k_logprob_join
// merges a row's splits in order (no atomics on results: the same call gives
// the same bits).
#pragma once

#include "common.cuh"

namespace fgm {
namespace score {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxTop = FGM_MAX_TOP;
constexpr int kVals = 32;                     // logits of a lane and chunk
constexpr float kClamp = -200.0f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kNone = 0x7FFFFFFF;

// A split's (or a row's) result.
struct Part {
    float m, l, w;
    int nan;
    float v[kMaxTop];
    int32_t i[kMaxTop];
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

__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// An order of floats as unsigned integers (NaN does not occur).
__device__ __forceinline__ unsigned ordered(float x)
{
    const unsigned u = __float_as_uint(x);
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
};

__device__ __forceinline__ Sums warp_sums(Sums s, float c)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        s.add(Sums{__shfl_xor_sync(0xFFFFFFFFu, s.m, o), __shfl_xor_sync(0xFFFFFFFFu, s.l, o),
                   __shfl_xor_sync(0xFFFFFFFFu, s.w, o)},
              c);
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
    static __device__ float one(const float *p) { return __ldg(p); }
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
        return bf16_to_f32(__ldg(reinterpret_cast<const uint16_t *>(p)));
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
        r.x = __ldg(reinterpret_cast<const uint16_t *>(p));
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
__global__ void __launch_bounds__(kThreads, 2)
    k_logprobs(const E *z, int64_t stride, int splits, Part *part, const Outs o)
{
    using L = Load<E>;
    constexpr int kVec = L::kVec, kLoads = kVals / kVec;
    __shared__ unsigned s_thr;
    __shared__ Sums s_sum[kWarps];
    __shared__ float s_v[kWarps][kMaxTop];
    __shared__ int32_t s_i[kWarps][kMaxTop];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, k = o.k;
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
    const int chunks = (v1 - v0 + 32 * kLoads - 1) / (32 * kLoads);
    const float c = kLog2e / o.T;
    if (tid == 0)
        s_thr = 0;

    Sums s;
    s.clear();
    TopList top;
    top.clear();
    int nan = 0;
    uint4 raw[kLoads];
    float v[kVals];
    auto fetch = [&](int ch) {                 // one chunk's vectors of this lane
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int at = v0 + (ch * kLoads + i) * 32 + lane;
            if (at < v1)
                raw[i] = __ldcs(zv + at);
        }
    };
    auto spread = [&](int ch) {                // to fp32; past the end: -inf
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            L::unpack(raw[i], v + i * kVec);
            if (v0 + (ch * kLoads + i) * 32 + lane >= v1)
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    v[i * kVec + j] = -INFINITY;
        }
    };
    // ch < 0: the logits before the first and after the last vector
    auto index = [&](int ch, int j, int src) -> int32_t {
        if (ch < 0)
            return j == 0 ? src : V - tail + src;
        return head + (v0 + (ch * kLoads + j / kVec) * 32 + src) * kVec + j % kVec;
    };

    bool first = true;
    const int begin = split == 0 && warp == 0 && head + tail > 0 ? -kWarps : warp;
    int ch = begin;
    if (ch >= 0 && ch < chunks)
        fetch(ch);
    for (;;) {
        const bool work = ch < chunks;
        if (work) {
            if (ch >= 0) {
                spread(ch);
            } else {
#pragma unroll
                for (int j = 0; j < kVals; ++j)
                    v[j] = -INFINITY;
                if (lane < head)
                    v[0] = L::one(zr + lane);
                if (lane < tail)
                    v[1] = L::one(zr + V - tail + lane);
            }
        } else if (!first) {
            break;
        }
        const int next = ch + kWarps;
        if (next >= 0 && next < chunks)
            fetch(next);
        float mx[4];
        float cm = -INFINITY;
        if (work) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                mx[g] = v[g * 8];
#pragma unroll
                for (int j = 1; j < 8; ++j)
                    mx[g] = max_nan(mx[g], v[g * 8 + j]);
            }
            cm = max_nan(max_nan(mx[0], mx[1]), max_nan(mx[2], mx[3]));
            if (cm != cm) {                    // NaN counts as -inf
                nan = 1;
#pragma unroll
                for (int j = 0; j < kVals; ++j)
                    v[j] = v[j] == v[j] ? v[j] : -INFINITY;
                cm = -INFINITY;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    mx[g] = -INFINITY;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        mx[g] = fmaxf(mx[g], v[g * 8 + j]);
                    cm = fmaxf(cm, mx[g]);
                }
            }
            if (cm > s.m)
                s.rise(cm, c);
            float l0 = 0.0f, l1 = 0.0f, w0 = 0.0f, w1 = 0.0f;
            if (fabsf(s.m) < 1.0e30f) {        // one fused step: z c cannot overflow unless the result is below the clamp
                const float mc = s.m * c;
#pragma unroll
                for (int j = 0; j < kVals; j += 2) {
                    const float d0 = fmaxf(fmaf(v[j], c, -mc), kClamp), d1 = fmaxf(fmaf(v[j + 1], c, -mc), kClamp);
                    const float e0 = ex2(d0), e1 = ex2(d1);
                    l0 += e0;
                    l1 += e1;
                    w0 = fmaf(e0, d0, w0);
                    w1 = fmaf(e1, d1, w1);
                }
            } else {
#pragma unroll
                for (int j = 0; j < kVals; ++j) {
                    const float d = fmaxf((v[j] - s.m) * c, kClamp), e = ex2(d);
                    l0 += e;
                    w0 = fmaf(e, d, w0);
                }
            }
            s.l += l0 + l1;
            s.w += w0 + w1;
        }
        if (k) {
            if (first) {
                // a bound that k logits of the row reach, from the first chunk's lane maxima
                float x = cm, kth = -INFINITY;
                for (int j = 0; j < k; ++j) {
                    kth = x;
#pragma unroll
                    for (int q = 16; q > 0; q >>= 1)
                        kth = fmaxf(kth, __shfl_xor_sync(0xFFFFFFFFu, kth, q));
                    const unsigned b = __ballot_sync(0xFFFFFFFFu, x == kth);
                    if (lane == __ffs(b) - 1)
                        x = -INFINITY;
                }
                __syncthreads();               // s_thr is set
                if (lane == 0)
                    atomicMax(&s_thr, ordered(kth));
                __syncthreads();
            }
            if (work) {
                float bound = unordered(*reinterpret_cast<volatile unsigned *>(&s_thr));
                if (__any_sync(0xFFFFFFFFu, cm >= bound)) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        if (!__any_sync(0xFFFFFFFFu, mx[g] >= bound))
                            continue;
#pragma unroll
                        for (int j = g * 8; j < g * 8 + 8; ++j)
                            if (__any_sync(0xFFFFFFFFu, v[j] >= bound)) {
                                const bool in = v[j] >= bound && (ch >= 0 || (j == 0 ? lane < head : j == 1 && lane < tail)) &&
                                                (ch < 0 || v0 + (ch * kLoads + j / kVec) * 32 + lane < v1);
                                top.offer(in ? v[j] : -INFINITY, in ? index(ch, j, lane) : kNone, k, lane);
                            }
                    }
                    const float kth = __shfl_sync(0xFFFFFFFFu, top.v, k - 1);
                    if (lane == 0 && kth > bound)
                        atomicMax(&s_thr, ordered(kth));
                }
            }
        }
        first = false;
        ch = next;
    }

    // ------------------------------------------------------------ the CTA's split
    s = warp_sums(s, c);
    nan = __any_sync(0xFFFFFFFFu, nan);
    if (lane == 0)
        s_sum[warp] = s;
    if (lane < k) {
        s_v[warp][lane] = top.v;
        s_i[warp][lane] = top.i;
    }
    nan = __syncthreads_or(nan);
    if (warp)
        return;
    for (int w = 1; w < kWarps; ++w)
        s.add(s_sum[w], c);
    if (k)
        for (int w = 1; w < kWarps; ++w)
            top.offer(lane < k ? s_v[w][lane] : -INFINITY, lane < k ? s_i[w][lane] : kNone, k, lane);
    if (splits == 1) {
        float zt = -INFINITY;
        if (o.logp) {
            const int32_t t = __ldg(o.tokens + row);
            if (t >= 0 && t < V)
                zt = L::one(zr + t);
            if (zt != zt)
                zt = -INFINITY;
        }
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

// A warp per row merges its splits in order. The given token's logit comes from
// z, or (z NULL) from ztok.
template <typename E>
__global__ void __launch_bounds__(kThreads)
    k_logprob_join(const E *z, int64_t stride, const float *ztok, int64_t N, int splits, const Part *part, const Outs o)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = o.k;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (row >= N)
        return;
    const float c = kLog2e / o.T;
    const Part *p = part + row * splits;
    Sums s;
    s.clear();
    int nan = 0;
    TopList top;
    top.clear();
    for (int i = lane; i < splits; i += 32) {
        s.add(Sums{__ldcg(&p[i].m), __ldcg(&p[i].l), __ldcg(&p[i].w)}, c);
        nan |= __ldcg(&p[i].nan);
    }
    s = warp_sums(s, c);
    nan = __any_sync(0xFFFFFFFFu, nan);
    for (int i0 = 0; i0 < splits * k; i0 += 32) {
        const int i = i0 + lane;
        const bool in = i < splits * k;
        const int sp = in ? i / k : 0, j = in ? i - sp * k : 0;
        top.offer(in ? __ldcg(&p[sp].v[j]) : -INFINITY, in ? __ldcg(&p[sp].i[j]) : kNone, k, lane);
    }
    float zt = -INFINITY;
    if (o.logp) {
        if (z) {
            const int32_t t = __ldg(o.tokens + row);
            if (t >= 0 && t < o.V)
                zt = Load<E>::one(z + row * stride + t);
        } else {
            zt = __ldcg(ztok + row);
        }
        if (zt != zt)
            zt = -INFINITY;
    }
    write_row(o, row, s, top, nan, zt, lane);
}

}  // namespace score
}  // namespace fgm
