// What stands around the products of grouped.cuh: slots grouped by expert
// (fgm_moe_group, fgm_moe_route), activations as E4M3 terms, and the weighted sum
// of the experts' rows (fgm_moe_experts_fwd).
#pragma once

#include "tensor.cuh"

namespace fgm {
namespace rows {

// ---------------------------------------------------------------- grouping
//
// Slots 0 .. n - 1 with ids[i] in [0, E) (others belong to no expert), stably sorted
// by id: each chunk of slots is counted by a CTA; then each adds up the counts before
// it (of smaller ids, and of its own id in earlier chunks) and deals its slots, a
// warp a run of consecutive ones. No order of CTAs or atomics enters the result.

constexpr int kGroupThreads = 256;
constexpr int kGroupWarps = kGroupThreads / 32;
constexpr int kMaxChunks = 256;
constexpr int kMaxE = 1024;

struct GroupArgs {
    const int32_t *ids;
    int64_t n;               // slots
    int E;
    int chunk;               // slots of a CTA, a multiple of kGroupThreads
    int chunks;
    int32_t *count;          // [chunks][E] (chunks > 1)
    int32_t *offsets;        // [E + 1]
    int32_t *order;          // [n] slots by expert, or NULL
    int32_t *src;            // [n] their tokens, or NULL
    int32_t *pos;            // [n] each slot's place, -1 without an expert, or NULL
    int per;                 // slots of a token
    int shared;              // tokens that one more expert takes behind the others (offsets has E + 2 entries), 0: none
};

// Counts of a warp's run of slots in its own row of hist.
__device__ __forceinline__ void count_run(const GroupArgs &p, int64_t i0, int64_t i1, int *hist, int lane)
{
    for (int64_t i = i0; i < i1; i += 32) {
        const int id = i + lane < i1 ? __ldcg(p.ids + i + lane) : -1;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, id);
        if (id >= 0 && id < p.E && lane == __ffs(same) - 1)
            hist[id] += __popc(same);
        __syncwarp();
    }
}

__device__ __forceinline__ void run_of(const GroupArgs &p, int warp, int64_t &i0, int64_t &i1)
{
    const int64_t each = p.chunk / kGroupWarps;
    i0 = static_cast<int64_t>(blockIdx.x) * p.chunk + warp * each;
    i1 = i0 + each < p.n ? i0 + each : p.n;
}

__global__ void __launch_bounds__(kGroupThreads) k_group_count(const GroupArgs p)
{
    extern __shared__ int hist[];                // [kGroupWarps][E]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < kGroupWarps * p.E; i += kGroupThreads)
        hist[i] = 0;
    tc::after_previous();
    tc::let_next_start();
    __syncthreads();
    int64_t i0, i1;
    run_of(p, warp, i0, i1);
    count_run(p, i0, i1, hist + warp * p.E, lane);
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kGroupThreads) {
        int s = 0;
        for (int w = 0; w < kGroupWarps; ++w)
            s += hist[w * p.E + e];
        p.count[static_cast<int64_t>(blockIdx.x) * p.E + e] = s;
    }
}

__global__ void __launch_bounds__(kGroupThreads) k_group_deal(const GroupArgs p)
{
    extern __shared__ int hist[];                // [kGroupWarps][E], then [E] totals
    __shared__ int warp_sum[kGroupWarps];
    int *total = hist + kGroupWarps * p.E;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < kGroupWarps * p.E; i += kGroupThreads)
        hist[i] = 0;
    tc::after_previous();
    tc::let_next_start();
    __syncthreads();
    int64_t i0, i1;
    run_of(p, warp, i0, i1);
    count_run(p, i0, i1, hist + warp * p.E, lane);
    __syncthreads();
    // a warp's first place of each expert, from the chunk's first, and the expert's slots in all
    for (int e = threadIdx.x; e < p.E; e += kGroupThreads) {
        int before = 0, all = 0, mine = 0;
        if (p.chunks > 1)
#pragma unroll 8
            for (int c = 0; c < p.chunks; ++c) {
                const int v = __ldcg(p.count + static_cast<int64_t>(c) * p.E + e);
                before += c < static_cast<int>(blockIdx.x) ? v : 0;
                all += v;
            }
        for (int w = 0; w < kGroupWarps; ++w) {
            const int v = hist[w * p.E + e];
            hist[w * p.E + e] = before + mine;
            mine += v;
        }
        total[e] = p.chunks > 1 ? all : mine;
    }
    __syncthreads();
    // places before each expert: a thread scans E / 256 experts, rounded up
    const int each = (p.E + kGroupThreads - 1) / kGroupThreads, e0 = threadIdx.x * each;
    int sum = 0;
    for (int e = e0; e < e0 + each && e < p.E; ++e)
        sum += total[e];
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        incl += lane >= o ? u : 0;
    }
    if (lane == 31)
        warp_sum[warp] = incl;
    __syncthreads();
    int base = incl - sum;
    for (int w = 0; w < warp; ++w)
        base += warp_sum[w];
    for (int e = e0; e < e0 + each && e < p.E; ++e) {
        const int v = total[e];
        total[e] = base;
        if (blockIdx.x == 0)
            p.offsets[e] = base;
        base += v;
    }
    int all = 0;
    for (int w = 0; w < kGroupWarps; ++w)
        all += warp_sum[w];
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        p.offsets[p.E] = all;
        if (p.shared)
            p.offsets[p.E + 1] = all + p.shared;
    }
    __syncthreads();
    int *at = hist + warp * p.E;
    for (int64_t i = i0; i < i1; i += 32) {
        const int id = i + lane < i1 ? __ldcg(p.ids + i + lane) : -1;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, id);
        const bool in = id >= 0 && id < p.E;
        int to = -1;
        if (in)
            to = total[id] + at[id] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (in && lane == __ffs(same) - 1)
            at[id] += __popc(same);
        __syncwarp();
        if (i + lane < i1) {
            if (p.pos)
                p.pos[i + lane] = to;
            if (in && p.order)
                p.order[to] = static_cast<int32_t>(i + lane);
            if (in && p.src)
                p.src[to] = static_cast<int32_t>((i + lane) / p.per);
        }
    }
    if (p.shared) {
        const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.chunk / p.per;
        for (int64_t t = t0 + threadIdx.x; t < t0 + p.chunk / p.per && t < p.shared; t += kGroupThreads)
            p.src[all + t] = static_cast<int32_t>(t);
    }
}

// ---------------------------------------------------------------- terms
//
// A row v[0 .. K) as two E4M3 terms under a power of two s that puts its largest
// element into [128, 256): t1 = e4m3(v / s), t2 = e4m3(v / s - t1), in blocks of 32
// elements, t1's and then t2's, so that one copy of 128 bytes brings both. K is
// filled up with zeros to a multiple of 32. |v - s (t1 + t2)| is at most 2^-9 |v| or
// 2^-10 s, whichever is larger; of a bf16 number it is 0 or at most 2^-10 s. A row
// with an element that is not finite has s = NaN.

__device__ __forceinline__ uint32_t e4m3x4(const float *v)
{
    const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE, __NV_E4M3);
    return a | b << 16;
}

// Terms of elements k .. k + 7, written to the row.
__device__ __forceinline__ void write_terms(uint8_t *row, int k, const float *v)
{
    uint32_t hi[2], lo[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float d[4], r[4];
        hi[h] = e4m3x4(v + 4 * h);
        e4m3x4_to_f32(hi[h], d);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            r[q] = v[4 * h + q] - d[q];
        lo[h] = e4m3x4(r);
    }
    uint8_t *to = row + (k >> 5) * 64 + (k & 31);
    *reinterpret_cast<uint2 *>(to) = make_uint2(hi[0], hi[1]);
    *reinterpret_cast<uint2 *>(to + 32) = make_uint2(lo[0], lo[1]);
}

// 2^(e - 134), for a row whose largest exponent field is e: below 2^(e - 126), above 2^8 times less.
__device__ __forceinline__ float row_scale(int e) { return e == 255 ? __int_as_float(0x7FC00000) : __int_as_float((e - 7) << 23); }

constexpr int kTermWarps = 8;

// Rows of bf16: a warp each.
__global__ void __launch_bounds__(32 * kTermWarps) k_terms(const uint16_t *x, int64_t stride, int64_t n, int K, uint8_t *terms, float *scale)
{
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kTermWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, K32 = (K + 31) & ~31;
    tc::after_previous();
    tc::let_next_start();
    if (row >= n)
        return;
    const uint16_t *xr = x + row * stride;
    uint32_t m = 0;
    for (int k = lane * 8; k < K; k += 256) {
        const uint4 u = __ldcg(reinterpret_cast<const uint4 *>(xr + k));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int q = 0; q < 4; ++q)
            m = max(m, max(w[q] & 0x7FFFu, w[q] >> 16 & 0x7FFFu));
    }
    int e = static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, m) >> 7);
    e = e < 14 ? 14 : e;
    if (lane == 0)
        scale[row] = row_scale(e);
    const float up = __int_as_float((261 - e) << 23);         // 1 / s (e = 255: whatever it is, s is NaN)
    for (int k = lane * 8; k < K32; k += 256) {
        float v[8];
        uint4 u = make_uint4(0, 0, 0, 0);
        if (k < K)
            u = __ldcg(reinterpret_cast<const uint4 *>(xr + k));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 f = bf16x2_to_f32(w[q]);
            v[2 * q] = f.x * up;
            v[2 * q + 1] = f.y * up;
        }
        write_terms(terms + row * (2 * static_cast<int64_t>(K32)), k, v);
    }
}

// Rows of the gated activations (grouped.cuh: f16 under a power of two per 32), a
// warp each; only those of some expert.
__global__ void __launch_bounds__(32 * kTermWarps) k_act_terms(const uint16_t *act, const uint8_t *exps, const int32_t *n, uint8_t *terms,
                                                               float *scale)
{
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kTermWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    tc::after_previous();
    tc::let_next_start();
    if (row >= __ldcg(n))
        return;
    constexpr int kBlocks = kF / 32;
    const int mine = lane < kBlocks ? __ldcg(exps + row * kBlocks + lane) : 14;
    const int e = __reduce_max_sync(0xFFFFFFFFu, mine);
    if (lane == 0)
        scale[row] = row_scale(e);
#pragma unroll
    for (int i = 0; i < (kF + 255) / 256; ++i) {
        const int k = i * 256 + lane * 8, eb = __shfl_sync(0xFFFFFFFFu, mine, (k >> 5) & 31);
        if (k < kF) {
            const uint4 u = __ldcg(reinterpret_cast<const uint4 *>(act + row * kF + k));
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
            // a = f16 2^(eb - 141); over s: 2^(eb - e - 7)
            const int d = eb - e - 7 + 127;
            const float up = d > 0 ? __int_as_float(d << 23) : 0.0f;
            float v[8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[q]));
                v[2 * q] = f.x * up;
                v[2 * q + 1] = f.y * up;
            }
            write_terms(terms + row * (2 * kF), k, v);
        }
    }
}

// A power of two that is not below any of an expert's scales (its absolute value), 1 for none.
__global__ void __launch_bounds__(256) k_scale_max(const float *s, int n, float *smax)
{
    __shared__ uint32_t part[8];
    tc::after_previous();
    tc::let_next_start();
    uint32_t m = 0;
    for (int i = threadIdx.x; i < n; i += 256)
        m = max(m, __float_as_uint(__ldcg(s + static_cast<int64_t>(blockIdx.x) * n + i)) & 0x7FFFFFFFu);
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 8; ++w)
            m = max(m, part[w]);
        // (of scales beyond 2^126, infinite or NaN ones 2^127: what they give shows in the products)
        const uint32_t e = (m >> 23) + 1;
        smax[blockIdx.x] = m == 0 ? 1.0f : __uint_as_float((e > 254 ? 254 : e) << 23);
    }
}

// ---------------------------------------------------------------- weighted sum
//
// y_t = sum_k w_tk y[pos_tk] (+ the shared expert's row), k in order: rows of f16,
// which grouped.cuh wrote as f16(a 2^-12 / (sa smax)).
struct CombineArgs {
    const uint16_t *rows;    // [.][2816] f16
    const float *sa;         // [.] scales of the activations' terms
    const float *smax;       // [129]
    const int32_t *ids;      // [T][8]
    const float *w;          // [T][8]
    const int32_t *pos;      // [T][8]
    const int32_t *offsets;  // [129] or more; the shared expert's rows begin at offsets[128]
    int shared;
    uint16_t *y;             // [T][2816]
};

constexpr int kCombineThreads = kH / 8;

__global__ void __launch_bounds__(kCombineThreads) k_combine(const CombineArgs p)
{
    tc::after_previous();
    tc::let_next_start();
    const int64_t t = blockIdx.x;
    const int k0 = threadIdx.x * 8;
    uint4 u[kK + 1];
    float f[kK + 1];
#pragma unroll
    for (int k = 0; k <= kK; ++k) {
        int at = -1, e = kE;
        float w = 1.0f;
        if (k < kK) {
            at = __ldcg(p.pos + t * kK + k);
            if (at >= 0) {
                e = __ldcg(p.ids + t * kK + k);
                w = __ldcg(p.w + t * kK + k);
            }
        } else if (p.shared) {
            at = __ldcg(p.offsets + kE) + static_cast<int>(t);
        }
        u[k] = make_uint4(0, 0, 0, 0);
        f[k] = 0.0f;
        if (at >= 0) {
            u[k] = __ldcg(reinterpret_cast<const uint4 *>(p.rows + static_cast<int64_t>(at) * kH + k0));
            f[k] = w * (__ldcg(p.sa + at) * (__ldcg(p.smax + e) * 4096.0f));
        }
    }
    float o[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
        o[q] = 0.0f;
#pragma unroll
    for (int k = 0; k <= kK; ++k) {
        const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w[q]));
            o[2 * q] = fmaf(f[k], v.x, o[2 * q]);
            o[2 * q + 1] = fmaf(f[k], v.y, o[2 * q + 1]);
        }
    }
    uint32_t r[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
        r[q] = f32_to_bf16(o[2 * q]) | static_cast<uint32_t>(f32_to_bf16(o[2 * q + 1])) << 16;
    *reinterpret_cast<uint4 *>(p.y + t * kH + k0) = make_uint4(r[0], r[1], r[2], r[3]);
}

}  // namespace rows
}  // namespace fgm
