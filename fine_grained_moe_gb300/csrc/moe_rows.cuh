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
// by id: each chunk of slots is counted by a CTA (a router's by k_route_top); then each adds up the counts before
// it (of smaller ids, and of its own id in earlier chunks) and deals its slots, a
// warp a run of consecutive ones. From 33 chunks on a kernel between them adds up the
// counts once for all. No order of CTAs or atomics enters the result.

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

constexpr int kIdsAhead = 4;

__device__ __forceinline__ void load_ids(const GroupArgs &p, int64_t i, int64_t i1, int (&id)[kIdsAhead])
{
#pragma unroll
    for (int j = 0; j < kIdsAhead; ++j)
        id[j] = i + 32 * j < i1 ? __ldcg(p.ids + i + 32 * j) : -1;
}

// Counts of a warp's run of slots in its own row of hist; the run's first ids are in `head`.
__device__ __forceinline__ void count_run(const GroupArgs &p, int64_t i0, int64_t i1, const int (&head)[kIdsAhead], int *hist, int lane)
{
    for (int64_t i = i0; i < i1; i += 32 * kIdsAhead) {
        int id[kIdsAhead];
#pragma unroll
        for (int j = 0; j < kIdsAhead; ++j)
            id[j] = head[j];
        if (i > i0)
            load_ids(p, i + lane, i1, id);
#pragma unroll
        for (int j = 0; j < kIdsAhead; ++j) {
            const unsigned same = __match_any_sync(0xFFFFFFFFu, id[j]);
            if (id[j] >= 0 && id[j] < p.E && lane == __ffs(same) - 1)
                hist[id[j]] += __popc(same);
            __syncwarp();
        }
    }
}

__device__ __forceinline__ void run_of(const GroupArgs &p, int chunk, int warp, int64_t &i0, int64_t &i1)
{
    const int64_t each = p.chunk / kGroupWarps;
    i0 = static_cast<int64_t>(chunk) * p.chunk + warp * each;
    i1 = i0 + each < p.n ? i0 + each : p.n;
}

// Of chunk `chunk`, by a CTA; hist: shared, [kGroupWarps][E].
__device__ __forceinline__ void group_count(const GroupArgs &p, int chunk, int *hist)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t i0, i1;
    int head[kIdsAhead];
    run_of(p, chunk, warp, i0, i1);
    load_ids(p, i0 + lane, i1, head);
    for (int i = threadIdx.x; i < kGroupWarps * p.E; i += kGroupThreads)
        hist[i] = 0;
    __syncthreads();
    count_run(p, i0, i1, head, hist + warp * p.E, lane);
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kGroupThreads) {
        int s = 0;
        for (int w = 0; w < kGroupWarps; ++w)
            s += hist[w * p.E + e];
        p.count[static_cast<int64_t>(chunk) * p.E + e] = s;
    }
}

constexpr int kDirectChunks = 32;

// Counts to sums: count[c][e] becomes those of earlier chunks, offsets all of smaller experts; one CTA. (Each
// dealing CTA adding up 128 chunks for itself: 21 us for 131,048 slots, where the three kernels take 14.)
constexpr int kScanThreads = 1024;

__global__ void __launch_bounds__(kScanThreads) k_group_scan(const GroupArgs p)
{
    __shared__ int part_sum[kScanThreads], warp_sum[32];
    const int parts = kScanThreads / p.E, e = threadIdx.x % p.E, part = threadIdx.x / p.E, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = p.chunks * part / parts, c1 = p.chunks * (part + 1) / parts;
    int32_t *at = p.count + e;
    tc::after_previous();
    tc::let_next_start();
    int sum = 0;
    if (part < parts)
#pragma unroll 16
        for (int c = c0; c < c1; ++c)
            sum += __ldcg(at + static_cast<int64_t>(c) * p.E);
    part_sum[threadIdx.x] = sum;
    __syncthreads();
    int before = 0, all = 0;
    if (part < parts)
        for (int q = 0; q < parts; ++q) {
            const int v = part_sum[q * p.E + e];
            before += q < part ? v : 0;
            all += v;
        }
    if (part < parts)
        for (int c = c0; c < c1; c += 16) {
            int v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                v[i] = c + i < c1 ? __ldcg(at + static_cast<int64_t>(c + i) * p.E) : 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (c + i < c1)
                    at[static_cast<int64_t>(c + i) * p.E] = before;
                before += v[i];
            }
        }
    int mine = part == 0 ? all : 0, incl = mine; // (the first E threads have an expert each)
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        incl += lane >= o ? u : 0;
    }
    if (lane == 31)
        warp_sum[warp] = incl;
    __syncthreads();
    for (int w = 0; w < warp; ++w)
        incl += warp_sum[w];
    if (part == 0) {
        if (e == 0)
            p.offsets[0] = 0;
        p.offsets[e + 1] = incl;
        if (e == p.E - 1 && p.shared)
            p.offsets[p.E + 1] = incl + p.shared;
    }
}

// The same CTA's slots dealt; hist: [kGroupWarps][E], then [2][E] totals.
__device__ __forceinline__ void group_deal(const GroupArgs &p, int chunk, int *hist)
{
    __shared__ int warp_sum[kGroupWarps];
    int *total = hist + kGroupWarps * p.E;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t i0, i1;
    int head[kIdsAhead];
    run_of(p, chunk, warp, i0, i1);
    load_ids(p, i0 + lane, i1, head);
    for (int i = threadIdx.x; i < kGroupWarps * p.E; i += kGroupThreads)
        hist[i] = 0;
    __syncthreads();
    count_run(p, i0, i1, head, hist + warp * p.E, lane);
    __syncthreads();
    // slots of each expert in all chunks and in those before: threads share out the chunks where experts are few
    int *before = total + p.E;
    const int parts = p.E < kGroupThreads ? kGroupThreads / p.E : 1;
    const bool scanned = p.chunks > kDirectChunks;
    for (int e = threadIdx.x; e < p.E; e += kGroupThreads) {
        total[e] = scanned ? __ldcg(p.offsets + e) : 0;
        before[e] = scanned ? __ldcg(p.count + static_cast<int64_t>(chunk) * p.E + e) : 0;
    }
    __syncthreads();
    if (p.chunks > 1 && !scanned)
        for (int i = threadIdx.x; i < p.E * parts; i += kGroupThreads) {
            const int e = i % p.E, part = i / p.E;
            int sum = 0, sum_before = 0;
#pragma unroll 16
            for (int c = part; c < p.chunks; c += parts) {
                const int v = __ldcg(p.count + static_cast<int64_t>(c) * p.E + e);
                sum_before += c < chunk ? v : 0;
                sum += v;
            }
            atomicAdd(total + e, sum);
            atomicAdd(before + e, sum_before);
        }
    __syncthreads();
    // a warp's first place of each expert
    for (int e = threadIdx.x; e < p.E; e += kGroupThreads) {
        int mine = before[e];
        for (int w = 0; w < kGroupWarps; ++w) {
            const int v = hist[w * p.E + e];
            hist[w * p.E + e] = mine;
            mine += v;
        }
        if (p.chunks == 1)
            total[e] = mine;
    }
    __syncthreads();
    int all = scanned ? __ldcg(p.offsets + p.E) : 0;
    if (!scanned) {
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
            if (chunk == 0)
                p.offsets[e] = base;
            base += v;
        }
        for (int w = 0; w < kGroupWarps; ++w)
            all += warp_sum[w];
        if (chunk == 0 && threadIdx.x == 0) {
            p.offsets[p.E] = all;
            if (p.shared)
                p.offsets[p.E + 1] = all + p.shared;
        }
    }
    __syncthreads();
    int *at = hist + warp * p.E;
    for (int64_t i = i0; i < i1; i += 32 * kIdsAhead) {
        int ids[kIdsAhead];
#pragma unroll
        for (int j = 0; j < kIdsAhead; ++j)
            ids[j] = head[j];
        if (i > i0)
            load_ids(p, i + lane, i1, ids);
#pragma unroll
        for (int j = 0; j < kIdsAhead; ++j) {
            const int id = ids[j];
            const int64_t slot = i + 32 * j + lane;
            const unsigned same = __match_any_sync(0xFFFFFFFFu, id);
            const bool in = id >= 0 && id < p.E;
            int to = -1;
            if (in)
                to = total[id] + at[id] + __popc(same & ((1u << lane) - 1u));
            __syncwarp();
            if (in && lane == __ffs(same) - 1)
                at[id] += __popc(same);
            __syncwarp();
            if (slot < i1) {
                if (p.pos)
                    p.pos[slot] = to;
                if (in && p.order)
                    p.order[to] = static_cast<int32_t>(slot);
                if (in && p.src)
                    p.src[to] = static_cast<int32_t>(slot / p.per);
            }
        }
    }
    if (p.shared) {
        const int64_t t0 = static_cast<int64_t>(chunk) * p.chunk / p.per;
        for (int64_t t = t0 + threadIdx.x; t < t0 + p.chunk / p.per && t < p.shared; t += kGroupThreads)
            p.src[all + t] = static_cast<int32_t>(t);
    }
}

__global__ void __launch_bounds__(kGroupThreads) k_group_count(const GroupArgs p)
{
    extern __shared__ int hist[];
    tc::after_previous();
    tc::let_next_start();
    group_count(p, blockIdx.x, hist);
}

__global__ void __launch_bounds__(kGroupThreads) k_group_deal(const GroupArgs p)
{
    extern __shared__ int hist[];
    tc::after_previous();
    tc::let_next_start();
    group_deal(p, blockIdx.x, hist);
}

// ---------------------------------------------------------------- terms
//
// A row v[0 .. K) as two E4M3 terms under a power of two s that puts its largest
// element into [128, 256): t1 = e4m3(v / s), t2 = e4m3(v / s - t1), in blocks of 32
// elements, t1's and then t2's, so that one copy of 128 bytes brings both. K is
// filled up with zeros to a multiple of 32. |v - s (t1 + t2)| is at most 2^-9 |v| or
// 2^-10 s, whichever is larger; of a bf16 number it is 0 or at most 2^-10 s. A row
// with an element that is not finite has s = NaN. Bound by HBM: 147,429 rows of 704 take 62
// us, 6.7 TB/s; a few rows, all of whose elements are on their way at once, 4 us.

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

constexpr int kTermThreads = 256;
constexpr int kTermHeld = 4;                     // vectors of 8 that a thread holds (longer rows are read twice)

// Threads of a row: a warp up to 1,024 elements, else four.
__host__ __device__ __forceinline__ int term_row(int K) { return K <= 32 * 8 * kTermHeld ? 32 : 128; }

struct TermArgs {
    const uint16_t *x;       // bf16 rows of K, `stride` apart
    int64_t stride, n;
    int K;
    uint8_t *terms;          // [n][2 K rounded up to 32]
    float *scale;            // [n]
};

// Eight or two rows of bf16, the CTA's `part`th of them. All of a row is on its way
// before its largest element is known.
template <int kTermRow>
__device__ __forceinline__ void row_terms(const TermArgs &p, int64_t part)
{
    __shared__ uint32_t most[kTermThreads / 32];
    const int t = threadIdx.x % kTermRow, warp = threadIdx.x >> 5, K32 = (p.K + 31) & ~31;
    const int64_t row = part * (kTermThreads / kTermRow) + threadIdx.x / kTermRow;
    const uint16_t *xr = p.x + row * p.stride;
    uint4 u[kTermHeld];
    uint32_t m = 0;
    auto largest = [&](const uint4 &v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 4; ++q)
            m = max(m, max(w[q] & 0x7FFFu, w[q] >> 16 & 0x7FFFu));
    };
    auto take = [&](int k) { return row < p.n && k < p.K ? __ldcg(reinterpret_cast<const uint4 *>(xr + k)) : make_uint4(0, 0, 0, 0); };
#pragma unroll
    for (int i = 0; i < kTermHeld; ++i)
        u[i] = take((i * kTermRow + t) * 8);
#pragma unroll
    for (int i = 0; i < kTermHeld; ++i)
        largest(u[i]);
    for (int k = (kTermHeld * kTermRow + t) * 8; k < p.K; k += kTermRow * 8)
        largest(take(k));
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if (kTermRow > 32) {
        if ((threadIdx.x & 31) == 0)
            most[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kTermRow / 32; ++w)
            m = max(m, most[(warp & ~(kTermRow / 32 - 1)) + w]);
    }
    if (row >= p.n)
        return;
    int e = static_cast<int>(m >> 7);
    e = e < 14 ? 14 : e;
    if (t == 0)
        p.scale[row] = row_scale(e);
    const float up = __int_as_float((261 - e) << 23);         // 1 / s (e = 255: whatever it is, s is NaN)
    uint8_t *to = p.terms + row * (2 * static_cast<int64_t>(K32));
    auto write = [&](const uint4 &x, int k) {
        float v[8];
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 f = bf16x2_to_f32(w[q]);
            v[2 * q] = f.x * up;
            v[2 * q + 1] = f.y * up;
        }
        write_terms(to, k, v);
    };
#pragma unroll
    for (int i = 0; i < kTermHeld; ++i)
        if ((i * kTermRow + t) * 8 < K32)
            write(u[i], (i * kTermRow + t) * 8);
    for (int k = (kTermHeld * kTermRow + t) * 8; k < K32; k += kTermRow * 8)
        write(take(k), k);
}

__global__ void __launch_bounds__(kTermThreads) k_terms(const TermArgs p)
{
    tc::after_previous();
    tc::let_next_start();
    if (term_row(p.K) == 32)
        row_terms<32>(p, blockIdx.x);
    else
        row_terms<128>(p, blockIdx.x);
}

// Rows of the gated activations (grouped.cuh: f16 under a power of two per 32), a
// warp each; only those of some expert.
__global__ void __launch_bounds__(kTermThreads) k_act_terms(const uint16_t *act, const uint8_t *exps, const int32_t *n, int64_t most,
                                                            uint8_t *terms, float *scale)
{
    constexpr int kBlocks = kF / 32, kMine = (kF / 8 + 31) / 32;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kTermThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    tc::after_previous();
    tc::let_next_start();
    if (row >= most)
        return;
    const int rows = __ldcg(n);                  // (known when the row's values are: they are there, whatever they are)
    const int mine = lane < kBlocks ? __ldcg(exps + row * kBlocks + lane) : 0;
    uint4 u[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i)
        u[i] = i * 32 + lane < kF / 8 ? __ldcg(reinterpret_cast<const uint4 *>(act + row * kF) + i * 32 + lane) : make_uint4(0, 0, 0, 0);
    if (row >= rows)
        return;
    const int e = __reduce_max_sync(0xFFFFFFFFu, mine);
    if (lane == 0)
        scale[row] = row_scale(e);
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int at = i * 32 + lane, eb = __shfl_sync(0xFFFFFFFFu, mine, at >> 2);
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
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
        if (at < kF / 8)
            write_terms(terms + row * (2 * kF), at * 8, v);
    }
}

// A power of two that is not below any of an expert's n scales (their absolute values), 1 for none; by a CTA.
__device__ __forceinline__ void scale_max(const float *s, int n, float *smax, int e)
{
    __shared__ uint32_t part[8];
    uint32_t m = 0;
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += 256)
        m = max(m, __float_as_uint(__ldcg(s + static_cast<int64_t>(e) * n + i)) & 0x7FFFFFFFu);
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 8; ++w)
            m = max(m, part[w]);
        // (of scales beyond 2^126, infinite or NaN ones 2^127: what they give shows in the products)
        const uint32_t b = (m >> 23) + 1;
        smax[e] = m == 0 ? 1.0f : __uint_as_float((b > 254 ? 254 : b) << 23);
    }
}

// What the experts' products wait for, side by side: slots grouped (or counted, where
// they take several CTAs), x as terms, the experts' largest down scales.
struct PrepArgs {
    GroupArgs group;
    TermArgs terms;
    const float *down_s;
    float *smax;
};

__global__ void __launch_bounds__(256) k_prep(const PrepArgs p)
{
    extern __shared__ int hist[];
    static_assert(kGroupThreads == 256 && kTermThreads == 256, "one block size");
    tc::after_previous();
    tc::let_next_start();
    int b = blockIdx.x;
    if (b < p.group.chunks) {
        if (p.group.chunks == 1)
            group_deal(p.group, 0, hist);
        else
            group_count(p.group, b, hist);
    } else if ((b -= p.group.chunks) < kNE) {
        scale_max(p.down_s, kH, p.smax, b);
    } else {
        row_terms<128>(p.terms, b - kNE);
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
    int64_t T;
    uint16_t *y;             // [T][2816]
    int32_t *status;
    long long timeout_ns;
};

// A CTA takes tokens in turn, four at a time on their way: four warps each bring a
// token's rows, nine copies of 5,632 bytes (one warp for all was bound by the two loads
// that lead to a row's place: 253 us for 16,381 tokens, now 135, 6.8 TB/s), and two teams
// of others add them up by turns.
constexpr int kCombineTeam = kH / 8;
constexpr int kCombineTeams = 2;
constexpr int kCombineStages = 4;
constexpr int kCombineThreads = kCombineTeams * kCombineTeam + 32 * kCombineStages;
constexpr int kCombineStage = (kK + 1) * 2 * kH;
constexpr int kCombineSmem = kCombineStages * kCombineStage + 128;

__global__ void __launch_bounds__(kCombineThreads, 1) k_combine(const CombineArgs p)
{
    extern __shared__ uint8_t dsm_raw[];
    __shared__ unsigned long long full[kCombineStages], empty[kCombineStages];
    __shared__ float factor[kCombineStages][kK + 1];
    __shared__ uint32_t present[kCombineStages];
    __shared__ int abort_;
    const uint32_t ring = (tc::saddr(dsm_raw) + 127u) & ~127u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kCombineStages; ++i) {
            tc::bar_init(&full[i], 2);           // the copies' bytes, and the factors
            tc::bar_init(&empty[i], kCombineTeam / 32);
        }
        abort_ = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    tc::after_previous();
    tc::let_next_start();
    const tc::Waiter wait{&abort_, p.status, p.timeout_ns};
    uint32_t n = 0;                              // round of a stage, then the CTA's n-th token
    if (warp >= kCombineTeams * kCombineTeam / 32) {
        const int slot = warp - kCombineTeams * kCombineTeam / 32;
        bool ok = true;
        for (int64_t t = blockIdx.x + static_cast<int64_t>(slot) * gridDim.x; t < p.T; t += static_cast<int64_t>(kCombineStages) * gridDim.x, ++n) {
            // lane k: choice k's row, and what its elements are multiplied by; lane 8: the shared expert's
            int at = -1, e = kE;
            float w = 1.0f;
            if (lane < kK) {
                at = __ldcg(p.pos + t * kK + lane);
                e = __ldcg(p.ids + t * kK + lane);
                w = __ldcg(p.w + t * kK + lane);
            } else if (lane == kK && p.shared) {
                at = __ldcg(p.offsets + kE) + static_cast<int>(t);
            }
            const uint32_t rows_of = __ballot_sync(0xFFFFFFFFu, at >= 0), bar = tc::saddr(&full[slot]);
            if (n)
                ok = wait(&empty[slot], n - 1, 44, static_cast<int>(t));
            if (!(ok = __all_sync(0xFFFFFFFFu, ok)))
                break;
            if (lane == 0)
                tc::bar_expect(bar, __popc(rows_of) * 2 * kH);
            __syncwarp();
            if (at >= 0)
                asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                 ring + slot * kCombineStage + lane * 2 * kH),
                             "l"(reinterpret_cast<uint64_t>(p.rows + static_cast<int64_t>(at) * kH)), "r"(2 * kH), "r"(bar)
                             : "memory");
            if (lane <= kK)
                factor[slot][lane] = at >= 0 ? w * (__ldcg(p.sa + at) * __ldcg(p.smax + e) * 4096.0f) : 0.0f;
            if (lane == 0)
                present[slot] = rows_of;         // (without a row a place of the ring holds anything)
            __syncwarp();
            if (lane == 0)
                tc::bar_arrive(bar);
        }
        if (n)                                   // the last copies land before the CTA ends
            tc::bar_drain(tc::saddr(&full[slot]), (n - 1) & 1);
        return;
    }
    const int team = threadIdx.x / kCombineTeam, at = threadIdx.x - team * kCombineTeam;
    n = team;
    for (int64_t t = blockIdx.x + static_cast<int64_t>(team) * gridDim.x; t < p.T; t += static_cast<int64_t>(kCombineTeams) * gridDim.x, n += kCombineTeams) {
        const uint32_t slot = n % kCombineStages;
        if (!__all_sync(0xFFFFFFFFu, wait(&full[slot], n / kCombineStages, 45, static_cast<int>(t))))
            break;
        const uint32_t rows_of = present[slot];
        uint32_t w[kK + 1][4];
#pragma unroll
        for (int k = 0; k <= kK; ++k)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[k][0]), "=r"(w[k][1]), "=r"(w[k][2]), "=r"(w[k][3])
                         : "r"(ring + slot * kCombineStage + k * 2 * kH + at * 16)
                         : "memory");
        float o[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
            o[q] = 0.0f;
#pragma unroll
        for (int k = 0; k <= kK; ++k) {
            const float f = factor[slot][k];
            const bool in = rows_of >> k & 1;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t x = in ? w[k][q] : 0u;
                const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&x));
                o[2 * q] = fmaf(f, v.x, o[2 * q]);
                o[2 * q + 1] = fmaf(f, v.y, o[2 * q + 1]);
            }
        }
        __syncwarp();
        if (lane == 0)
            tc::bar_arrive(tc::saddr(&empty[slot]));
        uint32_t r[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            r[q] = f32_to_bf16(o[2 * q]) | static_cast<uint32_t>(f32_to_bf16(o[2 * q + 1])) << 16;
        *reinterpret_cast<uint4 *>(p.y + t * kH + at * 8) = make_uint4(r[0], r[1], r[2], r[3]);
    }
}

}  // namespace rows
}  // namespace fgm
