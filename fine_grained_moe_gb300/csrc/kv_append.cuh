// Writing keys and values into the 8-bit cache (fgm_kv_append).
//
// Per (64-token block, kv head), K and V apart, with a = max |x| over the
// call's tokens in the block:
//   s_new = 2^ceil(log2(a / 448)),  s = kept tokens ? max(s_old, s_new) : s_new,
//   code = e4m3(x / s),  kept code = e4m3(e4m3(code) s_old / s).
// Every factor is a power of two, so each division is exact and a new code
// carries one rounding (half an E4M3 step, 2^-4 of the value).
//
// One CTA per (touched block, kv head, K or V): the block's scale needs all of
// its tokens, and 64 tokens x D are small enough to stay in registers between
// the maximum and the rounding, so the input is read once. K rows go out as
// they came in, 8 codes a lane; V is turned through shared memory, so that the
// cache's token-contiguous rows leave in 16-byte pieces.
//
// What bounds it: HBM, with the instructions close behind. The maximum is taken
// and the scale applied two elements at a time in bf16 form (17.7 -> about 9
// instructions an element; a prompt of 16,381 tokens, 8 heads of 256: 47.8 ->
// 35.8 us, 5.6 TB/s). A decode step's few tokens take a launch.
#pragma once

#include "common.cuh"

namespace fgm {
namespace kv {

constexpr int kBlock = FGM_KV_BLOCK;
constexpr float kE4m3Max = 448.0f;

struct Cache {
    uint8_t *k_q;
    float *k_s;
    uint8_t *v_q;
    float *v_s;
    int64_t n_blocks;
    int heads;
};

struct AppendArgs {
    Cache c;
    const uint16_t *k, *v;
    int64_t stride;          // elements between tokens of k, v
    int N;
    const int32_t *lens;
    const int32_t *table;    // NULL: block b * max_blocks + j
    int max_blocks;
    int32_t *status;
};

// A sequence's length, held to [0, max_blocks * 64].
__device__ __forceinline__ int clamp_len(int len, int max_blocks, int32_t *status, bool report)
{
    const int64_t top = static_cast<int64_t>(max_blocks) * kBlock;
    if (len >= 0 && len <= top)
        return len;
    if (report)
        atomicOr(status, FGM_STATUS_BAD_BLOCK);
    return len < 0 ? 0 : static_cast<int>(top);
}

// Physical block of a sequence's block j, -1 when the table names none.
__device__ __forceinline__ int64_t phys_block(const int32_t *table, int b, int j, int max_blocks, int64_t n_blocks)
{
    const int64_t at = static_cast<int64_t>(b) * max_blocks + j;
    const int64_t p = table ? __ldcg(table + at) : at;
    return p >= 0 && p < n_blocks ? p : -1;
}

// Smallest power of two s with a / s <= 448 (a = m 2^e with m in [1, 2); 448 =
// 1.75 * 2^8), at least 2^-60. a is finite and not negative.
__device__ __forceinline__ float pow2_scale(float a)
{
    const unsigned u = __float_as_uint(a);
    const int e = static_cast<int>(u >> 23) + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);   // biased
    return __uint_as_float(static_cast<unsigned>(max(e - 8, 127 - 60)) << 23);
}

__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d)
{
    const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Four codes times a power of two, rounded to codes again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f)
{
    float x[4];
    e4m3x4_to_f32(w, x);
    return to_e4m3x4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    uint32_t y;
    asm("max.u16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t w, __nv_bfloat162 f)
{
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&w), f);
    return *reinterpret_cast<const uint32_t *>(&y);
}

// Two bf16 with NaN replaced by 0; the finite ones' bits of |x| go into amax.
__device__ __forceinline__ uint32_t drop_nan(uint32_t w, unsigned &amax)
{
    const unsigned a0 = w & 0x7FFFu, a1 = (w >> 16) & 0x7FFFu;
    amax = max(amax, max(a0 < 0x7F80u ? a0 : 0u, a1 < 0x7F80u ? a1 : 0u));
    return (a0 > 0x7F80u ? 0u : w & 0xFFFFu) | (a1 > 0x7F80u ? 0u : w & 0xFFFF0000u);
}

// Bytes of `a` where the byte's slot is in [lo, hi), of `b` elsewhere; the
// word holds slots s .. s + 3.
__device__ __forceinline__ uint32_t pick4(uint32_t a, uint32_t b, int s, int lo, int hi)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m |= (s + i >= lo && s + i < hi) ? 0xFFu << (8 * i) : 0u;
    return (a & m) | (b & ~m);
}

template <int D>
struct Append {
    static constexpr int kThreads = D == 64 ? 128 : 256;
    static constexpr int kSlices = D / 64;                              // 64-wide slices of a token
    static constexpr int kItems = 4 * kSlices / (kThreads / 32);        // (4-slot group, 8-wide piece) a thread holds
    static constexpr int kRow = kBlock + 4;                             // bytes of a V row in shared memory
};

template <int D>
__global__ void __launch_bounds__(Append<D>::kThreads) k_kv_append(const AppendArgs p)
{
    using A = Append<D>;
    constexpr int kRow = A::kRow, kItems = A::kItems, kThreads = A::kThreads;
    __shared__ __align__(16) uint8_t vt[D * kRow];
    __shared__ float smax[kThreads / 32];
    const int tid = threadIdx.x, h = blockIdx.y >> 1, b = blockIdx.z;
    const bool is_v = blockIdx.y & 1;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int len0 = __ldcg(p.lens + b);
    const int len = clamp_len(len0, p.max_blocks, p.status, tid == 0 && blockIdx.x == 0 && blockIdx.y == 0);
    // the call's tokens are positions [start, len); start counts from the length as given
    const int64_t first = static_cast<int64_t>(len0) - p.N;
    const int start = first > 0 ? static_cast<int>(min(first, static_cast<int64_t>(len))) : 0;
    const int j = start / kBlock + blockIdx.x;
    if (static_cast<int64_t>(j) * kBlock >= len || start >= len)
        return;
    const int64_t phys = phys_block(p.table, b, j, p.max_blocks, p.c.n_blocks);
    if (phys < 0) {
        if (tid == 0)
            atomicOr(p.status, FGM_STATUS_BAD_BLOCK);
        return;
    }
    const int lo = max(start - j * kBlock, 0), hi = min(len - j * kBlock, kBlock);   // new slots
    const int n = hi - lo;
    const int64_t tok0 = static_cast<int64_t>(j) * kBlock + lo - first;              // their first token in the call
    const uint16_t *src = (is_v ? p.v : p.k) + (static_cast<int64_t>(b) * p.N + tok0) * p.stride + h * D;
    float *scale = (is_v ? p.c.v_s : p.c.k_s) + phys * p.c.heads + h;
    uint8_t *dst = (is_v ? p.c.v_q : p.c.k_q) + (phys * p.c.heads + h) * static_cast<int64_t>(kBlock * D);

    // A warp takes a 64-wide slice of 16 slots: lane = 8-wide piece (0..7) and
    // group of 4 slots (0..3), so that a row's loads and K's stores are whole
    // 128- and 64-byte pieces and a thread packs 4 slots of V into one word
    // (two lanes to a bank: rows are 17 words apart).
    const int piece = tid & 7;
    auto slice_of = [&](int i) { return ((tid >> 5) + i * (kThreads / 32)) % A::kSlices; };
    auto slot_of = [&](int i) { return ((tid >> 5) + i * (kThreads / 32)) / A::kSlices * 16 + ((tid >> 3) & 3) * 4; };
    uint4 x[kItems][4];
#pragma unroll
    for (int i = 0; i < kItems; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = slot_of(i) + r - lo;
            x[i][r] = make_uint4(0, 0, 0, 0);
            if (t >= 0 && t < n)
                x[i][r] = __ldcs(reinterpret_cast<const uint4 *>(src + t * p.stride + slice_of(i) * 64 + piece * 8));
        }
    // |x| as bf16 bits orders like the values, Inf and NaN above all others
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kItems; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint4 w = x[i][r];
            top = max_u16x2(max_u16x2(top, w.x & 0x7FFF7FFFu), w.y & 0x7FFF7FFFu);
            top = max_u16x2(max_u16x2(top, w.z & 0x7FFF7FFFu), w.w & 0x7FFF7FFFu);
        }
    unsigned amax = max(top & 0xFFFFu, top >> 16);
    if (amax >= 0x7F80u) {    // the finite ones' maximum; NaN becomes 0
        atomicOr(p.status, FGM_STATUS_NONFINITE_KV);
        amax = 0;
#pragma unroll
        for (int i = 0; i < kItems; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                x[i][r].x = drop_nan(x[i][r].x, amax);
                x[i][r].y = drop_nan(x[i][r].y, amax);
                x[i][r].z = drop_nan(x[i][r].z, amax);
                x[i][r].w = drop_nan(x[i][r].w, amax);
            }
    }
    amax = __reduce_max_sync(0xFFFFFFFFu, amax);
    if ((tid & 31) == 0)
        smax[tid >> 5] = __uint_as_float(amax << 16);
    const float old = lo > 0 ? *scale : 0.0f;
    __syncthreads();
    float a = 0.0f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w)
        a = fmaxf(a, smax[w]);
    const float fresh = pow2_scale(a);
    const float s = lo > 0 ? fmaxf(old, fresh) : fresh;
    const bool grow = lo > 0 && s > old;
    const float up = 1.0f / s;                    // a power of two, exact
    const float fk = grow ? old * up : 1.0f;
    // x / s in bf16 already: a power of two changes no bit of it that a code keeps
    const __nv_bfloat162 up2 = __float2bfloat162_rn(up);
    auto codes = [&](uint32_t w0, uint32_t w1) -> uint32_t {
        const float2 p0 = bf16x2_to_f32(mul_bf16x2(w0, up2)), p1 = bf16x2_to_f32(mul_bf16x2(w1, up2));
        return to_e4m3x4(p0.x, p0.y, p1.x, p1.y);
    };
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int slot = slot_of(i), slice = slice_of(i);
        if (slot + 4 <= lo || slot >= hi)
            continue;
        uint32_t q0[4], q1[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            q0[r] = codes(x[i][r].x, x[i][r].y);
            q1[r] = codes(x[i][r].z, x[i][r].w);
            if (!is_v && slot + r >= lo && slot + r < hi)
                *reinterpret_cast<uint2 *>(dst + slice * (kBlock * 64) + (slot + r) * 64 + piece * 8) = make_uint2(q0[r], q1[r]);
        }
        if (is_v) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint32_t *q = half ? q1 : q0;
                // 4 x 4 bytes turned: word k holds dim k of the four slots
                const uint32_t t0 = __byte_perm(q[0], q[1], 0x5140), t1 = __byte_perm(q[2], q[3], 0x5140);
                const uint32_t t2 = __byte_perm(q[0], q[1], 0x7362), t3 = __byte_perm(q[2], q[3], 0x7362);
                const uint32_t o[4] = {__byte_perm(t0, t1, 0x5410), __byte_perm(t0, t1, 0x7632),
                                       __byte_perm(t2, t3, 0x5410), __byte_perm(t2, t3, 0x7632)};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    *reinterpret_cast<uint32_t *>(vt + (slice * 64 + piece * 8 + half * 4 + k) * kRow + slot) = o[k];
            }
        }
    }
    if (!is_v) {
        if (grow)   // the kept tokens' rows, 16 codes at a time
            for (int e = tid; e < lo * (D / 16); e += kThreads) {
                const int c = e / (lo * 4), r = e % (lo * 4);
                uint4 *at = reinterpret_cast<uint4 *>(dst + c * (kBlock * 64) + r * 16);
                uint4 w = *at;
                w.x = rescale4(w.x, fk);
                w.y = rescale4(w.y, fk);
                w.z = rescale4(w.z, fk);
                w.w = rescale4(w.w, fk);
                *at = w;
            }
    } else {
        __syncthreads();
        // pieces of 16 slots from the first that changes to the last new one
        const int c0 = grow ? 0 : lo / 16, c1 = (hi + 15) / 16, nc = c1 - c0;
        for (int e = tid; e < D * nc; e += kThreads) {
            const int d = e / nc, s0 = (c0 + e % nc) * 16;
            uint4 *at = reinterpret_cast<uint4 *>(dst + d * kBlock + s0);
            const uint32_t *row = reinterpret_cast<const uint32_t *>(vt + d * kRow + s0);
            uint4 w = make_uint4(row[0], row[1], row[2], row[3]);
            if (s0 < lo || s0 + 16 > hi) {
                const uint4 o = *at;
                uint32_t nw[4] = {w.x, w.y, w.z, w.w};
                const uint32_t ow[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t kept = grow ? pick4(rescale4(ow[q], fk), ow[q], s0 + 4 * q, 0, lo) : ow[q];
                    nw[q] = pick4(nw[q], kept, s0 + 4 * q, lo, hi);
                }
                w = make_uint4(nw[0], nw[1], nw[2], nw[3]);
            }
            *at = w;
        }
    }
    if (tid == 0)
        *scale = s;
}

}  // namespace kv
}  // namespace fgm
