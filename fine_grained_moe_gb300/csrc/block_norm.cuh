// The norms around a block (fgm_block_norm):
//   h' = a h + b gate * post(y),   xn = pre(h'),
//   post(y) = y / sqrt(mean(y^2) + eps) * (post_gain + offset), pre(h') alike.
//
// 10 operations an element: bound by HBM. One pass: a row's y and h are read once, both
// norms' sums are taken in registers, and h' and xn written once. Sums and h' itself are
// fp32; xn goes by the fp32 h', not by the rounded one that is stored.
//
// Each row waits for two sums in turn, so the memory is kept busy by the rows behind it:
// a CTA owns a row at a time and walks through many, the gains stay in its shared memory,
// and each thread copies its own pieces of the next two rows there meanwhile
// (cp.async; nobody else reads them). There are as many threads as a row has eights of
// elements, or a multiple of a warp above that. 16,381 bf16 rows of 2,816 take 68 us, 5.4 TB/s; with a
// CTA a row and nothing ahead 152 us. Rows that do not allow 16-byte accesses go element by
// element, the next one's in registers.
#pragma once

#include <type_traits>

#include "tensor.cuh"

namespace fgm {
namespace norm {

struct Rows {
    void *p;                 // NULL: absent
    int64_t stride;          // elements between rows
    int type;                // FGM_F32, FGM_BF16 or FGM_F16
    int step;                // elements between columns: 1, or 0 (one value a row)
};

struct Args {
    Rows h, y, gate, h_out, xn;
    const void *post, *pre;  // [D] gains, NULL: 1
    int gain_type;
    int64_t N;
    int D;
    int post_norm;
    int keep;                // gains in shared memory (else, where they do not fit, read with every row)
    float a, b, offset, eps;
    float per_d;             // 1 / D
};

template <int VEC>
__device__ __forceinline__ void load(const void *p, int type, int64_t i, float (&v)[VEC])
{
    if constexpr (VEC == 8) {
        if (type == FGM_F32) {
            const float4 a = __ldcg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i)),
                         b = __ldcg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i) + 1);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            const uint4 u = __ldcg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i));
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 f = type == FGM_BF16 ? bf16x2_to_f32(w[q]) : __half22float2(*reinterpret_cast<const __half2 *>(&w[q]));
                v[2 * q] = f.x;
                v[2 * q + 1] = f.y;
            }
        }
    } else {
        if (type == FGM_F32) {
            v[0] = __ldcg(static_cast<const float *>(p) + i);
        } else {
            const uint16_t u = __ldcg(static_cast<const uint16_t *>(p) + i);
            v[0] = type == FGM_BF16 ? bf16_to_f32(u) : __half2float(__ushort_as_half(u));
        }
    }
}

__device__ __forceinline__ uint32_t narrow2(float a, float b, int type)
{
    if (type == FGM_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint16_t narrow(float v, int type) { return type == FGM_BF16 ? f32_to_bf16(v) : __half_as_ushort(__float2half_rn(v)); }

template <int VEC>
__device__ __forceinline__ void store(void *p, int type, int64_t i, const float (&v)[VEC])
{
    if constexpr (VEC == 8) {
        if (type == FGM_F32) {
            float4 *to = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
            to[0] = make_float4(v[0], v[1], v[2], v[3]);
            to[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                w[q] = narrow2(v[2 * q], v[2 * q + 1], type);
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
        if (type == FGM_F32)
            static_cast<float *>(p)[i] = v[0];
        else
            static_cast<uint16_t *>(p)[i] = narrow(v[0], type);
    }
}

// Sum over a row's threads, all of the CTA's, the same order and so the same bits in each.
__device__ __forceinline__ float row_sum(float v, float *part)
{
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    v = warp_sum(v);
    if (warps == 1)
        return v;
    if (lane == 0)
        part[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < warps ? part[lane] : 0.0f);
}

// Gains plus their offset to shared memory as fp32, post's and then pre's.
__device__ __forceinline__ void keep_gains(const Args &p, float *g)
{
    if (!p.keep)
        return;
    for (int which = 0; which < 2; ++which) {
        const void *from = which ? p.pre : p.post;
        if (from)
            for (int d = threadIdx.x; d < p.D; d += blockDim.x) {
                float v[1];
                load<1>(from, p.gain_type, d, v);
                g[which * p.D + d] = v[0] + p.offset;
            }
    }
}

// VEC gains from d on.
template <int VEC>
__device__ __forceinline__ void gain(const Args &p, const float *gains, int which, int d, float (&g)[VEC])
{
    if (p.keep) {
        if constexpr (VEC == 8) {                // (D is a multiple of 8, too)
            const float4 a = *reinterpret_cast<const float4 *>(gains + which * p.D + d), b = *reinterpret_cast<const float4 *>(gains + which * p.D + d + 4);
            g[0] = a.x, g[1] = a.y, g[2] = a.z, g[3] = a.w, g[4] = b.x, g[5] = b.y, g[6] = b.z, g[7] = b.w;
        } else {
            g[0] = gains[which * p.D + d];
        }
    } else {
        load<VEC>(which ? p.pre : p.post, p.gain_type, d, g);
#pragma unroll
        for (int q = 0; q < VEC; ++q)
            g[q] += p.offset;
    }
}

// One row: y, h and, where it has an element each, the gate in registers (fp32); `one`: its
// gate where that is a value a row. VPT vectors of VEC elements a thread.
template <int VPT, int VEC>
__device__ __forceinline__ void one_row(const Args &p, int64_t row, float (&y)[VPT][VEC], float (&h)[VPT][VEC], float (&gate)[VPT][VEC], float one,
                                        const float *gains, float (*part)[32])
{
    const int t = threadIdx.x, TPR = blockDim.x;
    if (p.y.p) {
        float r = p.b * one;
        if (p.post_norm) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int q = 0; q < VEC; ++q)
                    s = fmaf(y[i][q], y[i][q], s);
            r *= rsqrtf(row_sum(s, part[0]) * p.per_d + p.eps);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int d = (i * TPR + t) * VEC;
            if (p.post && d < p.D) {
                float g[VEC];
                gain<VEC>(p, gains, 0, d, g);
#pragma unroll
                for (int q = 0; q < VEC; ++q)
                    y[i][q] *= g[q];
            }
#pragma unroll
            for (int q = 0; q < VEC; ++q) {
                if (p.gate.p && p.gate.step)
                    y[i][q] *= gate[i][q];
                h[i][q] = fmaf(r, y[i][q], p.a * h[i][q]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int q = 0; q < VEC; ++q)
                h[i][q] *= p.a;
    }
    if (p.h_out.p)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int d = (i * TPR + t) * VEC;
            if (d < p.D)
                store<VEC>(p.h_out.p, p.h.type, row * p.h_out.stride + d, h[i]);
        }
    if (!p.xn.p)
        return;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int q = 0; q < VEC; ++q)
            s = fmaf(h[i][q], h[i][q], s);
    const float r = rsqrtf(row_sum(s, part[1]) * p.per_d + p.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int d = (i * TPR + t) * VEC;
        if (d < p.D) {
            float g[VEC];
            if (p.pre)
                gain<VEC>(p, gains, 1, d, g);
#pragma unroll
            for (int q = 0; q < VEC; ++q)
                g[q] = p.pre ? g[q] * (h[i][q] * r) : h[i][q] * r;
            store<VEC>(p.xn.p, p.xn.type, row * p.xn.stride + d, g);
        }
    }
}

// A value a row of the gate, else 1; a gate of one row for all of them (stride 0) is one, too.
__device__ __forceinline__ float row_gate(const Args &p, int64_t row)
{
    float one[1] = {1.0f};
    if (p.gate.p && !p.gate.step)
        load<1>(p.gate.p, p.gate.type, row * p.gate.stride, one);
    return one[0];
}

// Bytes of a row's pieces of a tensor in shared memory: padded to whole vectors of all threads.
__host__ __device__ __forceinline__ int piece_bytes(const Rows &r, int type, int vectors) { return r.p && r.step ? vectors * 8 * (type == FGM_F32 ? 4 : 2) : 0; }

// Rows of 16-byte accesses; STAGES rows in shared memory, the current one and those ahead. (Beyond 8,192 elements
// its 1,024 threads' two vectors each spill some 200 bytes: 8,191 bf16 rows of 8,200 167 us, of 8,192 the same.)
template <int VPT, int STAGES>
__global__ void __launch_bounds__(1024) k_block_norm(const Args p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float part[2][32];
    const int t = threadIdx.x, TPR = blockDim.x;
    const int yb = piece_bytes(p.y, p.y.type, TPR * VPT), hb = piece_bytes(p.h, p.h.type, TPR * VPT),
              gb = piece_bytes(p.gate, p.gate.type, TPR * VPT), stage = yb + hb + gb;
    float *gains = reinterpret_cast<float *>(smem + STAGES * stage);
    tc::after_previous();
    tc::let_next_start();
    // this thread's pieces of a row: vector i at (i * TPR + t) * its bytes
    auto bring = [&](const Rows &r, int type, int64_t row, uint32_t to) {
        const int size = type == FGM_F32 ? 4 : 2;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * TPR + t;
            if (v * 8 < p.D) {
                const uint8_t *from = static_cast<const uint8_t *>(r.p) + (row * r.stride + v * 8) * size;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + v * 8 * size), "l"(from) : "memory");
                if (size == 4)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + v * 32 + 16), "l"(from + 16) : "memory");
            }
        }
    };
    auto ahead = [&](int64_t row, int slot) {
        if (row < p.N) {
            const uint32_t to = tc::saddr(smem) + slot * stage;
            if (yb)
                bring(p.y, p.y.type, row, to);
            bring(p.h, p.h.type, row, to + yb);
            if (gb)
                bring(p.gate, p.gate.type, row, to + yb + hb);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto take = [&](int type, const uint8_t *from, float (&v)[VPT][8]) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int at = i * TPR + t;
#pragma unroll
            for (int q = 0; q < 8; ++q)
                v[i][q] = 0.0f;
            if (at * 8 >= p.D)
                continue;
            if (type == FGM_F32) {
                const float4 a = reinterpret_cast<const float4 *>(from)[2 * at], b = reinterpret_cast<const float4 *>(from)[2 * at + 1];
                v[i][0] = a.x, v[i][1] = a.y, v[i][2] = a.z, v[i][3] = a.w, v[i][4] = b.x, v[i][5] = b.y, v[i][6] = b.z, v[i][7] = b.w;
            } else {
                const uint4 u = reinterpret_cast<const uint4 *>(from)[at];
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float2 f = type == FGM_BF16 ? bf16x2_to_f32(w[q]) : __half22float2(*reinterpret_cast<const __half2 *>(&w[q]));
                    v[i][2 * q] = f.x;
                    v[i][2 * q + 1] = f.y;
                }
            }
        }
    };
    int64_t next = blockIdx.x;
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i, next += gridDim.x)
        ahead(next, i);
    keep_gains(p, gains);
    __syncthreads();
    int slot = 0;
    for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x, next += gridDim.x) {
        const float one = row_gate(p, row);
        ahead(next, slot + STAGES - 1 < STAGES ? slot + STAGES - 1 : slot - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
        float y[VPT][8], h[VPT][8], g[VPT][8];
        const uint8_t *at = smem + slot * stage;
        if (yb)
            take(p.y.type, at, y);
        take(p.h.type, at + yb, h);
        if (gb)
            take(p.gate.type, at + yb + hb, g);
        slot = slot + 1 < STAGES ? slot + 1 : 0;
        one_row<VPT, 8>(p, row, y, h, g, one, gains, part);
        if (!(p.post_norm && p.y.p && p.xn.p))   // (the barriers of two sums keep rows apart; without one of them this does)
            __syncthreads();
    }
}

// ---------------------------------------------------------------- the usual rows
//
// bf16 y and xn, bf16 or fp32 h, no gate of an element each, up to 512 eights of elements (a sum's
// warps are 16 at most): a vector a thread. The general kernel above spends 490 instructions a warp and row, most of
// them on types and options (16,381 rows of 2,816: 114 us, issue-bound); this one has the
// types built in, addresses that advance, and two fp32 operations to an instruction. 16,381 bf16
// rows of 3,080 take 82 us here and 153 there, of 4,096 102 and 170.

__device__ __forceinline__ uint64_t pair(float a, float b) { return static_cast<uint64_t>(__float_as_uint(a)) | static_cast<uint64_t>(__float_as_uint(b)) << 32; }
__device__ __forceinline__ float low(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float high(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }

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

__device__ __forceinline__ float square_sum(const uint64_t (&v)[4])
{
    uint64_t s = mul2(v[0], v[0]);
#pragma unroll
    for (int q = 1; q < 4; ++q)
        s = fma2(v[q], v[q], s);
    return low(s) + high(s);
}

// Sum over a CTA of at most 16 warps.
__device__ __forceinline__ float sum16(float v, float *part, int lane, int warps)
{
    v = warp_sum(v);
    if (lane == 0)
        part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (lane & 15) < warps ? part[lane & 15] : 0.0f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Eight values of a bf16 (16 bytes) or fp32 (32 bytes) vector from shared memory.
template <bool F32>
__device__ __forceinline__ void take8(uint32_t at, uint64_t (&v)[4])
{
    uint32_t w[8];
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
    if (F32) {
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]) : "r"(at + 16) : "memory");
#pragma unroll
        for (int q = 0; q < 4; ++q)
            v[q] = static_cast<uint64_t>(w[2 * q]) | static_cast<uint64_t>(w[2 * q + 1]) << 32;
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            v[q] = static_cast<uint64_t>(w[q] << 16) | static_cast<uint64_t>(w[q] & 0xFFFF0000u) << 32;
    }
}

template <bool F32>
__device__ __forceinline__ void give8(uint8_t *to, const uint64_t (&v)[4])
{
    if (F32) {
        reinterpret_cast<float4 *>(to)[0] = make_float4(low(v[0]), high(v[0]), low(v[1]), high(v[1]));
        reinterpret_cast<float4 *>(to)[1] = make_float4(low(v[2]), high(v[2]), low(v[3]), high(v[3]));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            w[q] = narrow2(low(v[q]), high(v[q]), FGM_BF16);
        *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

constexpr int kUsualThreads = 512;               // at most
constexpr int kUsualStages = 3;

// F32: h. The gate is one value a row, or a channel's, which joins post's gain.
template <bool F32>
__global__ void __launch_bounds__(kUsualThreads, 3) k_block_norm_usual(const Args p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float part[2][16];
    constexpr int kHBytes = F32 ? 32 : 16;
    const int t = threadIdx.x, lane = t & 31, TPR = blockDim.x, warps = TPR >> 5, d = t * 8;
    const bool in = d < p.D, channel_gate = p.gate.p && p.gate.step, row_gated = p.gate.p && !p.gate.step, scaled = p.post || channel_gate,
               sums = p.post_norm && p.y.p, both = sums && p.xn.p;
    const int stage = (16 + kHBytes) * TPR;
    const uint32_t mine = tc::saddr(smem) + t * 16, mine_h = tc::saddr(smem) + 16 * TPR + t * kHBytes;
    float4 *gains = reinterpret_cast<float4 *>(smem + kUsualStages * stage) + t;     // [post, pre][halves of eight][threads]
    tc::after_previous();
    tc::let_next_start();
    const uint8_t *y_from = static_cast<const uint8_t *>(p.y.p) + (blockIdx.x * p.y.stride + d) * 2,
                  *h_from = static_cast<const uint8_t *>(p.h.p) + (blockIdx.x * p.h.stride + d) * (kHBytes / 8);
    const int64_t y_step = gridDim.x * p.y.stride * 2, h_step = gridDim.x * p.h.stride * (kHBytes / 8);
    int64_t next = blockIdx.x;
    auto ahead = [&](uint32_t slot) {
        if (next < p.N && in) {
            if (p.y.p)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(mine + slot), "l"(y_from) : "memory");
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(mine_h + slot), "l"(h_from) : "memory");
            if (F32)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(mine_h + slot + 16), "l"(h_from + 16) : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        next += gridDim.x;
        y_from += y_step;
        h_from += h_step;
    };
#pragma unroll
    for (int i = 0; i < kUsualStages - 1; ++i)
        ahead(i * stage);
    if (in) {
        float g[8], c[8];
        if (scaled) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                g[q] = 1.0f;
            if (p.post) {
                load<8>(p.post, p.gain_type, d, g);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    g[q] += p.offset;
            }
            if (channel_gate) {
                load<8>(p.gate.p, p.gate.type, d, c);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    g[q] *= c[q];
            }
            gains[0] = make_float4(g[0], g[1], g[2], g[3]);
            gains[TPR] = make_float4(g[4], g[5], g[6], g[7]);
        }
        if (p.pre) {
            load<8>(p.pre, p.gain_type, d, g);
            gains[2 * TPR] = make_float4(g[0] + p.offset, g[1] + p.offset, g[2] + p.offset, g[3] + p.offset);
            gains[3 * TPR] = make_float4(g[4] + p.offset, g[5] + p.offset, g[6] + p.offset, g[7] + p.offset);
        }
    }
    auto times_gain = [&](const float4 *at, uint64_t (&v)[4]) {
        const float4 a = at[0], b = at[TPR];
        v[0] = mul2(v[0], pair(a.x, a.y));
        v[1] = mul2(v[1], pair(a.z, a.w));
        v[2] = mul2(v[2], pair(b.x, b.y));
        v[3] = mul2(v[3], pair(b.z, b.w));
    };
    const uint64_t a2 = pair(p.a, p.a);
    uint8_t *h_to = static_cast<uint8_t *>(p.h_out.p) + (blockIdx.x * p.h_out.stride + d) * (kHBytes / 8),
            *n_to = static_cast<uint8_t *>(p.xn.p) + (blockIdx.x * p.xn.stride + d) * 2;
    const int64_t ho_step = gridDim.x * p.h_out.stride * (kHBytes / 8), n_step = gridDim.x * p.xn.stride * 2;
    uint32_t slot = 0;
    for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x) {
        float r = p.b;
        if (row_gated)
            r *= row_gate(p, row);
        ahead(slot ? slot - stage : (kUsualStages - 1) * stage);
        asm volatile("cp.async.wait_group %0;" ::"n"(kUsualStages - 1) : "memory");
        uint64_t y[4] = {0, 0, 0, 0}, h[4] = {0, 0, 0, 0};
        if (in) {
            if (p.y.p)
                take8<false>(mine + slot, y);
            take8<F32>(mine_h + slot, h);
        }
        slot = slot == (kUsualStages - 1) * stage ? 0 : slot + stage;
        if (sums)
            r *= rsqrtf(sum16(square_sum(y), part[0], lane, warps) * p.per_d + p.eps);
        if (scaled && in)
            times_gain(gains, y);
        const uint64_t r2 = pair(r, r);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            h[q] = mul2(a2, h[q]);
        if (p.y.p)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                h[q] = fma2(r2, y[q], h[q]);
        if (p.h_out.p && in)
            give8<F32>(h_to, h);
        if (p.xn.p) {
            const float n = rsqrtf(sum16(square_sum(h), part[1], lane, warps) * p.per_d + p.eps);
            const uint64_t n2 = pair(n, n);
            if (in) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    h[q] = mul2(h[q], n2);
                if (p.pre)
                    times_gain(gains + 2 * TPR, h);
                give8<false>(n_to, h);
            }
        }
        h_to += ho_step;
        n_to += n_step;
        if (!both)                               // (the barriers of two sums keep rows apart; without one of them this does)
            __syncthreads();
    }
}

// ---------------------------------------------------------------- the usual types, rows of any alignment
//
// Four elements a thread, blockDim.x apart; their gains stay in registers, the next row's
// values are on their way as they are. (The kernel below issues 187 instructions an
// element on these types, this one 50: 4,099 rows of 1,409 with a gate 55 us and 22.)
constexpr int kOddVals = 4;

template <bool F32, bool GATE>
__global__ void __launch_bounds__(1024) k_block_norm_odd(const Args p)
{
    __shared__ float part[2][32];
    using HT = typename std::conditional<F32, float, uint16_t>::type;
    const int t = threadIdx.x, TPR = blockDim.x;
    const bool channel_gate = !GATE && p.gate.p && p.gate.step, row_gated = p.gate.p && !p.gate.step, sums = p.post_norm && p.y.p,
               both = sums && p.xn.p;
    tc::after_previous();
    tc::let_next_start();
    const uint16_t *y = static_cast<const uint16_t *>(p.y.p) + blockIdx.x * p.y.stride + t,
                   *g = static_cast<const uint16_t *>(p.gate.p) + blockIdx.x * p.gate.stride + t;
    const HT *h = static_cast<const HT *>(p.h.p) + blockIdx.x * p.h.stride + t;
    HT *ho = static_cast<HT *>(p.h_out.p) + blockIdx.x * p.h_out.stride + t;
    uint16_t *xn = static_cast<uint16_t *>(p.xn.p) + blockIdx.x * p.xn.stride + t;
    const int64_t y_step = gridDim.x * p.y.stride, g_step = gridDim.x * p.gate.stride, h_step = gridDim.x * p.h.stride,
                  ho_step = gridDim.x * p.h_out.stride, n_step = gridDim.x * p.xn.stride;
    bool in[kOddVals];
    float post[kOddVals], pre[kOddVals];
    uint32_t yr[kOddVals], gr[kOddVals], hr[kOddVals];
#pragma unroll
    for (int i = 0; i < kOddVals; ++i) {
        const int d = i * TPR + t;
        in[i] = d < p.D;
        float v[1];
        post[i] = pre[i] = 1.0f;
        yr[i] = gr[i] = hr[i] = 0;
        if (in[i] && p.post) {
            load<1>(p.post, p.gain_type, d, v);
            post[i] = v[0] + p.offset;
        }
        if (in[i] && channel_gate) {
            load<1>(p.gate.p, p.gate.type, d, v);
            post[i] *= v[0];
        }
        if (in[i] && p.pre) {
            load<1>(p.pre, p.gain_type, d, v);
            pre[i] = v[0] + p.offset;
        }
    }
    auto ahead = [&](int64_t row) {
        if (row >= p.N)
            return;
#pragma unroll
        for (int i = 0; i < kOddVals; ++i)
            if (in[i]) {
                if (p.y.p)
                    yr[i] = __ldcg(y + i * TPR);
                if (GATE)
                    gr[i] = __ldcg(g + i * TPR);
                if constexpr (F32)
                    hr[i] = __float_as_uint(__ldcg(h + i * TPR));
                else
                    hr[i] = __ldcg(h + i * TPR);
            }
        y += y_step;
        g += g_step;
        h += h_step;
    };
    ahead(blockIdx.x);
    for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x) {
        float r = p.b;
        if (row_gated)
            r *= row_gate(p, row);
        float v[kOddVals], w[kOddVals], s = 0.0f;
#pragma unroll
        for (int i = 0; i < kOddVals; ++i) {
            v[i] = __uint_as_float(yr[i] << 16);
            w[i] = p.a * __uint_as_float(F32 ? hr[i] : hr[i] << 16);
            s = fmaf(v[i], v[i], s);
            v[i] *= post[i];
            if (GATE)
                v[i] *= __uint_as_float(gr[i] << 16);
        }
        ahead(row + gridDim.x);
        if (sums)
            r *= rsqrtf(row_sum(s, part[0]) * p.per_d + p.eps);
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < kOddVals; ++i) {
            w[i] = fmaf(r, v[i], w[i]);
            s = fmaf(w[i], w[i], s);
            if (in[i] && p.h_out.p) {
                if constexpr (F32)
                    ho[i * TPR] = w[i];
                else
                    ho[i * TPR] = f32_to_bf16(w[i]);
            }
        }
        if (p.xn.p) {
            r = rsqrtf(row_sum(s, part[1]) * p.per_d + p.eps);
#pragma unroll
            for (int i = 0; i < kOddVals; ++i)
                if (in[i])
                    xn[i * TPR] = f32_to_bf16(pre[i] * (w[i] * r));
        }
        ho += ho_step;
        xn += n_step;
        if (!both)
            __syncthreads();
    }
}

// Rows of any alignment, element by element, the next row's on their way (VPT = 4). (VPT = 16, beyond 4,096 elements,
// spills some 200 bytes and is slow: 4,099 bf16 rows of 8,195 643 us.)
template <int VPT>
__global__ void __launch_bounds__(1024) k_block_norm_any(const Args p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float part[2][32];
    const int t = threadIdx.x, TPR = blockDim.x;
    constexpr bool kAhead = VPT == 4;
    float *gains = reinterpret_cast<float *>(smem);
    tc::after_previous();
    tc::let_next_start();
    auto bring = [&](const Rows &r, int64_t row, float (&v)[VPT][1]) {
        const int64_t first = row * r.stride + t;
        const bool live = r.p && r.step && row < p.N;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            v[i][0] = 0.0f;
            if (live && i * TPR + t < p.D)
                load<1>(r.p, r.type, first + i * TPR, v[i]);
        }
    };
    float y[VPT][1], h[VPT][1], g[VPT][1], y1[VPT][1], h1[VPT][1], g1[VPT][1];
    auto bring_all = [&](int64_t row, float (&y)[VPT][1], float (&h)[VPT][1], float (&g)[VPT][1]) {
        bring(p.y, row, y);
        bring(p.h, row, h);
        bring(p.gate, row, g);
    };
    if (kAhead)
        bring_all(blockIdx.x, y1, h1, g1);
    keep_gains(p, gains);
    __syncthreads();
    for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x) {
        const float one = row_gate(p, row);
        if (kAhead) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                y[i][0] = y1[i][0];
                h[i][0] = h1[i][0];
                g[i][0] = g1[i][0];
            }
            bring_all(row + gridDim.x, y1, h1, g1);
        } else {
            bring_all(row, y, h, g);
        }
        one_row<VPT, 1>(p, row, y, h, g, one, gains, part);
        if (!(p.post_norm && p.y.p && p.xn.p))
            __syncthreads();
    }
}

}  // namespace norm
}  // namespace fgm
