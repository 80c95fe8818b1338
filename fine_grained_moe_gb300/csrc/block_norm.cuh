// The norms around a block (fgm_block_norm):
//   h' = a h + b gate * post(y),   xn = pre(h'),
//   post(y) = y / sqrt(mean(y^2) + eps) * (post_gain + offset), pre(h') alike.
//
// 10 operations an element: bound by HBM. One pass: a row's y and h are read once into
// registers, both norms' sums are taken there, and h' and xn written once. Sums and
// h' itself are fp32; xn goes by the fp32 h', not by the rounded one that is stored.
// TPR threads own a row, VPT vectors of VEC elements each (VEC = 8 where rows allow
// 16-byte accesses, else 1).
#pragma once

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
    float a, b, offset, eps;
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
                w[q] = narrow(v[2 * q], type) | static_cast<uint32_t>(narrow(v[2 * q + 1], type)) << 16;
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
        if (type == FGM_F32)
            static_cast<float *>(p)[i] = v[0];
        else
            static_cast<uint16_t *>(p)[i] = narrow(v[0], type);
    }
}

constexpr int kMinThreads = 128;

// Sum over a row's threads, the same order and so the same bits in each.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *part)
{
    v = warp_sum(v);
    if constexpr (TPR > 32) {
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0)
            part[warp] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < TPR / 32; ++w)
            v += part[w];
    }
    return v;
}

template <int TPR, int VPT, int VEC>
__global__ void __launch_bounds__(TPR < kMinThreads ? kMinThreads : TPR) k_block_norm(const Args p)
{
    constexpr int kRows = TPR < kMinThreads ? kMinThreads / TPR : 1;
    __shared__ float part[2][TPR > 32 ? TPR / 32 : 1];
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / TPR;
    const int t = threadIdx.x % TPR;
    tc::after_previous();
    tc::let_next_start();
    if (row >= p.N)                              // (whole warps; with several a row there is one row a CTA)
        return;
    float h[VPT][VEC], y[VPT][VEC], s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int d = (i * TPR + t) * VEC;
#pragma unroll
        for (int q = 0; q < VEC; ++q)
            h[i][q] = y[i][q] = 0.0f;
        if (d < p.D) {
            if (p.y.p)
                load<VEC>(p.y.p, p.y.type, row * p.y.stride + d, y[i]);
            load<VEC>(p.h.p, p.h.type, row * p.h.stride + d, h[i]);
        }
    }
    if (p.y.p) {
        float r = p.b;
        if (p.post_norm) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int q = 0; q < VEC; ++q)
                    s = fmaf(y[i][q], y[i][q], s);
            r *= rsqrtf(row_sum<TPR>(s, part[0]) / p.D + p.eps);
        }
        float one[1] = {1.0f};
        if (p.gate.p && !p.gate.step) {
            load<1>(p.gate.p, p.gate.type, row * p.gate.stride, one);
            r *= one[0];
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int d = (i * TPR + t) * VEC;
            if (d < p.D) {
                float g[VEC];
                if (p.post) {
                    load<VEC>(p.post, p.gain_type, d, g);
#pragma unroll
                    for (int q = 0; q < VEC; ++q)
                        y[i][q] *= g[q] + p.offset;
                }
                if (p.gate.p && p.gate.step) {
                    load<VEC>(p.gate.p, p.gate.type, row * p.gate.stride + d, g);
#pragma unroll
                    for (int q = 0; q < VEC; ++q)
                        y[i][q] *= g[q];
                }
            }
#pragma unroll
            for (int q = 0; q < VEC; ++q)
                h[i][q] = fmaf(r, y[i][q], p.a * h[i][q]);
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
                store<VEC>(p.h_out.p, p.h_out.type, row * p.h_out.stride + d, h[i]);
        }
    if (!p.xn.p)
        return;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int q = 0; q < VEC; ++q)
            s = fmaf(h[i][q], h[i][q], s);
    const float r = rsqrtf(row_sum<TPR>(s, part[1]) / p.D + p.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int d = (i * TPR + t) * VEC;
        if (d < p.D) {
            float g[VEC];
            if (p.pre) {
                load<VEC>(p.pre, p.gain_type, d, g);
#pragma unroll
                for (int q = 0; q < VEC; ++q)
                    g[q] = (g[q] + p.offset) * (h[i][q] * r);
            } else {
#pragma unroll
                for (int q = 0; q < VEC; ++q)
                    g[q] = h[i][q] * r;
            }
            store<VEC>(p.xn.p, p.xn.type, row * p.xn.stride + d, g);
        }
    }
}

}  // namespace norm
}  // namespace fgm
