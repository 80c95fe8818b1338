// Attention of M <= 8 new tokens per sequence over the 8-bit cache
// (fgm_attn_fwd): simplest form, one CTA per (query row, kv head, sequence),
// fp32 on the CUDA cores, an online softmax over the blocks.
#pragma once

#include "kv_append.cuh"

namespace fgm {
namespace kv {

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
};

template <int D>
__global__ void __launch_bounds__(128) k_attn_simple(const AttnArgs p)
{
    __shared__ float q[D], pr[64];
    const int tid = threadIdx.x, h = blockIdx.y, b = blockIdx.z, i = blockIdx.x / p.G, g = blockIdx.x % p.G;
    const int hq = h * p.G + g;
    const int len = clamp_len(__ldg(p.lens + b), p.max_blocks, p.status, tid == 0 && blockIdx.x == 0 && h == 0);
    for (int d = tid; d < D; d += 128)
        q[d] = bf16_to_f32(p.q[(static_cast<int64_t>(b) * p.M + i) * p.stride + hq * D + d]);
    const int pos = len - p.M + i;
    const int t0 = p.window > 0 ? max(0, pos - p.window + 1) : 0;
    float m = -INFINITY, l = 0.0f, acc[(D + 127) / 128] = {};
    for (int j = t0 / 64; j * 64 <= pos; ++j) {
        const int64_t ph = phys_block(p.table, b, j, p.max_blocks, p.c.n_blocks);
        if (ph < 0) {
            if (tid == 0)
                atomicOr(p.status, FGM_STATUS_BAD_BLOCK);
            continue;
        }
        const uint8_t *k = p.c.k_q + (ph * p.c.heads + h) * (64 * D), *v = p.c.v_q + (ph * p.c.heads + h) * (64 * D);
        __syncthreads();
        if (tid < 64) {
            const int t = j * 64 + tid;
            float s = -INFINITY;
            if (t >= t0 && t <= pos) {
                float a = 0.0f, x[4];
                for (int d = 0; d < D; d += 4) {
                    e4m3x4_to_f32(*reinterpret_cast<const uint32_t *>(k + (d >> 6) * 4096 + tid * 64 + (d & 63)), x);
                    a += q[d] * x[0] + q[d + 1] * x[1] + q[d + 2] * x[2] + q[d + 3] * x[3];
                }
                s = a * p.scale * p.c.k_s[ph * p.c.heads + h];
            }
            pr[tid] = s;
        }
        __syncthreads();
        float mx = m;
        for (int t = 0; t < 64; ++t)
            mx = fmaxf(mx, pr[t]);
        const float f = m == -INFINITY ? 0.0f : expf(m - mx), vs = p.c.v_s[ph * p.c.heads + h];
        l *= f;
        for (int e = 0; e < (D + 127) / 128; ++e)
            acc[e] *= f;
        for (int t = 0; t < 64; ++t) {
            if (pr[t] == -INFINITY)
                continue;
            const float w = expf(pr[t] - mx);
            l += w;
            for (int e = 0; e < (D + 127) / 128; ++e) {
                const int d = tid + e * 128;
                if (d < D) {
                    const __half_raw x = __nv_cvt_fp8_to_halfraw(v[d * 64 + t], __NV_E4M3);
                    acc[e] += w * vs * __half2float(__half(x));
                }
            }
        }
        m = mx;
    }
    const int64_t row = (static_cast<int64_t>(b) * p.M + i) * p.Hq + hq;
    for (int e = 0; e < (D + 127) / 128; ++e) {
        const int d = tid + e * 128;
        if (d < D)
            p.out[row * D + d] = f32_to_bf16(l == 0.0f ? 0.0f : acc[e] / l);
    }
    if (tid == 0 && p.lse)
        p.lse[row] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace kv
}  // namespace fgm
