// C ABI of the 8-bit KV cache (declared in include/fgm.h): argument checks and
// launches of kv_append.cuh and kv_attn.cuh.
#include <cmath>

#include "host.h"
#include "kv_append.cuh"
#include "kv_attn.cuh"

namespace fgm {
namespace {

bool head_dim_ok(int D) { return D == 64 || D == 128 || D == 256; }

int check_cache(const fgm_kv_cache *c)
{
    if (!c)
        return failf(FGM_ERR_INVALID_ARG, "cache is NULL");
    if (!head_dim_ok(c->head_dim))
        return failf(FGM_ERR_INVALID_ARG, "head_dim = %d: 64, 128 or 256", c->head_dim);
    if (c->n_kv_heads < 1 || c->n_kv_heads > 1024)
        return failf(FGM_ERR_INVALID_ARG, "n_kv_heads = %d outside [1, 1024]", c->n_kv_heads);
    if (c->n_blocks < 1 || c->n_blocks > 0x7FFFFFFFLL)
        return failf(FGM_ERR_INVALID_ARG, "n_blocks = %lld outside [1, 2^31)", (long long)c->n_blocks);
    if (!c->k_q || !c->v_q || !is_aligned(c->k_q, 16) || !is_aligned(c->v_q, 16))
        return failf(FGM_ERR_INVALID_ARG, "cache codes NULL or not 16-byte aligned");
    if (!c->k_s || !c->v_s || !is_aligned(c->k_s, 4) || !is_aligned(c->v_s, 4))
        return failf(FGM_ERR_INVALID_ARG, "cache scales NULL or not 4-byte aligned");
    return FGM_OK;
}

int check_seqs(int B, const int32_t *lens, const int32_t *table, int max_blocks)
{
    if (B < 1 || B > 1024)
        return failf(FGM_ERR_INVALID_ARG, "B = %d outside [1, 1024]", B);
    if (!lens || !is_aligned(lens, 4) || !is_aligned(table, 4))
        return failf(FGM_ERR_INVALID_ARG, "lens NULL, or lens or block_table not 4-byte aligned");
    if (max_blocks < 1 || max_blocks > (1 << 24))
        return failf(FGM_ERR_INVALID_ARG, "max_blocks = %d outside [1, 2^24]", max_blocks);
    return FGM_OK;
}

int check_rows(const char *name, const void *p, int64_t stride, int heads, int D)
{
    if (!p || !is_aligned(p, 16))
        return failf(FGM_ERR_INVALID_ARG, "%s NULL or not 16-byte aligned", name);
    if (stride < static_cast<int64_t>(heads) * D || stride % 8)
        return failf(FGM_ERR_INVALID_ARG, "token_stride = %lld: a multiple of 8, at least heads * head_dim = %lld",
                     (long long)stride, (long long)heads * D);
    return FGM_OK;
}

int32_t *status_word(void *ws) { return reinterpret_cast<int32_t *>(static_cast<char *>(ws) + ws_offsets().status); }

kv::Cache device_cache(const fgm_kv_cache *c)
{
    return kv::Cache{c->k_q, c->k_s, c->v_q, c->v_s, c->n_blocks, c->n_kv_heads};
}

template <int D>
void launch_append(const kv::AppendArgs &a, dim3 grid, cudaStream_t st)
{
    kv::k_kv_append<D><<<grid, kv::Append<D>::kThreads, 0, st>>>(a);
}

}  // namespace
}  // namespace fgm

using namespace fgm;

extern "C" {

int fgm_kv_append(const fgm_kv_cache *cache, const uint16_t *k, const uint16_t *v, int64_t token_stride, int B, int N,
                  const int32_t *lens, const int32_t *block_table, int max_blocks, void *ws, size_t ws_bytes,
                  void *stream)
{
    FGM_HOST_TRY(check_cache(cache));
    FGM_HOST_TRY(check_seqs(B, lens, block_table, max_blocks));
    if (N < 1 || N > (1 << 24))
        return failf(FGM_ERR_INVALID_ARG, "N = %d outside [1, 2^24]", N);
    FGM_HOST_TRY(check_rows("k", k, token_stride, cache->n_kv_heads, cache->head_dim));
    FGM_HOST_TRY(check_rows("v", v, token_stride, cache->n_kv_heads, cache->head_dim));
    FGM_HOST_TRY(host_check_ws(ws, ws_bytes, ws_offsets().total));
    FGM_HOST_TRY(host_device_ready(nullptr));
    kv::AppendArgs a{device_cache(cache), k, v, token_stride, N, lens, block_table, max_blocks, status_word(ws)};
    const dim3 grid((N + FGM_KV_BLOCK - 2) / FGM_KV_BLOCK + 1, 2 * cache->n_kv_heads, B);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (cache->head_dim) {
    case 64: launch_append<64>(a, grid, st); break;
    case 128: launch_append<128>(a, grid, st); break;
    default: launch_append<256>(a, grid, st); break;
    }
    FGM_HOST_CUDA(cudaGetLastError());
    return FGM_OK;
}

size_t fgm_attn_workspace_bytes(int B, int M, int n_q_heads, int n_kv_heads, int head_dim)
{
    if (B < 1 || B > 1024 || M < 1 || M > kMaxM || n_kv_heads < 1 || n_kv_heads > 1024 || n_q_heads < 1 ||
        n_q_heads % n_kv_heads || !head_dim_ok(head_dim) || M * (n_q_heads / n_kv_heads) > FGM_ATTN_MAX_ROWS)
        return 0;
    return ws_offsets().total;
}

int fgm_attn_fwd(const fgm_kv_cache *cache, const uint16_t *q, int64_t token_stride, int B, int M, int n_q_heads,
                 const int32_t *lens, const int32_t *block_table, int max_blocks, float scale, int window,
                 uint16_t *out, float *lse, void *ws, size_t ws_bytes, void *stream)
{
    FGM_HOST_TRY(check_cache(cache));
    FGM_HOST_TRY(check_seqs(B, lens, block_table, max_blocks));
    if (M < 1 || M > kMaxM)
        return failf(FGM_ERR_INVALID_ARG, "M = %d outside [1, %d]", M, kMaxM);
    if (n_q_heads < 1 || n_q_heads % cache->n_kv_heads)
        return failf(FGM_ERR_INVALID_ARG, "n_q_heads = %d: a multiple of n_kv_heads = %d", n_q_heads, cache->n_kv_heads);
    if (M * (n_q_heads / cache->n_kv_heads) > FGM_ATTN_MAX_ROWS)
        return failf(FGM_ERR_INVALID_ARG, "M * n_q_heads / n_kv_heads = %d above %d", M * (n_q_heads / cache->n_kv_heads),
                     FGM_ATTN_MAX_ROWS);
    FGM_HOST_TRY(check_rows("q", q, token_stride, n_q_heads, cache->head_dim));
    if (!(scale > 0.0f) || !std::isfinite(scale))
        return failf(FGM_ERR_INVALID_ARG, "scale = %g: needs a finite scale > 0", (double)scale);
    if (window < 0)
        return failf(FGM_ERR_INVALID_ARG, "window = %d: 0 (none) or a positive number of tokens", window);
    if (!out || !is_aligned(out, 16) || !is_aligned(lse, 4))
        return failf(FGM_ERR_INVALID_ARG, "out NULL or not 16-byte aligned, or lse not 4-byte aligned");
    FGM_HOST_TRY(host_check_ws(ws, ws_bytes, fgm_attn_workspace_bytes(B, M, n_q_heads, cache->n_kv_heads, cache->head_dim)));
    FGM_HOST_TRY(host_device_ready(nullptr));
    const int G = n_q_heads / cache->n_kv_heads;
    kv::AttnArgs a{device_cache(cache), q, token_stride, B, M, G, n_q_heads, lens, block_table, max_blocks, scale,
                   window < (1 << 30) ? window : 1 << 30, out, lse, status_word(ws)};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const dim3 grid(M * G, cache->n_kv_heads, B);
    switch (cache->head_dim) {
    case 64: kv::k_attn_simple<64><<<grid, 128, 0, st>>>(a); break;
    case 128: kv::k_attn_simple<128><<<grid, 128, 0, st>>>(a); break;
    default: kv::k_attn_simple<256><<<grid, 128, 0, st>>>(a); break;
    }
    FGM_HOST_CUDA(cudaGetLastError());
    return FGM_OK;
}

}  // extern "C"
