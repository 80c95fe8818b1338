// C ABI of the 8-bit KV cache (declared in include/fgm.h): argument checks and
// launches of kv_append.cuh and kv_attn.cuh.
#include <atomic>
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
int launch_append(const kv::AppendArgs &a, dim3 grid, cudaStream_t st)
{
    return launch_overlapped(kv::k_kv_append<D>, grid, kv::Append<D>::kThreads, 0, st, a);
}

// Rows of the products: the instantiations. Padding costs softmax work only (the
// 128-lane products take the same time up to 64 columns, 1.3 times that at 128).
int attn_rows(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 48 ? 48 : 64; }

// The attention's regions behind the common workspace.
struct AttnWs {
    size_t part, rec, total;
};

AttnWs attn_ws(int rows, int D)
{
    AttnWs o;
    o.part = align_up(ws_offsets().total, 256);
    o.rec = align_up(o.part + sizeof(float) * 2 * kv::kMaxGrid * kv::partial_floats(attn_rows(rows), D), 256);
    o.total = align_up(o.rec + sizeof(int4) * kv::kMaxGrid, 256);
    return o;
}

template <int D, int R>
int launch_attn_t(kv::AttnArgs &a, int sms, cudaStream_t st)
{
    const int grid = sms < kv::kMaxGrid ? sms : kv::kMaxGrid;
    a.n_rec = a.B * a.c.heads < grid ? a.B * a.c.heads : grid;
    // what is left of the shared memory goes to the rings, V's first: its stages are freed last
    constexpr size_t side = static_cast<size_t>(kv::kTile) * D;
    a.q_ring = kv::query_bytes(R, D) <= 16384 ? 2 : 1;
    const size_t fixed = a.q_ring * kv::query_bytes(R, D) + 2 * kv::prob_bytes(R) + (D == 64 ? kv::kBlock * D : 0) +
                         align_up(sizeof(int) * (3 * static_cast<size_t>(a.B) + 2), 128) + 1024;
    const size_t most = kv::kSmemMax - sizeof(kv::AttnShared) - 256;
    const int stages = static_cast<int>((most - fixed) / side);
    a.v_ring = (stages + 1) / 2 < kv::kMaxRing ? (stages + 1) / 2 : kv::kMaxRing;
    a.k_ring = stages - a.v_ring < kv::kMaxRing ? stages - a.v_ring : kv::kMaxRing;
    const size_t bytes = fixed + (a.k_ring + a.v_ring) * side;
    CUtensorMap kmap, vmap;
    const uint64_t n_rows = static_cast<uint64_t>(a.c.n_blocks) * a.c.heads * D;
    FGM_HOST_TRY(host_rows64_map(&kmap, a.c.k_q, n_rows, kv::kBlock));
    FGM_HOST_TRY(host_rows64_map(&vmap, a.c.v_q, n_rows, D));
    static std::atomic<bool> ready[64];        // per device; setting it twice does no harm
    int dev = 0;
    FGM_HOST_CUDA(cudaGetDevice(&dev));
    if (!ready[dev & 63]) {
        FGM_HOST_CUDA(cudaFuncSetAttribute(kv::k_attn<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(most)));
        ready[dev & 63] = true;
    }
    FGM_HOST_TRY(launch_overlapped(kv::k_attn<D, R>, dim3(grid), kv::kAttnThreads, bytes, st, kmap, vmap, a));
    // a CTA a row where the records are few, else enough to fill the device
    const int rows = a.M * a.G, y = a.n_rec * rows <= 2432 ? rows : 2432 / a.n_rec;
    return launch_overlapped(kv::k_attn_join<D>, dim3(a.n_rec, y), 256, 0, st, a);
}

template <int D>
int launch_attn(kv::AttnArgs &a, int sms, cudaStream_t st)
{
    switch (a.rows) {
    case 8: return launch_attn_t<D, 8>(a, sms, st);
    case 16: return launch_attn_t<D, 16>(a, sms, st);
    case 32: return launch_attn_t<D, 32>(a, sms, st);
    case 48: return launch_attn_t<D, 48>(a, sms, st);
    default: return launch_attn_t<D, 64>(a, sms, st);
    }
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
    case 64: return launch_append<64>(a, grid, st);
    case 128: return launch_append<128>(a, grid, st);
    default: return launch_append<256>(a, grid, st);
    }
}

size_t fgm_attn_workspace_bytes(int B, int M, int n_q_heads, int n_kv_heads, int head_dim)
{
    if (B < 1 || B > 1024 || M < 1 || M > kMaxM || n_kv_heads < 1 || n_kv_heads > 1024 || n_q_heads < 1 ||
        n_q_heads % n_kv_heads || !head_dim_ok(head_dim) || n_q_heads / n_kv_heads > FGM_ATTN_MAX_ROWS / M)
        return 0;
    return attn_ws(M * (n_q_heads / n_kv_heads), head_dim).total;
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
    if (n_q_heads / cache->n_kv_heads > FGM_ATTN_MAX_ROWS / M)
        return failf(FGM_ERR_INVALID_ARG, "M * n_q_heads / n_kv_heads = %lld above %d",
                     static_cast<long long>(M) * (n_q_heads / cache->n_kv_heads), FGM_ATTN_MAX_ROWS);
    FGM_HOST_TRY(check_rows("q", q, token_stride, n_q_heads, cache->head_dim));
    if (!(scale > 0.0f) || !std::isfinite(scale))
        return failf(FGM_ERR_INVALID_ARG, "scale = %g: needs a finite scale > 0", (double)scale);
    if (window < 0)
        return failf(FGM_ERR_INVALID_ARG, "window = %d: 0 (none) or a positive number of tokens", window);
    if (!out || !is_aligned(out, 16) || !is_aligned(lse, 4))
        return failf(FGM_ERR_INVALID_ARG, "out NULL or not 16-byte aligned, or lse not 4-byte aligned");
    FGM_HOST_TRY(host_check_ws(ws, ws_bytes, fgm_attn_workspace_bytes(B, M, n_q_heads, cache->n_kv_heads, cache->head_dim)));
    if (static_cast<int64_t>(B) * max_blocks * cache->n_kv_heads > (1LL << 30))
        return failf(FGM_ERR_INVALID_ARG, "B * max_blocks * n_kv_heads = %lld above 2^30",
                     (long long)B * max_blocks * cache->n_kv_heads);
    if (cache->n_blocks * cache->n_kv_heads > 0x7FFFFFFFLL / cache->head_dim)
        return failf(FGM_ERR_INVALID_ARG, "cache of %lld blocks: n_blocks * n_kv_heads * head_dim above 2^31 - 1",
                     (long long)cache->n_blocks);
    int sms = 0;
    FGM_HOST_TRY(host_device_ready(&sms));
    kv::AttnArgs a = {};
    a.c = device_cache(cache);
    a.q = q;
    a.stride = token_stride;
    a.B = B;
    a.M = M;
    a.G = n_q_heads / cache->n_kv_heads;
    a.Hq = n_q_heads;
    a.lens = lens;
    a.table = block_table;
    a.max_blocks = max_blocks;
    a.scale = scale;
    a.window = window < (1 << 30) ? window : 1 << 30;
    a.out = out;
    a.lse = lse;
    a.status = status_word(ws);
    const AttnWs o = attn_ws(M * a.G, cache->head_dim);
    a.part = reinterpret_cast<float *>(static_cast<char *>(ws) + o.part);
    a.rec = reinterpret_cast<int4 *>(static_cast<char *>(ws) + o.rec);
    a.rows = attn_rows(M * a.G);
    a.timeout_ns = host_wait_limit_ns();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (cache->head_dim) {
    case 64: return launch_attn<64>(a, sms, st);
    case 128: return launch_attn<128>(a, sms, st);
    default: return launch_attn<256>(a, sms, st);
    }
}

}  // extern "C"
