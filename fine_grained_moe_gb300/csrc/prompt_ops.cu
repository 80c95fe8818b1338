// C ABI of a prompt's way through the experts (declared in include/fgm.h): argument
// checks and launches of route.cuh, moe_rows.cuh and grouped.cuh.
#include <atomic>

#include "grouped.cuh"
#include "host.h"
#include "moe_rows.cuh"
#include "route.cuh"

namespace fgm {
namespace {

constexpr int64_t kMaxT = FGM_MAX_TOKENS;
constexpr int64_t kMaxSlotsN = kMaxT * kK;
constexpr int64_t kMaxGemmRows = 1 << 24;
constexpr int kMaxPairs = 80;                    // CTA pairs of a full sm_103 part

size_t common_bytes() { return align_up(ws_offsets().total, 256); }
int32_t *status_word(void *ws) { return reinterpret_cast<int32_t *>(static_cast<char *>(ws) + ws_offsets().status); }

// Regions of a workspace behind the common one.
struct Carve {
    size_t at = common_bytes();

    size_t take(size_t bytes)
    {
        const size_t a = at;
        at = align_up(at + bytes, 256);
        return a;
    }
};

template <typename T>
T *region(void *ws, size_t at) { return reinterpret_cast<T *>(static_cast<char *>(ws) + at); }

// ---------------------------------------------------------------- grouping

// A CTA's slots: 1,024, more from 256 CTAs on (each reads the counts of all).
int group_chunk(int64_t n)
{
    const int64_t each = (n + rows::kMaxChunks - 1) / rows::kMaxChunks;
    return each <= 1024 ? 1024 : static_cast<int>(align_up(each, rows::kGroupThreads));
}

// Room for the counts of n slots, and of fewer (262,144 have more chunks than 262,145).
size_t group_count_bytes(int64_t n, int E)
{
    const int64_t most = (n + 1023) / 1024, chunks = most < rows::kMaxChunks ? most : rows::kMaxChunks;
    return chunks > 1 ? sizeof(int32_t) * chunks * E : 0;
}

void cut_group(rows::GroupArgs &a)
{
    a.chunk = group_chunk(a.n);
    a.chunks = static_cast<int>((a.n + a.chunk - 1) / a.chunk);
}

size_t group_smem(int E) { return sizeof(int) * (rows::kGroupWarps + 2) * E; }

int launch_deal(const rows::GroupArgs &a, cudaStream_t st)
{
    if (a.chunks > rows::kDirectChunks)
        FGM_HOST_TRY(launch_overlapped(rows::k_group_scan, dim3(1), rows::kScanThreads, 0, st, a));
    return launch_overlapped(rows::k_group_deal, dim3(a.chunks), rows::kGroupThreads, group_smem(a.E), st, a);
}

int launch_group(rows::GroupArgs a, cudaStream_t st)
{
    cut_group(a);
    if (a.chunks > 1)
        FGM_HOST_TRY(launch_overlapped(rows::k_group_count, dim3(a.chunks), rows::kGroupThreads, group_smem(a.E), st, a));
    return launch_deal(a, st);
}

// ---------------------------------------------------------------- routing

constexpr int64_t kRouteCtas = 152;

// K is split while the tiles of 128 tokens leave SMs idle.
int route_splits(int64_t T)
{
    const int64_t s = kRouteCtas / ((T + 127) / 128);
    return static_cast<int>(s < 1 ? 1 : s > route::kChunks ? route::kChunks : s);
}

struct RouteWs {
    size_t part, xn2, wn2, count, total;
};

RouteWs route_ws(int64_t T)
{
    RouteWs o;
    Carve c;
    // Rows of partial sums, for T tokens and for fewer, whose K may be cut into more parts: a split K has at
    // most 128 rows a CTA.
    const int64_t split = route::kChunks * T < kRouteCtas * 128 ? route::kChunks * T : kRouteCtas * 128, n = split < T ? T : split;
    o.part = c.take(sizeof(float) * n * kE);
    o.xn2 = c.take(sizeof(float) * n);
    o.wn2 = c.take(sizeof(float) * route::kChunks * 4);
    o.count = c.take(group_count_bytes(T * kK, kE));
    o.total = c.at;
    return o;
}

// ---------------------------------------------------------------- grouped products

// Rows of a tile at most: as many as tensor memory holds, 64 where experts have fewer than
// four on average (the ring then has more stages of weights: 208 rows on 128 experts 24.6 us, with 256 26.6; 200
// tokens' experts, 12 rows each but some with all, 106 us with 256 and 122 with 64).
int tile_cols(int64_t R, int E, int most) { return R < 4 * static_cast<int64_t>(E) ? 64 : most; }

// bf16 rows or terms as 128-byte boxes: single rows for gathering, else 8 to 128 at a time.
int x_maps(grouped::Maps &m, const void *x, int64_t row_bytes, int64_t stride_bytes, int64_t n, bool gathered)
{
    const uint64_t dims[2] = {static_cast<uint64_t>(row_bytes), static_cast<uint64_t>(n)}, strides[1] = {static_cast<uint64_t>(stride_bytes)};
    for (int i = 0; i < (gathered ? 1 : 5); ++i) {
        const uint32_t box[2] = {128, gathered ? 1u : 8u << i};
        FGM_HOST_TRY(host_map(&m.x[i], x, 1, 2, dims, strides, box, true));
    }
    return FGM_OK;
}

int weight_map(CUtensorMap *map, const void *w, int elem, int E, int N, int K)
{
    const uint64_t dims[3] = {static_cast<uint64_t>(K), static_cast<uint64_t>(N), static_cast<uint64_t>(E)},
                   strides[2] = {static_cast<uint64_t>(K) * elem, static_cast<uint64_t>(K) * elem * N};
    const uint32_t box[3] = {128u / elem, 128, 1};
    return host_map(map, w, elem, 3, dims, strides, box, true);
}

template <grouped::Mode MODE, bool BYTES>
int launch_grouped(const grouped::Maps &m, grouped::Args a, int sms, cudaStream_t st)
{
    const auto kernel = grouped::k_grouped<MODE, BYTES>;
    constexpr int kSmem = grouped::kSmem;
    static std::atomic<int> fit_pairs[64];       // CTA pairs at a time, per device; finding it twice does no harm
    int dev = 0;
    FGM_HOST_CUDA(cudaGetDevice(&dev));
    int most = fit_pairs[dev & 63];
    if (!most) {
        FGM_HOST_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(sms / 2 * 2);
        cfg.blockDim = dim3(grouped::kGatherThreads);
        cfg.dynamicSmemBytes = kSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        FGM_HOST_CUDA(cudaOccupancyMaxActiveClusters(&most, kernel, &cfg));
        if (most < 1)
            return failf(FGM_ERR_DEVICE, "no CTA pair of the grouped products fits this device");
        most = most < kMaxPairs ? most : kMaxPairs;
        fit_pairs[dev & 63] = most;
    }
    const int fit = grouped::kRing / grouped::stage_bytes<MODE, BYTES>(a.cols);
    for (a.log_cols = 0; 1 << a.log_cols < a.cols; ++a.log_cols)
        ;
    a.stages = fit < grouped::kMaxStages ? fit : grouped::kMaxStages;
    // tiles: an expert has at most its rows / cols, rounded up, and no more experts than rows have any
    const int64_t across = (a.N + 255) / 256, tiles = (a.R / a.cols + (a.E < a.R ? a.E : a.R)) * across;
    const int64_t pairs = tiles < most ? tiles : most;
    return launch_overlapped(kernel, dim3(static_cast<unsigned>(2 * pairs)), a.src ? grouped::kGatherThreads : grouped::kThreads, kSmem, st, m, a);
}

// CTAs for the terms of n rows.
unsigned term_ctas(int64_t n, int K)
{
    const int each = rows::kTermThreads / rows::term_row(K);
    return static_cast<unsigned>((n + each - 1) / each);
}

bool gemm_sizes_ok(int64_t x_rows, int64_t R, int E, int N, int K)
{
    return x_rows >= 1 && x_rows <= kMaxGemmRows && R >= 1 && R <= kMaxGemmRows && E >= 1 && E <= FGM_MAX_GROUPS && N >= 1 && N <= 65536 &&
           K >= 8 && K <= 65536 && K % 8 == 0;
}

struct GemmWs {
    size_t terms, xs, total;
};

GemmWs gemm_ws(int64_t x_rows, int K)
{
    GemmWs o;
    Carve c;
    o.terms = c.take(2 * align_up(K, 32) * x_rows);
    o.xs = c.take(sizeof(float) * x_rows);
    o.total = c.at;
    return o;
}

struct ExpertsWs {
    size_t offsets, src, pos, count, terms, xs, exps, act_terms, sa, rows, smax, total;
};

ExpertsWs experts_ws(int64_t T)
{
    ExpertsWs o;
    Carve c;
    const int64_t R = T * (kK + 1);
    o.offsets = c.take(sizeof(int32_t) * (kE + 2));
    o.src = c.take(sizeof(int32_t) * R);
    o.pos = c.take(sizeof(int32_t) * T * kK);
    o.count = c.take(group_count_bytes(T * kK, kE));
    o.terms = c.take(2 * static_cast<size_t>(kH) * T);
    o.xs = c.take(sizeof(float) * T);
    o.exps = c.take(static_cast<size_t>(kF / 32) * R);
    o.act_terms = c.take(2 * static_cast<size_t>(kF) * R);
    o.sa = c.take(sizeof(float) * R);
    o.rows = c.take(sizeof(uint16_t) * kH * R);  // (first the activations, 704 of 2816, which end as terms)
    o.smax = c.take(sizeof(float) * kNE);
    o.total = c.at;
    return o;
}

int check_x(const uint16_t *x, int64_t stride, int64_t width)
{
    if (!x || !is_aligned(x, 16))
        return failf(FGM_ERR_INVALID_ARG, "x NULL or not 16-byte aligned");
    if (stride < width || stride % 8 || stride > (int64_t(1) << 32))
        return failf(FGM_ERR_INVALID_ARG, "x_stride = %lld: a multiple of 8, at least %lld, at most 2^32", (long long)stride, (long long)width);
    return FGM_OK;
}

int check_tokens(int64_t T)
{
    if (T < 1 || T > kMaxT)
        return failf(FGM_ERR_INVALID_ARG, "T = %lld outside [1, %lld]", (long long)T, (long long)kMaxT);
    return FGM_OK;
}

int check_words(const char *name, const void *p)
{
    if (!p || !is_aligned(p, 4))
        return failf(FGM_ERR_INVALID_ARG, "%s NULL or not 4-byte aligned", name);
    return FGM_OK;
}

}  // namespace
}  // namespace fgm

using namespace fgm;

extern "C" {

size_t fgm_moe_route_workspace_bytes(int64_t T) { return T < 1 || T > kMaxT ? 0 : route_ws(T).total; }

int fgm_moe_route(const uint16_t *router_w, const float *router_b, const uint16_t *x, int64_t x_stride, int64_t T, int32_t *ids,
                  float *w, int32_t *offsets, int32_t *order, void *ws, size_t ws_bytes, void *stream)
{
    FGM_HOST_TRY(check_tokens(T));
    if (!router_w || !is_aligned(router_w, 16))
        return failf(FGM_ERR_INVALID_ARG, "router_w NULL or not 16-byte aligned");
    if (!is_aligned(router_b, 4))
        return failf(FGM_ERR_INVALID_ARG, "router_b not 4-byte aligned");
    FGM_HOST_TRY(check_x(x, x_stride, kH));
    FGM_HOST_TRY(check_words("ids", ids));
    FGM_HOST_TRY(check_words("w", w));
    if (!offsets != !order)
        return failf(FGM_ERR_INVALID_ARG, "offsets and order: both or neither");
    if (!is_aligned(offsets, 4) || !is_aligned(order, 4))
        return failf(FGM_ERR_INVALID_ARG, "offsets or order not 4-byte aligned");
    const RouteWs o = route_ws(T);
    FGM_HOST_TRY(host_check_ws(ws, ws_bytes, o.total));
    FGM_HOST_TRY(host_device_ready(nullptr));
    CUtensorMap xmap, wmap;
    const uint64_t xdims[2] = {kH, static_cast<uint64_t>(T)}, xstr[1] = {2 * static_cast<uint64_t>(x_stride)}, wdims[2] = {kH, kE}, wstr[1] = {2 * kH};
    const uint32_t box[2] = {64, 128};
    FGM_HOST_TRY(host_map(&xmap, x, 2, 2, xdims, xstr, box, true));
    FGM_HOST_TRY(host_map(&wmap, router_w, 2, 2, wdims, wstr, box, true));
    static std::atomic<bool> ready[64];          // per device; setting it twice does no harm
    int dev = 0;
    FGM_HOST_CUDA(cudaGetDevice(&dev));
    if (!ready[dev & 63]) {
        FGM_HOST_CUDA(cudaFuncSetAttribute(route::k_router_logits_tc, cudaFuncAttributeMaxDynamicSharedMemorySize, route::kSmem));
        ready[dev & 63] = true;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    route::LogitArgs a = {};
    a.T = T;
    a.splits = route_splits(T);
    a.part = region<float>(ws, o.part);
    a.xn2 = region<float>(ws, o.xn2);
    a.wn2 = region<float>(ws, o.wn2);
    a.w = router_w;
    a.status = status_word(ws);
    a.timeout_ns = host_wait_limit_ns();
    rows::GroupArgs g = {};
    g.ids = ids;
    g.n = T * kK;
    g.E = kE;
    g.count = region<int32_t>(ws, o.count);
    g.offsets = offsets;
    g.order = order;
    g.per = 1;
    cut_group(g);
    if (offsets && g.chunks > 1) {               // (counted by the choice)
        a.count = g.count;
        a.counts = g.chunks * kE;
    }
    FGM_HOST_TRY(launch_overlapped(route::k_router_logits_tc, dim3(static_cast<unsigned>((T + 127) / 128), a.splits), route::kThreads,
                                   route::kSmem, st, xmap, wmap, a));
    const route::TopArgs b{a.part, a.xn2, a.wn2, router_b, x, x_stride, router_w, T, a.splits, ids, w, a.count, static_cast<unsigned>(g.chunk / kK), a.status};
    const dim3 tops(static_cast<unsigned>((T + route::kTopWarps - 1) / route::kTopWarps));
    FGM_HOST_TRY(a.splits == 1 ? launch_overlapped(route::k_route_top<1>, tops, 32 * route::kTopWarps, 0, st, b)
                               : launch_overlapped(route::k_route_top<route::kChunks>, tops, 32 * route::kTopWarps, 0, st, b));
    if (!offsets)
        return FGM_OK;
    return launch_deal(g, st);
}

size_t fgm_moe_group_workspace_bytes(int64_t n, int E)
{
    if (n < 1 || n > kMaxSlotsN || E < 1 || E > FGM_MAX_GROUPS)
        return 0;
    return align_up(common_bytes() + group_count_bytes(n, E), 256);
}

int fgm_moe_group(const int32_t *ids, int64_t n, int E, int32_t *offsets, int32_t *order, void *ws, size_t ws_bytes, void *stream)
{
    if (n < 1 || n > kMaxSlotsN)
        return failf(FGM_ERR_INVALID_ARG, "n = %lld outside [1, %lld]", (long long)n, (long long)kMaxSlotsN);
    if (E < 1 || E > FGM_MAX_GROUPS)
        return failf(FGM_ERR_INVALID_ARG, "E = %d outside [1, %d]", E, FGM_MAX_GROUPS);
    FGM_HOST_TRY(check_words("ids", ids));
    FGM_HOST_TRY(check_words("offsets", offsets));
    FGM_HOST_TRY(check_words("order", order));
    FGM_HOST_TRY(host_check_ws(ws, ws_bytes, fgm_moe_group_workspace_bytes(n, E)));
    // (a CTA may read its ids when others have written)
    auto meet = [](const void *a, int64_t na, const void *b, int64_t nb) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
        return x < y + 4 * nb && y < x + 4 * na;
    };
    if (meet(ids, n, offsets, E + 1) || meet(ids, n, order, n) || meet(offsets, E + 1, order, n))
        return failf(FGM_ERR_INVALID_ARG, "ids, offsets and order overlap");
    FGM_HOST_TRY(host_device_ready(nullptr));
    rows::GroupArgs g = {};
    g.ids = ids;
    g.n = n;
    g.E = E;
    g.count = region<int32_t>(ws, common_bytes());
    g.offsets = offsets;
    g.order = order;
    g.per = 1;
    return launch_group(g, static_cast<cudaStream_t>(stream));
}

size_t fgm_grouped_gemm_workspace_bytes(int64_t x_rows, int64_t R, int E, int N, int K)
{
    return gemm_sizes_ok(x_rows, R, E, N, K) ? gemm_ws(x_rows, K).total : 0;
}

int fgm_grouped_gemm(const uint16_t *x, int64_t x_stride, int64_t x_rows, const int32_t *src, int per, const int32_t *offsets,
                     const void *w, int w_type, const float *w_s, int E, int N, int K, uint16_t *out, int64_t R, void *ws,
                     size_t ws_bytes, void *stream)
{
    if (!gemm_sizes_ok(x_rows, R, E, N, K))
        return failf(FGM_ERR_INVALID_ARG, "x_rows = %lld, R = %lld (1 to 2^24), E = %d (1 to %d), N = %d, K = %d (1 to 65536, K a multiple of 8)",
                     (long long)x_rows, (long long)R, E, FGM_MAX_GROUPS, N, K);
    if (w_type != FGM_E4M3 && w_type != FGM_BF16)
        return failf(FGM_ERR_INVALID_ARG, "w_type = %d: FGM_E4M3 or FGM_BF16", w_type);
    if (w_type == FGM_E4M3 && K % 16)
        return failf(FGM_ERR_INVALID_ARG, "K = %d: a multiple of 16 with E4M3 weights", K);
    FGM_HOST_TRY(check_x(x, x_stride, K));
    if (per < 1)
        return failf(FGM_ERR_INVALID_ARG, "per = %d: at least 1", per);
    if (!src && x_rows != R)
        return failf(FGM_ERR_INVALID_ARG, "without rows x has R = %lld rows, not %lld", (long long)R, (long long)x_rows);
    if (!is_aligned(src, 4) || !is_aligned(w_s, 4))
        return failf(FGM_ERR_INVALID_ARG, "rows or w_s not 4-byte aligned");
    FGM_HOST_TRY(check_words("offsets", offsets));
    if (!w || !is_aligned(w, 16))
        return failf(FGM_ERR_INVALID_ARG, "w NULL or not 16-byte aligned");
    if (!out || !is_aligned(out, 2))
        return failf(FGM_ERR_INVALID_ARG, "out NULL or not aligned to an element");
    const bool bytes = w_type == FGM_E4M3;
    const GemmWs o = gemm_ws(x_rows, K);
    FGM_HOST_TRY(host_check_ws(ws, ws_bytes, bytes ? o.total : common_bytes()));      // (bf16 rows enter as they are)
    int sms = 0;
    FGM_HOST_TRY(host_device_ready(&sms));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    grouped::Maps m;
    FGM_HOST_TRY(weight_map(&m.w, w, bytes ? 1 : 2, E, N, K));
    m.w2 = m.w;
    const int64_t row = 2 * static_cast<int64_t>(bytes ? align_up(K, 32) : K);
    FGM_HOST_TRY(x_maps(m, bytes ? region<void>(ws, o.terms) : static_cast<const void *>(x), row, bytes ? row : 2 * x_stride, x_rows, src != nullptr));
    if (bytes)
        FGM_HOST_TRY(launch_overlapped(rows::k_terms, dim3(term_ctas(x_rows, K)), rows::kTermThreads, 0, st,
                                       rows::TermArgs{x, x_stride, x_rows, K, region<uint8_t>(ws, o.terms), region<float>(ws, o.xs)}));
    grouped::Args a = {};
    a.offsets = offsets;
    a.E = E;
    a.R = R;
    a.src = src;
    a.per = per;
    a.x_rows = static_cast<int>(x_rows);
    a.N = N;
    a.K = K;
    a.s0 = w_s;
    a.xs = bytes ? region<float>(ws, o.xs) : nullptr;
    a.out = out;
    a.wide = N % 8 == 0 && is_aligned(out, 16);
    a.cols = tile_cols(R, E, 256);
    a.status = status_word(ws);
    a.timeout_ns = host_wait_limit_ns();
    return bytes ? launch_grouped<grouped::kGemm, true>(m, a, sms, st)
                 : launch_grouped<grouped::kGemm, false>(m, a, sms, st);
}

size_t fgm_moe_experts_workspace_bytes(int64_t T) { return T < 1 || T > kMaxT ? 0 : experts_ws(T).total; }

int fgm_moe_experts_fwd(const fgm_layer *layer, const uint16_t *x, int64_t x_stride, int64_t T, const int32_t *ids, const float *w,
                        int shared, uint16_t *y, void *ws, size_t ws_bytes, void *stream)
{
    if (!layer)
        return failf(FGM_ERR_INVALID_ARG, "layer is NULL");
    FGM_HOST_TRY(check_tokens(T));
    const void *codes[3] = {layer->gate_q, layer->up_q, layer->down_q};
    for (const void *q : codes)
        if (!q || !is_aligned(q, 16))
            return failf(FGM_ERR_INVALID_ARG, "gate_q, up_q or down_q NULL or not 16-byte aligned");
    FGM_HOST_TRY(check_words("gate_s", layer->gate_s));
    FGM_HOST_TRY(check_words("up_s", layer->up_s));
    FGM_HOST_TRY(check_words("down_s", layer->down_s));
    FGM_HOST_TRY(check_x(x, x_stride, kH));
    FGM_HOST_TRY(check_words("ids", ids));
    FGM_HOST_TRY(check_words("w", w));
    if (!y || !is_aligned(y, 16))
        return failf(FGM_ERR_INVALID_ARG, "y NULL or not 16-byte aligned");
    const ExpertsWs o = experts_ws(T);
    FGM_HOST_TRY(host_check_ws(ws, ws_bytes, o.total));
    int sms = 0;
    FGM_HOST_TRY(host_device_ready(&sms));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int E = shared ? kNE : kE;
    const int64_t R = T * (shared ? kK + 1 : kK);
    grouped::Maps up, down;
    FGM_HOST_TRY(weight_map(&up.w, layer->gate_q, 1, kNE, kF, kH));
    FGM_HOST_TRY(weight_map(&up.w2, layer->up_q, 1, kNE, kF, kH));
    FGM_HOST_TRY(weight_map(&down.w, layer->down_q, 1, kNE, kH, kF));
    down.w2 = down.w;
    FGM_HOST_TRY(x_maps(up, region<void>(ws, o.terms), 2 * kH, 2 * kH, T, true));
    FGM_HOST_TRY(x_maps(down, region<void>(ws, o.act_terms), 2 * kF, 2 * kF, R, false));

    rows::PrepArgs prep = {};
    rows::GroupArgs &g = prep.group;
    g.ids = ids;
    g.n = T * kK;
    g.E = kE;
    g.count = region<int32_t>(ws, o.count);
    g.offsets = region<int32_t>(ws, o.offsets);
    g.src = region<int32_t>(ws, o.src);
    g.pos = region<int32_t>(ws, o.pos);
    g.per = kK;
    g.shared = shared ? static_cast<int>(T) : 0;
    cut_group(g);
    prep.terms = rows::TermArgs{x, x_stride, T, kH, region<uint8_t>(ws, o.terms), region<float>(ws, o.xs)};
    prep.down_s = layer->down_s;
    prep.smax = region<float>(ws, o.smax);
    FGM_HOST_TRY(launch_overlapped(rows::k_prep, dim3(g.chunks + kNE + term_ctas(T, kH)), 256, group_smem(kE), st, prep));
    if (g.chunks > 1)
        FGM_HOST_TRY(launch_deal(g, st));

    grouped::Args a = {};
    a.offsets = g.offsets;
    a.E = E;
    a.R = R;
    a.src = g.src;
    a.per = 1;
    a.x_rows = static_cast<int>(T);
    a.N = kF;
    a.K = kH;
    a.s0 = layer->gate_s;
    a.s1 = layer->up_s;
    a.xs = region<float>(ws, o.xs);
    a.out = region<uint16_t>(ws, o.rows);
    a.wide = 1;
    a.exps = region<uint8_t>(ws, o.exps);
    a.cols = tile_cols(T * kK, E, 128);
    a.status = status_word(ws);
    a.timeout_ns = host_wait_limit_ns();
    FGM_HOST_TRY((launch_grouped<grouped::kGated, true>(up, a, sms, st)));
    FGM_HOST_TRY(launch_overlapped(rows::k_act_terms, dim3(static_cast<unsigned>((R + 7) / 8)), rows::kTermThreads, 0, st, static_cast<const uint16_t *>(a.out), static_cast<const uint8_t *>(a.exps),
                                   a.offsets + E, R, region<uint8_t>(ws, o.act_terms), region<float>(ws, o.sa)));
    grouped::Args d = a;
    d.src = nullptr;
    d.x_rows = static_cast<int>(R);
    d.N = kH;
    d.K = kF;
    d.s0 = layer->down_s;
    d.s1 = nullptr;
    d.xs = nullptr;
    d.exps = nullptr;
    d.smax = region<float>(ws, o.smax);
    d.cols = tile_cols(T * kK, E, 256);
    FGM_HOST_TRY((launch_grouped<grouped::kDown, true>(down, d, sms, st)));
    const rows::CombineArgs c{d.out, region<float>(ws, o.sa), d.smax, ids, w, g.pos, g.offsets, shared ? 1 : 0, T, y, a.status, a.timeout_ns};
    static std::atomic<bool> ready[64];          // per device; setting it twice does no harm
    int dev = 0;
    FGM_HOST_CUDA(cudaGetDevice(&dev));
    if (!ready[dev & 63]) {
        FGM_HOST_CUDA(cudaFuncSetAttribute(rows::k_combine, cudaFuncAttributeMaxDynamicSharedMemorySize, rows::kCombineSmem));
        ready[dev & 63] = true;
    }
    return launch_overlapped(rows::k_combine, dim3(static_cast<unsigned>(T < sms ? T : sms)), rows::kCombineThreads, rows::kCombineSmem, st, c);
}

}  // extern "C"
