// C ABI of the log probabilities (declared in include/fgm.h): argument checks
// and launches of logprobs.cuh and lm_score.cuh.
#include <atomic>
#include <cmath>

#include "host.h"
#include "lm_score.cuh"
#include "logprobs.cuh"

namespace fgm {
namespace {

constexpr int64_t kMaxRows = 1 << 24;

bool score_sizes_ok(int64_t N, int64_t V, int k)
{
    return N >= 1 && N <= kMaxRows && V >= 1 && V <= 0x7FFFFFFFLL && k >= 0 && k <= FGM_MAX_TOP && k <= V;
}

int check_scores(int64_t N, int64_t V, float T, const int32_t *tokens, int k, const float *logp, const float *entropy,
                 const int32_t *top_ids, const float *top_logp)
{
    if (N < 1 || N > kMaxRows)
        return failf(FGM_ERR_INVALID_ARG, "N = %lld outside [1, 2^24]", (long long)N);
    if (V < 1 || V > 0x7FFFFFFFLL)
        return failf(FGM_ERR_INVALID_ARG, "V = %lld outside [1, 2^31)", (long long)V);
    if (k < 0 || k > FGM_MAX_TOP || k > V)
        return failf(FGM_ERR_INVALID_ARG, "k = %d outside [0, min(%d, V)]", k, FGM_MAX_TOP);
    if (!(T > 0.0f) || !std::isfinite(T) || !std::isfinite(1.0f / T))
        return failf(FGM_ERR_INVALID_ARG, "temperature T = %g: needs a finite T > 0 with 1/T finite", (double)T);
    if (logp && !tokens)
        return failf(FGM_ERR_INVALID_ARG, "logp without tokens");
    if (k > 0 && (!top_ids || !top_logp))
        return failf(FGM_ERR_INVALID_ARG, "top_ids/top_logp NULL with k = %d", k);
    if (!is_aligned(tokens, 4) || !is_aligned(logp, 4) || !is_aligned(entropy, 4) || !is_aligned(top_ids, 4) ||
        !is_aligned(top_logp, 4))
        return failf(FGM_ERR_INVALID_ARG, "tokens or an output not 4-byte aligned");
    return FGM_OK;
}

// Splits of a row. 608 CTAs run at a time (152 SMs, four each); a CTA's start and
// end (first loads, the k best, the sums) take about as long as 56 KB of its
// share of HBM, and the join of split rows as long as 80 KB: the number of splits
// that makes waves * (56 KB + a split's bytes) + 80 KB least. Measured: 1,013 rows
// of 100 KB, one split 28 us, four 51 us; 300 rows of 100 KB, one 13.9 us, two
// 17.0; 152 rows of 64 KB, one 7.7 us, three 10.0; 5 rows of 1 MB: 32. A split has
// 8,192 logits at least. A function of the sizes alone, so that results do not
// depend on the device.
int64_t most_row_splits(int64_t N, int64_t V)
{
    const int64_t by_grid = 8 * 608 / N + 1, by_size = V / 8192;
    const int64_t s = by_grid < by_size ? by_grid : by_size;
    return s < 1 ? 1 : s > 128 ? 128 : s;
}

int row_splits(int64_t N, int64_t V, int64_t elem)
{
    const int64_t most = most_row_splits(N, V);
    int64_t best = 1, cost = 0;
    for (int64_t s = 1; s <= most; ++s) {
        const int64_t c = (N * s + 607) / 608 * (56 * 1024 + V * elem / s) + (s > 1 ? 80 * 1024 : 0);
        if (s == 1 || c < cost) {
            best = s;
            cost = c;
        }
    }
    return static_cast<int>(best);
}

// Whether a warp takes a row: the same measure of both, a warp having an eighth of
// a CTA's share of HBM and 4,864 of them running at a time. Rows above 32 KB stay
// with a CTA, as the k best have a warp read k / 32 of its row again. Measured at
// k = 8 (warp : CTA, us): 4,864 fp32 rows of 8 KB 15 : 36, 16 KB 21 : 39, 24 KB
// 33 : 45, 32 KB 47 : 49, 48 KB 69 : 59, 64 KB 102 : 70; 2,500 rows of 32 KB 27 : 29,
// 48 KB 40 : 35. At k = 0 the warp is ahead to 48 KB (37 : 45); the choice is made
// for k > 0 and does not depend on it. Of 92 sizes (1 to 64 KB, 700 to 20,000 rows,
// fp32 and bf16) the rule's pick is 12 % slower than the other at worst (2,500 bf16
// rows of 24 KB, 34 : 31).
bool row_a_warp(int64_t N, int64_t V, int64_t elem)
{
    const int64_t bytes = V * elem;
    return bytes <= 32 * 1024 && row_splits(N, V, elem) == 1 &&
           (N + 4863) / 4864 * (56 * 1024 + 8 * bytes) < (N + 607) / 608 * (56 * 1024 + bytes);
}

size_t part_offset() { return align_up(ws_offsets().total, 256); }

score::Outs outs(const int32_t *tokens, float *logp, float *entropy, int32_t *top_ids, float *top_logp, int k, float T,
                 int64_t V, void *ws)
{
    return score::Outs{tokens, logp, entropy, top_ids, top_logp, k, T, V,
                       reinterpret_cast<int32_t *>(static_cast<char *>(ws) + ws_offsets().status)};
}

template <typename E>
int run_logprobs(const void *z, int64_t stride, int64_t N, const score::Outs &o, void *ws, cudaStream_t st)
{
    const int splits = row_splits(N, o.V, sizeof(E));
    score::Part *part = reinterpret_cast<score::Part *>(static_cast<char *>(ws) + part_offset());
    const E *zp = static_cast<const E *>(z);
    if (row_a_warp(N, o.V, sizeof(E)))
        return launch_overlapped(score::k_logprob_rows<E>, dim3(static_cast<unsigned>((N + score::kWarps - 1) / score::kWarps)),
                                 score::kThreads, 0, st, zp, stride, N, o);
    FGM_HOST_TRY(launch_overlapped(score::k_logprobs<E>, dim3(static_cast<unsigned>(N * splits)), score::kThreads, 0, st, zp,
                                   stride, splits, part, o));
    if (splits == 1)
        return FGM_OK;
    return launch_overlapped(score::k_logprob_join<E>, dim3(static_cast<unsigned>((N + score::kWarps - 1) / score::kWarps)),
                             score::kThreads, 0, st, zp, stride, N, splits, static_cast<const score::Part *>(part), o);
}

size_t logits_bytes(int64_t N, int64_t V) { return align_up(sizeof(float) * static_cast<size_t>(N) * V, 256); }

constexpr int kMaxPairs = 80;                  // CTA pairs of a full sm_103 part

int64_t row_tiles(int64_t N) { return (N + score::kLmRows - 1) / score::kLmRows; }

// Word ranges of a row tile of fgm_lm_head_logprobs on a device that runs `pairs`
// CTA pairs at a time: those that fill 1 to 4 waves of pairs, whichever makes
// waves * (a range's tiles + 1) least; an item's start and end cost about a tile.
// (How many pairs fit is asked of the device: 76 on one with 152 SMs.)
int word_splits(int64_t N, int64_t V, int pairs)
{
    const int64_t tiles = (V + score::kLmWords - 1) / score::kLmWords, rows = row_tiles(N);
    int64_t best = 1, cost = 0;
    for (int w = 1; w <= 4; ++w) {
        int64_t s = w * pairs / rows;
        s = s < 1 ? 1 : s > tiles ? tiles : s;
        const int64_t c = (rows * s + pairs - 1) / pairs * ((tiles + s - 1) / s + 1);
        if (w == 1 || c < cost) {
            best = s;
            cost = c;
        }
    }
    return static_cast<int>(best);
}

// The most ranges that word_splits gives on any device.
int64_t most_splits(int64_t N) { return N <= score::kLmRows ? kMaxPairs : 4 * kMaxPairs / row_tiles(N) + 1; }

template <int L>
int run_lm_score(const uint16_t *emb, const uint16_t *h, score::LmArgs &a, const score::Outs &o, int sms, cudaStream_t st)
{
    CUtensorMap hmap, emap;
    a.h_rows = a.N < 128 ? static_cast<int>(align_up(a.N, 8)) : 128;
    const int stage = score::kLmBoxes * (a.h_rows * 128 + score::kLmBox), fit = (score::kLmSmem - 1024) / stage;
    a.stages = fit < score::kLmStages ? fit : score::kLmStages;
    FGM_HOST_TRY(host_hidden_map(&hmap, h, a.N, a.h_rows, score::kLmBoxes));
    FGM_HOST_TRY(host_hidden_map(&emap, emb, a.V, 128, score::kLmBoxes));
    static std::atomic<int> fit_pairs[64];     // CTA pairs at a time, per device; finding it twice does no harm
    int dev = 0;
    FGM_HOST_CUDA(cudaGetDevice(&dev));
    int most = fit_pairs[dev & 63];
    if (!most) {
        FGM_HOST_CUDA(cudaFuncSetAttribute(score::k_lm_score<L>, cudaFuncAttributeMaxDynamicSharedMemorySize, score::kLmSmem));
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(sms / 2 * 2);
        cfg.blockDim = dim3(score::kLmThreads);
        cfg.dynamicSmemBytes = score::kLmSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        FGM_HOST_CUDA(cudaOccupancyMaxActiveClusters(&most, score::k_lm_score<L>, &cfg));
        if (most < 1)
            return failf(FGM_ERR_DEVICE, "no CTA pair of the lm_head kernel fits this device");
        most = most < kMaxPairs ? most : kMaxPairs;
        fit_pairs[dev & 63] = most;
    }
    a.splits = word_splits(a.N, a.V, most);
    a.items = row_tiles(a.N) * a.splits;
    const int64_t pairs = a.items < most ? a.items : most;
    FGM_HOST_TRY(launch_overlapped(score::k_lm_score<L>, dim3(static_cast<unsigned>(2 * pairs)), score::kLmThreads,
                                   score::kLmSmem, st, hmap, emap, a));
    return launch_overlapped(score::k_lm_join<L>, dim3(static_cast<unsigned>(a.N)), 32 * score::kJoinWarps, 0, st, emb, h, a, o);
}

}  // namespace
}  // namespace fgm

using namespace fgm;

extern "C" {

size_t fgm_logprobs_workspace_bytes(int64_t N, int64_t V, int k)
{
    if (!score_sizes_ok(N, V, k))
        return 0;
    const int64_t s = most_row_splits(N, V);
    return align_up(part_offset() + (s == 1 ? 0 : sizeof(score::Part) * static_cast<size_t>(N) * s), 256);
}

int fgm_logprobs(const void *z, int dtype, int64_t row_stride, int64_t N, int64_t V, float T, const int32_t *tokens,
                 int k, float *logp, float *entropy, int32_t *top_ids, float *top_logp, void *ws, size_t ws_bytes,
                 void *stream)
{
    FGM_HOST_TRY(check_scores(N, V, T, tokens, k, logp, entropy, top_ids, top_logp));
    if (dtype != FGM_F32 && dtype != FGM_BF16 && dtype != FGM_F16)
        return failf(FGM_ERR_INVALID_ARG, "dtype = %d: FGM_F32, FGM_BF16 or FGM_F16", dtype);
    if (!z || !is_aligned(z, dtype == FGM_F32 ? 4 : 2))
        return failf(FGM_ERR_INVALID_ARG, "z NULL or not aligned to an element");
    if (row_stride < V || row_stride > (int64_t(1) << 40))
        return failf(FGM_ERR_INVALID_ARG, "row_stride = %lld below V = %lld or above 2^40", (long long)row_stride, (long long)V);
    FGM_HOST_TRY(host_check_ws(ws, ws_bytes, fgm_logprobs_workspace_bytes(N, V, k)));
    FGM_HOST_TRY(host_device_ready(nullptr));
    const score::Outs o = outs(tokens, logp, entropy, top_ids, top_logp, k, T, V, ws);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (dtype) {
    case FGM_F32: return run_logprobs<float>(z, row_stride, N, o, ws, st);
    case FGM_BF16: return run_logprobs<__nv_bfloat16>(z, row_stride, N, o, ws, st);
    default: return run_logprobs<__half>(z, row_stride, N, o, ws, st);
    }
}

size_t fgm_lm_head_logprobs_workspace_bytes(int64_t N, int64_t V, int k)
{
    if (!score_sizes_ok(N, V, k))
        return 0;
    if (N <= kMaxM)
        return fgm_logprobs_workspace_bytes(N, V, k) + logits_bytes(N, V);
    return align_up(part_offset() + sizeof(score::Part) * 2 * static_cast<size_t>(N) * most_splits(N), 256);
}

int fgm_lm_head_logprobs(const uint16_t *emb, int64_t V, const uint16_t *h, int64_t N, float T, const int32_t *tokens,
                         int k, float *logp, float *entropy, int32_t *top_ids, float *top_logp, void *ws,
                         size_t ws_bytes, void *stream)
{
    FGM_HOST_TRY(check_scores(N, V, T, tokens, k, logp, entropy, top_ids, top_logp));
    if (!emb || !is_aligned(emb, 16) || !h || !is_aligned(h, 16))
        return failf(FGM_ERR_INVALID_ARG, "emb/h NULL or not 16-byte aligned");
    FGM_HOST_TRY(host_check_ws(ws, ws_bytes, fgm_lm_head_logprobs_workspace_bytes(N, V, k)));
    int sms = 0;
    FGM_HOST_TRY(host_device_ready(&sms));
    const score::Outs o = outs(tokens, logp, entropy, top_ids, top_logp, k, T, V, ws);
    if (N <= kMaxM) {
        // The persistent lm_head kernel, whose whole-row copies stream the embedding at 6.8 TB/s where the pair
        // kernel's boxes reach 5.9 (5 rows 217 us, 9 rows 251), with its logits (0.4 % of the bytes) scored by k_logprobs.
        char *z = static_cast<char *>(ws) + fgm_logprobs_workspace_bytes(N, V, k);
        FGM_HOST_TRY(host_lm_logits(emb, V, h, static_cast<int>(N), reinterpret_cast<float *>(z), ws, stream));
        return run_logprobs<float>(z, V, N, o, ws, static_cast<cudaStream_t>(stream));
    }
    score::LmArgs a = {};
    a.N = N;
    a.V = static_cast<int>(V);
    a.T = T;
    a.part = reinterpret_cast<score::Part *>(static_cast<char *>(ws) + part_offset());
    a.status = o.status;
    a.timeout_ns = host_wait_limit_ns();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return k <= 8 ? run_lm_score<12>(emb, h, a, o, sms, st) : run_lm_score<20>(emb, h, a, o, sms, st);
}

}  // extern "C"
