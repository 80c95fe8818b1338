// C ABI of the log probabilities (declared in include/fgm.h): argument checks
// and launches of logprobs.cuh.
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
// share of HBM: the number of splits that makes waves * (56 KB + a split's bytes)
// least. 1,013 rows of 100 KB: one split 28 us, four 51 us (measured); 600 rows
// of 1 MB: one; 5 rows of 1 MB: 32. A split has 8,192 logits at least. A function
// of the sizes alone, so that results do not depend on the device.
int row_splits(int64_t N, int64_t V, int64_t elem)
{
    const int64_t most = V / 8192;
    int64_t best = 1, cost = 0;
    for (int64_t s = 1; s == 1 || (s <= most && s <= 128); ++s) {
        const int64_t c = (N * s + 607) / 608 * (56 * 1024 + V * elem / s);
        if (s == 1 || c < cost) {
            best = s;
            cost = c;
        }
    }
    return static_cast<int>(best);
}

size_t part_offset() { return align_up(ws_offsets().total, 256); }

score::Outs outs(const int32_t *tokens, float *logp, float *entropy, int32_t *top_ids, float *top_logp, int k, float T,
                 int64_t V, void *ws)
{
    return score::Outs{tokens, logp, entropy, top_ids, top_logp, k, T, V,
                       reinterpret_cast<int32_t *>(static_cast<char *>(ws) + ws_offsets().status)};
}

template <typename E>
int launch_join(const E *z, int64_t stride, const float *ztok, int64_t N, int splits, const score::Part *part,
                const score::Outs &o, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((N + score::kWarps - 1) / score::kWarps));
    cfg.blockDim = dim3(score::kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    FGM_HOST_CUDA(cudaLaunchKernelEx(&cfg, score::k_logprob_join<E>, z, stride, ztok, N, splits, part, o));
    return FGM_OK;
}

template <typename E>
int run_logprobs(const void *z, int64_t stride, int64_t N, const score::Outs &o, void *ws, cudaStream_t st)
{
    const int splits = row_splits(N, o.V, sizeof(E));
    score::Part *part = reinterpret_cast<score::Part *>(static_cast<char *>(ws) + part_offset());
    score::k_logprobs<E><<<static_cast<unsigned>(N * splits), score::kThreads, 0, st>>>(static_cast<const E *>(z), stride,
                                                                                         splits, part, o);
    FGM_HOST_CUDA(cudaGetLastError());
    return splits == 1 ? FGM_OK : launch_join<E>(static_cast<const E *>(z), stride, nullptr, N, splits, part, o, st);
}

// Word ranges of a row tile of fgm_lm_head_logprobs: the number that makes waves *
// (a range's tiles + 1) least, for the 76 pairs of a 152-SM part; an item's start
// and end cost about one tile.
int word_splits(int64_t N, int64_t V)
{
    const int64_t tiles = (V + score::kLmWords - 1) / score::kLmWords, rows = (N + score::kLmRows - 1) / score::kLmRows;
    int64_t best = 1, cost = 0;
    for (int64_t s = 1; s <= tiles && s <= 152; ++s) {
        const int64_t c = (rows * s + 75) / 76 * ((tiles + s - 1) / s + 1);
        if (s == 1 || c < cost) {
            best = s;
            cost = c;
        }
    }
    return static_cast<int>(best);
}

// The regions behind the common workspace: partial results, the given tokens' logits.
struct LmWs {
    size_t part, ztok, total;
};

LmWs lm_ws(int64_t N, int64_t V)
{
    LmWs o;
    o.part = part_offset();
    o.ztok = align_up(o.part + sizeof(score::Part) * static_cast<size_t>(N) * word_splits(N, V), 256);
    o.total = align_up(o.ztok + sizeof(float) * static_cast<size_t>(N), 256);
    return o;
}

}  // namespace
}  // namespace fgm

using namespace fgm;

extern "C" {

size_t fgm_logprobs_workspace_bytes(int64_t N, int64_t V, int k)
{
    if (!score_sizes_ok(N, V, k))
        return 0;
    const int s4 = row_splits(N, V, 4), s2 = row_splits(N, V, 2), s = s4 > s2 ? s4 : s2;
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
    return score_sizes_ok(N, V, k) ? lm_ws(N, V).total : 0;
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
    CUtensorMap hmap, emap;
    FGM_HOST_TRY(host_hidden_map(&hmap, h, N));
    FGM_HOST_TRY(host_hidden_map(&emap, emb, V));
    const LmWs w = lm_ws(N, V);
    const score::Outs o = outs(tokens, logp, entropy, top_ids, top_logp, k, T, V, ws);
    score::LmArgs a = {};
    a.N = N;
    a.V = static_cast<int>(V);
    a.tokens = tokens;
    a.T = T;
    a.k = k;
    a.splits = word_splits(N, V);
    a.items = (N + score::kLmRows - 1) / score::kLmRows * a.splits;
    a.part = reinterpret_cast<score::Part *>(static_cast<char *>(ws) + w.part);
    a.ztok = reinterpret_cast<float *>(static_cast<char *>(ws) + w.ztok);
    a.status = o.status;
    a.timeout_ns = host_wait_limit_ns();
    static bool ready[64];                     // per device; setting it twice does no harm
    int dev = 0;
    FGM_HOST_CUDA(cudaGetDevice(&dev));
    if (!ready[dev & 63]) {
        FGM_HOST_CUDA(cudaFuncSetAttribute(score::k_lm_score, cudaFuncAttributeMaxDynamicSharedMemorySize, score::kLmSmem));
        ready[dev & 63] = true;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t pairs = a.items < sms / 2 ? a.items : sms / 2;
    score::k_lm_score<<<static_cast<unsigned>(2 * pairs), score::kLmThreads, score::kLmSmem, st>>>(hmap, emap, a);
    FGM_HOST_CUDA(cudaGetLastError());
    return launch_join<float>(nullptr, 0, a.ztok, N, a.splits, a.part, o, st);
}

}  // extern "C"
