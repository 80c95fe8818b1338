// C ABI of the block norms (declared in include/fgm.h): argument checks and launches
// of block_norm.cuh.
#include <atomic>
#include <cmath>

#include "block_norm.cuh"
#include "host.h"

namespace fgm {
namespace {

constexpr int kNormSmem = 226 * 1024;            // dynamic shared memory at most

int64_t elem_bytes(int type) { return type == FGM_F32 ? 4 : 2; }
bool type_ok(int type) { return type == FGM_F32 || type == FGM_BF16 || type == FGM_F16; }

// The bytes of a tensor's rows: `rows` of them, `width` bytes each, `stride` bytes apart.
struct Span {
    uintptr_t at;
    int64_t rows, stride, width;
};

Span span(const void *p, int64_t rows, int64_t stride, int64_t cols, int type)
{
    return Span{reinterpret_cast<uintptr_t>(p), rows, stride * elem_bytes(type), cols * elem_bytes(type)};
}

bool same(const Span &a, const Span &b) { return a.at == b.at && a.width == b.width && (a.rows == 1 || a.stride == b.stride); }

// Whether two tensors share no byte: apart, or interleaved rows at one stride.
bool apart(const Span &a, const Span &b)
{
    const uintptr_t a1 = a.at + (a.rows - 1) * a.stride + a.width, b1 = b.at + (b.rows - 1) * b.stride + b.width;
    if (a1 <= b.at || b1 <= a.at)
        return true;
    // (a single row goes with any stride)
    const int64_t s = a.rows == 1 ? b.stride : a.stride;
    if ((b.rows != 1 && b.stride != s) || s <= 0)
        return false;
    const int64_t d = a.at <= b.at ? static_cast<int64_t>((b.at - a.at) % s) : static_cast<int64_t>((s - (a.at - b.at) % s) % s);
    return d >= a.width && d + b.width <= s;
}

int check_tensor(const char *name, const void *p, int type, int64_t stride, int D)
{
    if (!type_ok(type))
        return failf(FGM_ERR_INVALID_ARG, "%s: type %d is not FGM_F32, FGM_BF16 or FGM_F16", name, type);
    if (!p || !is_aligned(p, elem_bytes(type)))
        return failf(FGM_ERR_INVALID_ARG, "%s NULL or not aligned to an element", name);
    if (stride < D || stride > (int64_t(1) << 32))
        return failf(FGM_ERR_INVALID_ARG, "%s: stride %lld below D = %d or above 2^32", name, (long long)stride, D);
    return FGM_OK;
}

bool wide(const void *p, int64_t stride, int type) { return !p || (is_aligned(p, 16) && stride * elem_bytes(type) % 16 == 0); }

// CTAs of a kernel at a time on this device; found once per device (twice does no harm) for its most shared memory and asked for less.
template <typename K>
int norm_grid(K kernel, std::atomic<bool> (&ready)[64], int threads, size_t smem, int sms, int64_t N, int64_t *grid)
{
    int dev = 0, each = 0;
    FGM_HOST_CUDA(cudaGetDevice(&dev));
    if (!ready[dev & 63]) {
        FGM_HOST_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem));
        ready[dev & 63] = true;
    }
    *grid = N;
    if (N > sms) {
        FGM_HOST_CUDA(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&each, kernel, threads, smem));
        *grid = N < static_cast<int64_t>(each) * sms ? N : static_cast<int64_t>(each) * sms;
    }
    return FGM_OK;
}

size_t gain_bytes(const norm::Args &a) { return sizeof(float) * (a.pre ? 2 : a.post ? 1 : 0) * a.D; }

template <int VPT, int STAGES>
int launch_staged(norm::Args &a, int threads, size_t row, int sms, cudaStream_t st)
{
    static std::atomic<bool> ready[64];
    int64_t grid = 0;
    a.keep = STAGES * row + gain_bytes(a) <= kNormSmem;
    const size_t smem = STAGES * row + (a.keep ? gain_bytes(a) : 0);
    FGM_HOST_TRY(norm_grid(norm::k_block_norm<VPT, STAGES>, ready, threads, smem, sms, a.N, &grid));
    return launch_overlapped(norm::k_block_norm<VPT, STAGES>, dim3(static_cast<unsigned>(grid)), threads, smem, st, a);
}

// Three rows in shared memory, or one where three do not fit.
template <int VPT>
int launch_norm(norm::Args &a, int sms, cudaStream_t st)
{
    const int threads = (a.D + 256 * VPT - 1) / (256 * VPT) * 32, n = threads * VPT;
    const size_t row = norm::piece_bytes(a.y, a.y.type, n) + norm::piece_bytes(a.h, a.h.type, n) + norm::piece_bytes(a.gate, a.gate.type, n);
    if (3 * row + gain_bytes(a) <= kNormSmem)
        return launch_staged<VPT, 3>(a, threads, row, sms, st);
    return launch_staged<VPT, 1>(a, threads, row, sms, st);
}

template <bool F32>
int launch_usual(const norm::Args &a, int sms, cudaStream_t st)
{
    static std::atomic<bool> ready[64];
    int64_t grid = 0;
    const int threads = (a.D + 255) / 256 * 32;
    const bool scaled = a.post || (a.gate.p && a.gate.step);
    const size_t smem = threads * (norm::kUsualStages * (F32 ? 48 : 32) + 32 * (a.pre ? 2 : scaled ? 1 : 0));
    FGM_HOST_TRY(norm_grid(norm::k_block_norm_usual<F32>, ready, threads, smem, sms, a.N, &grid));
    return launch_overlapped(norm::k_block_norm_usual<F32>, dim3(static_cast<unsigned>(grid)), threads, smem, st, a);
}

template <bool F32, bool GATE>
int launch_odd(const norm::Args &a, int sms, cudaStream_t st)
{
    static std::atomic<bool> ready[64];
    int64_t grid = 0;
    const int threads = (a.D + 32 * norm::kOddVals - 1) / (32 * norm::kOddVals) * 32;
    FGM_HOST_TRY(norm_grid(norm::k_block_norm_odd<F32, GATE>, ready, threads, 0, sms, a.N, &grid));
    return launch_overlapped(norm::k_block_norm_odd<F32, GATE>, dim3(static_cast<unsigned>(grid)), threads, 0, st, a);
}

template <int VPT>
int launch_any(norm::Args &a, int sms, cudaStream_t st)
{
    static std::atomic<bool> ready[64];
    int64_t grid = 0;
    const int threads = (a.D + 32 * VPT - 1) / (32 * VPT) * 32;
    a.keep = 1;
    const size_t smem = gain_bytes(a);
    FGM_HOST_TRY(norm_grid(norm::k_block_norm_any<VPT>, ready, threads, smem, sms, a.N, &grid));
    return launch_overlapped(norm::k_block_norm_any<VPT>, dim3(static_cast<unsigned>(grid)), threads, smem, st, a);
}

}  // namespace
}  // namespace fgm

using namespace fgm;

extern "C" int fgm_block_norm(const fgm_block *b, void *stream)
{
    if (!b)
        return failf(FGM_ERR_INVALID_ARG, "block is NULL");
    if (b->N < 1 || b->N > 0x7FFFFFFFLL)
        return failf(FGM_ERR_INVALID_ARG, "N = %lld outside [1, 2^31)", (long long)b->N);
    if (b->D < 1 || b->D > 16384)
        return failf(FGM_ERR_INVALID_ARG, "D = %d outside [1, 16384]", b->D);
    if (!std::isfinite(b->residual_scale) || !std::isfinite(b->block_scale) || !std::isfinite(b->gain_offset) || !std::isfinite(b->eps) || b->eps < 0)
        return failf(FGM_ERR_INVALID_ARG, "scales and gain_offset must be finite, eps finite and not negative");
    if (!b->h_out && !b->xn)
        return failf(FGM_ERR_INVALID_ARG, "h_out and xn both NULL: no output");
    FGM_HOST_TRY(check_tensor("h", b->h, b->h_type, b->h_stride, b->D));
    if (b->y)
        FGM_HOST_TRY(check_tensor("y", b->y, b->y_type, b->y_stride, b->D));
    if (!b->y && (b->gate || b->post_gain))
        return failf(FGM_ERR_INVALID_ARG, "gate or post_gain without y");
    if (b->post_gain && !b->post_norm)
        return failf(FGM_ERR_INVALID_ARG, "post_gain without post_norm");
    if (b->pre_gain && !b->xn)
        return failf(FGM_ERR_INVALID_ARG, "pre_gain without xn");
    if (b->h_out)
        FGM_HOST_TRY(check_tensor("h_out", b->h_out, b->h_type, b->h_out_stride, b->D));
    if (b->xn)
        FGM_HOST_TRY(check_tensor("xn", b->xn, b->xn_type, b->xn_stride, b->D));
    const int64_t gate_cols = b->gate_col_stride ? b->D : 1;
    if (b->gate) {
        if (!type_ok(b->gate_type) || !is_aligned(b->gate, elem_bytes(b->gate_type)))
            return failf(FGM_ERR_INVALID_ARG, "gate: type %d, or not aligned to an element", b->gate_type);
        if (b->gate_col_stride != 0 && b->gate_col_stride != 1)
            return failf(FGM_ERR_INVALID_ARG, "gate_col_stride = %d: 0 or 1", b->gate_col_stride);
        if (b->gate_row_stride != 0 && (b->gate_row_stride < gate_cols || b->gate_row_stride > (int64_t(1) << 32)))
            return failf(FGM_ERR_INVALID_ARG, "gate_row_stride = %lld: 0, or at least %lld and at most 2^32", (long long)b->gate_row_stride, (long long)gate_cols);
    }
    const void *gains[2] = {b->post_gain, b->pre_gain};
    for (const void *g : gains)
        if (g && (!type_ok(b->gain_type) || !is_aligned(g, elem_bytes(b->gain_type))))
            return failf(FGM_ERR_INVALID_ARG, "gains: type %d, or not aligned to an element", b->gain_type);
    // outputs: no byte of theirs is another tensor's, but for rows taken over whole
    const Span h = span(b->h, b->N, b->h_stride, b->D, b->h_type), y = span(b->y, b->N, b->y_stride, b->D, b->y_type),
               ho = span(b->h_out, b->N, b->h_out_stride, b->D, b->h_type), xn = span(b->xn, b->N, b->xn_stride, b->D, b->xn_type),
               gate = span(b->gate, b->gate_row_stride ? b->N : 1, b->gate_row_stride, gate_cols, b->gate_type);
    bool clash = false;
    if (b->h_out)
        clash |= !(same(ho, h) || apart(ho, h)) || (b->y && !apart(ho, y)) || (b->gate && !apart(ho, gate)) || (b->xn && !apart(ho, xn));
    if (b->xn)
        clash |= !(same(xn, h) || apart(xn, h)) || (b->y && !(same(xn, y) || apart(xn, y))) || (b->gate && !apart(xn, gate));
    for (const void *g : gains)
        if (g) {
            const Span s = span(g, 1, 0, b->D, b->gain_type);
            clash |= (b->h_out && !apart(ho, s)) || (b->xn && !apart(xn, s));
        }
    if (clash)
        return failf(FGM_ERR_INVALID_ARG, "an output overlaps another tensor (h_out may be h; xn may be y or h)");
    int sms = 0;
    FGM_HOST_TRY(host_device_ready(&sms));

    norm::Args a = {};
    a.h = {const_cast<void *>(b->h), b->h_stride, b->h_type, 1};
    a.y = {const_cast<void *>(b->y), b->y_stride, b->y_type, 1};
    a.gate = {const_cast<void *>(b->gate), b->gate_row_stride, b->gate_type, b->gate_col_stride};
    a.h_out = {b->h_out, b->h_out_stride, b->h_type, 1};
    a.xn = {b->xn, b->xn_stride, b->xn_type, 1};
    a.post = b->post_gain;
    a.pre = b->pre_gain;
    a.gain_type = b->gain_type;
    a.N = b->N;
    a.D = b->D;
    a.post_norm = b->post_norm;
    a.a = b->residual_scale;
    a.b = b->block_scale;
    a.offset = b->gain_offset;
    a.eps = b->eps;
    a.per_d = 1.0f / b->D;
    const bool vec = b->D % 8 == 0 && wide(b->h, b->h_stride, b->h_type) && wide(b->y, b->y_stride, b->y_type) &&
                     (!b->gate_col_stride || wide(b->gate, b->gate_row_stride, b->gate_type)) && wide(b->h_out, b->h_out_stride, b->h_type) &&
                     wide(b->xn, b->xn_stride, b->xn_type) && wide(b->post_gain, 0, b->gain_type) && wide(b->pre_gain, 0, b->gain_type);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (vec) {
        const bool usual = b->D <= 8 * norm::kUsualThreads && (!b->y || b->y_type == FGM_BF16) && (!b->xn || b->xn_type == FGM_BF16) &&
                           (!b->gate || !b->gate_col_stride || !b->gate_row_stride || b->N == 1);
        if (usual && b->h_type == FGM_BF16)
            return launch_usual<false>(a, sms, st);
        if (usual && b->h_type == FGM_F32)
            return launch_usual<true>(a, sms, st);
        return b->D <= 8192 ? launch_norm<1>(a, sms, st) : launch_norm<2>(a, sms, st);
    }
    if (b->D > 4096)
        return launch_any<16>(a, sms, st);
    const bool full = b->gate && b->gate_col_stride && b->gate_row_stride,
               usual = (!b->y || b->y_type == FGM_BF16) && (!b->xn || b->xn_type == FGM_BF16) && (!full || b->gate_type == FGM_BF16);
    if (usual && b->h_type == FGM_BF16)
        return full ? launch_odd<false, true>(a, sms, st) : launch_odd<false, false>(a, sms, st);
    if (usual && b->h_type == FGM_F32)
        return full ? launch_odd<true, true>(a, sms, st) : launch_odd<true, false>(a, sms, st);
    return launch_any<4>(a, sms, st);
}
