// Matrix products grouped by expert (fgm_grouped_gemm, and the two products of
// fgm_moe_experts_fwd): with rows [off[e], off[e + 1]) belonging to expert e,
//   D[n][r] = sum_k W_e[n][k] x[src(r)][k],
// W_e in E4M3 codes or bf16, x in bf16.
//
// 8-bit weights go to the tensor pipe as they are stored. An activation enters as
// two E4M3 terms under a power of two per row, t1 = e4m3(x / s), t2 = e4m3(x / s - t1):
// a bf16 number has 8 significant bits and a term 4, so t1 + t2 is x / s exactly
// where that is 1/4 or more, else to 2^-10 (s puts the row's largest element into
// [128, 256), moe_rows.cuh). Two 8-bit products take as long as one bf16 product would,
// and the weights as half the bytes, without a conversion anywhere. A third term would cost half
// the products' time again, and a prompt's are bound by it; the experts' outputs are 1.8e-3 off 64 bits
// (root mean square), of which their own rounding to bf16 is 1.65e-3.
//
// 2 N K operations a row: bound by the weights' bytes while experts have few rows (208
// rows on 128 experts of 1408 x 2816 take 87 us, 5.8 TB/s), by the tensor pipe from a few
// hundred a piece on (32,768 rows on 8 experts of 2816 x 2816 336 us with their terms,
// 1.55 PFLOP/s, in bf16 281 us, 1.85; a 16,381-token prompt's gate and up products 737 us, 1.6;
// its down products, whose 704 of K end a tile every 6 stages, 414 us, 1.4). Weights are the products' first operand:
//  * A pair of CTAs (cta_group::2) holds 256 features x up to 256 rows (gate and up: two
//    such products of up to 128 rows) in one of two halves of tensor memory; an expert's
//    rows are cut into equal tiles, whose width is the products' N, so that a few rows
//    cost few columns. Each CTA copies its 128 features and half of the rows.
//  * Stages of 128 elements of K in the 128-byte swizzle, as many as fit. A row brings 128
//    bytes with both terms of 64 elements (blocks of 32 of one and then of the other).
//    Gathered rows come four a copy (tile::gather4) from six warps' lanes, the others in
//    boxes of 8 to 128; a copy costs its warp some 80 cycles, whatever it brings
//    (32,768 gathered rows of 2816 on 2816 features of 128 experts: 1103 us by one warp in the
//    first kernel, 404 now; in order 369).
//  * Both terms' products take the weights from one reading (collector::a).
//  * Tiles of an expert go feature by feature, so that its rows are read from HBM once
//    and its weights stay in L2 (rows first: 412 us where 344).
//  * Sixteen epilogue warps; accumulators are read as products hold them, scaled,
//    rounded to 16 bits, transposed by stmatrix and stored in whole lines.
#pragma once

#include <cuda.h>

#include "pair_copies.h"
#include "tensor.cuh"

namespace fgm {
namespace grouped {

constexpr int kSides = 4;                        // epilogue warps of a 32-lane quarter, which share out its columns
constexpr int kEpilogue = 4 * kSides;
constexpr int kThreads = 128 + 32 * kEpilogue;   // weights, products, rows (two warps), epilogue,
constexpr int kGatherThreads = kThreads + 128;   // and four more warps for rows where they are gathered
constexpr int kGatherWarps = 6;
constexpr int kMaxStages = 12;
constexpr int kMaxExperts = 1024;
constexpr int kStageK = 128;                     // elements of K in a stage
constexpr int kBox = 128 * 128;                  // 128 weight rows x 128 bytes
constexpr int kRing = 192 * 1024;                // bytes of the ring at most
constexpr int kOutRow = 256 + 16;                // 128 features of a row on their way out (and 16 bytes: rows begin in other banks),
constexpr int kOutBuf = 8 * kOutRow;             // eight rows, twice for each side
constexpr int kOutBytes = kSides * 2 * kOutBuf;
constexpr int kSmem = kRing + kOutBytes + 1024;

enum Mode {
    kGemm = 0,   // out[r][n] = bf16(s[n] xs[r] D)
    kGated = 1,  // a[r][n] = gelu(s_g[n] xs[r] D_g) * (s_u[n] xs[r] D_u), f16 under a power of two per 32 of n
    kDown = 2,   // y[r][n] = f16(s[n] / smax[e] 2^-12 D)
};

struct Args {
    const int32_t *offsets;  // [E + 1]
    int E;
    int64_t R;               // rows at most
    const int32_t *src;      // row r takes x row src[r] / per; NULL: x row r
    int per;
    int x_rows;
    int N, K;
    const float *s0, *s1;    // [E][N] row scales (gate and up), or NULL
    const float *xs;         // [x_rows] scales of the terms
    uint16_t *out;           // [R][N]
    uint8_t *exps;           // kGated: [R][N / 32] exponents
    const float *smax;       // kDown: [E] a power of two not below the expert's scales
    int wide;                // 16-byte stores to out
    int cols, log_cols;      // rows of a tile at most: a power of two, 32 to 256
    int stages;
    int32_t *status;
    long long timeout_ns;
};

struct Shared {
    unsigned long long full[kMaxStages], empty[kMaxStages], tfull[2], tempty[2], drained;
    uint32_t tmem;
    int abort;
    uint32_t issued, passed;  // stages that the weights' warp has copied for at the end, and up to the first one of its tile, found free
    uint32_t bytes[kMaxStages];                  // of a CTA in each stage
    uint32_t rows_issued[kGatherWarps];          // stages that each rows' warp has copied for at the end,
    score::TileNote sent[kGatherWarps][kMaxStages];          // and its last tiles
    int row0[kMaxExperts], count[kMaxExperts], cum[kMaxExperts + 1];   // rows and tiles before, by expert
};

// Weight boxes of a stage: gate and up rows, or one of 8-bit rows (128 of K), or two of bf16 (64 of K each).
template <Mode MODE, bool BYTES>
__host__ __device__ constexpr int weight_boxes() { return MODE == kGated || !BYTES ? 2 : 1; }

// Bytes of a stage whose tiles have up to `cols` rows (half of them in each CTA, 2 x 128 bytes a row).
template <Mode MODE, bool BYTES>
__host__ __device__ constexpr int stage_bytes(int cols) { return weight_boxes<MODE, BYTES>() * kBox + cols * 128; }

__device__ __forceinline__ void copy_weights(uint32_t dst, const CUtensorMap *map, int k, int n, int e, uint32_t bar, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(k), "r"(n), "r"(e), "r"(bar), "l"(policy)
        : "memory");
}

// A box of rows x 128 bytes,
__device__ __forceinline__ void copy_rows(uint32_t dst, const CUtensorMap *map, int at, int row, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(at), "r"(row), "r"(bar)
        : "memory");
}

// or four rows anywhere.
__device__ __forceinline__ void copy_gathered(uint32_t dst, const CUtensorMap *map, int at, int4 rows, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(at), "r"(rows.x), "r"(rows.y), "r"(rows.z), "r"(rows.w), "r"(bar)
        : "memory");
}

// gelu_tanh (common.cuh) as x times a sigmoid: 0.5 (1 + tanh z) = 1 / (1 + exp(-2 z)).
__device__ __forceinline__ float gelu(float x)
{
    const float z = 0.7978845608028654f * (x + 0.044715f * x * x * x);
    return __fdividef(x, 1.0f + __expf(-2.0f * z));
}

// A place in the ring and the parity of its round, counted: a thread that divides for
// them takes longer than a stage of few rows (122 us where it now takes 105).
struct Place {
    uint32_t slot = 0, phase = 0;

    __device__ __forceinline__ void next(uint32_t stages)
    {
        if (++slot == stages) {
            slot = 0;
            phase ^= 1;
        }
    }
    // n places on (once a tile at most)
    __device__ __forceinline__ void skip(uint32_t n, uint32_t stages)
    {
        const uint32_t to = slot + n;
        phase ^= to / stages & 1;
        slot = to % stages;
    }
};

// The tensor maps of a launch. x: boxes of 8, 16, .. 128 rows; for gathering the first, of one row.
struct Maps {
    CUtensorMap w, w2, x[5];
};

// Rows of the boxes that bring `half` (a multiple of 8, at most 128) rows or a few
// more: the next power of two, or three quarters of it in two boxes. (A copy costs its
// warp about 80 cycles to issue, whatever it brings.)
struct RowBoxes {
    int first, second;       // log2 of the rows / 8; second < 0: none

    __device__ __forceinline__ explicit RowBoxes(int half)
    {
        const int up = 32 - __clz((half >> 3) - 1);
        const bool three = up >= 2 && half * 4 <= (8 << up) * 3;
        first = three ? up - 1 : up;
        second = three ? up - 2 : -1;
    }
    __device__ __forceinline__ int rows() const { return (8 << first) + (second < 0 ? 0 : 8 << second); }
};

// Whether all four warps of a side say so, and the same without a question.
__device__ __forceinline__ bool side_all(int side, bool yes)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(yes)), "r"(1 + side)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ void side_sync(int side) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + side) : "memory"); }

// Four words of two rows x a feature a lane, as products hold them (a word: features l / 4,
// + 8, + 16, + 24), to shared memory by rows: lane l names where row l % 8's features 8 (l / 8) to
// + 7 go.
__device__ __forceinline__ void put_rows(uint32_t at, const uint32_t (&w)[4])
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                 : "memory");
}

// A tile: rows [r0, r0 + live) of expert e against 256 of its output features (of
// each product) from n0 on. A pair's items come in ascending order.
struct Tile {
    int e, n0, r0, live;

    __device__ __forceinline__ void find(const Shared &sh, const Args &p, int item)
    {
        while (item >= sh.cum[e + 1])
            ++e;
        const unsigned c = sh.count[e], nt = (c + p.cols - 1) >> p.log_cols, across = (p.N + 255u) >> 8, local = item - sh.cum[e],
                       n = local / across;
        n0 = (local - n * across) * 256;
        // (the expert's eights of rows, shared out)
        const unsigned eights = (c + 7) >> 3, each = eights / nt, more = eights - each * nt, a = n * each + min(n, more),
                       b = a + each + (n < more);
        r0 = sh.row0[e] + a * 8;
        live = min(b * 8, c) - a * 8;
    }

    // columns of the products in each CTA's half of the second operand
    __device__ __forceinline__ int half() const { return (live + 15) / 16 * 8; }
};

// After waits that ran out (pair_copies.h), in the pair's first CTA: the stages' barriers made up for what was not sent, of which
// each CTA's weights are `weights` bytes a stage. Returns how far to wait for stages.
__device__ __noinline__ uint32_t settle(Shared &sh, uint32_t stages, uint32_t K, uint32_t weights)
{
    const uint32_t steps = (K + kStageK - 1) / kStageK;
    const uint32_t here = sh.issued, there = tc::of_second(tc::saddr(&sh.issued));
    score::StagesLeft left;
    left.warp(here);
    left.warp(there);
    for (int w = 0; w < kGatherWarps; ++w) {
        left.warp(sh.rows_issued[w]);
        left.warp(tc::of_second(tc::saddr(&sh.rows_issued[w])));
    }
    for (uint32_t i = left.first(stages); i < left.to; ++i) {
        const uint32_t slot = i % stages, bar = tc::saddr(&sh.full[slot]);
        uint32_t sent = (i < here ? weights : 0) + (i < there ? weights : 0);
        for (int w = 0; w < kGatherWarps; ++w) {
            const uint32_t got = tc::of_second(tc::saddr(&sh.rows_issued[w]));
            for (int k = 0; k < kMaxStages; ++k) {
                const uint32_t at = tc::saddr(&sh.sent[w][k]);
                sent += score::sent_bytes(sh.sent[w][k], steps, sh.rows_issued[w], i) +
                        score::sent_bytes({tc::of_second(at), tc::of_second(at + 4)}, steps, got, i);
            }
        }
        if (i >= here)
            tc::bar_expect(bar, sent);
        else if (sent != 2 * sh.bytes[slot])
            asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(2 * sh.bytes[slot] - sent) : "memory");
    }
    return left.to;
}

template <Mode MODE, bool BYTES>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGatherThreads, 1) k_grouped(const __grid_constant__ Maps maps, const Args p)
{
    constexpr int kWBoxes = weight_boxes<MODE, BYTES>();
    extern __shared__ uint8_t dsm_raw[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = tc::cluster_rank();
    const uint32_t ring = (tc::saddr(dsm_raw) + 1023u) & ~1023u, xbox = p.cols * 64, rows_at = kWBoxes * kBox,
                   stage = rows_at + 2 * xbox, stages = p.stages;
    const int pairs = gridDim.x / 2, pair = blockIdx.x / 2, steps = (p.K + kStageK - 1) / kStageK;

    if (tid == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            tc::bar_init(&sh.full[i], 1);
            tc::bar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::bar_init(&sh.tfull[i], 1);
            tc::bar_init(&sh.tempty[i], 2 * kEpilogue);      // of both CTAs
        }
        tc::bar_init(&sh.drained, 1);
        sh.abort = 0;
        sh.passed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    for (int i = tid; i < kGatherWarps * kMaxStages; i += blockDim.x)
        sh.sent[i / kMaxStages][i % kMaxStages].first = ~0u;
    if (tid < kGatherWarps)
        sh.rows_issued[tid] = 0;
    tc::after_previous();
    if (warp == 1)
        tc::memory_take<2>(&sh.tmem);
    if (warp == 2) {
        // tiles before each expert: 32 experts at a time, their loads ahead
        const int across = (p.N + 255) / 256;
        int base = 0;
        constexpr int kAhead = 4;
        for (int e1 = 0; e1 < p.E; e1 += 32 * kAhead) {
            int32_t from[kAhead], to[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int e = e1 + i * 32 + lane;
                from[i] = e < p.E ? __ldcg(p.offsets + e) : 0;
                to[i] = e < p.E ? __ldcg(p.offsets + e + 1) : 0;
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int e = e1 + i * 32 + lane;
                int64_t a = from[i], b = to[i];
                a = a < 0 ? 0 : a > p.R ? p.R : a;
                b = b < a ? a : b > p.R ? p.R : b;
                int sum = (static_cast<int>(b - a) + p.cols - 1) / p.cols * across;
                if (e < p.E) {
                    sh.row0[e] = static_cast<int>(a);
                    sh.count[e] = static_cast<int>(b - a);
                }
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int u = __shfl_up_sync(0xFFFFFFFFu, sum, o);
                    sum += lane >= o ? u : 0;
                }
                if (e < p.E)
                    sh.cum[e + 1] = base + sum;
                base += __shfl_sync(0xFFFFFFFFu, sum, 31);
            }
        }
        if (lane == 0)
            sh.cum[0] = 0;
    }
    tc::fence_before();
    __syncthreads();
    tc::cluster_sync();
    tc::fence_after();
    tc::let_next_start();
    const uint32_t tmem = sh.tmem;
    const tc::Waiter wait{&sh.abort, p.status, p.timeout_ns};
    const int items = sh.cum[p.E];
    const uint32_t bar0 = tc::saddr(&sh.full[0]), full0 = tc::in_first(bar0);
    Tile t;
    t.e = 0;

    if (warp == 0) {
        // ------------------------------------------------------------ copies of weights (each CTA its own; rows below)
        if (lane == 0) {
            tc::prefetch_map(&maps.w);
            tc::prefetch_map(&maps.w2);
            uint64_t once, again;
            asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
            asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(again));
            bool ok = true;
            uint32_t n = 0;
            Place at;
            for (int item = pair; item < items && ok; item += pairs) {
                t.find(sh, p, item);
                const int half = t.half();
                const uint32_t mine = kWBoxes * kBox + (p.src ? half : RowBoxes(half).rows()) * 256;
                const uint64_t policy = sh.count[t.e] <= p.cols ? once : again;
                const int w0 = t.n0 + rank * 128;
                for (int ks = 0; ks < steps; ++ks, ++n, at.next(stages)) {
                    if (n >= stages && !(ok = wait(&sh.empty[at.slot], at.phase ^ 1, 34, ks)))
                        break;
                    if (p.src && ks == 0)
                        asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(tc::saddr(&sh.passed)), "r"(n + 1) : "memory");
                    const uint32_t bar = full0 + at.slot * 8, dst = ring + at.slot * stage;
                    if (rank == 0)
                        tc::bar_expect(bar0 + at.slot * 8, 2 * mine);
                    sh.bytes[at.slot] = mine;
                    copy_weights(dst, &maps.w, ks * kStageK, w0, t.e, bar, policy);
                    if (MODE == kGated)
                        copy_weights(dst + kBox, &maps.w2, ks * kStageK, w0, t.e, bar, policy);
                    else if (!BYTES)
                        copy_weights(dst + kBox, &maps.w, ks * kStageK + 64, w0, t.e, bar, policy);
                }
            }
            sh.issued = n;
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ products (the first CTA's warp for both)
        if (rank == 0) {
            const bool lead = tc::elect();
            bool ok = true;
            uint32_t tile = 0;
            Place at;
            for (int item = pair; item < items && ok; item += pairs, ++tile) {
                t.find(sh, p, item);
                const uint32_t buf = tile & 1, d = tmem + buf * 256, idesc = tc::product_desc(256, 2 * t.half(), BYTES);
                if (tile >= 2)
                    ok = wait(&sh.tempty[buf], (tile >> 1) - 1, 35, t.e);
                for (int ks = 0; ks < steps; ++ks, at.next(stages)) {
                    const uint32_t slot = at.slot;
                    ok = ok && wait(&sh.full[slot], at.phase, 36, ks);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok)
                        break;
                    if (lead) {
                        tc::fence_after();
                        const uint64_t a = tc::operand(ring + slot * stage), b = tc::operand(ring + slot * stage + rows_at);
                        const int left = p.K - ks * kStageK;
                        if constexpr (BYTES) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (j * 32 < left) {
                                    const uint64_t aj = a + j * 2, bj = b + (j >> 1) * (xbox >> 4) + (j & 1) * 4;
                                    const bool add = (ks | j) != 0;
                                    tc::product_twice<2>(d, aj, bj, bj + 2, idesc, add);
                                    if constexpr (MODE == kGated)
                                        tc::product_twice<2>(d + 128, aj + (kBox >> 4), bj, bj + 2, idesc, add);
                                }
                        } else {
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                if (j * 16 < left)
                                    tc::product<2, false>(d, a + (j >> 2) * (kBox >> 4) + (j & 3) * 2,
                                                          b + (j >> 2) * (xbox >> 4) + (j & 3) * 2, idesc, (ks | j) != 0);
                        }
                        tc::commit_both(&sh.empty[slot]);
                        if (ks == steps - 1)
                            tc::commit_both(&sh.tfull[buf]);
                    }
                    __syncwarp();
                }
            }
            // every issued product completes before the tensor memory is released
            if (lead) {
                tc::commit<2>(&sh.drained);
                tc::bar_drain(tc::saddr(&sh.drained), 0);
            }
            __syncwarp();
        }
    } else if (warp < 4 || warp >= 4 + kEpilogue) {
        // ------------------------------------------------------------ rows: gathered ones four a copy, a lane's of one half of K; else boxes
        if (p.src) {
            const int mate = warp < 4 ? warp - 2 : warp - kEpilogue - 2, h = lane & 1, group = (lane >> 1) * kGatherWarps + mate;
            // A warp that has rows in a tile keeps the products from running on, so that no stage is used again behind its back.
            // Without any it would have to see each of their phases in time (they turn after two); it leaves the tile out,
            // and goes by the weights' warp when it comes back.
            bool ok = true, left = false;
            uint32_t n = 0;
            Place place;
            for (int item = pair; item < items && ok; item += pairs) {
                t.find(sh, p, item);
                const int half = t.half(), at = rank * half + 4 * group;
                const bool mine = 4 * group < half;
                if (4 * mate >= half) {
                    n += steps;
                    place.skip(steps, stages);
                    left = true;
                    continue;
                }
                if (lane == 0)                   // (its groups of four rows, in two copies each)
                    sh.sent[mate][n / steps % kMaxStages] = {n, ((half >> 2) - mate + kGatherWarps - 1u) / kGatherWarps * 1024};
                if (left && !(ok = __all_sync(0xFFFFFFFFu, wait.passed(&sh.passed, n, 43, t.e))))
                    break;
                left = false;
                int v[4] = {0, 0, 0, 0};
                // (places behind the tile's rows, and rows of x that are not there, take row 0: never stored)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (mine && at + j < t.live) {
                        const int s = __ldcg(p.src + t.r0 + at + j);
                        v[j] = s >= 0 && s / p.per < p.x_rows ? s / p.per : 0;
                    }
                const int4 idx = make_int4(v[0], v[1], v[2], v[3]);
                for (int ks = 0; ks < steps; ++ks, ++n, place.next(stages)) {
                    ok = wait(&sh.empty[place.slot], place.phase ^ 1, 43, ks);       // (a new barrier has this parity behind it)
                    if (!(ok = __all_sync(0xFFFFFFFFu, ok)))
                        break;
                    if (mine)
                        copy_gathered(ring + place.slot * stage + rows_at + h * xbox + group * 512, &maps.x[0], ks * 256 + h * 128, idx,
                                      full0 + place.slot * 8);
                    __syncwarp();
                }
                if (lane == 0)
                    sh.rows_issued[mate] = n;
            }
        } else if (warp == 2 && lane == 0) {
            bool ok = true;
            uint32_t n = 0;
            Place place;
            for (int item = pair; item < items && ok; item += pairs) {
                t.find(sh, p, item);
                const int half = t.half(), row = t.r0 + rank * half;
                const RowBoxes box(half);
                sh.sent[0][n / steps % kMaxStages] = {n, static_cast<uint32_t>(box.rows() * 256)};
                for (int ks = 0; ks < steps; ++ks, ++n, place.next(stages)) {
                    if (n >= stages && !(ok = wait(&sh.empty[place.slot], place.phase ^ 1, 43, ks)))
                        break;
                    const uint32_t dst = ring + place.slot * stage + rows_at, bar = full0 + place.slot * 8;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        copy_rows(dst + h * xbox, &maps.x[box.first], ks * 256 + h * 128, row, bar);
                        if (box.second >= 0)
                            copy_rows(dst + h * xbox + (1024 << box.first), &maps.x[box.second], ks * 256 + h * 128, row + (8 << box.first), bar);
                    }
                }
            }
            sh.rows_issued[0] = n;
        }
    } else {
        // ------------------------------------------------------------ epilogue: a lane is an output feature, a column a row of x
        // (columns by eights, a side's each fourth: with two sides, what a warp waits for itself took longer than the products)
        const int quarter = warp & 3, side = (warp - 4) >> 2;
        constexpr int kEights = (MODE == kGated ? 128 : 256) / 8 / kSides;
        const uint32_t out0 = ring + kRing + side * 2 * kOutBuf, put_at = out0 + (lane & 7) * kOutRow + quarter * 64 + (lane >> 3) * 16,
                       take_at = out0 + (quarter * 2 + (lane >> 4)) * kOutRow + (lane & 15) * 16;
        uint32_t outs = 0;
        bool alive = true;
        uint32_t tile = 0;
        for (int item = pair; item < items; item += pairs, ++tile) {
            t.find(sh, p, item);
            const uint32_t buf = tile & 1;
            const int n0 = t.n0 + rank * 128, nw = n0 + quarter * 32;
            // what this lane's rows and features (see below) are multiplied by, on its way while the products end
            constexpr int kX = MODE == kGated ? 2 : 1;
            float xs[kEights][kX], s0[4], s1[4];
#pragma unroll
            for (int i = 0; i < kEights; ++i)
#pragma unroll
                for (int j = 0; j < kX; ++j) {
                    const int c = (i * kSides + side) * 8 + (MODE == kGated ? 2 * (lane & 3) + j : quarter * 2 + (lane >> 4));
                    xs[i][j] = 1.0f;
                    if (MODE != kDown && c < t.live) {
                        int row = t.r0 + c;
                        bool there = true;
                        if (p.src) {
                            row = __ldcg(p.src + row);
                            there = row >= 0 && row / p.per < p.x_rows;
                            row = there ? row / p.per : 0;
                        }
                        // (negative: no such row of x, the output is zero)
                        xs[i][j] = there ? (BYTES ? __ldcg(p.xs + row) : 1.0f) : -1.0f;
                    }
                }
            const float norm = MODE == kDown ? 0x1p-12f / __ldcg(p.smax + t.e) : 1.0f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int n = nw + (lane >> 2) + 8 * q;
                s0[q] = s1[q] = norm;
                if (n < p.N && p.s0) {
                    s0[q] *= __ldcg(p.s0 + static_cast<int64_t>(t.e) * p.N + n);
                    if (MODE == kGated)
                        s1[q] = __ldcg(p.s1 + static_cast<int64_t>(t.e) * p.N + n);
                }
            }
            if (alive)
                alive = wait(&sh.tfull[buf], tile >> 1, 37, t.e);
            alive = side_all(side, alive);       // (a side's warps meet at barriers below)
            tc::fence_after();
            if (alive && n0 < p.N) {
                const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + buf * 256;
                auto read = [&](int c, uint32_t (&u)[8], uint32_t (&v)[8]) {
                    tc::read_pairs(from + c, u);
                    if (MODE == kGated)
                        tc::read_pairs(from + 128 + c, v);
                };
                // this side's eights, the next on its way meanwhile
                uint32_t u[2][8], v[2][8];
                if (side * 8 < t.live)
                    read(side * 8, u[0], v[0]);
#pragma unroll
                for (int i = 0; i < kEights; ++i) {
                    const int c = (i * kSides + side) * 8;
                    if (c >= t.live)
                        break;
                    const uint32_t ob = (outs++ & 1) * kOutBuf;
                    __syncwarp();
                    tc::read_wait();
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        asm volatile("" : "+r"(u[i & 1][q]));
                        if (MODE == kGated)
                            asm volatile("" : "+r"(v[i & 1][q]));
                    }
                    if (i + 1 < kEights && c + kSides * 8 < t.live)
                        read(c + kSides * 8, u[(i + 1) & 1], v[(i + 1) & 1]);
                    // (of features l / 4 + 8 q rows 2 (l % 4) and the next: u[2 q], u[2 q + 1])
                    uint32_t pk[4];
                    if (MODE == kGated) {
                        float a[8];
                        uint32_t m[2] = {0, 0};
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const float x = xs[i][kX == 2 ? q & 1 : 0];
                            a[q] = gelu(__uint_as_float(u[i & 1][q]) * s0[q >> 1] * x) * (__uint_as_float(v[i & 1][q]) * s1[q >> 1] * x);
                            m[q & 1] = max(m[q & 1], __float_as_uint(a[q]) & 0x7FFFFFFFu);
                        }
                        // |a| < 2^(e - 126) for all 32 features of a row: below 2^15 in f16, which has 11 bits down to 2^-14
                        float up[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1)
                                m[j] = max(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], o));
                            const uint32_t e = max(m[j] >> 23, 14u);
                            up[j] = __uint_as_float((268 - e) << 23);
                            const int r = c + 2 * lane + j;
                            if (lane < 4 && r < t.live && nw < p.N)
                                p.exps[static_cast<int64_t>(t.r0 + r) * (p.N >> 5) + (nw >> 5)] = static_cast<uint8_t>(e);
                        }
                        // (f16, not fp32: half the bytes out and back in; 2^-11 beside the terms' 2^-9)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const __half2 h = __floats2half2_rn(a[2 * q] * up[0], a[2 * q + 1] * up[1]);
                            pk[q] = *reinterpret_cast<const uint32_t *>(&h);
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float a = __uint_as_float(u[i & 1][2 * q]) * s0[q], b = __uint_as_float(u[i & 1][2 * q + 1]) * s0[q];
                            if (MODE == kDown) {         // (f16: a quarter of the rounding of bf16, at its bytes, down to 2^-14)
                                const __half2 h = __floats2half2_rn(a, b);
                                pk[q] = *reinterpret_cast<const uint32_t *>(&h);
                            } else {
                                const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
                                pk[q] = *reinterpret_cast<const uint32_t *>(&h);
                            }
                        }
                    }
                    // The side's four warps lay 128 features of eight rows side by side, and each takes two rows of
                    // them out again: whole lines, where a warp's own 32 features are 64 bytes of a row (50
                    // cycles a store of 512 bytes instead of 18; 32,768 rows of 704 on 2816 features 156 us, now 116). The products read their operands over the same
                    // wires, so that what passes through shared memory here is to be little.
                    put_rows(put_at + ob, pk);
                    side_sync(side);
                    uint32_t w[4];
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                 : "r"(take_at + ob)
                                 : "memory");
                    if (MODE == kGemm) {
                        // (a row's scale is a power of two: it may follow the rounding)
                        const __nv_bfloat162 x2 = __float2bfloat162_rn(xs[i][0]);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if (BYTES) {
                                const __nv_bfloat162 h = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&w[q]), x2);
                                w[q] = *reinterpret_cast<const uint32_t *>(&h);
                            }
                            w[q] = xs[i][0] < 0.0f ? 0u : w[q];
                        }
                    }
                    const int r = c + quarter * 2 + (lane >> 4), first = n0 + (lane & 15) * 8;
                    if (r < t.live) {
                        uint16_t *to = p.out + static_cast<int64_t>(t.r0 + r) * p.N + first;
                        if (p.wide) {
                            if (first < p.N)
                                *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
                        } else {
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                if (first + q < p.N)
                                    to[q] = static_cast<uint16_t>(q & 1 ? w[q >> 1] >> 16 : w[q >> 1]);
                        }
                    }
                }
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0)
                asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(tc::in_first(tc::saddr(&sh.tempty[buf])))
                             : "memory");
        }
    }
    tc::fence_before();
    __syncthreads();
    // neither CTA leaves while the other's products or arrivals may reach it,
    tc::cluster_sync();
    // nor before every copy that either issued has landed (the first sees both CTAs' bytes)
    if (rank == 0 && tid == 0) {
        // (without a wait that ran out all warps have copied for all stages)
        const uint32_t to = sh.abort || tc::of_second(tc::saddr(&sh.abort)) ? settle(sh, p.stages, p.K, kWBoxes * kBox) : sh.issued;
        for (uint32_t i = to > stages ? to - stages : 0; i < to; ++i)
            tc::bar_drain(tc::saddr(&sh.full[i % stages]), (i / stages) & 1);
    }
    __syncthreads();
    tc::cluster_sync();
    if (warp == 1) {
        tc::fence_after();
        tc::memory_free<2>(tmem);
    }
}

}  // namespace grouped
}  // namespace fgm
