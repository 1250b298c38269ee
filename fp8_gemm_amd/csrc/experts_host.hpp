// Argument checks, shape classes and launches shared by the experts' entry
// points (experts_bf16.hip, experts_int8.hip).
#pragma once

#include "../../include/fp8_gemm_experts.h"
#include "experts.hpp"
#include "fused_host.hpp"

namespace {

using fp8g::PLACE_GROUPS;
using fp8g::PLACE_REST;
using fp8g::PLACE_SUMS;
using fp8g::RaggedParams;

// Sizes of a ragged product (`unit` bytes per element).
int check_ragged_sizes(int M, int G, int N, int K, int unit) {
    if (G < 0 || G > 65535) return fail(FP8G_ERR_SHAPE, "G=%d is not in 0 .. 65535", G);
    if (const int st = check_sizes(M, N, K, unit)) return st;
    if (N % 8) return fail(FP8G_ERR_SHAPE, "N=%d is not a multiple of 8", N);
    if ((int64_t)N * 2 > kMaxRowStride) return fail(FP8G_ERR_SHAPE, "N=%d exceeds the row-stride limit %lld bytes", N, (long long)kMaxRowStride);
    return FP8G_OK;
}

constexpr int kMaxIntK = 131056;                   // 2^14 K < 2^31
int check_int8_sizes(int K) {
    if (K > kMaxIntK) return fail(FP8G_ERR_SHAPE, "K=%d exceeds %d: a sum could leave 32 bits", K, kMaxIntK);
    return FP8G_OK;
}

// Token rows of a backward pass: the weight gradients' longest sum, counted in
// K steps.
constexpr int kMaxSumRows = 1 << 30;
int check_sum_rows(int M) {
    if (M > kMaxSumRows) return fail(FP8G_ERR_SHAPE, "M=%d exceeds %d", M, kMaxSumRows);
    return FP8G_OK;
}

// A BF16 output whose tiles are addressed with 32-bit offsets.
int check_tile_output(const char *name, const void *ptr, int64_t ld, int cols) {
    if (const int st = check_output(name, ptr, ld, cols)) return st;
    if (2 * ld > kMaxRowStride) return fail(FP8G_ERR_STRIDE, "row stride of %s above %lld bytes", name, (long long)kMaxRowStride);
    return FP8G_OK;
}

int check_offsets(const int32_t *offsets) {
    if (!offsets) return fail(FP8G_ERR_NULL, "offsets is required");
    if (!aligned4(offsets)) return fail(FP8G_ERR_ALIGN, "offsets must be 4-byte aligned");
    return FP8G_OK;
}

// The distance between experts' [N x K] matrices, in elements.
int check_stride(const char *name, int64_t stride, int64_t ld, int G, int N, int K, int unit) {
    if (G <= 1 || N == 0 || K == 0) return FP8G_OK;
    if (stride < (N - 1) * ld + K) return fail(FP8G_ERR_STRIDE, "experts of %s overlap: stride %lld", name, (long long)stride);
    if (stride * unit % 16) return fail(FP8G_ERR_ALIGN, "expert stride %lld of %s is not a multiple of 16 bytes", (long long)stride, name);
    return FP8G_OK;
}

// G matrices of [N x K]: row by row where they follow one another evenly, else
// each as one block.
Area experts_area(const char *name, const void *ptr, int64_t ld, int64_t stride, int64_t G, int64_t N, int64_t K, int unit) {
    if (G <= 1 || stride == N * ld) return area(name, ptr, ld, G * N, K, unit);
    return area(name, ptr, stride, N > 0 ? G : 0, (N - 1) * ld + K, unit);
}

// Tiles of `rows` rows that any division of M rows into that many segments can
// need.
int64_t tiles_bound(int64_t M, int64_t segments, int rows) {
    const int64_t live = segments < M ? segments : M;
    return (M + live * (rows - 1)) / rows;
}

// ---------------------------------------------------------------------------
// Shape classes of the ragged and integer products: the one with the smallest
// estimated time, as in fused_host.hpp, with the number of tiles that M rows
// divided among G experts make on average (half a tile more per expert than
// whole tiles alone).
//
// The constants (us; the persistent kernels: launch, and per round of 256
// workgroups a fixed part and the K steps, a last round of at most 128 tiles
// counting 0.7) are fitted to 2555 measured cases, every class each: 2 .. 160
// experts, 1 .. 65536 rows divided unevenly, N 32 .. 14336, K 64 .. 8192, the
// weights read from memory.  On average the choice takes longer than the fastest
// class by 3.4% (BF16), 2.0% (8-bit integers), 0.7% (token gradients), 1.3%
// (weight gradients) and 0.1% (dense integers).  Most of what is left are
// products of few columns, where the number of rows of the largest experts
// matters, which the host does not know: at worst 1.8 times (BF16 1086 rows of
// 7 experts, 224 x 7936: 41 against 22 us) and 1.7 times (integers, 5305 rows of
// 57 experts, 152 x 4736: 39 against 23 us).
// ---------------------------------------------------------------------------
enum RaggedOp { R_BF16, R_INT8, R_TOKEN_GRAD, R_WEIGHT_GRAD };

constexpr ClassCost kRaggedCost[4][3] = {{{1.8, 2.5, 0.385, 0.233}, {1.4, 4.0, 0.640, 0.331}, {1.2, 4.8, 0.859, 0.543}},
                                         {{2.9, 3.2, 0.405, 0.158}, {2.7, 4.9, 0.655, 0.282}, {3.1, 6.2, 0.840, 0.486}},
                                         {{2.8, 2.6, 0.426, 0.161}, {3.1, 3.6, 0.902, 0.158}, {2.6, 3.9, 0.910, 0.470}},
                                         {{4.1, 2.4, 0.519, 0.100}, {4.3, 3.5, 1.075, 0.140}, {3.4, 5.2, 0.982, 0.676}}};
struct FewCost {
    double launch, round, copy, memory;            // copy: bytes per ns and CU; memory: bytes per us / 1e6
};
constexpr FewCost kRaggedFew[2] = {{3.1, 2.3, 74.2, 5.6}, {4.5, 2.4, 75.8, 6.2}};

double expected_tiles(double M, double live, int rows) {
    const double t = M / rows + 0.5 * live;
    return t > live ? t : live;
}

double ragged_time(RaggedOp op, int c, double tiles, double steps) {
    const ClassCost &k = kRaggedCost[op][c];
    const int64_t n = (int64_t)tiles, left = n % 256;
    double rounds = (double)(n / 256) + (left == 0 ? 0.0 : (left <= 128 ? 0.7 : 1.0));
    if (rounds < 0.7) rounds = 0.7;
    const double busy = n >= 256 ? 1.0 : (double)(left <= 128 ? 2 * left : left) / 256.0;
    return k.launch + rounds * (k.wave + steps * (k.step + k.load * busy));
}

// M rows [K] of G experts times weights [N][K] (op R_TOKEN_GRAD: N and K are
// those of the gradient's product).
Choice pick_ragged(RaggedOp op, int64_t M, int64_t G, int64_t N, int64_t K) {
    const int unit = op == R_INT8 ? 1 : 2;
    const double kbytes = (double)K * unit, live = (double)(G < 1 ? 1 : (G < M ? G : M));
    const double bytes = kbytes * ((double)N * live + (double)M) + 2.0 * (double)M * (double)N;
    Choice best = {C_256x256, {}};
    double least = 1e300;
    auto consider = [&](double t, double memory, const Choice &c) {
        t = (t > 2.0 + memory ? t : 2.0 + memory) + 0.05 * t;
        if (t < least) least = t, best = c;
    };
    for (int cb = 1; op <= R_INT8 && cb <= 4; cb *= 2) {
        const int64_t tiles = tiles_bound(M, G, 16 * cb);
        if (tiles > 65535) continue;               // (grid y)
        const FewCost &k = kRaggedFew[op];
        for (int rb = 1; rb <= 4; rb *= 2) {
            int fit = 160 * 1024 / (kFewWaves * (rb + cb) * 2048 * few_slots(rb, cb));
            if (fit > 3) fit = 3;
            const double wgs = (double)cdiv(N, 16 * rb) * expected_tiles((double)M, live, 16 * cb);
            double rounds = fit == 1 ? (double)cdiv((int64_t)wgs, 256) : wgs / 256.0;
            if (rounds < 1.0) rounds = 1.0;
            consider(k.launch + rounds * (k.round / fit + 16.0 * (rb + cb) * kbytes / (k.copy * 1e3)), bytes / (k.memory * 1e6),
                     Choice{C_FEW, FewShape{rb, cb, cdiv(N, 16 * rb) * tiles}});
        }
    }
    for (int c = 0; c < 3; ++c)
        consider(ragged_time(op, c, expected_tiles((double)M, live, (int)kClassRows[c]) * (double)cdiv(N, kClassCols[c]),
                             (double)cdiv(K * unit, 128)),
                 bytes / 5.0e6, Choice{(ShapeClass)(C_128x128 + c), {}});
    return best;
}

// Weight gradients: G of N x K, each reduced over M / G rows on average.
ShapeClass pick_sums(int64_t M, int64_t G, int64_t N, int64_t K) {
    ShapeClass best = C_256x256;
    double least = 1e300;
    const double steps = (double)M / (64.0 * (double)(G > 0 ? G : 1)) + 0.5;
    for (int c = 0; c < 3; ++c) {
        const double t = ragged_time(R_WEIGHT_GRAD, c, (double)(cdiv(N, kClassRows[c]) * cdiv(K, kClassCols[c]) * G), steps);
        if (t < least) least = t, best = (ShapeClass)(C_128x128 + c);
    }
    return best;
}

// The dense integer product.  Few tokens or not as for FP8, by the constants of
// that form's tiles, which are slower than the persistent ones: between 256 and
// 1024 rows with K of 8192 and more the few-token kernel is taken where
// ragged_time puts the tiles up to 30% lower (not measured).  `direct`: the
// tiled kernel is the persistent one, and its class the one with the least of
// its own estimates; the staged form's goes by FP8's too.
Choice pick_dense(int64_t M, int64_t N, int64_t K, bool direct) {
    Choice best = pick_class(M, N, K, 1, false);
    if (best.c == C_FEW || !direct) return best;
    double least = 1e300;
    for (int c = 0; c < 3; ++c) {
        const double t = ragged_time(R_INT8, c, (double)(cdiv(M, kClassRows[c]) * cdiv(N, kClassCols[c])), (double)cdiv(K, 128));
        if (t < least) least = t, best.c = (ShapeClass)(C_128x128 + c);
    }
    return best;
}

template <int E, bool SCALED, int PLACE>
RaggedParams<E, SCALED, PLACE> with_offsets(const FusedArgs &a, const int32_t *offsets, int rows = 0) {
    RaggedParams<E, SCALED, PLACE> p = {};
    static_cast<FusedArgs &>(p) = a;
    p.offsets = offsets;
    p.rows = rows;
    return p;
}

// The persistent kernels count their tiles in 32 bits, with room for the step
// from one to the next.
constexpr int64_t kMaxTiles = int64_t(1) << 30;
int check_tiles(int64_t tiles) {
    if (tiles > kMaxTiles) return fail(FP8G_ERR_SHAPE, "%lld tiles: too many for one launch", (long long)tiles);
    return FP8G_OK;
}

// Persistent workgroups: one per CU (few tiles are cut in two).
int64_t persistent_grid(int64_t tiles) { return 2 * tiles < 256 ? 2 * tiles : 256; }

template <int BM, int BN, int STAGES, bool INT, bool TB, int PLACE, int EPI>
int launch_rows_shape(const FusedArgs &a, const int32_t *offsets, hipStream_t s) {
    auto p = with_offsets<EPI, INT, PLACE>(a, offsets);
    p.tiles_n = (int)cdiv(p.N, BN);
    const int64_t bound = tiles_bound(p.M, p.G + (PLACE == PLACE_REST ? 2 : 0), BM), wgs = bound * p.tiles_n;
    if (const int st = check_tiles(wgs)) return st;
    p.tiles_m = (int)bound;
    const dim3 grid((unsigned)persistent_grid(wgs)), block(256);
    if (p.K % (INT ? 128 : 64))
        hipLaunchKernelGGL((fp8g::ragged_tile_kernel<BM, BN, STAGES, INT, false, TB, true, PLACE, EPI>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((fp8g::ragged_tile_kernel<BM, BN, STAGES, INT, false, TB, false, PLACE, EPI>), grid, block, 0, s, p);
    return launch_status("ragged tiled kernel");
}

template <bool INT, bool TB, int PLACE, int EPI>
int launch_rows(ShapeClass c, const FusedArgs &a, const int32_t *offsets, hipStream_t s) {
    if (c == C_128x128) return launch_rows_shape<128, 128, 4, INT, TB, PLACE, EPI>(a, offsets, s);
    if (c == C_128x256) return launch_rows_shape<128, 256, 3, INT, TB, PLACE, EPI>(a, offsets, s);
    return launch_rows_shape<256, 256, 2, INT, TB, PLACE, EPI>(a, offsets, s);
}

// Few rows per expert (K and the strides in bytes).
template <int RB, int CB, bool INT>
int launch_ragged_few(const FusedArgs &a, const int32_t *offsets, hipStream_t s) {
    const auto p = with_offsets<fp8g::EPI_ACT, INT, PLACE_GROUPS>(a, offsets);
    // (N is below 2^22 here, and pick_ragged keeps grid y below 2^16)
    const dim3 grid((unsigned)cdiv(p.N, 16 * RB), (unsigned)tiles_bound(p.M, p.G, 16 * CB)), block(256);
    hipLaunchKernelGGL((fp8g::ragged_decode_kernel<RB, CB, INT, few_slots(RB, CB)>), grid, block, 0, s, p);
    return launch_status("ragged few-token kernel");
}

template <int RB, bool INT>
int launch_ragged_few_rb(const FusedArgs &a, int cb, const int32_t *offsets, hipStream_t s) {
    if (cb == 1) return launch_ragged_few<RB, 1, INT>(a, offsets, s);
    if (cb == 2) return launch_ragged_few<RB, 2, INT>(a, offsets, s);
    return launch_ragged_few<RB, 4, INT>(a, offsets, s);
}

template <bool INT>
int launch_ragged_few_shape(const FusedArgs &a, const FewShape &f, const int32_t *offsets, hipStream_t s) {
    if (f.rb == 1) return launch_ragged_few_rb<1, INT>(a, f.cb, offsets, s);
    if (f.rb == 2) return launch_ragged_few_rb<2, INT>(a, f.cb, offsets, s);
    return launch_ragged_few_rb<4, INT>(a, f.cb, offsets, s);
}

// A product of rows [M][lda] with experts' weights; strides in bytes.
FusedArgs ragged_args(const void *A, int64_t lda, const void *B, int64_t ldb, int64_t b_stride, void *D, int64_t ldd,
                      int M, int G, int N, int K, int unit) {
    FusedArgs p = {};
    p.A = static_cast<const uint8_t *>(A);
    p.B = static_cast<const uint8_t *>(B);
    p.B2 = p.B;
    p.D = static_cast<uint16_t *>(D);
    p.D2 = p.D;
    p.lda = lda * unit; p.ldb = ldb * unit; p.ldb2 = p.ldb; p.ldd = ldd;
    p.b_gstride = b_stride * unit;
    p.M = M; p.N = N; p.K = K; p.G = G; p.cap = M;
    p.ksplit = 1 << 30;
    p.krows = K;
    return p;
}

}  // namespace
