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
// Shape classes of the ragged products: the one with the smallest estimated
// time, by fused_host.hpp's estimates with the number of tiles that M rows
// divided among G experts make on average (half a tile more per expert than
// whole tiles alone).
// ---------------------------------------------------------------------------
double expected_tiles(double M, double live, int rows) {
    const double t = M / rows + 0.5 * live;
    return t > live ? t : live;
}

Choice pick_ragged(int64_t M, int64_t G, int64_t N, int64_t K, int unit, bool few) {
    const double kbytes = (double)K * unit, live = (double)(G < 1 ? 1 : (G < M ? G : M));
    const double memory = 2.0 + (kbytes * ((double)N * live + (double)M) + 2.0 * (double)M * (double)N) / 5.0e6;
    auto floored = [&](double t) { return (t > memory ? t : memory) + 0.05 * t; };
    Choice best = {C_256x256, {}};
    double least = 1e300;
    for (int cb = 1; few && cb <= 4; cb *= 2) {
        const int64_t tiles = tiles_bound(M, G, 16 * cb);
        if (tiles > 65535) continue;               // (grid y)
        for (int rb = 1; rb <= 4; rb *= 2) {
            int fit = 160 * 1024 / (kFewWaves * (rb + cb) * 2048 * few_slots(rb, cb));
            if (fit > 3) fit = 3;
            double rounds = (double)cdiv(N, 16 * rb) * expected_tiles((double)M, live, 16 * cb) / 256.0;
            if (rounds < 1.0) rounds = 1.0;
            const double t = floored(2.5 + rounds * (1.5 / fit + 16.0 * (rb + cb) * kbytes / 70e3));
            if (t < least) least = t, best = Choice{C_FEW, FewShape{rb, cb, cdiv(N, 16 * rb) * tiles}};
        }
    }
    for (int c = 0; c < 3; ++c) {
        const double tiles = expected_tiles((double)M, live, (int)kClassRows[c]) * (double)cdiv(N, kClassCols[c]);
        const double t = floored(tiled_time(c, 2, (int64_t)tiles, cdiv(K * unit, 128)));
        if (t < least) least = t, best = Choice{(ShapeClass)(C_128x128 + c), {}};
    }
    return best;
}

// Weight gradients: G of N x K, each reduced over M / G rows on average.
ShapeClass pick_sums(int64_t M, int64_t G, int64_t N, int64_t K) {
    ShapeClass best = C_256x256;
    double least = 1e300;
    for (int c = 0; c < 3; ++c) {
        const int64_t tiles = cdiv(N, kClassRows[c]) * cdiv(K, kClassCols[c]) * G;
        const double t = tiled_time(c, 2, tiles, cdiv(M, 64 * (G > 0 ? G : 1)));
        if (t < least) least = t, best = (ShapeClass)(C_128x128 + c);
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

// A grid of at most 2^32 threads.
int check_grid(int64_t workgroups) {
    if (workgroups >= (int64_t(1) << 24)) return fail(FP8G_ERR_SHAPE, "%lld workgroups: too many for one launch", (long long)workgroups);
    return FP8G_OK;
}

template <int BM, int BN, int STAGES, int FMT, bool TB, int PLACE, int EPI>
int launch_rows_shape(const FusedArgs &a, const int32_t *offsets, hipStream_t s) {
    auto p = with_offsets<EPI, FMT == fp8g::FMT_I8, PLACE>(a, offsets);
    p.tiles_n = (int)cdiv(p.N, BN);
    const int64_t wgs = tiles_bound(p.M, p.G + (PLACE == PLACE_REST ? 2 : 0), BM) * p.tiles_n;
    if (const int st = check_grid(wgs)) return st;
    const dim3 grid((unsigned)wgs), block(256);
    if (p.K % (FMT == fp8g::FMT_I8 ? 128 : 64))
        hipLaunchKernelGGL((fp8g::ragged_tile_kernel<BM, BN, STAGES, FMT, false, TB, true, PLACE, EPI>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((fp8g::ragged_tile_kernel<BM, BN, STAGES, FMT, false, TB, false, PLACE, EPI>), grid, block, 0, s, p);
    return launch_status("ragged tiled kernel");
}

template <int FMT, bool TB, int PLACE, int EPI>
int launch_rows(ShapeClass c, const FusedArgs &a, const int32_t *offsets, hipStream_t s) {
    if (c == C_128x128) return launch_rows_shape<128, 128, 4, FMT, TB, PLACE, EPI>(a, offsets, s);
    if (c == C_128x256) return launch_rows_shape<128, 256, 3, FMT, TB, PLACE, EPI>(a, offsets, s);
    return launch_rows_shape<256, 256, 2, FMT, TB, PLACE, EPI>(a, offsets, s);
}

// Few rows per expert (K and the strides in bytes).
template <int RB, int CB, int FMT>
int launch_ragged_few(const FusedArgs &a, const int32_t *offsets, hipStream_t s) {
    const auto p = with_offsets<fp8g::EPI_ACT, FMT == fp8g::FMT_I8, PLACE_GROUPS>(a, offsets);
    const dim3 grid((unsigned)cdiv(p.N, 16 * RB), (unsigned)tiles_bound(p.M, p.G, 16 * CB)), block(256);
    if (const int st = check_grid((int64_t)grid.x * grid.y)) return st;
    hipLaunchKernelGGL((fp8g::ragged_decode_kernel<RB, CB, FMT, few_slots(RB, CB)>), grid, block, 0, s, p);
    return launch_status("ragged few-token kernel");
}

template <int RB, int FMT>
int launch_ragged_few_rb(const FusedArgs &a, int cb, const int32_t *offsets, hipStream_t s) {
    if (cb == 1) return launch_ragged_few<RB, 1, FMT>(a, offsets, s);
    if (cb == 2) return launch_ragged_few<RB, 2, FMT>(a, offsets, s);
    return launch_ragged_few<RB, 4, FMT>(a, offsets, s);
}

template <int FMT>
int launch_ragged_few_shape(const FusedArgs &a, const FewShape &f, const int32_t *offsets, hipStream_t s) {
    if (f.rb == 1) return launch_ragged_few_rb<1, FMT>(a, f.cb, offsets, s);
    if (f.rb == 2) return launch_ragged_few_rb<2, FMT>(a, f.cb, offsets, s);
    return launch_ragged_few_rb<4, FMT>(a, f.cb, offsets, s);
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
