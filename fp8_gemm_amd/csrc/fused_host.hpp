// Argument checks and launch helpers shared by the fused entry points
// (fused_fp8.hip, fused_bf16.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/fp8_gemm_fused.h"
#include "fused.hpp"
#include "host_common.hpp"

namespace {

using namespace fp8g_host;
using fp8g::FusedArgs;
using fp8g::FusedParams;

constexpr int kFewMaxM = 64;                       // few-token kernel up to here

template <int E>
FusedParams<E> with_epilogue(const FusedArgs &a) {
    FusedParams<E> p = {};
    static_cast<FusedArgs &>(p) = a;
    return p;
}

// Sizes: every product's M, N, K.  `kbytes` = bytes of a row of K.
int check_sizes(int M, int N, int K, int unit) {
    if (M < 0 || N < 0 || K < 0) return fail(FP8G_ERR_SHAPE, "negative size (M=%d N=%d K=%d)", M, N, K);
    if (K % (16 / unit)) return fail(FP8G_ERR_SHAPE, "K=%d is not a multiple of %d", K, 16 / unit);
    if ((int64_t)K * unit > kMaxRowStride) return fail(FP8G_ERR_SHAPE, "K=%d exceeds the row-stride limit %lld bytes", K, (long long)kMaxRowStride);
    return FP8G_OK;
}

// A K-contiguous operand (ld in elements of `unit` bytes); nothing is read
// from it when K = 0.
int check_operand(const char *name, const void *ptr, int64_t ld, int K, int unit) {
    if (K > 0 && !ptr) return fail(FP8G_ERR_NULL, "%s is required", name);
    if (!aligned16(ptr)) return fail(FP8G_ERR_ALIGN, "%s must be 16-byte aligned", name);
    if (ld < K) return fail(FP8G_ERR_STRIDE, "row stride %lld of %s below K=%d", (long long)ld, name, K);
    if (ld * unit % 16) return fail(FP8G_ERR_ALIGN, "row stride %lld of %s is not a multiple of 16 bytes", (long long)ld, name);
    if (ld > kMaxRowStride / unit) return fail(FP8G_ERR_STRIDE, "row stride of %s above %lld bytes", name, (long long)kMaxRowStride);
    return FP8G_OK;
}

// A BF16 output with `cols` columns.
int check_output(const char *name, const void *ptr, int64_t ld, int cols) {
    if (!ptr) return fail(FP8G_ERR_NULL, "%s is required", name);
    if (!aligned16(ptr)) return fail(FP8G_ERR_ALIGN, "%s must be 16-byte aligned", name);
    if (ld < cols) return fail(FP8G_ERR_STRIDE, "row stride %lld of %s below %d", (long long)ld, name, cols);
    if (ld % 8) return fail(FP8G_ERR_ALIGN, "row stride %lld of %s is not a multiple of 8 elements", (long long)ld, name);
    return FP8G_OK;
}

// A matrix read or written element by element (unit bytes each); *vec = its
// rows start 16-byte aligned.
int check_rows(const char *name, const void *ptr, int64_t ld, int cols, int unit, int *vec) {
    if (reinterpret_cast<uintptr_t>(ptr) % unit) return fail(FP8G_ERR_ALIGN, "%s must be %d-byte aligned", name, unit);
    if (ld < cols) return fail(FP8G_ERR_STRIDE, "row stride %lld of %s below %d", (long long)ld, name, cols);
    *vec = aligned16(ptr) && ld * unit % 16 == 0;
    return FP8G_OK;
}

int check_floats(const char *name, const void *ptr) {
    if (!aligned4(ptr)) return fail(FP8G_ERR_ALIGN, "%s must be 4-byte aligned", name);
    return FP8G_OK;
}

int check_activation(int act) {
    if (act < FP8G_ACT_NONE || act > FP8G_ACT_GELU_TANH) return fail(FP8G_ERR_ARG, "unknown activation %d", act);
    return FP8G_OK;
}

// A scale vector of n values for `rows` rows or channels; *step = 1 or 0.
int check_scale(const char *name, const float *ptr, int n, int rows, int *step) {
    *step = 0;
    if (!ptr) return FP8G_OK;
    if (n != rows && n != 1) return fail(FP8G_ERR_ARG, "%s has %d values: 1 or %d are wanted", name, n, rows);
    *step = n == rows && rows != 1;
    return check_floats(name, ptr);
}

// ---------------------------------------------------------------------------
// Few tokens (M <= 64; larger M in tiles of 64, grid y): 16 RB weight rows per
// workgroup of 4 waves (gated: 8 RB of each matrix).
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 4;

template <int RB, int CB, int FA, int FB, int EPI>
int launch_few(const FusedArgs &a, hipStream_t s) {
    constexpr int D = RB == 1 && CB == 1 ? 3 : 2;
    constexpr int out = EPI == fp8g::EPI_GATED ? 8 * RB : 16 * RB;
    const FusedParams<EPI> p = with_epilogue<EPI>(a);
    const dim3 grid((unsigned)cdiv(p.N, out), (unsigned)cdiv(p.M, 64));
    const dim3 block(64 * kFewWaves);
    if ((int64_t)grid.x * grid.y <= 256)
        hipLaunchKernelGGL((fp8g::fused_decode_kernel<kFewWaves, RB, CB, FA, FB, D, EPI, 1>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((fp8g::fused_decode_kernel<kFewWaves, RB, CB, FA, FB, D, EPI, 2>), grid, block, 0, s, p);
    return launch_status("fused few-token kernel");
}

template <int RB, int FA, int FB, int EPI>
int launch_few_cb(const FusedArgs &a, hipStream_t s) {
    if (a.M <= 16) return launch_few<RB, 1, FA, FB, EPI>(a, s);
    if (a.M <= 32) return launch_few<RB, 2, FA, FB, EPI>(a, s);
    return launch_few<RB, 4, FA, FB, EPI>(a, s);
}

template <int FA, int FB, int EPI>
int launch_few_fmt(const FusedArgs &a, hipStream_t s) {
    constexpr int R0 = EPI == fp8g::EPI_GATED ? 2 : 1;
    const int64_t wide = EPI == fp8g::EPI_GATED ? cdiv(a.N, 16) : cdiv(a.N, 32);
    if (wide >= 512) return launch_few_cb<2 * R0, FA, FB, EPI>(a, s);
    return launch_few_cb<R0, FA, FB, EPI>(a, s);
}

// The tile rows of the 256-column tiled kernels, by the same estimate as the
// plain dense forms: waves of 256 workgroups times the cost of a tile.
int tile_rows(int64_t M, int64_t cols, int64_t tile_cols) {
    const double c256 = (double)cdiv(cdiv(M, 256) * cdiv(cols, tile_cols), 256) * 2.0;
    const double c128 = (double)cdiv(cdiv(M, 128) * cdiv(cols, tile_cols), 256) * 1.15;
    return c128 < c256 ? 128 : 256;
}

}  // namespace
