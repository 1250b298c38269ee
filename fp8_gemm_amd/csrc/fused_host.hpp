// Argument checks and launch helpers shared by the fused entry points
// (fused_fp8.hip, fused_bf16.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <initializer_list>

#include "../../include/fp8_gemm_fused.h"
#include "fused.hpp"
#include "host_common.hpp"

namespace {

using namespace fp8g_host;
using fp8g::FusedArgs;
using fp8g::FusedParams;

template <int E, bool SCALED>
FusedParams<E, SCALED> with_epilogue(const FusedArgs &a) {
    FusedParams<E, SCALED> p = {};
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

// A matrix in memory: rows of `width` bytes, `ld` bytes apart (ld >= width).
struct Area {
    const char *name;
    const void *ptr;
    int64_t ld, rows, width;
};

Area area(const char *name, const void *ptr, int64_t ld, int64_t rows, int64_t cols, int unit) {
    return Area{name, ptr, ld * unit, ptr ? rows : 0, cols * unit};
}
Area area(const char *name, const void *ptr, int64_t count, int unit) { return area(name, ptr, count, 1, count, unit); }

// Whether two matrices share a byte (rows of one may lie between rows of the
// other).  Rows are gone through one by one only where the strides differ and
// the spans of memory meet.
bool share(const Area &x, const Area &y) {
    if (x.rows <= 0 || y.rows <= 0 || x.width <= 0 || y.width <= 0) return false;
    const int64_t a = (int64_t)reinterpret_cast<uintptr_t>(x.ptr), b = (int64_t)reinterpret_cast<uintptr_t>(y.ptr);
    if (a >= b + (y.rows - 1) * y.ld + y.width || b >= a + (x.rows - 1) * x.ld + x.width) return false;
    auto floor_div = [](int64_t n, int64_t d) { return n / d - (n % d < 0); };
    // whether -before < gap + t ld < after for some t in lo .. hi
    auto meets = [&](int64_t gap, int64_t ld, int64_t before, int64_t after, int64_t lo, int64_t hi) {
        const int64_t first = -floor_div(before - 1 + gap, ld), last = floor_div(after - 1 - gap, ld);
        return (first > lo ? first : lo) <= (last < hi ? last : hi);
    };
    // (t: row of y less row of x)
    if (x.ld == y.ld) return meets(b - a, x.ld, y.width, x.width, 1 - x.rows, y.rows - 1);
    const bool swap = x.rows > y.rows;
    const Area &few = swap ? y : x, &many = swap ? x : y;
    const int64_t gap = swap ? a - b : b - a;
    for (int64_t i = 0; i < few.rows; ++i)
        if (meets(gap - i * few.ld, many.ld, many.width, few.width, 0, many.rows - 1)) return true;
    return false;
}

// No output may share memory with another output or an operand: tiles are
// written while others are still being read.
int check_apart(std::initializer_list<Area> outputs, std::initializer_list<Area> operands) {
    for (const Area *o = outputs.begin(); o != outputs.end(); ++o) {
        for (const Area *q = o + 1; q != outputs.end(); ++q)
            if (share(*o, *q)) return fail(FP8G_ERR_ARG, "%s and %s overlap", o->name, q->name);
        for (const Area &q : operands)
            if (share(*o, q)) return fail(FP8G_ERR_ARG, "%s overlaps %s", o->name, q.name);
    }
    return FP8G_OK;
}

// The residual of an output: another matrix, or the output itself.
Area residual_area(const void *R, int64_t ldr, const void *D, int64_t ldd, int M, int N) {
    const bool same = R == D && (ldr == ldd || M == 1);
    return area("R", same ? nullptr : R, ldr, M, N, 2);
}

// ---------------------------------------------------------------------------
// Shape classes: the few-token kernel (tokens in blocks of 16, 32 or 64, grid
// y over the 64-token tiles) and the tiled kernels of 128 x 128, 128 x 256 and
// 256 x 256 ring rows (gated: half as many output columns).
// ---------------------------------------------------------------------------
enum ShapeClass { C_FEW, C_128x128, C_128x256, C_256x256 };

struct FewShape {
    int rb, cb;                // 16-row weight blocks and 16-token blocks per workgroup
    int64_t workgroups;
};

constexpr int kFewWaves = 4;
constexpr int few_slots(int rb, int cb) { return rb == 1 && cb == 1 ? 3 : 2; }

FewShape few_shape(int64_t M, int64_t N, bool gated, int rb) {
    FewShape f;
    f.rb = rb;
    f.cb = M <= 16 ? 1 : (M <= 32 ? 2 : 4);
    f.workgroups = cdiv(N, gated ? 8 * rb : 16 * rb) * cdiv(M, 64);
    return f;
}

// The class with the smallest estimated time in us.  A tiled kernel's: a
// launch, and per wave of 256 workgroups (one per CU) a fixed part (prologue
// and epilogue) and its 128-byte K steps, each the slower the more CUs work
// (clock and memory); the few-token kernel's, for each number of weight rows
// per workgroup (more rows: fewer copies of the tokens, fewer workgroups): its
// rounds of workgroups, each a fixed part shared by the workgroups that fit a
// CU and the bytes that its copies bring in; all of them at least the time
// that memory takes for the operands and the output.  The constants are fitted
// to 540 measured cases (M 1 .. 2048 by nine N x K from 512 x 512 to 28672 x
// 1024 and 1024 x 8192, FP8 and BF16, fused and gated, every class each, the
// weights read from memory as a serving pass does): on average the choice
// takes 0.7% longer than the fastest class, in 16 cases over 10%, at worst 32%
// (FP8 fused 64 x 28672 x 1024: 64 rows 14.5 us, 128 x 128 tiles 11.0; gated
// BF16 64 x 14336 x 4096 54.1 against 46.1).  Most of those are few-token
// builds of 8 blocks, of which one workgroup fits a CU: the estimate is 11 to
// 16% too low there.  Narrower outputs and more tokens than the set's are
// extrapolated.  Some, FP8 fused, few-token with
// 16, 32 and 64 rows | 128 x 128 | 128 x 256 tiles, in us: 64 x 14336 x 4096
// 24.7, 20.7, 17.2 | 22.1 | 32.4; 256 x 4096 x 14336 61.1, 42.3, 33.3 | 72.0 |
// 99.2; 512 x 4096 x 4096 36.9, 28.8, 21.7 | 23.1 | 33.2; 64 x 4096 x 4096
// 8.8, 10.3, - | 19.9 | 30.8.
struct ClassCost {
    double launch, wave, step, load;
};
constexpr ClassCost kCost[2][3] = {{{1.6, 3.3, 0.416, 0.19}, {1.6, 5.4, 0.696, 0.219}, {0.9, 8.3, 1.266, 0.405}},
                                   {{2.0, 3.1, 0.416, 0.16}, {2.1, 4.6, 0.708, 0.191}, {-0.6, 11.0, 1.026, 0.258}}};
constexpr int64_t kClassRows[3] = {128, 128, 256}, kClassCols[3] = {128, 256, 256};

// us of a tiled kernel of class C_128x128 + c over `wgs` workgroups of `steps`
// 128-byte K steps.
double tiled_time(int c, int unit, int64_t wgs, int64_t steps) {
    const ClassCost &k = kCost[unit - 1][c];
    const double full = wgs < 256 ? (double)wgs / 256.0 : 1.0;
    return k.launch + (double)cdiv(wgs, 256) * (k.wave + (double)steps * (k.step + k.load * full));
}

constexpr int64_t kFewMaxM = 2048;                 // (its 64-token tiles re-read the weights from the caches)

struct Choice {
    ShapeClass c;
    FewShape few;              // C_FEW
};

// unit: bytes per element.
Choice pick_class(int64_t M, int64_t N, int64_t K, int unit, bool gated) {
    const double kbytes = (double)K * unit;
    const int64_t cols = gated ? 2 * N : N;
    const double memory = 2.0 + (kbytes * ((double)cols + (double)M) + 2.0 * (double)M * (double)N) / 5.0e6;
    auto floored = [&](double t) { return (t > memory ? t : memory) + 0.05 * t; };
    Choice best = {C_256x256, {}};
    double least = 1e300;
    if (M <= kFewMaxM) {
        for (int rb = gated ? 2 : 1; rb <= 4; rb *= 2) {
            const FewShape f = few_shape(M, N, gated, rb);
            int fit = 160 * 1024 / (kFewWaves * (f.rb + f.cb) * 2048 * few_slots(f.rb, f.cb));
            if (fit > 3) fit = 3;
            double rounds = fit == 1 ? (double)cdiv(f.workgroups, 256) : (double)f.workgroups / 256.0;
            if (rounds < 1.0) rounds = 1.0;
            const double t = floored(2.5 + rounds * (1.5 / fit + 16.0 * (f.rb + f.cb) * kbytes / 70e3));
            if (t < least) least = t, best = Choice{C_FEW, f};
        }
    }
    for (int c = 0; c < 3; ++c) {
        const double t = floored(tiled_time(c, unit, cdiv(M, kClassRows[c]) * cdiv(cols, kClassCols[c]), cdiv(K * unit, 128)));
        if (t < least) least = t, best = Choice{(ShapeClass)(C_128x128 + c), {}};
    }
    return best;
}

// A BF16 backward product (ny of M x N outputs, N a multiple of 8, reduced over
// K): its class, and the splits of K where the output has few tiles and K is
// long.  The splits' FP32 sums are written to the workspace and joined by a
// kernel of their own (3 us and the sums' way to memory and back), at most
// kJoinBytes of them.
struct BackwardShape {
    ShapeClass c;
    int splits, ksteps;
    int64_t bytes;             // workspace of the sums
};
constexpr int64_t kJoinBytes = int64_t(128) << 20;

BackwardShape backward_shape(int64_t M, int64_t N, int64_t K, int ny) {
    BackwardShape best = {C_256x256, 1, 0, 0};
    const int64_t steps = cdiv(2 * K, 128);
    double least = 1e300;
    for (int c = 0; c < 3; ++c) {
        const int64_t tiles = cdiv(M, kClassRows[c]) * cdiv(N, kClassCols[c]) * ny;
        for (int64_t want = 1; want <= 64; want *= 2) {
            if (want > 1 && (tiles * want > 512 || steps < 2 * want)) break;
            const int64_t per = steps ? cdiv(steps, want) : 0, splits = steps ? cdiv(steps, per) : 1;
            const int64_t bytes = splits > 1 ? splits * ny * M * N * 4 : 0;
            if (bytes > kJoinBytes) break;
            const double t = tiled_time(c, 2, tiles * splits, per) + (splits > 1 ? 3.0 + (double)bytes / 2.0e6 : 0.0);
            if (t < least) least = t, best = BackwardShape{(ShapeClass)(C_128x128 + c), (int)splits, (int)per, bytes};
        }
    }
    return best;
}

// ---------------------------------------------------------------------------
// Few-token launch: 16 RB weight rows per workgroup of 4 waves (gated: 8 RB of
// each matrix).
// ---------------------------------------------------------------------------
template <int RB, int CB, int FA, int FB, int EPI>
int launch_few(const FusedArgs &a, int64_t workgroups, hipStream_t s) {
    const auto p = with_epilogue<EPI, FA != fp8g::FMT_BF16>(a);
    const unsigned tiles = (unsigned)cdiv(p.M, 64);
    const dim3 grid((unsigned)(workgroups / tiles), tiles), block(64 * kFewWaves);
    hipLaunchKernelGGL((fp8g::fused_decode_kernel<kFewWaves, RB, CB, FA, FB, few_slots(RB, CB), EPI>), grid, block, 0, s, p);
    return launch_status("fused few-token kernel");
}

template <int RB, int FA, int FB, int EPI>
int launch_few_rb(const FusedArgs &a, const FewShape &f, hipStream_t s) {
    if (f.cb == 1) return launch_few<RB, 1, FA, FB, EPI>(a, f.workgroups, s);
    if (f.cb == 2) return launch_few<RB, 2, FA, FB, EPI>(a, f.workgroups, s);
    return launch_few<RB, 4, FA, FB, EPI>(a, f.workgroups, s);
}

template <int FA, int FB, int EPI>
int launch_few_fmt(const FusedArgs &a, const FewShape &f, hipStream_t s) {
    if constexpr (EPI != fp8g::EPI_GATED) {
        if (f.rb == 1) return launch_few_rb<1, FA, FB, EPI>(a, f, s);
    }
    if (f.rb == 2) return launch_few_rb<2, FA, FB, EPI>(a, f, s);
    return launch_few_rb<4, FA, FB, EPI>(a, f, s);
}

}  // namespace
