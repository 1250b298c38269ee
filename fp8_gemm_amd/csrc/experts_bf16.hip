// BF16 entry points of include/fp8_gemm_experts.h.
#include "experts_host.hpp"

namespace {

using fp8g::EPI_STORE;

template <int BM, int BN, int STAGES>
int launch_sums_shape(const FusedArgs &a, const int32_t *offsets, int rows, hipStream_t s) {
    auto p = with_offsets<EPI_STORE, false, PLACE_SUMS>(a, offsets, rows);
    p.tiles_m = (int)cdiv(p.M, BM);
    p.tiles_n = (int)cdiv(p.N, BN);
    // Weight gradients larger than the last-level cache (256 MB) are stored past
    // it: 32 experts of 4096 x 2048 over 8192 rows 242 -> 189 us, 8 of 14336 x
    // 4096 908 -> 886 us; ones that fit it stay there for whoever reads them
    // next (17 of 1032 x 2056: 42.7 us, 48.1 past it).
    p.stream = (int64_t)p.G * p.M * p.N * 2 > (int64_t(256) << 20);
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
    if (const int st = check_tiles(tiles * p.G)) return st;
    const dim3 grid((unsigned)persistent_grid(tiles * p.G)), block(256);
    hipLaunchKernelGGL((fp8g::ragged_tile_kernel<BM, BN, STAGES, false, true, true, false, PLACE_SUMS, EPI_STORE>), grid,
                       block, 0, s, p);
    return launch_status("ragged weight gradient kernel");
}

}  // namespace

extern "C" {

int fp8_gemm_experts_plan(int op, int m, int n, int k, int groups, fp8g_plan *out) {
    if (!out) return fail(FP8G_ERR_NULL, "plan output pointer is NULL");
    *out = fp8g_plan{};
    out->k_splits = 1;
    if (op < 0 || op > 4) return fail(FP8G_ERR_ARG, "unknown op %d", op);
    const int unit = op == 1 || op == 4 ? 1 : 2;
    if (const int st = op == 4 ? check_sizes(m, n, k, 1) : check_ragged_sizes(m, groups, n, k, unit)) return st;
    const bool none = op == 4 ? m == 0 || n == 0 : op == 3 ? groups == 0 || n == 0 || k == 0 : m == 0 || (op == 2 ? k == 0 : n == 0 || groups == 0);
    // (sizes that the call itself refuses: no kernel either)
    if (none || (unit == 1 && check_int8_sizes(k)) || ((op == 2 || op == 3) && check_sum_rows(m))) return ok();
    ShapeClass c;
    int64_t tiles, cols;
    if (op == 3) {
        c = pick_sums(m, groups, n, k);
        tiles = cdiv(n, kClassRows[c - C_128x128]) * groups;
        cols = k;
    } else {
        const Choice choice = op == 4 ? pick_dense(m, n, k, n % 8 == 0)
                                      : op == 2 ? pick_ragged(R_TOKEN_GRAD, m, groups, k, n)
                                                : pick_ragged(op == 0 ? R_BF16 : R_INT8, m, groups, n, k);
        c = choice.c;
        if (c == C_FEW) {
            out->variant = 4;
            out->tile_m = 16 * choice.few.cb;
            out->tile_n = 16 * choice.few.rb;
            out->token_blocks = choice.few.cb;
            out->workgroups = choice.few.workgroups;
            return ok();
        }
        const int rows = (int)kClassRows[c - C_128x128];
        tiles = op == 4 ? cdiv(m, rows) : tiles_bound(m, groups + (op == 2 ? 2 : 0), rows);
        cols = op == 2 ? k : n;
    }
    tiles *= cdiv(cols, kClassCols[c - C_128x128]);
    if (tiles > (op == 4 && n % 8 ? kMaxWorkgroups : kMaxTiles)) return ok();
    out->variant = c == C_128x128 ? 7 : (c == C_128x256 ? 2 : 1);
    out->tile_m = (int)kClassRows[c - C_128x128];
    out->tile_n = (int)kClassCols[c - C_128x128];
    out->workgroups = tiles;
    return ok();
}

int bf16_grouped_gemm_ragged(const void *A, int64_t lda, const void *B, int64_t ldb, int64_t b_stride,
                             const int32_t *offsets, void *D, int64_t ldd, int M, int G, int N, int K, void *stream) {
    int st;
    if ((st = check_ragged_sizes(M, G, N, K, 2))) return st;
    if (M == 0 || N == 0 || G == 0) return ok();
    if ((st = check_operand("A", A, lda, K, 2)) || (st = check_operand("B", B, ldb, K, 2)) ||
        (st = check_stride("B", b_stride, ldb, G, N, K, 2)) || (st = check_offsets(offsets)) ||
        (st = check_tile_output("D", D, ldd, N)) ||
        (st = check_apart({area("D", D, ldd, M, N, 2)},
                          {area("A", A, lda, M, K, 2), experts_area("B", B, ldb, b_stride, G, N, K, 2),
                           area("offsets", offsets, G + 1, 4)})) ||
        (st = check_device()))
        return st;
    FusedArgs p = ragged_args(A, lda, B, ldb, b_stride, D, ldd, M, G, N, K, 2);
    const Choice c = pick_ragged(R_BF16, M, G, N, K);
    if (c.c != C_FEW) return launch_rows<false, false, PLACE_GROUPS, EPI_STORE>(c.c, p, offsets, static_cast<hipStream_t>(stream));
    p.K *= 2;
    return launch_ragged_few_shape<false>(p, c.few, offsets, static_cast<hipStream_t>(stream));
}

int bf16_grouped_gemm_ragged_backward(const void *dD, int64_t ldg, const void *A, int64_t lda, const void *B,
                                      int64_t ldb, int64_t b_stride, const int32_t *offsets, void *dA, int64_t ldda,
                                      void *dB, int64_t lddb, int64_t db_stride, int M, int G, int N, int K,
                                      void *stream) {
    int st;
    if ((st = check_ragged_sizes(M, G, N, K, 2))) return st;
    if ((st = check_sum_rows(M))) return st;
    const bool want_a = dA && M > 0 && K > 0, want_b = dB && G > 0 && N > 0 && K > 0;
    if (!want_a && !want_b) return ok();
    const bool sums = M > 0 && N > 0 && G > 0;       // anything to add up
    if ((st = check_offsets(offsets)) || (sums && (st = check_operand("dD", dD, ldg, N, 2)))) return st;
    if (want_a && ((sums && ((st = check_operand("B", B, ldb, K, 2)) || (st = check_stride("B", b_stride, ldb, G, N, K, 2)))) ||
                   (st = check_tile_output("dA", dA, ldda, K))))
        return st;
    if (want_b && ((sums && (st = check_operand("A", A, lda, K, 2))) || (st = check_tile_output("dB", dB, lddb, K)) ||
                   (st = check_stride("dB", db_stride, lddb, G, N, K, 2))))
        return st;
    if ((st = check_apart({area("dA", want_a ? dA : nullptr, ldda, M, K, 2),
                           experts_area("dB", want_b ? dB : nullptr, lddb, db_stride, G, N, K, 2)},
                          {area("dD", dD, ldg, M, N, 2), area("A", A, lda, want_b ? M : 0, K, 2),
                           experts_area("B", want_a ? B : nullptr, ldb, b_stride, G, N, K, 2),
                           area("offsets", offsets, G + 1, 4)})) ||
        (st = check_device()))
        return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (want_a) {
        const FusedArgs p = ragged_args(dD, ldg, B, ldb, b_stride, dA, ldda, M, G, K, N, 2);
        if ((st = launch_rows<false, true, PLACE_REST, EPI_STORE>(pick_ragged(R_TOKEN_GRAD, M, G, K, N).c, p, offsets, s))) return st;
    }
    if (want_b) {
        FusedArgs p = ragged_args(dD, ldg, A, lda, 0, dB, lddb, N, G, K, M, 2);
        p.d_gstride = db_stride;
        const ShapeClass c = pick_sums(M, G, N, K);
        if (c == C_128x128) return launch_sums_shape<128, 128, 4>(p, offsets, M, s);
        if (c == C_128x256) return launch_sums_shape<128, 256, 3>(p, offsets, M, s);
        return launch_sums_shape<256, 256, 2>(p, offsets, M, s);
    }
    return ok();
}

}  // extern "C"
