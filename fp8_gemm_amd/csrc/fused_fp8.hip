// FP8 entry points of include/fp8_gemm_fused.h: checks, shape classes, launch.
#include "fused_host.hpp"

namespace {

using fp8g::EPI_ACT;
using fp8g::EPI_GATED;

template <int BM, int BN, int STAGES, int FA, int FB, int EPI>
int launch_tile(const FusedArgs &a, hipStream_t s) {
    auto p = with_epilogue<EPI, true>(a);
    p.tiles_m = (int)cdiv(p.M, BM);
    p.tiles_n = (int)cdiv(p.N, EPI == EPI_GATED ? BN / 2 : BN);
    const dim3 grid((unsigned)(p.tiles_m * p.tiles_n)), block(256);
    if (p.K % 128)
        hipLaunchKernelGGL((fp8g::fused_tile16_kernel<BM, BN, STAGES, FA, FB, true, EPI>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((fp8g::fused_tile16_kernel<BM, BN, STAGES, FA, FB, false, EPI>), grid, block, 0, s, p);
    return launch_status("fused tiled kernel");
}

template <int FA, int FB, int EPI>
int launch_fmt(const FusedArgs &a, hipStream_t s) {
    const Choice c = pick_class(a.M, a.N, a.K, 1, EPI == EPI_GATED);
    switch (c.c) {
    case C_FEW: return launch_few_fmt<FA, FB, EPI>(a, c.few, s);
    case C_128x128: return launch_tile<128, 128, 4, FA, FB, EPI>(a, s);
    case C_128x256: return launch_tile<128, 256, 3, FA, FB, EPI>(a, s);
    default: return launch_tile<256, 256, 2, FA, FB, EPI>(a, s);
    }
}

template <int EPI>
int launch(int fa, int fb, const FusedArgs &a, hipStream_t s) {
    if (fa == 0 && fb == 0) return launch_fmt<0, 0, EPI>(a, s);
    if (fa == 0 && fb == 1) return launch_fmt<0, 1, EPI>(a, s);
    if (fa == 1 && fb == 0) return launch_fmt<1, 0, EPI>(a, s);
    return launch_fmt<1, 1, EPI>(a, s);
}

}  // namespace

extern "C" {

int fp8_gemm_fused_plan(int op, int m, int n, int k, fp8g_plan *out) {
    if (!out) return fail(FP8G_ERR_NULL, "plan output pointer is NULL");
    *out = fp8g_plan{};
    out->k_splits = 1;
    const int products = op == 4 + FP8G_PLAN_PAIR ? 2 : 1;
    if (products == 2) op = 4;
    if (op < 0 || op > 4) return fail(FP8G_ERR_ARG, "unknown op %d", op);
    if (op < 4) {
        if (const int st = check_sizes(m, n, k, op < 2 ? 1 : 2)) return st;
    } else if (m < 0 || n < 0 || k < 0) {
        return fail(FP8G_ERR_SHAPE, "negative size (m=%d n=%d k=%d)", m, n, k);
    }
    if (m == 0 || n == 0) return ok();
    const bool gated = op == 1 || op == 3;
    ShapeClass c;
    if (op == 4) {
        const BackwardShape b = backward_shape(m, n, k, products);
        c = b.c;
        out->k_splits = b.splits;
    } else {
        const Choice choice = pick_class(m, n, k, op < 2 ? 1 : 2, gated);
        c = choice.c;
        if (c == C_FEW) {
            const FewShape &f = choice.few;
            out->variant = 4;
            out->tile_m = 16 * f.cb;
            out->tile_n = gated ? 8 * f.rb : 16 * f.rb;
            out->token_blocks = f.cb;
            out->workgroups = f.workgroups;
            return ok();
        }
    }
    out->variant = c == C_128x128 ? 7 : (c == C_128x256 ? 2 : 1);
    out->tile_m = c == C_256x256 ? 256 : 128;
    out->tile_n = (c == C_128x128 ? 128 : 256) / (gated ? 2 : 1);
    out->workgroups = cdiv(m, out->tile_m) * cdiv(n, out->tile_n) * out->k_splits * products;
    return ok();
}

int fp8_gemm_nt_fused(const void *A, int64_t lda, int a_dtype, const void *B, int64_t ldb, int b_dtype,
                      const float *scale_a, int scale_a_n, const float *scale_b, int scale_b_n, const float *bias,
                      int activation, const void *R, int64_t ldr, void *D, int64_t ldd, int M, int N, int K,
                      void *stream) {
    FusedArgs p = {};
    int st;
    if (!dtype_ok(a_dtype) || !dtype_ok(b_dtype)) return fail(FP8G_ERR_DTYPE, "dtypes %d, %d", a_dtype, b_dtype);
    if ((st = check_sizes(M, N, K, 1)) || (st = check_activation(activation))) return st;
    if (M == 0 || N == 0) return ok();
    if ((st = check_operand("A", A, lda, K, 1)) || (st = check_operand("B", B, ldb, K, 1)) ||
        (st = check_output("D", D, ldd, N)) || (st = check_scale("scale_a", scale_a, scale_a_n, M, &p.sa_step)) ||
        (st = check_scale("scale_b", scale_b, scale_b_n, N, &p.sb_step)) || (st = check_floats("bias", bias)))
        return st;
    if (R && (st = check_rows("R", R, ldr, N, 2, &p.r_vec))) return st;
    if ((st = check_apart({area("D", D, ldd, M, N, 2)},
                          {area("A", A, lda, M, K, 1), area("B", B, ldb, N, K, 1), residual_area(R, ldr, D, ldd, M, N),
                           area("scale_a", scale_a, scale_a_n, 4), area("scale_b", scale_b, scale_b_n, 4),
                           area("bias", bias, N, 4)})) ||
        (st = check_device()))
        return st;
    p.A = static_cast<const uint8_t *>(A);
    p.B = static_cast<const uint8_t *>(B);
    p.D = static_cast<uint16_t *>(D);
    p.lda = lda; p.ldb = ldb; p.ldd = ldd;
    p.M = M; p.N = N; p.K = K; p.G = 1; p.cap = M;
    p.ch_sa = scale_a; p.ch_sb = scale_b; p.bias = bias;
    p.act = activation;
    p.R = static_cast<const uint16_t *>(R); p.ldr = ldr;
    return launch<EPI_ACT>(a_dtype, b_dtype, p, static_cast<hipStream_t>(stream));
}

int fp8_gated_nt(const void *A, int64_t lda, int a_dtype, const void *Wg, int64_t ldg, const void *Wu, int64_t ldu,
                 int w_dtype, const float *scale_a, int scale_a_n, const float *scale_g, const float *scale_u,
                 int scale_w_n, int activation, void *D, int64_t ldd, int M, int N, int K, void *stream) {
    FusedArgs p = {};
    int st, step_u = 0;
    if (!dtype_ok(a_dtype) || !dtype_ok(w_dtype)) return fail(FP8G_ERR_DTYPE, "dtypes %d, %d", a_dtype, w_dtype);
    if ((st = check_sizes(M, N, K, 1)) || (st = check_activation(activation))) return st;
    if (M == 0 || N == 0) return ok();
    if ((st = check_operand("A", A, lda, K, 1)) || (st = check_operand("Wg", Wg, ldg, K, 1)) ||
        (st = check_operand("Wu", Wu, ldu, K, 1)) || (st = check_output("D", D, ldd, N)) ||
        (st = check_scale("scale_a", scale_a, scale_a_n, M, &p.sa_step)) ||
        (st = check_scale("scale_g", scale_g, scale_w_n, N, &p.sb_step)) ||
        (st = check_scale("scale_u", scale_u, scale_w_n, N, &step_u)))
        return st;
    if ((st = check_apart({area("D", D, ldd, M, N, 2)},
                          {area("A", A, lda, M, K, 1), area("Wg", Wg, ldg, N, K, 1), area("Wu", Wu, ldu, N, K, 1),
                           area("scale_a", scale_a, scale_a_n, 4), area("scale_g", scale_g, scale_w_n, 4),
                           area("scale_u", scale_u, scale_w_n, 4)})) ||
        (st = check_device()))
        return st;
    p.A = static_cast<const uint8_t *>(A);
    p.B = static_cast<const uint8_t *>(Wg);
    p.B2 = static_cast<const uint8_t *>(Wu);
    p.D = static_cast<uint16_t *>(D);
    p.lda = lda; p.ldb = ldg; p.ldb2 = ldu; p.ldd = ldd;
    p.M = M; p.N = N; p.K = K; p.G = 1; p.cap = M;
    p.ch_sa = scale_a; p.ch_sb = scale_g; p.ch_sb2 = scale_u;
    p.sb_step = scale_g ? p.sb_step : step_u;      // (one length for both)
    p.act = activation;
    return launch<EPI_GATED>(a_dtype, w_dtype, p, static_cast<hipStream_t>(stream));
}

}  // extern "C"
