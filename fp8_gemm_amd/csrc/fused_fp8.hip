// FP8 entry points of include/fp8_gemm_fused.h: checks, shape classes, launch.
#include "fused_host.hpp"

namespace {

using fp8g::EPI_ACT;
using fp8g::EPI_GATED;

template <int BM, int STAGES, int FA, int FB, int EPI>
int launch_tile(const FusedArgs &a, hipStream_t s) {
    FusedParams<EPI> p = with_epilogue<EPI>(a);
    p.tiles_m = (int)cdiv(p.M, BM);
    p.tiles_n = (int)cdiv(p.N, EPI == EPI_GATED ? 128 : 256);
    const dim3 grid((unsigned)(p.tiles_m * p.tiles_n)), block(256);
    if (p.K % 128)
        hipLaunchKernelGGL((fp8g::fused_tile16_kernel<BM, STAGES, FA, FB, true, EPI>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((fp8g::fused_tile16_kernel<BM, STAGES, FA, FB, false, EPI>), grid, block, 0, s, p);
    return launch_status("fused tiled kernel");
}

template <int FA, int FB, int EPI>
int launch_fmt(const FusedArgs &a, hipStream_t s) {
    if (a.M <= kFewMaxM) return launch_few_fmt<FA, FB, EPI>(a, s);
    if (tile_rows(a.M, a.N, EPI == EPI_GATED ? 128 : 256) == 128) return launch_tile<128, 3, FA, FB, EPI>(a, s);
    return launch_tile<256, 2, FA, FB, EPI>(a, s);
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
    if ((st = check_device())) return st;
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
    if ((st = check_device())) return st;
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
