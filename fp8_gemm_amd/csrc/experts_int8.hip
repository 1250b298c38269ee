// Entry points of include/fp8_gemm_experts.h in 8-bit integers.
#include "experts_host.hpp"
#include "quantize.hpp"

namespace {

using fp8g::EPI_ACT;
using fp8g::EPI_SCALED;
using fp8g::FMT_I8;
using fp8g::QuantParams;

template <int BM, int BN, int STAGES, int EPI>
int launch_epilogue(const FusedArgs &a, hipStream_t s) {
    fp8g::Int8Params<EPI> p = {};
    static_cast<FusedArgs &>(p) = a;
    p.tiles_m = (int)cdiv(p.M, BM);
    p.tiles_n = (int)cdiv(p.N, BN);
    const int64_t wgs = (int64_t)p.tiles_m * p.tiles_n;
    if (EPI != EPI_SCALED && wgs > kMaxWorkgroups) return fail(FP8G_ERR_SHAPE, "%lld workgroups: too many for one launch", (long long)wgs);
    if (const int st = check_tiles(wgs)) return st;
    const dim3 grid((unsigned)(EPI == EPI_SCALED ? persistent_grid(wgs) : wgs)), block(256);
    if (p.K % 128) hipLaunchKernelGGL((fp8g::int8_tile_kernel<BM, BN, STAGES, true, EPI>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((fp8g::int8_tile_kernel<BM, BN, STAGES, false, EPI>), grid, block, 0, s, p);
    return launch_status("int8 tiled kernel");
}

// Scales and bias alone, in whole chunks of 8 columns, take the persistent
// form, whose offsets into a tile's output are 32-bit.
bool direct_epilogue(const FusedArgs &a) {
    return a.act == FP8G_ACT_NONE && !a.R && a.N % 8 == 0 && 2 * a.ldd <= kMaxRowStride;
}

template <int BM, int BN, int STAGES>
int launch_dense(const FusedArgs &a, bool direct, hipStream_t s) {
    return direct ? launch_epilogue<BM, BN, STAGES, EPI_SCALED>(a, s) : launch_epilogue<BM, BN, STAGES, EPI_ACT>(a, s);
}

// Workgroups of `threads` threads over `rows` rows each.  A launch holds fewer
// than 2^32 threads; more rows take another one.
int launch_quant_rows(void (*kernel)(QuantParams), QuantParams p, int rows, int threads, hipStream_t s) {
    const int64_t most = ((int64_t(1) << 32) - 1) / threads * rows;
    for (int64_t left = p.M; left > 0; left -= most) {
        p.M = (int)(left < most ? left : most);
        hipLaunchKernelGGL(kernel, dim3((unsigned)cdiv(p.M, rows)), dim3(threads), 0, s, p);
        if (const int st = launch_status("row quantisation kernel")) return st;
        p.X += most * p.ldx;
        p.Q += most * p.ldq;
        p.scale += most;
    }
    return ok();
}

template <int T, int R>
int launch_quant(const QuantParams &p, hipStream_t s) {
    return launch_quant_rows(fp8g::quantize_rows_kernel<T, R>, p, T < 256 ? 256 / T : 1, T < 256 ? 256 : T, s);
}

// (the numbers of chunks that the rule of int8_quantize_rows leaves each T)
template <int T>
int launch_quant_chunks(const QuantParams &p, hipStream_t s) {
    const int64_t chunks = cdiv(p.K, 8 * T);
    if constexpr (T < 1024) {
        if (chunks <= 1) return launch_quant<T, 1>(p, s);
    }
    if (chunks <= 2) return launch_quant<T, 2>(p, s);
    if constexpr (T > 64) {
        if (chunks > 4) return launch_quant<T, 8>(p, s);
    }
    return launch_quant<T, 4>(p, s);
}

}  // namespace

extern "C" {

int int8_grouped_gemm_ragged(const void *A, int64_t lda, const void *B, int64_t ldb, int64_t b_stride,
                             const float *scale_a, const float *scale_b, const int32_t *offsets, void *D, int64_t ldd,
                             int M, int G, int N, int K, void *stream) {
    int st;
    if ((st = check_ragged_sizes(M, G, N, K, 1)) || (st = check_int8_sizes(K))) return st;
    if (M == 0 || N == 0 || G == 0) return ok();
    if ((st = check_operand("A", A, lda, K, 1)) || (st = check_operand("B", B, ldb, K, 1)) ||
        (st = check_stride("B", b_stride, ldb, G, N, K, 1)) || (st = check_offsets(offsets)) ||
        (st = check_floats("scale_a", scale_a)) || (st = check_floats("scale_b", scale_b)) ||
        (st = check_tile_output("D", D, ldd, N)) ||
        (st = check_apart({area("D", D, ldd, M, N, 2)},
                          {area("A", A, lda, M, K, 1), experts_area("B", B, ldb, b_stride, G, N, K, 1),
                           area("scale_a", scale_a, M, 4), area("scale_b", scale_b, (int64_t)G * N, 4),
                           area("offsets", offsets, G + 1, 4)})) ||
        (st = check_device()))
        return st;
    FusedArgs p = ragged_args(A, lda, B, ldb, b_stride, D, ldd, M, G, N, K, 1);
    p.ch_sa = scale_a; p.ch_sb = scale_b;
    p.sa_step = p.sb_step = 1;
    p.act = FP8G_ACT_NONE;
    const Choice c = pick_ragged(R_INT8, M, G, N, K);
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (c.c == C_FEW) return launch_ragged_few_shape<true>(p, c.few, offsets, s);
    return launch_rows<true, false, PLACE_GROUPS, EPI_SCALED>(c.c, p, offsets, s);
}

int int8_gemm_nt_fused(const void *A, int64_t lda, const void *B, int64_t ldb, const float *scale_a, int scale_a_n,
                       const float *scale_b, int scale_b_n, const float *bias, int activation, const void *R,
                       int64_t ldr, void *D, int64_t ldd, int M, int N, int K, void *stream) {
    FusedArgs p = {};
    int st;
    if ((st = check_sizes(M, N, K, 1)) || (st = check_int8_sizes(K)) || (st = check_activation(activation))) return st;
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
    p.B2 = p.B;
    p.D = static_cast<uint16_t *>(D);
    p.D2 = p.D;
    p.lda = lda; p.ldb = ldb; p.ldb2 = ldb; p.ldd = ldd;
    p.M = M; p.N = N; p.K = K; p.G = 1; p.cap = M;
    p.ch_sa = scale_a; p.ch_sb = scale_b; p.bias = bias;
    p.act = activation;
    p.R = static_cast<const uint16_t *>(R); p.ldr = ldr;
    p.ksplit = 1 << 30;
    p.krows = K;
    const bool direct = direct_epilogue(p);
    const Choice c = pick_dense(M, N, K, direct);
    hipStream_t s = static_cast<hipStream_t>(stream);
    switch (c.c) {
    case C_FEW: return launch_few_fmt<FMT_I8, FMT_I8, EPI_ACT>(p, c.few, s);
    case C_128x128: return launch_dense<128, 128, 4>(p, direct, s);
    case C_128x256: return launch_dense<128, 256, 3>(p, direct, s);
    default: return launch_dense<256, 256, 2>(p, direct, s);
    }
}

int int8_quantize_rows(const void *X, int64_t ldx, void *Q, int64_t ldq, float *scale, int M, int K, void *stream) {
    if (M < 0 || K < 0) return fail(FP8G_ERR_SHAPE, "negative size (M=%d K=%d)", M, K);
    if (K % 16) return fail(FP8G_ERR_SHAPE, "K=%d is not a multiple of 16", K);
    if (M == 0) return ok();
    int st;
    if (!scale) return fail(FP8G_ERR_NULL, "scale is required");
    if ((st = check_floats("scale", scale)) || (st = check_operand("X", X, ldx, K, 2))) return st;
    if (K > 0 && !Q) return fail(FP8G_ERR_NULL, "Q is required");
    if (!aligned16(Q)) return fail(FP8G_ERR_ALIGN, "Q must be 16-byte aligned");
    if (ldq < K) return fail(FP8G_ERR_STRIDE, "row stride %lld of Q below K=%d", (long long)ldq, K);
    if (ldq % 16) return fail(FP8G_ERR_ALIGN, "row stride %lld of Q is not a multiple of 16 bytes", (long long)ldq);
    if ((st = check_apart({area("Q", Q, ldq, M, K, 1), area("scale", scale, M, 4)}, {area("X", X, ldx, M, K, 2)})) ||
        (st = check_device()))
        return st;
    QuantParams p = {};
    p.X = static_cast<const uint16_t *>(X);
    p.Q = static_cast<int8_t *>(Q);
    p.scale = scale;
    p.ldx = ldx; p.ldq = ldq;
    p.M = M; p.K = K;
    hipStream_t s = static_cast<hipStream_t>(stream);
    // Threads per row: enough of them to have a row's loads in flight at once,
    // few where rows are many and short.  Measured (us in a graph; 64 | 256 |
    // 1024 threads): 512 x 1024 values 2.56 | 2.69 | 3.37, 64 x 2048 2.87 | 2.57 |
    // 2.66, 8192 x 2048 9.8 | 10.9 | 24, 256 x 4096 3.57 | 2.82 | 2.91, 2048 x 8192
    // - | 9.4 | 12.7, 64 x 14336 - | 3.62 | 3.35, 1024 x 14336 - | 8.6 | 9.1, 8192 x
    // 14336 - | 65.2 | 60.9.  On another box, three inputs in turn, 256 | 1024
    // threads: 512 x 10240 4.65 | 5.16, 2048 x 10240 11.6 | 13.3, 4096 x 10240 21.3 |
    // 23.7, 256 x 12288 3.70 | 3.66, 1024 x 12288 8.97 | 9.16, 4096 x 12288 25.1 |
    // 25.6, 8192 x 12288 50.1 | 47.1, 256 x 16384 4.20 | 3.94, 512 x 16384 7.26 |
    // 7.06, 2048 x 16384 16.9 | 17.6, 4096 x 16384 32.6 | 34.0, 8192 x 16384 73.8 |
    // 70.0: what is taken is within 5% of the other but for 4096 and more rows of
    // about 10000 values (7 to 12%).
    if (K <= 1024 || (K <= 2048 && M >= 1024)) return launch_quant_chunks<64>(p, s);
    if (K <= 8192 || (K <= 16384 && M >= 512 && M < 4096)) return launch_quant_chunks<256>(p, s);
    if (K <= 65536) return launch_quant_chunks<1024>(p, s);
    return launch_quant_rows(fp8g::quantize_long_rows_kernel, p, 1, 1024, s);
}

}  // extern "C"
