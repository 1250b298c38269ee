// BF16 entry points of include/fp8_gemm_fused.h: checks, shape classes, launch.
#include "fused_bf16.hpp"
#include "fused_host.hpp"

namespace {

using fp8g::EPI_ACT;
using fp8g::EPI_GATED;
using fp8g::EPI_PARTIAL;
using fp8g::EPI_STORE;
using fp8g::FMT_BF16;
using fp8g::GradParams;

// grid: y over products sharing the launch, z over splits of K.
template <int BM, int BN, int STAGES, bool TA, bool TB, int EPI>
int launch_shape(const FusedArgs &a, int ny, int splits, hipStream_t s) {
    auto p = with_epilogue<EPI, false>(a);
    p.tiles_m = (int)cdiv(p.M, BM);
    p.tiles_n = (int)cdiv(p.N, EPI == EPI_GATED ? BN / 2 : BN);
    const dim3 grid((unsigned)(p.tiles_m * p.tiles_n), (unsigned)ny, (unsigned)splits), block(256);
    if (!(TA && TB) && p.K % 64)
        hipLaunchKernelGGL((fp8g::bf16_tile_kernel<BM, BN, STAGES, TA, TB, !(TA && TB), EPI>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((fp8g::bf16_tile_kernel<BM, BN, STAGES, TA, TB, false, EPI>), grid, block, 0, s, p);
    return launch_status("fused BF16 tiled kernel");
}

template <bool TA, bool TB, int EPI>
int launch_tile(ShapeClass c, const FusedArgs &a, int ny, int splits, hipStream_t s) {
    if (c == C_128x128) return launch_shape<128, 128, 4, TA, TB, EPI>(a, ny, splits, s);
    if (c == C_128x256) return launch_shape<128, 256, 3, TA, TB, EPI>(a, ny, splits, s);
    return launch_shape<256, 256, 2, TA, TB, EPI>(a, ny, splits, s);
}

// The forward products.  The few-token kernel counts K and the operands'
// strides in bytes, the tiled kernel K in elements.
template <int EPI>
int launch_forward(FusedArgs p, hipStream_t s) {
    const Choice c = pick_class(p.M, p.N, p.K, 2, EPI == EPI_GATED);
    if (c.c == C_FEW) {
        p.K *= 2;
        return launch_few_fmt<FMT_BF16, FMT_BF16, EPI>(p, c.few, s);
    }
    return launch_tile<false, false, EPI>(c.c, p, 1, 1, s);
}

// A backward product (ny of them), its split sums in `sums`.
template <bool TA, bool TB>
int launch_backward(FusedArgs p, int ny, float *sums, hipStream_t s) {
    const BackwardShape b = backward_shape(p.M, p.N, p.K, ny);
    if (b.splits == 1) return launch_tile<TA, TB, EPI_STORE>(b.c, p, ny, 1, s);
    p.ws = sums;
    p.ksteps = b.ksteps;
    if (const int st = launch_tile<TA, TB, EPI_PARTIAL>(b.c, p, ny, b.splits, s)) return st;
    const dim3 grid((unsigned)cdiv((int64_t)p.M * p.N, 256 * 8), (unsigned)ny);
    hipLaunchKernelGGL(fp8g::join_kernel, grid, dim3(256), 0, s, sums, b.splits, p.M, p.N, p.D, p.D2, p.ldd);
    return launch_status("join kernel");
}

FusedArgs base_args(const void *A, int64_t lda, const void *B, int64_t ldb, void *D, int64_t ldd, int M, int N, int K) {
    FusedArgs p = {};
    p.A = static_cast<const uint8_t *>(A);
    p.B = static_cast<const uint8_t *>(B);
    p.B2 = p.B;
    p.D = static_cast<uint16_t *>(D);
    p.D2 = p.D;
    p.lda = 2 * lda; p.ldb = 2 * ldb; p.ldb2 = p.ldb; p.ldd = ldd;
    p.M = M; p.N = N; p.K = K; p.G = 1; p.cap = M;
    p.ksplit = 1 << 30;
    p.krows = K;
    return p;
}

int64_t pad64(int64_t n) { return (n + 63) / 64 * 64; }
int64_t pad256(int64_t n) { return (n + 255) / 256 * 256; }

// Parts of the backward workspaces: the gradients of the pre-activations, the
// bias gradient's partial sums, and the split sums of either product (dA [M x
// K] reduced over `cols`, nw weight gradients [N x K] reduced over M), which
// follow one another.
int64_t grad_bytes(int64_t M, int64_t cols) { return pad256(2 * M * cols); }
// Rows per block of the pre-activation gradients: 64, or fewer while there
// are not 1024 blocks.
int grad_rows(int64_t M, int64_t cols) {
    int rows = fp8g::kGradMaxRows;
    while (rows > 8 && cdiv(M, rows) * cdiv(cols, 256) < 1024) rows /= 2;
    return rows;
}
int64_t bias_bytes(int64_t M, int64_t N) { return pad256(4 * cdiv(M, grad_rows(M, pad64(N))) * N); }
int64_t join_bytes(int64_t M, int64_t N, int64_t K, int64_t cols, int nw) {
    if (K == 0) return 0;
    const int64_t a = backward_shape(M, K, cols, 1).bytes, w = backward_shape(N, K, M, nw).bytes;
    return a > w ? a : w;
}

int check_workspace(const void *ws, int64_t bytes, int64_t need) {
    if (need == 0) return FP8G_OK;
    if (!ws) return fail(FP8G_ERR_NULL, "workspace is required");
    if (reinterpret_cast<uintptr_t>(ws) % 256) return fail(FP8G_ERR_ALIGN, "workspace must be 256-byte aligned");
    if (bytes < need) return fail(FP8G_ERR_ARG, "workspace of %lld bytes: %lld are needed", (long long)bytes, (long long)need);
    return FP8G_OK;
}

int check_grad_sizes(int M, int N) {
    if (M < 0 || N < 0) return fail(FP8G_ERR_SHAPE, "negative size (M=%d N=%d)", M, N);
    // gradients of the pre-activations: rows of at most two matrices' columns
    if (4 * pad64(N) > kMaxRowStride) return fail(FP8G_ERR_SHAPE, "N=%d exceeds the workspace's row limit", N);
    // M is the reduction length of the weight gradients, counted in K steps
    if (M > (1 << 30)) return fail(FP8G_ERR_SHAPE, "M=%d exceeds %d", M, 1 << 30);
    return FP8G_OK;
}

template <bool GATED, bool BIAS>
int launch_grad(GradParams g, int cols, hipStream_t s) {
    g.rows = grad_rows(g.M, cols);
    const dim3 grid((unsigned)cdiv(g.M, g.rows), (unsigned)cdiv(cols, 256));
    hipLaunchKernelGGL((fp8g::grad_kernel<GATED, BIAS>), grid, dim3(256), 0, s, g);
    return launch_status("pre-activation gradient kernel");
}

}  // namespace

extern "C" {

int bf16_gemm_nt_fused(const void *A, int64_t lda, const void *B, int64_t ldb, const float *bias, int activation,
                       const void *R, int64_t ldr, void *D, int64_t ldd, float *preact, int64_t ldp, int M, int N,
                       int K, void *stream) {
    int st, r_vec = 0, p_vec = 0;
    if ((st = check_sizes(M, N, K, 2)) || (st = check_activation(activation))) return st;
    if (M == 0 || N == 0) return ok();
    if ((st = check_operand("A", A, lda, K, 2)) || (st = check_operand("B", B, ldb, K, 2)) ||
        (st = check_output("D", D, ldd, N)) || (st = check_floats("bias", bias)))
        return st;
    if (R && (st = check_rows("R", R, ldr, N, 2, &r_vec))) return st;
    if (preact && (st = check_rows("preact", preact, ldp, N, 4, &p_vec))) return st;
    if ((st = check_apart({area("D", D, ldd, M, N, 2), area("preact", preact, ldp, M, N, 4)},
                          {area("A", A, lda, M, K, 2), area("B", B, ldb, N, K, 2), area("bias", bias, N, 4),
                           residual_area(R, ldr, D, ldd, M, N)})) ||
        (st = check_device()))
        return st;
    FusedArgs p = base_args(A, lda, B, ldb, D, ldd, M, N, K);
    p.bias = bias;
    p.act = activation;
    p.R = static_cast<const uint16_t *>(R); p.ldr = ldr; p.r_vec = r_vec;
    p.pre = preact; p.ldp = ldp; p.p_vec = p_vec;
    return launch_forward<EPI_ACT>(p, static_cast<hipStream_t>(stream));
}

int64_t bf16_gemm_nt_fused_backward_workspace(int M, int N, int K) {
    int st;
    if ((st = check_sizes(M, N, K, 2)) || (st = check_grad_sizes(M, N))) return st;
    return grad_bytes(M, pad64(N)) + bias_bytes(M, N) + join_bytes(M, N, K, pad64(N), 1);
}

int bf16_gemm_nt_fused_backward(const void *G, int64_t ldg, const void *A, int64_t lda, const void *B, int64_t ldb,
                                const float *preact, int64_t ldp, int activation, void *dA, int64_t ldda, void *dB,
                                int64_t lddb, float *dbias, void *workspace, int64_t workspace_bytes, int M, int N,
                                int K, void *stream) {
    int st, g_vec = 0, p_vec = 0;
    if ((st = check_sizes(M, N, K, 2)) || (st = check_grad_sizes(M, N)) || (st = check_activation(activation))) return st;
    if (N == 0 && (M == 0 || K == 0 || !dA)) return ok();
    if (N > 0 && M > 0) {
        if (!G) return fail(FP8G_ERR_NULL, "G is required");
        if ((st = check_rows("G", G, ldg, N, 2, &g_vec))) return st;
        if (activation != FP8G_ACT_NONE && !preact) return fail(FP8G_ERR_NULL, "preact is required");
        if (activation != FP8G_ACT_NONE && (st = check_rows("preact", preact, ldp, N, 4, &p_vec))) return st;
        if ((st = check_workspace(workspace, workspace_bytes, bf16_gemm_nt_fused_backward_workspace(M, N, K)))) return st;
    }
    const bool want_a = dA && M > 0 && K > 0, want_b = dB && N > 0 && K > 0;
    if (want_a && ((N > 0 && (st = check_operand("B", B, ldb, K, 2))) || (st = check_output("dA", dA, ldda, K)))) return st;
    if (want_b && ((M > 0 && (st = check_operand("A", A, lda, K, 2))) || (st = check_output("dB", dB, lddb, K)))) return st;
    if ((st = check_floats("dbias", dbias)) ||
        (st = check_apart({area("dA", want_a ? dA : nullptr, ldda, M, K, 2), area("dB", want_b ? dB : nullptr, lddb, N, K, 2),
                           area("dbias", dbias, N, 4),
                           area("workspace", workspace, M > 0 && N > 0 ? bf16_gemm_nt_fused_backward_workspace(M, N, K) : 0, 1)},
                          {area("G", G, ldg, M, N, 2), area("A", A, lda, want_b ? M : 0, K, 2),
                           area("B", B, ldb, want_a ? N : 0, K, 2),
                           area("preact", activation != FP8G_ACT_NONE ? preact : nullptr, ldp, M, N, 4)})) ||
        (st = check_device()))
        return st;
    hipStream_t s = static_cast<hipStream_t>(stream);

    // dZ: G itself where there is no activation and its rows are whole chunks,
    // else formed in the workspace
    const bool direct = activation == FP8G_ACT_NONE && g_vec && N % 8 == 0 && 2 * ldg <= kMaxRowStride;
    const int64_t cols = pad64(N);
    uint16_t *const w = static_cast<uint16_t *>(workspace);
    float *const part = reinterpret_cast<float *>(static_cast<char *>(workspace) + grad_bytes(M, cols));
    float *const sums = reinterpret_cast<float *>(static_cast<char *>(workspace) + grad_bytes(M, cols) + bias_bytes(M, N));
    if (M > 0 && N > 0 && (dbias || (!direct && (want_a || want_b)))) {
        GradParams g = {};
        g.G = static_cast<const uint16_t *>(G); g.ldg = ldg; g.g_vec = g_vec;
        if (activation != FP8G_ACT_NONE) { g.pre = preact; g.ldp = ldp; g.p_vec = p_vec; }
        g.W = direct || !(want_a || want_b) ? nullptr : w;
        g.ldw = cols;
        g.part = part;
        g.M = M; g.N = N; g.act = activation;
        st = dbias ? launch_grad<false, true>(g, (int)cols, s) : launch_grad<false, false>(g, (int)cols, s);
        if (st) return st;
    }
    if (dbias && N > 0) {
        hipLaunchKernelGGL(fp8g::bias_grad_kernel, dim3((unsigned)cdiv(N, 32)), dim3(256), 0, s, part,
                           (int)cdiv(M, grad_rows(M, cols)), N, dbias);
        if ((st = launch_status("bias gradient kernel"))) return st;
    }
    const void *dz = direct ? G : w;
    const int64_t ldz = direct ? ldg : cols;
    if (want_a) {
        // dA [M x K] = dZ [M x N] . B [N x K]: the padding columns of the
        // workspace's dZ are zero, and B's rows past N read as zeros
        FusedArgs p = base_args(dz, ldz, B, ldb, dA, ldda, M, K, direct ? N : (int)cols);
        p.krows = N;
        if ((st = launch_backward<false, true>(p, 1, sums, s))) return st;
    }
    if (want_b) {
        FusedArgs p = base_args(dz, ldz, A, lda, dB, lddb, N, K, M);
        if ((st = launch_backward<true, true>(p, 1, sums, s))) return st;
    }
    return ok();
}

int bf16_gated_nt(const void *A, int64_t lda, const void *Wg, int64_t ldg, const void *Wu, int64_t ldu, int activation,
                  void *D, int64_t ldd, float *pre_g, float *pre_u, int64_t ldp, int M, int N, int K, void *stream) {
    int st, p_vec = 0, p_vec2 = 0;
    if ((st = check_sizes(M, N, K, 2)) || (st = check_activation(activation))) return st;
    if (M == 0 || N == 0) return ok();
    if ((st = check_operand("A", A, lda, K, 2)) || (st = check_operand("Wg", Wg, ldg, K, 2)) ||
        (st = check_operand("Wu", Wu, ldu, K, 2)) || (st = check_output("D", D, ldd, N)))
        return st;
    if (!pre_g != !pre_u) return fail(FP8G_ERR_NULL, "pre_g and pre_u are given together or not at all");
    if (pre_g && ((st = check_rows("pre_g", pre_g, ldp, N, 4, &p_vec)) || (st = check_rows("pre_u", pre_u, ldp, N, 4, &p_vec2))))
        return st;
    if ((st = check_apart({area("pre_g", pre_g, ldp, M, N, 4), area("pre_u", pre_u, ldp, M, N, 4), area("D", D, ldd, M, N, 2)},
                          {area("A", A, lda, M, K, 2), area("Wg", Wg, ldg, N, K, 2), area("Wu", Wu, ldu, N, K, 2)})) ||
        (st = check_device()))
        return st;
    FusedArgs p = base_args(A, lda, Wg, ldg, D, ldd, M, N, K);
    p.B2 = static_cast<const uint8_t *>(Wu);
    p.ldb2 = 2 * ldu;
    p.act = activation;
    p.pre = pre_g; p.pre2 = pre_u; p.ldp = ldp; p.p_vec = p_vec && p_vec2;
    return launch_forward<EPI_GATED>(p, static_cast<hipStream_t>(stream));
}

int64_t bf16_gated_nt_backward_workspace(int M, int N, int K) {
    int st;
    if ((st = check_sizes(M, N, K, 2)) || (st = check_grad_sizes(M, N))) return st;
    return grad_bytes(M, 2 * pad64(N)) + join_bytes(M, N, K, 2 * pad64(N), 2);
}

int bf16_gated_nt_backward(const void *G, int64_t ldgrad, const void *A, int64_t lda, const void *Wg, int64_t ldg,
                           const void *Wu, int64_t ldu, const float *pre_g, const float *pre_u, int64_t ldp,
                           int activation, void *dA, int64_t ldda, void *dWg, void *dWu, int64_t lddw, void *workspace,
                           int64_t workspace_bytes, int M, int N, int K, void *stream) {
    int st, g_vec = 0, p_vec = 0, p_vec2 = 0;
    if ((st = check_sizes(M, N, K, 2)) || (st = check_grad_sizes(M, N)) || (st = check_activation(activation))) return st;
    if (!dWg != !dWu) return fail(FP8G_ERR_NULL, "dWg and dWu are given together or not at all");
    const bool want_a = dA && M > 0 && K > 0, want_w = dWg && N > 0 && K > 0;
    if (!want_a && !want_w) return ok();
    if (N > 0 && M > 0) {
        if (!G || !pre_g || !pre_u) return fail(FP8G_ERR_NULL, "G, pre_g and pre_u are required");
        if ((st = check_rows("G", G, ldgrad, N, 2, &g_vec)) || (st = check_rows("pre_g", pre_g, ldp, N, 4, &p_vec)) ||
            (st = check_rows("pre_u", pre_u, ldp, N, 4, &p_vec2)) ||
            (st = check_workspace(workspace, workspace_bytes, bf16_gated_nt_backward_workspace(M, N, K))))
            return st;
    }
    if (want_a) {
        if (N > 0 && ((st = check_operand("Wg", Wg, ldg, K, 2)) || (st = check_operand("Wu", Wu, ldu, K, 2)))) return st;
        if (N > 0 && ldg != ldu) return fail(FP8G_ERR_STRIDE, "dA needs Wg and Wu with one row stride (%lld, %lld)", (long long)ldg, (long long)ldu);
        if ((st = check_output("dA", dA, ldda, K))) return st;
    }
    if (want_w && ((M > 0 && (st = check_operand("A", A, lda, K, 2))) || (st = check_output("dWg", dWg, lddw, K)) ||
                   (st = check_output("dWu", dWu, lddw, K))))
        return st;
    if ((st = check_apart({area("dWg", want_w ? dWg : nullptr, lddw, N, K, 2), area("dWu", want_w ? dWu : nullptr, lddw, N, K, 2),
                           area("dA", want_a ? dA : nullptr, ldda, M, K, 2),
                           area("workspace", workspace, M > 0 && N > 0 ? bf16_gated_nt_backward_workspace(M, N, K) : 0, 1)},
                          {area("G", G, ldgrad, M, N, 2), area("A", A, lda, want_w ? M : 0, K, 2),
                           area("Wg", Wg, ldg, want_a ? N : 0, K, 2), area("Wu", Wu, ldu, want_a ? N : 0, K, 2),
                           area("pre_g", pre_g, ldp, M, N, 4), area("pre_u", pre_u, ldp, M, N, 4)})) ||
        (st = check_device()))
        return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t cols = pad64(N);
    uint16_t *const w = static_cast<uint16_t *>(workspace);
    float *const sums = reinterpret_cast<float *>(static_cast<char *>(workspace) + grad_bytes(M, 2 * cols));
    if (M > 0 && N > 0) {
        GradParams g = {};
        g.G = static_cast<const uint16_t *>(G); g.ldg = ldgrad; g.g_vec = g_vec;
        g.pre = pre_g; g.pre2 = pre_u; g.ldp = ldp; g.p_vec = p_vec && p_vec2;
        g.W = w; g.ldw = 2 * cols;
        g.M = M; g.N = N; g.act = activation;
        if ((st = launch_grad<true, false>(g, (int)cols, s))) return st;
    }
    if (want_a) {
        // one product over both halves: [dP | dU] (M x 2 cols) . [Wg; Wu],
        // whose rows past N of each half read as zeros
        FusedArgs p = base_args(w, 2 * cols, Wg, ldg, dA, ldda, M, K, (int)(2 * cols));
        p.B2 = static_cast<const uint8_t *>(Wu);
        p.ksplit = (int)(cols / 64);
        p.krows = N;
        if ((st = launch_backward<false, true>(p, 1, sums, s))) return st;
    }
    if (want_w) {
        FusedArgs p = base_args(w, 2 * cols, A, lda, dWg, lddw, N, K, M);
        p.D2 = static_cast<uint16_t *>(dWu);
        p.a_gstride = 2 * cols;
        if ((st = launch_backward<true, true>(p, 2, sums, s))) return st;
    }
    return ok();
}

}  // extern "C"
