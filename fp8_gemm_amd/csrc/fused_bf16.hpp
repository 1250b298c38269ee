// BF16 tiled kernel with fused epilogues, for the forward product and both
// backward products, and the kernels that form the gradients of the
// pre-activations and of the bias.
#pragma once

#include "tile_halves.hpp"

namespace fp8g {

// The BF16 products (tile_halves_body).
template <int BM, int BN, int STAGES, bool TA, bool TB, bool TAIL, int EPI>
__global__ __launch_bounds__(256, 1) void bf16_tile_kernel(FusedParams<EPI, false> p) {
    tile_halves_body<BM, BN, STAGES, FMT_BF16, TA, TB, TAIL, PLACE_DENSE>(p);
}

// act'(z), for z within a range outside of which act' has its limit value in
// FP32; the clamp keeps z, z^2 and z^3 finite (0 times infinity).  Above 30
// that holds for every activation here, below -30 for both forms of GELU
// (their slopes fall faster than exp(-z^2 / 2 + log |z|)); the slope of SiLU
// falls like |z| exp(z) only, down to the FP32 exponential's overflow at z =
// -88.7, past which the sigmoid, and with it the slope, is 0.
template <int ACT>
__device__ __forceinline__ float act_slope(float z0) {
    constexpr float lo = ACT == ACT_SILU ? -100.0f : -30.0f;
    const float z = z0 > 30.0f ? 30.0f : (z0 < lo ? lo : z0);
    if constexpr (ACT == ACT_RELU) {
        return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
    } else if constexpr (ACT == ACT_SILU) {
        const float s = 1.0f / (1.0f + expf(-z));
        return s * (1.0f + z * (1.0f - s));
    } else if constexpr (ACT == ACT_GELU) {
        return 0.5f * erfcf(-kSqrtHalf * z) + kInvSqrt2Pi * z * expf(-0.5f * z * z);
    } else if constexpr (ACT == ACT_GELU_TANH) {
        const float s = 1.0f / (1.0f + expf(-kGeluC * (z + kGeluA * z * z * z)));
        return s + z * s * (1.0f - s) * kGeluC * (1.0f + 3.0f * kGeluA * z * z);
    } else {
        return 1.0f;
    }
}

// act(z) of the backward pass, with the full-precision exponential and erfc
// (that kernel waits on memory).
template <int ACT>
__device__ __forceinline__ float act_value_exact(float z) {
    if constexpr (ACT == ACT_SILU) return z / (1.0f + expf(-z));
    else if constexpr (ACT == ACT_GELU_TANH) return z / (1.0f + expf(-kGeluC * (z + kGeluA * z * z * z)));
    else if constexpr (ACT == ACT_GELU) return 0.5f * z * erfcf(-kSqrtHalf * z);
    else return act_value<ACT>(z);
}

// ---------------------------------------------------------------------------
// Gradients of the pre-activations: fused dZ = dD act'(Z), gated dG = dH U
// act'(G) and dU = dH act(G), rounded to BF16 once, the operands of the
// backward products, into W [M][ldw] (gated: dU from column ldw / 2 on), whose
// columns past N hold zeros.  Bound by memory: 6 bytes read and 2 written per
// element (fused), 10 and 4 (gated); gated 4096 x 14336 188 us, 4.4 TB/s.
// The rounding: the products' matrix instructions take 16-bit operands, and dZ
// held to 16 bits as two BF16 terms would double both products' work.  Each
// term of a gradient's sum is off by at most 2^-8 of it, independently of the
// others, which moves the gradient about as much as its own rounding to BF16
// does: relative errors of 0.0023 where unrounded dZ give 0.0017.
// BIAS: also the column sums of the FP32 dZ over the block's rows into
// part[block row][N], added over the rows in a fixed order.
// A block is 32 groups of 8 columns x 8 rows of threads over `rows` rows: as
// few as 8 where M x N is small, so that every row's loads are in flight at
// once (301 x 1111, unaligned rows: 25.7 us with 64 rows per block, which 25
// blocks ran through 8 at a time).
// ---------------------------------------------------------------------------
constexpr int kGradMaxRows = 64;

struct GradParams {
    const uint16_t *G;         // output gradient [M][ldg] BF16
    const float *pre, *pre2;   // pre-activations [M][ldp] (not read with act none, ungated)
    uint16_t *W;               // NULL: column sums only
    float *part;
    int64_t ldg, ldp, ldw;
    int M, N, act, g_vec, p_vec, rows;
};

__device__ __forceinline__ void load_f32_row8(const float *src, int nv, bool vec, float (&out)[8]) {
    if (vec && nv >= 8) {
        const v4f a = *reinterpret_cast<const v4f *>(src), b = *reinterpret_cast<const v4f *>(src + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) { out[e] = a[e]; out[4 + e] = b[e]; }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) out[e] = e < nv ? src[e] : 0.0f;
    }
}

template <bool GATED, bool BIAS>
__global__ __launch_bounds__(256) void grad_kernel(GradParams p) {
    __shared__ float sums[BIAS ? 8 * 256 : 1];
    const int tid = threadIdx.x;
    const int n = blockIdx.y * 256 + (tid & 31) * 8;
    const int nv = p.N - n;                        // <= 0: padding columns
    const int half = GATED ? (int)(p.ldw / 2) : (int)p.ldw;   // columns of W per matrix
    float bsum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const int r0 = blockIdx.x * p.rows, r1 = min(p.M, r0 + p.rows);
    with_activation(p.act, [&](auto act) {
        for (int r = r0 + (tid >> 5); r < r1; r += 8) {
            float g[8], z[8], z2[8], dz[8], du[8];
            load_bf16_row<8>(p.G + (int64_t)r * p.ldg + n, nv, p.g_vec, g);
            if (GATED || act.value != ACT_NONE) load_f32_row8(p.pre + (int64_t)r * p.ldp + n, nv, p.p_vec, z);
            if (GATED) load_f32_row8(p.pre2 + (int64_t)r * p.ldp + n, nv, p.p_vec, z2);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (e >= nv) {                         // (a padding column is zero whatever its gradient)
                    dz[e] = du[e] = 0.0f;
                } else if (GATED) {
                    dz[e] = g[e] * z2[e] * act_slope<act.value>(z[e]);
                    du[e] = g[e] * act_value_exact<act.value>(z[e]);
                } else {
                    dz[e] = act.value != ACT_NONE ? g[e] * act_slope<act.value>(z[e]) : g[e];
                }
                if (BIAS) bsum[e] += dz[e];
            }
            if (p.W && n < half) {                     // (half is a multiple of 64: whole groups)
                const v2u lo = pack_bf16x4(dz[0], dz[1], dz[2], dz[3]), hi = pack_bf16x4(dz[4], dz[5], dz[6], dz[7]);
                *reinterpret_cast<v4u *>(p.W + (int64_t)r * p.ldw + n) = (v4u){lo[0], lo[1], hi[0], hi[1]};
                if (GATED) {
                    const v2u l2 = pack_bf16x4(du[0], du[1], du[2], du[3]), h2 = pack_bf16x4(du[4], du[5], du[6], du[7]);
                    *reinterpret_cast<v4u *>(p.W + (int64_t)r * p.ldw + half + n) = (v4u){l2[0], l2[1], h2[0], h2[1]};
                }
            }
        }
    });
    if constexpr (BIAS) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[(tid >> 5) * 256 + (tid & 31) * 8 + e] = bsum[e];
        __syncthreads();
        float total = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) total += sums[k * 256 + tid];
        const int c = blockIdx.y * 256 + tid;
        if (c < p.N) p.part[(int64_t)blockIdx.x * p.N + c] = total;
    }
}

// Outputs of a product split over K: the splits' sums added in split order,
// rounded to BF16.  ws [splits][ny][M][N], N a multiple of 8; 8 columns per
// thread, product y = blockIdx.y.
__global__ __launch_bounds__(256) void join_kernel(const float *ws, int splits, int M, int N, uint16_t *d0, uint16_t *d1,
                                                   int64_t ldd) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8, out = (int64_t)M * N;
    if (i >= out) return;
    const float *src = ws + blockIdx.y * out + i;
    const int64_t step = (int64_t)gridDim.y * out;
    v4f lo = *reinterpret_cast<const v4f *>(src), hi = *reinterpret_cast<const v4f *>(src + 4);
    for (int s = 1; s < splits; ++s) {
        lo += *reinterpret_cast<const v4f *>(src + s * step);
        hi += *reinterpret_cast<const v4f *>(src + s * step + 4);
    }
    uint16_t *const d = (blockIdx.y ? d1 : d0) + (i / N) * ldd + i % N;
    const v2u a = pack_bf16x4(lo[0], lo[1], lo[2], lo[3]), b = pack_bf16x4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<v4u *>(d) = (v4u){a[0], a[1], b[0], b[1]};
}

// Column sums of part [rows][N]: 32 columns per block, 8 threads per column
// over every 8th row, their sums added in order.
__global__ __launch_bounds__(256) void bias_grad_kernel(const float *part, int rows, int n, float *out) {
    __shared__ float sums[8][32];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), lane = threadIdx.x >> 5;
    float total = 0.0f;
    if (c < n) {
        int r = lane;
        for (; r + 24 < rows; r += 32) {           // four rows' loads at a time
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = part[(int64_t)(r + 8 * k) * n + c];
#pragma unroll
            for (int k = 0; k < 4; ++k) total += v[k];
        }
        for (; r < rows; r += 8) total += part[(int64_t)r * n + c];
    }
    sums[lane][threadIdx.x & 31] = total;
    __syncthreads();
    if (lane || c >= n) return;
#pragma unroll
    for (int k = 1; k < 8; ++k) total += sums[k][threadIdx.x];
    out[c] = total;
}

}  // namespace fp8g
