// Products with fused epilogues: bias, activation and residual, and the gated
// product of two weight matrices, in FP8 and BF16, with the BF16 backward
// products.
//
//   fused   Z = sa[m] sb[n] (A . B^T) + bias[n],  D = act(Z) + R
//   gated   G = sa[m] sg[n] (A . Wg^T),  U = sa[m] su[n] (A . Wu^T),  H = act(G) U
//
// FP8 runs on the dense forms' loops (tile16_body, decode_body of kernels.hpp)
// with the epilogue below; BF16 with few tokens on decode_body, otherwise on
// bf16_tile_kernel, whose operands may each be K-contiguous or K-strided, so
// that it also computes the backward products
//   dA = dZ . B        (A operand K-contiguous, B operand K-strided)
//   dB = dZ^T . A      (both K-strided)
// with dZ = dD act'(Z) (gated: dG = dH U act'(G), dU = dH act(G)) formed once
// by grad_kernel from the FP32 pre-activations that the forward pass kept.
#pragma once

#include "kernels.hpp"

namespace fp8g {

enum { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3, ACT_GELU_TANH = 4 };

struct FusedArgs : GemmParams {
    // Gated: the second weight matrix and its channel scales (p.B / ch_sb: the
    // first).  K-strided B of the backward pass: the rows of K steps from
    // ksplit on.
    const uint8_t *B2;
    int64_t ldb2;
    const float *ch_sb2;
    int sa_step, sb_step;      // 1: one scale per row of A / channel, 0: one for all of them
    int act;
    const uint16_t *R;         // residual [M][ldr] BF16 or NULL
    int64_t ldr;
    float *pre;                // pre-activations out [M][ldp] or NULL
    float *pre2;               // gated: those of the second matrix
    int64_t ldp;
    int r_vec, p_vec;          // rows of R / pre start 16-byte aligned
    // Backward products: the second output (grid y = 1, whose A operand starts
    // a_gstride bytes later), the K step where B2's rows begin and the rows of
    // each of B and B2.
    uint16_t *D2;
    int ksplit, krows;
};

template <int E>
struct FusedParams : FusedArgs {
    static constexpr int kEpilogue = E;
};

// ---------------------------------------------------------------------------
// Activations, in FP32.  x sigmoid(v) is x / (1 + exp(-v)): no cancellation at
// either end (exp overflows to infinity for v < -88, and the quotient is then
// -0).  The tanh form of GELU is x sigmoid(2 u), since (1 + tanh u) / 2 =
// sigmoid(2 u); the exact form is x erfc(-x / sqrt 2) / 2, which keeps its
// relative precision where 1 + erf would cancel.
// ---------------------------------------------------------------------------
constexpr float kGeluC = 1.5957691216057308f;      // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

__device__ __forceinline__ float sigmoid_times(float x, float v) {
    return x * __builtin_amdgcn_rcpf(1.0f + __expf(-v));
}

__device__ __forceinline__ float act_value(int act, float z) {
    switch (act) {
    case ACT_NONE: return z;
    case ACT_RELU: return z < 0.0f ? 0.0f : z;     // (NaN stays NaN)
    case ACT_SILU: return sigmoid_times(z, z);
    case ACT_GELU: return 0.5f * z * erfcf(-kSqrtHalf * z);
    default: return sigmoid_times(z, kGeluC * (z + kGeluA * z * z * z));
    }
}

// act'(z).  Beyond |z| = 30 every activation here has its limit slope to FP32
// precision; the clamp keeps z^2 and z^3 finite (0 times infinity).
__device__ __forceinline__ float act_slope(int act, float z0) {
    const float z = z0 > 30.0f ? 30.0f : (z0 < -30.0f ? -30.0f : z0);
    switch (act) {
    case ACT_NONE: return 1.0f;
    case ACT_RELU: return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
    case ACT_SILU: {
        const float s = 1.0f / (1.0f + expf(-z));
        return s * (1.0f + z * (1.0f - s));
    }
    case ACT_GELU: return 0.5f * erfcf(-kSqrtHalf * z) + kInvSqrt2Pi * z * expf(-0.5f * z * z);
    default: {
        const float s = 1.0f / (1.0f + expf(-kGeluC * (z + kGeluA * z * z * z)));
        return s + z * s * (1.0f - s) * kGeluC * (1.0f + 3.0f * kGeluA * z * z);
    }
    }
}

// act(z) of the backward pass, with the full-precision exponential.
__device__ __forceinline__ float act_value_exact(int act, float z) {
    switch (act) {
    case ACT_SILU: return z / (1.0f + expf(-z));
    case ACT_GELU_TANH: return z / (1.0f + expf(-kGeluC * (z + kGeluA * z * z * z)));
    default: return act_value(act, z);
    }
}

__device__ __forceinline__ float bf16_float(uint16_t b) { return __builtin_bit_cast(float, (uint32_t)b << 16); }

// NV (4 or 8) consecutive values of a BF16 / FP32 row, `nv` of which exist;
// `vec`: the address is aligned for whole-vector access where all exist.
template <int NV>
__device__ __forceinline__ void load_bf16_row(const uint16_t *src, int nv, bool vec, float (&out)[NV]) {
    if (vec && nv >= NV) {
        uint32_t w[NV / 2];
        if constexpr (NV == 8) {
            const v4u v = *reinterpret_cast<const v4u *>(src);
            w[0] = v[0]; w[1] = v[1]; w[2] = v[2]; w[3] = v[3];
        } else {
            const v2u v = *reinterpret_cast<const v2u *>(src);
            w[0] = v[0]; w[1] = v[1];
        }
#pragma unroll
        for (int e = 0; e < NV; ++e) out[e] = bf16_float((uint16_t)(w[e / 2] >> (16 * (e & 1))));
    } else {
#pragma unroll
        for (int e = 0; e < NV; ++e) out[e] = e < nv ? bf16_float(src[e]) : 0.0f;
    }
}

template <int NV>
__device__ __forceinline__ void store_f32_row(float *dst, int nv, bool vec, const float (&v)[NV]) {
    if (vec && nv >= NV) {
#pragma unroll
        for (int e = 0; e < NV; e += 4) *reinterpret_cast<v4f *>(dst + e) = (v4f){v[e], v[e + 1], v[e + 2], v[e + 3]};
    } else {
#pragma unroll
        for (int e = 0; e < NV; ++e)
            if (e < nv) dst[e] = v[e];
    }
}

// Column terms of NV consecutive output columns (absent arrays: 1, 0).
template <int NV>
struct ColumnTerms {
    float s[NV], s2[NV], b[NV];
};

template <int NV, class P>
__device__ __forceinline__ ColumnTerms<NV> column_terms(const P &p, int n, int nv) {
    ColumnTerms<NV> t;
#pragma unroll
    for (int e = 0; e < NV; ++e) {
        const bool in = e < nv;
        t.s[e] = in && p.ch_sb ? p.ch_sb[(n + e) * p.sb_step] : 1.0f;
        t.s2[e] = P::kEpilogue == EPI_GATED && in && p.ch_sb2 ? p.ch_sb2[(n + e) * p.sb_step] : 1.0f;
        t.b[e] = P::kEpilogue == EPI_ACT && in && p.bias ? p.bias[n + e] : 0.0f;
    }
    return t;
}

// The epilogue of NV consecutive outputs of row m from column n on (z: the
// sums; gated: z of the first matrix, z2 of the second): scales and bias, the
// pre-activations kept for the backward pass, activation, residual or product,
// all in FP32; `out` is rounded once by the caller.
template <int NV, class P>
__device__ __forceinline__ void fused_outputs(const P &p, int m, int n, int nv, const ColumnTerms<NV> &t,
                                              float (&z)[NV], float (&z2)[NV], float (&out)[NV]) {
    constexpr int EPI = P::kEpilogue;
    if constexpr (EPI == EPI_STORE) {
#pragma unroll
        for (int e = 0; e < NV; ++e) out[e] = z[e];
    } else {
        const float sa = p.ch_sa ? p.ch_sa[(int64_t)m * p.sa_step] : 1.0f;
#pragma unroll
        for (int e = 0; e < NV; ++e) {
            z[e] = z[e] * sa * t.s[e] + t.b[e];
            if (EPI == EPI_GATED) z2[e] = z2[e] * sa * t.s2[e];
        }
        if (p.pre) {
            store_f32_row<NV>(p.pre + (int64_t)m * p.ldp + n, nv, p.p_vec, z);
            if (EPI == EPI_GATED) store_f32_row<NV>(p.pre2 + (int64_t)m * p.ldp + n, nv, p.p_vec, z2);
        }
#pragma unroll
        for (int e = 0; e < NV; ++e) out[e] = act_value(p.act, z[e]);
        if constexpr (EPI == EPI_GATED) {
#pragma unroll
            for (int e = 0; e < NV; ++e) out[e] *= z2[e];
        } else if (p.R) {
            float r[NV];
            load_bf16_row<NV>(p.R + (int64_t)m * p.ldr + n, nv, p.r_vec, r);
#pragma unroll
            for (int e = 0; e < NV; ++e) out[e] += r[e];
        }
    }
}

// Four outputs of a few-token lane: row m, columns n .. n + 3.
template <class P>
__device__ __forceinline__ void fused_store4(const P &p, int m, int n, v4f a, v4f b) {
    const int nv = p.N - n;
    if (nv <= 0) return;
    const ColumnTerms<4> t = column_terms<4>(p, n, nv);
    float z[4] = {a[0], a[1], a[2], a[3]}, z2[4] = {b[0], b[1], b[2], b[3]}, o[4];
    fused_outputs<4>(p, m, n, nv, t, z, z2, o);
    store_bf16x4(p.D + (int64_t)m * p.ldd + n, 0, nv, pack_bf16x4(o[0], o[1], o[2], o[3]));
}

// ---------------------------------------------------------------------------
// Epilogue of the tiled kernels.  The tile's FP32 sums are staged in the freed
// LDS ring (row s at s * BN * 4 bytes, its 16-byte chunk c at c ^ (s % 16), so
// that the 16 or 32 rows that one write instruction touches, and the chunks of
// one row that a read touches, lie in different banks), as many rows as fit at
// a time; then each thread takes 8 consecutive output columns, always the same
// ones, of every RPI-th row.  Against an epilogue in the accumulator layout:
// one copy of the activations' code instead of one per accumulator, column
// terms loaded once per thread, and 16-byte accesses of whole row segments for
// the residual, the pre-activations and the output.
// ---------------------------------------------------------------------------
template <int BN>
__device__ __forceinline__ void stage_f32(uint8_t *smem, int s, int col, v4f v) {
    *reinterpret_cast<v4f *>(smem + s * (BN * 4) + (((uint32_t)col >> 2) ^ ((uint32_t)s & 15u)) * 16) = v;
}

template <int BN, int ROWS, int THREADS, int IB, class P, class RowOf>
__device__ __forceinline__ void fused_store_rows(const P &p, const uint8_t *smem, int tid, int m0, int rows_m, int n0,
                                                 uint16_t *d, RowOf row_of) {
    constexpr bool GATED = P::kEpilogue == EPI_GATED;
    constexpr int GROUPS = (GATED ? BN / 2 : BN) / 8, RPI = THREADS / GROUPS;
    static_assert(THREADS % GROUPS == 0 && ROWS % RPI == 0, "rows split evenly over the threads");
    const int g = tid % GROUPS;
    const int n = n0 + 8 * g;
    const int nv = p.N - n;
    if (nv <= 0) return;
    const ColumnTerms<8> t = column_terms<8>(p, n, nv);
    // first 16-byte chunk of the group's sums (gated: blocks of IB columns of
    // the two matrices alternate)
    const uint32_t c0 = GATED ? (uint32_t)((g / (IB / 8)) * (IB / 2) + (g % (IB / 8)) * 2) : (uint32_t)(2 * g);
#pragma unroll 2
    for (int s = tid / GROUPS; s < ROWS; s += RPI) {
        const int r = row_of(s);
        if (r >= rows_m) continue;
        const uint8_t *row = smem + s * (BN * 4);
        auto read8 = [&](uint32_t c, float (&z)[8]) {
            const v4f lo = *reinterpret_cast<const v4f *>(row + (c ^ ((uint32_t)s & 15u)) * 16);
            const v4f hi = *reinterpret_cast<const v4f *>(row + ((c + 1) ^ ((uint32_t)s & 15u)) * 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) { z[e] = lo[e]; z[4 + e] = hi[e]; }
        };
        float z[8], z2[8], o[8];
        read8(c0, z);
        if (GATED) read8(c0 + IB / 4, z2);
        const int m = m0 + r;
        fused_outputs<8>(p, m, n, nv, t, z, z2, o);
        const v2u lo = pack_bf16x4(o[0], o[1], o[2], o[3]), hi = pack_bf16x4(o[4], o[5], o[6], o[7]);
        store_chunk<MODE_DENSE>(d + (int64_t)m * p.ldd + n, (v4u){lo[0], lo[1], hi[0], hi[1]}, nv);
    }
}

// ---------------------------------------------------------------------------
// FP8: the dense loops of kernels.hpp with a fused epilogue.
// ---------------------------------------------------------------------------
template <int BM, int STAGES, int FA, int FB, bool KTAIL, int EPI>
__global__ __launch_bounds__(256, 1) void fused_tile16_kernel(FusedParams<EPI> p) {
    tile16_body<BM, 256, STAGES, FA, FB, MODE_DENSE, SCALE_CHANNEL, KTAIL>(p);
}

// Few tokens, FP8 and BF16.
template <int WAVES, int RB, int CB, int FA, int FB, int D, int EPI, int OCC>
__global__ __launch_bounds__(64 * WAVES, OCC) void fused_decode_kernel(FusedParams<EPI> p) {
    decode_body<WAVES, RB, CB, FA, FB, D, SCALE_CHANNEL>(p);
}

}  // namespace fp8g
