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

// One split of a backward product: FP32 sums into the workspace.
constexpr int EPI_PARTIAL = 3;
// Scales and bias alone, applied in the accumulators' layout (tile_halves.hpp).
constexpr int EPI_SCALED = 4;

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
    // each of B and B2.  Split over K (grid z, ksteps steps each): the sums of
    // split z of product y go to ws [z][y][M][N].
    uint16_t *D2;
    int ksplit, krows;
};

// SCALED: the sums take scales (FP8, 8-bit integers); BF16 sums do not.  INT:
// they are 32-bit integers.
template <int E, bool SCALED, bool INT = false>
struct FusedParams : FusedArgs {
    static constexpr int kEpilogue = E;
    static constexpr bool kScaled = SCALED;
    static constexpr bool kIntSums = INT;
};

// 8-bit integers (experts.hpp): the sums are staged as they are and become FP32
// (rounded to nearest even) where the epilogue reads them.  Converted before,
// they took registers that the 256 x 256 tile does not have (5 spilled).
template <int E>
struct Int8Params : FusedParams<E, true, true> {};

// Over ragged groups of rows (ragged.hpp): expert g's weights begin b_gstride
// bytes after those of expert g - 1, its channel scales N floats, its weight
// gradient d_gstride elements.  rows: PLACE_SUMS, the number of token rows (M
// and N are the gradient's); stream: its stores bypass the caches.  Scales
// come with 8-bit integers only.
template <int E, bool SCALED, int PLACE>
struct RaggedParams : FusedParams<E, SCALED, SCALED> {
    static constexpr int kPlace = PLACE;
    const int32_t *offsets;
    int rows, stream;
};

// ---------------------------------------------------------------------------
// Activations, in FP32.  x sigmoid(v) is x / (1 + exp(-v)): no cancellation at
// either end.  The reciprocal instruction returns 0 for results below 2^-126,
// so it is taken of (1 + exp(-v)) / 4, which stays in its range up to the
// exponential's overflow at -v = 88.7 (silu(-88) = -5.3e-37 is a normal BF16
// number); past that the quotient is -0.  The tanh form of GELU is
// x sigmoid(2 u), since (1 + tanh u) / 2 = sigmoid(2 u).
// The exact form is x Phi(x), Phi the normal distribution: x Q for x < 0 and
// x (1 - Q) otherwise, with Q = Phi(-|x|) = exp(-x^2 / 2) h(|x|), which keeps
// its relative precision where 1 + erf would cancel.  h(x) = erfcx(x / sqrt 2)
// / 2 is smooth and falls like 1 / x: a polynomial of degree 7 in t = 1 / (1 +
// 0.36 x) without constant term, fitted by least squares reweighted towards
// the largest relative error, is within 8.1e-7 of it in FP32 up to x = 13.5
// (past which Q underflows).  erfcf, with its two branches, made the epilogue of a
// 2048 x 4096 x 14336 product 10 us longer.
// ---------------------------------------------------------------------------
constexpr float kGeluC = 1.5957691216057308f;      // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

__device__ __forceinline__ float sigmoid_times(float x, float v) {
    return (0.25f * x) * __builtin_amdgcn_rcpf(0.25f + 0.25f * __expf(-v));
}

__device__ __forceinline__ float normal_cdf(float z) {
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.36f * __builtin_fabsf(z));
    float h = 0.04734533f;
    h = h * t - 0.18075425f;
    h = h * t + 0.18230114f;
    h = h * t + 0.02562137f;
    h = h * t + 0.14005832f;
    h = h * t + 0.14171051f;
    h = h * t + 0.14371745f;
    const float q = h * t * __expf(-0.5f * z * z);
    return z < 0.0f ? q : 1.0f - q;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == ACT_RELU) return z < 0.0f ? 0.0f : z;     // (NaN stays NaN)
    else if constexpr (ACT == ACT_SILU) return sigmoid_times(z, z);
    else if constexpr (ACT == ACT_GELU) return z * normal_cdf(z);
    else if constexpr (ACT == ACT_GELU_TANH) return sigmoid_times(z, kGeluC * (z + kGeluA * z * z * z));
    else return z;
}

// Calls f with the activation as a compile-time value (f(int_c<ACT>{})): the
// choice is made once per workgroup, around whole loops.  Made per value it
// put five activations' code into the innermost loop, and the epilogue of one
// 256 x 256 tile took 23 us.
template <class F>
__device__ __forceinline__ void with_activation(int act, F f) {
    switch (act) {
    case ACT_NONE: f(int_c<ACT_NONE>{}); break;
    case ACT_RELU: f(int_c<ACT_RELU>{}); break;
    case ACT_SILU: f(int_c<ACT_SILU>{}); break;
    case ACT_GELU: f(int_c<ACT_GELU>{}); break;
    default: f(int_c<ACT_GELU_TANH>{}); break;
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
        t.s[e] = P::kScaled && in && p.ch_sb ? p.ch_sb[(n + e) * p.sb_step] : 1.0f;
        t.s2[e] = P::kScaled && P::kEpilogue == EPI_GATED && in && p.ch_sb2 ? p.ch_sb2[(n + e) * p.sb_step] : 1.0f;
        t.b[e] = P::kEpilogue == EPI_ACT && in && p.bias ? p.bias[n + e] : 0.0f;
    }
    return t;
}

// The scale of a row of integer sums in two factors, for z first (sb rest).  A
// sum of up to 2^31 times a scale above 2^96 could leave FP32 although the
// output, with a small channel scale, does not (rows quantised from values above
// 2^103): such a row leaves 2^32 of its scale to the channel's.  At the other end
// nothing is lost: whole multiples of a scale below the normal numbers are exact
// there.  Both factors are powers of two away from the scale, so that no output
// within FP32 depends on the split.  (Where both scales are above 2^96, every sum
// but 0 leaves FP32, and 0 becomes NaN.)  It costs one product per output: 0.4 to
// 0.8% of prompts (4096 x 14336 x 4096 191.6 against 190.5 us), 1.6% where K is
// short (8192 x 8192 x 512 57.9 against 56.9), 0.16 us of few tokens.  A branch
// around it, per 4 outputs or with the whole epilogue twice, took more: scalar
// instructions in every pass, or 8 to 41 spilled registers.
struct RowFactors {
    float first, rest;
};
__device__ __forceinline__ RowFactors row_factors(float sa) {
    const bool large = __builtin_fabsf(sa) > 0x1p+96f;
    return {large ? sa * 0x1p-32f : sa, large ? 0x1p+32f : 1.0f};
}

// The epilogue of NV consecutive outputs of row m from column n on (z: the
// sums; gated: z of the first matrix, z2 of the second; sa: the row's scale;
// r: the residual): scales and bias, the pre-activations kept for the backward
// pass, activation, residual or product, all in FP32; `out` is rounded once by
// the caller.
template <int ACT, int NV, class P>
__device__ __forceinline__ void fused_outputs(const P &p, int m, int n, int nv, const ColumnTerms<NV> &t, float sa,
                                              const float (&r)[NV], float (&z)[NV], float (&z2)[NV], float (&out)[NV]) {
    constexpr bool GATED = P::kEpilogue == EPI_GATED;
    const RowFactors f = P::kIntSums ? row_factors(sa) : RowFactors{sa, 1.0f};
#pragma unroll
    for (int e = 0; e < NV; ++e) {
        if (P::kScaled) z[e] = z[e] * f.first * (P::kIntSums ? t.s[e] * f.rest : t.s[e]);
        if (P::kScaled && GATED) z2[e] = z2[e] * sa * t.s2[e];
        if (!GATED) z[e] += t.b[e];
    }
    if (!P::kScaled && p.pre) {                   // (kept by the BF16 forms only)
        store_f32_row<NV>(p.pre + (int64_t)m * p.ldp + n, nv, p.p_vec, z);
        if (GATED) store_f32_row<NV>(p.pre2 + (int64_t)m * p.ldp + n, nv, p.p_vec, z2);
    }
#pragma unroll
    for (int e = 0; e < NV; ++e) {
        out[e] = act_value<ACT>(z[e]);
        out[e] = GATED ? out[e] * z2[e] : out[e] + r[e];
    }
}

template <class P>
__device__ __forceinline__ float row_scale(const P &p, int m) {
    return P::kScaled && p.ch_sa ? p.ch_sa[(int64_t)m * p.sa_step] : 1.0f;
}

// Four outputs of a few-token lane: row m, columns n .. n + 3.
template <class P>
__device__ __forceinline__ void fused_store4(const P &p, int m, int n, v4f a, v4f b) {
    const int nv = p.N - n;
    if (nv <= 0) return;
    const ColumnTerms<4> t = column_terms<4>(p, n, nv);
    const float sa = row_scale(p, m);
    float z[4] = {a[0], a[1], a[2], a[3]}, z2[4] = {b[0], b[1], b[2], b[3]}, o[4], r[4] = {0, 0, 0, 0};
    if (P::kEpilogue == EPI_ACT && p.R) load_bf16_row<4>(p.R + (int64_t)m * p.ldr + n, nv, p.r_vec, r);
    with_activation(p.act, [&](auto act) { fused_outputs<act.value, 4>(p, m, n, nv, t, sa, r, z, z2, o); });
    store_bf16x4(p.D + (int64_t)m * p.ldd + n, 0, nv, pack_bf16x4(o[0], o[1], o[2], o[3]));
}

// ---------------------------------------------------------------------------
// Epilogue of the tiled kernels.  The tile's FP32 sums are staged in the freed
// LDS ring (row s at s * BN * 4 bytes, its 16-byte chunk c at c ^ (s % 16), so
// that the 16 or 32 rows that one write instruction touches, and the chunks of
// one row that a read touches, lie in different banks), as many rows as fit at
// a time; then each thread takes 8 consecutive output columns, always the same
// ones, of every RPI-th row.  Against an epilogue in the accumulator layout:
// one copy of the activations' code instead of one per accumulator, and
// 16-byte accesses of whole row segments for the residual, the pre-activations
// and the output (4 columns and 8 bytes per thread measured 17% slower on
// 8192 x 14336 x 4096).
//
// The row scales, column scales and biases wait in LDS (copy_tile_terms, before
// the main loop), and the residuals of the next batch of U rows are loaded
// before this batch is computed and stored: a load after a store is answered,
// in order, only once the write-through store has reached memory.  The first
// batch's go out before the sums are staged (`stage`, which ends in a barrier).
// ---------------------------------------------------------------------------
template <int BN>
__device__ __forceinline__ void stage_f32(uint8_t *smem, int s, int col, v4f v) {
    *reinterpret_cast<v4f *>(smem + s * (BN * 4) + (((uint32_t)col >> 2) ^ ((uint32_t)s & 15u)) * 16) = v;
}

// Copies the tile's terms into LDS: floats [0, 256) row scales, [256, 512)
// column scales (gated: [256, 384) the first matrix's, [384, 512) the
// second's), [512, 768) biases, 64 of each per wave, one dword per lane,
// asynchronously (the wait for the ring's step 0 covers them).  Entries past
// the tile's rows or columns read as zeros; absent scales are ones, absent
// biases zeros.
template <class P>
__device__ __forceinline__ void copy_tile_terms(const P &p, uint8_t *terms, uint32_t lds, int wave, int lane, int m0,
                                                int rows_m, int n0, int rows_n) {
    constexpr bool GATED = P::kEpilogue == EPI_GATED;
    float *const own = reinterpret_cast<float *>(terms) + wave * 64 + lane;
    auto copy = [&](const float *src, int step, int first, int count, int idx, int at, float absent) {
        // (the persistent kernels are short of scalar registers: the compiler
        // would keep the LDS address in a vector register, which M0 cannot take)
        auto address = [](uint32_t a) { return P::kEpilogue == EPI_SCALED ? (uint32_t)__builtin_amdgcn_readfirstlane((int)a) : a; };
        if (src)
            dma4(make_srd(src + (int64_t)first * step, step ? rows_bytes(count, 4) : 4u),
                 idx < count ? 4u * (uint32_t)(idx * step) : kOobOffset, address(lds + (uint32_t)(at + wave * 64) * 4u));
        else
            own[at] = absent;
    };
    const int idx = wave * 64 + lane;
    if (P::kScaled) {
        copy(p.ch_sa, p.sa_step, m0, rows_m, idx, 0, 1.0f);
        if (GATED && wave >= 2) copy(p.ch_sb2, p.sb_step, n0, rows_n, idx - 128, 256, 1.0f);
        else copy(p.ch_sb, p.sb_step, n0, rows_n, idx, 256, 1.0f);
    }
    if (P::kEpilogue == EPI_ACT || P::kEpilogue == EPI_SCALED) copy(p.bias, 1, n0, rows_n, idx, 512, 0.0f);
}

template <int BN, int ROWS, class P, class RowOf, class Stage>
__device__ __forceinline__ void fused_store_rows(const P &p, const uint8_t *smem, const uint8_t *terms, int tid, int m0,
                                                 int rows_m, int n0, uint16_t *d, RowOf row_of, Stage stage) {
    constexpr int EPI = P::kEpilogue;
    constexpr bool GATED = EPI == EPI_GATED;
    constexpr int THREADS = 256, GROUPS = (GATED ? BN / 2 : BN) / 8, RPI = THREADS / GROUPS, NIT = ROWS / RPI;
    constexpr int U = 4;                           // rows per batch
    constexpr int IB = 16;                         // gated: columns of a block of one matrix
    static_assert(THREADS % GROUPS == 0 && ROWS % RPI == 0 && NIT % U == 0, "rows split evenly over the threads");
    const int g = tid % GROUPS;
    const int n = n0 + 8 * g;
    const int nv = p.N - n;
    const int s0 = tid / GROUPS;
    // the residual of U rows as loaded (whole 16-byte chunks), or element by
    // element at the matrix' edge and for unaligned rows
    const bool res = EPI == EPI_ACT && p.R, whole = res && p.r_vec && nv >= 8;
    auto load_residuals = [&](v4u (&rb)[U], int i) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = row_of(s0 + (i + u) * RPI);
            if (whole && r < rows_m) rb[u] = *reinterpret_cast<const v4u *>(p.R + (int64_t)(m0 + r) * p.ldr + n);
        }
    };
    v4u rb[2][U];
    if constexpr (EPI == EPI_ACT) load_residuals(rb[0], 0);
    stage();
    if (nv <= 0) return;
    // first 16-byte chunk of the group's sums (gated: the two matrices' blocks
    // alternate)
    const uint32_t c0 = GATED ? (uint32_t)((g / (IB / 8)) * (IB / 2) + (g % (IB / 8)) * 2) : (uint32_t)(2 * g);
    auto read8 = [&](int s, uint32_t c, float (&z)[8]) {
        const uint8_t *row = smem + s * (BN * 4);
        const v4f lo = *reinterpret_cast<const v4f *>(row + (c ^ ((uint32_t)s & 15u)) * 16);
        const v4f hi = *reinterpret_cast<const v4f *>(row + ((c + 1) ^ ((uint32_t)s & 15u)) * 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (P::kIntSums) {           // (the vectors as wholes: a bit cast of one element takes the first)
                z[e] = (float)__builtin_bit_cast(v4i, lo)[e];
                z[4 + e] = (float)__builtin_bit_cast(v4i, hi)[e];
            } else {
                z[e] = lo[e];
                z[4 + e] = hi[e];
            }
        }
    };
    auto write8 = [&](int m, const float (&o)[8]) {
        const v2u lo = pack_bf16x4(o[0], o[1], o[2], o[3]), hi = pack_bf16x4(o[4], o[5], o[6], o[7]);
        store_chunk<MODE_DENSE>(d + (int64_t)m * p.ldd + n, (v4u){lo[0], lo[1], hi[0], hi[1]}, nv);
    };
    if constexpr (EPI == EPI_PARTIAL) {
        float *const sums = p.ws + ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * p.M * p.N;
#pragma unroll U
        for (int i = 0; i < NIT; ++i) {
            const int s = s0 + i * RPI, r = row_of(s);
            float z[8];
            read8(s, c0, z);
            if (r < rows_m) store_f32_row<8>(sums + (int64_t)(m0 + r) * p.N + n, nv, true, z);
        }
    } else if constexpr (EPI == EPI_STORE) {
#pragma unroll U
        for (int i = 0; i < NIT; ++i) {
            const int s = s0 + i * RPI, r = row_of(s);
            float z[8];
            read8(s, c0, z);
            if (r < rows_m) write8(m0 + r, z);
        }
    } else {
        const float *const tf = reinterpret_cast<const float *>(terms);
        ColumnTerms<8> t;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            t.s[e] = P::kScaled ? tf[256 + 8 * g + e] : 1.0f;
            t.s2[e] = P::kScaled && GATED ? tf[384 + 8 * g + e] : 1.0f;
            t.b[e] = GATED ? 0.0f : tf[512 + 8 * g + e];
        }
        with_activation(p.act, [&](auto act) {
            auto batch = [&](const v4u (&rb)[U], int i) {
                float o[U][8];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int s = s0 + (i + u) * RPI, r = row_of(s);
                    float z[8], z2[8], rv[8];
                    read8(s, c0, z);
                    if (GATED) read8(s, c0 + IB / 4, z2);
                    const float sa = P::kScaled ? tf[r] : 1.0f;
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) rv[e] = bf16_float((uint16_t)(rb[u][e / 2] >> (16 * (e & 1))));
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) rv[e] = 0.0f;
                        if (res && r < rows_m) load_bf16_row<8>(p.R + (int64_t)(m0 + r) * p.ldr + n, nv, false, rv);
                    }
                    fused_outputs<act.value, 8>(p, m0 + r, n, r < rows_m ? nv : 0, t, sa, rv, z, z2, o[u]);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int r = row_of(s0 + (i + u) * RPI);
                    if (r < rows_m) write8(m0 + r, o[u]);
                }
            };
            if constexpr (EPI == EPI_ACT) {
                static_assert(NIT % (2 * U) == 0, "pairs of batches");
#pragma unroll 1
                for (int i = 0; i < NIT; i += 2 * U) {
                    load_residuals(rb[1], i + U);
                    batch(rb[0], i);
                    if (i + 2 * U < NIT) load_residuals(rb[0], i + 2 * U);
                    batch(rb[1], i + U);
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < NIT; i += U) batch(rb[0], i);
            }
        });
    }
}

// ---------------------------------------------------------------------------
// FP8: the dense loops of kernels.hpp with a fused epilogue, which is all that
// they cost beyond the plain form: gated 8192 x 14336 x 4096 770 us back to back
// (2.5 PFLOP/s, the clock under load; the plain product of half the size takes
// 350), 2048 x 4096 x 14336 with residual 101 us (95).
// ---------------------------------------------------------------------------
template <int BM, int BN, int STAGES, int FA, int FB, bool KTAIL, int EPI>
__global__ __launch_bounds__(256, 1) void fused_tile16_kernel(FusedParams<EPI, true> p) {
    tile16_body<BM, BN, STAGES, FA, FB, MODE_DENSE, SCALE_CHANNEL, KTAIL>(p);
}

// Few tokens, FP8 and BF16.  Bound by the weights' way from memory for up to
// 16 tokens (gated FP8 1 x 14336 x 4096 24 us, 4.9 TB/s), by the copies of
// tokens and weights into each CU for more (64 tokens 28 us): every wave
// copies the tokens of its K steps beside 16 to 64 weight rows.  The plain
// form's decode_rows_kernel, whose waves share one copy of the tokens, needs
// fewer and has no fused epilogue (64 x 4096 x 14336: 22.8 us here, 18.5 the
// plain product there).  (Builds for one workgroup per CU, as the dense form
// has for grids of up to 256, measured within 1% of these for two.)
template <int WAVES, int RB, int CB, int FA, int FB, int D, int EPI>
__global__ __launch_bounds__(64 * WAVES, 2) void fused_decode_kernel(FusedParams<EPI, FA != FMT_BF16, FA == FMT_I8> p) {
    decode_body<WAVES, RB, CB, FA, FB, D, SCALE_CHANNEL>(p);
}

}  // namespace fp8g
