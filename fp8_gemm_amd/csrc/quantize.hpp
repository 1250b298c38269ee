// Rows of BF16 values in 8-bit integers with a scale each.
#pragma once

#include "fused.hpp"

namespace fp8g {

// ---------------------------------------------------------------------------
// Quantisation of rows.  T threads hold one row in registers, 8 values per
// thread and chunk, up to R chunks: one pass over memory (2 bytes read, 1
// written per value), which bounds it: 8192 x 14336 values 61.4 us, 5.7 TB/s; a
// few rows take the launch and the latency of one load (16 x 14336: 3.6 us).
// The maximum is that of the BF16 magnitudes as integers, which also orders
// infinities and NaN behind every finite value: a row that holds one gets the
// scale NaN (and codes 0), so that every product of the row is NaN.
//
// Each code is round(127 x / a), a the row's largest magnitude, rounded to
// even at halves, exactly: t = 127 x has 15 significant bits and is exact in
// FP32; y = t / a is corrected once with the exact remainder t - y a, after
// which a quotient that is a half (8 bits) is met exactly, and any other
// quotient of 8-bit significands lies at least 2^-18 away from a half, far
// outside the correction's error.  Row maxima near FP32's ends are moved by a
// power of two first, so that neither 127 x nor 1 / a leaves its range; what
// that flushes quantises to 0 either way.
// ---------------------------------------------------------------------------
struct QuantParams {
    const uint16_t *X;         // [M][ldx] BF16
    int8_t *Q;                 // [M][ldq]
    float *scale;              // [M]
    int64_t ldx, ldq;
    int M, K;
};

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    typedef unsigned short v2us __attribute__((ext_vector_type(2)));
    const v2us x = __builtin_bit_cast(v2us, a), y = __builtin_bit_cast(v2us, b);
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(x, y));
}

// The factors of one row: code = round(fma(t - y a, r, y)), y = t r, t = x c.
struct QuantRow {
    float c, a, r, scale;
    bool finite;
};

__device__ __forceinline__ QuantRow quant_row(uint32_t most) {      // the largest magnitude's BF16 bits
    QuantRow q;
    q.finite = most < 0x7F80u;
    const float m = bf16_float((uint16_t)most);
    const float s = m > 0x1p+60f ? 0x1p-64f : (m < 0x1p-60f ? 0x1p+64f : 1.0f);
    q.a = m * s;
    q.c = 127.0f * s;
    q.r = most ? 1.0f / q.a : 0.0f;
    q.scale = q.finite ? m / 127.0f : __builtin_nanf("");
    return q;
}

// 4 codes of two words of BF16 pairs; the rounding adds 1.5 2^23, after which
// the low byte of the sum's bits is the code.
__device__ __forceinline__ uint32_t quant4(const QuantRow &q, uint32_t w0, uint32_t w1) {
    auto code = [&](uint32_t bits) {
        const float t = __builtin_bit_cast(float, bits) * q.c;
        const float y = t * q.r;
        const float z = __builtin_fmaf(__builtin_fmaf(-y, q.a, t), q.r, y);
        return __builtin_bit_cast(uint32_t, z + 12582912.0f);
    };
    const uint32_t c0 = code(w0 << 16), c1 = code(w0 & 0xFFFF0000u), c2 = code(w1 << 16), c3 = code(w1 & 0xFFFF0000u);
    const uint32_t lo = __builtin_amdgcn_perm(c1, c0, 0x0C0C0400u), hi = __builtin_amdgcn_perm(c3, c2, 0x0C0C0400u);
    return lo | (hi << 16);
}

__device__ __forceinline__ v2u quant8(const QuantRow &q, v4u w) {
    if (!q.finite) return (v2u){0, 0};
    return (v2u){quant4(q, w[0], w[1]), quant4(q, w[2], w[3])};
}

__device__ __forceinline__ uint32_t most_of(uint32_t m, v4u w) {
#pragma unroll
    for (int e = 0; e < 4; ++e) m = max_u16x2(m, w[e] & 0x7FFF7FFFu);
    return m;
}

// The largest of T threads' pairs (T = 64: within the wave).
template <int T>
__device__ __forceinline__ uint32_t row_most(uint32_t m, uint32_t *part) {
#pragma unroll
    for (int d = 32; d > 0; d /= 2) m = max_u16x2(m, (uint32_t)__shfl_xor((int)m, d));
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
        __syncthreads();
        m = part[0];
#pragma unroll
        for (int w = 1; w < T / 64; ++w) m = max_u16x2(m, part[w]);
    }
    return max(m & 0xFFFFu, m >> 16);
}

// Rows of up to 8 T R values; a workgroup of max(T, 256) threads.
template <int T, int R>
__global__ __launch_bounds__(T < 256 ? 256 : T) void quantize_rows_kernel(QuantParams p) {
    __shared__ uint32_t part[T > 64 ? T / 64 : 1];
    constexpr int ROWS = T < 256 ? 256 / T : 1;
    const int64_t row = (int64_t)blockIdx.x * ROWS + (ROWS > 1 ? threadIdx.x / T : 0);
    if (row >= p.M) return;                        // (whole waves: T = 64)
    const int t = threadIdx.x % T;
    const uint16_t *x = p.X + row * p.ldx;
    v4u w[R];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int k = (i * T + t) * 8;
        w[i] = (v4u){0, 0, 0, 0};
        if (k < p.K) w[i] = *reinterpret_cast<const v4u *>(x + k);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) m = most_of(m, w[i]);
    const QuantRow q = quant_row(row_most<T>(m, part));
    int8_t *const out = p.Q + row * p.ldq;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int k = (i * T + t) * 8;
        if (k < p.K) *reinterpret_cast<v2u *>(out + k) = quant8(q, w[i]);
    }
    if (t == 0) p.scale[row] = q.scale;
}

// Longer rows: read twice, the second time from the caches.
__global__ __launch_bounds__(1024) void quantize_long_rows_kernel(QuantParams p) {
    __shared__ uint32_t part[16];
    const uint16_t *x = p.X + (int64_t)blockIdx.x * p.ldx;
    uint32_t m = 0;
    for (int k = threadIdx.x * 8; k < p.K; k += 8192) m = most_of(m, *reinterpret_cast<const v4u *>(x + k));
    const QuantRow q = quant_row(row_most<1024>(m, part));
    int8_t *const out = p.Q + (int64_t)blockIdx.x * p.ldq;
    for (int k = threadIdx.x * 8; k < p.K; k += 8192)
        *reinterpret_cast<v2u *>(out + k) = quant8(q, *reinterpret_cast<const v4u *>(x + k));
    if (threadIdx.x == 0) p.scale[blockIdx.x] = q.scale;
}

}  // namespace fp8g
