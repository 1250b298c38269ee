// BF16 tiled kernel with fused epilogues, for the forward product and both
// backward products, and the kernels that form the gradients of the
// pre-activations and of the bias.
#pragma once

#include <utility>

#include "fused.hpp"

namespace fp8g {

// ---------------------------------------------------------------------------
// BF16 tiled kernel.  BM x BN outputs per workgroup of 4 waves (2 x 2) on
// v_mfma 16x16x32, K in steps of 64 elements through a direct-to-LDS ring of
// STAGES slots.  A step is two K halves (32 elements, one instruction per block
// pair) of T / 2 matrix instructions each:
//   - 0 .. T / 4: the fragments of the step's second half are read;
//   - barrier A, at 17 T / 64: everyone has read the step's slot, and its
//     refill (step kt + STAGES) is spread over the rest of the step;
//   - barrier B, at 5 T / 8: step kt + 1 has landed for everyone, and its first
//     half's fragments are read up to the step's end.
// With two slots a step's copies thus have 5 T / 8 instructions or more to land
// and go out over 47 T / 64 of them; one barrier in the middle of the step, for
// both, left T / 2 and T / 2.  The loop waits on its copies (in that form 4096 x
// 4096 x 16384 took 448 us, 326 without the loop's copies, 444 without its
// fragment reads), and the more evenly they go out the less: 4096^3 103.2 ->
// 99.7 us; token gradient of the gated 4096 x 14336 x 4096 851 (one barrier),
// 848 (copies over T / 2 from A on) -> 811 us (to the end), weight gradients
// 908, 929 -> 900 us.  Steps of 32 elements with twice the slots measured 8%
// slower than the one-barrier form on K-contiguous operands, whose rows are
// then fetched half a cache line at a time, and no faster on K-strided ones.
//
// Either operand may be K-contiguous (rows of K elements: ring rows of 128
// bytes, read with ds_read_b128; 16-byte chunk c of row r stored at c ^ ((r >>
// 1) & 7), as in tile16_body) or K-strided (TA / TB: rows of the operand's
// other dimension, one per K element: ring rows of BM or BN elements), so that
// the backward products need no transposed copies of the weights, tokens or
// gradients.  A K-strided fragment comes from ds_read_b64_tr_b16, which gives
// lane i of each 16 lanes column i of a 4 x 16 block of 16-bit values: 4 K
// elements of one row of the operand.  Two of them make the 16 bytes of a
// lane's fragment, in the K order of the K-contiguous form.  The 32-byte
// segments of a K-strided ring row k are stored at segment ^ strided_key(k):
// the 4 rows that 16 lanes read, and the 8 rows of 32 lanes, lie in different
// banks.
//
// Gated: blocks of 16 ring rows alternate between p.B and p.B2.
// ---------------------------------------------------------------------------
__device__ __forceinline__ int strided_key(int k) { return 2 * (k & 3) + ((k >> 3) & 1); }

// f(int_c<0>{}), ..., f(int_c<N - 1>{})
template <class F, int... I>
__device__ __forceinline__ void static_for_each(F f, std::integer_sequence<int, I...>) {
    (f(int_c<I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void static_for(F f) {
    static_for_each(f, std::make_integer_sequence<int, N>{});
}

typedef short v4s __attribute__((ext_vector_type(4)));
__device__ __forceinline__ v2u lds_read_tr16(const uint8_t *a) {
    return __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s *)a));
}

// TAIL: a K-contiguous operand whose K is not a multiple of 64.
template <int BM, int BN, int STAGES, bool TA, bool TB, bool TAIL, int EPI>
__global__ __launch_bounds__(256, 1) void bf16_tile_kernel(FusedParams<EPI, false> p) {
    constexpr bool GATED = EPI == EPI_GATED;
    static_assert(!GATED || (!TA && !TB), "gated: K-contiguous operands");
    constexpr int BK = 128, KE = BK / 2;           // a K step: bytes, elements
    constexpr int WM = 2, WN = 2, WAVES = WM * WN, THREADS = 64 * WAVES;
    constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
    constexpr int SLOT = (BM + BN) * BK;
    constexpr int CPA = BM / 8 / WAVES, CPB = BN / 8 / WAVES, CPW = CPA + CPB;   // 1 KB copies per wave per step
    constexpr int RING = STAGES * SLOT;
    constexpr int FPASS = (BM * BN * 4 + RING - 1) / RING, RW = TM / FPASS;   // epilogue passes, rows of a wave in each
    static_assert(CPA % 4 == 0 && CPB % 4 == 0, "copies split evenly");
    static_assert(STAGES >= 2 && CPW * (STAGES - 1) < 64, "ring");
    static_assert(FPASS <= 2 && RW % 16 == 0, "epilogue rows");
    constexpr int TERMS = EPI == EPI_ACT ? 3 * 1024 : 0;   // (copy_tile_terms; the biases are used)
    static_assert(RING + TERMS <= 160 * 1024, "LDS");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[RING + TERMS];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)smem;

    constexpr int BNO = GATED ? BN / 2 : BN;       // output columns of a tile
    int tm, tn;
    tile_coords<false>(blockIdx.x, p.tiles_m, p.tiles_n, tm, tn);
    const int m0 = tm * BM, n0 = tn * BNO;
    const int rows_m = min(p.M - m0, BM), rows_n = min(p.N - n0, BNO);
    const int y = blockIdx.y;
    uint16_t *const d = y ? p.D2 : p.D;
    // this split's K steps: kb .. kb + nk - 1
    constexpr bool SPLIT = EPI == EPI_PARTIAL;
    const int kb = SPLIT ? (int)blockIdx.z * p.ksteps : 0;
    const int nk = SPLIT ? min((p.K + KE - 1) / KE - kb, p.ksteps) : (p.K + KE - 1) / KE;

    // ---- copies ----
    // K-contiguous: copy qq fills ring rows 8 qq .. 8 qq + 7, lane l row l / 8,
    // stored chunk l % 8 holding logical chunk (l % 8) ^ key(row); the key
    // depends on qq through its parity only.  K-strided: copy qq fills 512 /
    // rows elements (2 or 4 K rows), lane l stored chunk l % (rows / 8) of row
    // l / (rows / 8).  A lane's offset within the tile is fixed per copy; each
    // step moves the descriptor's base and byte count.
    auto key16 = [](uint32_t row) { return (row >> 1) & 7u; };
    const uint32_t lr = (uint32_t)lane / 8;
    const uint32_t kc0 = (((uint32_t)lane % 8) ^ key16(lr)) * 16u;
    const uint32_t kc1 = (((uint32_t)lane % 8) ^ key16(8 + lr)) * 16u;
    auto strided_off = [&](int qq, int rows, int valid, int64_t ld) -> uint32_t {
        const int cpr = rows / 8;                  // 16-byte chunks per ring row
        const int k = qq * (512 / rows) + lane / cpr, pos = lane % cpr;
        const int col = ((pos >> 1) ^ strided_key(k)) * 16 + (pos & 1) * 8;
        // (columns come in whole chunks: the caller's `valid` is rounded up to 8)
        return col < valid ? (uint32_t)k * (uint32_t)ld + 2u * (uint32_t)col : kOobOffset;
    };
    // Gated: copies 4 q, 4 q + 1 fill ring rows 32 q .. + 15 with rows 16 q ..
    // + 15 of p.B, 4 q + 2 and 4 q + 3 the next 16 with those of p.B2 (a second
    // descriptor).
    uint32_t lo_a[CPA], lo_b[CPB];
#pragma unroll
    for (int i = 0; i < CPA; ++i) {
        const int qq = wave * CPA + i;
        lo_a[i] = TA ? strided_off(qq, BM, (rows_m + 7) & ~7, p.lda)
                     : (uint32_t)(qq * 8 + (int)lr) * (uint32_t)p.lda + ((i & 1) ? kc1 : kc0);
    }
#pragma unroll
    for (int i = 0; i < CPB; ++i) {
        const int qq = wave * CPB + i;
        const int row = GATED ? (qq / 4) * 16 + (qq & 1) * 8 + (int)lr : qq * 8 + (int)lr;
        lo_b[i] = TB ? strided_off(qq, BN, (rows_n + 7) & ~7, p.ldb)
                     : (uint32_t)row * (uint32_t)(GATED && (i & 2) ? p.ldb2 : p.ldb) + ((i & 1) ? kc1 : kc0);
    }
    const uint8_t *const a0 = p.A + (int64_t)y * p.a_gstride + (TA ? (int64_t)m0 * 2 : (int64_t)m0 * p.lda);
    const uint8_t *const b0 = p.B + (TB ? (int64_t)n0 * 2 : (int64_t)n0 * p.ldb);
    // K-strided: rows of K steps from ksplit on; gated: the second matrix
    const uint8_t *const b1 = p.B2 + (TB ? (int64_t)n0 * 2 : (int64_t)n0 * p.ldb2);
    const uint32_t bytes_a = rows_bytes(rows_m, p.lda), bytes_b = rows_bytes(rows_n, p.ldb);
    const uint32_t bytes_b1 = rows_bytes(rows_n, p.ldb2);
    v4i srdA, srdB, srdB1 = {0, 0, 0, 0};
    uint32_t lds_a = 0, lds_b = 0, ko0 = 0, ko1 = 0;
    auto set_step = [&](int kd) {                  // the copies of local step kd follow
        const int k = kb + kd;
        const bool in = kd < nk;
        if constexpr (TA) {
            srdA = make_srd(a0 + (int64_t)k * KE * p.lda, in ? rows_bytes(min(KE, p.K - k * KE), p.lda) : 0u);
        } else {
            srdA = make_srd(a0 + (int64_t)k * BK, in ? bytes_a - (uint32_t)(k * BK) : 0u);
        }
        if constexpr (TB) {
            const bool late = k >= p.ksplit;
            const int ks = late ? k - p.ksplit : k;
            srdB = make_srd((late ? b1 : b0) + (int64_t)ks * KE * p.ldb, in ? rows_bytes(min(KE, p.krows - ks * KE), p.ldb) : 0u);
        } else {
            srdB = make_srd(b0 + (int64_t)k * BK, in ? bytes_b - (uint32_t)(k * BK) : 0u);
            if constexpr (GATED) srdB1 = make_srd(b1 + (int64_t)k * BK, in ? bytes_b1 - (uint32_t)(k * BK) : 0u);
        }
        lds_a = lds0 + (uint32_t)(kd % STAGES) * SLOT + (uint32_t)(wave * CPA) * 1024u;
        lds_b = lds0 + (uint32_t)(kd % STAGES) * SLOT + (uint32_t)BM * BK + (uint32_t)(wave * CPB) * 1024u;
        // K-contiguous: lanes whose chunk starts at or past K
        if constexpr (TAIL) {
            const int lim = 2 * (p.K - k * KE);
            ko0 = (int)kc0 < lim ? 0u : kOobOffset;
            ko1 = (int)kc1 < lim ? 0u : kOobOffset;
        }
    };
    auto issue_one = [&](int i) {
        const uint32_t ko = (i & 1) ? ko1 : ko0;   // (CPA is even)
        if (i < CPA) dma16_m0(srdA, TA || !TAIL ? lo_a[i] : lo_a[i] + ko, lds_a + (uint32_t)i * 1024u);
        else dma16_m0(GATED && ((i - CPA) & 2) ? srdB1 : srdB, TB || !TAIL ? lo_b[i - CPA] : lo_b[i - CPA] + ko,
                      lds_b + (uint32_t)(i - CPA) * 1024u);
    };

    // ---- fragments: lane l carries row l % 16 of a 16-row block and, of K
    // half h, elements 8 (l / 16) .. + 7
    const int r16 = lane & 15, kg = lane >> 4;
    const uint32_t key = key16((uint32_t)r16);
    const uint32_t fo0 = (uint32_t)r16 * BK + (((uint32_t)kg ^ key) & 7u) * 16u;
    const uint32_t fo1 = (uint32_t)r16 * BK + (((uint32_t)(4 + kg) ^ key) & 7u) * 16u;
    // K-strided: offset of segment f of the wave's part
    const int trow = 8 * kg + (r16 >> 2);
    uint32_t to_a[FM], to_b[FN];
#pragma unroll
    for (int f = 0; f < FM; ++f)
        to_a[f] = (uint32_t)(trow * BM * 2 + ((wm * FM + f) ^ strided_key(trow)) * 32 + (lane & 3) * 8);
#pragma unroll
    for (int f = 0; f < FN; ++f)
        to_b[f] = (uint32_t)(trow * BN * 2 + ((wn * FN + f) ^ strided_key(trow)) * 32 + (lane & 3) * 8);
    auto frag = [&](auto strided, const uint8_t *base, uint32_t to, int rowb, int h) -> v4u {
        if constexpr (strided.value) {
            const uint8_t *r = base + to + 32 * h * rowb;
            const v2u p0 = lds_read_tr16(r), p1 = lds_read_tr16(r + 4 * rowb);
            return (v4u){p0[0], p0[1], p1[0], p1[1]};
        } else {
            return *reinterpret_cast<const v4u *>(base + (h ? fo1 : fo0));
        }
    };
    // fragment q of K half h: weight block q < FN, else token block q - FN
    auto read_frag = [&](v4u (&bf)[FN], v4u (&af)[FM], const uint8_t *slot, int h, int q) {
        if (q < FN) bf[q] = frag(int_c<TB>{}, slot + BM * BK + (TB ? 0 : (wn * TN + q * 16) * BK), to_b[q], BN * 2, h);
        else af[q - FN] = frag(int_c<TA>{}, slot + (TA ? 0 : (wm * TM + (q - FN) * 16) * BK), to_a[q - FN], BM * 2, h);
    };

    v4f acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = (v4f){0, 0, 0, 0};

    // One K step (see above).  (Unrolled by the template: the loop pragma gave
    // up on K-strided operands.)
    constexpr int NMF = FN * FM, NFR = FN + FM, T = 2 * NMF;
    constexpr int kRead1 = T / 4, kBarA = 17 * T / 64, kCopyTo = T, kBarB = 5 * T / 8;
    static_assert(kRead1 <= kBarA && kBarA < NMF && kBarB >= NMF && kCopyTo <= T, "schedule");
    // copies out at barrier B: those issued from barrier A on
    constexpr int kIssued = ((kBarB - kBarA) * CPW) / (kCopyTo - kBarA);
    static_assert(CPW * (STAGES - 2) + kIssued < 64, "copies in flight");
    v4u f0b[FN], f0a[FM], f1b[FN], f1a[FM];
    auto step = [&](int kt) {
        const uint8_t *cur = smem + (kt % STAGES) * SLOT;
        const uint8_t *nxt = smem + ((kt + 1) % STAGES) * SLOT;
        static_for<T>([&](auto tc) {
            constexpr int t = tc.value, i = (t % NMF) / FM, j = (t % NMF) % FM;
            if constexpr (t == kBarA) {
                __syncthreads();                   // step kt's slot is no longer read
                set_step(kt + STAGES);
            }
            if constexpr (t == kBarB) {
                vmcnt_wait<CPW * (STAGES - 2) + kIssued>();   // this wave's part of step kt + 1 has landed
                __syncthreads();                   // everyone's has
            }
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, t < NMF ? f0b[i] : f1b[i]),
                                                                __builtin_bit_cast(v8bf, t < NMF ? f0a[j] : f1a[j]),
                                                                acc[i][j], 0, 0, 0);
            if constexpr (t < kRead1) {
#pragma unroll
                for (int q = (t * NFR) / kRead1; q < ((t + 1) * NFR) / kRead1; ++q) read_frag(f1b, f1a, cur, 1, q);
            }
            if constexpr (t >= kBarA && t < kCopyTo) {
#pragma unroll
                for (int q = ((t - kBarA) * CPW) / (kCopyTo - kBarA); q < ((t - kBarA + 1) * CPW) / (kCopyTo - kBarA); ++q)
                    issue_one(q);
            }
            if constexpr (t >= kBarB) {
#pragma unroll
                for (int q = ((t - kBarB) * NFR) / (T - kBarB); q < ((t - kBarB + 1) * NFR) / (T - kBarB); ++q)
                    read_frag(f0b, f0a, nxt, 0, q);
            }
            __builtin_amdgcn_sched_barrier(0);
        });
    };

    if constexpr (EPI == EPI_ACT) copy_tile_terms(p, smem + RING, lds0 + (uint32_t)RING, wave, lane, m0, rows_m, n0, rows_n);
#pragma unroll
    for (int s = 0; s < STAGES; ++s) {
        set_step(s);
#pragma unroll
        for (int i = 0; i < CPW; ++i) issue_one(i);
    }
    vmcnt_wait<CPW * (STAGES - 1)>();              // this wave's part of step 0 has landed
    __syncthreads();
#pragma unroll
    for (int q = 0; q < NFR; ++q) read_frag(f0b, f0a, smem, 0, q);
    for (int kt = 0; kt < nk; ++kt) {
        __builtin_amdgcn_sched_barrier(0);
        step(kt);
    }
    vmcnt_wait<0>();                               // drain the copies past the last step
    __syncthreads();                               // every wave's have landed; the ring is free

    // (pinned to AGPRs at the loop's exit: without this the 128-row builds carry
    // the sums in VGPRs around the loop and copy them to AGPRs and back in every
    // step)
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) asm volatile("" : "+a"(acc[i][j]));

    // ---- epilogue: register r of a block holds weight row 4 (l / 16) + r and
    // token l % 16
    auto stage = [&](auto pass) {
#pragma unroll
        for (int jj = 0; jj < RW / 16; ++jj)
#pragma unroll
            for (int i = 0; i < FN; ++i)
                stage_f32<BN>(smem, wm * RW + jj * 16 + r16, wn * TN + i * 16 + kg * 4, acc[i][pass.value * (RW / 16) + jj]);
    };
#pragma unroll 1
    for (int h = 0; h < FPASS; ++h)
        fused_store_rows<BN, WM * RW>(
            p, smem, smem + RING, tid, m0, rows_m, n0, d, [=](int s) { return (s / RW) * TM + h * RW + s % RW; },
            [&] {
                if (h == 0) {
                    stage(int_c<0>{});
                } else {
                    __syncthreads();               // the staged rows have been read
                    stage(int_c<FPASS - 1>{});
                }
                __syncthreads();
            });
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
