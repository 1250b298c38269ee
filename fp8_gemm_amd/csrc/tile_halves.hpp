// Tiled kernel body of the products whose 128-byte K step is two instructions
// per block pair (BF16, 8-bit integers), dense or over ragged groups of rows.
#pragma once

#include <utility>

#include "fused.hpp"
#include "ragged.hpp"

namespace fp8g {

// ---------------------------------------------------------------------------
// BM x BN outputs per workgroup of 4 waves (2 x 2), K in steps of 128 bytes
// through a direct-to-LDS ring of STAGES slots.  A step is two K halves of 64
// bytes, one instruction per block pair and half: v_mfma 16x16x32 with BF16
// operands, 16x16x64 with 8-bit integers, which has the same operand layout in
// bytes (lane l: row l % 16, 16 bytes from 16 (l / 16) on) and takes the same
// time, so that all of the following, measured with BF16, holds for both.  A
// half is T / 2 matrix instructions:
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
//
// PLACE: whose rows the tile holds (ragged.hpp).  Ragged groups cost the loop
// nothing: a tile's rows are consecutive rows of one expert, the descriptors
// end behind the last of them, and only where they begin comes from the
// offsets (one round of loads and a scan over the experts before the first
// copy).
//
// Persistent workgroups (every placement but the dense BF16 products'): one per
// CU, each on tiles blockIdx.x, + gridDim.x, ..., so that the number of tiles
// need not be known to the host.  A tile's first copies go out before the
// tile before it is written, which hides their way from memory, the launch and
// most of the offsets' loads behind the epilogue.  Tiles of at most BM / 2 rows (an expert's
// last rows, the cut tiles of the last round) run a step of half the matrix
// instructions, which takes about 0.7 of a whole one's time: 4096 x 14336 x 4096
// in 8-bit integers, 3.5 rounds, 196 -> 189 us; 2048 x 4096 x 14336, half a
// round, 121 -> 95 us.  They stay in the order of the rows: moved behind all
// whole tiles, for a balanced end, each expert's weights came from memory twice,
// 8 experts of 14336 x 4096 over 8192 rows 795 against 757 us.
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

// TAIL: a K-contiguous operand whose K is not a multiple of the K step.
template <int BM, int BN, int STAGES, int FMT, bool TA, bool TB, bool TAIL, int PLACE, class P>
__device__ __forceinline__ void tile_halves_body(P p) {
    constexpr int EPI = P::kEpilogue;
    constexpr bool GATED = EPI == EPI_GATED, I8 = FMT == FMT_I8;
    static_assert(!GATED || (!TA && !TB), "gated: K-contiguous operands");
    static_assert(I8 ? !TA && !TB : FMT == FMT_BF16, "8-bit integers: K-contiguous operands");
    static_assert(I8 == P::kIntSums, "the epilogue reads the sums' type");
    static_assert(PLACE == PLACE_SUMS ? TA && TB : PLACE == PLACE_DENSE || !TA, "ragged rows or ragged sums");
    constexpr int ES = I8 ? 1 : 2;                 // bytes of an element
    constexpr int BK = 128, KE = BK / ES;          // a K step: bytes, elements
    using Acc = typename AccOf<FMT>::type;
    constexpr int WM = 2, WN = 2, WAVES = WM * WN, THREADS = 64 * WAVES;
    constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
    constexpr int SLOT = (BM + BN) * BK;
    constexpr int CPA = BM / 8 / WAVES, CPB = BN / 8 / WAVES, CPW = CPA + CPB;   // 1 KB copies per wave per step
    constexpr int RING = STAGES * SLOT;
    constexpr int FPASS = (BM * BN * 4 + RING - 1) / RING, RW = TM / FPASS;   // epilogue passes, rows of a wave in each
    static_assert(CPA % 4 == 0 && CPB % 4 == 0, "copies split evenly");
    static_assert(STAGES >= 2 && CPW * (STAGES - 1) < 64, "ring");
    static_assert(FPASS <= 2 && RW % 16 == 0, "epilogue rows");
    // Persistent workgroups with the direct epilogue (see above).
    constexpr bool PERSIST = PLACE != PLACE_DENSE || EPI == EPI_SCALED;
    static_assert(!PERSIST || EPI == EPI_STORE || EPI == EPI_SCALED, "direct epilogues");
    // row scales, column scales and biases (copy_tile_terms); persistent: of
    // two tiles in turn
    constexpr int TERMS = EPI == EPI_ACT || EPI == EPI_SCALED ? 3 * 1024 : 0;
    constexpr int STAGE_AT = RING + 2 * TERMS, STAGE = 2048;       // direct epilogue: 16 rows x 64 columns per wave
    constexpr int SMEM = PERSIST ? STAGE_AT + WAVES * STAGE : RING + TERMS;
    static_assert(SMEM <= 160 * 1024, "LDS");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[SMEM];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)smem;
    constexpr int BNO = GATED ? BN / 2 : BN;       // output columns of a tile

    // ---- the tiles of this workgroup
    struct Where {
        int g, m0, rows, tn;                       // expert, first row and rows, column of tiles
    };
    // Persistent: whole tiles in rounds of one per workgroup, and if the last
    // round has work for at most half of them, its `cut` tiles in two halves
    // each, by rows.
    using Tiles = RaggedTiles<BM, PLACE == PLACE_REST>;
    Tiles tiles = {};
    int row_tiles = 0, whole = 0, cut = 0;
    if constexpr (PERSIST) {
        if constexpr (PLACE == PLACE_GROUPS || PLACE == PLACE_REST) {
            tiles = Tiles{p.offsets, p.G, p.M, lane, 0, 0, 0};
            row_tiles = tiles.count(p.tiles_m);
        } else {
            row_tiles = PLACE == PLACE_SUMS ? p.G * p.tiles_m : p.tiles_m;
        }
        whole = row_tiles * p.tiles_n;
        const int left = whole % (int)gridDim.x;
        if (2 * left <= (int)gridDim.x) cut = left;
        whole -= cut;
    }
    auto place = [&](int t, Where &w) -> bool {
        int tm, tn;
        if constexpr (!PERSIST) {
            tile_coords<false>(t, p.tiles_m, p.tiles_n, tm, tn);
            w = Where{0, tm * BM, min(p.M - tm * BM, BM), tn};
            return true;
        }
        const int u = t - whole;                   // >= 0: half u / cut of a tile
        if (u >= 2 * cut) return false;
        // (the dense order keeps each XCD on its own part of the matrix, the
        // other one all of them on the same experts)
        tile_coords<PLACE != PLACE_DENSE>(u < cut ? t : t - cut, row_tiles, p.tiles_n, tm, tn);
        if constexpr (PLACE == PLACE_GROUPS || PLACE == PLACE_REST) {
            typename Tiles::Spot spot;
            if (!tiles.find(tm, spot, false)) return false;
            w = Where{spot.g, spot.m0, spot.rows, tn};
        } else {
            const int m0 = (PLACE == PLACE_SUMS ? tm % p.tiles_m : tm) * BM;
            w = Where{PLACE == PLACE_SUMS ? tm / p.tiles_m : 0, m0, min(p.M - m0, BM), tn};
        }
        if (u >= cut) w.m0 += BM / 2;
        if (u >= 0) w.rows = u < cut ? min(w.rows, BM / 2) : max(0, w.rows - BM / 2);
        return true;
    };
    Where now;
    if (!place(blockIdx.x, now) && PERSIST) return;
    const int y = PERSIST ? 0 : blockIdx.y;
    // this split's K steps: kb .. kb + nk - 1
    constexpr bool SPLIT = EPI == EPI_PARTIAL;
    const int kb = SPLIT ? (int)blockIdx.z * p.ksteps : 0;

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
    // The tile being copied: operands, rows, K; set by `aim`.
    uint32_t lo_a[CPA], lo_b[CPB], bytes_a, bytes_b, bytes_b1;
    const uint8_t *a0, *b0, *b1;
    uint16_t *d;
    int m0, n0, rows_m, rows_n, K = p.K, krows = p.krows, nk;
    const float *const expert_sb = P::kScaled ? p.ch_sb : nullptr;
    auto aim = [&](const Where &w) {
        // (uniform, which the compiler does not see through the persistent
        // loop; the branches and the copies' LDS addresses depend on it)
        auto uniform = [](int v) { return PERSIST ? __builtin_amdgcn_readfirstlane(v) : v; };
        m0 = uniform(w.m0);
        rows_m = uniform(w.rows);
        n0 = uniform(w.tn) * BNO;
        rows_n = min(p.N - n0, BNO);
        const uint8_t *A = p.A + (int64_t)y * p.a_gstride, *B = p.B;
        d = y ? p.D2 : p.D;
        if constexpr (PLACE == PLACE_GROUPS || PLACE == PLACE_REST) {
            if (PLACE == PLACE_REST) K = w.g < 0 ? 0 : p.K;        // (the empty sum)
            B += (int64_t)max(w.g, 0) * p.b_gstride;
            if (P::kScaled && expert_sb) p.ch_sb = expert_sb + (int64_t)w.g * p.N;
        }
        if constexpr (PLACE == PLACE_SUMS) {
            // the expert's rows are the K elements of both operands
            const int first = row_offset(p.offsets, w.g, p.rows);
            K = krows = max(0, row_offset(p.offsets, w.g + 1, p.rows) - first);
            A += (int64_t)first * p.lda;
            B += (int64_t)first * p.ldb;
            d += (int64_t)w.g * p.d_gstride;
        }
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
        a0 = A + (TA ? (int64_t)m0 * 2 : (int64_t)m0 * p.lda);
        b0 = B + (TB ? (int64_t)n0 * 2 : (int64_t)n0 * p.ldb);
        // K-strided: rows of K steps from ksplit on; gated: the second matrix
        b1 = p.B2 + (TB ? (int64_t)n0 * 2 : (int64_t)n0 * p.ldb2);
        bytes_a = rows_bytes(rows_m, p.lda);
        bytes_b = rows_bytes(rows_n, p.ldb);
        bytes_b1 = rows_bytes(rows_n, p.ldb2);
        nk = SPLIT ? min((K + KE - 1) / KE - kb, p.ksteps) : (K + KE - 1) / KE;
        // the second half of a cut tile may have no rows: no steps then, whose
        // descriptors would count bytes down from 0
        if (PERSIST && rows_m <= 0) nk = 0;
    };
    aim(now);
    v4i srdA, srdB, srdB1 = {0, 0, 0, 0};
    uint32_t lds_a = 0, lds_b = 0, ko0 = 0, ko1 = 0;
    auto set_step = [&](int kd) {                  // the copies of local step kd follow
        const int k = kb + kd;
        const bool in = kd < nk;
        if constexpr (TA) {
            srdA = make_srd(a0 + (int64_t)k * KE * p.lda, in ? rows_bytes(min(KE, K - k * KE), p.lda) : 0u);
        } else {
            srdA = make_srd(a0 + (int64_t)k * BK, in ? bytes_a - (uint32_t)(k * BK) : 0u);
        }
        if constexpr (TB) {
            const bool late = PLACE == PLACE_DENSE && k >= p.ksplit;
            const int ks = late ? k - p.ksplit : k;
            srdB = make_srd((late ? b1 : b0) + (int64_t)ks * KE * p.ldb, in ? rows_bytes(min(KE, krows - ks * KE), p.ldb) : 0u);
        } else {
            srdB = make_srd(b0 + (int64_t)k * BK, in ? bytes_b - (uint32_t)(k * BK) : 0u);
            if constexpr (GATED) srdB1 = make_srd(b1 + (int64_t)k * BK, in ? bytes_b1 - (uint32_t)(k * BK) : 0u);
        }
        lds_a = lds0 + (uint32_t)(kd % STAGES) * SLOT + (uint32_t)(wave * CPA) * 1024u;
        lds_b = lds0 + (uint32_t)(kd % STAGES) * SLOT + (uint32_t)BM * BK + (uint32_t)(wave * CPB) * 1024u;
        // K-contiguous: lanes whose chunk starts at or past K
        if constexpr (TAIL) {
            const int lim = ES * (K - k * KE);
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

    // Row blocks of 16 of the token side: the wave's part in one piece, or
    // (persistent) every second one, so that a tile's rows, however few, are
    // shared by both waves.
    auto row_block = [&](int f) { return PERSIST ? 2 * f + wm : wm * FM + f; };

    // ---- fragments: lane l carries row l % 16 of a 16-row block and, of K
    // half h, bytes 16 (l / 16) .. + 15
    const int r16 = lane & 15, kg = lane >> 4;
    const uint32_t key = key16((uint32_t)r16);
    const uint32_t fo0 = (uint32_t)r16 * BK + (((uint32_t)kg ^ key) & 7u) * 16u;
    const uint32_t fo1 = (uint32_t)r16 * BK + (((uint32_t)(4 + kg) ^ key) & 7u) * 16u;
    // K-strided: offset of segment f of the wave's part
    const int trow = 8 * kg + (r16 >> 2);
    uint32_t to_a[FM], to_b[FN];
#pragma unroll
    for (int f = 0; f < FM; ++f)
        to_a[f] = (uint32_t)(trow * BM * 2 + (row_block(f) ^ strided_key(trow)) * 32 + (lane & 3) * 8);
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
        else af[q - FN] = frag(int_c<TA>{}, slot + (TA ? 0 : row_block(q - FN) * 16 * BK), to_a[q - FN], BM * 2, h);
    };

    // The sums of FN x FMV blocks: FMV = FM, or (half tiles) FM / 2.
    auto clear = [&](auto &acc) {
        constexpr int FMV = sizeof(acc[0]) / sizeof(Acc);
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FMV; ++j) acc[i][j] = (Acc){0, 0, 0, 0};
    };
    auto pin = [&](auto &acc) {
        constexpr int FMV = sizeof(acc[0]) / sizeof(Acc);
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FMV; ++j) asm volatile("" : "+a"(acc[i][j]));
    };

    // One K step (see above).  (Unrolled by the template: the loop pragma gave
    // up on K-strided operands.)
    v4u f0b[FN], f0a[FM], f1b[FN], f1a[FM];
    auto step = [&](auto &acc, int kt) {
        constexpr int FMV = sizeof(acc[0]) / sizeof(Acc);
        constexpr int NMF = FN * FMV, NFR = FN + FMV, T = 2 * NMF;
        constexpr int kRead1 = T / 4, kBarA = 17 * T / 64, kCopyTo = T, kBarB = 5 * T / 8;
        static_assert(kRead1 <= kBarA && kBarA < NMF && kBarB >= NMF && kCopyTo <= T, "schedule");
        // copies out at barrier B: those issued from barrier A on
        constexpr int kIssued = ((kBarB - kBarA) * CPW) / (kCopyTo - kBarA);
        static_assert(CPW * (STAGES - 2) + kIssued < 64, "copies in flight");
        const uint8_t *cur = smem + (kt % STAGES) * SLOT;
        const uint8_t *nxt = smem + ((kt + 1) % STAGES) * SLOT;
        static_for<T>([&](auto tc) {
            constexpr int t = tc.value, i = (t % NMF) / FMV, j = (t % NMF) % FMV;
            if constexpr (t == kBarA) {
                __syncthreads();                   // step kt's slot is no longer read
                set_step(kt + STAGES);
            }
            if constexpr (t == kBarB) {
                vmcnt_wait<CPW * (STAGES - 2) + kIssued>();   // this wave's part of step kt + 1 has landed
                __syncthreads();                   // everyone's has
            }
            acc[i][j] = mfma_half<FMT>(t < NMF ? f0b[i] : f1b[i], t < NMF ? f0a[j] : f1a[j], acc[i][j]);
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

    // The copies ahead of a tile's first step: its terms (into slot `part`), STAGES steps.
    auto begin = [&](int part) {
        if constexpr (TERMS > 0)
            copy_tile_terms(p, smem + RING + part * TERMS, lds0 + (uint32_t)(RING + part * TERMS), wave, lane, m0, rows_m, n0, rows_n);
#pragma unroll
        for (int s = 0; s < STAGES; ++s) {
            set_step(s);
#pragma unroll
            for (int i = 0; i < CPW; ++i) issue_one(i);
        }
    };
    auto sum = [&](auto &acc) {
        constexpr int FMV = sizeof(acc[0]) / sizeof(Acc);
        __syncthreads();                           // everyone's part of step 0 has landed
#pragma unroll
        for (int q = 0; q < FN + FMV; ++q) read_frag(f0b, f0a, smem, 0, q);
        // (pinned to AGPRs at the loop's exit: without this the 128-row builds
        // carry the sums in VGPRs around the loop and copy them to AGPRs and
        // back in every step.  Integer sums, and those of the persistent forms,
        // need it at both ends of the loop's body as well: 450 copies beside
        // the 128 matrix instructions of a step otherwise, and 4096 x 14336 x
        // 4096 in 8-bit integers took 305 us.)
        constexpr bool kPin = I8 || PERSIST;
        if constexpr (kPin) pin(acc);
        for (int kt = 0; kt < nk; ++kt) {
            __builtin_amdgcn_sched_barrier(0);
            step(acc, kt);
            if constexpr (kPin) pin(acc);
        }
    };

    begin(0);
    if constexpr (PERSIST) {
        // The direct epilogue, a wave by itself: 16 rows x 64 columns of its
        // part at a time are rounded, laid out by rows in its own 2 KB of LDS
        // (chunk c of row r at c ^ (r % 8)) and stored as whole 128-byte row
        // segments, while the next tile's copies are under way.  Stores outside
        // the matrix get an offset past the descriptor's end instead of a
        // branch, so that their number is known to the wait for those copies.
        constexpr int PASS_N = TN / 64;
        constexpr int STORES = FM * PASS_N * 2;    // of a wave (half tiles: half of them)
        static_assert(TN % 64 == 0 && CPW * (STAGES - 1) + STORES < 64, "stores in flight");
        uint8_t *const st = smem + STAGE_AT + wave * STAGE;
        const uint32_t ld2 = (uint32_t)p.ldd * 2u;
        auto store = [&](const auto &acc, uint16_t *out, int rows, int col0, const uint8_t *terms) {
            constexpr int PASSES = sizeof(acc[0]) / sizeof(Acc) * PASS_N;
            // (the lane taken afresh: nothing of this is kept live across the loop)
            const int el = lane_id_here(), r16 = el & 15, kg = el >> 4, er = el >> 3, ec = el & 7;
            uint32_t put[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                put[i] = (uint32_t)(r16 * 128 + (((i * 2 + (kg >> 1)) ^ (r16 & 7)) * 16) + (kg & 1) * 8);
            const uint32_t get = (uint32_t)(er * 128 + ((ec ^ er) * 16));
            const __amdgpu_buffer_rsrc_t to = make_rsrc(out, rows_bytes(rows, (int64_t)ld2));
            const float *const tf = reinterpret_cast<const float *>(terms);
            v4u held[2];
            uint32_t at[2];
            RowFactors sa = {1.0f, 1.0f};          // of the 16 rows at hand
            static_for<PASSES + 1>([&](auto pc) {
                constexpr int pass = pc.value, j = pass / PASS_N, h = pass % PASS_N;
                v4u v[2];
                if constexpr (pass < PASSES) {
                    if constexpr (EPI == EPI_SCALED && h == 0) sa = row_factors(tf[row_block(j) * 16 + r16]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v4f z = sums_f32(acc[h * 4 + i][j]);
                        if constexpr (EPI == EPI_SCALED) {
                            const int c = wn * TN + (h * 4 + i) * 16 + kg * 4;
                            const v4f sb = *reinterpret_cast<const v4f *>(tf + 256 + c), b = *reinterpret_cast<const v4f *>(tf + 512 + c);
#pragma unroll
                            for (int e = 0; e < 4; ++e) z[e] = z[e] * sa.first * (sb[e] * sa.rest) + b[e];
                        }
                        *reinterpret_cast<v2u *>(st + put[i]) = pack_bf16x4(z[0], z[1], z[2], z[3]);
                    }
                    // (a wave's LDS accesses keep their order: the next pass may write behind these reads)
                    v[0] = *reinterpret_cast<const v4u *>(st + get);
                    v[1] = *reinterpret_cast<const v4u *>(st + get + 1024);
                }
                if constexpr (pass > 0) {
                    bool stream = false;
                    if constexpr (PLACE == PLACE_SUMS) stream = p.stream;
                    if (stream) {                  // (cache bit 2: nontemporal)
                        __builtin_amdgcn_raw_buffer_store_b128(held[0], to, at[0], 0, 2);
                        __builtin_amdgcn_raw_buffer_store_b128(held[1], to, at[1], 0, 2);
                    } else {
                        __builtin_amdgcn_raw_buffer_store_b128(held[0], to, at[0], 0, 0);
                        __builtin_amdgcn_raw_buffer_store_b128(held[1], to, at[1], 0, 0);
                    }
                }
                if constexpr (pass < PASSES) {
                    const int col = wn * TN + h * 64 + ec * 8;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int row = row_block(j) * 16 + q * 8 + er;
                        at[q] = row < rows && col0 + col < p.N ? (uint32_t)row * ld2 + 2u * (uint32_t)col : kOobOffset;
                        held[q] = v[q];
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            });
        };
        int t = blockIdx.x, part = 0, stores = 0;  // stores issued behind the copies of the tile at hand
        // One tile (each kind with registers of its own for the sums: shared by
        // both loops they were spilled); true: another one is under way.
        auto tile = [&](auto fmv) -> bool {
            constexpr int FMV = fmv.value;
            Acc acc[FN][FMV];
            clear(acc);
            // this wave's part of step 0 has landed
            if (stores == 0) vmcnt_wait<CPW * (STAGES - 1)>();
            else if (stores == 1) vmcnt_wait<CPW * (STAGES - 1) + STORES / 2>();
            else vmcnt_wait<CPW * (STAGES - 1) + STORES>();
            t += gridDim.x;
            Where next;
            // (the offsets of more than 64 segments are loaded here, before the
            // loop, and waited for with the copies at hand; a weight gradient's
            // two offsets behind it, in aim)
            const bool more = __builtin_amdgcn_readfirstlane(place(t, next));
            sum(acc);
            uint16_t *const out = d + (int64_t)m0 * p.ldd + n0;
            const int rows = rows_m, col0 = n0;
            vmcnt_wait<0>();                       // the copies past the last step (zeros)
            // (No barrier: the slots refilled now were last read before the last
            // step's first barrier, but for fragments that nobody uses.)
            if (more) {
                aim(next);
                begin(part ^ 1);
            }
            // the last matrix instruction's result may be read: the pins above
            // hide it from the compiler, which would have waited itself
            asm volatile("s_nop 15\n\ts_nop 7" ::: "memory");
            pin(acc);
            store(acc, out, rows, col0, smem + RING + part * TERMS);
            part ^= 1;
            stores = FMV == FM ? 2 : 1;
            return more;
        };
        while (rows_m <= BM / 2 ? tile(int_c<FM / 2>{}) : tile(int_c<FM>{})) {}
    } else {
    Acc acc[FN][FM];
    clear(acc);
    vmcnt_wait<CPW * (STAGES - 1)>();              // this wave's part of step 0 has landed
    sum(acc);
    vmcnt_wait<0>();                               // drain the copies past the last step
    __syncthreads();                               // every wave's have landed; the ring is free
    pin(acc);

    // ---- epilogue: register r of a block holds weight row 4 (l / 16) + r and
    // token l % 16
    auto stage = [&](auto pass) {
#pragma unroll
        for (int jj = 0; jj < RW / 16; ++jj)
#pragma unroll
            for (int i = 0; i < FN; ++i)
                stage_f32<BN>(smem, wm * RW + jj * 16 + r16, wn * TN + i * 16 + kg * 4,
                              __builtin_bit_cast(v4f, acc[i][pass.value * (RW / 16) + jj]));
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
}

}  // namespace fp8g
