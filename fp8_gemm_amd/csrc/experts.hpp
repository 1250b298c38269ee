// Products over ragged groups of rows (BF16 and 8-bit integers) and the dense
// product in 8-bit integers.
//
//   groups  D[r] = sa[r] sb[g] (A[r] . B[g]^T)      r a row of expert g
//           dA[r] = dD[r] . B[g]   (zeros for the rows of no expert)
//           dB[g] = sum over g's rows of dD[r]^T . A[r]
//   int8    D = act(sa[m] sb[n] (A . B^T) + bias[n]) + R
#pragma once

#include "tile_halves.hpp"

namespace fp8g {

// ---------------------------------------------------------------------------
// Tiles of one expert's rows (tile_halves_body with the placements of
// ragged.hpp): the product, the token gradient (TB: weights read along N) and
// the weight gradients (TA and TB: both operands read along the rows, which are
// summed).  The matrix instructions bound the longest sums and, before them, the
// path of the copies into LDS; a tile's epilogue the short ones.  8 experts of
// 14336 x 4096 over 8192 rows, operands from memory: product 716 us (1340
// TFLOP/s), token gradient 842 us (2.25 rounds of 256 tiles, the last a quarter
// full), weight gradients 969 us (16 steps per tile; with operands from the
// caches 895, and 785 without the stores); 64 experts of 2048 x 4096 over 65536
// rows in 8-bit integers 504 us (2180 TOP/s).
// ---------------------------------------------------------------------------
template <int BM, int BN, int STAGES, bool INT, bool TA, bool TB, bool TAIL, int PLACE, int EPI>
__global__ __launch_bounds__(256, 1) void ragged_tile_kernel(RaggedParams<EPI, INT, PLACE> p) {
    tile_halves_body<BM, BN, STAGES, INT ? FMT_I8 : FMT_BF16, TA, TB, TAIL, PLACE>(p);
}

// Few rows per expert: 16 CB rows of one expert times 16 RB of its weight rows
// per workgroup, the waves splitting K (decode_body).  Reading the weights
// bounds it: 64 experts of 2048 x 4096 with 512 rows in all 188 us in BF16 (5.7
// TB/s), of 2048 x 7168 in 8-bit integers 159 us (5.9 TB/s).
template <int RB, int CB, bool INT, int D>
__global__ __launch_bounds__(256, 2) void ragged_decode_kernel(RaggedParams<EPI_ACT, INT, PLACE_GROUPS> p) {
    constexpr int FMT = INT ? FMT_I8 : FMT_BF16;
    decode_body<4, RB, CB, FMT, FMT, D, SCALE_CHANNEL>(p);
}

// The dense product in 8-bit integers (few tokens: fused_decode_kernel, 64 x
// 14336 x 4096 13.7 us).  Persistent for whole chunks of columns with neither
// activation nor residual (EPI_SCALED), bound as above: 4096 x 14336 x 4096 192
// us (2500 TOP/s), 4096^3 52 us.  With either, or columns that are no whole
// chunks, one tile per workgroup and the staged epilogue: the same with SiLU 241
// us, 4096 x 4096 x 14336 with a residual 172 us.
template <int BM, int BN, int STAGES, bool TAIL, int EPI>
__global__ __launch_bounds__(256, 1) void int8_tile_kernel(Int8Params<EPI> p) {
    tile_halves_body<BM, BN, STAGES, FMT_I8, false, false, TAIL, PLACE_DENSE>(p);
}

}  // namespace fp8g
