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
// ragged.hpp).
// ---------------------------------------------------------------------------
template <int BM, int BN, int STAGES, bool INT, bool TA, bool TB, bool TAIL, int PLACE, int EPI>
__global__ __launch_bounds__(256, 1) void ragged_tile_kernel(RaggedParams<EPI, INT, PLACE> p) {
    tile_halves_body<BM, BN, STAGES, INT ? FMT_I8 : FMT_BF16, TA, TB, TAIL, PLACE>(p);
}

// Few rows per expert: 16 CB rows of one expert times 16 RB of its weight rows
// per workgroup, the waves splitting K (decode_body).
template <int RB, int CB, bool INT, int D>
__global__ __launch_bounds__(256, 2) void ragged_decode_kernel(RaggedParams<EPI_ACT, INT, PLACE_GROUPS> p) {
    constexpr int FMT = INT ? FMT_I8 : FMT_BF16;
    decode_body<4, RB, CB, FMT, FMT, D, SCALE_CHANNEL>(p);
}

// The dense product in 8-bit integers (few tokens: fused_decode_kernel).
template <int BM, int BN, int STAGES, bool TAIL, int EPI>
__global__ __launch_bounds__(256, 1) void int8_tile_kernel(Int8Params<EPI> p) {
    tile_halves_body<BM, BN, STAGES, FMT_I8, false, false, TAIL, PLACE_DENSE>(p);
}

}  // namespace fp8g
