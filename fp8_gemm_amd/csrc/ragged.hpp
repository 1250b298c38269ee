// Ragged groups of rows: which rows, of which expert, a workgroup computes.
//
// The rows of expert g are offsets[g] .. offsets[g + 1] - 1, any number of
// them, starting anywhere.  The offsets are read on the device, so no count
// passes through the host: the host launches as many tiles as any offsets can
// need, and the workgroups past the actual number leave at once.
#pragma once

#include "device_common.hpp"

namespace fp8g {

// Placement of a workgroup's tile:
//   PLACE_DENSE   tile (tm, tn) of one product
//   PLACE_GROUPS  BM consecutive rows of one expert, times its weights
//   PLACE_REST    the same, and tiles of zeros over the rows of no expert
//                 (before offsets[0] and from offsets[G] on)
//   PLACE_SUMS    one expert's weight gradient, summed over its rows
enum { PLACE_DENSE = 0, PLACE_GROUPS = 1, PLACE_REST = 2, PLACE_SUMS = 3 };

// Row number from memory: offsets outside [0, M] count as the nearer end, so
// that no value in them leads outside the matrices.
__device__ __forceinline__ int row_offset(const int32_t *offsets, int i, int M) { return min(max(offsets[i], 0), M); }

// Inclusive sum of v over the wave's lanes up to this one.
__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int u = __shfl_up(v, d);
        if (lane >= d) v += u;
    }
    return v;
}

// The tiles of BM rows of all experts, in order of their rows.  Each wave
// works on its own, a lane per segment (an expert; with REST also the rows
// before the first and behind the last of them), 64 segments at a time.  Up to
// 64 segments (64 experts, or 62 with REST) are read once; more are read again,
// a batch of 64 after the other, for every tile that is looked for.
template <int BM, bool REST>
struct RaggedTiles {
    const int32_t *offsets;
    int G, M, lane;
    int lo, hi, upto;          // of the lane's expert in the batch read last: its rows, the tiles up to and with it

    // Tiles of a segment's rows (the sum in 32 bits without a sign: up to 2^31 - 1
    // rows, and a tile's more).
    __device__ __forceinline__ static int tiles_of(int rows) { return (int)(((unsigned)rows + (BM - 1)) / BM); }

    // Segment j: expert j, or with REST expert j - 1 between the rows before
    // the first expert (j = 0) and those behind the last (j = G + 1).
    __device__ __forceinline__ int segments() const { return REST ? G + 2 : G; }
    __device__ __forceinline__ int bound(int j) const {
        if (REST) return j == 0 ? 0 : (j == G + 2 ? M : row_offset(offsets, j - 1, M));
        return row_offset(offsets, j, M);
    }
    __device__ __forceinline__ int read(int first) {       // the batch's number of tiles
        const int j = min(first + lane, segments());
        lo = bound(j);
        hi = max(lo, bound(min(j + 1, segments())));
        upto = wave_scan(tiles_of(hi - lo), lane);
        return __builtin_amdgcn_readlane(upto, 63);
    }
    // The number of tiles, of which `most` (up to 2^30) suffice for offsets that
    // do not decrease.
    __device__ __forceinline__ int count(int most) {
        int n = 0;
        for (int first = 0; first < segments(); first += 64) n = min(max(n + read(first), 0), most);
        return n;
    }
    // Tile t: expert (-1: a tile of zeros), first row, rows; false if there is
    // no such tile.
    struct Spot {
        int g, m0, rows;
    };
    __device__ __forceinline__ bool find(int t, Spot &s, bool fresh) {
        for (int first = 0; first < segments(); first += 64) {
            if (fresh || segments() > 64) read(first);
            const unsigned long long past = __ballot(upto > t);
            if (past) {
                const int l = __builtin_ctzll(past);
                const int g = first + l - (REST ? 1 : 0);
                const int begin = __builtin_amdgcn_readlane(lo, l), end = __builtin_amdgcn_readlane(hi, l);
                const int tiles = tiles_of(end - begin);
                const int nth = t - (__builtin_amdgcn_readlane(upto, l) - tiles);
                // (offsets that decrease can overflow the sums of tiles)
                if ((unsigned)nth >= (unsigned)tiles) return false;
                s.g = REST && (g < 0 || g >= G) ? -1 : g;
                s.m0 = begin + nth * BM;
                s.rows = min(BM, end - s.m0);
                return true;
            }
            t -= __builtin_amdgcn_readlane(upto, 63);
        }
        return false;
    }
};

}  // namespace fp8g
