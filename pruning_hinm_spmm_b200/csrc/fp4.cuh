// The 4-bit matrices' geometry (hinm.h, section b1), shared by the quantiser, the products
// and the argument checks.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/hinm.h"

namespace hinm {

constexpr int kFp4RowTile = 128;     // rows whose scales one 512-byte chunk holds
constexpr int kFp4ChunkBytes = 512;  // 128 rows x 4 blocks
constexpr int kFp4DepthPad = 128;    // depth is stored in multiples of it
constexpr int kFp4MaxGroups = 512;  // ragged groups (the products keep a table of them)

__host__ __device__ constexpr int fp4_block(int format) { return format == HINM_FP4_NV ? 16 : 32; }

struct Fp4Geom {
  long long depth_pad;  // stored depth
  long long row_tiles;  // scale tiles of 128 rows of one matrix of the batch
  __host__ __device__ long long pitch() const { return depth_pad / 2; }  // bytes of a row
  __host__ __device__ long long chunks(int format) const {
    return depth_pad / (4 * fp4_block(format));
  }
};

// Ragged rows: group e's scale tiles start at tile o_e / 128 + e, so that every group starts
// a tile of its own without a sum over the groups before it: with n rows the next group's
// first tile is at least ceil(n / 128) further on.  Ragged depth: the same in steps of 128
// of the stored depth.
__host__ __device__ inline Fp4Geom fp4_geom(int rows, int depth, int ragged, int groups) {
  Fp4Geom g;
  g.depth_pad = ragged == HINM_RAGGED_DEPTH
                    ? ((long long)depth / kFp4DepthPad + groups) * kFp4DepthPad
                    : ((long long)depth + kFp4DepthPad - 1) / kFp4DepthPad * kFp4DepthPad;
  g.row_tiles = ragged == HINM_RAGGED_ROWS ? (long long)rows / kFp4RowTile + groups
                                           : ((long long)rows + kFp4RowTile - 1) / kFp4RowTile;
  return g;
}

// First scale tile (ragged rows) or first 128-step of the stored depth (ragged depth) of the
// group that starts at `offset`.
__host__ __device__ inline long long fp4_group_tile(int offset, int e) {
  return (long long)(offset / kFp4RowTile) + e;
}

}  // namespace hinm
