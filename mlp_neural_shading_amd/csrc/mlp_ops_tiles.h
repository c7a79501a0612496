// mlp_ops_tiles.h -- which rows the tiles of a grouped product take: the arithmetic, the same on the GPU and on the host
// (where its edges can be checked without a GPU).
#pragma once

#include <hip/hip_runtime.h>

namespace mlpk {

// Tiles of bn rows that the rows [begin, end) make.
__host__ __device__ inline int tiles_in(int begin, int end, int bn) { return end > begin ? (end - begin - 1) / bn + 1 : 0; }

// The first row of tile `tile` of the rows from `begin` on, for a tile there is; any number for others.
__host__ __device__ inline int tile_begin(int begin, int bn, int tile)
{
    return (int)((unsigned)begin + (unsigned)tile * (unsigned)bn);
}

// The row behind the last of the tile that begins at row0 < end: row0 + bn may pass INT_MAX.
__host__ __device__ inline int tile_end(int row0, int end, int bn) { return end - row0 > bn ? row0 + bn : end; }

}  // namespace mlpk
