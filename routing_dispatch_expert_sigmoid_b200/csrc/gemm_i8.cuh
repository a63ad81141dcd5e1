// Tile lists of the int8 products, shared by their engines: the rows of each
// group, cut into chunks, times the column tiles.
#pragma once

#include "tcgen05_common.cuh"

namespace moe {
namespace tc {

// Row offsets and tile starts in shared memory: s_off[0..G] and the exclusive
// scan of the groups' tile counts s_tstart[0..G].  All threads of the block;
// ends with a barrier.  Returns the number of tiles, 0 after bad offsets.
__device__ __forceinline__ int build_tiles(const int32_t *offsets, int G, int fixed_rows,
                                           int rows_cap, int tile_rows, int col_tiles,
                                           int32_t *s_off, int32_t *s_tstart, int *abort_flag,
                                           uint32_t *err) {
  const int tid = threadIdx.x, lane = tid % 32;
  bool bad = false;
  for (int g = tid; g <= G; g += blockDim.x) {
    const int v = offsets ? offsets[g] : (g == 0 ? 0 : fixed_rows);
    s_off[g] = v;
    if (v < 0 || v > rows_cap) bad = true;
  }
  __syncthreads();
  for (int g = tid; g < G; g += blockDim.x) {
    const int rows = s_off[g + 1] - s_off[g];
    if (rows < 0) bad = true;
    s_tstart[g] = rows > 0 ? ((rows + tile_rows - 1) / tile_rows) * col_tiles : 0;
  }
  if (bad) {
    *abort_flag = 1;
    raise_error(err, kErrIndex);
  }
  __syncthreads();
  if (tid < 32) {  // in-place exclusive scan, 32 groups per step
    int carry = 0;
    for (int base = 0; base < G; base += 32) {
      const int g = base + lane;
      const int v = g < G ? s_tstart[g] : 0;
      int incl = v;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
      }
      if (g < G) s_tstart[g] = carry + incl - v;
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) s_tstart[G] = carry;
  }
  __syncthreads();
  return *abort_flag ? 0 : s_tstart[G];
}

// Tile -> group, column tile, first row and rows.  Tiles run group by group,
// row chunks fastest, so CTAs running at the same time share a weight tile; a
// role's tiles ascend, so the group is looked for from the last one on.
struct Tile {
  int g, c, row0, nr;
};
__device__ __forceinline__ Tile tile_at(int tile, int tile_rows, int G, const int32_t *s_off,
                                        const int32_t *s_tstart, int &cursor) {
  while (cursor + 1 < G && s_tstart[cursor + 1] <= tile) ++cursor;
  Tile t;
  t.g = cursor;
  const int rows = s_off[t.g + 1] - s_off[t.g];
  const int chunks = (rows + tile_rows - 1) / tile_rows;
  const int local = tile - s_tstart[t.g];
  t.c = local / chunks;
  const int m = local - t.c * chunks;
  t.row0 = s_off[t.g] + m * tile_rows;
  t.nr = min(tile_rows, rows - m * tile_rows);
  return t;
}

}  // namespace tc
}  // namespace moe
