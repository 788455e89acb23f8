// Token tiles of expert-sorted rows, written by one block of a launch that runs
// before the products.
#pragma once

#include <hip/hip_runtime.h>

namespace moe {

struct TileList {
  const int* offsets;
  int E, tile;
  int4* tiles;
  int* ntiles;
};

// By 256 threads of one block: tiles[i] = (expert, first row, first tile of its group, tiles in the group), groups of up
// to GROUP tiles of one expert, which share a weight slab next to each other.
template <int GROUP>
__device__ __forceinline__ void write_tiles(const TileList& l) {
  __shared__ int part[4];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  int base = 0;
  for (int e0 = 0; e0 < l.E; e0 += 256) {
    const int e = e0 + tid;
    int first = 0, c = 0;
    if (e < l.E) {
      first = l.offsets[e];
      c = (max(0, l.offsets[e + 1] - first) + l.tile - 1) / l.tile;
    }
    int s = c;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(s, d, 64);
      if (lane >= d) s += o;
    }
    if (lane == 63) part[wv] = s;
    __syncthreads();
    int at = base + s - c;
    for (int i = 0; i < 4; ++i) {
      if (i < wv) at += part[i];
      base += part[i];
    }
    for (int i = 0; i < c; ++i) {
      const int g = i / GROUP * GROUP;
      l.tiles[at + i] = make_int4(e, first + i * l.tile, at + g, min(GROUP, c - g));
    }
    __syncthreads();
  }
  if (tid == 0) *l.ntiles = base;
}

}  // namespace moe
