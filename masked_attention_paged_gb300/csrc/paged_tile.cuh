// paged_tile.cuh -- a 128-key tile of a paged cache in shared memory, gathered
// from eight 16-token blocks with one TMA load each.
//
// A load brings all 16 rows of a (block, KV head), 64-column halves and 8-row
// groups as box dimensions: [row group][half][8 rows x 128 bytes], 128-byte
// swizzle.  Groups of 8 rows are then a constant H * 1024 bytes apart through the
// whole tile (H = D / 64 halves), which is all a K-major (K) or MN-major (V)
// matrix descriptor asks for.
//
// A load brings 4 KB (D = 128), so a tile of K and V takes sixteen; their issue is
// no small matter: a single producer warp spent 1200 to 2400 cycles a tile on it
// (its code is fetched anew each time, the softmax warps' having displaced it),
// against the 2780 that the tile's bytes take.  So four producer warps share a
// tile, kWarpBlocks blocks each, one lane a block.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace attn {

constexpr int kBlockTokens = 16;
constexpr int kTileBlocks = 8;  // of 16 tokens
constexpr int kWarpBlocks = 4;  // of a tile, or of a pair of tiles, per producer warp

template <int D>
struct PagedTile {
  static constexpr uint32_t kHalf = 1024;              // next 64 columns
  static constexpr uint32_t kGroup = D / 64 * 1024;    // next 8 rows
  static constexpr uint32_t kBlock = 2 * kGroup;       // next 16 rows
};

// byte offset of 16-byte chunk ch of row r, halves and 8-row groups `half` and
// `group` bytes apart
__device__ __forceinline__ uint32_t swizzled_off(int r, int ch, uint32_t half, uint32_t group) {
  return static_cast<uint32_t>(r >> 3) * group + static_cast<uint32_t>(ch >> 3) * half +
         static_cast<uint32_t>((r & 7) * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

// The block `id` (negative: not loaded) to block place `i` of the tile.
template <int D>
__device__ __forceinline__ void load_block(uint8_t* tile, int i, const void* map, uint64_t* bar, int id, int Hkv,
                                           int g) {
  if (id >= 0) tma_load_5d(tile + i * PagedTile<D>::kBlock, map, bar, 0, 0, 0, 0, id * Hkv + g);
}

}  // namespace attn
