// How a latent prefill's query block cuts its keys into parts, and which (sequence, head)
// units' blocks are launched together.
#pragma once

namespace da {

constexpr int kPrefillPartTiles = 4;  // a block has a part for every 4 key tiles begun, at most

// Parts of a block that sees `tiles` key tiles in a launch of `parts` CTAs a block: by the block's own
// tiles, so that the cache's capacity has no say in it; never more than the launch has.
__host__ __device__ constexpr int prefill_block_parts(int tiles, int parts) {
  const int most = tiles / kPrefillPartTiles + (tiles % kPrefillPartTiles != 0);
  return most < 1 || parts < 2 ? 1 : most < parts ? most : parts;
}

// The first of its tiles in part i, of nparts nearly equal ones.
__host__ __device__ constexpr int prefill_part_begin(int tiles, int i, int nparts) {
  return (int)((long long)tiles * i / nparts);
}

// Units of a launch group: as many as have their K and V, of the longest sequence's tokens, in about
// 96 MB of L2 together.
__host__ __device__ constexpr int prefill_group(int longest, int D, long long units) {
  const long long g = (96LL << 20) / (4LL * D * (longest < 1 ? 1 : longest));
  return (int)(g < 1 ? 1 : g < units ? g : units);
}

}  // namespace da
