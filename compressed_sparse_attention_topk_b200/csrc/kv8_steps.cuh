// Steps of the many-row attention's line of work (kv8_chunk.cuh).  Host code
// too, so that the counts can be checked as whole numbers at sizes that no
// test attends over.
#pragma once

#include <cstdint>

namespace csa2 {
namespace kv8 {

constexpr int kChunkRows = 256;  // query rows of a tile
constexpr int kChunkKeys = 64;   // positions of a step

// A sequence's new tokens, the position of the first, its tiles per kv head,
// and the positions that its table holds.
struct ChunkSeq {
  int t0, T, pos0, tiles, reach;
};

// Steps of tile x, at most 2^30 / 64: its keys end at its last row's position.
// (A sequence has fewer than 2^31 rows, but its last tile may end at 2^31.)
__host__ __device__ inline int chunk_steps(const ChunkSeq &s, int G, int x) {
  const long long end = ((long long)x + 1) * kChunkRows, all = (long long)s.T * G;
  const int at = s.pos0 + ((int)((end < all ? end : all) - 1)) / G;
  const int last = at < s.reach - 1 ? at : s.reach - 1;
  return last < 0 ? 1 : last / kChunkKeys + 1;
}

// Steps of the tiles x0, x0 + stride, ... of a sequence and kv head: some
// rows * positions / (256 * 64) over all of them, which passes 2^31.
__host__ __device__ inline long long chunk_steps_of(const ChunkSeq &s, int G, int x0, int stride) {
  long long steps = 0;
  for (int x = x0; x < s.tiles; x += stride) steps += chunk_steps(s, G, x);
  return steps;
}

}  // namespace kv8
}  // namespace csa2
