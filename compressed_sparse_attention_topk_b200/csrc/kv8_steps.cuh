// Counts of the attention kernels' work: steps of the many-row attention's
// line (kv8_chunk.cuh), uses of a ring of buffers.  Host code too, so that
// they can be checked as whole numbers at sizes that no test attends over.
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

// The n-th use of a ring of SLOTS buffers: which one, and the parity of the
// barrier phase that this use completes.  A block may use a ring more than
// 2^32 times: the count then wraps, which a power of two of slots does not
// notice.  (Waiting for the phase before the first, parity 1 of a barrier just
// made, is answered at once.)
template <int SLOTS>
__host__ __device__ inline int ring_slot(uint32_t n) {
  static_assert((SLOTS & (SLOTS - 1)) == 0, "a wrapped count must stay in step");
  return (int)(n % SLOTS);
}
template <int SLOTS>
__host__ __device__ inline uint32_t ring_parity(uint32_t n) {
  return (n / SLOTS) & 1u;
}

// A ring of any number of slots: the count after `used` (at most 2^26) more
// uses, kept below two rounds, which leaves slot and parity as they are.
__host__ __device__ inline int ring_after(int n, int used, int slots) {
  return (n + used) % (2 * slots);
}

}  // namespace kv8
}  // namespace csa2
