// Attention over the 8-bit paged cache (contract of csa2_kv8_attn in
// include/csa2.h).
#pragma once

#include "kv8_cache.cuh"

namespace csa2 {
namespace kv8 {

struct AttnParams {
  Cache c;
  Steps s;
  const uint16_t *q;
  int64_t q_stride;
  int32_t G;            // query heads per kv head
  const int32_t *sel;   // [n, Hk, n_sel] or null: every block
  int32_t n_sel;
  float sm_scale;
  uint16_t *out;        // [n, H, D]
  float *lse;           // [n, H] or null
};

// One warp per token and query head; a lane holds D / 32 dims.  One pass over
// the keys with the running maximum and sum of the softmax in fp32.
template <int D>
__global__ void __launch_bounds__(128) kv8_attn_kernel(const AttnParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t H = (int64_t)p.G * p.c.Hk;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int64_t i = item / H;
  const int head = (int)(item - i * H), h = head / p.G;
  if (i >= p.s.n) return;
  const int b = seq_of(p.s, i);
  if (b < 0) return;
  const int64_t pos = (int64_t)p.s.lens[b] - p.s.cu[b + 1] + i;
  float q[E], o[E];
  for (int e = 0; e < E; ++e) {
    q[e] = bf16_to_f32_bits(p.q[i * p.q_stride + (int64_t)head * D + lane * E + e]);
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int64_t nblk = pos < 0 ? 0 : (pos >> p.c.bs_shift) + 1;
  const int64_t count = p.sel ? p.n_sel : nblk;
  for (int64_t x = 0; x < count; ++x) {
    const int64_t j = p.sel ? p.sel[(i * p.c.Hk + h) * p.n_sel + x] : x;
    if (j < 0 || j >= nblk) continue;
    const int32_t page = j < p.s.width ? p.s.table[(int64_t)b * p.s.width + j] : -1;
    if (page < 0 || page >= p.c.pages) {
      if (lane == 0) raise_status(kStatusBadIndex);
      continue;
    }
    const int64_t ph = (int64_t)page * p.c.Hk + h;
    const float ks = p.c.k_scale[ph] * p.sm_scale, vs = p.c.v_scale[ph];
    const int rows = (int)min64(p.c.bs, pos + 1 - (j << p.c.bs_shift));
    for (int r = 0; r < rows; ++r) {
      const int64_t at = ((ph << p.c.bs_shift) + r) * D + lane * E;
      float dot = 0.f;
      for (int e = 0; e < E; ++e) dot += q[e] * (float)p.c.k[at + e];
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
      const float y = dot * ks;
      const float mn = fmaxf(m, y);
      const float corr = m == mn ? 1.f : expf(m - mn), w = expf(y - mn);
      m = mn;
      l = l * corr + w;
      for (int e = 0; e < E; ++e) o[e] = o[e] * corr + w * vs * (float)p.c.v[at + e];
    }
  }
  for (int e = 0; e < E; ++e) {
    const float y = l == 0.f ? 0.f : o[e] / l;
    p.out[(i * H + head) * D + lane * E + e] = __bfloat16_as_ushort(__float2bfloat16(y));
  }
  if (lane == 0 && p.lse) p.lse[i * H + head] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace kv8
}  // namespace csa2
