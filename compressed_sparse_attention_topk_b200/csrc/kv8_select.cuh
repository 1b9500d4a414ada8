// Blocks of the 8-bit cache chosen for each token by a cheap score: the dot
// of the token's int8 group query with each block's sum of key codes
// (contract of csa2_kv8_select in include/csa2.h).
#pragma once

#include "kv8_cache.cuh"

namespace csa2 {
namespace kv8 {

struct SelectParams {
  Cache c;
  Steps s;
  const uint16_t *q;
  int64_t q_stride;
  int32_t G;       // query heads per kv head
  int32_t n_sel, n_first, n_last;
  int32_t *sel;    // [n, Hk, n_sel]
  float *scores;   // [n, Hk, width]
};

constexpr int kSelectThreads = 256;

// One CTA per token and kv head.
__global__ void __launch_bounds__(kSelectThreads) kv8_select_kernel(const SelectParams p) {
  __shared__ int8_t s_q[128];
  __shared__ float s_red[8];
  __shared__ uint32_t s_hist[256], s_scan[33], s_pick[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int D = p.c.D;
  const int h = blockIdx.y;
  for (int64_t i = blockIdx.x; i < p.s.n; i += gridDim.x) {
    const int b = seq_of(p.s, i);
    if (b < 0) return;  // only padding from here on
    const int64_t pos = (int64_t)p.s.lens[b] - p.s.cu[b + 1] + i;
    const int nblk = pos < 0 ? 0 : (int)min64((pos >> p.c.bs_shift) + 1, p.s.width);
    // the group's query, in 8 bits
    float qs = 0.f;
    if (tid < D) {
      double sum = 0.0;
      for (int g = 0; g < p.G; ++g)
        sum += (double)bf16_to_f32_bits(p.q[i * p.q_stride + (int64_t)(h * p.G + g) * D + tid]);
      qs = (float)sum;
    }
    const float wm = warp_max(fabsf(qs) == fabsf(qs) ? fabsf(qs) : INFINITY);
    if (lane == 0) s_red[warp] = wm;
    __syncthreads();
    float big = 0.f;
    for (int w = 0; w < 8; ++w) big = fmaxf(big, s_red[w]);
    const bool dead = !(big > 0.f && big < INFINITY);
    if (tid < D)
      s_q[tid] = dead ? (int8_t)0 : (int8_t)__float2int_rn(__fmul_rn(qs, __fdiv_rn(127.f, big)));
    __syncthreads();
    // scores
    float *row = p.scores + (i * p.c.Hk + h) * p.s.width;
    const int first = min(p.n_first, nblk);
    const int last = max(first, nblk - p.n_last);  // candidates: [first, last)
    for (int j = first + tid; j < last; j += kSelectThreads) {
      const int32_t page = p.s.table[(int64_t)b * p.s.width + j];
      float sc = -INFINITY;
      if (page < 0 || page >= p.c.pages) {
        raise_status(kStatusBadIndex);
      } else {
        const int64_t ph = (int64_t)page * p.c.Hk + h;
        const int16_t *ks = p.c.k_sum + ph * D;
        int dot = 0;
        for (int d = 0; d < D; ++d) dot += (int)s_q[d] * ks[d];
        sc = __fadd_rn(__fmul_rn((float)dot, p.c.k_scale[ph]), 0.f);
      }
      row[j] = sc;
    }
    __syncthreads();
    // the want-th largest candidate by radix selection, 8 bits at a time
    const int want = min(p.n_sel - (first + nblk - last), last - first);
    uint32_t prefix = 0u, need = (uint32_t)want;
    for (int shift = 24; shift >= 0 && want > 0; shift -= 8) {
      s_hist[tid] = 0u;
      __syncthreads();
      for (int j = first + tid; j < last; j += kSelectThreads) {
        const uint32_t k = score_key(row[j]);
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
          atomicAdd(&s_hist[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      radix_threshold<kSelectThreads, 256>(s_hist, need, s_scan, s_pick);
      prefix |= s_pick[0] << shift;
      need -= s_pick[1];
      __syncthreads();
    }
    // kept blocks in ascending order: candidates above the threshold, and the
    // lowest `need` of those at it
    int32_t *out = p.sel + (i * p.c.Hk + h) * p.n_sel;
    uint32_t at = 0u, ties = 0u;
    for (int j0 = 0; j0 < nblk; j0 += kSelectThreads) {
      const int j = j0 + tid;
      uint32_t keep = 0u, tie = 0u;
      if (j < nblk) {
        if (j < first || j >= last) {
          keep = 1u;
        } else if (want > 0) {
          const uint32_t k = score_key(row[j]);
          keep = k > prefix ? 1u : 0u;
          tie = k == prefix ? 1u : 0u;
        }
      }
      uint32_t total;
      const uint32_t before = block_excl_scan<kSelectThreads>(tie, s_scan, total);
      if (tie && ties + before < need) keep = 1u;
      ties += total;
      const uint32_t o = block_excl_scan<kSelectThreads>(keep, s_scan, total);
      if (keep && at + o < (uint32_t)p.n_sel) out[at + o] = j;
      at += total;
    }
    for (uint32_t o = at + tid; o < (uint32_t)p.n_sel; o += kSelectThreads) out[o] = -1;
    __syncthreads();
  }
}

}  // namespace kv8
}  // namespace csa2
