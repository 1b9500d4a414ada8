// Blocks of the 8-bit cache chosen for each token by a cheap score: the dot
// of the token's int8 group query with each block's sum of key codes
// (contract of csa2_kv8_select in include/csa2.h).
//
// Two launches.  kv8_score_kernel forms every score a token sees,
//   score_j = fl(sum_d q8[d] ksum_j[d]) * k_scale_j,
// exactly: the int16 sums are 256 hi + lo with hi int8 and lo uint8, so a dot
// is two exact int8 products on the tensor cores (mma.sync m16n8k32, 16
// blocks x 8 tokens), 256 times the first plus the second (< 2^28).  A
// sequence's sums (2 D bytes per block and head) are read once per 8 or 32
// tokens; bound by those bytes for a few tokens, by the scores' own traffic
// for a chunk.  kv8_pick_*_kernel then takes each row's n_sel best: a score is
// ordered as an unsigned key, forced blocks get the largest key, and the
// n_sel-th largest key is found by bisection within a warp (rows of up to
// 2,048 blocks) or by digits over a CTA.  Four tokens over 4,096 blocks are
// bound by latency (11 and 11 us, 17 MB).  4,096 tokens over 1,024 blocks and 4
// heads move 67 MB of scores to L2 and back beside 18 MB of sums (42 and 42 us;
// instructions issue in 43 and 72 % of the cycles): that traffic is this cut's,
// not the operator's, whose own bytes take 3 us.
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

constexpr int kScoreThreads = 256;
constexpr int kScoreWarps = kScoreThreads / 32;

// Blocks that position pos sees in a table of `width` blocks.
__device__ __forceinline__ int seen_blocks(int64_t pos, int shift, int width) {
  return pos < 0 ? 0 : (int)min64((pos >> shift) + 1, width);
}

// grid (token tiles, kv heads, splits of the blocks).  Tiles of 8 R tokens of
// one sequence: with f(b) = cu[b] / (8 R) + b, tiles f(b) .. f(b + 1) - 1
// belong to sequence b (enough for its tokens; a last one may be empty).
template <int D, int R>
__global__ void __launch_bounds__(kScoreThreads, 2) kv8_score_kernel(const SelectParams p) {
  constexpr int TT = 8 * R;
  static_assert(TT == kScoreWarps * R, "R tokens per warp");
  constexpr int KS = D / 32;       // k-steps
  constexpr int LD = D + 32;       // bytes per token of q8: its reads meet no bank twice
  __shared__ __align__(16) int8_t s_q[TT][LD];
  __shared__ int s_b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int h = blockIdx.y;
  pdl_allow_dependents();
  if (tid == 0) s_b = -1;
  __syncthreads();
  for (int b = tid; b < p.s.B; b += kScoreThreads) {
    const int lo = p.s.cu[b] / TT + b, hi = p.s.cu[b + 1] / TT + b + 1;
    if (lo <= (int)blockIdx.x && (int)blockIdx.x < hi) s_b = b;
  }
  __syncthreads();
  const int b = s_b;
  if (b < 0) return;
  const int cu0 = max(p.s.cu[b], 0), cu1 = p.s.cu[b + 1];
  const int64_t T = min64(cu1, p.s.n) - cu0;
  const int64_t x0 = (int64_t)((int)blockIdx.x - (cu0 / TT + b)) * TT;  // first token
  if (x0 < 0 || x0 >= T) return;
  const int count = (int)min64(TT, T - x0);
  const int64_t tok0 = cu0 + x0;
  const int64_t pos_last = (int64_t)p.s.lens[b] - cu1 + tok0 + count - 1;
  const int nblk = seen_blocks(pos_last, p.c.bs_shift, p.s.width);
  if (tid == 0 && blockIdx.y == 0 && blockIdx.z == 0 && pos_last >> p.c.bs_shift >= p.s.width)
    raise_status(kStatusBadIndex);  // (blocks past the table's width)
  const int groups = (nblk + 15) / 16;
  const int stride = kScoreWarps * gridDim.z;
  int gi = blockIdx.z * kScoreWarps + warp;

  // this thread's two blocks of group gi: their page and head, or -1
  int ph[2];
  auto pages = [&](int grp) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int j = grp * 16 + g + 8 * e;
      ph[e] = -1;
      if (j < nblk) {
        const int page = p.s.table[(int64_t)b * p.s.width + j];
        if (page >= 0 && page < p.c.pages) ph[e] = page * p.c.Hk + h;
        else raise_status(kStatusBadIndex);
      }
    }
  };
  uint4 x[2][KS];
  float ks[2];
  auto load = [&]() {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      ks[e] = ph[e] >= 0 ? p.c.k_scale[ph[e]] : 0.f;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        x[e][s] = make_uint4(0u, 0u, 0u, 0u);
        if (ph[e] >= 0)
          x[e][s] = *reinterpret_cast<const uint4 *>(p.c.k_sum + (int64_t)ph[e] * D +
                                                     (4 * s + t) * 8);
      }
    }
  };
  if (gi < groups) {
    pages(gi);
    load();
  }

  // ---- the tokens' group queries in 8 bits: R tokens per warp, their heads'
  // loads in flight together, four heads at a time ----
  constexpr int E = D / 32;  // dims per lane
  double sum[R][E];
#pragma unroll
  for (int x = 0; x < R; ++x)
#pragma unroll
    for (int e = 0; e < E; ++e) sum[x][e] = 0.0;
  for (int k0 = 0; k0 < p.G; k0 += 4) {
    uint32_t w[R][4][E / 2];
#pragma unroll
    for (int x = 0; x < R; ++x) {
      const int i = warp + x * kScoreWarps;
      const uint16_t *src =
          p.q + (tok0 + i) * p.q_stride + ((int64_t)h * p.G + k0) * D + lane * E;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool in = i < count && k0 + k < p.G;
        if constexpr (D == 128) {
          const uint2 y = in ? *reinterpret_cast<const uint2 *>(src + k * D) : make_uint2(0u, 0u);
          w[x][k][0] = y.x;
          w[x][k][E / 2 - 1] = y.y;
        } else {
          w[x][k][0] = in ? *reinterpret_cast<const uint32_t *>(src + k * D) : 0u;
        }
      }
    }
#pragma unroll
    for (int x = 0; x < R; ++x)
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          sum[x][2 * e] += (double)__uint_as_float(w[x][k][e] << 16);
          sum[x][2 * e + 1] += (double)__uint_as_float(w[x][k][e] & 0xffff0000u);
        }
  }
#pragma unroll
  for (int x = 0; x < R; ++x) {
    const int i = warp + x * kScoreWarps;
    float qs[E];
    float big = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      qs[e] = (float)sum[x][e];
      const float a = fabsf(qs[e]);
      big = fmaxf(big, a == a ? a : INFINITY);
    }
    big = warp_max(big);
    const bool dead = !(big > 0.f && big < INFINITY);
    const float r = dead ? 0.f : __fdiv_rn(127.f, big);
    uint32_t word = 0u;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int q8 = dead ? 0 : __float2int_rn(__fmul_rn(qs[e], r));
      word |= (uint32_t)(uint8_t)(int8_t)q8 << (8 * e);
    }
    if constexpr (D == 128) *reinterpret_cast<uint32_t *>(&s_q[i][lane * 4]) = word;
    else *reinterpret_cast<uint16_t *>(&s_q[i][lane * 2]) = (uint16_t)word;
  }
  __syncthreads();
  uint32_t qb[R][KS][2];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const uint2 y = *reinterpret_cast<const uint2 *>(&s_q[r * 8 + g][(4 * s + t) * 8]);
      qb[r][s][0] = y.x;
      qb[r][s][1] = y.y;
    }

  // ---- 16 blocks at a time; this thread's tokens are 2 t, 2 t + 1 of each 8 ----
  const int row_step = p.c.Hk * p.s.width;  // < 2^23 floats from token to token
  const int mine = count - 2 * t;           // r * 8 + e < mine: it is one of the tile's
  float *const rows = p.scores + ((tok0 + 2 * t) * p.c.Hk + h) * p.s.width;
  for (; gi < groups; gi += stride) {
    int32_t acc[R][4];  // 256 times the high bytes' dots, then the low bytes' on top
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[r][e] = 0;
#pragma unroll
    for (int low = 0; low < 2; ++low) {
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        // bytes of dims 0..3 (first word) and 4..7 of the thread's 8
        const uint32_t pick = low ? 0x6420u : 0x7531u;
        const uint32_t a[4] = {__byte_perm(x[0][s].x, x[0][s].y, pick),
                               __byte_perm(x[1][s].x, x[1][s].y, pick),
                               __byte_perm(x[0][s].z, x[0][s].w, pick),
                               __byte_perm(x[1][s].z, x[1][s].w, pick)};
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if (low) mma_i8<true>(acc[r], a, qb[r][s][0], qb[r][s][1]);
          else mma_i8<false>(acc[r], a, qb[r][s][0], qb[r][s][1]);
        }
      }
      if (!low) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[r][e] *= 256;
      }
    }
    const int j0 = gi * 16 + g;
    const float k0 = ks[0], k1 = ks[1];
    const bool bad0 = ph[0] < 0, bad1 = ph[1] < 0;
    if (gi + stride < groups) {
      pages(gi + stride);
      load();
    }
    float *at = rows + j0;
#pragma unroll
    for (int half = 0; half < 2; ++half, at += 8) {
      if (j0 + 8 * half >= nblk) break;
      const float kk = half ? k1 : k0;
      const bool bad = half ? bad1 : bad0;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float sc = __fadd_rn(__fmul_rn((float)acc[r][half * 2 + e], kk), 0.f);
          if (r * 8 + e < mine) at[(r * 8 + e) * row_step] = bad ? -INFINITY : sc;
        }
    }
  }
}

// ---------------------------------------------------------------------------
// The n_sel best of a row.
// ---------------------------------------------------------------------------
// Key of block j of nblk: 0 when there is none, the largest for a block that
// is always kept.
__device__ __forceinline__ uint32_t pick_key(const SelectParams &p, const float *row, int j,
                                             int nblk) {
  if (j >= nblk) return 0u;
  if (j < p.n_first || j >= nblk - p.n_last) return 0xffffffffu;
  return max(score_key(row[j]), 1u);
}

// One warp per row of up to 32 K blocks.  Where at most 32 are wanted the
// smallest of the lanes' largest keys is a bound that at least 32 keys reach:
// only those keys (some 130 of 1,024 in a random order) are listed, in block
// order, and searched.
constexpr int kPickWarps = 4;

template <int K>
__global__ void __launch_bounds__(32 * kPickWarps) kv8_pick_warp_kernel(const SelectParams p) {
  __shared__ uint32_t s_key[kPickWarps][32 * K];
  __shared__ uint16_t s_block[kPickWarps][32 * K];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t item = (int64_t)blockIdx.x * kPickWarps + warp;
  const int64_t i = item / p.c.Hk;
  if (i >= p.s.n) return;
  const int b = seq_of(p.s, i, lane);
  if (b < 0) {
    pdl_wait_primary();  // (or this launch, and what follows it, could overtake the scores')
    return;
  }
  const int64_t pos = (int64_t)p.s.lens[b] - p.s.cu[b + 1] + i;
  const int nblk = seen_blocks(pos, p.c.bs_shift, p.s.width);
  int32_t *out = p.sel + item * p.n_sel;
  const int first = min(p.n_first, nblk), last = max(first, nblk - p.n_last);
  const int want = min(p.n_sel - (first + nblk - last), last - first);
  pdl_wait_primary();
  if (want == last - first) {  // all of them
    for (int o = lane; o < p.n_sel; o += 32) out[o] = o < nblk ? o : -1;
    return;
  }
  const float *row = p.scores + item * p.s.width;
  uint32_t key[K];
  uint32_t top = 0u;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int j = k * 32 + lane;
    key[k] = j >= first && j < last ? max(score_key(row[j]), 1u) : 0u;
    top = max(top, key[k]);
  }
  // lo: at least `want` keys reach it; hi: fewer do
  uint32_t lo = want <= 32 ? max(__reduce_min_sync(0xffffffffu, top), 1u) : 1u;
  uint64_t hi = (uint64_t)__reduce_max_sync(0xffffffffu, top) + 1;
  uint32_t *keys = s_key[warp];
  uint16_t *blocks = s_block[warp];
  const uint32_t lt = lanemask_lt_u32();
  int n = 0;  // listed
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const bool in = key[k] >= lo;
    const uint32_t who = __ballot_sync(0xffffffffu, in);
    if (in) {
      const int at = n + __popc(who & lt);
      keys[at] = key[k];
      blocks[at] = (uint16_t)(k * 32 + lane);
    }
    n += __popc(who);
  }
  __syncwarp();
  uint32_t above = 0u;  // keys that reach hi
  bool ties = n != want;
  while (ties && hi - lo > 1) {
    const uint32_t mid = (uint32_t)((lo + hi) >> 1);
    uint32_t reach = 0;
    for (int x = lane; x < n; x += 32) reach += keys[x] >= mid ? 1u : 0u;
    reach = __reduce_add_sync(0xffffffffu, reach);
    if (reach >= (uint32_t)want) {
      lo = mid;
      ties = reach != (uint32_t)want;
    } else {
      hi = mid;
      above = reach;
    }
  }
  // kept: keys that reach lo, of those that equal it the lowest blocks only
  uint32_t left = ties ? (uint32_t)want - above : 0xffffffffu;
  int at = first;
  for (int x0 = 0; x0 < n; x0 += 32) {
    const uint32_t k = x0 + lane < n ? keys[x0 + lane] : 0u;
    bool keep = k >= lo;
    if (ties) {
      const uint32_t who = __ballot_sync(0xffffffffu, k == lo);
      if (k == lo) keep = (uint32_t)__popc(who & lt) < left;
      left -= min(left, (uint32_t)__popc(who));
    }
    const uint32_t kept = __ballot_sync(0xffffffffu, keep);
    if (keep) out[at + __popc(kept & lt)] = blocks[x0 + lane];
    at += __popc(kept);
  }
  for (int o = lane; o < first; o += 32) out[o] = o;
  for (int o = lane; o < nblk - last; o += 32) out[at + o] = last + o;
}

// One CTA per row: the threshold by three digits (11, 11 and 10 bits), each
// from a histogram of the keys that share the digits so far.
constexpr int kPickThreads = 512;

__global__ void __launch_bounds__(kPickThreads) kv8_pick_cta_kernel(const SelectParams p,
                                                                   int staged) {
  extern __shared__ uint32_t pick_smem[];  // the row's keys, when they fit
  __shared__ uint32_t s_hist[kBins1], s_scan[33], s_out[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t item = blockIdx.x;
  const int64_t i = item / p.c.Hk;
  const int b = seq_of(p.s, i, lane);
  if (b < 0) {
    pdl_wait_primary();  // (as above)
    return;
  }
  const int64_t pos = (int64_t)p.s.lens[b] - p.s.cu[b + 1] + i;
  const int nblk = seen_blocks(pos, p.c.bs_shift, p.s.width);
  for (int k = tid; k < kBins1; k += kPickThreads) s_hist[k] = 0u;
  pdl_wait_primary();
  const float *row = p.scores + item * p.s.width;
  int32_t *out = p.sel + item * p.n_sel;
  const int want = min(p.n_sel, nblk);
  __syncthreads();
  for (int j = tid; j < nblk; j += kPickThreads) {
    const uint32_t k = pick_key(p, row, j, nblk);
    if (staged) pick_smem[j] = k;
    atomicAdd(&s_hist[key_d1(k)], 1u);
  }
  __syncthreads();
  auto key = [&](int j) { return staged ? pick_smem[j] : pick_key(p, row, j, nblk); };
  uint32_t need = (uint32_t)want, thr;
  radix_threshold<kPickThreads, kBins1>(s_hist, need, s_scan, s_out);
  thr = s_out[0] << 21;
  need -= s_out[1];
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    const int shift = pass == 0 ? 10 : 0, bins = pass == 0 ? kBins2 : kBins3;
    __syncthreads();
    for (int k = tid; k < bins; k += kPickThreads) s_hist[k] = 0u;
    __syncthreads();
    const int above = pass == 0 ? 21 : 10;
    for (int j = tid; j < nblk; j += kPickThreads) {
      const uint32_t k = key(j);
      if (k >> above == thr >> above) atomicAdd(&s_hist[(k >> shift) & (bins - 1)], 1u);
    }
    __syncthreads();
    if (pass == 0) radix_threshold<kPickThreads, kBins2>(s_hist, need, s_scan, s_out);
    else radix_threshold<kPickThreads, kBins3>(s_hist, need, s_scan, s_out);
    thr |= s_out[0] << shift;
    need -= s_out[1];
  }
  // each warp takes a run of blocks; one scan over the warps' counts of keys
  // above the threshold and at it, then every warp writes its own
  const int run = (((nblk + kPickThreads - 1) / kPickThreads)) * 32;
  const int j0 = warp * run, j1 = min(nblk, j0 + run);
  uint32_t n_gt = 0u, n_eq = 0u;
  for (int j = j0 + lane; j < j1; j += 32) {
    const uint32_t k = key(j);
    n_gt += k > thr ? 1u : 0u;
    n_eq += k == thr ? 1u : 0u;
  }
  n_gt = __reduce_add_sync(0xffffffffu, n_gt);
  n_eq = __reduce_add_sync(0xffffffffu, n_eq);
  __syncthreads();
  if (lane == 0) {
    s_hist[warp] = n_gt;
    s_hist[64 + warp] = n_eq;
  }
  __syncthreads();
  uint32_t at = 0u, eq = 0u;  // kept and equal ones before this warp's run
  for (int w = 0; w < warp; ++w) {
    at += s_hist[w];
    eq += s_hist[64 + w];
  }
  at += min(eq, need);
  const uint32_t lt = lanemask_lt_u32();
  for (int base = j0; base < j1; base += 32) {
    const int j = base + lane;
    const uint32_t k = j < j1 ? key(j) : 0u;
    const bool is_eq = j < j1 && k == thr;
    const uint32_t who = __ballot_sync(0xffffffffu, is_eq);
    const bool keep = (j < j1 && k > thr) || (is_eq && eq + __popc(who & lt) < need);
    const uint32_t kept = __ballot_sync(0xffffffffu, keep);
    if (keep) out[at + __popc(kept & lt)] = j;
    at += __popc(kept);
    eq += __popc(who);
  }
  for (int o = want + tid; o < p.n_sel; o += kPickThreads) out[o] = -1;
}

}  // namespace kv8
}  // namespace csa2
