// Attention over the 8-bit paged cache (contract of csa2_kv8_attn in
// include/csa2.h).
//
// Mathematics, per query row (token, head) and page with scales ks, vs:
//   x_j = (sm_scale log2(e) ks) <q, kcode_j>,  p_j = 2^(x_j - m),
//   out = sum_j p_j vs vcode_j / sum_j p_j,   lse = ln 2 (m + log2 sum_j p_j)
// in one pass over the keys with the running maximum m.  The codes are exact
// in fp16, and so is q once its row is scaled by a power of two: its largest
// magnitude goes to [1, 2), and an element less than 2^-17 of that is off by at
// most 2^-25 of it (half the last place of an fp16 subnormal).  So the products
// are exact and their sums fp32.  m follows the running maximum only when that has grown by more
// than kSlack, which one vote of the warp finds out; so a row's maximum is
// seldom reduced and its output seldom rescaled.  The weights are rounded once
// to fp16, 2^10 at m: 2^-11 of each weight, and weights down to 2^-34 of the
// largest are not lost.  Sums of weights and outputs stay in fp32; a page's
// scale multiplies its fp32 partial output, so scales far apart lose nothing.
#pragma once

#include <cuda.h>

#include "kv8_cache.cuh"
#include "kv8_steps.cuh"

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
  float *part;          // split tiles: partial results, two per CTA
  int4 *rec;            // split tiles: one record per CTA
  int32_t split_rows;   // > 0: sequences of more rows are kv8_chunk_kernel's, the others
                        // kv8_split_kernel's; 0: the kernel serves them all
};

__device__ __forceinline__ void tma_load_rows(void *smem, const CUtensorMap *map, int row,
                                              uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3, %4}], [%5];" ::"r"(smem_u32(smem)),
      "l"(map), "r"(0), "r"(row), "r"(0), "r"(smem_u32(bar))
      : "memory");
}

// Bounded wait whose polls may suspend the warp, leaving its issue slots to
// the others of the SM: ~2^32 cycles at most, then recorded (bit 1).
__device__ __forceinline__ bool mbar_wait_suspended(uint64_t *bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long start = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - start > (1ll << 32)) {
      raise_status(kStatusWaitTimeout);
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, "
      "%9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The first product of a sum.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, "
      "%9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A word whose bytes 0 and 2 are codes -> two fp16 codes: one three-input
// logic operation, (w & 0x00ff00ff) ^ 0x64806480, makes 1024 + (code + 128) of
// each, less 1152.  `flip` is that second constant in a register that the
// compiler cannot see through: with both as immediates it takes two operations.
constexpr uint32_t kFlip = 0x64806480u;
__device__ __forceinline__ uint32_t codes_f16(uint32_t w, uint32_t flip) {
  uint32_t u;
  asm("lop3.b32 %0, %1, 0x00ff00ff, %2, 0x6a;" : "=r"(u) : "r"(w), "r"(flip));
  const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&u), bias);
  return *reinterpret_cast<const uint32_t *>(&r);
}

// 8 x 8 transpose of 16-bit elements over the warp (row lane / 4, columns
// 2 (lane % 4) and the next).
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 r = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&r);
}

// ---------------------------------------------------------------------------
// Few query rows per sequence (decode, drafts) or a list of blocks per token:
// the work is the stream of the cache's bytes.
//
// A tile is 4, 8, 16, 24 or 32 query rows (token-major, the group's heads
// inside) of one sequence and kv head; its keys are cut into units of 32
// positions.  The
// units of all tiles form one line, cut evenly over the CTAs (lengths differ
// by orders of magnitude between sequences), so a CTA works on the end of a
// tile, whole tiles and the beginning of one; a tile that several CTAs share
// leaves a partial (z, l, O) per CTA, merged in order by kv8_merge_kernel.
// Within a CTA the warps take a tile's units in turn, each with its own ring
// of units (TMA, one lane), its own softmax state and no barrier until the
// tile's end: the 8-bit codes become fp16 fragments in registers, and the
// products are mma.sync m16n8k16 with the cache as the 16-row operand and the
// query rows as the 8 columns, S^T = K Q^T and O^T = V^T P^T (so 4 or 8 query
// heads do not pay for 16, and P^T is an 8 x 8 transpose of S^T).  The tensor
// work is a fraction of the time the bytes take; a 128-row tcgen05 tile would
// be mostly padding.
//
// Beside the bytes it is the instructions around the products that bound it
// (717 of a warp per unit of 8 KB at D = 128 and 8 rows, half of them the
// codes' conversion): 28 decode tokens of 8 heads over 1.26 GB take 205 us
// (6.1 TB/s) and the merge 8.  A tile of at most 4 rows therefore takes its
// logits in whole numbers: a query row is scaled to 30 bits and split into four
// signed bytes d3 .. d0, the columns of a product hold d3 and d2 of row t side
// by side, those of a second product d1 and d0, and 2^24 d3 + 2^16 d2 + 2^8 d1
// + d0 is the dot with the codes themselves, without their conversion (q is off
// by at most 2^-29 of its row's largest magnitude).  A thread then has one row,
// so the softmax and the outputs' arithmetic halve too: 585 instructions (lists
// of 32 blocks for 1,024 tokens of 4 heads 305 -> 268 us).
// ---------------------------------------------------------------------------
constexpr int kSplitWarps = 4;
constexpr int kSplitThreads = 32 * kSplitWarps;
constexpr int kUnit = 32;
constexpr int kNoPos = 1 << 30;  // a table reaches fewer positions; no row sees this one
constexpr float kPBias = 10.f, kSlack = 5.f;  // weights are at most 2^(10 + 5) < 65504

template <int D, int ROWS>
struct SplitShape {
  static constexpr int CTAS = ROWS <= 8 ? 3 : 2;          // per SM
  static constexpr int STAGES = (ROWS <= 8 ? 2 : 3) * (128 / D);
  static constexpr int TILE = kUnit * D;                  // bytes of a unit's keys (or values)
  static constexpr int RING = STAGES * 2 * TILE;          // per warp
  static constexpr int LDO = D + 4;                       // floats per row of a warp's result
  static constexpr size_t SMEM = size_t(kSplitWarps) * RING + 1024;
  static constexpr size_t PART = size_t(ROWS) * (D + 2);  // floats of one partial
  static_assert(ROWS * LDO * 4 <= RING, "a warp's result reuses its ring");
};

// A tile: rows row0 .. row0 + nrows - 1 (row = token of the sequence * G +
// head of the group).
struct Tile {
  int32_t b, h, row0, nrows, tok0;
  int32_t pos0;      // position of the sequence's first new token
  int32_t pos_first, pos_last;  // positions of the tile's first and last row
  int32_t units;
};

// Work of sequence b: tiles per kv head and units per tile.
template <int ROWS>
__device__ __forceinline__ void seq_work(const AttnParams &p, int b, int &tiles, int &units,
                                         int &t0, int &T, int &pos0) {
  const int32_t lo = max(p.s.cu[b], 0), hi = p.s.cu[b + 1];
  t0 = lo;
  T = (int)max((int64_t)0, min64(hi, p.s.n) - lo);
  const int64_t len = p.s.lens[b];
  pos0 = (int)max((int64_t)-0x40000000, len - hi + lo);
  const int64_t rows = (int64_t)T * p.G;
  tiles = p.split_rows && rows > p.split_rows ? 0 : (int)((rows + ROWS - 1) / ROWS);
  const int64_t reach = (int64_t)p.s.width << p.c.bs_shift;
  const int64_t seen = min64(max(len, (int64_t)0), reach);
  units = max(1, (int)((seen + kUnit - 1) / kUnit));
}

template <int D, int ROWS, bool P16>
__global__ void __launch_bounds__(kSplitThreads, SplitShape<D, ROWS>::CTAS)
    kv8_split_kernel(const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const AttnParams p) {
  using S = SplitShape<D, ROWS>;
  constexpr bool QUAD = ROWS == 4;
  constexpr int R8 = QUAD ? 1 : ROWS / 8;  // groups of 8 columns
  constexpr int EC = QUAD ? 1 : 2;         // rows of a group that a thread has
  constexpr int DT = D / 16;   // k-steps of a dot; 16-dim tiles of the output
  constexpr int kStages = S::STAGES;
  extern __shared__ unsigned char split_smem[];
  __shared__ uint64_t s_bar[kSplitWarps][kStages];
  __shared__ float s_z[kSplitWarps][ROWS], s_l[kSplitWarps][ROWS];
  __shared__ long long s_sum[kSplitWarps], s_tiles[kSplitWarps];
  __shared__ long long s_pre;
  __shared__ int s_b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  unsigned char *const ring0 = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(split_smem) + 1023) & ~uintptr_t(1023));
  unsigned char *const ring = ring0 + warp * S::RING;
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&s_bar[warp][i], 1);
    fence_barrier_init();
  }
  pdl_allow_dependents();
  uint32_t flip;
  asm volatile("mov.b32 %0, %1;" : "=r"(flip) : "n"(kFlip));

  // ---- the line of units: its length, and this CTA's stretch of it ----
  long long W, u0, u1, n_tiles = 0;
  int b = 0;            // first tile's sequence (dense)
  long long pre = 0;    // units before sequence b
  const int xt = (p.G + ROWS - 1) / ROWS;  // tiles of a (token, kv head) with a list
  const int list_units = P16 ? (p.n_sel + 1) / 2 : p.n_sel << (p.c.bs_shift - 5);
  if (p.sel) {
    const int64_t tokens = min64(p.s.n, p.s.cu[p.s.B]);
    n_tiles = max((long long)tokens, 0ll) * p.c.Hk * xt;
    W = n_tiles * list_units;
  } else {
    long long mine = 0, count = 0;
    for (int i = tid; i < p.s.B; i += kSplitThreads) {
      int tiles, units, t0, T, pos0;
      seq_work<ROWS>(p, i, tiles, units, t0, T, pos0);
      mine += (long long)tiles * units;
      count += tiles;
      if (tiles > 0 && blockIdx.x == 0 &&
          (int64_t)p.s.lens[i] > ((int64_t)p.s.width << p.c.bs_shift))
        raise_status(kStatusBadIndex);
    }
    mine = warp_sum64(mine);
    count = warp_sum64(count);
    if (lane == 0) {
      s_sum[warp] = mine;
      s_tiles[warp] = count;
    }
    __syncthreads();
    W = 0;
    for (int w = 0; w < kSplitWarps; ++w) {
      W += s_sum[w];
      n_tiles += s_tiles[w];
    }
    W *= p.c.Hk;
    n_tiles *= p.c.Hk;
  }
  // as many CTAs as there are, but no tile in pieces of fewer units than two
  // for each warp (every piece is a partial to merge)
  const long long ctas =
      max(1ll, min((long long)gridDim.x, max(n_tiles, W / (2 * kSplitWarps))));
  const long long c = blockIdx.x;
  u0 = c < ctas ? W * c / ctas : W;
  u1 = c < ctas ? W * (c + 1) / ctas : W;
  if (p.sel && W > 0 && n_tiles * 2 <= gridDim.x) {
    // few lists, all as long: the same number of CTAs for each, so that none
    // works on two
    const long long each = min((long long)gridDim.x / n_tiles,
                               max(1ll, (long long)list_units / (2 * kSplitWarps)));
    u0 = u1 = W;
    if (c < n_tiles * each) {
      u0 = c / each * list_units + list_units * (c % each) / each;
      u1 = c / each * list_units + list_units * (c % each + 1) / each;
    }
  }
  if (u0 >= u1) {
    if (tid == 0) p.rec[c] = make_int4(-1, 0, 0, 0);
    return;
  }
  if (!p.sel) {  // the sequence that holds unit u0
    long long before = 0;
    for (int i0 = 0; i0 < p.s.B; i0 += kSplitThreads) {
      const int i = i0 + tid;
      long long w = 0;
      if (i < p.s.B) {
        int tiles, units, t0, T, pos0;
        seq_work<ROWS>(p, i, tiles, units, t0, T, pos0);
        w = (long long)tiles * units * p.c.Hk;
      }
      const long long incl = warp_incl_scan64(w);
      __syncthreads();
      if (lane == 31) s_sum[warp] = incl;
      __syncthreads();
      long long base = before;
      for (int k = 0; k < kSplitWarps; ++k) {
        if (k < warp) base += s_sum[k];
        before += s_sum[k];
      }
      const long long lo = base + incl - w;
      if (w > 0 && lo <= u0 && u0 < lo + w) {
        s_b = i;
        s_pre = lo;
      }
      if (before > u0) break;  // uniform
    }
    __syncthreads();
    b = s_b;
    pre = s_pre;
  }

  int n_issued = 0;     // units issued by this warp so far, in two rounds of the ring
  bool broken = false;  // a copy did not arrive: this warp reads no more
  int4 rec = make_int4(-1, 0, 0, 0);
  for (long long u = u0; u < u1;) {
    // ---- the tile that holds unit u ----
    Tile tl;
    long long tile_begin;
    int64_t list_at = 0;
    if (p.sel) {
      const long long idx = u / list_units;
      tile_begin = idx * list_units;
      const int x = (int)(idx % xt);
      const long long th = idx / xt;
      const int64_t tok = th / p.c.Hk;
      tl.h = (int)(th - tok * p.c.Hk);
      tl.b = max(seq_of(p.s, tok, lane), 0);
      tl.tok0 = (int)tok;
      tl.pos0 = (int)max((int64_t)-0x40000000,
                         (int64_t)p.s.lens[tl.b] - p.s.cu[tl.b + 1] + tok);
      tl.row0 = x * ROWS;
      tl.nrows = min(ROWS, p.G - tl.row0);
      tl.units = list_units;
      list_at = (tok * p.c.Hk + tl.h) * p.n_sel;
    } else {
      int tiles, units, t0, T, pos0;
      seq_work<ROWS>(p, b, tiles, units, t0, T, pos0);
      while (u - pre >= (long long)tiles * units * p.c.Hk) {
        pre += (long long)tiles * units * p.c.Hk;
        ++b;
        seq_work<ROWS>(p, b, tiles, units, t0, T, pos0);
      }
      const long long idx = (u - pre) / units;
      tile_begin = pre + idx * units;
      const int x = (int)(idx / p.c.Hk);
      tl.b = b;
      tl.h = (int)(idx - (long long)x * p.c.Hk);
      tl.row0 = x * ROWS;
      tl.nrows = min(ROWS, T * p.G - tl.row0);
      tl.tok0 = t0;
      tl.pos0 = pos0;
      tl.units = units;
    }
    // (at most as a row's own position below: a missing page's, kNoPos, is past it)
    tl.pos_first = min(tl.pos0 + tl.row0 / p.G, kNoPos - 1);
    tl.pos_last = tl.pos0 + (tl.row0 + tl.nrows - 1) / p.G;
    const int first = (int)(u - tile_begin);
    const int last = (int)min(u1 - tile_begin, (long long)tl.units);  // units [first, last)

    // ---- query rows.  Thread (g, t) holds dims 64 hh + 16 t + 4 w + 0 .. 3
    // for k-step 4 hh + w, as the cache's words below: of row g of each group
    // of 8, power-of-two scaled fp16 (0, 2 | 1, 3); or (QUAD) of row g / 2,
    // bytes: of the upper two the higher (g even) or the lower, and of the
    // lower two ----
    uint32_t qb[R8][DT][2];
    float fac[R8][EC];     // of the thread's rows: the columns of S^T and O^T
    int row_pos[R8][EC];
#pragma unroll
    for (int q8 = 0; q8 < R8; ++q8) {
      const int R = tl.row0 + min(QUAD ? g >> 1 : q8 * 8 + g, tl.nrows - 1);
      const int tok = R / p.G;
      const uint16_t *src = p.q + (int64_t)(tl.tok0 + tok) * p.q_stride +
                            (int64_t)(tl.h * p.G + R - tok * p.G) * D;
      float big = 0.f;
      bool finite = true;
#pragma unroll
      for (int hh = 0; hh < D / 64; ++hh) {
        const uint4 a = *reinterpret_cast<const uint4 *>(src + 64 * hh + 16 * t);
        const uint4 c4 = *reinterpret_cast<const uint4 *>(src + 64 * hh + 16 * t + 8);
        const uint32_t ws[8] = {a.x, a.y, a.z, a.w, c4.x, c4.y, c4.z, c4.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x0 = fabsf(__uint_as_float(ws[e] << 16));
          const float x1 = fabsf(__uint_as_float(ws[e] & 0xffff0000u));
          qb[q8][hh * 4 + e / 2][e & 1] = ws[e];
          big = fmaxf(big, fmaxf(x0, x1));
          finite &= x0 < INFINITY && x1 < INFINITY;
        }
      }
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // 2^-e with 2^e <= big < 2^(e+1), kept normal; 1 for zero or infinity
      const uint32_t eb = __float_as_uint(big) >> 23;
      const uint32_t sb =
          min((big > 0.f && eb < 255u) ? max(254u - eb, 1u) : 127u, 253u);
      const float down = __uint_as_float(sb << 23);
      float f = p.sm_scale * 1.44269504088896340736f * __uint_as_float((254u - sb) << 23);
      if constexpr (QUAD) {
        f *= 0x1p-28f;  // the digits are of 2^28 times the scaled value
        // bytes carry no NaN or infinity: the row's scale does
        const uint32_t who = __ballot_sync(0xffffffffu, finite);
        if ((who >> (lane & 28) & 15u) != 15u) f = __int_as_float(0x7fffffff);
      }
      const int pos = min(tl.pos0 + tok, kNoPos - 1);
#pragma unroll
      for (int e = 0; e < EC; ++e) {
        fac[q8][e] = __shfl_sync(0xffffffffu, f, (2 * t + e) * 4);
        row_pos[q8][e] = __shfl_sync(0xffffffffu, pos, (2 * t + e) * 4);
      }
#pragma unroll
      for (int s = 0; s < DT; ++s) {
        const uint32_t w0 = qb[q8][s][0], w1 = qb[q8][s][1];  // dims 0, 1 and 2, 3
        if constexpr (QUAD) {
          const float y[4] = {__uint_as_float(w0 << 16), __uint_as_float(w0 & 0xffff0000u),
                              __uint_as_float(w1 << 16), __uint_as_float(w1 & 0xffff0000u)};
          uint32_t upper = 0u, low = 0u;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int d0123 = __float2int_rn(y[e] * down * 0x1p28f);  // |.| <= 2^30
            const int d0 = (int8_t)d0123, d123 = (d0123 - d0) >> 8;
            const int d1 = (int8_t)d123, d23 = (d123 - d1) >> 8;
            const int d2 = (int8_t)d23, d3 = (d23 - d2) >> 8;         // |d3| <= 64
            upper |= (uint32_t)(uint8_t)(g & 1 ? d2 : d3) << (8 * e);
            low |= (uint32_t)(uint8_t)(g & 1 ? d0 : d1) << (8 * e);
          }
          qb[q8][s][0] = upper;
          qb[q8][s][1] = low;
        } else {
          qb[q8][s][0] =
              pack_f16(__uint_as_float(w0 << 16) * down, __uint_as_float(w1 << 16) * down);
          qb[q8][s][1] = pack_f16(__uint_as_float(w0 & 0xffff0000u) * down,
                                  __uint_as_float(w1 & 0xffff0000u) * down);
        }
      }
    }

    // ---- state: weights are 2^(x - z); one above 2^lim moves z (any does
    // where z is not set yet) ----
    float o[R8][DT][2 * EC], lim[R8][EC], z[R8][EC], l[R8][EC];
#pragma unroll
    for (int q8 = 0; q8 < R8; ++q8) {
#pragma unroll
      for (int j = 0; j < DT; ++j)
#pragma unroll
        for (int e = 0; e < 2 * EC; ++e) o[q8][j][e] = 0.f;
#pragma unroll
      for (int e = 0; e < EC; ++e) {
        lim[q8][e] = -INFINITY;
        z[q8][e] = l[q8][e] = 0.f;
      }
    }

    // ---- this warp's units: first + warp, + kSplitWarps, ... ----
    const int mine = last - first > warp ? (last - first - warp + kSplitWarps - 1) / kSplitWarps : 0;
    // What a lane knows of unit 32 k + lane of this warp: the row of its keys
    // in the cache (-1: nothing to do), its first position and its scales.
    // With 16-token pages a unit is two pages.
    struct Meta {
      int row[P16 ? 2 : 1], pos[P16 ? 2 : 1];
      float ks[P16 ? 2 : 1], vs[P16 ? 2 : 1];
    } cur, nxt;
    auto load_meta = [&](Meta &M, int k) {
      const int i = k * 32 + lane;  // of this warp
      const int un = first + warp + i * kSplitWarps;
#pragma unroll
      for (int e = 0; e < (P16 ? 2 : 1); ++e) {
        M.row[e] = -1;
        M.pos[e] = kNoPos;
        M.ks[e] = M.vs[e] = 0.f;
        if (i >= mine) continue;
        int j, sub = 0;
        if (p.sel) {
          const int at = P16 ? 2 * un + e : un >> (p.c.bs_shift - 5);
          if (!P16) sub = un & ((p.c.bs >> 5) - 1);
          j = at < p.n_sel ? p.sel[list_at + at] : -1;
        } else {
          j = P16 ? 2 * un + e : un >> (p.c.bs_shift - 5);
          if (!P16) sub = un & ((p.c.bs >> 5) - 1);
        }
        if (j < 0 || (int64_t)j << p.c.bs_shift > tl.pos_last) continue;
        const int pos = (j << p.c.bs_shift) + sub * kUnit;
        if (pos > tl.pos_last) continue;
        const int page = j < p.s.width ? p.s.table[(int64_t)tl.b * p.s.width + j] : -1;
        if (page < 0 || page >= p.c.pages) {
          raise_status(kStatusBadIndex);
          continue;
        }
        const int ph = page * p.c.Hk + tl.h;
        M.row[e] = (ph << p.c.bs_shift) + sub * kUnit;
        M.pos[e] = pos;
        M.ks[e] = p.c.k_scale[ph];
        M.vs[e] = p.c.v_scale[ph];
      }
    };
    load_meta(cur, 0);
    load_meta(nxt, 1);
    int group = 0;      // cur holds units 32 group .. of this warp
    const int base = n_issued;
    auto issue = [&](int i) {  // unit i of this warp into its stage
      int row[P16 ? 2 : 1];
#pragma unroll
      for (int e = 0; e < (P16 ? 2 : 1); ++e) {
        const int rc = __shfl_sync(0xffffffffu, cur.row[e], i & 31);
        const int rn = __shfl_sync(0xffffffffu, nxt.row[e], i & 31);
        row[e] = (i >> 5) == group ? rc : rn;
      }
      if (lane == 0) {
        const int st = (base + i) % kStages;
        unsigned char *kt = ring + st * 2 * S::TILE, *vt = kt + S::TILE;
        uint64_t *bar = &s_bar[warp][st];
        if (!P16) {
          mbar_arrive_expect_tx(bar, row[0] >= 0 ? 2 * S::TILE : 0);
          if (row[0] >= 0) {
            tma_load_rows(kt, &kmap, row[0], bar);
            tma_load_rows(vt, &vmap, row[0], bar);
          }
        } else {
          mbar_arrive_expect_tx(bar, ((row[0] >= 0) + (row[P16 ? 1 : 0] >= 0)) * S::TILE);
#pragma unroll
          for (int e = 0; e < (P16 ? 2 : 1); ++e)
            if (row[e] >= 0) {
              tma_load_rows(kt + e * (S::TILE / 2), &kmap, row[e], bar);
              tma_load_rows(vt + e * (S::TILE / 2), &vmap, row[e], bar);
            }
        }
      }
    };
    for (int i = 0; i < (broken ? 0 : min(mine, kStages)); ++i) issue(i);

    for (int i = 0; i < (broken ? 0 : mine); ++i) {
      if ((i >> 5) != group) {
        cur = nxt;
        ++group;
        load_meta(nxt, group + 1);
      }
      const int st = (base + i) % kStages;
      const bool landed =
          mbar_wait_suspended(&s_bar[warp][st], (uint32_t)((base + i) / kStages) & 1u);
      if (!__all_sync(0xffffffffu, landed)) {
        // given up: no more copies, and those under way get the same chance
        for (int k = i + 1; k < min(mine, i + kStages); ++k)
          mbar_wait_suspended(&s_bar[warp][(base + k) % kStages],
                              (uint32_t)((base + k) / kStages) & 1u);
        broken = true;
        break;
      }
      float ks[2], vs[2];
      int pos[2];
      bool any = false;
#pragma unroll
      for (int e = 0; e < (P16 ? 2 : 1); ++e) {
        ks[e] = __shfl_sync(0xffffffffu, cur.ks[e], i & 31);
        vs[e] = __shfl_sync(0xffffffffu, cur.vs[e], i & 31);
        pos[e] = __shfl_sync(0xffffffffu, cur.pos[e], i & 31);
        any |= pos[e] != kNoPos;
      }
      if (!P16) {
        ks[1] = ks[0];
        vs[1] = vs[0];
        pos[1] = pos[0] + 16;
      }
      if (any) {
        const unsigned char *kt = ring + st * 2 * S::TILE, *vt = kt + S::TILE;
        // ---- S^T = K Q^T: 16 positions per row tile ----
        float sc[R8][2][2 * EC];  // [..][16 positions][position g, g + 8][row]
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int r = k * 16 + g;  // and r + 8: the same place in the swizzle
          float dot[R8][4];
          int32_t upper[4] = {0, 0, 0, 0}, low[4] = {0, 0, 0, 0};
#pragma unroll
          for (int hh = 0; hh < D / 64; ++hh) {
            const int chunk = D == 128 ? ((t + 4 * hh) ^ g) : (t ^ ((g >> 1) & 3));
            const uint4 x = *reinterpret_cast<const uint4 *>(kt + r * D + chunk * 16);
            const uint4 y = *reinterpret_cast<const uint4 *>(kt + (r + 8) * D + chunk * 16);
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
            if constexpr (QUAD) {
#pragma unroll
              for (int w = 0; w < 4; w += 2) {
                const uint32_t a[4] = {xs[w], ys[w], xs[w + 1], ys[w + 1]};
                mma_i8<false>(upper, a, qb[0][hh * 4 + w][0], qb[0][hh * 4 + w + 1][0]);
                mma_i8<false>(low, a, qb[0][hh * 4 + w][1], qb[0][hh * 4 + w + 1][1]);
              }
            } else {
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const uint32_t a[4] = {codes_f16(xs[w], flip), codes_f16(ys[w], flip),
                                       codes_f16(xs[w] >> 8, flip), codes_f16(ys[w] >> 8, flip)};
#pragma unroll
                for (int q8 = 0; q8 < R8; ++q8) {
                  if (hh == 0 && w == 0)
                    mma_f16_first(dot[q8], a, qb[q8][0][0], qb[q8][0][1]);
                  else
                    mma_f16(dot[q8], a, qb[q8][hh * 4 + w][0], qb[q8][hh * 4 + w][1]);
                }
              }
            }
          }
          // x - z, a thread's positions g, g + 8 and rows (2 t, 2 t + 1 of each
          // group, or t)
#pragma unroll
          for (int q8 = 0; q8 < R8; ++q8)
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
              for (int e = 0; e < EC; ++e) {
                float x;
                if constexpr (QUAD)  // 2^8 d3 + d2 < 2^29, 2^8 d1 + d0 < 2^30
                  x = fmaf((float)(upper[2 * half] * 256 + upper[2 * half + 1]), 65536.f,
                           (float)(low[2 * half] * 256 + low[2 * half + 1]));
                else
                  x = dot[q8][half * 2 + e];
                sc[q8][k][half * EC + e] = fmaf(x, fac[q8][e] * ks[k], -z[q8][e]);
              }
        }
        // ---- softmax ----
        if (max(pos[0], pos[1]) + 15 > tl.pos_first) {  // not seen whole by every row
#pragma unroll
          for (int q8 = 0; q8 < R8; ++q8)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int e = 0; e < 2 * EC; ++e)
                if (pos[k] + g + (e / EC) * 8 > row_pos[q8][e % EC]) sc[q8][k][e] = -INFINITY;
        }
        float top[R8][EC];
        bool move = false;
#pragma unroll
        for (int q8 = 0; q8 < R8; ++q8)
#pragma unroll
          for (int e = 0; e < EC; ++e) {
            top[q8][e] = fmaxf(fmaxf(sc[q8][0][e], sc[q8][0][EC + e]),
                               fmaxf(sc[q8][1][e], sc[q8][1][EC + e]));
            move |= top[q8][e] > lim[q8][e];
          }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int q8 = 0; q8 < R8; ++q8) {
            float corr[EC];
#pragma unroll
            for (int e = 0; e < EC; ++e) {
              float mx = top[q8][e];
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
              corr[e] = 1.f;
              if (mx > lim[q8][e]) {
                const float to = z[q8][e] + (mx - kPBias), by = to - z[q8][e];
                if (lim[q8][e] > 0.f) corr[e] = ex2(-by);  // (else there are no weights yet)
                z[q8][e] = to;
                lim[q8][e] = kPBias + kSlack;
                l[q8][e] *= corr[e];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  sc[q8][k][e] -= by;
                  sc[q8][k][EC + e] -= by;
                }
              }
            }
#pragma unroll
            for (int j = 0; j < DT; ++j)
#pragma unroll
              for (int e = 0; e < 2 * EC; ++e) o[q8][j][e] *= corr[e % EC];
          }
        }
        // weights; QUAD: row t in column 2 t, zeros beside it
        uint32_t pb[R8][2][2];
#pragma unroll
        for (int q8 = 0; q8 < R8; ++q8) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int e = 0; e < 2 * EC; ++e) sc[q8][k][e] = ex2(sc[q8][k][e]);
#pragma unroll
            for (int half = 0; half < 2; ++half)
              pb[q8][k][half] = transpose_8x8(
                  pack_f16(sc[q8][k][half * EC], QUAD ? 0.f : sc[q8][k][half * EC + EC - 1]));
          }
#pragma unroll
          for (int e = 0; e < EC; ++e)
            l[q8][e] += (sc[q8][0][e] + sc[q8][0][EC + e]) + (sc[q8][1][e] + sc[q8][1][EC + e]);
        }
        // ---- O^T += vs * V^T P^T: rows g and g + 8 of 16-dim tile j are
        // dims g DT 2 + j and + DT + j, so a thread's bytes of a token are
        // consecutive ----
        uint32_t vw[2][4][D / 32];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            const int r = k * 16 + 2 * t + (i4 & 1) + (i4 >> 1) * 8;
            if constexpr (D == 128) {
              const uint4 x = *reinterpret_cast<const uint4 *>(vt + r * D + ((g ^ (r & 7)) * 16));
              vw[k][i4][0] = x.x;
              vw[k][i4][1] = x.y;
              vw[k][i4][2] = x.z;
              vw[k][i4][3] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2 *>(
                  vt + r * D + (((g >> 1) ^ ((r >> 1) & 3)) * 16) + (g & 1) * 8);
              vw[k][i4][0] = x.x;
              vw[k][i4][1] = x.y;
            }
          }
#pragma unroll
        for (int j = 0; j < DT; ++j) {
          // byte j % 4 of words j / 4 (dim row g) and j / 4 + D / 64 (row g + 8)
          const int lo = j / 4, hi = lo + D / 64;
          const uint32_t pick = (uint32_t)((4 + j % 4) << 8 | j % 4);
          float part[R8][4];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t a[4] = {
                codes_f16(__byte_perm(vw[k][0][lo], vw[k][1][lo], pick), flip),
                codes_f16(__byte_perm(vw[k][0][hi], vw[k][1][hi], pick), flip),
                codes_f16(__byte_perm(vw[k][2][lo], vw[k][3][lo], pick), flip),
                codes_f16(__byte_perm(vw[k][2][hi], vw[k][3][hi], pick), flip)};
#pragma unroll
            for (int q8 = 0; q8 < R8; ++q8) {
              if (P16 || k == 0)
                mma_f16_first(part[q8], a, pb[q8][k][0], pb[q8][k][1]);
              else
                mma_f16(part[q8], a, pb[q8][k][0], pb[q8][k][1]);
            }
            if (P16 || k == 1) {
#pragma unroll
              for (int q8 = 0; q8 < R8; ++q8)
#pragma unroll
                for (int e = 0; e < 2 * EC; ++e)
                  o[q8][j][e] = fmaf(vs[k], part[q8][(e / EC) * 2 + e % EC], o[q8][j][e]);
            }
          }
        }
      }
      __syncwarp();
      if (i + kStages < mine) issue(i + kStages);
    }
    n_issued = ring_after(base, mine, kStages);

    // ---- the warps' results into their rings, then merged ----
    float *res = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int q8 = 0; q8 < R8; ++q8)
#pragma unroll
      for (int e = 0; e < EC; ++e) {
        float sum = l[q8][e];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int r = QUAD ? t : q8 * 8 + 2 * t + e;
        if (g == 0) {
          s_z[warp][r] = sum == 0.f ? -INFINITY : z[q8][e];
          s_l[warp][r] = sum;
        }
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int j = 0; j < DT; j += 4)
            *reinterpret_cast<float4 *>(res + r * S::LDO + (2 * g + half) * DT + j) = make_float4(
                o[q8][j][half * EC + e], o[q8][j + 1][half * EC + e],
                o[q8][j + 2][half * EC + e], o[q8][j + 3][half * EC + e]);
      }
    __syncthreads();
    const bool whole = first == 0 && last == tl.units;
    const int slot = first > 0 ? 0 : 1;  // the end of a tile, or its beginning
    float *part = p.part + (2 * c + slot) * S::PART;
    for (int item = tid; item < tl.nrows * (D / 4); item += kSplitThreads) {
      const int r = item / (D / 4), d = (item % (D / 4)) * 4;
      float mx = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kSplitWarps; ++w) mx = fmaxf(mx, s_z[w][r]);
      const float zero = mx == -INFINITY ? 0.f : mx;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kSplitWarps; ++w) {
        const float f = ex2(s_z[w][r] - zero);
        const float4 x = *reinterpret_cast<const float4 *>(
            reinterpret_cast<float *>(ring0 + w * S::RING) + r * S::LDO + d);
        sum = fmaf(s_l[w][r], f, sum);
        acc.x = fmaf(x.x, f, acc.x);
        acc.y = fmaf(x.y, f, acc.y);
        acc.z = fmaf(x.z, f, acc.z);
        acc.w = fmaf(x.w, f, acc.w);
      }
      if (whole) {
        const int R = tl.row0 + r, tok = R / p.G;
        const int64_t at = (int64_t)(tl.tok0 + tok) * (p.G * p.c.Hk) + tl.h * p.G + R - tok * p.G;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        uint2 w2;
        w2.x = (uint32_t)__bfloat16_as_ushort(__float2bfloat16(acc.x * inv)) |
               ((uint32_t)__bfloat16_as_ushort(__float2bfloat16(acc.y * inv)) << 16);
        w2.y = (uint32_t)__bfloat16_as_ushort(__float2bfloat16(acc.z * inv)) |
               ((uint32_t)__bfloat16_as_ushort(__float2bfloat16(acc.w * inv)) << 16);
        *reinterpret_cast<uint2 *>(p.out + at * D + d) = w2;
        if (d == 0 && p.lse)
          p.lse[at] = sum == 0.f ? -INFINITY
                                 : fmaf(zero, 0.693147180559945309417f, logf(sum));
      } else {
        *reinterpret_cast<float4 *>(part + r * D + d) = acc;
        if (d == 0) {
          part[ROWS * D + r] = mx;
          part[ROWS * D + ROWS + r] = sum;
        }
      }
    }
    if (!whole) {
      if (first > 0) {
        rec.z = last == tl.units;          // this CTA ends a tile begun earlier
      } else {                             // it begins one that later CTAs end
        const int R = tl.row0;
        rec.x = tl.tok0;
        rec.y = tl.h | (tl.nrows << 8);
        rec.w = R;
      }
    }
    fence_proxy_async_smem();  // the rings are written by TMA again
    __syncthreads();
    u = tile_begin + last;
  }
  if (tid == 0) p.rec[c] = rec;
}

// ---------------------------------------------------------------------------
// Tiles of ROWS query rows that several CTAs shared (of kv8_split_kernel, or
// of kv8_chunk_kernel): block (c, y) merges rows RPB y .. of the tile that CTA
// c begins and later CTAs end, in CTA order.  RPB 32: a warp takes a row at a
// time (a chunk's 256 rows, of few partials each).  RPB 4 and 1: the block's
// warps share a row's partials, eight, four or two to a row, as many rows as
// the block has; RPB 1 where so few tiles share the CTAs that a row can have
// hundreds of partials.
// ---------------------------------------------------------------------------
constexpr int kMergeThreads = 256;

template <int D, int ROWS, int RPB>
__global__ void __launch_bounds__(kMergeThreads) kv8_merge_kernel(const AttnParams p, int ctas) {
  constexpr size_t PART = size_t(ROWS) * (D + 2);
  constexpr int E = D / 32;
  __shared__ float s_o[8][D], s_ml[8][2];
  const int c = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait_primary();
  const int4 rec = p.rec[c];
  const int nrows = rec.y >> 8;
  if (rec.x < 0 || (int)blockIdx.y * RPB >= nrows) return;
  // the tile's partials: (c, 1), (c + 1, 0), ..., up to the CTA that ends it
  int end = c + 1;
  for (; end < ctas; end += 32) {
    const bool ends = end + lane < ctas && p.rec[end + lane].z;
    const uint32_t who = __ballot_sync(0xffffffffu, ends);
    if (who) {
      end += __ffs(who) - 1;
      break;
    }
  }
  const int count = min(end, ctas - 1) - c + 1;
  const int here = min(RPB, nrows - (int)blockIdx.y * RPB);
  const int wpr = RPB > 4 ? 1 : here == 1 ? 8 : here == 2 ? 4 : 2;  // warps per row
  const int piece = (count + wpr - 1) / wpr;
  const int k0 = (warp % wpr) * piece, k1 = min(count, k0 + piece);
  auto at = [&](int k) { return p.part + (k == 0 ? 2 * c + 1 : 2 * (c + k)) * PART; };
#pragma unroll 1
  for (int r = blockIdx.y * RPB + warp / wpr; r < (int)(blockIdx.y + 1) * RPB; r += 8 / wpr) {
    float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    if (r < nrows) {
      for (int k = k0 + lane; k < k1; k += 32) m = fmaxf(m, at(k)[ROWS * D + r]);
      m = warp_max(m);
      const float zero = m == -INFINITY ? 0.f : m;
#pragma unroll 8
      for (int k = k0; k < k1; ++k) {
        const float *src = at(k);
        const float f = ex2(src[ROWS * D + r] - zero);
        l = fmaf(src[ROWS * D + ROWS + r], f, l);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(src[r * D + lane * E + e], f, o[e]);
      }
    }
    float sum = l, zero = m == -INFINITY ? 0.f : m;
    if constexpr (RPB <= 4) {  // (one turn of the loop: 8 / wpr rows are all there are)
#pragma unroll
      for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
      if (lane == 0) {
        s_ml[warp][0] = m;
        s_ml[warp][1] = l;
      }
      __syncthreads();
      if (warp % wpr) return;
      float mx = m;
      for (int w = 1; w < wpr; ++w) mx = fmaxf(mx, s_ml[warp + w][0]);
      zero = mx == -INFINITY ? 0.f : mx;
      float f = ex2(m - zero);
      sum = l * f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= f;
      for (int w = 1; w < wpr; ++w) {
        f = ex2(s_ml[warp + w][0] - zero);
        sum = fmaf(s_ml[warp + w][1], f, sum);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(s_o[warp + w][lane * E + e], f, o[e]);
      }
    }
    if (r < nrows) {
      const int R = rec.w + r, tok = R / p.G;
      const int64_t row =
          (int64_t)(rec.x + tok) * (p.G * p.c.Hk) + (rec.y & 255) * p.G + R - tok * p.G;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int e = 0; e < E; ++e)
        p.out[row * D + lane * E + e] = __bfloat16_as_ushort(__float2bfloat16(o[e] * inv));
      if (lane == 0 && p.lse)
        p.lse[row] =
            sum == 0.f ? -INFINITY : fmaf(zero, 0.693147180559945309417f, logf(sum));
    }
    if constexpr (RPB <= 4) return;
  }
}

}  // namespace kv8
}  // namespace csa2
