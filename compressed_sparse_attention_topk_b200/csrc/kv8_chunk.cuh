// Attention over the 8-bit paged cache for many query rows per sequence (a
// prompt or a chunk of one): the mathematics of kv8_attn.cuh on the
// 5th-generation tensor cores.
//
// A CTA holds 256 query rows (token-major, the group's heads inside) of one
// sequence and kv head as two 128-row tiles, and passes over its keys 64 at a
// time.  Per step and tile: S = Q K^T (tcgen05, fp16 x fp16 -> fp32 in TMEM),
// one thread per row takes the softmax (its 64 logits in registers) and
// leaves the weights in TMEM over S, O += P V (the weights as the TMEM
// operand).  Six further warps turn the codes into fp16 tiles in shared
// memory, up to four steps ahead, once for both row tiles.  S is double
// buffered, so the products of the next step run while a tile's rows are in
// the softmax.
//
// The products are exact (codes and power-of-two scaled queries are fp16),
// sums fp32.  A page's value scale joins its logits instead of its values:
//   y_j = x_j + log2(vs / vref),  P_j = 2^(y_j - m),  m >= max y - kSlack,
// so P_j vcode_j vref is p_j vs vcode_j in the row's own units; the softmax
// sum takes P_j (vref / vs) page by page.  vref is the largest scale of the
// sequence's pages; one below 2^-80 of it counts as 0.  P is rounded
// once to fp16, 2^kPBias at m: 2^-11 of a weight, down to 2^-34 of the
// largest.  m follows the running maximum only when that has grown by more
// than kSlack, so O is rarely rescaled.
//
// Bound: 128 x 128 weights take 1,024 clocks of the exponential unit and
// their two products the same of the tensor core.  2,048 tokens of 16 heads
// over 16,384 positions (4 kv heads, D = 128) take 345 us, 747 TFLOP/s: some
// 2,600 clocks for a step of both row tiles, which is the chain of one tile's
// step (logits, maximum, weights, product) rather than any unit.
#pragma once

#include "kv8_attn.cuh"
#include "tcgen05.cuh"

namespace csa2 {
namespace kv8 {

using namespace tc;

constexpr int kChunkGroups = kChunkKeys / 16;  // no page ends inside 16 positions
constexpr int kChunkSlots = 4;                 // steps of fp16 tiles
constexpr int kSoftWarps = 8;
constexpr int kConvWarps = 6;
constexpr int kMmaWarps = 2;   // one per row tile; 16 warps in all: 128 registers a thread
constexpr int kChunkThreads = 32 * (kSoftWarps + kConvWarps + kMmaWarps);
constexpr int kMetaSlots = 8;
constexpr float kLvsFloor = -80.f;  // log2 of the smallest value scale that counts

template <int D>
struct ChunkShape {
  static constexpr int DH = D / 64;          // 128-byte wide sub-tiles of a row
  static constexpr int QSUB = 128 * 128;     // bytes of a sub-tile of the queries
  static constexpr int SUB = kChunkKeys * 128;  // and of the keys or values
  static constexpr size_t PART = size_t(kChunkRows) * (D + 2);  // floats of one partial
};

// Scales of a step's groups of 16 positions: keys; values as log2(vs / vref)
// and vref / vs; vref.
struct ChunkMeta {
  float ks[kChunkGroups], lvs[kChunkGroups], ivs[kChunkGroups], vref;
};

template <int D>
struct ChunkSmem {
  alignas(1024) uint8_t q[2][ChunkShape<D>::DH * ChunkShape<D>::QSUB];
  alignas(1024) uint8_t k[kChunkSlots][ChunkShape<D>::DH * ChunkShape<D>::SUB];
  alignas(1024) uint8_t v[kChunkSlots][ChunkShape<D>::DH * ChunkShape<D>::SUB];
  ChunkMeta meta[kMetaSlots];
  uint64_t q_full[2], s_full[2][2], p_full[2][2], o_done[2][2];  // [row tile][buffer of S]
  uint64_t k_full[kChunkSlots], k_empty[kChunkSlots], v_full[kChunkSlots], v_empty[kChunkSlots];
  uint64_t meta_full[kMetaSlots], drained;
  uint32_t tmem_base;
  volatile uint32_t abort_flag;
  long long sum[kChunkThreads / 32], tiles[kChunkThreads / 32];
  long long pre;
  int b, h, x, from;
};

template <int D>
constexpr size_t chunk_smem_bytes() {
  return sizeof(ChunkSmem<D>) + 1024 < 120 * 1024 ? 120 * 1024 : sizeof(ChunkSmem<D>) + 1024;
}

// Bounded wait that also gives up once another role has.
template <int D>
__device__ __forceinline__ bool chunk_wait(ChunkSmem<D> &sm, uint64_t *bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long start = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (sm.abort_flag) return false;
    if (clock64() - start > (1ll << 32)) {
      raise_status(kStatusWaitTimeout);
      sm.abort_flag = 1u;
      return false;
    }
  }
  return true;
}

// Operand rows of 128 bytes, 128-byte swizzle, 8-row groups 1,024 bytes apart.
// K-major: a k-step of 16 is 32 bytes on.  MN-major (values: 64 dims of a key
// per row): `lead` bytes to the next 64 dims, 1,024 to the next 8 keys.
__device__ __forceinline__ uint64_t chunk_desc(const void *smem, uint32_t lead) {
  const uint64_t addr = smem_u32(smem);
  return ((addr >> 4) & 0x3FFFull) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}

// One thread of a whole warp, chosen in a way that the compiler knows to be
// one: the operands of the products then live in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// fp16 x fp16 -> fp32, M = 128, N = n; B K-major or MN-major.
__host__ __device__ constexpr uint32_t chunk_idesc(int n, bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(128 >> 4) << 24);
}

__device__ __forceinline__ void umma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The wait that makes loaded TMEM values usable, tied to their registers.
__device__ __forceinline__ void tie(uint32_t (&v)[32]) {
  asm volatile(""
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                 "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                 "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])::"memory");
  asm volatile(""
               : "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]),
                 "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]),
                 "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])::"memory");
}
__device__ __forceinline__ void tmem_landed(uint32_t (&v)[32]) {
  tmem_wait_ld();
  tie(v);
}
__device__ __forceinline__ void tmem_landed(uint32_t (&v)[32], uint32_t (&w)[32]) {
  tmem_wait_ld();
  tie(v);
  tie(w);
}

// Largest of 16 values: three-input maxima.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max16(const uint32_t *v) {
  float m0 = max3(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]));
  float m1 = max3(__uint_as_float(v[3]), __uint_as_float(v[4]), __uint_as_float(v[5]));
#pragma unroll
  for (int j = 6; j < 14; j += 4) {
    m0 = max3(m0, __uint_as_float(v[j]), __uint_as_float(v[j + 1]));
    m1 = max3(m1, __uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]));
  }
  m0 = max3(m0, __uint_as_float(v[14]), __uint_as_float(v[15]));
  return fmaxf(m0, m1);
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Weights of 16 columns of a row: 2^(s fk + add), packed as fp16 into w[0..7];
// returns their sum.
__device__ __forceinline__ float weights16(const uint32_t *v, float fk, float add, uint32_t *w) {
  const uint64_t f2 = pack2(fk, fk), a2 = pack2(add, add);
  uint64_t sum = pack2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    float x0, x1;
    unpack2(fma2(pack2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), f2, a2), x0, x1);
    const float e0 = ex2(x0), e1 = ex2(x1);
    sum = add2(sum, pack2(e0, e1));
    w[j / 2] = pack_f16(e0, e1);
  }
  float s0, s1;
  unpack2(sum, s0, s1);
  return s0 + s1;
}

// 16 columns, landed.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// ---------------------------------------------------------------------------
// The line of steps (a tile's 64-key steps), cut evenly over the CTAs as in
// kv8_attn.cuh (kv8_steps.cuh counts them).
// ---------------------------------------------------------------------------
__device__ __forceinline__ ChunkSeq chunk_seq(const AttnParams &p, int b) {
  ChunkSeq s;
  const int32_t lo = max(p.s.cu[b], 0), hi = p.s.cu[b + 1];
  s.t0 = lo;
  s.T = (int)max((int64_t)0, min64(hi, p.s.n) - lo);
  s.pos0 = (int)max((int64_t)-0x40000000, (int64_t)p.s.lens[b] - hi + lo);
  const int64_t rows = (int64_t)s.T * p.G;
  s.tiles = rows <= p.split_rows ? 0 : (int)((rows + kChunkRows - 1) / kChunkRows);
  s.reach = p.s.width << p.c.bs_shift;
  return s;
}

struct ChunkWalk {
  const AttnParams &p;
  long long u, u1;   // the CTA's stretch from here on
  ChunkSeq s;
  int b, h, x;
  int steps, first, last;  // of the tile; the CTA's steps of it are [first, last)
  int row0, nrows, pos_first, pos_last;

  __device__ ChunkWalk(const AttnParams &p_, long long u0_, long long u1_, int b_, int h_, int x_,
                       int from)
      : p(p_), u(u0_), u1(u1_), s(chunk_seq(p_, b_)), b(b_), h(h_), x(x_) {
    set(from);
  }
  __device__ void set(int from) {
    steps = chunk_steps(s, p.G, x);
    first = from;
    last = (int)min64(steps, from + (u1 - u));
    row0 = x * kChunkRows;
    nrows = min(kChunkRows, s.T * p.G - row0);
    pos_first = s.pos0 + row0 / p.G;
    pos_last = s.pos0 + (row0 + nrows - 1) / p.G;
  }
  __device__ bool next() {
    u += last - first;
    if (u >= u1) return false;
    if (++x >= s.tiles) {
      x = 0;
      if (++h >= p.c.Hk) {
        h = 0;
        do {
          s = chunk_seq(p, ++b);
        } while (s.tiles == 0 && b < p.s.B - 1);
      }
    }
    set(0);
    return true;
  }
};

// The unit of a sequence's values: the largest value scale of its pages (of a
// kv head), found by each converter warp.  lvs is then at most 0, and the
// sums of weights keep fp32's range down to kLvsFloor below it: a weight whose
// P underflows (2^-126) adds less than 2^(-126 + 80) to a sum of at least 2^5.
// (a call: inlined at its places it costs the kernel registers)
__device__ __noinline__ float chunk_top(const int32_t *row, int n, const float *scale, int Hk,
                                        int pages) {
  float top = 0.f;
  for (int j0 = threadIdx.x & 31; j0 < n; j0 += 4 * 32) {
    int page[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) page[e] = j0 + 32 * e < n ? row[j0 + 32 * e] : -1;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float v = page[e] >= 0 && page[e] < pages ? scale[page[e] * Hk] : 0.f;
      top = v < INFINITY ? fmaxf(top, v) : top;
    }
  }
  top = warp_max(top);
  return top > 0.f ? top : 1.f;
}
__device__ __forceinline__ float chunk_vref(const AttnParams &p, int b, int h) {
  const int64_t len = max(p.s.lens[b], 0);
  return chunk_top(p.s.table + (int64_t)b * p.s.width,
                   (int)min64((len + p.c.bs - 1) >> p.c.bs_shift, p.s.width), p.c.v_scale + h,
                   p.c.Hk, p.c.pages);
}

template <int D>
__global__ void __launch_bounds__(kChunkThreads, 1) kv8_chunk_kernel(const AttnParams p) {
  using S = ChunkShape<D>;
  extern __shared__ __align__(1024) unsigned char chunk_smem_raw[];
  ChunkSmem<D> &sm = *reinterpret_cast<ChunkSmem<D> *>(
      (reinterpret_cast<uintptr_t>(chunk_smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kWarps = kChunkThreads / 32;
  pdl_allow_dependents();
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], kSoftWarps / 2);
      for (int k = 0; k < 2; ++k) {
        mbar_init(&sm.s_full[i][k], 1);
        mbar_init(&sm.o_done[i][k], 1);
        mbar_init(&sm.p_full[i][k], kSoftWarps / 2);
      }
    }
    for (int i = 0; i < kChunkSlots; ++i) {
      mbar_init(&sm.k_full[i], kChunkGroups);
      mbar_init(&sm.k_empty[i], kMmaWarps);
      mbar_init(&sm.v_full[i], kChunkGroups);
      mbar_init(&sm.v_empty[i], kMmaWarps);
    }
    for (int i = 0; i < kMetaSlots; ++i) mbar_init(&sm.meta_full[i], kChunkGroups);
    mbar_init(&sm.drained, kMmaWarps);
    sm.abort_flag = 0u;
    sm.b = sm.h = sm.x = sm.from = 0;
    sm.pre = 0;
    fence_barrier_init();
  }
  // ---- this CTA's stretch of the line.  Steps per sequence and kv head first
  // (a warp each, a lane per tile), kept where the queries go later ----
  long long *const per_seq = reinterpret_cast<long long *>(sm.q[0]);
  static_assert(sizeof(sm.q) >= kMaxSeqs * sizeof(long long), "every sequence's steps");
  long long tiles = 0;
  for (int b = warp; b < p.s.B; b += kWarps) {
    const ChunkSeq s = chunk_seq(p, b);
    const long long steps = warp_sum64(chunk_steps_of(s, p.G, lane, 32));
    if (lane == 0) {
      per_seq[b] = steps;
      if (s.tiles > 0 && blockIdx.x == 0 && p.s.lens[b] > s.reach) raise_status(kStatusBadIndex);
    }
    tiles += s.tiles;
  }
  if (lane == 0) sm.tiles[warp] = tiles;
  __syncthreads();
  long long mine = 0;
  for (int b = tid; b < p.s.B; b += kChunkThreads) mine += per_seq[b];
  mine = warp_sum64(mine);
  if (lane == 0) sm.sum[warp] = mine;
  __syncthreads();
  long long W = 0;
  tiles = 0;
  for (int w = 0; w < kWarps; ++w) {
    W += sm.sum[w];
    tiles += sm.tiles[w];
  }
  W *= p.c.Hk;
  // as many CTAs as there are, but no tile in pieces of fewer than 8 steps
  const long long ctas = max(1ll, min((long long)gridDim.x, max(tiles * p.c.Hk, W / 8)));
  const long long c = blockIdx.x;
  const long long u0 = c < ctas ? W * c / ctas : W, u1 = c < ctas ? W * (c + 1) / ctas : W;
  if (u0 >= u1) {
    if (tid == 0) p.rec[c] = make_int4(-1, 0, 0, 0);
    return;
  }
  long long before = 0;
  for (int b0 = 0; b0 < p.s.B; b0 += kChunkThreads) {
    const int b = b0 + tid;
    const long long w = b < p.s.B ? per_seq[b] * p.c.Hk : 0;
    const long long incl = warp_incl_scan64(w);
    __syncthreads();
    if (lane == 31) sm.sum[warp] = incl;
    __syncthreads();
    long long base = before;
    for (int k = 0; k < kWarps; ++k) {
      if (k < warp) base += sm.sum[k];
      before += sm.sum[k];
    }
    const long long lo = base + incl - w;
    if (w > 0 && lo <= u0 && u0 < lo + w) {
      sm.b = b;
      sm.pre = lo;
    }
    if (before > u0) break;  // uniform
  }
  __syncthreads();
  if (warp == 0) {  // its kv head and tile
    const int b = sm.b;
    const ChunkSeq s = chunk_seq(p, b);
    const long long per = max(per_seq[b], 1ll);
    const int h = (int)((u0 - sm.pre) / per);
    long long r = u0 - sm.pre - h * per;  // steps of that head before u0
    for (int x0 = 0; x0 < s.tiles; x0 += 32) {
      const int x = x0 + lane, n = x < s.tiles ? chunk_steps(s, p.G, x) : 0;
      const int incl = (int)warp_incl_scan((uint32_t)n);
      const uint32_t who = __ballot_sync(0xffffffffu, r < incl);
      if (who) {
        if (lane == __ffs(who) - 1) {
          sm.h = h;
          sm.x = x;
          sm.from = (int)r - (incl - n);
        }
        break;
      }
      r -= __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  if (warp == kWarps - 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sm.tmem_base)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  ChunkWalk walk(p, u0, u1, sm.b, sm.h, sm.x, sm.from);

  if (warp < kSoftWarps) {
    // ---------------- softmax: one thread per query row ----------------
    const int tile = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_at = (uint32_t)(quarter * 32) << 16;
    const uint32_t t_o = tmem + lane_at + 256u + (uint32_t)(tile * D);
    uint32_t n_steps = 0;    // of this tile so far: buffers and phases
    uint32_t k_index = 0;    // steps of both tiles so far: slots of the page facts
    int4 rec = make_int4(-1, 0, 0, 0);
    do {
      const bool whole = walk.first == 0 && walk.last == walk.steps;
      if (tile * 128 >= walk.nrows) {  // warp-uniform: no row of this tile
        k_index += (uint32_t)(walk.last - walk.first);
        continue;
      }
      const int r = tile * 128 + row;
      const int R = walk.row0 + min(r, walk.nrows - 1);
      const int tok = R / p.G;
      const int64_t head = (int64_t)walk.h * p.G + R - tok * p.G;
      const int my_pos = min(walk.s.pos0 + tok, kNoPos - 1);
      float f;  // logit per product, without the page's key scale
      {
        const uint4 *src = reinterpret_cast<const uint4 *>(
            p.q + (int64_t)(walk.s.t0 + tok) * p.q_stride + head * D);
        uint4 w[D / 8];
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          w[i] = src[i];
          const uint32_t ws[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            big = fmaxf(big, fabsf(__uint_as_float(ws[e] << 16)));
            big = fmaxf(big, fabsf(__uint_as_float(ws[e] & 0xffff0000u)));
          }
        }
        const uint32_t eb = __float_as_uint(big) >> 23;
        const uint32_t sb = min((big > 0.f && eb < 255u) ? max(254u - eb, 1u) : 127u, 253u);
        f = fabsf(p.sm_scale) * 1.44269504088896340736f * __uint_as_float((254u - sb) << 23);
        const float down = copysignf(__uint_as_float(sb << 23), p.sm_scale);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {  // dims 0, 2, 1, 3 of each 4, as the codes
          uint4 x;
          x.x = pack_f16(__uint_as_float(w[i].x << 16) * down, __uint_as_float(w[i].y << 16) * down);
          x.y = pack_f16(__uint_as_float(w[i].x & 0xffff0000u) * down,
                         __uint_as_float(w[i].y & 0xffff0000u) * down);
          x.z = pack_f16(__uint_as_float(w[i].z << 16) * down, __uint_as_float(w[i].w << 16) * down);
          x.w = pack_f16(__uint_as_float(w[i].z & 0xffff0000u) * down,
                         __uint_as_float(w[i].w & 0xffff0000u) * down);
          *reinterpret_cast<uint4 *>(sm.q[tile] + (i >> 3) * S::QSUB + row * 128 +
                                     (((i & 7) ^ (row & 7)) << 4)) = x;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_full[tile]);

      float m = -INFINITY, l = 0.f;
      for (int t = walk.first; t < walk.last; ++t, ++k_index, ++n_steps) {
        const ChunkMeta &me = sm.meta[ring_slot<kMetaSlots>(k_index)];
        // the products first: once they are there, the page facts of this very
        // step are (a row tile that skipped steps could mistake an older phase)
        const uint32_t buf = n_steps & 1u, phase = (n_steps >> 1) & 1u;
        bool ok = chunk_wait(sm, &sm.s_full[tile][buf], phase);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        const uint32_t t_s = tmem + lane_at + (uint32_t)(tile * 128) + buf * 64u;
        uint32_t a[32], b2[32];
        tmem_ld32(t_s, a);
        tmem_ld32(t_s + 32, b2);
        ok = chunk_wait(sm, &sm.meta_full[ring_slot<kMetaSlots>(k_index)],
                        ring_parity<kMetaSlots>(k_index));
        const int seen = my_pos - t * kChunkKeys;  // columns 0 .. seen are visible
        float fk[4], lv[4];
#pragma unroll
        for (int part = 0; part < 4; ++part) {
          // (never 0: a masked column's -inf must stay one)
          fk[part] = fmaxf(f * me.ks[part], 1e-37f);
          lv[part] = me.lvs[part];
        }
        tmem_landed(a, b2);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (__any_sync(0xffffffffu, seen < kChunkKeys - 1)) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            if (j > seen) a[j] = 0xff800000u;  // -inf
            if (j + 32 > seen) b2[j] = 0xff800000u;
          }
        }
        // ---- the row's maximum ----
        float mx = m;
#pragma unroll
        for (int part = 0; part < 4; ++part)
          mx = fmaxf(mx, fmaf(max16((part & 2 ? b2 : a) + (part & 1) * 16), fk[part], lv[part]));
        // ---- the unit of the weights ----
        float corr = 1.f;
        if (mx > m + kSlack || (m == -INFINITY && mx > -INFINITY)) {
          corr = m == -INFINITY ? 1.f : ex2(m - mx);  // (no weights yet: nothing to rescale)
          m = mx;
        }
        l *= corr;
        if (t > walk.first && __any_sync(0xffffffffu, corr != 1.f)) {
          // the products so far
          ok = chunk_wait(sm, &sm.o_done[tile][buf ^ 1u], ((n_steps - 1) >> 1) & 1u);
          if (!__all_sync(0xffffffffu, ok)) break;
          tc_fence_after();
#pragma unroll 1
          for (int ch = 0; ch < D; ch += 16) {
            uint32_t x[16];
            tmem_ld16(t_o + ch, x);
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * corr);
            tmem_st16(t_o + ch, x);
          }
        }
        // ---- weights over S, sums ----
        const float zero = (m == -INFINITY ? 0.f : m) - kPBias;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int part = half * 2 + e;
            l = fmaf(weights16((half ? b2 : a) + e * 16, fk[part], lv[part] - zero, w + e * 8),
                     me.ivs[part], l);
          }
          tmem_st16(t_s + 16 * half, w);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[tile][buf]);
      }
      // ---- out ----
      // (a barrier per buffer: the products of the step before the last may be
      // under way too, and one barrier's parity cannot tell the two apart)
      bool ok = chunk_wait(sm, &sm.o_done[tile][(n_steps - 1) & 1u], ((n_steps - 1) >> 1) & 1u);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const bool mine_out = r < walk.nrows;
      const int64_t at = (int64_t)(walk.s.t0 + tok) * (p.G * p.c.Hk) + head;
      const float zero = m - kPBias;
      float *part = p.part + (2 * c + (walk.first > 0 ? 0 : 1)) * S::PART;
      // (a partial is kept in units 2^24 larger: O vref stays in range)
      const float vref = sm.meta[ring_slot<kMetaSlots>(k_index - 1)].vref;  // (not yet rewritten)
      const float mul = whole ? (l == 0.f ? 0.f : vref / l) : vref * 0x1p-24f;
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t v[32];
        tmem_ld32(t_o + 32 * ch, v);
        tmem_landed(v);
        if (mine_out) {
          float y[32];
#pragma unroll
          for (int j = 0; j < 32; j += 4) {  // columns 0, 2, 1, 3 of each 4
            y[j] = __uint_as_float(v[j]) * mul;
            y[j + 2] = __uint_as_float(v[j + 1]) * mul;
            y[j + 1] = __uint_as_float(v[j + 2]) * mul;
            y[j + 3] = __uint_as_float(v[j + 3]) * mul;
          }
          if (whole) {
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = (uint32_t)__bfloat16_as_ushort(
                           __float2bfloat16(l == 0.f ? 0.f : y[j + 2 * e])) |
                       ((uint32_t)__bfloat16_as_ushort(
                            __float2bfloat16(l == 0.f ? 0.f : y[j + 2 * e + 1]))
                        << 16);
              *reinterpret_cast<uint4 *>(p.out + at * D + 32 * ch + j) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<float4 *>(part + r * D + 32 * ch + j) =
                  make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
          }
        }
      }
      if (mine_out && whole && p.lse)
        p.lse[at] = l == 0.f ? -INFINITY : fmaf(zero, 0.693147180559945309417f, logf(l));
      if (mine_out && !whole) {
        part[kChunkRows * D + r] = l == 0.f ? -INFINITY : zero + 24.f;
        part[kChunkRows * D + kChunkRows + r] = l * 0x1p-24f;
      }
      if (!whole && tile == 0) {
        if (walk.first > 0) {
          rec.z = walk.last == walk.steps;   // this CTA ends a tile begun earlier
        } else {                             // it begins one that later CTAs end
          rec.x = walk.s.t0;
          rec.y = walk.h | (walk.nrows << 8);
          rec.w = walk.row0;
        }
      }
      tc_fence_before();  // these reads come before the next tile's products
    } while (walk.next());
    if (tid == 0) p.rec[c] = rec;
  } else if (warp < kSoftWarps + kConvWarps) {
    // ---------------- codes -> fp16 tiles ----------------
    // A task is 16 positions of one page, keys or values: eight to a step, keys
    // first, dealt to the warps in turn.  8 consecutive lanes store 2 rows x 4
    // places of a 128-byte line: no two in the same banks under the swizzle.
    constexpr int RPP = D == 128 ? 4 : 8;  // rows per pass
    constexpr int PASSES = 16 / RPP;
    const int piece = D == 128 ? ((lane & 3) | ((lane >> 3) & 1) << 2) : (lane & 3);
    const int sub = D == 128 ? (((lane >> 2) & 1) | ((lane >> 4) & 1) << 1) : (lane >> 2);
    uint32_t flip;
    asm volatile("mov.b32 %0, %1;" : "=r"(flip) : "n"(kFlip));
    uint4 reg[PASSES];
    // Where a step's positions are: their page as the table has it (on the way
    // from one iteration to the next), and what it takes to use it.
    struct Place {
      uint32_t step;       // of the CTA
      int part;            // 0 .. 3 keys, 4 .. 7 values
      int raw, key, h;     // table entry, first position, kv head
      bool seen;           // the entry was read: the positions are seen
      float vref;
    };
    int t = walk.first;
    float vref_now = chunk_vref(p, walk.b, walk.h);
    uint32_t step = 0;  // of the task that `look` is at
    int part = warp - kSoftWarps;
    auto look = [&](Place &at) {
      at.step = step;
      at.part = part;
      at.key = t * kChunkKeys + (part % kChunkGroups) * 16;
      const int j = at.key >> p.c.bs_shift;
      at.h = walk.h;
      at.vref = vref_now;
      at.seen = (int64_t)j << p.c.bs_shift <= walk.pos_last && j < p.s.width;
      at.raw = at.seen ? p.s.table[(int64_t)walk.b * p.s.width + j] : -1;
    };
    auto advance = [&]() {  // to this warp's next task; false: there is none
      part += kConvWarps;
      if (part < 2 * kChunkGroups) return true;
      part -= 2 * kChunkGroups;
      ++step;
      if (++t < walk.last) return true;
      const int b = walk.b, h = walk.h;
      if (!walk.next()) return false;
      t = walk.first;
      if (walk.b != b || walk.h != h) vref_now = chunk_vref(p, walk.b, walk.h);
      return true;
    };
    // page and head, or -1 where nothing is seen or the page is not the cache's
    auto page_head = [&](const Place &at) {
      if (at.raw >= 0 && at.raw < p.c.pages) return at.raw * p.c.Hk + at.h;
      if (at.seen && lane == 0) raise_status(kStatusBadIndex);
      return -1;
    };
    auto load = [&](int ph, const Place &at) {
      const int key = at.key;
      const int8_t *src = (at.part < kChunkGroups ? p.c.k : p.c.v) +
                          (((int64_t)max(ph, 0) << p.c.bs_shift) + (key & (p.c.bs - 1)) + sub) * D +
                          piece * 16;
#pragma unroll
      for (int i = 0; i < PASSES; ++i)
        reg[i] = ph < 0 ? make_uint4(0u, 0u, 0u, 0u)
                        : *reinterpret_cast<const uint4 *>(src + i * RPP * D);
    };
    auto store = [&](uint8_t *tile, int row0, bool zeros) {
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const int r = row0 + i * RPP + sub;
        const uint32_t ws[4] = {reg[i].x, reg[i].y, reg[i].z, reg[i].w};
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[2 * e] = codes_f16(ws[e], flip);
          o[2 * e + 1] = codes_f16(ws[e] >> 8, flip);
        }
        if (zeros) {  // a value scale of 0: whatever the codes are
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = 0u;
        }
        uint8_t *line = tile + (piece >> 2) * S::SUB + r * 128;
        const int at = (((piece & 3) * 2) ^ (r & 7)) << 4;
        *reinterpret_cast<uint4 *>(line + at) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4 *>(line + (at ^ 16)) = make_uint4(o[4], o[5], o[6], o[7]);
      }
    };
    Place here, there;  // of this step and of the next
    look(here);
    int ph = page_head(here);
    bool more = advance();
    if (more) look(there);
    float ks = ph >= 0 ? p.c.k_scale[ph] : 0.f, vs = ph >= 0 ? p.c.v_scale[ph] : 0.f;
    load(ph, here);
    for (;;) {
      const int slot = ring_slot<kChunkSlots>(here.step);
      const int cw = here.part % kChunkGroups;
      const bool vals = here.part >= kChunkGroups;
      if (!chunk_wait(sm, vals ? &sm.v_empty[slot] : &sm.k_empty[slot],
                      ring_parity<kChunkSlots>(here.step) ^ 1u))
        break;
      // (a page without values must not raise the maximum: it takes the floor)
      const bool zero = vs == 0.f || vs < here.vref * 0x1p-80f;
      store(vals ? sm.v[slot] : sm.k[slot], cw * 16, vals && zero);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(vals ? &sm.v_full[slot] : &sm.k_full[slot]);
        if (!vals) {  // (the softmax is never a ring of these behind)
          const int at = ring_slot<kMetaSlots>(here.step);
          sm.meta[at].ks[cw] = ks;
          if (cw == 0) sm.meta[at].vref = here.vref;
          sm.meta[at].lvs[cw] = ph < 0 ? -INFINITY : zero ? kLvsFloor : log2f(vs / here.vref);
          sm.meta[at].ivs[cw] = ph < 0 ? 0.f : zero ? 0x1p80f : here.vref / vs;
          mbar_arrive(&sm.meta_full[at]);
        }
      }
      __syncwarp();
      if (!more) break;
      here = there;
      ph = page_head(here);
      load(ph, here);
      ks = ph >= 0 ? p.c.k_scale[ph] : 0.f;
      vs = ph >= 0 ? p.c.v_scale[ph] : 0.f;
      more = advance();
      if (more) look(there);
    }
  } else if (elect_one()) {
    // ---------------- products: one thread per row tile ----------------
    // (its waits for weights then never hold up the other tile's products)
    const int tile = warp - kSoftWarps - kConvWarps;
    constexpr uint32_t kIdQK = chunk_idesc(kChunkKeys, false), kIdPV = chunk_idesc(D, true);
    uint32_t n_seg = 0u, n_s = 0u, n_p = 0u;  // tiles, logits and weights so far
    uint32_t k_index = 0u;
    bool ok = true;
    const uint64_t q_desc = chunk_desc(sm.q[tile], 16), k_desc = chunk_desc(sm.k[0], 16);
    const uint64_t v_desc = chunk_desc(sm.v[0], S::SUB);
    const uint32_t t_s = tmem + (uint32_t)(tile * 128), t_o = tmem + 256u + (uint32_t)(tile * D);
    // the logits of step k
    auto qk = [&](uint32_t k) {
      const int slot = ring_slot<kChunkSlots>(k);
      ok = chunk_wait(sm, &sm.k_full[slot], ring_parity<kChunkSlots>(k));
      if (!ok) return;
      tc_fence_after();
      const uint32_t buf = n_s++ & 1u;
      const uint64_t b = k_desc + (uint64_t)(slot * S::DH * S::SUB >> 4);
#pragma unroll
      for (int s = 0; s < D / 16; ++s)
        umma_f16_ss(t_s + buf * 64u, q_desc + (uint64_t)((s >> 2) * S::QSUB >> 4) + 2 * (s & 3),
                    b + (uint64_t)((s >> 2) * S::SUB >> 4) + 2 * (s & 3), kIdQK, s > 0 ? 1u : 0u);
      umma_commit(&sm.s_full[tile][buf]);
      umma_commit(&sm.k_empty[slot]);
    };
    do {
      const int n = walk.last - walk.first;
      if (tile * 128 >= walk.nrows) {  // no row of this tile: the slots pass by
        for (int t = 0; t < n && ok; ++t, ++k_index) {
          const int slot = ring_slot<kChunkSlots>(k_index);
          const uint32_t phase = ring_parity<kChunkSlots>(k_index);
          ok = chunk_wait(sm, &sm.k_full[slot], phase);
          if (ok) mbar_arrive(&sm.k_empty[slot]);
          ok = ok && chunk_wait(sm, &sm.v_full[slot], phase);
          if (ok) mbar_arrive(&sm.v_empty[slot]);
        }
        continue;
      }
      ok = chunk_wait(sm, &sm.q_full[tile], n_seg++ & 1u);
      // logits two steps ahead of the weights: a buffer of S is free again as
      // soon as the product of its weights has been issued
      for (int at = 0; at < min(n, 2) && ok; ++at) qk(k_index + at);
      for (int t = 0; t < n && ok; ++t, ++k_index) {
        const int slot = ring_slot<kChunkSlots>(k_index);
        const uint32_t buf = n_p & 1u, phase = (n_p >> 1) & 1u;
        ++n_p;
        ok = chunk_wait(sm, &sm.v_full[slot], ring_parity<kChunkSlots>(k_index)) &&
             chunk_wait(sm, &sm.p_full[tile][buf], phase);
        if (!ok) break;
        tc_fence_after();
        const uint64_t b = v_desc + (uint64_t)(slot * S::DH * S::SUB >> 4);
#pragma unroll
        for (int s = 0; s < kChunkKeys / 16; ++s)
          umma_f16_ts(t_o, t_s + buf * 64u + (uint32_t)(8 * s), b + (uint64_t)(s * 2048 >> 4),
                      kIdPV, t > 0 || s > 0 ? 1u : 0u);
        umma_commit(&sm.o_done[tile][buf]);
        umma_commit(&sm.v_empty[slot]);
        if (t + 2 < n) qk(k_index + 2);
      }
    } while (ok && walk.next());
    // every product done before the tensor memory is freed
    umma_commit(&sm.drained);
    mbar_wait_bounded(&sm.drained, 0u);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarps - 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

}  // namespace kv8
}  // namespace csa2
