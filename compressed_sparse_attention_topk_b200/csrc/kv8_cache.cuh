// The 8-bit paged key/value cache: block tables and slot maps, the writer,
// the reader (contracts in include/csa2.h).
#pragma once

#include "common.cuh"

namespace csa2 {
namespace kv8 {

constexpr uint32_t kStatusBadLength = 4u;  // block tables: bad length, or no page or room
constexpr int kMaxSeqs = 4096;

struct Cache {
  int8_t *k, *v;
  float *k_scale, *v_scale;
  int16_t *k_sum;
  int32_t pages, Hk, bs, bs_shift, D;
};

// ---------------------------------------------------------------------------
// Block tables and slot maps.
//
// Two prefix sums over the requests (tokens added, pages taken), then a
// gather per token and a copy per new page.  Latency-bound: B <= 4096 lengths
// are 32 KB, so every CTA repeats the scan (L2 reads) instead of waiting for
// another one's, and the tokens are dealt over the CTAs (6 us for 32 requests
// of a token as for 512 of 69,792).
// ---------------------------------------------------------------------------
constexpr int kTableThreads = 512;

struct TableParams {
  const int32_t *lens, *add;
  int32_t *table;
  const int32_t *free_pages;
  int32_t *lens_out, *cu;
  int64_t *slots;
  int32_t *pos, *used;
  int64_t cap;
  int32_t B, bs_shift, width, n_free;
};

__device__ __forceinline__ long long warp_incl_scan64(long long v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  return v;
}

__device__ __forceinline__ long long warp_sum64(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ int32_t sat32(long long v) {
  return v > 0x7fffffffll ? 0x7fffffff : (int32_t)v;
}

__global__ void __launch_bounds__(kTableThreads) block_tables_kernel(const TableParams p) {
  // per request: first token and first page taken, then totals
  extern __shared__ int32_t table_smem[];
  int32_t *s_cu = table_smem, *s_page = table_smem + p.B + 1;
  __shared__ long long s_warp[2][kTableThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bs1 = (1 << p.bs_shift) - 1;
  bool bad = false;
  long long run_t = 0, run_p = 0;  // totals of the chunks before this one
  for (int b0 = 0; b0 < p.B; b0 += kTableThreads) {
    const int b = b0 + tid;
    long long len = 0, add = 0;
    if (b < p.B) {
      len = p.lens[b];
      add = p.add[b];
      bad |= len < 0 || add < 0;
      len = len < 0 ? 0 : len;
      add = add < 0 ? 0 : add;
    }
    const long long have = min64((len + bs1) >> p.bs_shift, p.width);
    const long long need = min64((len + add + bs1) >> p.bs_shift, p.width);
    const long long it = warp_incl_scan64(add), ip = warp_incl_scan64(need - have);
    if (lane == 31) {
      s_warp[0][warp] = it;
      s_warp[1][warp] = ip;
    }
    __syncthreads();
    long long bt = run_t, bp = run_p;
    for (int w = 0; w < kTableThreads / 32; ++w) {
      if (w < warp) {
        bt += s_warp[0][w];
        bp += s_warp[1][w];
      }
      run_t += s_warp[0][w];
      run_p += s_warp[1][w];
    }
    if (b < p.B) {
      s_cu[b] = sat32(bt + it - add);
      s_page[b] = sat32(bp + ip - (need - have));
      if (blockIdx.x == 0) {
        p.lens_out[b] = sat32(len + add);
        p.cu[b] = sat32(bt + it - add);
      }
    }
    __syncthreads();
  }
  const int32_t total = sat32(run_t);
  if (tid == 0) {
    s_cu[p.B] = total;
    if (blockIdx.x == 0) {
      p.cu[p.B] = total;
      p.used[0] = sat32(run_p);
      bad |= run_t > p.cap || run_p > p.n_free;
    }
  }
  __syncthreads();

  // new pages: one warp per request
  const int nwarps = gridDim.x * (kTableThreads / 32);
  for (int b = blockIdx.x * (kTableThreads / 32) + warp; b < p.B; b += nwarps) {
    const long long len = max(p.lens[b], 0);
    const long long end = len + max(p.add[b], 0);
    const int have = (int)min64((len + bs1) >> p.bs_shift, p.width);
    const int need = (int)min64((end + bs1) >> p.bs_shift, p.width);
    bad |= ((end + bs1) >> p.bs_shift) > p.width;
    for (int j = have + lane; j < need; j += 32) {
      const long long f = (long long)s_page[b] + j - have;
      p.table[(int64_t)b * p.width + j] = f < p.n_free ? p.free_pages[f] : -1;
    }
  }
  // tokens
  const int64_t step = (int64_t)gridDim.x * kTableThreads;
  for (int64_t i = (int64_t)blockIdx.x * kTableThreads + tid; i < p.cap; i += step) {
    int64_t slot = -1;
    int32_t at = -1;
    if (i < total) {
      int lo = 0, hi = p.B;  // s_cu[lo] <= i < s_cu[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_cu[mid] <= i) lo = mid;
        else hi = mid;
      }
      const long long len = max(p.lens[lo], 0);
      const long long pos = len + (i - s_cu[lo]);
      const long long j = pos >> p.bs_shift;
      const long long have = min64((len + bs1) >> p.bs_shift, p.width);
      int32_t page = -1;
      if (j < have) {
        page = p.table[(int64_t)lo * p.width + j];
      } else if (j < p.width) {
        const long long f = (long long)s_page[lo] + j - have;
        if (f < p.n_free) page = p.free_pages[f];
      }
      if (page >= 0) slot = ((int64_t)page << p.bs_shift) + (pos & bs1);
      else bad = true;
      at = sat32(pos);
    }
    p.slots[i] = slot;
    p.pos[i] = at;
  }
  if (bad) raise_status(kStatusBadLength);
}

// ---------------------------------------------------------------------------
// The writer.
//
// A run is the tokens of one page in a call: consecutive tokens at ascending
// slots.  A CTA per (group of tokens, kv head, keys or values) finds the runs
// that begin in its group (one look at the slots for all of them) and takes
// them in turn.  It loads the whole page at once, each row either a code row
// from before or a new one, and keeps it in registers: largest magnitude,
// scale, requantised old codes if the scale grew, new codes, and for keys the
// code sums.  Bound by bytes (4 D read + 2 D written per token and head; a
// decode step's page is mostly its earlier rows), in practice by the chain
// slots -> rows -> scale -> codes of a run: 6.5 us for 28 tokens of 4 heads,
// 18 us for 10,241 (31 MB, 1.7 TB/s; instructions issue in 53 % of the cycles,
// and between them a warp waits for rows, code and barriers in equal parts).
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 128;
constexpr int kAppendGroup = 32;  // tokens per CTA at most

struct AppendParams {
  Cache c;
  const uint16_t *x[2];
  int64_t stride[2];
  const int64_t *slots;
  int64_t n;
  int32_t group;  // tokens per CTA
};

// rint(x / s) of eight values (two to a word), |x| <= 127 s.  inv = fl(1 / s), or
// NaN for s below 2^-100.  x inv is within 127 2^-24 of x / s, and the rounded
// quotient within 127 2^-25: unless x inv lies within 2^-14 of a half, both
// round to the integer n that adding 1.5 2^23 leaves in the low bits; where one
// of the eight does, or is not finite, the divisions decide.
__device__ __forceinline__ void kv8_codes(const uint32_t (&w)[4], float s, float inv,
                                          int32_t (&c)[8]) {
  constexpr float kMagic = 12582912.f;
  bool sure = true;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = __uint_as_float((e & 1) ? (w[e >> 1] & 0xffff0000u) : (w[e >> 1] << 16));
    const float t = fmaf(x, inv, kMagic);
    const float n = t - kMagic;
    sure &= fabsf(fmaf(x, inv, -n)) <= 0.5f - 0x1p-14f;
    c[e] = __float_as_int(t) - __float_as_int(kMagic);
  }
  if (sure) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = __uint_as_float((e & 1) ? (w[e >> 1] & 0xffff0000u) : (w[e >> 1] << 16));
    c[e] = max(-127, min(127, __float2int_rn(__fdiv_rn(x, s))));
  }
}

template <int D, int BS>
__global__ void __launch_bounds__(kAppendThreads) kv8_append_kernel(const AppendParams p) {
  constexpr int CPR = D / 8;                    // 8-element pieces of a row
  constexpr int RPP = kAppendThreads / CPR;     // rows per pass
  constexpr int PASSES = (BS + RPP - 1) / RPP;
  __shared__ float s_max[kAppendThreads / 32];
  __shared__ int64_t s_slot[kAppendGroup + BS];  // of tokens g0 - 1 ..
  __shared__ uint32_t s_runs;
  __shared__ int s_len[2];                      // by parity of the run: one barrier less
  __shared__ int32_t s_sum[RPP][D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.y;
  const bool vals = blockIdx.z != 0;
  const uint16_t *x_in = vals ? p.x[1] : p.x[0];
  const int64_t stride = vals ? p.stride[1] : p.stride[0];
  const int col = (tid % CPR) * 8, rsub = tid / CPR;
  const int64_t slots_end = (int64_t)p.c.pages * BS;
  const int64_t g0 = (int64_t)blockIdx.x * p.group;
  const int count = (int)min64(p.group, p.n - g0);
  // the group's slots, the one before them and what its last run may reach
  for (int k = tid; k < kAppendGroup + BS; k += kAppendThreads) {
    const int64_t at = g0 + k - 1;
    s_slot[k] = at >= 0 && at < p.n ? p.slots[at] : -2;
  }
  __syncthreads();
  // the tokens of the group at which a run begins
  if (warp == 0) {
    bool begins = false;
    if (lane < count) {
      const int64_t s = s_slot[lane + 1];
      if (s >= slots_end) raise_status(kStatusBadIndex);
      begins = s >= 0 && s < slots_end && ((s & (BS - 1)) == 0 || s_slot[lane] != s - 1);
    }
    const uint32_t who = __ballot_sync(0xffffffffu, begins);
    if (lane == 0) {
      s_runs = who;
      s_len[0] = s_len[1] = BS;
    }
  }
  __syncthreads();
  uint32_t runs = s_runs;
  for (int turn = 0; runs; ++turn, runs &= runs - 1) {
    const int in_group = __ffs(runs) - 1;
    const int64_t i = g0 + in_group;
    const int64_t slot = s_slot[in_group + 1];
    const int r0 = (int)(slot & (BS - 1));
    const int64_t ph = slot / BS * p.c.Hk + h;
    int8_t *codes = (vals ? p.c.v : p.c.k) + ph * BS * D;
    float *scale_at = (vals ? p.c.v_scale : p.c.k_scale) + ph;
    const float s_old = r0 ? *scale_at : 0.f;
    // the run's length: the first row whose token does not follow
    if (tid < BS - r0 && s_slot[in_group + 1 + tid] != slot + tid)
      atomicMin(&s_len[turn & 1], tid);
    // the page's rows: 8 codes (x, y) before r0, 8 new values from there
    uint4 x[PASSES];
#pragma unroll
    for (int a = 0; a < PASSES; ++a) {
      const int r = a * RPP + rsub;
      x[a] = make_uint4(0u, 0u, 0u, 0u);
      if (r < r0) {
        const uint2 w = *reinterpret_cast<const uint2 *>(codes + r * D + col);
        x[a].x = w.x;
        x[a].y = w.y;
      }
    }
    __syncthreads();
    const int end = min(r0 + s_len[turn & 1], BS);
    const uint16_t *src = x_in + (i - r0) * stride + (int64_t)h * D + col;
#pragma unroll
    for (int a = 0; a < PASSES; ++a) {
      const int r = a * RPP + rsub;
      if (r >= r0 && r < end) x[a] = *reinterpret_cast<const uint4 *>(src + r * stride);
    }
    float big = 0.f;
#pragma unroll
    for (int a = 0; a < PASSES; ++a) {
      if (a * RPP + rsub < r0) continue;
      const uint32_t w[4] = {x[a].x, x[a].y, x[a].z, x[a].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        big = fmaxf(big, fabsf(__uint_as_float(w[e] << 16)));
        big = fmaxf(big, fabsf(__uint_as_float(w[e] & 0xffff0000u)));
      }
    }
    big = warp_max(big);
    if (lane == 0) s_max[warp] = big;
    __syncthreads();  // (also: every thread has read the old scale and the length)
#pragma unroll
    for (int w = 0; w < kAppendThreads / 32; ++w) big = fmaxf(big, s_max[w]);
    const float s = fmaxf(s_old, __fdiv_rn(big, 127.f));
    const bool grew = s > s_old;
    const float ratio = grew ? __fdiv_rn(s_old, s) : 1.f;
    const float inv = s >= 0x1p-100f ? __fdiv_rn(1.f, s) : __int_as_float(0x7fffffff);
    if (tid == 0) {
      *scale_at = s;
      s_len[(turn & 1) ^ 1] = BS;
    }
    int32_t sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int a = 0; a < PASSES; ++a) {
      const int r = a * RPP + rsub;
      if (r >= end) continue;
      const bool old = r < r0;
      const uint32_t w[4] = {x[a].x, x[a].y, x[a].z, x[a].w};
      int32_t cs[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (old) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          cs[e] = (int8_t)(w[e >> 2] >> (8 * (e & 3)));
          if (grew) cs[e] = __float2int_rn(__fmul_rn((float)cs[e], ratio));
        }
      } else if (s > 0.f) {
        kv8_codes(w, s, inv, cs);
      }
      uint32_t o[2] = {0u, 0u};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        o[e >> 2] |= (uint32_t)(uint8_t)cs[e] << (8 * (e & 3));
        sum[e] += cs[e];
      }
      if (!old || grew)
        *reinterpret_cast<uint2 *>(codes + r * D + col) = make_uint2(o[0], o[1]);
    }
    if (!vals) {
#pragma unroll
      for (int e = 0; e < 8; ++e) s_sum[rsub][col + e] = sum[e];
      __syncthreads();
      if (tid < D) {
        int32_t t = 0;
#pragma unroll
        for (int r = 0; r < RPP; ++r) t += s_sum[r][tid];
        p.c.k_sum[ph * D + tid] = (int16_t)t;
      }
    }
    __syncthreads();  // s_max, s_sum and s_len are free again
  }
}

// ---------------------------------------------------------------------------
// The reader: one thread per 4 codes of a row and head, so that a warp reads
// 128 bytes and writes 512 in one piece.  Bound by bytes (D read and 4 D
// written per row, head and array): 10,496 rows of 4 heads (54 MB) in 16 us
// (instructions issue in 64 % of the cycles, else the warps wait for the codes).
// ---------------------------------------------------------------------------
constexpr int kUnpackThreads = 256;

template <int D>
__global__ void __launch_bounds__(kUnpackThreads) kv8_unpack_kernel(
    const Cache c, const int64_t *__restrict__ slots, int64_t n, float *k_out, float *v_out) {
  constexpr int TPR = D / 4;  // threads per row
  float *out = blockIdx.y ? v_out : k_out;
  if (!out) return;
  const int8_t *codes = blockIdx.y ? c.v : c.k;
  const float *scales = blockIdx.y ? c.v_scale : c.k_scale;
  const int piece = threadIdx.x % TPR;
  const int64_t rows = n * c.Hk, step = (int64_t)gridDim.x * (kUnpackThreads / TPR);
  const int64_t end = (int64_t)c.pages << c.bs_shift;
#pragma unroll 4
  for (int64_t row = (int64_t)blockIdx.x * (kUnpackThreads / TPR) + threadIdx.x / TPR; row < rows;
       row += step) {
    const int64_t i = row / c.Hk;
    const int64_t slot = slots[i];
    uint32_t w = 0u;
    float s = 0.f;
    if (slot >= end) {
      if (piece == 0) raise_status(kStatusBadIndex);
    } else if (slot >= 0) {
      const int64_t ph = (slot >> c.bs_shift) * c.Hk + (row - i * c.Hk);
      const int64_t at = (ph << c.bs_shift) + (slot & (c.bs - 1));
      w = *reinterpret_cast<const uint32_t *>(codes + at * D + piece * 4);
      s = scales[ph];
    }
    float4 f;
    f.x = __fmul_rn((float)(int8_t)(w), s);
    f.y = __fmul_rn((float)(int8_t)(w >> 8), s);
    f.z = __fmul_rn((float)(int8_t)(w >> 16), s);
    f.w = __fmul_rn((float)(int8_t)(w >> 24), s);
    reinterpret_cast<float4 *>(out)[row * TPR + piece] = f;
  }
}

// 16 x 32 (signed or unsigned bytes) times 32 x 8 signed bytes, exact.
template <bool A_UNSIGNED>
__device__ __forceinline__ void mma_i8(int32_t (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                       uint32_t b1) {
  if constexpr (A_UNSIGNED)
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, "
        "%9}, {%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, "
        "%9}, {%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------------------
// Sequences of a step.
// ---------------------------------------------------------------------------
struct Steps {
  const int32_t *cu, *lens, *table;
  int32_t B, width;
  int64_t n;
};

// The sequence that owns token i (cu[b] <= i < cu[b+1]), or -1 for padding: a
// whole warp looks at 32 offsets a round.
__device__ __forceinline__ int seq_of(const Steps &s, int64_t i, int lane) {
  const int32_t total = s.cu[s.B];
  int lo = 0, n = s.B;  // cu[lo] <= i, and the owner is among lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const uint32_t who = __ballot_sync(0xffffffffu, lane * step < n && s.cu[at] <= i);
    const int k = who ? 31 - __clz(who) : 0;
    lo += k * step;
    n = min(step, n - k * step);
  }
  return i < total ? lo : -1;
}

}  // namespace kv8
}  // namespace csa2
