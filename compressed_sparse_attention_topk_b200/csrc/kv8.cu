// C ABI of the 8-bit paged key/value cache (see include/csa2.h).  A
// translation unit of its own, with a device status word of its own:
// csa2_get_device_status reports both.
#include "csa2.h"

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "host.cuh"
#include "kv8_attn.cuh"
#include "kv8_cache.cuh"
#include "kv8_chunk.cuh"
#include "kv8_select.cuh"

namespace csa2 {

namespace {
// A kernel of this unit was launched, or captured, so its word may be set: a
// process that never uses the cache has nothing to copy (12 us of the call).
std::atomic<bool> g_launched{false};

void note_launch() {
  if (!g_launched.load(std::memory_order_relaxed))
    g_launched.store(true, std::memory_order_release);
}
}  // namespace

// Reads and clears this unit's device status word (the stream has been
// synchronised).
csa2_status kv8_take_status(uint32_t *v) {
  const uint32_t zero = 0;
  *v = 0;
  if (!g_launched.load(std::memory_order_acquire)) return CSA2_OK;
  if (cudaMemcpyFromSymbol(v, g_device_status, sizeof(*v)) != cudaSuccess) return CSA2_ERR_CUDA;
  if (*v && cudaMemcpyToSymbol(g_device_status, &zero, sizeof(zero)) != cudaSuccess)
    return CSA2_ERR_CUDA;
  return CSA2_OK;
}

}  // namespace csa2

using namespace csa2;

namespace {

int log2_of(int32_t block) {
  return block == 16 ? 4 : block == 32 ? 5 : block == 64 ? 6 : block == 128 ? 7 : -1;
}

// Checks a cache and makes the kernels' view of it.
csa2_status cache_view(const csa2_kv8 *c, kv8::Cache *out) {
  if (!c || c->Hk < 1 || c->D < 1 || c->block < 1 || c->pages < 1) return CSA2_ERR_INVALID_ARG;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->k_sum || !aligned(c->k, 16) ||
      !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
      !aligned(c->k_sum, 16))
    return CSA2_ERR_INVALID_ARG;
  const int shift = log2_of(c->block);
  if (shift < 0 || (c->D != 64 && c->D != 128) || c->Hk > 128 ||
      c->pages >= (int64_t(1) << 31) / c->block / c->Hk)
    return CSA2_ERR_UNSUPPORTED;
  *out = {c->k,   c->v,     c->k_scale, c->v_scale, c->k_sum,
          (int32_t)c->pages, c->Hk,    c->block,   shift,      c->D};
  return CSA2_OK;
}

// Checks shared by the calls over a step's tokens (n > 0).
csa2_status check_step(const uint16_t *q, int64_t q_stride, const kv8::Cache &c,
                       const int32_t *table, int32_t width, const int32_t *cu,
                       const int32_t *lens, int32_t B, int32_t H) {
  if (!q || !table || !cu || !lens || !aligned(q, 16) || !aligned(table, 4) || !aligned(cu, 4) ||
      !aligned(lens, 4) || width < 1 || H < 1 || H % c.Hk != 0 || q_stride % 8 != 0 ||
      q_stride < int64_t(H) * c.D)
    return CSA2_ERR_INVALID_ARG;
  if (H > 128 || B > kv8::kMaxSeqs) return CSA2_ERR_UNSUPPORTED;
  return CSA2_OK;
}

struct Bytes {
  const void *at;
  size_t n;
};

// Whether any of the first `written` ranges shares a byte with another range.
template <size_t N>
bool overlap(const Bytes (&r)[N], size_t written) {
  for (size_t i = 0; i < written; ++i)
    for (size_t j = i + 1; j < N; ++j) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(r[i].at);
      const uintptr_t b = reinterpret_cast<uintptr_t>(r[j].at);
      if (r[i].n && r[j].n && a < b + r[j].n && b < a + r[i].n) return true;
    }
  return false;
}

template <int D, int BS>
void launch_append(const kv8::AppendParams &p, cudaStream_t st) {
  const dim3 grid((unsigned)ceil_div(p.n, p.group), (unsigned)p.c.Hk, 2);
  kv8::kv8_append_kernel<D, BS><<<grid, kv8::kAppendThreads, 0, st>>>(p);
}

template <int D>
csa2_status launch_append_d(const kv8::AppendParams &p, cudaStream_t st) {
  switch (p.c.bs) {
    case 16: launch_append<D, 16>(p, st); break;
    case 32: launch_append<D, 32>(p, st); break;
    case 64: launch_append<D, 64>(p, st); break;
    default: launch_append<D, 128>(p, st); break;
  }
  return after_launch();
}

// A dependent launch: its blocks come up while the kernel before it ends.
template <class... Params, class... Args>
csa2_status launch_dependent(void (*kernel)(Params...), dim3 grid, int threads, size_t smem,
                             cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) return CSA2_ERR_CUDA;
  return after_launch();
}

template <int D, int R>
void launch_score(const kv8::SelectParams &p, dim3 grid, cudaStream_t st) {
  kv8::kv8_score_kernel<D, R><<<grid, kv8::kScoreThreads, 0, st>>>(p);
}

// Rows of more blocks than a warp's registers hold go to a CTA each, with
// their keys in shared memory up to this many.
constexpr int32_t kPickStaged = 40960;

csa2_status launch_select(const kv8::SelectParams &p, cudaStream_t st) {
  // tiles of 32 tokens where sequences have that many on average, else of 8
  // (both kernels, D = 128: 4 sequences of 4 tokens and 262,144 positions 27 us
  // with 8, 31 with 32; of 24 to 64 tokens and 65,536 positions the same within
  // 2 us; 64 sequences of 40 tokens and 8,192 positions 39 and 37); the blocks
  // split so that about three CTAs per SM share the work (each forms its
  // tokens' queries anew: a 4,096-token chunk 76 us with one split, 84 with two)
  const int32_t TT = p.s.n >= int64_t(32) * p.s.B ? 32 : 8;
  const int64_t tiles = p.s.n / TT + p.s.B;
  const int64_t most = std::max<int64_t>(1, ceil_div(p.s.width, 16 * kv8::kScoreWarps));
  const int64_t splits = std::min<int64_t>(
      std::min<int64_t>(most, 65535),
      std::max<int64_t>(1, 3 * device_sms() / std::max<int64_t>(1, tiles * p.c.Hk)));
  {
    const dim3 grid((unsigned)tiles, (unsigned)p.c.Hk, (unsigned)splits);
    TraceScope ts("kv8_score", st);
    if (p.c.D == 64) TT == 8 ? launch_score<64, 1>(p, grid, st) : launch_score<64, 4>(p, grid, st);
    else TT == 8 ? launch_score<128, 1>(p, grid, st) : launch_score<128, 4>(p, grid, st);
    const csa2_status rc = after_launch();
    if (rc != CSA2_OK) return rc;
  }
  const int64_t rows = p.s.n * p.c.Hk;
  TraceScope ts("kv8_pick", st);
  // a warp per row up to 2,048 blocks: as fast as a CTA per row for a few rows
  // (both kernels, 4 tokens: 14-21 us and 14-19), twice as fast for many (1,024
  // tokens over 2,048 blocks 50 us, 94 with a CTA per row)
  const dim3 warps((unsigned)ceil_div(rows, kv8::kPickWarps));
  if (p.s.width <= 256)
    return launch_dependent(kv8::kv8_pick_warp_kernel<8>, warps, 32 * kv8::kPickWarps, 0, st, p);
  if (p.s.width <= 1024)
    return launch_dependent(kv8::kv8_pick_warp_kernel<32>, warps, 32 * kv8::kPickWarps, 0, st, p);
  if (p.s.width <= 2048)
    return launch_dependent(kv8::kv8_pick_warp_kernel<64>, warps, 32 * kv8::kPickWarps, 0, st, p);
  const int staged = p.s.width <= kPickStaged ? 1 : 0;
  static std::atomic<bool> done[256];  // per device: attributes set
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 256 || !done[dev].load(std::memory_order_acquire)) {
    if (set_smem_attr(kv8::kv8_pick_cta_kernel, size_t(kPickStaged) * 4, false) != CSA2_OK)
      return CSA2_ERR_CUDA;
    if (dev >= 0 && dev < 256) done[dev].store(true, std::memory_order_release);
  }
  return launch_dependent(kv8::kv8_pick_cta_kernel, dim3((unsigned)rows), kv8::kPickThreads,
                          staged ? size_t(p.s.width) * 4 : 0, st, p, staged);
}

// One attention kernel of a call and its workspace.
struct AttnPart {
  int rows;        // query rows in a tile (0: the kernel is not used)
  int ctas;
  size_t rec_at, part_at;  // one record per CTA, and the partials
};

struct AttnPlan {
  AttnPart split, chunk;  // the split stream; 256-row tiles on tcgen05
  size_t bytes;
};

// Sequences of up to 32 query rows (tokens x heads of a group) belong to the
// split stream, with as many rows in a tile as they have -- every row of a
// tile reads the same fragments of the cache -- and longer ones to the
// tensor-core tiles.  Both kernels on both sides (us, split stream / tcgen05
// tiles, 2 kv heads, D = 128): 4 sequences of 65,536 positions with 24 rows
// 64 / 152, 32 rows 88 / 156, 40 rows (two tiles) 139 / 156, 64 rows 139 / 158,
// 96 rows 199 / 160, 256 rows 461 / 178; 16 sequences of 4,096 positions and 4
// kv heads with 32 rows 66 / 78, 40 rows 90 / 78, 64 rows 92 / 80.  The exception
// is a long context alone: one sequence of 262,144 positions with 40 to 64 rows
// takes 240 us here, 135 as two tiles of the split stream.
// The host knows the numbers of tokens and sequences only.
// Where one of several sequences may have a tile's 256 rows beyond a token for
// each, both kernels run, each on its own sequences (31 decode tokens of
// 32,768 positions and 512 tokens of 16,384 in one step: 320 us instead of 768;
// a kernel that finds no sequence costs about 8 us, so not where the tables
// reach fewer than 2^17 positions and kv heads in all: what one kernel loses
// there is of that size; tables far wider than their sequences lose nothing, 7
// decode tokens of 500 positions and a prompt of 300 55 us with either plan, of
// 2,000 64 us with both kernels and 72 with one); else the average decides.
// The split stream's tile is then the average, or a decode token's group where
// the tokens cannot be the same for all.  With lists everything is the split
// stream's, by the heads of a group.
constexpr int64_t kSplitRows = 32;

constexpr int64_t kBothReach = int64_t(1) << 17;

AttnPlan attn_plan(int64_t n, int32_t B, int32_t G, int32_t D, int32_t n_sel, bool far) {
  AttnPlan a{};
  const int64_t rows = n_sel > 0 ? G : ceil_div(n * G, std::max(B, 1));
  const bool mixed = far && n_sel == 0 && B > 1 && (n - B) * G >= kv8::kChunkRows;
  auto tile = [](int64_t r) { return r <= 4 ? 4 : 8 * (int)std::min<int64_t>(4, ceil_div(r, 8)); };
  if (mixed) a.split.rows = tile(n % B == 0 && rows <= kSplitRows ? rows : G);
  else if (n_sel > 0 || rows <= kSplitRows) a.split.rows = tile(rows);
  if (mixed || (n_sel == 0 && rows > kSplitRows)) a.chunk.rows = kv8::kChunkRows;
  a.split.ctas = (a.split.rows <= 8 ? 3 : 2) * device_sms();
  a.chunk.ctas = device_sms();
  for (AttnPart *part : {&a.split, &a.chunk}) {
    if (!part->rows) continue;
    part->rec_at = a.bytes;
    part->part_at = part->rec_at + align_up(size_t(part->ctas) * sizeof(int4), 256);
    a.bytes = part->part_at + align_up(size_t(part->ctas) * 2 * part->rows * (D + 2) * 4, 256);
  }
  return a;
}

// Merges the tiles that several CTAs shared; its blocks come up while the
// attention kernel's last ones run.
template <int D, int ROWS, int RPB>
csa2_status launch_merge(const kv8::AttnParams &p, const AttnPart &a, cudaStream_t st) {
  TraceScope ts("kv8_attn_merge", st);
  return launch_dependent(kv8::kv8_merge_kernel<D, ROWS, RPB>,
                          dim3((unsigned)a.ctas, ROWS / RPB), kv8::kMergeThreads, 0, st, p,
                          a.ctas);
}

template <int D>
csa2_status launch_chunk(const kv8::AttnParams &p, const AttnPart &a, cudaStream_t st) {
  const size_t smem = kv8::chunk_smem_bytes<D>();
  static std::atomic<bool> done[256];  // per device: attributes set
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 256 || !done[dev].load(std::memory_order_acquire)) {
    if (set_smem_attr(kv8::kv8_chunk_kernel<D>, smem, false) != CSA2_OK) return CSA2_ERR_CUDA;
    if (dev >= 0 && dev < 256) done[dev].store(true, std::memory_order_release);
  }
  {
    TraceScope ts("kv8_attn_chunk", st);
    kv8::kv8_chunk_kernel<D><<<(unsigned)a.ctas, kv8::kChunkThreads, smem, st>>>(p);
    const csa2_status rc = after_launch();
    if (rc != CSA2_OK) return rc;
  }
  return launch_merge<D, kv8::kChunkRows, 32>(p, a, st);
}

template <int D, int ROWS, bool P16>
csa2_status launch_split(const kv8::AttnParams &p, const AttnPart &a, cudaStream_t st) {
  using S = kv8::SplitShape<D, ROWS>;
  static std::atomic<bool> done[256];  // per device: attributes set
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 256 || !done[dev].load(std::memory_order_acquire)) {
    if (set_smem_attr(kv8::kv8_split_kernel<D, ROWS, P16>, S::SMEM, false) != CSA2_OK)
      return CSA2_ERR_CUDA;
    if (dev >= 0 && dev < 256) done[dev].store(true, std::memory_order_release);
  }
  const uint64_t rows = uint64_t(p.c.pages) * p.c.Hk * p.c.bs;
  const uint32_t box = P16 ? 16 : kv8::kUnit;
  CUtensorMap km, vm;
  if (!make_map_u8(&km, p.c.k, D, rows, 1, D, rows * D, box, 1) ||
      !make_map_u8(&vm, p.c.v, D, rows, 1, D, rows * D, box, 1))
    return CSA2_ERR_CUDA;
  {
    TraceScope ts("kv8_attn_split", st);
    kv8::kv8_split_kernel<D, ROWS, P16>
        <<<(unsigned)a.ctas, kv8::kSplitThreads, S::SMEM, st>>>(km, vm, p);
    const csa2_status rc = after_launch();
    if (rc != CSA2_OK) return rc;
  }
  // at most this many tiles share the CTAs: with few, a row has hundreds of
  // partials, and a block to itself (one sequence and kv head of 262,144
  // positions: 66 us with four rows to a block)
  const int64_t tiles = (p.s.n * p.G / ROWS + p.s.B) * p.c.Hk;
  return tiles * 32 <= a.ctas ? launch_merge<D, ROWS, 1>(p, a, st)
                              : launch_merge<D, ROWS, 4>(p, a, st);
}

template <int D, bool P16>
csa2_status launch_split_rows(const kv8::AttnParams &p, const AttnPart &a, cudaStream_t st) {
  switch (a.rows) {
    case 4: return launch_split<D, 4, P16>(p, a, st);
    case 8: return launch_split<D, 8, P16>(p, a, st);
    case 16: return launch_split<D, 16, P16>(p, a, st);
    case 24: return launch_split<D, 24, P16>(p, a, st);
    default: return launch_split<D, 32, P16>(p, a, st);
  }
}

csa2_status launch_attn(kv8::AttnParams p, const AttnPlan &a, char *ws, cudaStream_t st) {
  const bool both = a.split.rows && a.chunk.rows;
  p.split_rows = both ? (int32_t)kSplitRows : 0;
  if (a.chunk.rows) {
    p.rec = reinterpret_cast<int4 *>(ws + a.chunk.rec_at);
    p.part = reinterpret_cast<float *>(ws + a.chunk.part_at);
    const csa2_status rc = p.c.D == 64 ? launch_chunk<64>(p, a.chunk, st)
                                       : launch_chunk<128>(p, a.chunk, st);
    if (rc != CSA2_OK || !both) return rc;
  }
  p.rec = reinterpret_cast<int4 *>(ws + a.split.rec_at);
  p.part = reinterpret_cast<float *>(ws + a.split.part_at);
  if (p.c.bs == 16)
    return p.c.D == 64 ? launch_split_rows<64, true>(p, a.split, st)
                       : launch_split_rows<128, true>(p, a.split, st);
  return p.c.D == 64 ? launch_split_rows<64, false>(p, a.split, st)
                     : launch_split_rows<128, false>(p, a.split, st);
}

}  // namespace

extern "C" {

csa2_status csa2_block_tables(const int32_t *lens, const int32_t *add, int32_t B, int32_t block,
                              int32_t *table, int32_t width, const int32_t *free_pages,
                              int32_t n_free, int32_t *lens_out, int32_t *cu, int64_t *slots,
                              int32_t *pos, int64_t cap, int32_t *used, void *stream) {
  if (B < 0 || width < 1 || n_free < 0 || cap < 0 || block < 1) return CSA2_ERR_INVALID_ARG;
  if (!cu || !used || (B > 0 && (!lens || !add || !table || !lens_out)) ||
      (n_free > 0 && !free_pages) || (cap > 0 && (!slots || !pos)) ||
      !aligned(lens, 4) || !aligned(add, 4) || !aligned(table, 4) || !aligned(free_pages, 4) ||
      !aligned(lens_out, 4) || !aligned(cu, 4) || !aligned(used, 4) || !aligned(slots, 8) ||
      !aligned(pos, 4))
    return CSA2_ERR_INVALID_ARG;
  const int shift = log2_of(block);
  if (shift < 0 || B > kv8::kMaxSeqs || int64_t(width) * block >= (int64_t(1) << 31) ||
      cap >= (int64_t(1) << 31))
    return CSA2_ERR_UNSUPPORTED;
  // every block reads the lengths, the lists and the tables again
  const size_t b4 = size_t(B) * 4;
  const Bytes ranges[] = {{lens_out, b4},           {cu, b4 + 4},
                          {slots, size_t(cap) * 8}, {pos, size_t(cap) * 4},
                          {used, 4},                {table, b4 * width},
                          {lens, b4},               {add, b4},
                          {free_pages, size_t(n_free) * 4}};
  if (overlap(ranges, 6)) return CSA2_ERR_INVALID_ARG;
  const kv8::TableParams p{lens, add, table, free_pages, lens_out, cu,    slots, pos,
                           used, cap, B,     shift,      width,    n_free};
  const int64_t blocks = std::min<int64_t>(
      std::max<int64_t>({1, ceil_div(cap, kv8::kTableThreads), ceil_div(B, 64)}), device_sms());
  note_launch();
  TraceScope ts("block_tables", as_stream(stream));
  kv8::block_tables_kernel<<<(unsigned)blocks, kv8::kTableThreads, (2 * size_t(B) + 1) * 4,
                             as_stream(stream)>>>(p);
  return after_launch();
}

csa2_status csa2_kv8_append(const csa2_kv8 *cache, const uint16_t *k_new, int64_t k_stride,
                            const uint16_t *v_new, int64_t v_stride, const int64_t *slots,
                            int64_t n, void *stream) {
  kv8::AppendParams p{};
  csa2_status rc = cache_view(cache, &p.c);
  if (rc != CSA2_OK) return rc;
  if (n < 0) return CSA2_ERR_INVALID_ARG;
  if (n == 0) return CSA2_OK;
  const int64_t row = int64_t(p.c.Hk) * p.c.D;
  if (!k_new || !v_new || !slots || !aligned(k_new, 16) || !aligned(v_new, 16) ||
      !aligned(slots, 8) || k_stride % 8 != 0 || v_stride % 8 != 0 || k_stride < row ||
      v_stride < row)
    return CSA2_ERR_INVALID_ARG;
  if (n >= (int64_t(1) << 31)) return CSA2_ERR_UNSUPPORTED;
  p.x[0] = k_new;
  p.x[1] = v_new;
  p.stride[0] = k_stride;
  p.stride[1] = v_stride;
  p.slots = slots;
  p.n = n;
  // a decode step: a token per CTA, so that its runs go side by side; more
  // tokens: 32, so that fewer CTAs find no run.  The host does not know which
  // it is (us for a run per token / one prompt, 4 heads): 512 tokens 27 / 14
  // with 1, 84 / 12 with 32; 1,024: 41 / 16 and 86 / 12; 2,048: 74 / 23 and 98 /
  // 14; 4,096: 137 / 35 and 133 / 16.  (10,241 tokens written and read back: 31.4
  // us, 32.5 with 16.)
  p.group = n <= 1024 ? 1 : kv8::kAppendGroup;
  note_launch();
  TraceScope ts("kv8_append", as_stream(stream));
  return p.c.D == 64 ? launch_append_d<64>(p, as_stream(stream))
                     : launch_append_d<128>(p, as_stream(stream));
}

csa2_status csa2_kv8_unpack(const csa2_kv8 *cache, const int64_t *slots, int64_t n, float *k_out,
                            float *v_out, void *stream) {
  kv8::Cache c;
  csa2_status rc = cache_view(cache, &c);
  if (rc != CSA2_OK) return rc;
  if (n < 0 || !aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(slots, 8))
    return CSA2_ERR_INVALID_ARG;
  if (n == 0 || (!k_out && !v_out)) return CSA2_OK;
  if (!slots) return CSA2_ERR_INVALID_ARG;
  const int64_t blocks = std::min<int64_t>(ceil_div(n * c.Hk * (c.D / 4), kv8::kUnpackThreads),
                                           int64_t(device_sms()) * 8);
  const dim3 grid((unsigned)blocks, 2);
  note_launch();
  TraceScope ts("kv8_unpack", as_stream(stream));
  if (c.D == 64)
    kv8::kv8_unpack_kernel<64>
        <<<grid, kv8::kUnpackThreads, 0, as_stream(stream)>>>(c, slots, n, k_out, v_out);
  else
    kv8::kv8_unpack_kernel<128>
        <<<grid, kv8::kUnpackThreads, 0, as_stream(stream)>>>(c, slots, n, k_out, v_out);
  return after_launch();
}

size_t csa2_kv8_select_workspace_size(int64_t n, int32_t Hk, int32_t width) {
  if (n < 0 || Hk < 1 || Hk > 128 || width < 1 || width > 65536) return 0;
  return std::max<size_t>(256, align_up(size_t(n) * Hk * width * 4, 256));
}

csa2_status csa2_kv8_select(const uint16_t *q, int64_t q_stride, const csa2_kv8 *cache,
                            const int32_t *table, int32_t width, const int32_t *cu,
                            const int32_t *lens, int32_t B, int64_t n, int32_t H, int32_t n_sel,
                            int32_t n_first, int32_t n_last, int32_t *sel, void *ws,
                            size_t ws_bytes, void *stream) {
  kv8::SelectParams p{};
  csa2_status rc = cache_view(cache, &p.c);
  if (rc != CSA2_OK) return rc;
  if (n < 0 || B < 0 || n_sel < 1 || n_first < 0 || n_last < 1 ||
      int64_t(n_first) + n_last > n_sel)
    return CSA2_ERR_INVALID_ARG;
  if (n == 0 || B == 0) return CSA2_OK;
  rc = check_step(q, q_stride, p.c, table, width, cu, lens, B, H);
  if (rc != CSA2_OK) return rc;
  if (!sel || !aligned(sel, 4)) return CSA2_ERR_INVALID_ARG;
  if (n_sel > 4096 || width > 65536 || n >= (int64_t(1) << 31) / p.c.Hk)
    return CSA2_ERR_UNSUPPORTED;
  if (!ws || ws_bytes < csa2_kv8_select_workspace_size(n, p.c.Hk, width) || !aligned(ws, 16))
    return CSA2_ERR_WORKSPACE;
  p.s = {cu, lens, table, B, width, n};
  p.q = q;
  p.q_stride = q_stride;
  p.G = H / p.c.Hk;
  p.n_sel = n_sel;
  p.n_first = n_first;
  p.n_last = n_last;
  p.sel = sel;
  p.scores = static_cast<float *>(ws);
  note_launch();
  return launch_select(p, as_stream(stream));
}

size_t csa2_kv8_attn_workspace_size(int64_t n, int32_t B, int32_t H, int32_t Hk, int32_t D,
                                    int32_t n_sel) {
  if (n < 0 || B < 0 || H < 1 || Hk < 1 || H % Hk != 0 || (D != 64 && D != 128) || n_sel < 0)
    return 0;
  return std::max(attn_plan(n, B, H / Hk, D, n_sel, false).bytes,
                  attn_plan(n, B, H / Hk, D, n_sel, true).bytes);
}

csa2_status csa2_kv8_attn(const uint16_t *q, int64_t q_stride, const csa2_kv8 *cache,
                          const int32_t *table, int32_t width, const int32_t *cu,
                          const int32_t *lens, int32_t B, int64_t n, int32_t H,
                          const int32_t *sel, int32_t n_sel, float sm_scale, uint16_t *out,
                          float *lse, void *ws, size_t ws_bytes, void *stream) {
  kv8::AttnParams p{};
  csa2_status rc = cache_view(cache, &p.c);
  if (rc != CSA2_OK) return rc;
  if (n < 0 || B < 0 || n_sel < 0 || !std::isfinite(sm_scale)) return CSA2_ERR_INVALID_ARG;
  if (n == 0 || B == 0) return CSA2_OK;
  if ((sel != nullptr) != (n_sel > 0)) return CSA2_ERR_INVALID_ARG;
  rc = check_step(q, q_stride, p.c, table, width, cu, lens, B, H);
  if (rc != CSA2_OK) return rc;
  if (!out || !aligned(out, 16) || !aligned(lse, 4) || !aligned(sel, 4))
    return CSA2_ERR_INVALID_ARG;
  if (n_sel > 65536 || n >= (int64_t(1) << 31) / H ||
      int64_t(width) * p.c.bs > kv8::kNoPos)
    return CSA2_ERR_UNSUPPORTED;
  if (!ws || ws_bytes < csa2_kv8_attn_workspace_size(n, B, H, p.c.Hk, p.c.D, n_sel) ||
      !aligned(ws, 16))
    return CSA2_ERR_WORKSPACE;
  p.s = {cu, lens, table, B, width, n};
  p.q = q;
  p.q_stride = q_stride;
  p.G = H / p.c.Hk;
  p.sel = sel;
  p.n_sel = n_sel;
  p.sm_scale = sm_scale;
  p.out = out;
  p.lse = lse;
  note_launch();
  const bool far = int64_t(B) * width * p.c.bs * p.c.Hk >= kBothReach;
  const AttnPlan plan = attn_plan(n, B, p.G, p.c.D, n_sel, far);
  return launch_attn(p, plan, static_cast<char *>(ws), as_stream(stream));
}

}  // extern "C"
