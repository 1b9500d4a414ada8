// Host helpers that the library's translation units share: argument and
// launch checks, the kernel timing trace, tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "csa2.h"

namespace csa2 {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline cudaStream_t as_stream(void *s) { return reinterpret_cast<cudaStream_t>(s); }

inline int device_sms() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  static std::atomic<int> cache[256];  // per device: 0 unknown
  if (dev >= 0 && dev < 256) {
    const int c = cache[dev].load(std::memory_order_relaxed);
    if (c) return c;
  }
  int v = 148;
  if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) v = 148;
  if (dev >= 0 && dev < 256) cache[dev].store(v, std::memory_order_relaxed);
  return v;
}

inline csa2_status after_launch() { return cudaGetLastError() == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA; }

// ---------------------------------------------------------------------------
// Kernel timing trace: event pairs around launches while enabled.
// ---------------------------------------------------------------------------
struct TraceRecord {
  const char *name;
  cudaEvent_t start, stop;
};
constexpr size_t kTraceMax = size_t(1) << 16;
inline bool g_trace_on = false;
inline TraceRecord *g_trace = nullptr;
inline size_t g_trace_n = 0;

inline void trace_clear() {
  for (size_t i = 0; i < g_trace_n; ++i) {
    cudaEventDestroy(g_trace[i].start);
    cudaEventDestroy(g_trace[i].stop);
  }
  g_trace_n = 0;
}

// Records an event on `st`; while `st` is being captured into a CUDA graph
// the record becomes an event-record node of the graph (timed on every
// replay) instead of a capture-internal dependency.
inline void trace_record(cudaEvent_t ev, cudaStream_t st) {
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(st, &cs) == cudaSuccess && cs == cudaStreamCaptureStatusActive)
    cudaEventRecordWithFlags(ev, st, cudaEventRecordExternal);
  else
    cudaEventRecord(ev, st);
}

// Brackets one launch: records `start` on construction and `stop` on
// destruction when the trace is on and has room.
struct TraceScope {
  TraceRecord *rec = nullptr;
  cudaStream_t st;
  TraceScope(const char *name, cudaStream_t s) : st(s) {
    if (!g_trace_on || g_trace_n >= kTraceMax) return;
    if (!g_trace) g_trace = new TraceRecord[kTraceMax];
    TraceRecord &r = g_trace[g_trace_n];
    if (cudaEventCreate(&r.start) != cudaSuccess) return;
    if (cudaEventCreate(&r.stop) != cudaSuccess) {
      cudaEventDestroy(r.start);
      return;
    }
    r.name = name;
    rec = &r;
    ++g_trace_n;
    trace_record(r.start, st);
  }
  ~TraceScope() {
    if (rec) trace_record(rec->stop, st);
  }
};

// Per-device one-time kernel attribute setup (dynamic shared memory above
// 48 KiB, non-portable cluster size).  Must run before any stream capture;
// the entry points call it on their first use on a device.
template <typename K>
csa2_status set_smem_attr(K kernel, size_t bytes, bool big_cluster) {
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) !=
      cudaSuccess)
    return CSA2_ERR_CUDA;
  if (big_cluster &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
          cudaSuccess)
    return CSA2_ERR_CUDA;
  return CSA2_OK;
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (no link
// dependency on the driver library).
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = [] {  // looked up once (thread-safe initialisation)
    EncodeTiledFn f = nullptr;
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      f = reinterpret_cast<EncodeTiledFn>(ptr);
    cudaGetLastError();
    return f;
  }();
  return fn;
}

// 3-D byte tensor map: dims {d0, d1, d2}, byte strides of dims 1 and 2, box
// {d0, b1, b2}, swizzled over d0 bytes (d0 in {32, 64, 128}).
inline bool make_map_u8(CUtensorMap *m, const void *base, uint64_t d0, uint64_t d1, uint64_t d2,
                 uint64_t s1, uint64_t s2, uint32_t b1, uint32_t b2) {
  EncodeTiledFn f = encode_tiled();
  if (!f || d1 == 0 || d2 == 0) return false;
  const cuuint64_t dims[3] = {d0, d1, d2};
  const cuuint64_t strides[2] = {s1, s2};
  const cuuint32_t box[3] = {(cuuint32_t)d0, b1, b2};
  const cuuint32_t es[3] = {1, 1, 1};
  const CUtensorMapSwizzle sw = d0 == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                : d0 == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                           : CU_TENSOR_MAP_SWIZZLE_32B;
  return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box, es,
           CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace csa2
