// Host-side helpers shared by the entry points of the operators around the LM
// head (norm, 8-bit operands and their product, logits processing).
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "../../include/flce.h"

namespace flce {

constexpr int kScaleGroup = 128;          // columns that share a scale
constexpr float kFp8Max = 448.f;          // largest e4m3 value
constexpr float kAmaxMin = 0x1p-100f;     // floor of a block's max |v|: its scale stays normal
constexpr int64_t kMaxRowElems = 1 << 16; // longest norm row / contraction

// FLCE_OK and the SM count of the current device, if it is an sm_103 one.
flce_status check_device(int* sms);

// NVTX range over the host side of one call (a pointer check when no tool is
// attached).
struct OpRange {
  explicit OpRange(const char* name) { nvtxRangePushA(name); }
  ~OpRange() { nvtxRangePop(); }
  OpRange(const OpRange&) = delete;
  OpRange& operator=(const OpRange&) = delete;
};

// Raises a kernel's dynamic shared-memory limit to `smem`, on its first launch
// on a device; one SmemLimit per kernel.  Atomic: racing first launches set the
// same attribute.
struct SmemLimit {
  std::atomic<int> set[64] = {};
};
cudaError_t allow_smem(const void* kernel, int smem, SmemLimit* limit);

// Launches `kernel` so that it may start while the stream's previous kernel
// ends: its blocks take the places that become free, set themselves up and wait
// (griddep_wait, before their first access of global memory) until that kernel
// is complete.  Only where that kernel allows it (griddep_launch_dependents, or
// at its end); after anything else this is a plain launch.  cluster: CTAs per
// cluster, where the kernel does not fix it.
template <class... P, class... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, dim3 block, int smem,
                              cudaStream_t s, int cluster, const A&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

inline bool valid_dtype(flce_dtype t) { return t == FLCE_BF16 || t == FLCE_F32; }
inline size_t dtype_bytes(flce_dtype t) { return t == FLCE_F32 ? 4 : 2; }
inline bool aligned_to(const void* p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// Bytes from the first to the last element of a [rows][cols] matrix.
inline size_t span_bytes(int64_t rows, int64_t cols, int64_t ld, size_t elem) {
  if (rows <= 0 || cols <= 0) return 0;
  return (static_cast<size_t>(rows - 1) * static_cast<size_t>(ld) + static_cast<size_t>(cols)) *
         elem;
}

struct Range {
  const void* p;
  size_t n;
};

// Whether two byte ranges share a byte (a null range shares none).
inline bool ranges_overlap(const Range& a, const Range& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.n > 0 && b.n > 0 && x < y + b.n && y < x + a.n;
}

}  // namespace flce
