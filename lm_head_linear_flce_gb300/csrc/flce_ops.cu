// Host-side helpers shared by the operators around the LM head (flce_ops.h).
#include "flce_ops.h"

#include <atomic>

namespace flce {
namespace {

// Per device: 0 until the first query there, then (SM count << 1) | (compute
// capability is 10.3).  Atomic: racing first queries store the same value.
std::atomic<int> g_devices[64];

}  // namespace

flce_status check_device(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FLCE_ERR_CUDA;
  const bool cached = dev >= 0 && dev < 64;
  int v = cached ? g_devices[dev].load(std::memory_order_acquire) : 0;
  if (v == 0) {
    int major = 0, minor = 0, n = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return FLCE_ERR_CUDA;
    v = (n < 1 ? 2 : n << 1) | ((major == 10 && minor == 3) ? 1 : 0);
    if (cached) g_devices[dev].store(v, std::memory_order_release);
  }
  *sms = v >> 1;
  return (v & 1) ? FLCE_OK : FLCE_ERR_UNSUPPORTED_DEVICE;
}

bool make_tmap_sw64(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t outer,
                    uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer,
                    CUtensorMapDataType dtype) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return static_cast<Encode>(nullptr);
    return reinterpret_cast<Encode>(p);
  }();
  if (!encode) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {row_bytes};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t ones[2] = {1, 1};
  return encode(m, dtype, 2, const_cast<void*>(ptr), dims, strides, box, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace flce
