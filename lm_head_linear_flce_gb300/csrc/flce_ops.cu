// Host-side helpers shared by the operators around the LM head (flce_ops.h).
#include "flce_ops.h"

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

cudaError_t allow_smem(const void* kernel, int smem, SmemLimit* limit) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool cached = dev >= 0 && dev < 64;
  if (cached && limit->set[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && cached) limit->set[dev].store(1, std::memory_order_release);
  return e;
}

}  // namespace flce
