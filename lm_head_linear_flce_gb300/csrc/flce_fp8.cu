// Matrix product on 8-bit operands with block scales (flce_matmul_fp8).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "flce_internal.h"
#include "flce_ops.h"

namespace flce {
namespace {

constexpr int kTile = 64;  // output rows and columns per block
constexpr int kKStep = 32; // K per shared-memory step (4 steps per scale block)

__device__ __forceinline__ float e4m3_to_f(uint8_t b) {
  __nv_fp8_e4m3 v;
  v.__x = b;
  return static_cast<float>(v);
}

__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float v) {
  *p = __float2bfloat16_rn(v);
}

// 64 x 64 outputs per block of 256 threads, 4 x 4 per thread; each 128-column
// block of K is summed by itself, then scaled into the result.
template <class O>
__global__ void __launch_bounds__(256)
    matmul_fp8_kernel(const uint8_t* __restrict__ A, int64_t lda,
                      const float* __restrict__ a_scale, const uint8_t* __restrict__ B,
                      int64_t ldb, const float* __restrict__ b_scale, int64_t M, int64_t V, int K,
                      O* __restrict__ y, int64_t ldy) {
  __shared__ float as[kKStep][kTile + 1], bs[kKStep][kTile + 1];
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * kTile;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int groups = (K + kScaleGroup - 1) / kScaleGroup;
  float acc[4][4] = {};
  for (int j = 0; j < groups; ++j) {
    float part[4][4] = {};
    for (int k0 = j * kScaleGroup; k0 < min(K, (j + 1) * kScaleGroup); k0 += kKStep) {
      for (int i = threadIdx.x; i < kTile * kKStep; i += 256) {
        const int k = i % kKStep, r = i / kKStep;
        const bool in_k = k0 + k < K;
        as[k][r] = in_k && m0 + r < M ? e4m3_to_f(A[(m0 + r) * lda + k0 + k]) : 0.f;
        bs[k][r] = in_k && v0 + r < V ? e4m3_to_f(B[(v0 + r) * ldb + k0 + k]) : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kKStep; ++k) {
        float a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = as[k][ty * 4 + i];
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = bs[k][tx + 16 * i];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int n = 0; n < 4; ++n) part[i][n] = fmaf(a[i], b[n], part[i][n]);
      }
      __syncthreads();
    }
    const float sb = b_scale[v0 / kScaleGroup * groups + j];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t m = m0 + ty * 4 + i;
      const float s = m < M ? a_scale[m * groups + j] * sb : 0.f;
#pragma unroll
      for (int n = 0; n < 4; ++n) acc[i][n] = fmaf(s, part[i][n], acc[i][n]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int64_t m = m0 + ty * 4 + i, v = v0 + tx + 16 * n;
      if (m < M && v < V) store_out(y + m * ldy + v, acc[i][n]);
    }
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" flce_status flce_matmul_fp8(const void* A, int64_t lda, const float* a_scale,
                                       const void* B, int64_t ldb, const float* b_scale, int64_t M,
                                       int64_t V, int64_t K, void* y, int64_t ldy,
                                       flce_dtype out_dtype, flce_stream_t stream) {
  constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1024;
  if (M < 0 || V <= 0 || K <= 0 || !valid_dtype(out_dtype)) return FLCE_ERR_INVALID_ARG;
  if (K % 16 != 0 || K > kMaxRowElems || M > kMaxDim || V > kMaxDim)
    return FLCE_ERR_UNSUPPORTED_SHAPE;
  if (M == 0) return FLCE_OK;
  if (!A || !B || !a_scale || !b_scale || !y) return FLCE_ERR_INVALID_ARG;
  if (lda < K || ldb < K || ldy < V || lda % 16 != 0 || ldb % 16 != 0) return FLCE_ERR_INVALID_ARG;
  const size_t e = dtype_bytes(out_dtype);
  if (!aligned_to(A, 16) || !aligned_to(B, 16) || !aligned_to(a_scale, 4) ||
      !aligned_to(b_scale, 4) || !aligned_to(y, e))
    return FLCE_ERR_INVALID_ARG;
  const int64_t gk = (K + kScaleGroup - 1) / kScaleGroup, gv = (V + kScaleGroup - 1) / kScaleGroup;
  const Range yr = {y, span_bytes(M, V, ldy, e)};
  const Range ins[] = {{A, span_bytes(M, K, lda, 1)},
                       {B, span_bytes(V, K, ldb, 1)},
                       {a_scale, span_bytes(M, gk, gk, 4)},
                       {b_scale, span_bytes(gv, gk, gk, 4)}};
  for (const Range& r : ins)
    if (ranges_overlap(yr, r)) return FLCE_ERR_INVALID_ARG;
  int sms = 0;
  const flce_status st = check_device(&sms);
  if (st != FLCE_OK) return st;
  const auto s = reinterpret_cast<cudaStream_t>(stream);
  if ((M + kTile - 1) / kTile > 65535) return FLCE_ERR_UNSUPPORTED_SHAPE;
  const dim3 grid(static_cast<unsigned>((V + kTile - 1) / kTile),
                  static_cast<unsigned>((M + kTile - 1) / kTile));
  const auto* a8 = static_cast<const uint8_t*>(A);
  const auto* b8 = static_cast<const uint8_t*>(B);
  if (out_dtype == FLCE_BF16)
    matmul_fp8_kernel<<<grid, 256, 0, s>>>(a8, lda, a_scale, b8, ldb, b_scale, M, V,
                                           static_cast<int>(K), static_cast<__nv_bfloat16*>(y),
                                           ldy);
  else
    matmul_fp8_kernel<<<grid, 256, 0, s>>>(a8, lda, a_scale, b8, ldb, b_scale, M, V,
                                           static_cast<int>(K), static_cast<float*>(y), ldy);
  note_launch();
  return cudaGetLastError() == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}
