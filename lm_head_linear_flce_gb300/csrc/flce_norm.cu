// RMS norm with the residual's addition (forward, 8-bit output, backward) and
// the block quantiser.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "flce_internal.h"
#include "flce_ops.h"

namespace flce {
namespace {

constexpr int kNormThreads = 256;
constexpr int kDwRows = 64;  // rows per partial sum of dweight

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Sum over the block, the same on every thread.
__device__ float block_sum(float v) {
  __shared__ float part[kNormThreads / 32];
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
  for (int w = 0; w < kNormThreads / 32; ++w) t += part[w];
  __syncthreads();
  return t;
}

__device__ __forceinline__ uint8_t to_e4m3(float v) {
  return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}

// A block per row; a warp per group of 128 columns in the second pass.
template <class T, class W, bool FP8>
__global__ void __launch_bounds__(kNormThreads)
    norm_fwd_kernel(const T* __restrict__ x, int64_t ldx, const T* residual, int64_t ldr,
                    const W* __restrict__ weight, int H, float eps, T* y, uint8_t* q,
                    float* scale, T* h_out, float* rstd) {
  const int64_t row = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* xr = x + row * ldx;
  const T* rr = residual ? residual + row * ldr : nullptr;
  float ss = 0.f;
  for (int c = threadIdx.x; c < H; c += kNormThreads) {
    const float h = to_f(xr[c]) + (rr ? to_f(rr[c]) : 0.f);
    ss += h * h;
  }
  const float r = rsqrtf(block_sum(ss) / static_cast<float>(H) + eps);
  if (rstd && threadIdx.x == 0) rstd[row] = r;
  const int groups = (H + kScaleGroup - 1) / kScaleGroup;
  for (int g = warp; g < groups; g += kNormThreads / 32) {
    float v[4];
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = g * kScaleGroup + i * 32 + lane;
      v[i] = 0.f;
      if (c < H) {
        const float h = to_f(xr[c]) + (rr ? to_f(rr[c]) : 0.f);
        if (h_out) h_out[row * H + c] = from_f<T>(h);
        v[i] = h * r * to_f(weight[c]);
        if (!FP8) y[row * H + c] = from_f<T>(v[i]);
        a = fmaxf(a, fabsf(v[i]));
      }
    }
    if (FP8) {
      a = fmaxf(warp_max(a), kAmaxMin);
      const float inv = kFp8Max / a;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = g * kScaleGroup + i * 32 + lane;
        if (c < H) q[row * H + c] = to_e4m3(v[i] * inv);
      }
      if (lane == 0) scale[row * groups + g] = a / kFp8Max;
    }
  }
}

template <class T, class W>
__global__ void __launch_bounds__(kNormThreads)
    norm_bwd_dx_kernel(const T* __restrict__ dy, const T* __restrict__ dh,
                       const T* __restrict__ h, int64_t ldh, const W* __restrict__ weight,
                       const float* __restrict__ rstd, int H, T* __restrict__ dx) {
  const int64_t row = blockIdx.x;
  const float r = rstd[row];
  float dot = 0.f;
  for (int c = threadIdx.x; c < H; c += kNormThreads)
    dot += to_f(dy[row * H + c]) * to_f(weight[c]) * to_f(h[row * ldh + c]);
  const float k = r * r * block_sum(dot) / static_cast<float>(H);
  for (int c = threadIdx.x; c < H; c += kNormThreads) {
    float v = r * (to_f(dy[row * H + c]) * to_f(weight[c]) - to_f(h[row * ldh + c]) * k);
    if (dh) v += to_f(dh[row * H + c]);
    dx[row * H + c] = from_f<T>(v);
  }
}

// Partial sums of dweight over kDwRows rows, then their sum in order.
template <class T>
__global__ void __launch_bounds__(kNormThreads)
    norm_bwd_dw_kernel(const T* __restrict__ dy, const T* __restrict__ h, int64_t ldh,
                       const float* __restrict__ rstd, int64_t N, int H,
                       float* __restrict__ part) {
  const int c = blockIdx.y * kNormThreads + threadIdx.x;
  if (c >= H) return;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kDwRows;
  const int64_t n1 = min(N, n0 + kDwRows);
  float s = 0.f;
  for (int64_t n = n0; n < n1; ++n)
    s += to_f(dy[n * H + c]) * to_f(h[n * ldh + c]) * rstd[n];
  part[static_cast<int64_t>(blockIdx.x) * H + c] = s;
}

template <class W>
__global__ void __launch_bounds__(kNormThreads)
    norm_dw_sum_kernel(const float* __restrict__ part, int64_t parts, int H, W* __restrict__ dw) {
  const int c = blockIdx.x * kNormThreads + threadIdx.x;
  if (c >= H) return;
  float s = 0.f;
  for (int64_t p = 0; p < parts; ++p) s += part[p * H + c];
  dw[c] = from_f<W>(s);
}

// One block of block_rows x 128 elements per thread block.
template <class T>
__global__ void __launch_bounds__(kNormThreads)
    quantize_kernel(const T* __restrict__ x, int64_t ldx, int64_t R, int K, int block_rows,
                    uint8_t* __restrict__ q, float* __restrict__ scale) {
  __shared__ float part[kNormThreads / 32];
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * block_rows;
  const int c = blockIdx.y * kScaleGroup + (threadIdx.x & (kScaleGroup - 1));
  const int64_t r1 = min(R, r0 + block_rows);
  float a = 0.f;
  if (c < K)
    for (int64_t r = r0 + threadIdx.x / kScaleGroup; r < r1; r += kNormThreads / kScaleGroup)
      a = fmaxf(a, fabsf(to_f(x[r * ldx + c])));
  a = warp_max(a);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
  __syncthreads();
  for (int w = 0; w < kNormThreads / 32; ++w) a = fmaxf(a, part[w]);
  a = fmaxf(a, kAmaxMin);
  const float inv = kFp8Max / a;
  if (c < K)
    for (int64_t r = r0 + threadIdx.x / kScaleGroup; r < r1; r += kNormThreads / kScaleGroup)
      q[r * K + c] = to_e4m3(to_f(x[r * ldx + c]) * inv);
  if (threadIdx.x == 0) scale[static_cast<int64_t>(blockIdx.x) * gridDim.y + blockIdx.y] =
      a / kFp8Max;
}

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1;

// What both forward entry points check.
flce_status check_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                       const void* weight, int64_t N, int64_t H, flce_dtype dtype,
                       flce_dtype weight_dtype) {
  if (N < 0 || H <= 0 || !valid_dtype(dtype) || !valid_dtype(weight_dtype))
    return FLCE_ERR_INVALID_ARG;
  if (H > kMaxRowElems || N > kMaxRows) return FLCE_ERR_UNSUPPORTED_SHAPE;
  if (N == 0) return FLCE_OK;
  if (!x || !weight || ldx < H || (residual && ldr < H)) return FLCE_ERR_INVALID_ARG;
  const size_t e = dtype_bytes(dtype);
  if (!aligned_to(x, e) || !aligned_to(residual, e) ||
      !aligned_to(weight, dtype_bytes(weight_dtype)))
    return FLCE_ERR_INVALID_ARG;
  return FLCE_OK;
}

// No output overlaps an input or another output, but that h_out may be x or
// residual itself.
bool norm_outputs_apart(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                        const Range& weight, int64_t N, int64_t H, size_t e, const void* h_out,
                        const Range& a, const Range& b) {
  const Range ins[] = {{x, span_bytes(N, H, ldx, e)},
                       {residual, span_bytes(N, H, ldr, e)},
                       weight};
  const Range h = {h_out, span_bytes(N, H, H, e)};
  for (const Range& r : ins) {
    if (ranges_overlap(a, r) || ranges_overlap(b, r)) return false;
    const bool itself = h_out && r.p == h_out && r.p != weight.p &&
                        ((r.p == x && ldx == H) || (r.p == residual && ldr == H));
    if (!itself && ranges_overlap(h, r)) return false;
  }
  return !ranges_overlap(a, b) && !ranges_overlap(a, h) && !ranges_overlap(b, h);
}

template <class T, class W, bool FP8>
cudaError_t run_norm_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                         const void* weight, int64_t N, int64_t H, float eps, void* y, void* q,
                         float* scale, void* h_out, float* rstd, cudaStream_t s) {
  norm_fwd_kernel<T, W, FP8><<<static_cast<unsigned>(N), kNormThreads, 0, s>>>(
      static_cast<const T*>(x), ldx, static_cast<const T*>(residual), ldr,
      static_cast<const W*>(weight), static_cast<int>(H), eps, static_cast<T*>(y),
      static_cast<uint8_t*>(q), scale, static_cast<T*>(h_out), rstd);
  note_launch();
  return cudaGetLastError();
}

template <bool FP8, class... A>
cudaError_t norm_fwd_by_type(flce_dtype t, flce_dtype w, A... a) {
  if (t == FLCE_BF16)
    return w == FLCE_BF16 ? run_norm_fwd<__nv_bfloat16, __nv_bfloat16, FP8>(a...)
                          : run_norm_fwd<__nv_bfloat16, float, FP8>(a...);
  return w == FLCE_BF16 ? run_norm_fwd<float, __nv_bfloat16, FP8>(a...)
                        : run_norm_fwd<float, float, FP8>(a...);
}

int64_t dw_parts(int64_t N) { return (N + kDwRows - 1) / kDwRows; }

template <class T, class W>
cudaError_t run_norm_bwd(const void* dy, const void* dh, const void* h, int64_t ldh,
                         const void* weight, const float* rstd, int64_t N, int64_t H, void* dx,
                         void* dweight, void* ws, cudaStream_t s) {
  const int cols = static_cast<int>((H + kNormThreads - 1) / kNormThreads);
  if (dx && N > 0) {
    norm_bwd_dx_kernel<T, W><<<static_cast<unsigned>(N), kNormThreads, 0, s>>>(
        static_cast<const T*>(dy), static_cast<const T*>(dh), static_cast<const T*>(h), ldh,
        static_cast<const W*>(weight), rstd, static_cast<int>(H), static_cast<T*>(dx));
    note_launch();
  }
  if (dweight) {
    const int64_t parts = dw_parts(N);
    float* part = static_cast<float*>(ws);
    if (parts > 0) {
      norm_bwd_dw_kernel<T><<<dim3(static_cast<unsigned>(parts), cols), kNormThreads, 0, s>>>(
          static_cast<const T*>(dy), static_cast<const T*>(h), ldh, rstd, N,
          static_cast<int>(H), part);
      note_launch();
    }
    norm_dw_sum_kernel<W><<<cols, kNormThreads, 0, s>>>(part, parts, static_cast<int>(H),
                                                        static_cast<W*>(dweight));
    note_launch();
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

flce_status flce_rms_norm_forward(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                                  const void* weight, int64_t N, int64_t H, float eps,
                                  flce_dtype dtype, flce_dtype weight_dtype, void* y, void* h_out,
                                  float* rstd, flce_stream_t stream) {
  flce_status st = check_norm(x, ldx, residual, ldr, weight, N, H, dtype, weight_dtype);
  if (st != FLCE_OK || N == 0) return st;
  const size_t e = dtype_bytes(dtype);
  if (!y || !aligned_to(y, e) || !aligned_to(h_out, e)) return FLCE_ERR_INVALID_ARG;
  if (!norm_outputs_apart(x, ldx, residual, ldr,
                          {weight, static_cast<size_t>(H) * dtype_bytes(weight_dtype)}, N, H, e,
                          h_out, {y, span_bytes(N, H, H, e)},
                          {rstd, static_cast<size_t>(N) * 4}))
    return FLCE_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = check_device(&sms)) != FLCE_OK) return st;
  return norm_fwd_by_type<false>(dtype, weight_dtype, x, ldx, residual, ldr, weight, N, H, eps, y,
                                 static_cast<void*>(nullptr), static_cast<float*>(nullptr), h_out,
                                 rstd, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FLCE_OK
             : FLCE_ERR_CUDA;
}

flce_status flce_rms_norm_fp8(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                              const void* weight, int64_t N, int64_t H, float eps,
                              flce_dtype dtype, flce_dtype weight_dtype, void* q, float* scale,
                              void* h_out, flce_stream_t stream) {
  flce_status st = check_norm(x, ldx, residual, ldr, weight, N, H, dtype, weight_dtype);
  if (st != FLCE_OK || N == 0) return st;
  const size_t e = dtype_bytes(dtype);
  if (!q || !scale || !aligned_to(h_out, e)) return FLCE_ERR_INVALID_ARG;
  const int64_t groups = (H + kScaleGroup - 1) / kScaleGroup;
  if (!norm_outputs_apart(x, ldx, residual, ldr,
                          {weight, static_cast<size_t>(H) * dtype_bytes(weight_dtype)}, N, H, e,
                          h_out, {q, span_bytes(N, H, H, 1)},
                          {scale, span_bytes(N, groups, groups, 4)}))
    return FLCE_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = check_device(&sms)) != FLCE_OK) return st;
  return norm_fwd_by_type<true>(dtype, weight_dtype, x, ldx, residual, ldr, weight, N, H, eps,
                                static_cast<void*>(nullptr), q, scale, h_out,
                                static_cast<float*>(nullptr),
                                reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FLCE_OK
             : FLCE_ERR_CUDA;
}

size_t flce_rms_norm_workspace_size(int64_t N, int64_t H) {
  if (N < 0 || H <= 0 || H > kMaxRowElems || N > kMaxRows) return 0;
  const size_t n = static_cast<size_t>(dw_parts(N)) * static_cast<size_t>(H) * 4;
  return std::max<size_t>((n + 255) / 256 * 256, 256);
}

flce_status flce_rms_norm_backward(const void* dy, const void* dh, const void* h, int64_t ldh,
                                   const void* weight, const float* rstd, int64_t N, int64_t H,
                                   flce_dtype dtype, flce_dtype weight_dtype, void* dx,
                                   void* dweight, void* workspace, size_t workspace_bytes,
                                   flce_stream_t stream) {
  if (N < 0 || H <= 0 || !valid_dtype(dtype) || !valid_dtype(weight_dtype))
    return FLCE_ERR_INVALID_ARG;
  if (H > kMaxRowElems || N > kMaxRows) return FLCE_ERR_UNSUPPORTED_SHAPE;
  if (N > 0 && (!dy || !h || !weight || !rstd || ldh < H)) return FLCE_ERR_INVALID_ARG;
  const size_t e = dtype_bytes(dtype), we = dtype_bytes(weight_dtype);
  if (!aligned_to(dy, e) || !aligned_to(dh, e) || !aligned_to(h, e) || !aligned_to(dx, e) ||
      !aligned_to(weight, we) || !aligned_to(dweight, we))
    return FLCE_ERR_INVALID_ARG;
  if (dweight) {
    if (!workspace || !aligned_to(workspace, 256)) return FLCE_ERR_INVALID_ARG;
    if (workspace_bytes < flce_rms_norm_workspace_size(N, H)) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  }
  const size_t nh = span_bytes(N, H, H, e);
  const Range dxr = {dx, nh}, dwr = {dweight, static_cast<size_t>(H) * we};
  const Range ins[] = {{dy, nh},
                       {dh, nh},
                       {h, span_bytes(N, H, ldh, e)},
                       {weight, static_cast<size_t>(H) * we},
                       {rstd, static_cast<size_t>(N) * 4},
                       {workspace, workspace_bytes}};
  for (const Range& r : ins)
    if (ranges_overlap(dxr, r) || ranges_overlap(dwr, r)) return FLCE_ERR_INVALID_ARG;
  if (ranges_overlap(dxr, dwr)) return FLCE_ERR_INVALID_ARG;
  int sms = 0;
  const flce_status st = check_device(&sms);
  if (st != FLCE_OK) return st;
  const auto s = reinterpret_cast<cudaStream_t>(stream);
  const bool wb = weight_dtype == FLCE_BF16;
  cudaError_t err;
  if (dtype == FLCE_BF16)
    err = wb ? run_norm_bwd<__nv_bfloat16, __nv_bfloat16>(dy, dh, h, ldh, weight, rstd, N, H, dx,
                                                          dweight, workspace, s)
             : run_norm_bwd<__nv_bfloat16, float>(dy, dh, h, ldh, weight, rstd, N, H, dx, dweight,
                                                  workspace, s);
  else
    err = wb ? run_norm_bwd<float, __nv_bfloat16>(dy, dh, h, ldh, weight, rstd, N, H, dx, dweight,
                                                  workspace, s)
             : run_norm_bwd<float, float>(dy, dh, h, ldh, weight, rstd, N, H, dx, dweight,
                                          workspace, s);
  return err == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

flce_status flce_quantize_fp8(const void* x, int64_t ldx, int64_t R, int64_t K, flce_dtype dtype,
                              int block_rows, void* q, float* scale, flce_stream_t stream) {
  if (R < 0 || K <= 0 || !valid_dtype(dtype) || (block_rows != 1 && block_rows != kScaleGroup))
    return FLCE_ERR_INVALID_ARG;
  if (K > kMaxRowElems || R > kMaxRows) return FLCE_ERR_UNSUPPORTED_SHAPE;
  if (R == 0) return FLCE_OK;
  const size_t e = dtype_bytes(dtype);
  if (!x || !q || !scale || ldx < K || !aligned_to(x, e)) return FLCE_ERR_INVALID_ARG;
  const int64_t gr = (R + block_rows - 1) / block_rows, gk = (K + kScaleGroup - 1) / kScaleGroup;
  const Range xr = {x, span_bytes(R, K, ldx, e)}, qr = {q, span_bytes(R, K, K, 1)},
              sr = {scale, span_bytes(gr, gk, gk, 4)};
  if (ranges_overlap(xr, qr) || ranges_overlap(xr, sr) || ranges_overlap(qr, sr))
    return FLCE_ERR_INVALID_ARG;
  int sms = 0;
  const flce_status st = check_device(&sms);
  if (st != FLCE_OK) return st;
  const auto s = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(gr), static_cast<unsigned>(gk));
  if (dtype == FLCE_BF16)
    quantize_kernel<<<grid, kNormThreads, 0, s>>>(static_cast<const __nv_bfloat16*>(x), ldx, R,
                                                  static_cast<int>(K), block_rows,
                                                  static_cast<uint8_t*>(q), scale);
  else
    quantize_kernel<<<grid, kNormThreads, 0, s>>>(static_cast<const float*>(x), ldx, R,
                                                  static_cast<int>(K), block_rows,
                                                  static_cast<uint8_t*>(q), scale);
  note_launch();
  return cudaGetLastError() == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

}  // extern "C"
