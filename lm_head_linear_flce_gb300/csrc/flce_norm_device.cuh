// What the norms share: rows held in registers, their loads, stores and sums,
// 8-bit output, the plan of threads a row, and the check that outputs are apart.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <initializer_list>

#include "flce_device.cuh"
#include "flce_ops.h"

namespace flce {
namespace {

constexpr int kNormThreads = 256;   // of the kernels for rows past kMaxHeld, and the quantiser
constexpr int kMaxHeld = 16384;     // longest row held in registers (1024 threads x 16 values)

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
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

// ------------------------------------------------------- rows in registers
// A row is a block's (or, with 32 threads a row, a warp's), read once and held
// in registers between the sum of squares and the output.  A thread holds P
// slots of E elements:
//   VEC  H a multiple of E = 16 / sizeof(T): E consecutive columns, slot s of
//        thread t being piece t + s * threads, loaded as 16 bytes where the
//        rows are `aligned`; 16 (bf16) or 32 (float32) neighbouring lanes make a
//        group of 128 columns.  The same threads add the same columns in either
//        case, so that a view's alignment does not change the result;
//   else E = 4 columns 32 apart, a warp and slot being one group: rows of any
//        length, still read whole lines at a time.
template <class T, bool VEC>
struct Slots {
  static constexpr int kE = VEC ? 16 / static_cast<int>(sizeof(T)) : 4;
  static constexpr int kLanes = VEC ? kScaleGroup / kE : 32;  // lanes of a scale group
  __device__ static int first(int s) {  // column of the slot's first element
    const int t = threadIdx.x + s * blockDim.x;
    return VEC ? t * kE : (t >> 5) * kScaleGroup + (t & 31);
  }
  static constexpr int kStep = VEC ? 1 : 32;  // columns between a slot's elements
};

// A slot's elements as loaded (zero past the row), and as floats.
template <class T, bool VEC>
struct Piece {
  static constexpr int kE = Slots<T, VEC>::kE;
  uint32_t w[kE * sizeof(T) / 4];

  __device__ __forceinline__ void load(const T* __restrict__ row, int c, int H, bool aligned) {
    if constexpr (VEC) {
      // H is a multiple of E: a piece lies inside the row or past it
      if (aligned) {
        uint4 p = make_uint4(0, 0, 0, 0);
        if (c < H) p = *reinterpret_cast<const uint4*>(row + c);
        w[0] = p.x, w[1] = p.y, w[2] = p.z, w[3] = p.w;
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      const int k = c + i * Slots<T, VEC>::kStep;
      if constexpr (sizeof(T) == 4) {
        w[i] = k < H ? __float_as_uint(row[k]) : 0u;
      } else {
        const uint32_t u = k < H ? __bfloat16_as_ushort(row[k]) : 0u;
        w[i / 2] = i % 2 ? w[i / 2] | u << 16 : u;
      }
    }
  }
  __device__ __forceinline__ void set(const uint4& p) {
    if constexpr (VEC) w[0] = p.x, w[1] = p.y, w[2] = p.z, w[3] = p.w;
  }
  __device__ __forceinline__ void floats(float (&v)[kE]) const {
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w[i]);
      else v[i] = __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
  }
};

template <class T, bool VEC>
__device__ __forceinline__ void load_slot(const T* __restrict__ row, int c, int H, bool aligned,
                                          float (&v)[Slots<T, VEC>::kE]) {
  Piece<T, VEC> p;
  p.load(row, c, H, aligned);
  p.floats(v);
}

template <class T, bool VEC>
__device__ __forceinline__ void store_slot(T* __restrict__ row, int c, int H, bool aligned,
                                           const float (&v)[Slots<T, VEC>::kE]) {
  constexpr int kE = Slots<T, VEC>::kE;
  if constexpr (VEC) {
    if (c >= H) return;
    if (!aligned) {
#pragma unroll
      for (int i = 0; i < kE; ++i) row[c + i] = from_f<T>(v[i]);
      return;
    }
    uint4 p;
    if constexpr (sizeof(T) == 4) {
      p = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                     __float_as_uint(v[3]));
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<uint32_t*>(&h);
      }
      p = make_uint4(w[0], w[1], w[2], w[3]);
    }
    *reinterpret_cast<uint4*>(row + c) = p;
  } else {
#pragma unroll
    for (int i = 0; i < kE; ++i)
      if (c + 32 * i < H) row[c + 32 * i] = from_f<T>(v[i]);
  }
}

// The weight's elements of a slot (of either type).
template <class T, bool VEC>
__device__ __forceinline__ void load_weight(const void* __restrict__ w, int w_f32, int c, int H,
                                            bool aligned, float (&v)[Slots<T, VEC>::kE]) {
  constexpr int kE = Slots<T, VEC>::kE;
  if constexpr (VEC) {
    if (c >= H) {
#pragma unroll
      for (int i = 0; i < kE; ++i) v[i] = 0.f;
    } else if (!aligned) {
#pragma unroll
      for (int i = 0; i < kE; ++i)
        v[i] = w_f32 ? static_cast<const float*>(w)[c + i]
                     : to_f(static_cast<const __nv_bfloat16*>(w)[c + i]);
    } else if (w_f32) {
#pragma unroll
      for (int i = 0; i < kE / 4; ++i) {
        const float4 p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + c)[i];
        v[4 * i] = p.x;
        v[4 * i + 1] = p.y;
        v[4 * i + 2] = p.z;
        v[4 * i + 3] = p.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kE / 4; ++i) {
        const uint2 p = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(w) + c)[i];
        v[4 * i] = __uint_as_float(p.x << 16);
        v[4 * i + 1] = __uint_as_float(p.x & 0xffff0000u);
        v[4 * i + 2] = __uint_as_float(p.y << 16);
        v[4 * i + 3] = __uint_as_float(p.y & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      const int k = c + 32 * i;
      v[i] = k >= H ? 0.f
             : w_f32 ? static_cast<const float*>(w)[k]
                     : to_f(static_cast<const __nv_bfloat16*>(w)[k]);
    }
  }
}

// Sum over the threads of a row (blockDim.x of them), the same on every one.
// `part`: 2 x 32 floats, used in turn by `phase`, so that one barrier a sum is
// enough.
__device__ __forceinline__ float row_sum(float v, float* part, int phase) {
  v = warp_sum(v);
  if (blockDim.x == 32) return v;
  float* p = part + 32 * phase;
  if ((threadIdx.x & 31) == 0) p[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_sum(lane < static_cast<int>(blockDim.x >> 5) ? p[lane] : 0.f);
}

// A slot's values in 8 bits with their group's scale (every lane of the group calls
// it); qr and scale: the row's.
template <class T, bool VEC>
__device__ __forceinline__ void store_quantized(const float (&v)[Slots<T, VEC>::kE], int c, int H,
                                                bool aligned, uint8_t* __restrict__ qr,
                                                float* __restrict__ scale, int groups) {
  using S = Slots<T, VEC>;
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < S::kE; ++i) a = fmaxf(a, fabsf(v[i]));
#pragma unroll
  for (int o = S::kLanes / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  a = fmaxf(a, kAmaxMin);
  const float inv = kFp8Max / a;
  if constexpr (VEC) {
    uint32_t b[S::kE / 4];
#pragma unroll
    for (int i = 0; i < S::kE / 4; ++i)
      b[i] = pack_e4m3(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
    if (c < H && !aligned) {
#pragma unroll
      for (int i = 0; i < S::kE; ++i) qr[c + i] = static_cast<uint8_t>(b[i / 4] >> 8 * (i % 4));
    } else if (c < H) {
      if constexpr (S::kE == 8) *reinterpret_cast<uint2*>(qr + c) = make_uint2(b[0], b[1]);
      else *reinterpret_cast<uint32_t*>(qr + c) = b[0];
    }
  } else {
#pragma unroll
    for (int i = 0; i < S::kE; ++i)
      if (c + 32 * i < H) qr[c + 32 * i] = to_e4m3(v[i] * inv);
  }
  const int g = c / kScaleGroup;
  if ((threadIdx.x & (S::kLanes - 1)) == 0 && g < groups) scale[g] = a / kFp8Max;
}

__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
}

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1;

// No output of a norm's forward (h_out, `outs`) overlaps an input (x, residual,
// `params`) or another output, but that h_out may be x or residual itself.
inline bool norm_outputs_apart(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                               int64_t N, int64_t H, size_t e, const void* h_out,
                               std::initializer_list<Range> params,
                               std::initializer_list<Range> outs) {
  const Range ins[] = {{x, span_bytes(N, H, ldx, e)}, {residual, span_bytes(N, H, ldr, e)}};
  const Range h = {h_out, span_bytes(N, H, H, e)};
  for (const Range& r : ins) {
    const bool itself = h_out && r.p == h_out &&
                        ((r.p == x && ldx == H) || (r.p == residual && ldr == H));
    if (!itself && ranges_overlap(h, r)) return false;
    for (const Range& o : outs)
      if (ranges_overlap(o, r)) return false;
  }
  for (const Range& r : params) {
    if (ranges_overlap(h, r)) return false;
    for (const Range& o : outs)
      if (ranges_overlap(o, r)) return false;
  }
  for (const Range* o = outs.begin(); o != outs.end(); ++o) {
    if (ranges_overlap(*o, h)) return false;
    for (const Range* p = outs.begin(); p != o; ++p)
      if (ranges_overlap(*o, *p)) return false;
  }
  return true;
}

// How a row of H columns is spread over threads.  Few rows: as many threads as
// there are slots, for latency.  Many: a few slots a thread (16 values), so that
// more rows are in flight on an SM; short rows share a block, a warp each.
struct RowPlan {
  int threads, slots, rows;  // threads a row, slots a thread, rows a block
};
inline RowPlan plan_rows(int64_t N, int64_t H, int elems, bool vec) {
  const int64_t units = vec ? (H + elems - 1) / elems
                            : (H + kScaleGroup - 1) / kScaleGroup * 32;  // slots of a row
  const int most = 16 / elems;  // slots a thread may hold
  const bool few = N <= 304;    // at most two rows an SM
  int slots = 1;
  while (slots < most && units > (few ? 1024 : 32) * slots) slots *= 2;
  int64_t threads = (units + slots - 1) / slots;
  threads = std::max<int64_t>((threads + 31) / 32 * 32, 32);
  return {static_cast<int>(threads), slots, threads == 32 && !few ? 8 : 1};
}

}  // namespace
}  // namespace flce
