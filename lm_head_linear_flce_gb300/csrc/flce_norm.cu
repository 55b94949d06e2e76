// RMS norm with the residual's addition (forward, 8-bit output, backward) and
// the block quantiser.
#include "flce_internal.h"
#include "flce_norm_device.cuh"

namespace flce {
namespace {

constexpr int kDwRows = 64;         // rows per partial sum of dweight beyond that
// Rows the backward has in shared memory or on their way, and its threads on an
// SM.  Measured at 8192 x 3584: bf16 50 us with 1024 threads (54 with 768; three
// rows ahead 67), float32 76 us with 512, whose threads hold 80 registers (97
// with 768, 92 with 1024).
constexpr int kBwdAhead = 2;
template <class T>
constexpr int kBwdThreads = sizeof(T) == 4 ? 512 : 1024;

// Bytes bound it: 16-byte loads of every value once, all of a row's in flight
// at once.  8192 x 3584 with a residual, call after call: bf16 41 us (5.7 TB/s of
// its 8 bytes a value; the measured copy rate is 6.8), float32 71 (6.6); with 8-bit
// output 43 and 66 us; one row with 8-bit output 3 us, launch latency and two trips
// to memory.
template <class T, bool FP8, bool VEC, int P>
__global__ void __launch_bounds__(1024)
    norm_fwd_held_kernel(const T* x, int64_t ldx, const T* residual, int64_t ldr,
                         const void* __restrict__ weight, int w_f32, bool aligned, int64_t N, int H,
                         float eps, T* y, uint8_t* q, float* scale, T* h_out, float* rstd) {
  using S = Slots<T, VEC>;
  __shared__ float part[64];
  griddep_launch_dependents();
  griddep_wait();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (row >= N) return;  // a whole warp (rows share a block only as warps)
  float h[P][S::kE];
#pragma unroll
  for (int s = 0; s < P; ++s) load_slot<T, VEC>(x + row * ldx, S::first(s), H, aligned, h[s]);
  if (residual) {
#pragma unroll
    for (int s = 0; s < P; ++s) {
      float r[S::kE];
      load_slot<T, VEC>(residual + row * ldr, S::first(s), H, aligned, r);
#pragma unroll
      for (int i = 0; i < S::kE; ++i) h[s][i] += r[i];
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int s = 0; s < P; ++s)
#pragma unroll
    for (int i = 0; i < S::kE; ++i) ss = fmaf(h[s][i], h[s][i], ss);
  if (h_out) {
#pragma unroll
    for (int s = 0; s < P; ++s) store_slot<T, VEC>(h_out + row * H, S::first(s), H, aligned, h[s]);
  }
  const float r = rsqrtf(row_sum(ss, part, 0) / static_cast<float>(H) + eps);
  if (rstd && threadIdx.x == 0) rstd[row] = r;
  const int groups = (H + kScaleGroup - 1) / kScaleGroup;
#pragma unroll
  for (int s = 0; s < P; ++s) {
    const int c = S::first(s);
    float w[S::kE];
    load_weight<T, VEC>(weight, w_f32, c, H, aligned, w);
#pragma unroll
    for (int i = 0; i < S::kE; ++i) h[s][i] = h[s][i] * r * w[i];
    if constexpr (!FP8) {
      store_slot<T, VEC>(y + row * H, c, H, aligned, h[s]);
    } else {
      store_quantized<T, VEC>(h[s], c, H, aligned, q + row * H, scale + row * groups, groups);
    }
  }
}

// dx of a row and this block's share of dweight in one pass over dy, h (and
// dh): a block walks rows blockIdx.x, + gridDim.x, ... with the weight and the
// sums of its columns in registers, and leaves one partial sum per column.
//
// AHEAD: the rows' pieces come through shared memory, kBwdAhead rows at a time,
// each thread's own in slots that only it touches: the rows in flight cost no
// registers, and a row is read there twice (sum, then dx) instead of being held
// over the sum.  Without it (rows not aligned to 16 bytes, or too long for the
// slots) a row is loaded when its turn comes.
//
// h is the sum as the forward stored it, in T, where the forward normed the sum
// before it was rounded: keeping that would double what the forward writes and this
// reads.  In bf16 it is a rounding of up to 2^-8 of h in the gradients (8192 x 3584:
// 0.0023 off the gradient in 64 bits, where the outputs' own rounding alone makes
// 0.0017).
//
// 8192 x 3584 with dh, dweight's sum included: bf16 50 us (4.7 TB/s of 8 bytes a
// value), float32 76 us (6.2 TB/s); bf16 spends twice the instructions a byte.
template <class T, bool VEC, int P, int THREADS, bool AHEAD>
__global__ void __launch_bounds__(THREADS, AHEAD && THREADS <= 512 ? kBwdThreads<T> / THREADS : 1)
    norm_bwd_held_kernel(const T* __restrict__ dy, const T* __restrict__ dh,
                         const T* __restrict__ h, int64_t ldh, const void* __restrict__ weight,
                         int w_f32, bool aligned, const float* __restrict__ rstd, int64_t N, int H,
                         T* __restrict__ dx, float* __restrict__ dw_part) {
  using S = Slots<T, VEC>;
  __shared__ float part[64];
  extern __shared__ __align__(16) uint4 ring[];  // [kBwdAhead][3][P][threads of the block]
  const int64_t first = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
  float w[P][S::kE], dw[P][S::kE];
#pragma unroll
  for (int s = 0; s < P; ++s) {
    load_weight<T, VEC>(weight, w_f32, S::first(s), H, aligned, w[s]);
#pragma unroll
    for (int i = 0; i < S::kE; ++i) dw[s][i] = 0.f;
  }
  const float inv_h = 1.f / static_cast<float>(H);
  const bool with_dh = dh && dx;
  const int threads = blockDim.x * blockDim.y, tid = threadIdx.y * blockDim.x + threadIdx.x;
  const auto slot = [&](int stage, int array, int s) {
    return ring + ((stage * 3 + array) * P + s) * threads + tid;
  };
  const auto fetch = [&](int64_t row, int stage) {
    if (row < N) {
#pragma unroll
      for (int s = 0; s < P; ++s) {
        const int c = S::first(s);
        if (c >= H) continue;  // (stays zero)
        copy_async16(slot(stage, 0, s), dy + row * H + c);
        copy_async16(slot(stage, 1, s), h + row * ldh + c);
        if (with_dh) copy_async16(slot(stage, 2, s), dh + row * H + c);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if constexpr (AHEAD) {
    for (int i = 0; i < kBwdAhead * 3 * P; ++i) ring[i * threads + tid] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kBwdAhead; ++i) fetch(first + i * step, i);
  }
  int stage = 0, phase = 0;
  for (int64_t row = first; row < N; row += step, phase ^= 1) {
    const float r = rstd[row];
    Piece<T, VEC> held[3][P];  // without AHEAD
    const auto piece = [&](int array, int s) {
      Piece<T, VEC> p = held[array][s];
      if constexpr (AHEAD) p.set(*slot(stage, array, s));
      return p;
    };
    if constexpr (AHEAD) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kBwdAhead - 1) : "memory");
    } else {
#pragma unroll
      for (int s = 0; s < P; ++s) {
        const int c = S::first(s);
        held[0][s].load(dy + row * H, c, H, aligned);
        held[1][s].load(h + row * ldh, c, H, aligned);
        if (with_dh) held[2][s].load(dh + row * H, c, H, aligned);
      }
    }
    float dot = 0.f;
#pragma unroll
    for (int s = 0; s < P; ++s) {
      float d[S::kE], v[S::kE];
      piece(0, s).floats(d);
      piece(1, s).floats(v);
#pragma unroll
      for (int i = 0; i < S::kE; ++i) {
        const float t = d[i] * v[i];
        dw[s][i] = fmaf(t, r, dw[s][i]);
        dot = fmaf(t, w[s][i], dot);
      }
    }
    if (dx) {
      const float k = r * r * (row_sum(dot, part, phase) * inv_h);
#pragma unroll
      for (int s = 0; s < P; ++s) {
        float d[S::kE], v[S::kE];
        piece(0, s).floats(d);
        piece(1, s).floats(v);
#pragma unroll
        for (int i = 0; i < S::kE; ++i) d[i] = r * (d[i] * w[s][i] - v[i] * k);
        if (with_dh) {
          piece(2, s).floats(v);
#pragma unroll
          for (int i = 0; i < S::kE; ++i) d[i] += v[i];
        }
        store_slot<T, VEC>(dx + row * H, S::first(s), H, aligned, d);
      }
    }
    if constexpr (AHEAD) {
      fetch(row + kBwdAhead * step, stage);
      stage = stage + 1 == kBwdAhead ? 0 : stage + 1;
    }
  }
  if constexpr (AHEAD) asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (!dw_part) return;
#pragma unroll
  for (int s = 0; s < P; ++s) {
    const int c = S::first(s);
    float* p = dw_part + first * H;
#pragma unroll
    for (int i = 0; i < S::kE; ++i)
      if (c + i * S::kStep < H) p[c + i * S::kStep] = dw[s][i];
  }
}

// dweight = the partial sums, added in order: 32 columns a block, each of its
// 32 warps taking every 32nd partial, then the warps in order.
constexpr int kSumWarps = 32;
template <class W>
__global__ void __launch_bounds__(32 * kSumWarps)
    norm_dw_sum_kernel(const float* __restrict__ part, int64_t parts, int H, W* __restrict__ dw) {
  __shared__ float sums[kSumWarps][32];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < H) {
#pragma unroll 8
    for (int64_t p = warp; p < parts; p += kSumWarps) s += part[p * H + c];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= H) return;
  for (int k = 1; k < kSumWarps; ++k) s += sums[k][lane];
  dw[c] = from_f<W>(s);
}

// ----------------------------------------------------- small backwards
// dx needs a row's sum, dweight a column's, and neither needs the other: where
// the inputs stay in L2, one launch does both, the first `row_blocks` blocks rows
// (`tpr` threads each, 8 values a thread) and the others 16 columns each, over all
// rows.  Latency bounds it: 64 x 4096 bf16 4.5 us against 6.5 for the two launches
// above, 2048 x 64 5.1 against 7.2, 512 x 4096 13.3 against 14.6.  Where the rows
// are many or long for its two readings it is the slower kernel: 1021 x 1001 float32
// 8.3 against 6.9 (but 13.4 against 15.5 us a forward and backward where the host
// launches them one by one), 2048 x 1024 bf16 14.4 against 10.6, 256 x 8192 17.4
// against 13.7.
constexpr int kSmallThreads = 1024;
constexpr int kSmallValues = 8;
constexpr int kSmallCols = 16;
template <class T>
__global__ void __launch_bounds__(kSmallThreads)
    norm_bwd_small_kernel(const T* __restrict__ dy, const T* __restrict__ dh,
                          const T* __restrict__ h, int64_t ldh, const void* __restrict__ weight,
                          int w_f32, const float* __restrict__ rstd, int N, int H,
                          T* __restrict__ dx, void* __restrict__ dw, int row_blocks, int tpr) {
  __shared__ float part[kSmallThreads / 32][33];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (static_cast<int>(blockIdx.x) < row_blocks) {
    const int rows = kSmallThreads / tpr, r = threadIdx.x / tpr, t = threadIdx.x % tpr;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * rows + r;
    const bool live = r < rows && row < N;
    float g[kSmallValues], v[kSmallValues], e[kSmallValues], dot = 0.f;
#pragma unroll
    for (int i = 0; i < kSmallValues; ++i) {
      const int c = t + i * tpr;
      const bool in = live && c < H;
      g[i] = in ? to_f(dy[row * H + c]) : 0.f;
      v[i] = in ? to_f(h[row * ldh + c]) : 0.f;
      e[i] = in && dh ? to_f(dh[row * H + c]) : 0.f;
      const float w = !in     ? 0.f
                      : w_f32 ? static_cast<const float*>(weight)[c]
                              : to_f(static_cast<const __nv_bfloat16*>(weight)[c]);
      g[i] *= w;
      dot = fmaf(g[i], v[i], dot);
    }
    dot = warp_sum(dot);
    if (lane == 0) part[0][warp] = dot;
    __syncthreads();
    if (!live) return;
    dot = 0.f;
    for (int w = 0; w < tpr / 32; ++w) dot += part[0][r * (tpr / 32) + w];
    const float s = rstd[row], k = s * s * dot / static_cast<float>(H);
#pragma unroll
    for (int i = 0; i < kSmallValues; ++i) {
      const int c = t + i * tpr;
      if (c < H) dx[row * H + c] = from_f<T>(s * (g[i] - v[i] * k) + e[i]);
    }
    return;
  }
  // a half warp a row: 64 rows at a time
  const int c = (blockIdx.x - row_blocks) * kSmallCols + (lane & (kSmallCols - 1));
  float s = 0.f;
  if (c < H) {
#pragma unroll 8
    for (int n = threadIdx.x / kSmallCols; n < N; n += kSmallThreads / kSmallCols)
      s += to_f(dy[static_cast<int64_t>(n) * H + c]) * to_f(h[n * ldh + c]) * rstd[n];
  }
  s += __shfl_xor_sync(0xffffffffu, s, kSmallCols);
  part[warp][lane] = s;
  __syncthreads();
  if (threadIdx.x >= kSmallCols || c >= H) return;
  for (int w = 1; w < kSmallThreads / 32; ++w) s += part[w][lane];
  if (w_f32) static_cast<float*>(dw)[c] = s;
  else static_cast<__nv_bfloat16*>(dw)[c] = from_f<__nv_bfloat16>(s);
}

// ----------------------------------------------------- rows past kMaxHeld
// A block per row; a warp per group of 128 columns in the second pass, where a
// thread reads an element before it writes the sum in its place (h_out may be x or
// residual).
template <class T, class W, bool FP8>
__global__ void __launch_bounds__(kNormThreads)
    norm_fwd_kernel(const T* x, int64_t ldx, const T* residual, int64_t ldr,
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

// Partial sums of dweight over kDwRows rows.
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

// 128 x 128 blocks of a matrix with 16-byte rows: a thread block reads a block
// once into registers (8 values of bf16, 4 of float32 a load, all in flight),
// takes the maximum and writes it.  Bound by bytes, 2 + 1 a bf16 value: 152064 x
// 3584 in 248 us, 6.6 TB/s, with three blocks an SM (two: 288 us); float32 411 us,
// 6.6 TB/s.
template <class T>
__global__ void __launch_bounds__(kNormThreads, 3)
    quantize_tile_kernel(const T* __restrict__ x, int64_t ldx, int64_t R, int K,
                         uint8_t* __restrict__ q, float* __restrict__ scale) {
  constexpr int kE = 16 / static_cast<int>(sizeof(T));
  constexpr int kCols = kScaleGroup / kE;             // pieces of a row of the block
  constexpr int kRowStep = kNormThreads / kCols;
  constexpr int kN = kScaleGroup / kRowStep;          // pieces a thread holds
  __shared__ float part[kNormThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kScaleGroup + threadIdx.x / kCols;
  const int c = blockIdx.y * kScaleGroup + threadIdx.x % kCols * kE;
  uint4 v[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int64_t r = r0 + i * kRowStep;
    v[i] = make_uint4(0, 0, 0, 0);
    if (r < R && c < K) v[i] = *reinterpret_cast<const uint4*>(x + r * ldx + c);
  }
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (sizeof(T) == 4) {
        a = fmaxf(a, fabsf(__uint_as_float(w[k])));
      } else {
        a = fmaxf(a, fabsf(__uint_as_float(w[k] << 16)));
        a = fmaxf(a, fabsf(__uint_as_float(w[k] & 0xffff0000u)));
      }
    }
  }
  a = warp_max(a);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kNormThreads / 32; ++w) a = fmaxf(a, part[w]);
  a = fmaxf(a, kAmaxMin);
  const float inv = kFp8Max / a;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int64_t r = r0 + i * kRowStep;
    if (r >= R || c >= K) continue;
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<uint32_t*>(q + r * K + c) =
          pack_e4m3(__uint_as_float(w[0]) * inv, __uint_as_float(w[1]) * inv,
                    __uint_as_float(w[2]) * inv, __uint_as_float(w[3]) * inv);
    } else {
      uint32_t o[2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        o[k] = pack_e4m3(__uint_as_float(w[2 * k] << 16) * inv,
                         __uint_as_float(w[2 * k] & 0xffff0000u) * inv,
                         __uint_as_float(w[2 * k + 1] << 16) * inv,
                         __uint_as_float(w[2 * k + 1] & 0xffff0000u) * inv);
      *reinterpret_cast<uint2*>(q + r * K + c) = make_uint2(o[0], o[1]);
    }
  }
  if (threadIdx.x == 0)
    scale[static_cast<int64_t>(blockIdx.x) * gridDim.y + blockIdx.y] = a / kFp8Max;
}

// 1 x 128 groups: a half warp (bf16) or warp (float32, or unaligned rows, 4
// columns 32 apart a lane) per group; 152064 x 3584 bf16 in 312 us, 5.2 TB/s,
// float32 571 us, 4.8 TB/s.
template <class T, bool VEC>
__global__ void __launch_bounds__(kNormThreads)
    quantize_rows_kernel(const T* __restrict__ x, int64_t ldx, int64_t R, int K,
                         uint8_t* __restrict__ q, float* __restrict__ scale) {
  using S = Slots<T, VEC>;
  constexpr int kPer = kNormThreads / S::kLanes;  // groups per thread block
  griddep_launch_dependents();
  griddep_wait();
  const int groups = (K + kScaleGroup - 1) / kScaleGroup;
  const uint32_t u = blockIdx.x * kPer + threadIdx.x / S::kLanes;  // (the host bounds their number)
  const int64_t row = u / static_cast<uint32_t>(groups);
  const int g = static_cast<int>(u % static_cast<uint32_t>(groups));
  const int l = threadIdx.x % S::kLanes;
  // a group past the last row takes part in the shuffles with zeros
  const int c = row < R ? g * kScaleGroup + (VEC ? l * S::kE : l) : K;
  float v[S::kE];
  load_slot<T, VEC>(x + (row < R ? row : 0) * ldx, c, K, true, v);
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < S::kE; ++i) a = fmaxf(a, fabsf(v[i]));
#pragma unroll
  for (int o = S::kLanes / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  a = fmaxf(a, kAmaxMin);
  const float inv = kFp8Max / a;
  if (row >= R) return;
  uint8_t* qr = q + row * K;
  if constexpr (VEC) {
    if (c < K) {
      uint32_t b[S::kE / 4];
#pragma unroll
      for (int i = 0; i < S::kE / 4; ++i)
        b[i] = pack_e4m3(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv,
                         v[4 * i + 3] * inv);
      if constexpr (S::kE == 8) *reinterpret_cast<uint2*>(qr + c) = make_uint2(b[0], b[1]);
      else *reinterpret_cast<uint32_t*>(qr + c) = b[0];
    }
  } else {
#pragma unroll
    for (int i = 0; i < S::kE; ++i)
      if (c + 32 * i < K) qr[c + 32 * i] = to_e4m3(v[i] * inv);
  }
  if (l == 0) scale[u] = a / kFp8Max;
}

// 128 x 128 blocks of unaligned rows, read twice, the second time from L2:
// 152064 x 3583 bf16 in 642 us (held in registers, two bytes a load: 877).
template <class T>
__global__ void __launch_bounds__(kNormThreads)
    quantize_kernel(const T* __restrict__ x, int64_t ldx, int64_t R, int K,
                    uint8_t* __restrict__ q, float* __restrict__ scale) {
  __shared__ float part[kNormThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kScaleGroup;
  const int c = blockIdx.y * kScaleGroup + (threadIdx.x & (kScaleGroup - 1));
  const int64_t r1 = min(R, r0 + kScaleGroup);
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

// The backward's threads a row: up to 256 before a thread takes more slots.
RowPlan plan_bwd(int64_t N, int64_t H, int elems, bool vec) {
  RowPlan p = plan_rows(N, H, elems, vec);
  while (p.slots > 1 && p.rows == 1 && p.threads <= 128) {
    p.slots /= 2;
    p.threads *= 2;
  }
  return p;
}

// Partial sums of dweight: a block's rows at a time.  A fixed number, so that
// the order of additions depends on the sizes and the type alone: the blocks
// that 152 SMs hold at once.
int64_t held_parts(int64_t N, const RowPlan& p, size_t elem_bytes) {
  const int threads = p.threads * p.rows;
  const int block = threads <= 256 ? 256 : threads <= 512 ? 512 : 1024;
  const int per_sm = std::max((elem_bytes == 4 ? kBwdThreads<float> : kBwdThreads<__nv_bfloat16>) /
                                  block, 1);
  return std::min<int64_t>((N + p.rows - 1) / p.rows, 152 * per_sm) * p.rows;
}
int64_t dw_parts(int64_t N, int64_t H) {
  if (H > kMaxHeld) return (N + kDwRows - 1) / kDwRows;
  // whichever plan the call's types lead to
  return std::max({held_parts(N, plan_bwd(N, H, 8, true), 2),
                   held_parts(N, plan_bwd(N, H, 4, true), 4),
                   held_parts(N, plan_bwd(N, H, 4, false), 2)});
}

struct FwdArgs {
  const void* x;
  int64_t ldx;
  const void* residual;
  int64_t ldr;
  const void* weight;
  int w_f32;
  int64_t N;
  int H;
  float eps;
  void* y;
  void* q;
  float* scale;
  void* h_out;
  float* rstd;
};

template <class T, bool FP8, bool VEC, int P>
cudaError_t launch_fwd_held(const RowPlan& p, bool aligned, const FwdArgs& a, cudaStream_t s) {
  const unsigned blocks = static_cast<unsigned>((a.N + p.rows - 1) / p.rows);
  return launch_overlapped(
      norm_fwd_held_kernel<T, FP8, VEC, P>, dim3(blocks), dim3(p.threads, p.rows), 0, s, 1,
      static_cast<const T*>(a.x), a.ldx, static_cast<const T*>(a.residual), a.ldr, a.weight,
      a.w_f32, aligned, a.N, a.H, a.eps, static_cast<T*>(a.y), static_cast<uint8_t*>(a.q), a.scale,
      static_cast<T*>(a.h_out), a.rstd);
}

// Whether every row's pieces are 16-byte aligned.
template <class T>
bool fwd_aligned(const FwdArgs& a) {
  const int e = 16 / sizeof(T);
  return a.ldx % e == 0 && a.ldr % e == 0 && aligned_to(a.x, 16) &&
         aligned_to(a.residual, 16) && aligned_to(a.weight, 16) && aligned_to(a.y, 16) &&
         aligned_to(a.q, 8) && aligned_to(a.h_out, 16);
}

template <class T, bool FP8>
cudaError_t run_norm_fwd(const FwdArgs& a, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (a.H > kMaxHeld) {
    const auto launch = [&](auto w) {
      using W = decltype(w);
      norm_fwd_kernel<T, W, FP8><<<static_cast<unsigned>(a.N), kNormThreads, 0, s>>>(
          static_cast<const T*>(a.x), a.ldx, static_cast<const T*>(a.residual), a.ldr,
          static_cast<const W*>(a.weight), a.H, a.eps, static_cast<T*>(a.y),
          static_cast<uint8_t*>(a.q), a.scale, static_cast<T*>(a.h_out), a.rstd);
    };
    if (a.w_f32) launch(float{});
    else launch(__nv_bfloat16{});
  } else if (a.H % Slots<T, true>::kE == 0) {
    constexpr int kE = Slots<T, true>::kE;
    const bool al = fwd_aligned<T>(a);
    const RowPlan p = plan_rows(a.N, a.H, kE, true);
    if (p.slots == 1) e = launch_fwd_held<T, FP8, true, 1>(p, al, a, s);
    else if (p.slots == 2) e = launch_fwd_held<T, FP8, true, 2>(p, al, a, s);
    else if constexpr (kE == 4) e = launch_fwd_held<T, FP8, true, 4>(p, al, a, s);
  } else {
    const RowPlan p = plan_rows(a.N, a.H, 4, false);
    if (p.slots == 1) e = launch_fwd_held<T, FP8, false, 1>(p, false, a, s);
    else if (p.slots == 2) e = launch_fwd_held<T, FP8, false, 2>(p, false, a, s);
    else e = launch_fwd_held<T, FP8, false, 4>(p, false, a, s);
  }
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

struct BwdArgsN {
  const void* dy;
  const void* dh;
  const void* h;
  int64_t ldh;
  const void* weight;
  int w_f32;
  const float* rstd;
  int64_t N;
  int H;
  void* dx;
  void* dweight;
  float* part;
};

template <class T, bool VEC, int P>
cudaError_t launch_bwd_held(const RowPlan& p, bool aligned, int64_t parts,
                            const BwdArgsN& a, cudaStream_t s) {
  constexpr int kMost = 200 * 1024;
  const int threads = p.threads * p.rows, ring = kBwdAhead * 3 * P * threads * 16;
  const auto launch = [&](auto* k, int smem) {
    // A plain launch, and no early start for what follows: blocks that wait here
    // take shared memory from the kernel before them, and blocks of the sum that
    // wait take it from this one (8192 x 3584 bf16, a step: 91.1 us, plain 89.2).
    k<<<dim3(static_cast<unsigned>(parts / p.rows)), dim3(p.threads, p.rows), smem, s>>>(
        static_cast<const T*>(a.dy), static_cast<const T*>(a.dh), static_cast<const T*>(a.h),
        a.ldh, a.weight, a.w_f32, aligned, a.rstd, a.N, a.H, static_cast<T*>(a.dx),
        a.dweight ? a.part : static_cast<float*>(nullptr));
    return cudaGetLastError();
  };
  if constexpr (VEC) {
    if (aligned && ring <= kMost) {
      auto* k = threads <= 256   ? norm_bwd_held_kernel<T, VEC, P, 256, true>
                : threads <= 512 ? norm_bwd_held_kernel<T, VEC, P, 512, true>
                                 : norm_bwd_held_kernel<T, VEC, P, 1024, true>;
      static SmemLimit limits[3];  // one for each of them
      const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), kMost,
                                       &limits[threads <= 256 ? 0 : threads <= 512 ? 1 : 2]);
      return e != cudaSuccess ? e : launch(k, ring);
    }
  }
  return threads <= 512 ? launch(norm_bwd_held_kernel<T, VEC, P, 512, false>, 0)
                        : launch(norm_bwd_held_kernel<T, VEC, P, 1024, false>, 0);
}

// Rows that norm_bwd_small_kernel takes: a column's block adds at most 64 of them
// a warp, and 2^21 values are read twice from L2.  (Times on both sides: above.  By
// the GPU's time alone the limit would be lower.)
bool small_bwd(int64_t N, int64_t H) {
  return N <= 2048 && H <= kSmallThreads * kSmallValues && N * H <= int64_t{1} << 21;
}

template <class T>
cudaError_t run_norm_bwd(const BwdArgsN& a, cudaStream_t s) {
  if (small_bwd(a.N, a.H)) {
    const int tpr = (((a.H + kSmallValues - 1) / kSmallValues) + 31) / 32 * 32;
    const int rows = kSmallThreads / tpr;
    const int row_blocks = a.dx ? static_cast<int>((a.N + rows - 1) / rows) : 0;
    const int blocks = row_blocks + (a.dweight ? (a.H + kSmallCols - 1) / kSmallCols : 0);
    if (blocks == 0) return cudaSuccess;
    const cudaError_t e = launch_overlapped(
        norm_bwd_small_kernel<T>, dim3(blocks), dim3(kSmallThreads), 0, s, 1,
        static_cast<const T*>(a.dy), static_cast<const T*>(a.dh), static_cast<const T*>(a.h),
        a.ldh, a.weight, a.w_f32, a.rstd, static_cast<int>(a.N), a.H, static_cast<T*>(a.dx),
        a.dweight, row_blocks, tpr);
    note_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
  }
  int64_t parts = 0;
  if (a.N > 0 && a.H > kMaxHeld) {
    parts = dw_parts(a.N, a.H);
    const unsigned cols = static_cast<unsigned>((a.H + kNormThreads - 1) / kNormThreads);
    const T* dy = static_cast<const T*>(a.dy);
    const T* h = static_cast<const T*>(a.h);
    if (a.dx) {
      const auto launch = [&](auto w) {
        using W = decltype(w);
        norm_bwd_dx_kernel<T, W><<<static_cast<unsigned>(a.N), kNormThreads, 0, s>>>(
            dy, static_cast<const T*>(a.dh), h, a.ldh, static_cast<const W*>(a.weight), a.rstd,
            a.H, static_cast<T*>(a.dx));
      };
      if (a.w_f32) launch(float{});
      else launch(__nv_bfloat16{});
      note_launch();
    }
    if (a.dweight) {
      norm_bwd_dw_kernel<T><<<dim3(static_cast<unsigned>(parts), cols), kNormThreads, 0, s>>>(
          dy, h, a.ldh, a.rstd, a.N, a.H, a.part);
      note_launch();
    }
  } else if (a.N > 0 && (a.dx || a.dweight)) {
    constexpr int kE = Slots<T, true>::kE;
    const bool vec = a.H % kE == 0;
    const bool al = a.ldh % kE == 0 && aligned_to(a.dy, 16) && aligned_to(a.dh, 16) &&
                    aligned_to(a.h, 16) && aligned_to(a.weight, 16) && aligned_to(a.dx, 16);
    const RowPlan p = plan_bwd(a.N, a.H, vec ? kE : 4, vec);
    parts = held_parts(a.N, p, sizeof(T));
    cudaError_t e = cudaSuccess;
    if (vec) {
      if (p.slots == 1) e = launch_bwd_held<T, true, 1>(p, al, parts, a, s);
      else if (p.slots == 2) e = launch_bwd_held<T, true, 2>(p, al, parts, a, s);
      else if constexpr (kE == 4) e = launch_bwd_held<T, true, 4>(p, al, parts, a, s);
    } else {
      if (p.slots == 1) e = launch_bwd_held<T, false, 1>(p, al, parts, a, s);
      else if (p.slots == 2) e = launch_bwd_held<T, false, 2>(p, al, parts, a, s);
      else e = launch_bwd_held<T, false, 4>(p, al, parts, a, s);
    }
    if (e != cudaSuccess) return e;
    note_launch();
  }
  if (a.dweight) {
    const unsigned blocks = static_cast<unsigned>((a.H + 31) / 32);
    const dim3 block(32 * kSumWarps);
    const cudaError_t e =
        a.w_f32 ? launch_overlapped(norm_dw_sum_kernel<float>, dim3(blocks), block, 0, s, 1, a.part,
                                    parts, a.H, static_cast<float*>(a.dweight))
                : launch_overlapped(norm_dw_sum_kernel<__nv_bfloat16>, dim3(blocks), block, 0, s, 1,
                                    a.part, parts, a.H, static_cast<__nv_bfloat16*>(a.dweight));
    if (e != cudaSuccess) return e;
    note_launch();
  }
  return cudaGetLastError();
}

template <class T>
cudaError_t run_quantize(const void* xp, int64_t ldx, int64_t R, int64_t K64, int block_rows,
                         void* qp, float* scale, cudaStream_t s) {
  const T* x = static_cast<const T*>(xp);
  auto* q = static_cast<uint8_t*>(qp);
  const int K = static_cast<int>(K64), e = 16 / sizeof(T);
  const int64_t gk = (K + kScaleGroup - 1) / kScaleGroup;
  const bool vec = K % e == 0 && ldx % e == 0 && aligned_to(x, 16) && aligned_to(q, 8);
  if (block_rows == 1) {
    const int lanes = vec ? Slots<T, true>::kLanes : Slots<T, false>::kLanes;
    const int per = kNormThreads / lanes;
    const auto blocks = static_cast<unsigned>((R * gk + per - 1) / per);
    return launch_overlapped(vec ? quantize_rows_kernel<T, true> : quantize_rows_kernel<T, false>,
                             dim3(blocks), dim3(kNormThreads), 0, s, 1, x, ldx, R, K, q, scale);
  }
  const dim3 grid(static_cast<unsigned>((R + kScaleGroup - 1) / kScaleGroup),
                  static_cast<unsigned>(gk));
  return launch_overlapped(vec ? quantize_tile_kernel<T> : quantize_kernel<T>, grid,
                           dim3(kNormThreads), 0, s, 1, x, ldx, R, K, q, scale);
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

flce_status flce_rms_norm_forward(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                                  const void* weight, int64_t N, int64_t H, float eps,
                                  flce_dtype dtype, flce_dtype weight_dtype, void* y, void* h_out,
                                  float* rstd, flce_stream_t stream) {
  OpRange range("flce_rms_norm_forward");
  flce_status st = check_norm(x, ldx, residual, ldr, weight, N, H, dtype, weight_dtype);
  if (st != FLCE_OK || N == 0) return st;
  const size_t e = dtype_bytes(dtype);
  if (!y || !aligned_to(y, e) || !aligned_to(h_out, e) || !aligned_to(rstd, 4))
    return FLCE_ERR_INVALID_ARG;
  if (!norm_outputs_apart(x, ldx, residual, ldr, N, H, e, h_out,
                          {{weight, static_cast<size_t>(H) * dtype_bytes(weight_dtype)}},
                          {{y, span_bytes(N, H, H, e)}, {rstd, static_cast<size_t>(N) * 4}}))
    return FLCE_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = check_device(&sms)) != FLCE_OK) return st;
  const FwdArgs a = {x, ldx, residual, ldr, weight, weight_dtype == FLCE_F32, N,
                     static_cast<int>(H), eps, y, nullptr, nullptr, h_out, rstd};
  const auto s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t err = dtype == FLCE_BF16 ? run_norm_fwd<__nv_bfloat16, false>(a, s)
                                             : run_norm_fwd<float, false>(a, s);
  return err == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

flce_status flce_rms_norm_fp8(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                              const void* weight, int64_t N, int64_t H, float eps,
                              flce_dtype dtype, flce_dtype weight_dtype, void* q, float* scale,
                              void* h_out, flce_stream_t stream) {
  OpRange range("flce_rms_norm_fp8");
  flce_status st = check_norm(x, ldx, residual, ldr, weight, N, H, dtype, weight_dtype);
  if (st != FLCE_OK || N == 0) return st;
  const size_t e = dtype_bytes(dtype);
  if (!q || !scale || !aligned_to(h_out, e) || !aligned_to(scale, 4)) return FLCE_ERR_INVALID_ARG;
  const int64_t groups = (H + kScaleGroup - 1) / kScaleGroup;
  if (!norm_outputs_apart(x, ldx, residual, ldr, N, H, e, h_out,
                          {{weight, static_cast<size_t>(H) * dtype_bytes(weight_dtype)}},
                          {{q, span_bytes(N, H, H, 1)}, {scale, span_bytes(N, groups, groups, 4)}}))
    return FLCE_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = check_device(&sms)) != FLCE_OK) return st;
  const FwdArgs a = {x, ldx, residual, ldr, weight, weight_dtype == FLCE_F32, N,
                     static_cast<int>(H), eps, nullptr, q, scale, h_out, nullptr};
  const auto s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t err = dtype == FLCE_BF16 ? run_norm_fwd<__nv_bfloat16, true>(a, s)
                                             : run_norm_fwd<float, true>(a, s);
  return err == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

size_t flce_rms_norm_workspace_size(int64_t N, int64_t H) {
  if (N < 0 || H <= 0 || H > kMaxRowElems || N > kMaxRows) return 0;
  const size_t n = static_cast<size_t>(dw_parts(N, H)) * static_cast<size_t>(H) * 4;
  return std::max<size_t>((n + 255) / 256 * 256, 256);
}

flce_status flce_rms_norm_backward(const void* dy, const void* dh, const void* h, int64_t ldh,
                                   const void* weight, const float* rstd, int64_t N, int64_t H,
                                   flce_dtype dtype, flce_dtype weight_dtype, void* dx,
                                   void* dweight, void* workspace, size_t workspace_bytes,
                                   flce_stream_t stream) {
  OpRange range("flce_rms_norm_backward");
  if (N < 0 || H <= 0 || !valid_dtype(dtype) || !valid_dtype(weight_dtype))
    return FLCE_ERR_INVALID_ARG;
  if (H > kMaxRowElems || N > kMaxRows) return FLCE_ERR_UNSUPPORTED_SHAPE;
  if (N > 0 && (!dy || !h || !weight || !rstd || ldh < H)) return FLCE_ERR_INVALID_ARG;
  const size_t e = dtype_bytes(dtype), we = dtype_bytes(weight_dtype);
  if (!aligned_to(dy, e) || !aligned_to(dh, e) || !aligned_to(h, e) || !aligned_to(dx, e) ||
      !aligned_to(weight, we) || !aligned_to(dweight, we) || !aligned_to(rstd, 4))
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
  const BwdArgsN a = {dy, dh, h, ldh, weight, weight_dtype == FLCE_F32, rstd, N,
                      static_cast<int>(H), dx, dweight, static_cast<float*>(workspace)};
  const cudaError_t err =
      dtype == FLCE_BF16 ? run_norm_bwd<__nv_bfloat16>(a, s) : run_norm_bwd<float>(a, s);
  return err == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

flce_status flce_quantize_fp8(const void* x, int64_t ldx, int64_t R, int64_t K, flce_dtype dtype,
                              int block_rows, void* q, float* scale, flce_stream_t stream) {
  OpRange range("flce_quantize_fp8");
  if (R < 0 || K <= 0 || !valid_dtype(dtype) || (block_rows != 1 && block_rows != kScaleGroup))
    return FLCE_ERR_INVALID_ARG;
  if (K > kMaxRowElems || R > kMaxRows) return FLCE_ERR_UNSUPPORTED_SHAPE;
  if (R == 0) return FLCE_OK;
  const size_t e = dtype_bytes(dtype);
  if (!x || !q || !scale || ldx < K || !aligned_to(x, e) || !aligned_to(scale, 4))
    return FLCE_ERR_INVALID_ARG;
  const int64_t gr = (R + block_rows - 1) / block_rows, gk = (K + kScaleGroup - 1) / kScaleGroup;
  const Range xr = {x, span_bytes(R, K, ldx, e)}, qr = {q, span_bytes(R, K, K, 1)},
              sr = {scale, span_bytes(gr, gk, gk, 4)};
  if (ranges_overlap(xr, qr) || ranges_overlap(xr, sr) || ranges_overlap(qr, sr))
    return FLCE_ERR_INVALID_ARG;
  int sms = 0;
  const flce_status st = check_device(&sms);
  if (st != FLCE_OK) return st;
  const auto s = reinterpret_cast<cudaStream_t>(stream);
  if (block_rows == 1 && gr * gk > kMaxRows) return FLCE_ERR_UNSUPPORTED_SHAPE;
  const cudaError_t err =
      dtype == FLCE_BF16 ? run_quantize<__nv_bfloat16>(x, ldx, R, K, block_rows, q, scale, s)
                         : run_quantize<float>(x, ldx, R, K, block_rows, q, scale, s);
  note_launch();
  return err == cudaSuccess && cudaGetLastError() == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

}  // extern "C"
