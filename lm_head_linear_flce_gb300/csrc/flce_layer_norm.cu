// Layer norm with the residual's addition (forward, 8-bit output, backward).
#include <type_traits>

#include "flce_internal.h"
#include "flce_norm_device.cuh"
#include "flce_pairs.cuh"

namespace flce {
namespace {

constexpr int kLnDwRows = 64;  // rows per partial sum of dweight and dbias past kMaxHeld

template <int E>
__device__ __forceinline__ void to_pairs(const float (&v)[E], F2 (&p)[E / 2]) {
#pragma unroll
  for (int i = 0; i < E / 2; ++i) p[i] = pack2(v[2 * i], v[2 * i + 1]);
}
template <int E>
__device__ __forceinline__ void from_pairs(const F2 (&p)[E / 2], float (&v)[E]) {
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    const float2 f = unpack2(p[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// Sums of two values over the warp, in five exchanges: the first half's lanes end with
// the first one's, the others with the second's.
__device__ __forceinline__ float warp_sum_halves(float a, float b) {
  const bool low = (threadIdx.x & 16) == 0;
  float v = (low ? a : b) + __shfl_xor_sync(0xffffffffu, low ? b : a, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Sums of two values over the threads of a row, the same on every one.  `part`: the
// row's 2 x 32 pairs, used in turn by `phase`.  A block's rows wait for themselves
// alone, each at a barrier of its own.
__device__ __forceinline__ float2 row_sum2(float2 v, float (*part)[32][2], int phase) {
  const float s = warp_sum_halves(v.x, v.y);
  const int lane = threadIdx.x & 31;
  if (blockDim.x == 32)
    return make_float2(__shfl_sync(0xffffffffu, s, 0), __shfl_sync(0xffffffffu, s, 16));
  float(*p)[2] = part[phase];
  if ((lane & 15) == 0) p[threadIdx.x >> 5][lane >> 4] = s;
  asm volatile("bar.sync %0, %1;" ::"r"(threadIdx.y + 1), "r"(blockDim.x) : "memory");
  // both sums again in five exchanges where sixteen lanes hold the warps' parts
  const int warps = static_cast<int>(blockDim.x >> 5);
  if (warps <= 16) {
    const int k = lane & 15;
    float t = k < warps ? p[k][lane >> 4] : 0.f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    const float u = __shfl_xor_sync(0xffffffffu, t, 16);
    return lane < 16 ? make_float2(t, u) : make_float2(u, t);
  }
  v = lane < warps ? *reinterpret_cast<const float2*>(p[lane]) : make_float2(0.f, 0.f);
  return make_float2(warp_sum(v.x), warp_sum(v.y));
}

// The elements of a slot that lie in the row.
template <class T, bool VEC>
__device__ __forceinline__ bool in_row(int c, int i, int H) {
  return VEC ? c < H : c + 32 * i < H;
}

// A parameter's elements of a slot, `missing` where there is none, 0 past the row.
template <class T, bool VEC>
__device__ __forceinline__ void load_param(const void* __restrict__ w, int w_f32, float missing,
                                           int c, int H, bool aligned,
                                           float (&v)[Slots<T, VEC>::kE]) {
  if (w) {
    load_weight<T, VEC>(w, w_f32, c, H, aligned, v);
  } else {
#pragma unroll
    for (int i = 0; i < Slots<T, VEC>::kE; ++i) v[i] = in_row<T, VEC>(c, i, H) ? missing : 0.f;
  }
}

// A row in registers between its sums and the output, so that it is read once.
//
// Mean and variance in one meeting of the row's warps.  Each warp has its own mean m_w,
// and over its n_w values the sums d_w of what is left of them, h - m_w (m_w's
// rounding), and q_w of its squares; with m_0 the first warp's mean,
//     mean = m_0 + sum_w (n_w (m_w - m_0) + d_w) / H = m_0 + m_1
//     H variance = sum_w q_w + 2 (m_w - mean) d_w + n_w (m_w - mean)^2
// Nothing is lost where the mean is large: only differences are squared or added (h^2 -
// mean^2 would lose the variance of such rows), and h - mean is (h - m_w) + (m_w - mean).
//
// PLAIN: weight and bias there and of x's type, and with VEC 16-byte aligned rows.
//
// 8192 x 3584 bf16 with a residual 43 us (235 MB, 5.4 TB/s; a copy of as much 43), 16384 x
// 2048 float32 78 (537 MB, 6.9 TB/s): memory.  One row 1.9 us in a graph: a launch and two
// trips to memory.  Two values an instruction were slower here, and so was a second block
// barrier (mean, then squares).
template <class T, bool FP8, bool VEC, int P, bool PLAIN>
__global__ void __launch_bounds__(1024)
    ln_fwd_held_kernel(const T* x, int64_t ldx, const T* residual, int64_t ldr,
                       const void* __restrict__ weight, const void* __restrict__ bias, int w_f32,
                       bool al, int64_t N, int H, float inv_h, float eps, T* y, uint8_t* q,
                       float* scale, T* h_out, float* mean, float* rstd) {
  using S = Slots<T, VEC>;
  constexpr int kE = S::kE;
  __shared__ float4 part[32];
  griddep_launch_dependents();
  griddep_wait();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (row >= N) return;  // a whole warp (rows share a block only as warps)
  const bool aligned = PLAIN || al;
  const int lane = threadIdx.x & 31;
  float h[P][kE];
#pragma unroll
  for (int s = 0; s < P; ++s) load_slot<T, VEC>(x + row * ldx, S::first(s), H, aligned, h[s]);
  if (residual) {
#pragma unroll
    for (int s = 0; s < P; ++s) {
      float r[kE];
      load_slot<T, VEC>(residual + row * ldr, S::first(s), H, aligned, r);
#pragma unroll
      for (int i = 0; i < kE; ++i) h[s][i] += r[i];
    }
  }
  // columns from the warp's first one in a slot to the row's end
  const auto left = [&](int s) { return H - (S::first(s) - lane * (VEC ? kE : 1)); };
  float sum = 0.f;
  int count = 0;  // the warp's values
#pragma unroll
  for (int s = 0; s < P; ++s) {
#pragma unroll
    for (int i = 0; i < kE; ++i) sum += h[s][i];
    count += min(max(left(s), 0), 32 * kE);
  }
  if (h_out) {
#pragma unroll
    for (int s = 0; s < P; ++s) store_slot<T, VEC>(h_out + row * H, S::first(s), H, aligned, h[s]);
  }
  float4 own;  // n_w, m_w, d_w, q_w
  own.x = static_cast<float>(count);
  own.y = count ? __fdividef(warp_sum(sum), own.x) : 0.f;  // (d_w takes up what is lost here)
  own.z = own.w = 0.f;
#pragma unroll
  for (int s = 0; s < P; ++s) {  // h is h - m_w from here on (0 past the row)
    const float m = S::first(s) < H ? own.y : 0.f;
#pragma unroll
    for (int i = 0; i < kE; ++i) h[s][i] -= m;
    if (!VEC && left(s) < 32 * kE) {
#pragma unroll
      for (int i = 0; i < kE; ++i)
        if (!in_row<T, VEC>(S::first(s), i, H)) h[s][i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      own.z += h[s][i];
      own.w = fmaf(h[s][i], h[s][i], own.w);
    }
  }
  const float sums = warp_sum_halves(own.z, own.w);  // d_w or q_w
  const float mine = own.y;
  float m0 = own.y, m1, squares;
  if (blockDim.x == 32) {
    m1 = __shfl_sync(0xffffffffu, sums, 0) * inv_h;
    squares = __shfl_sync(0xffffffffu, sums, 16) - static_cast<float>(H) * m1 * m1;
  } else {
    auto* p = reinterpret_cast<float*>(&part[threadIdx.x >> 5]);
    if (lane == 0) p[0] = own.x, p[1] = own.y;
    if ((lane & 15) == 0) p[2 + (lane >> 4)] = sums;
    __syncthreads();
    m0 = part[0].y;
    own = lane < static_cast<int>(blockDim.x >> 5) ? part[lane] : make_float4(0.f, m0, 0.f, 0.f);
    const float apart = own.y - m0;
    m1 = warp_sum(fmaf(own.x, apart, own.z)) * inv_h;
    const float off = apart - m1;
    squares = warp_sum(fmaf(off, fmaf(own.x, off, 2.f * own.z), own.w));
  }
  // (a row with NaN or an infinity has a variance of NaN, and keeps it)
  const float r = rsqrtf(fmaf(squares < 0.f ? 0.f : squares, inv_h, eps));
  if (rstd && threadIdx.x == 0) {
    mean[row] = m0 + m1;
    rstd[row] = r;
  }
  const float back = (mine - m0) - m1;  // h - mean = (h - m_w) + back
  const int groups = (H + kScaleGroup - 1) / kScaleGroup;
#pragma unroll
  for (int s = 0; s < P; ++s) {
    const int c = S::first(s);
    float w[kE], b[kE];
    if constexpr (PLAIN) {
      load_slot<T, VEC>(static_cast<const T*>(weight), c, H, true, w);
      load_slot<T, VEC>(static_cast<const T*>(bias), c, H, true, b);
    } else {
      load_param<T, VEC>(weight, w_f32, 1.f, c, H, aligned, w);
      load_param<T, VEC>(bias, w_f32, 0.f, c, H, aligned, b);
    }
#pragma unroll
    for (int i = 0; i < kE; ++i) h[s][i] = fmaf((h[s][i] + back) * r, w[i], b[i]);
    if constexpr (!FP8) store_slot<T, VEC>(y + row * H, c, H, aligned, h[s]);
    else store_quantized<T, VEC>(h[s], c, H, aligned, q + row * H, scale + row * groups, groups);
  }
}

// With n = (h - mean) rstd and g = dy w:
//     dx = rstd (g - mean(g) - n mean(g n)) + dh,  dweight = sum dy n,  dbias = sum dy.
// One pass over dy, h (and dh): a block walks rows blockIdx.x, + gridDim.x, ... with
// the weight and the sums of its columns in registers, and leaves one partial sum
// of each per column; both means of a row in one sum over the block.
//
// AHEAD: the rows' pieces come through shared memory, kLnAhead rows at a time, each
// thread's own in slots that only it touches.  Without it (rows not aligned to 16
// bytes, or too long for the slots) a row is loaded when its turn comes.
//
// h is the sum as the forward stored it, in T (in bf16 rounded by up to 2^-8 of h),
// where mean and rstd are those of the sum before it was rounded.
//
// n is formed as (h - mean) rstd: h rstd + (-mean rstd) is an instruction less, but rounds
// the product for the whole row at once, 6e-5 in every n at a mean of 1000 deviations, where
// this has 1e-7 beside the mean's own rounding.  It costs 0.6 us of 47 at 8192 x 3584 bf16.
//
// Threads hold 16 values where the row has them (two slots of bf16, four of float32) and
// 128 registers, 512 of them an SM: what a row costs besides its values, two sums and a
// barrier, is a warp's, so few warps do it fastest.  8192 x 3584 bf16 with dh, dx alone:
// 43 us (5.4 TB/s; a copy of that size 43), with 8 values in 448 threads a row 62, 28 of
// whose warps an SM have more rows ahead; three or four rows ahead 45.
constexpr int kLnAhead = 2;
constexpr int kLnRing = 200 * 1024;  // of an SM's shared memory
// Blocks on an SM: up to 512 threads, or 1024 where a row takes more.
__host__ __device__ constexpr int ln_blocks(int slots, int threads) {
  return threads <= 512 && slots == 1 ? 2 : 1;
}
template <class T, bool VEC, int P, int THREADS, bool AHEAD>
__global__ void __launch_bounds__(THREADS, ln_blocks(P, THREADS))
    ln_bwd_held_kernel(const T* __restrict__ dy, const T* __restrict__ dh,
                       const T* __restrict__ h, int64_t ldh, const void* __restrict__ weight,
                       int w_f32, bool aligned, const float* __restrict__ mean,
                       const float* __restrict__ rstd, int64_t N, int H, T* __restrict__ dx,
                       float* __restrict__ sums) {
  using S = Slots<T, VEC>;
  __shared__ __align__(8) float part[THREADS <= 512 ? 8 : 1][2][32][2];
  extern __shared__ __align__(16) uint4 ring[];  // [kLnAhead][3][P][threads of the block]
  const int64_t first = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
  constexpr int kE = S::kE, kP = kE / 2;
  F2 w[P][kP], dw[P][kP], db[P][kP];
#pragma unroll
  for (int s = 0; s < P; ++s) {
    float v[kE];
    load_param<T, VEC>(weight, w_f32, 1.f, S::first(s), H, aligned, v);
    to_pairs<kE>(v, w[s]);
#pragma unroll
    for (int i = 0; i < kP; ++i) dw[s][i] = db[s][i] = 0;
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
    for (int i = 0; i < kLnAhead * 3 * P; ++i) ring[i * threads + tid] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kLnAhead; ++i) fetch(first + i * step, i);
  }
  // a row's statistics are fetched a row ahead
  float next_r = first < N ? rstd[first] : 0.f, next_m = first < N ? mean[first] : 0.f;
  int stage = 0, phase = 0;
  for (int64_t row = first; row < N; row += step, phase ^= 1) {
    const F2 r = both(next_r), minus_m = both(-next_m);
    const float minus_r = -next_r;
    if (row + step < N) {
      next_r = rstd[row + step];
      next_m = mean[row + step];
    }
    Piece<T, VEC> held[2][P];  // without AHEAD
    const auto pairs = [&](int array, int s, F2 (&p)[kP]) {
      Piece<T, VEC> piece;
      if constexpr (AHEAD) piece.set(*slot(stage, array, s));
      else if (array < 2) piece = held[array][s];
      else piece.load(dh + row * H, S::first(s), H, aligned);
      float v[kE];
      piece.floats(v);
      to_pairs<kE>(v, p);
    };
    if constexpr (AHEAD) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kLnAhead - 1) : "memory");
    } else {
#pragma unroll
      for (int s = 0; s < P; ++s) {
        const int c = S::first(s);
        held[0][s].load(dy + row * H, c, H, aligned);
        held[1][s].load(h + row * ldh, c, H, aligned);
      }
    }
    F2 dot1 = 0, dot2 = 0;
#pragma unroll
    for (int s = 0; s < P; ++s) {
      F2 d[kP], v[kP];
      pairs(0, s, d);
      pairs(1, s, v);
#pragma unroll
      for (int i = 0; i < kP; ++i) {
        // past the row d is 0, and with it every sum
        const F2 n = mul2(add2(v[i], minus_m), r), g = mul2(d[i], w[s][i]);
        dw[s][i] = fma2(d[i], n, dw[s][i]);
        db[s][i] = add2(db[s][i], d[i]);
        dot1 = add2(dot1, g);
        dot2 = fma2(g, n, dot2);
      }
    }
    if (dx) {
      const float2 dot =
          row_sum2(make_float2(sum2(dot1), sum2(dot2)), part[threadIdx.y & 7], phase);
      const F2 k1 = both(minus_r * (dot.x * inv_h)), k2 = both(minus_r * (dot.y * inv_h));
#pragma unroll
      for (int s = 0; s < P; ++s) {
        F2 d[kP], v[kP];
        pairs(0, s, d);
        pairs(1, s, v);
#pragma unroll
        for (int i = 0; i < kP; ++i) {
          const F2 n = mul2(add2(v[i], minus_m), r), g = mul2(d[i], w[s][i]);
          d[i] = fma2(g, r, fma2(n, k2, k1));
        }
        if (with_dh) {
          pairs(2, s, v);
#pragma unroll
          for (int i = 0; i < kP; ++i) d[i] = add2(d[i], v[i]);
        }
        float out[kE];
        from_pairs<kE>(d, out);
        store_slot<T, VEC>(dx + row * H, S::first(s), H, aligned, out);
      }
    }
    if constexpr (AHEAD) {
      fetch(row + kLnAhead * step, stage);
      stage = stage + 1 == kLnAhead ? 0 : stage + 1;
    }
  }
  if constexpr (AHEAD) asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (!sums) return;
  griddep_launch_dependents();  // the sum's blocks take the places that become free
  if (blockDim.y > 1) {
    // the block's rows one after another into the first one's registers (every copy
    // into the ring has been read)
    F2* all = reinterpret_cast<F2*>(ring) + threadIdx.x;  // [P][kE][threads of a row]
    for (int k = 1; k < static_cast<int>(blockDim.y); ++k) {
      __syncthreads();
      if (static_cast<int>(threadIdx.y) == k) {
#pragma unroll
        for (int s = 0; s < P; ++s)
#pragma unroll
          for (int i = 0; i < kP; ++i) {
            all[(s * kE + i) * blockDim.x] = dw[s][i];
            all[(s * kE + kP + i) * blockDim.x] = db[s][i];
          }
      }
      __syncthreads();
      if (threadIdx.y == 0) {
#pragma unroll
        for (int s = 0; s < P; ++s)
#pragma unroll
          for (int i = 0; i < kP; ++i) {
            dw[s][i] = add2(dw[s][i], all[(s * kE + i) * blockDim.x]);
            db[s][i] = add2(db[s][i], all[(s * kE + kP + i) * blockDim.x]);
          }
      }
    }
    if (threadIdx.y > 0) return;
  }
#pragma unroll
  for (int s = 0; s < P; ++s) {
    const int c = S::first(s);
    float* p = sums + static_cast<int64_t>(blockIdx.x) * 2 * H;
    float vw[kE], vb[kE];
    from_pairs<kE>(dw[s], vw);
    from_pairs<kE>(db[s], vb);
    if constexpr (VEC) {  // (H is a multiple of 4, and so is c)
      if (c >= H) continue;
#pragma unroll
      for (int i = 0; i < kE; i += 4) {
        *reinterpret_cast<float4*>(p + c + i) = make_float4(vw[i], vw[i + 1], vw[i + 2], vw[i + 3]);
        *reinterpret_cast<float4*>(p + H + c + i) =
            make_float4(vb[i], vb[i + 1], vb[i + 2], vb[i + 3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kE; ++i)
        if (c + i * S::kStep < H) {
          p[c + i * S::kStep] = vw[i];
          p[H + c + i * S::kStep] = vb[i];
        }
    }
  }
}

// dweight and dbias (blockIdx.y) = their partial sums, added in a fixed order: 32
// columns a block, each of its 32 warps taking every 32nd partial, then a warp a column.
constexpr int kLnSumWarps = 32;
template <class W>
__global__ void __launch_bounds__(32 * kLnSumWarps)
    ln_sum_kernel(const float* __restrict__ part, int64_t parts, int H, W* __restrict__ dweight,
                  W* __restrict__ dbias) {
  __shared__ float sums[kLnSumWarps][33];
  griddep_launch_dependents();
  griddep_wait();
  W* out = blockIdx.y == 0 ? dweight : dbias;
  if (!out) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const float* p0 = part + static_cast<int64_t>(blockIdx.y) * H + c;
  float s = 0.f;
  if (c < H) {
#pragma unroll 8
    for (int64_t p = warp; p < parts; p += kLnSumWarps) s += p0[p * 2 * H];
  }
  sums[warp][lane] = s;
  __syncthreads();
  s = warp_sum(sums[lane][warp]);
  if (lane == 0 && blockIdx.x * 32 + warp < H) out[blockIdx.x * 32 + warp] = from_f<W>(s);
}

// ----------------------------------------------------- small backwards
// dx needs a row's sums, dweight and dbias a column's, and neither needs the other's:
// where the inputs stay in L2, one launch does both, the first `row_blocks` blocks
// rows (`tpr` threads each, 8 values a thread) and the others 16 columns each, over
// all rows.
constexpr int kLnSmallThreads = 1024;
constexpr int kLnSmallValues = 8;
constexpr int kLnSmallCols = 16;
template <class T>
__global__ void __launch_bounds__(kLnSmallThreads)
    ln_bwd_small_kernel(const T* __restrict__ dy, const T* __restrict__ dh,
                        const T* __restrict__ h, int64_t ldh, const void* __restrict__ weight,
                        int w_f32, const float* __restrict__ mean, const float* __restrict__ rstd,
                        int N, int H, T* __restrict__ dx, void* __restrict__ dweight,
                        void* __restrict__ dbias, int row_blocks, int tpr) {
  __shared__ float2 part[kLnSmallThreads / 32][33];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (static_cast<int>(blockIdx.x) < row_blocks) {
    const int rows = kLnSmallThreads / tpr, k = threadIdx.x / tpr, t = threadIdx.x % tpr;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * rows + k;
    const bool live = k < rows && row < N;
    const float r = live ? rstd[row] : 0.f, m = live ? mean[row] : 0.f;
    float g[kLnSmallValues], n[kLnSmallValues], e[kLnSmallValues];
    float2 dot = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kLnSmallValues; ++i) {
      const int c = t + i * tpr;
      const bool in = live && c < H;
      g[i] = in ? to_f(dy[row * H + c]) : 0.f;
      n[i] = in ? (to_f(h[row * ldh + c]) - m) * r : 0.f;
      e[i] = in && dh ? to_f(dh[row * H + c]) : 0.f;
      if (in && weight)
        g[i] *= w_f32 ? static_cast<const float*>(weight)[c]
                      : to_f(static_cast<const __nv_bfloat16*>(weight)[c]);
      dot.x += g[i];
      dot.y = fmaf(g[i], n[i], dot.y);
    }
    dot.x = warp_sum(dot.x);
    dot.y = warp_sum(dot.y);
    if (lane == 0) part[0][warp] = dot;
    __syncthreads();
    if (!live) return;
    dot = make_float2(0.f, 0.f);
    for (int w = 0; w < tpr / 32; ++w) {
      const float2 p = part[0][k * (tpr / 32) + w];
      dot.x += p.x;
      dot.y += p.y;
    }
    const float inv_h = 1.f / static_cast<float>(H);
    const float k1 = -r * (dot.x * inv_h), k2 = -r * (dot.y * inv_h);
#pragma unroll
    for (int i = 0; i < kLnSmallValues; ++i) {
      const int c = t + i * tpr;
      if (c < H) dx[row * H + c] = from_f<T>(fmaf(g[i], r, fmaf(n[i], k2, k1)) + e[i]);
    }
    return;
  }
  // a half warp a row: 64 rows at a time
  const int c = (blockIdx.x - row_blocks) * kLnSmallCols + (lane & (kLnSmallCols - 1));
  float2 s = make_float2(0.f, 0.f);
  if (c < H) {
#pragma unroll 8
    for (int i = threadIdx.x / kLnSmallCols; i < N; i += kLnSmallThreads / kLnSmallCols) {
      const float d = to_f(dy[static_cast<int64_t>(i) * H + c]);
      s.x = fmaf(d, (to_f(h[i * ldh + c]) - mean[i]) * rstd[i], s.x);
      s.y += d;
    }
  }
  s.x += __shfl_xor_sync(0xffffffffu, s.x, kLnSmallCols);
  s.y += __shfl_xor_sync(0xffffffffu, s.y, kLnSmallCols);
  part[warp][lane] = s;
  __syncthreads();
  if (threadIdx.x >= kLnSmallCols || c >= H) return;
  for (int w = 1; w < kLnSmallThreads / 32; ++w) {
    s.x += part[w][lane].x;
    s.y += part[w][lane].y;
  }
  const auto put = [&](void* out, float v) {
    if (!out) return;
    if (w_f32) static_cast<float*>(out)[c] = v;
    else static_cast<__nv_bfloat16*>(out)[c] = from_f<__nv_bfloat16>(v);
  };
  put(dweight, s.x);
  put(dbias, s.y);
}

// ----------------------------------------------------- rows past kMaxHeld
__device__ __forceinline__ float param_at(const void* w, int w_f32, float missing, int c) {
  return !w ? missing
         : w_f32 ? static_cast<const float*>(w)[c]
                 : to_f(static_cast<const __nv_bfloat16*>(w)[c]);
}

// A block per row, read three times; a warp per group of 128 columns in the last
// pass, where a thread reads an element before it writes the sum in its place (h_out
// may be x or residual).
template <class T, bool FP8>
__global__ void __launch_bounds__(kNormThreads)
    ln_fwd_kernel(const T* x, int64_t ldx, const T* residual, int64_t ldr,
                  const void* __restrict__ weight, const void* __restrict__ bias, int w_f32, int H,
                  float eps, T* y, uint8_t* q, float* scale, T* h_out, float* mean, float* rstd) {
  const int64_t row = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* xr = x + row * ldx;
  const T* rr = residual ? residual + row * ldr : nullptr;
  const auto at = [&](int c) { return to_f(xr[c]) + (rr ? to_f(rr[c]) : 0.f); };
  const float n = static_cast<float>(H);
  float sum = 0.f;
  for (int c = threadIdx.x; c < H; c += kNormThreads) sum += at(c);
  const float m0 = block_sum(sum) / n;
  float rest = 0.f, squares = 0.f;
  for (int c = threadIdx.x; c < H; c += kNormThreads) {
    const float d = at(c) - m0;
    rest += d;
    squares = fmaf(d, d, squares);
  }
  const float m1 = block_sum(rest) / n;
  const float variance = block_sum(squares) / n - m1 * m1;
  const float r = rsqrtf((variance < 0.f ? 0.f : variance) + eps);  // (NaN stays NaN)
  if (rstd && threadIdx.x == 0) {
    mean[row] = m0 + m1;
    rstd[row] = r;
  }
  const int groups = (H + kScaleGroup - 1) / kScaleGroup;
  for (int g = warp; g < groups; g += kNormThreads / 32) {
    float v[4];
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = g * kScaleGroup + i * 32 + lane;
      v[i] = 0.f;
      if (c < H) {
        const float h = at(c);
        if (h_out) h_out[row * H + c] = from_f<T>(h);
        v[i] = fmaf((h - m0 - m1) * r, param_at(weight, w_f32, 1.f, c),
                    param_at(bias, w_f32, 0.f, c));
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

template <class T>
__global__ void __launch_bounds__(kNormThreads)
    ln_bwd_dx_kernel(const T* __restrict__ dy, const T* __restrict__ dh, const T* __restrict__ h,
                     int64_t ldh, const void* __restrict__ weight, int w_f32,
                     const float* __restrict__ mean, const float* __restrict__ rstd, int H,
                     T* __restrict__ dx) {
  const int64_t row = blockIdx.x;
  const float r = rstd[row], m = mean[row];
  float s1 = 0.f, s2 = 0.f;
  for (int c = threadIdx.x; c < H; c += kNormThreads) {
    const float g = to_f(dy[row * H + c]) * param_at(weight, w_f32, 1.f, c);
    s1 += g;
    s2 = fmaf(g, (to_f(h[row * ldh + c]) - m) * r, s2);
  }
  const float k1 = -r * (block_sum(s1) / static_cast<float>(H));
  const float k2 = -r * (block_sum(s2) / static_cast<float>(H));
  for (int c = threadIdx.x; c < H; c += kNormThreads) {
    const float g = to_f(dy[row * H + c]) * param_at(weight, w_f32, 1.f, c);
    float v = fmaf(g, r, fmaf((to_f(h[row * ldh + c]) - m) * r, k2, k1));
    if (dh) v += to_f(dh[row * H + c]);
    dx[row * H + c] = from_f<T>(v);
  }
}

// Partial sums of dweight and dbias over kLnDwRows rows.
template <class T>
__global__ void __launch_bounds__(kNormThreads)
    ln_bwd_sums_kernel(const T* __restrict__ dy, const T* __restrict__ h, int64_t ldh,
                       const float* __restrict__ mean, const float* __restrict__ rstd, int64_t N,
                       int H, float* __restrict__ part) {
  const int c = blockIdx.y * kNormThreads + threadIdx.x;
  if (c >= H) return;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kLnDwRows;
  const int64_t n1 = min(N, n0 + kLnDwRows);
  float s = 0.f, b = 0.f;
  for (int64_t n = n0; n < n1; ++n) {
    const float d = to_f(dy[n * H + c]);
    s = fmaf(d, (to_f(h[n * ldh + c]) - mean[n]) * rstd[n], s);
    b += d;
  }
  float* p = part + static_cast<int64_t>(blockIdx.x) * 2 * H + c;
  p[0] = s;
  p[H] = b;
}

// ------------------------------------------------------------- launching
// The backward's threads a row: 16 values each as far as the row has a warp of them.
// Rows share a block of up to 512 threads, whose sums are one partial sum: sixteen of a
// warp each, else up to eight (a barrier each).  8192 x 3584 bf16 with the sums, two
// rows a block 51 us, one 55.
RowPlan plan_ln_bwd(int64_t H, int elems, bool vec) {
  const int64_t units = vec ? (H + elems - 1) / elems
                            : (H + kScaleGroup - 1) / kScaleGroup * 32;
  const int most = 16 / elems;
  int slots = 1;
  while (slots < most && units > 32 * slots) slots *= 2;
  int64_t threads = (units + slots - 1) / slots;
  threads = std::max<int64_t>((threads + 31) / 32 * 32, 32);
  const int64_t rows = threads == 32 ? 16 : std::clamp<int64_t>(512 / threads, 1, 8);
  return {static_cast<int>(threads), slots, static_cast<int>(rows)};
}

// Partial sums of dweight and dbias, one of each a block.  A fixed number, so that the
// order of additions depends on the sizes and the type alone: the blocks that 152 SMs
// hold at once.
int64_t ln_held_parts(int64_t N, const RowPlan& p) {
  const int per_sm = ln_blocks(p.slots, p.threads * p.rows);
  return std::min<int64_t>((N + p.rows - 1) / p.rows, 152 * per_sm);
}
int64_t ln_parts(int64_t N, int64_t H) {
  if (H > kMaxHeld) return (N + kLnDwRows - 1) / kLnDwRows;
  // whichever plan the call's types lead to
  return std::max({ln_held_parts(N, plan_ln_bwd(H, 8, true)),
                   ln_held_parts(N, plan_ln_bwd(H, 4, true)),
                   ln_held_parts(N, plan_ln_bwd(H, 4, false))});
}

struct LnFwdArgs {
  const void* x;
  int64_t ldx;
  const void* residual;
  int64_t ldr;
  const void* weight;
  const void* bias;
  int w_f32;
  int64_t N;
  int H;
  float eps;
  void* y;
  void* q;
  float* scale;
  void* h_out;
  float* mean;
  float* rstd;
};

template <class T, bool FP8, bool VEC, int P, bool PLAIN>
cudaError_t launch_ln_fwd(const RowPlan& p, bool aligned, const LnFwdArgs& a, cudaStream_t s) {
  const unsigned blocks = static_cast<unsigned>((a.N + p.rows - 1) / p.rows);
  return launch_overlapped(
      ln_fwd_held_kernel<T, FP8, VEC, P, PLAIN>, dim3(blocks), dim3(p.threads, p.rows), 0, s, 1,
      static_cast<const T*>(a.x), a.ldx, static_cast<const T*>(a.residual), a.ldr, a.weight, a.bias,
      a.w_f32, aligned, a.N, a.H, static_cast<float>(1.0 / a.H), a.eps, static_cast<T*>(a.y),
      static_cast<uint8_t*>(a.q), a.scale, static_cast<T*>(a.h_out), a.mean, a.rstd);
}

// Whether every row's pieces are 16-byte aligned.
template <class T>
bool ln_fwd_aligned(const LnFwdArgs& a) {
  const int e = 16 / sizeof(T);
  return a.ldx % e == 0 && a.ldr % e == 0 && aligned_to(a.x, 16) && aligned_to(a.residual, 16) &&
         aligned_to(a.weight, 16) && aligned_to(a.bias, 16) && aligned_to(a.y, 16) &&
         aligned_to(a.q, 8) && aligned_to(a.h_out, 16);
}

template <class T, bool FP8>
cudaError_t run_ln_fwd(const LnFwdArgs& a, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const bool plain = a.weight && a.bias && a.w_f32 == (sizeof(T) == 4);
  if (a.H > kMaxHeld) {
    ln_fwd_kernel<T, FP8><<<static_cast<unsigned>(a.N), kNormThreads, 0, s>>>(
        static_cast<const T*>(a.x), a.ldx, static_cast<const T*>(a.residual), a.ldr, a.weight,
        a.bias, a.w_f32, a.H, a.eps, static_cast<T*>(a.y), static_cast<uint8_t*>(a.q), a.scale,
        static_cast<T*>(a.h_out), a.mean, a.rstd);
  } else if (a.H % Slots<T, true>::kE == 0) {
    constexpr int kE = Slots<T, true>::kE;
    const bool al = ln_fwd_aligned<T>(a);
    const RowPlan p = plan_rows(a.N, a.H, kE, true);
    const auto launch = [&](auto plain) {
      constexpr bool kPlain = decltype(plain)::value;
      if (p.slots == 1) return launch_ln_fwd<T, FP8, true, 1, kPlain>(p, al, a, s);
      if constexpr (kE == 4)
        if (p.slots == 4) return launch_ln_fwd<T, FP8, true, 4, kPlain>(p, al, a, s);
      return launch_ln_fwd<T, FP8, true, 2, kPlain>(p, al, a, s);
    };
    e = al && plain ? launch(std::true_type{}) : launch(std::false_type{});
  } else {
    const RowPlan p = plan_rows(a.N, a.H, 4, false);
    const auto launch = [&](auto plain) {
      constexpr bool kPlain = decltype(plain)::value;
      if (p.slots == 1) return launch_ln_fwd<T, FP8, false, 1, kPlain>(p, false, a, s);
      if (p.slots == 2) return launch_ln_fwd<T, FP8, false, 2, kPlain>(p, false, a, s);
      return launch_ln_fwd<T, FP8, false, 4, kPlain>(p, false, a, s);
    };
    e = plain ? launch(std::true_type{}) : launch(std::false_type{});
  }
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

struct LnBwdArgs {
  const void* dy;
  const void* dh;
  const void* h;
  int64_t ldh;
  const void* weight;
  int w_f32;
  const float* mean;
  const float* rstd;
  int64_t N;
  int H;
  void* dx;
  void* dweight;
  void* dbias;
  float* part;
};

template <class T, bool VEC, int P>
cudaError_t launch_ln_bwd(const RowPlan& p, bool aligned, int64_t parts, const LnBwdArgs& a,
                          cudaStream_t s) {
  const int threads = p.threads * p.rows, stage = 3 * P * threads * 16;
  const auto launch = [&](auto* k, int smem) {
    // the block's sums, where rows share it
    smem = std::max(smem, p.rows > 1 ? P * Slots<T, VEC>::kE * p.threads * 8 : 0);
    // a plain launch, as the RMS norm's: blocks that wait here would take shared
    // memory from the kernel before them
    k<<<dim3(static_cast<unsigned>(parts)), dim3(p.threads, p.rows), smem, s>>>(
        static_cast<const T*>(a.dy), static_cast<const T*>(a.dh), static_cast<const T*>(a.h),
        a.ldh, a.weight, a.w_f32, aligned, a.mean, a.rstd, a.N, a.H, static_cast<T*>(a.dx),
        a.dweight || a.dbias ? a.part : static_cast<float*>(nullptr));
    return cudaGetLastError();
  };
  // a row that takes more than 512 threads has 16 values in each
  constexpr int kMost = P * Slots<T, VEC>::kE == 16 ? 1024 : 512;
  if constexpr (VEC) {
    if (aligned && kLnAhead * stage * ln_blocks(P, threads) <= kLnRing) {
      auto* k = threads <= 512 ? ln_bwd_held_kernel<T, VEC, P, 512, true>
                               : ln_bwd_held_kernel<T, VEC, P, kMost, true>;
      static SmemLimit limits[2];  // one for each of them
      const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), kLnRing,
                                       &limits[threads <= 512 ? 0 : 1]);
      return e != cudaSuccess ? e : launch(k, kLnAhead * stage);
    }
  }
  return threads <= 512 ? launch(ln_bwd_held_kernel<T, VEC, P, 512, false>, 0)
                        : launch(ln_bwd_held_kernel<T, VEC, P, kMost, false>, 0);
}

// What ln_bwd_small_kernel takes: a column's block adds at most 64 rows a warp, and its
// inputs are read twice, from L2.  One launch and two, us in a graph over inputs larger than
// L2 / over inputs that are in L2 / called from the host, bf16 and float32 alike to 0.7:
//       64 x 4096  bf16      5.6, 7.0 / 5.2, 7.2 / 8.2, 10.0
//      482 x 1536  float32   8.0, 8.4 / 6.1, 8.1 / 8.6, 10.6
//     1021 x 1001  float32   9.7, 8.7 / -         / 9.7, 11.1   (1047 rows 8.6, 9.0: its rows
//                            are added 512 at a time, the last ones of them one by one)
//      409 x 2560  bf16      9.4, 8.7 / 7.7, 8.3 / 9.6, 11.1
//      608 x 2048  bf16      8.7, 8.3 / 7.7, 8.2 / 8.9, 10.5   (past the limit)
//     2097 x 1000  float32  15.7, 12.6 / -       / 16.1, 14.8  (past the limit)
//      218 x 3584  bf16      8.5, 7.9 / 6.8, 7.8 / 9.0, 10.6
//      292 x 3584  bf16     11.1, 8.4 / 8.8, 8.3 / 11.2, 10.8  (past the limit)
//      256 x 4096  float32  10.0, 8.9 / 7.9, 8.2 / 10.1, 10.7  (past the limit)
// So up to 2^20 values the host's time decides, where the two are close in a graph; from 3584
// columns on, whose blocks are more than the SMs, one launch falls behind from 3 2^18 on.
bool small_ln_bwd(int64_t N, int64_t H) {
  return N <= 2048 && H <= kLnSmallThreads * kLnSmallValues &&
         N * H <= int64_t{H <= 2560 ? 4 : 3} << 18;
}

template <class T>
cudaError_t run_ln_bwd(const LnBwdArgs& a, cudaStream_t s) {
  const bool want_sums = a.dweight || a.dbias;
  if (small_ln_bwd(a.N, a.H)) {
    const int tpr = (((a.H + kLnSmallValues - 1) / kLnSmallValues) + 31) / 32 * 32;
    const int rows = kLnSmallThreads / tpr;
    const int row_blocks = a.dx ? static_cast<int>((a.N + rows - 1) / rows) : 0;
    const int blocks = row_blocks + (want_sums ? (a.H + kLnSmallCols - 1) / kLnSmallCols : 0);
    if (blocks == 0) return cudaSuccess;
    const cudaError_t e = launch_overlapped(
        ln_bwd_small_kernel<T>, dim3(blocks), dim3(kLnSmallThreads), 0, s, 1,
        static_cast<const T*>(a.dy), static_cast<const T*>(a.dh), static_cast<const T*>(a.h),
        a.ldh, a.weight, a.w_f32, a.mean, a.rstd, static_cast<int>(a.N), a.H,
        static_cast<T*>(a.dx), a.dweight, a.dbias, row_blocks, tpr);
    note_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
  }
  int64_t parts = 0;
  const T* dy = static_cast<const T*>(a.dy);
  const T* h = static_cast<const T*>(a.h);
  if (a.N > 0 && a.H > kMaxHeld) {
    parts = ln_parts(a.N, a.H);
    const unsigned cols = static_cast<unsigned>((a.H + kNormThreads - 1) / kNormThreads);
    if (a.dx) {
      ln_bwd_dx_kernel<T><<<static_cast<unsigned>(a.N), kNormThreads, 0, s>>>(
          dy, static_cast<const T*>(a.dh), h, a.ldh, a.weight, a.w_f32, a.mean, a.rstd, a.H,
          static_cast<T*>(a.dx));
      note_launch();
    }
    if (want_sums) {
      ln_bwd_sums_kernel<T><<<dim3(static_cast<unsigned>(parts), cols), kNormThreads, 0, s>>>(
          dy, h, a.ldh, a.mean, a.rstd, a.N, a.H, a.part);
      note_launch();
    }
  } else if (a.N > 0 && (a.dx || want_sums)) {
    constexpr int kE = Slots<T, true>::kE;
    const bool vec = a.H % kE == 0;
    const bool al = a.ldh % kE == 0 && aligned_to(a.dy, 16) && aligned_to(a.dh, 16) &&
                    aligned_to(a.h, 16) && aligned_to(a.weight, 16) && aligned_to(a.dx, 16);
    const RowPlan p = plan_ln_bwd(a.H, vec ? kE : 4, vec);
    parts = ln_held_parts(a.N, p);
    cudaError_t e = cudaSuccess;
    if (vec) {
      if (p.slots == 1) e = launch_ln_bwd<T, true, 1>(p, al, parts, a, s);
      else if (p.slots == 2) e = launch_ln_bwd<T, true, 2>(p, al, parts, a, s);
      else if constexpr (kE == 4) e = launch_ln_bwd<T, true, 4>(p, al, parts, a, s);
    } else {
      if (p.slots == 1) e = launch_ln_bwd<T, false, 1>(p, al, parts, a, s);
      else if (p.slots == 2) e = launch_ln_bwd<T, false, 2>(p, al, parts, a, s);
      else e = launch_ln_bwd<T, false, 4>(p, al, parts, a, s);
    }
    if (e != cudaSuccess) return e;
    note_launch();
  }
  if (want_sums) {
    const dim3 grid(static_cast<unsigned>((a.H + 31) / 32), 2), block(32 * kLnSumWarps);
    const auto sum = [&](auto w) {
      using W = decltype(w);
      return launch_overlapped(ln_sum_kernel<W>, grid, block, 0, s, 1, a.part, parts, a.H,
                               static_cast<W*>(a.dweight), static_cast<W*>(a.dbias));
    };
    const cudaError_t e = a.w_f32 ? sum(float{}) : sum(__nv_bfloat16{});
    if (e != cudaSuccess) return e;
    note_launch();
  }
  return cudaGetLastError();
}

// What both forward entry points check.
flce_status check_layer_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                             const void* weight, const void* bias, int64_t N, int64_t H,
                             flce_dtype dtype, flce_dtype weight_dtype) {
  if (N < 0 || H <= 0 || !valid_dtype(dtype) || !valid_dtype(weight_dtype))
    return FLCE_ERR_INVALID_ARG;
  if (H > kMaxRowElems || N > kMaxRows) return FLCE_ERR_UNSUPPORTED_SHAPE;
  if (N == 0) return FLCE_OK;
  if (!x || ldx < H || (residual && ldr < H)) return FLCE_ERR_INVALID_ARG;
  const size_t e = dtype_bytes(dtype), we = dtype_bytes(weight_dtype);
  if (!aligned_to(x, e) || !aligned_to(residual, e) || !aligned_to(weight, we) ||
      !aligned_to(bias, we))
    return FLCE_ERR_INVALID_ARG;
  return FLCE_OK;
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

flce_status flce_layer_norm_forward(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                                    const void* weight, const void* bias, int64_t N, int64_t H,
                                    float eps, flce_dtype dtype, flce_dtype weight_dtype, void* y,
                                    void* h_out, float* mean, float* rstd, flce_stream_t stream) {
  OpRange range("flce_layer_norm_forward");
  flce_status st = check_layer_norm(x, ldx, residual, ldr, weight, bias, N, H, dtype, weight_dtype);
  if (st != FLCE_OK || N == 0) return st;
  const size_t e = dtype_bytes(dtype), nw = static_cast<size_t>(H) * dtype_bytes(weight_dtype);
  if (!y || !aligned_to(y, e) || !aligned_to(h_out, e) || !aligned_to(mean, 4) ||
      !aligned_to(rstd, 4) || !mean != !rstd)
    return FLCE_ERR_INVALID_ARG;
  if (!norm_outputs_apart(x, ldx, residual, ldr, N, H, e, h_out, {{weight, nw}, {bias, nw}},
                          {{y, span_bytes(N, H, H, e)},
                           {mean, static_cast<size_t>(N) * 4},
                           {rstd, static_cast<size_t>(N) * 4}}))
    return FLCE_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = check_device(&sms)) != FLCE_OK) return st;
  const LnFwdArgs a = {x, ldx, residual, ldr, weight, bias, weight_dtype == FLCE_F32, N,
                       static_cast<int>(H), eps, y, nullptr, nullptr, h_out, mean, rstd};
  const auto s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t err = dtype == FLCE_BF16 ? run_ln_fwd<__nv_bfloat16, false>(a, s)
                                             : run_ln_fwd<float, false>(a, s);
  return err == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

flce_status flce_layer_norm_fp8(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                                const void* weight, const void* bias, int64_t N, int64_t H,
                                float eps, flce_dtype dtype, flce_dtype weight_dtype, void* q,
                                float* scale, void* h_out, flce_stream_t stream) {
  OpRange range("flce_layer_norm_fp8");
  flce_status st = check_layer_norm(x, ldx, residual, ldr, weight, bias, N, H, dtype, weight_dtype);
  if (st != FLCE_OK || N == 0) return st;
  const size_t e = dtype_bytes(dtype), nw = static_cast<size_t>(H) * dtype_bytes(weight_dtype);
  if (!q || !scale || !aligned_to(h_out, e) || !aligned_to(scale, 4)) return FLCE_ERR_INVALID_ARG;
  const int64_t groups = (H + kScaleGroup - 1) / kScaleGroup;
  if (!norm_outputs_apart(x, ldx, residual, ldr, N, H, e, h_out, {{weight, nw}, {bias, nw}},
                          {{q, span_bytes(N, H, H, 1)}, {scale, span_bytes(N, groups, groups, 4)}}))
    return FLCE_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = check_device(&sms)) != FLCE_OK) return st;
  const LnFwdArgs a = {x, ldx, residual, ldr, weight, bias, weight_dtype == FLCE_F32, N,
                       static_cast<int>(H), eps, nullptr, q, scale, h_out, nullptr, nullptr};
  const auto s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t err = dtype == FLCE_BF16 ? run_ln_fwd<__nv_bfloat16, true>(a, s)
                                             : run_ln_fwd<float, true>(a, s);
  return err == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

size_t flce_layer_norm_workspace_size(int64_t N, int64_t H) {
  if (N < 0 || H <= 0 || H > kMaxRowElems || N > kMaxRows) return 0;
  const size_t n = static_cast<size_t>(ln_parts(N, H)) * static_cast<size_t>(H) * 8;
  return std::max<size_t>((n + 255) / 256 * 256, 256);
}

flce_status flce_layer_norm_backward(const void* dy, const void* dh, const void* h, int64_t ldh,
                                     const void* weight, const float* mean, const float* rstd,
                                     int64_t N, int64_t H, flce_dtype dtype,
                                     flce_dtype weight_dtype, void* dx, void* dweight, void* dbias,
                                     void* workspace, size_t workspace_bytes,
                                     flce_stream_t stream) {
  OpRange range("flce_layer_norm_backward");
  if (N < 0 || H <= 0 || !valid_dtype(dtype) || !valid_dtype(weight_dtype))
    return FLCE_ERR_INVALID_ARG;
  if (H > kMaxRowElems || N > kMaxRows) return FLCE_ERR_UNSUPPORTED_SHAPE;
  if (N > 0 && (!dy || !h || !mean || !rstd || ldh < H)) return FLCE_ERR_INVALID_ARG;
  const size_t e = dtype_bytes(dtype), we = dtype_bytes(weight_dtype);
  if (!aligned_to(dy, e) || !aligned_to(dh, e) || !aligned_to(h, e) || !aligned_to(dx, e) ||
      !aligned_to(weight, we) || !aligned_to(dweight, we) || !aligned_to(dbias, we) ||
      !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return FLCE_ERR_INVALID_ARG;
  if (dweight || dbias) {  // (else it is not used)
    if (!workspace || !aligned_to(workspace, 256)) return FLCE_ERR_INVALID_ARG;
    if (workspace_bytes < flce_layer_norm_workspace_size(N, H))
      return FLCE_ERR_WORKSPACE_TOO_SMALL;
  }
  const size_t nh = span_bytes(N, H, H, e), nw = static_cast<size_t>(H) * we,
               nr = static_cast<size_t>(N) * 4;
  const bool sums = dweight || dbias;
  const Range outs[] = {{dx, nh}, {dweight, nw}, {dbias, nw},
                        {sums ? workspace : nullptr, workspace_bytes}};
  const Range ins[] = {{dy, nh},     {dh, nh},   {h, span_bytes(N, H, ldh, e)},
                       {weight, nw}, {mean, nr}, {rstd, nr}};
  for (int i = 0; i < 4; ++i) {
    for (const Range& r : ins)
      if (ranges_overlap(outs[i], r)) return FLCE_ERR_INVALID_ARG;
    for (int k = 0; k < i; ++k)
      if (ranges_overlap(outs[i], outs[k])) return FLCE_ERR_INVALID_ARG;
  }
  int sms = 0;
  const flce_status st = check_device(&sms);
  if (st != FLCE_OK) return st;
  const auto s = reinterpret_cast<cudaStream_t>(stream);
  const LnBwdArgs a = {dy, dh, h, ldh, weight, weight_dtype == FLCE_F32, mean, rstd, N,
                       static_cast<int>(H), dx, dweight, dbias, static_cast<float*>(workspace)};
  const cudaError_t err =
      dtype == FLCE_BF16 ? run_ln_bwd<__nv_bfloat16>(a, s) : run_ln_bwd<float>(a, s);
  return err == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

}  // extern "C"
