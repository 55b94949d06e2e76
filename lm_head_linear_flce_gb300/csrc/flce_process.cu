// Penalties for repeated tokens, biases and grammar masks on logits
// (flce_process_logits).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "flce_internal.h"
#include "flce_ops.h"

namespace flce {
namespace {

struct ProcessArgs {
  int64_t ld_logits, ld_out, ld_tokens, ld_allowed;
  int64_t V, L;
  int n_bias;
  int cols;      // columns per block
  int in_place;  // out is logits
  const int* lengths;
  const int* prompt_lengths;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const float* bias_values;
  const int* allowed;
  const void* tokens;
  const void* bias_ids;
  int tokens_int64, bias_int64;
};

__device__ __forceinline__ int64_t id_at(const void* p, int is64, int64_t i) {
  return is64 ? static_cast<const int64_t*>(p)[i] : static_cast<const int*>(p)[i];
}

// ------------------------------------------------------------ the kernel
// A block takes `cols` columns of one row.  It counts the row's history into
// shared memory (every block of a row reads all of it and keeps the ids of its
// own columns), then streams its logits past the counts: bound by bytes, 2 + 4
// per bf16 -> float32 column.  The first logits are loaded before the counting,
// so that they arrive under it.
//
// A column's counter is its number of generated occurrences, and a top bit for
// "in the prompt": 16 bits where the history is shorter than 2^15 (half the
// shared memory, so twice the columns a block), else 32.  With biases, 16 more
// bits hold 1 + the largest index of the column's entries.
constexpr int kWin = 8;    // consecutive columns a thread takes at a time
constexpr int kBatch = 4;  // windows a thread has in flight

template <bool WIDE>
struct Counts {
  uint32_t* words;
  __device__ void add(int c, bool prompt) {
    if constexpr (WIDE) {
      if (prompt) atomicOr(words + c, 0x80000000u);
      else atomicAdd(words + c, 1u);
    } else {
      const int sh = 16 * (c & 1);
      if (prompt) atomicOr(words + (c >> 1), 0x8000u << sh);
      else atomicAdd(words + (c >> 1), 1u << sh);
    }
  }
  // Counters of the window at c (a multiple of kWin); false if all are zero.
  __device__ bool window(int c, uint32_t (&n)[kWin]) const {
    if constexpr (WIDE) {
      const uint4 p = *reinterpret_cast<const uint4*>(words + c);
      const uint4 q = *reinterpret_cast<const uint4*>(words + c + 4);
      n[0] = p.x, n[1] = p.y, n[2] = p.z, n[3] = p.w;
      n[4] = q.x, n[5] = q.y, n[6] = q.z, n[7] = q.w;
      return (p.x | p.y | p.z | p.w | q.x | q.y | q.z | q.w) != 0;
    } else {
      const uint4 p = *reinterpret_cast<const uint4*>(words + (c >> 1));
      const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) n[2 * i] = w[i] & 0xffffu, n[2 * i + 1] = w[i] >> 16;
      return (p.x | p.y | p.z | p.w) != 0;
    }
  }
  static constexpr uint32_t kPrompt = WIDE ? 0x80000000u : 0x8000u;
};

// Eight consecutive logits as loaded, and as floats.
template <class T>
struct Raw {
  uint4 p[sizeof(T) / 2];
};
__device__ __forceinline__ void floats(const Raw<float>& r, float (&v)[kWin]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[4 * i] = __uint_as_float(r.p[i].x);
    v[4 * i + 1] = __uint_as_float(r.p[i].y);
    v[4 * i + 2] = __uint_as_float(r.p[i].z);
    v[4 * i + 3] = __uint_as_float(r.p[i].w);
  }
}
__device__ __forceinline__ void floats(const Raw<__nv_bfloat16>& r, float (&v)[kWin]) {
  const uint32_t w[4] = {r.p[0].x, r.p[0].y, r.p[0].z, r.p[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <class T>
__device__ __forceinline__ Raw<T> load_raw(const T* p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
    r.p[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
__device__ __forceinline__ void store_window(float* p, const float (&v)[kWin]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store_window(__nv_bfloat16* p, const float (&v)[kWin]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float load_f(const float* p) { return *p; }
__device__ __forceinline__ float load_f(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_f(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <class T, class O, bool WIDE, bool BIAS, int THREADS>
__global__ void __launch_bounds__(THREADS)
    process_kernel(const T* logits, O* out, const ProcessArgs a) {
  extern __shared__ __align__(16) uint32_t smem[];
  const int64_t b = blockIdx.y;
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * a.cols;
  const int cols = static_cast<int>(min(int64_t{a.cols}, a.V - v0));
  const T* in_row = logits + b * a.ld_logits + v0;
  O* out_row = out + b * a.ld_out + v0;
  // Windows start `shift` columns before the block's first, where both rows are
  // 16-byte aligned; if no shift does that, every window goes column by column.
  constexpr int kEI = 16 / static_cast<int>(sizeof(T)), kEO = 16 / static_cast<int>(sizeof(O));
  const int mi = static_cast<int>(reinterpret_cast<uintptr_t>(in_row) / sizeof(T) % kEI);
  const int mo = static_cast<int>(reinterpret_cast<uintptr_t>(out_row) / sizeof(O) % kEO);
  const int shift = kEI > kEO ? mi : mo;
  const bool vec = (mi - shift) % kEI == 0 && (mo - shift) % kEO == 0;
  const int windows = (shift + cols + kWin - 1) / kWin;
  // a window wholly inside the block's columns
  const auto whole = [&](int k) {
    return vec && kWin * k >= shift && kWin * (k + 1) - shift <= cols;
  };

  Raw<T> raw[kBatch];
  const auto fetch = [&](int k0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int k = k0 + i * THREADS;
      if (k < windows && whole(k)) raw[i] = load_raw(in_row + kWin * k - shift);
    }
  };
  if (!a.in_place) fetch(threadIdx.x);

  // counters, then bias indices, one per window column
  const int slots = windows * kWin;
  Counts<WIDE> counts{smem};
  uint32_t* bias = smem + (WIDE ? slots : slots / 2);
  const int words = (WIDE ? slots : slots / 2) + (BIAS ? slots / 2 : 0);
  for (int i = threadIdx.x; i < words / 4; i += THREADS)
    reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  int64_t len = a.lengths ? a.lengths[b] : a.L;
  len = max(int64_t{0}, min(len, a.L));
  const int64_t prompt = a.prompt_lengths ? a.prompt_lengths[b] : 0;
  constexpr int kIds = 8;  // ids a thread has in flight
  for (int64_t i0 = threadIdx.x; i0 < len; i0 += THREADS * kIds) {
    int64_t id[kIds];
#pragma unroll
    for (int u = 0; u < kIds; ++u) {
      const int64_t i = i0 + u * THREADS;
      id[u] = i < len ? id_at(a.tokens, a.tokens_int64, b * a.ld_tokens + i) : -1;
    }
#pragma unroll
    for (int u = 0; u < kIds; ++u) {
      const int64_t c = id[u] - v0;
      if (id[u] >= 0 && c >= 0 && c < cols)
        counts.add(static_cast<int>(c) + shift, i0 + u * THREADS < prompt);
    }
  }
  if constexpr (BIAS) {
    for (int i = threadIdx.x; i < a.n_bias; i += THREADS) {
      const int64_t v = id_at(a.bias_ids, a.bias_int64, b * a.n_bias + i);
      if (v < v0 || v - v0 >= cols) continue;
      // the largest index stays, in whatever order the threads come
      const int c = static_cast<int>(v - v0) + shift, sh = 16 * (c & 1);
      uint32_t* w = bias + (c >> 1);
      uint32_t old = *w;
      while ((old >> sh & 0xffffu) < static_cast<uint32_t>(i + 1)) {
        const uint32_t seen =
            atomicCAS(w, old, (old & ~(0xffffu << sh)) | static_cast<uint32_t>(i + 1) << sh);
        if (seen == old) break;
        old = seen;
      }
    }
  }
  __syncthreads();

  const float rep = a.repetition ? a.repetition[b] : 1.f;
  const float freq = a.frequency ? a.frequency[b] : 0.f;
  const float pres = a.presence ? a.presence[b] : 0.f;
  const int* mask = a.allowed ? a.allowed + b * a.ld_allowed : nullptr;
  // One column: its counter n, bias entry e (0: none) and whether it is allowed.
  const auto apply = [&](float l, uint32_t n, uint32_t e, bool ok) {
    if (n) {
      l = l > 0.f ? l / rep : l * rep;
      const uint32_t c = n & ~Counts<WIDE>::kPrompt;
      l -= freq * static_cast<float>(c) + (c ? pres : 0.f);
    }
    if (BIAS && e) l += a.bias_values[b * a.n_bias + e - 1];
    return ok ? l : -INFINITY;
  };
  for (int k0 = threadIdx.x; k0 < windows; k0 += THREADS * kBatch) {
    if (!a.in_place && k0 != static_cast<int>(threadIdx.x)) fetch(k0);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int k = k0 + i * THREADS;
      if (k >= windows) break;
      const int c0 = kWin * k;  // the window's first counter
      uint32_t n[kWin];
      bool plain = !counts.window(c0, n);
      uint32_t e[kWin] = {};
      if constexpr (BIAS) {
        const uint4 p = *reinterpret_cast<const uint4*>(bias + (c0 >> 1));
        const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) e[2 * j] = w[j] & 0xffffu, e[2 * j + 1] = w[j] >> 16;
        plain = plain && (p.x | p.y | p.z | p.w) == 0;
      }
      const int64_t v = v0 + c0 - shift;  // the window's first column
      if (whole(k)) {
        uint32_t ok = 0xffu;
        if (mask) {
          const int sh = static_cast<int>(v & 31);
          ok = static_cast<uint32_t>(mask[v >> 5]) >> sh;
          if (sh > 32 - kWin) ok |= static_cast<uint32_t>(mask[(v >> 5) + 1]) << (32 - sh);
          ok &= 0xffu;
        }
        plain = plain && ok == 0xffu;
        if (a.in_place && plain) continue;  // nothing applies: not touched
        if (a.in_place) raw[i] = load_raw(in_row + c0 - shift);
        float l[kWin];
        floats(raw[i], l);
        if (!plain) {
#pragma unroll
          for (int j = 0; j < kWin; ++j) l[j] = apply(l[j], n[j], e[j], ok >> j & 1);
        }
        store_window(out_row + c0 - shift, l);
      } else {
#pragma unroll
        for (int j = 0; j < kWin; ++j) {
          const int c = c0 - shift + j;
          if (c < 0 || c >= cols) continue;
          const bool ok = !mask || (mask[(v + j) >> 5] >> ((v + j) & 31) & 1);
          store_f(out_row + c, apply(load_f(in_row + c), n[j], e[j], ok));
        }
      }
    }
  }
}

// Shared memory a block may take: two blocks an SM.
constexpr int kMaxSmem = 100 * 1024;

template <class T, class O, bool WIDE, bool BIAS, int THREADS>
cudaError_t launch_process(const void* logits, void* out, int64_t B, const ProcessArgs& a,
                           int smem, cudaStream_t s) {
  auto* k = process_kernel<T, O, WIDE, BIAS, THREADS>;
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid(static_cast<unsigned>((a.V + a.cols - 1) / a.cols), static_cast<unsigned>(B));
  k<<<grid, THREADS, smem, s>>>(static_cast<const T*>(logits), static_cast<O*>(out), a);
  note_launch();
  return cudaGetLastError();
}

template <class T, class O>
cudaError_t run_process(const void* logits, void* out, int64_t B, ProcessArgs a, int sms,
                        cudaStream_t s) {
  const bool wide = a.L >= 32768, bias = a.n_bias > 0;
  const int per_col = (wide ? 4 : 2) + (bias ? 2 : 0);
  // Columns a block: two blocks for every SM if the batch gives that, since
  // every block of a row reads the row's history; at least 1024, and at most
  // what shared memory holds (less the windows' shift).
  const int64_t most = kMaxSmem / per_col - 2 * kWin;
  int64_t cols = (B * a.V + 2 * sms - 1) / (2 * sms);
  cols = std::min(std::max<int64_t>(cols, 1024), most);
  const int64_t blocks = (a.V + cols - 1) / cols;
  cols = std::min(((a.V + blocks - 1) / blocks + 63) / 64 * 64, most / 64 * 64);
  a.cols = static_cast<int>(cols);
  // one window more for the shift; in steps of 16 bytes
  const int smem = static_cast<int>((cols + 2 * kWin) / kWin * kWin * per_col + 15) / 16 * 16;
  const bool small = cols <= 4096;
  if (wide && bias)
    return small ? launch_process<T, O, true, true, 256>(logits, out, B, a, smem, s)
                 : launch_process<T, O, true, true, 512>(logits, out, B, a, smem, s);
  if (wide)
    return small ? launch_process<T, O, true, false, 256>(logits, out, B, a, smem, s)
                 : launch_process<T, O, true, false, 512>(logits, out, B, a, smem, s);
  if (bias)
    return small ? launch_process<T, O, false, true, 256>(logits, out, B, a, smem, s)
                 : launch_process<T, O, false, true, 512>(logits, out, B, a, smem, s);
  return small ? launch_process<T, O, false, false, 256>(logits, out, B, a, smem, s)
               : launch_process<T, O, false, false, 512>(logits, out, B, a, smem, s);
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" flce_status flce_process_logits(
    const void* logits, int64_t ld_logits, flce_dtype dtype, int64_t B, int64_t V,
    const void* tokens, int64_t ld_tokens, int tokens_int64, int64_t L, const int32_t* lengths,
    const int32_t* prompt_lengths, const float* repetition, const float* frequency,
    const float* presence, const void* bias_ids, int bias_int64, const float* bias_values,
    int64_t n_bias, const int32_t* allowed, int64_t ld_allowed, void* out, int64_t ld_out,
    flce_dtype out_dtype, flce_stream_t stream) {
  if (B < 0 || V <= 0 || L < 0 || n_bias < 0 || !valid_dtype(dtype) || !valid_dtype(out_dtype))
    return FLCE_ERR_INVALID_ARG;
  if (B > 65535 || V > (int64_t{1} << 30) || L >= (int64_t{1} << 31) || n_bias > 65535)
    return FLCE_ERR_UNSUPPORTED_SHAPE;
  if (B == 0) return FLCE_OK;
  if (!logits || !out || ld_logits < V || ld_out < V) return FLCE_ERR_INVALID_ARG;
  if (L > 0 && (!tokens || ld_tokens < L)) return FLCE_ERR_INVALID_ARG;
  if (n_bias > 0 && (!bias_ids || !bias_values)) return FLCE_ERR_INVALID_ARG;
  const int64_t words = (V + 31) / 32;
  if (allowed && ld_allowed < words) return FLCE_ERR_INVALID_ARG;
  const size_t e = dtype_bytes(dtype), oe = dtype_bytes(out_dtype);
  if (!aligned_to(logits, e) || !aligned_to(out, oe) ||
      !aligned_to(tokens, tokens_int64 ? 8 : 4) || !aligned_to(bias_ids, bias_int64 ? 8 : 4) ||
      !aligned_to(bias_values, 4) || !aligned_to(allowed, 4) || !aligned_to(lengths, 4) ||
      !aligned_to(prompt_lengths, 4) || !aligned_to(repetition, 4) || !aligned_to(frequency, 4) ||
      !aligned_to(presence, 4))
    return FLCE_ERR_INVALID_ARG;
  const Range o = {out, span_bytes(B, V, ld_out, oe)};
  const Range in = {logits, span_bytes(B, V, ld_logits, e)};
  const bool in_place = out == logits && ld_out == ld_logits && dtype == out_dtype;
  const size_t nb = static_cast<size_t>(B);
  const Range others[] = {{tokens, span_bytes(B, L, ld_tokens, tokens_int64 ? 8 : 4)},
                          {lengths, nb * 4},
                          {prompt_lengths, nb * 4},
                          {repetition, nb * 4},
                          {frequency, nb * 4},
                          {presence, nb * 4},
                          {bias_ids, span_bytes(B, n_bias, n_bias, bias_int64 ? 8 : 4)},
                          {bias_values, span_bytes(B, n_bias, n_bias, 4)},
                          {allowed, span_bytes(B, words, ld_allowed, 4)}};
  if (!in_place && ranges_overlap(o, in)) return FLCE_ERR_INVALID_ARG;
  for (const Range& r : others)
    if (ranges_overlap(o, r)) return FLCE_ERR_INVALID_ARG;
  int sms = 0;
  const flce_status st = check_device(&sms);
  if (st != FLCE_OK) return st;
  ProcessArgs a = {};
  a.in_place = in_place;
  a.ld_logits = ld_logits;
  a.ld_out = ld_out;
  a.ld_tokens = ld_tokens;
  a.ld_allowed = ld_allowed;
  a.V = V;
  a.L = tokens ? L : 0;
  a.n_bias = static_cast<int>(n_bias);
  a.lengths = lengths;
  a.prompt_lengths = prompt_lengths;
  a.repetition = repetition;
  a.frequency = frequency;
  a.presence = presence;
  a.bias_values = bias_values;
  a.allowed = allowed;
  a.tokens = tokens;
  a.bias_ids = bias_ids;
  a.tokens_int64 = tokens_int64;
  a.bias_int64 = bias_int64;
  const auto s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t err;
  if (dtype == FLCE_BF16)
    err = out_dtype == FLCE_BF16 ? run_process<__nv_bfloat16, __nv_bfloat16>(logits, out, B, a, sms, s)
                                 : run_process<__nv_bfloat16, float>(logits, out, B, a, sms, s);
  else
    err = out_dtype == FLCE_BF16 ? run_process<float, __nv_bfloat16>(logits, out, B, a, sms, s)
                                 : run_process<float, float>(logits, out, B, a, sms, s);
  return err == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}
