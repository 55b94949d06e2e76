// Penalties for repeated tokens, biases and grammar masks on logits
// (flce_process_logits).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "flce_internal.h"
#include "flce_ops.h"

namespace flce {
namespace {

constexpr int kThreads = 512;
constexpr int kCols = 8192;  // columns per block

struct ProcessArgs {
  int64_t ld_logits, ld_out, ld_tokens, ld_allowed;
  int64_t V, L;
  int n_bias;
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

__device__ __forceinline__ float load_f(const float* p) { return *p; }
__device__ __forceinline__ float load_f(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_f(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Bits of a column's word: how often it was generated, and whether the prompt
// holds it.
constexpr unsigned kInPrompt = 0x80000000u;

template <class T, class O>
__global__ void __launch_bounds__(kThreads)
    process_kernel(const T* logits, O* out, const ProcessArgs a) {
  __shared__ unsigned hist[kCols];
  __shared__ unsigned short bias[kCols];  // 1 + index of the column's bias entry
  const int64_t b = blockIdx.y;
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * kCols;
  const int cols = static_cast<int>(min(int64_t{kCols}, a.V - v0));
  for (int c = threadIdx.x; c < kCols; c += kThreads) {
    hist[c] = 0u;
    bias[c] = 0;
  }
  __syncthreads();
  int64_t len = a.lengths ? a.lengths[b] : a.L;
  len = max(int64_t{0}, min(len, a.L));
  const int64_t prompt = a.prompt_lengths ? a.prompt_lengths[b] : 0;
  for (int64_t i = threadIdx.x; i < len; i += kThreads) {
    const int64_t c = id_at(a.tokens, a.tokens_int64, b * a.ld_tokens + i) - v0;
    if (c >= 0 && c < cols) {
      if (i < prompt) atomicOr(&hist[c], kInPrompt);
      else atomicAdd(&hist[c], 1u);
    }
  }
  if (threadIdx.x == 0)
    for (int i = 0; i < a.n_bias; ++i) {
      const int64_t c = id_at(a.bias_ids, a.bias_int64, b * a.n_bias + i) - v0;
      if (c >= 0 && c < cols) bias[c] = static_cast<unsigned short>(i + 1);
    }
  __syncthreads();
  const float rep = a.repetition ? a.repetition[b] : 1.f;
  const float freq = a.frequency ? a.frequency[b] : 0.f;
  const float pres = a.presence ? a.presence[b] : 0.f;
  for (int c = threadIdx.x; c < cols; c += kThreads) {
    const int64_t v = v0 + c;
    float l = load_f(logits + b * a.ld_logits + v);
    const unsigned h = hist[c];
    if (h) {
      l = l > 0.f ? l / rep : l * rep;
      const unsigned n = h & ~kInPrompt;
      l -= freq * static_cast<float>(n) + (n ? pres : 0.f);
    }
    if (bias[c]) l += a.bias_values[b * a.n_bias + bias[c] - 1];
    if (a.allowed && !((a.allowed[b * a.ld_allowed + (v >> 5)] >> (v & 31)) & 1)) l = -INFINITY;
    store_f(out + b * a.ld_out + v, l);
  }
}

template <class T, class O>
cudaError_t run_process(const void* logits, void* out, int64_t B, const ProcessArgs& a,
                        cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((a.V + kCols - 1) / kCols), static_cast<unsigned>(B));
  process_kernel<T, O><<<grid, kThreads, 0, s>>>(static_cast<const T*>(logits),
                                                 static_cast<O*>(out), a);
  note_launch();
  return cudaGetLastError();
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
    err = out_dtype == FLCE_BF16 ? run_process<__nv_bfloat16, __nv_bfloat16>(logits, out, B, a, s)
                                 : run_process<__nv_bfloat16, float>(logits, out, B, a, s);
  else
    err = out_dtype == FLCE_BF16 ? run_process<float, __nv_bfloat16>(logits, out, B, a, s)
                                 : run_process<float, float>(logits, out, B, a, s);
  return err == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}
