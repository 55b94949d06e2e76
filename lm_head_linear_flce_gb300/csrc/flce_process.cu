// Penalties for repeated tokens, biases and grammar masks on logits
// (flce_process_logits).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "flce_device.cuh"
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
// One row of 152064 takes 4.2 us, a launch and three trips to memory; 256 x 128255
// float32 with histories of 2000 47.6 us (5.6 TB/s), in place 63; 64 x 151936 bf16
// with masks 12.8 us without histories, with 2000 ids a row 14.9, to bf16 14.2, in
// place 15.8 (no loads ahead there), and 28 us with up to 32768 ids of a text's
// distribution a row, where the ids' instructions and the row's reading by each of
// its four blocks take over.  Where a row starts elsewhere in its 16 bytes than its
// output, its columns go one by one: 64 rows of 128255, 128256 apart, into rows 128255
// apart take 31 us, into rows 128256 apart 13.5.  (Counting in a kernel beside a
// streaming one: 62 us where this then took 45; grouping a warp's equal ids before the
// update was slower too.)
//
// A column's counter is its number of generated occurrences, and a top bit for
// "in the prompt".  16 bits do for a history of up to 2^15 (half the shared
// memory, so twice the columns a block): with a prompt at least one token is not
// generated and the count stays below the bit, without one no bit is set and all
// sixteen are the count.  Longer histories take 32.
//
// Biases: up to kBiasList entries a row, a block lists those of its columns and
// applies them after its windows, from the logit read beforehand; the list costs
// no shared memory per column.  More entries go by an index per column, 1 + the
// largest of the column's entries.
constexpr int kNoBias = 0, kListedBias = 1, kIndexedBias = 2;
constexpr int kBiasList = 512;

constexpr int kWin = 4;  // consecutive columns a thread takes at a time: neighbouring lanes
                         // then read and write whole lines in either type

template <bool WIDE>
struct Counts {
  static constexpr uint32_t kPrompt = WIDE ? 0x80000000u : 0x8000u;
  uint32_t* words;
  // Adds one to counter c, or sets its prompt bit; nothing if not `mine`.  (Both
  // updates under predicates: 128 ids of a warp rarely take one way.)
  __device__ __forceinline__ void add(uint32_t c, bool mine, bool prompt) const {
    const uint32_t w = static_cast<uint32_t>(__cvta_generic_to_shared(words)) +
                       (WIDE ? 4 * c : (2 * c & ~3u));
    const uint32_t sh = WIDE ? 0 : 16 * (c & 1);
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %0, 0;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "@p red.shared.add.u32 [%2], %3;\n\t"
        "@q red.shared.or.b32 [%2], %4;\n\t}" ::"r"(static_cast<uint32_t>(mine && !prompt)),
        "r"(static_cast<uint32_t>(mine && prompt)), "r"(w), "r"(1u << sh), "r"(kPrompt << sh)
        : "memory");
  }
  __device__ uint32_t at(int c) const {
    return WIDE ? words[c] : words[c >> 1] >> 16 * (c & 1) & 0xffffu;
  }
  // The window's counters, at c (a multiple of kWin).
  using Packed = typename std::conditional<WIDE, uint4, uint2>::type;
  __device__ Packed window(int c) const {
    return *reinterpret_cast<const Packed*>(words + (WIDE ? c : c >> 1));
  }
};
__device__ __forceinline__ bool any(const uint4& p) { return (p.x | p.y | p.z | p.w) != 0; }
__device__ __forceinline__ bool any(const uint2& p) { return (p.x | p.y) != 0; }
__device__ __forceinline__ void unpack(const uint4& p, uint32_t (&n)[kWin]) {
  n[0] = p.x, n[1] = p.y, n[2] = p.z, n[3] = p.w;
}
__device__ __forceinline__ void unpack(const uint2& p, uint32_t (&n)[kWin]) {
  n[0] = p.x & 0xffffu, n[1] = p.x >> 16, n[2] = p.y & 0xffffu, n[3] = p.y >> 16;
}

// Four consecutive logits as loaded, and as floats.
__device__ __forceinline__ uint4 load_raw(const float* p) {
  return *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ uint2 load_raw(const __nv_bfloat16* p) {
  return *reinterpret_cast<const uint2*>(p);
}
__device__ __forceinline__ void floats(const uint4& r, float (&v)[kWin]) {
  v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y);
  v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void floats(const uint2& r, float (&v)[kWin]) {
  v[0] = __uint_as_float(r.x << 16), v[1] = __uint_as_float(r.x & 0xffff0000u);
  v[2] = __uint_as_float(r.y << 16), v[3] = __uint_as_float(r.y & 0xffff0000u);
}
__device__ __forceinline__ void store_window(float* p, const float (&v)[kWin]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store_window(__nv_bfloat16* p, const float (&v)[kWin]) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}
__device__ __forceinline__ float load_f(const float* p) { return *p; }
__device__ __forceinline__ float load_f(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_f(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Blocks that share an SM, shared memory permitting.
template <int THREADS>
constexpr int kPerSm = THREADS <= 256 ? 4 : 3;

// Windows a thread has on their way, in slots of its own in shared memory, in
// bytes: 64 KB an SM with four small blocks there, 72 or 48 KB with three or two
// large ones, which need the room for counters.
template <int THREADS>
constexpr int kRingBytes = THREADS <= 256 ? 64 : 48;
template <class T, int THREADS>
constexpr int kRing = kRingBytes<THREADS> / (kWin * static_cast<int>(sizeof(T)));

template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(BYTES)
               : "memory");
}

// The column of an id relative to v0, all others (negative ids among them) as a
// number that no block has columns for.
__device__ __forceinline__ uint32_t column(int t, int v0) {
  return static_cast<uint32_t>(t) - static_cast<uint32_t>(v0);
}
__device__ __forceinline__ uint32_t column(int64_t t, int v0) {
  const uint64_t c = static_cast<uint64_t>(t) - static_cast<uint64_t>(v0);
  return c >> 32 ? ~0u : static_cast<uint32_t>(c);
}

// f(column, i) for each i < len of a row's history, THREADS threads together: 16
// bytes at a time, kIdLoads of them on their way while as many are counted (as
// many as registers allow: four in blocks of 512 spill and are 6% slower).
template <int THREADS>
constexpr int kIdLoads = THREADS <= 256 ? 4 : 2;
template <int THREADS, class I, class F>
__device__ __forceinline__ void each_id(const I* t, int len, int v0, const F& f) {
  constexpr int kPer = 16 / sizeof(I), kLoads = kIdLoads<THREADS>;
  const int tid = threadIdx.x;
  const int head =
      min(len, static_cast<int>((0 - reinterpret_cast<uintptr_t>(t)) / sizeof(I) % kPer));
  const int packs = (len - head) / kPer, tail = head + packs * kPer;
  if (tid < head + len - tail) {
    const int i = tid < head ? tid : tail + tid - head;
    f(column(t[i], v0), i);
  }
  const uint4* p = reinterpret_cast<const uint4*>(t + head);
  uint4 next[kLoads];
  const auto fetch = [&](int k0) {  // k0 + THREADS * kLoads < 2^31 / kPer + 4096
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      if (k0 + u * THREADS < packs) next[u] = p[k0 + u * THREADS];
  };
  fetch(tid);
  for (int k0 = tid; k0 < packs; k0 += THREADS * kLoads) {
    uint4 now[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) now[u] = next[u];
    fetch(k0 + THREADS * kLoads);
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int k = k0 + u * THREADS;
      if (k >= packs) break;
      alignas(16) I ids[kPer];
      *reinterpret_cast<uint4*>(ids) = now[u];
#pragma unroll
      for (int j = 0; j < kPer; ++j) f(column(ids[j], v0), head + k * kPer + j);
    }
  }
}

// The windows of a block of `cols` columns, the first starting `shift` columns
// before them: `all` of them, of which [lo, hi) lie wholly inside (none where
// `whole` is false, or where the columns do not fill one).
struct Windows {
  int all, lo, hi;
};
__host__ __device__ constexpr Windows windows_of(int shift, int cols, bool whole) {
  const int all = (shift + cols + kWin - 1) / kWin;
  if (!whole) return {all, all, all};
  const int lo = (shift + kWin - 1) / kWin, hi = (shift + cols) / kWin;
  return {all, lo, hi > lo ? hi : lo};
}
// The e-th window that is not whole.
__host__ __device__ constexpr int edge_window(const Windows& w, int e) {
  return e < w.lo ? e : e - w.lo + w.hi;
}
// Every window comes up once, as an edge or as a whole one: in place, a column
// that two threads take is a race.
constexpr bool each_window_once() {
  for (int whole = 0; whole < 2; ++whole)
    for (int shift = 0; shift < kWin; ++shift)
      for (int cols = 1; cols <= 5 * kWin; ++cols) {
        const Windows w = windows_of(shift, cols, whole);
        for (int k = 0; k < w.all; ++k) {
          int times = w.lo <= k && k < w.hi;
          for (int e = 0; e < w.all - (w.hi - w.lo); ++e) times += edge_window(w, e) == k;
          if (times != 1) return false;
        }
      }
  return true;
}
static_assert(each_window_once());

// Mask words a block of `cols` columns may touch, with one to spare for the
// word behind a window's first, in steps of 16 bytes.
__host__ __device__ constexpr int mask_words(int cols) { return (cols / 32 + 3 + 3) / 4 * 4; }

template <class T, class O, bool WIDE, int BIAS, int THREADS>
__global__ void __launch_bounds__(THREADS, kPerSm<THREADS>)
    process_kernel(const T* logits, O* out, const ProcessArgs a) {
  extern __shared__ __align__(16) uint32_t smem[];
  constexpr int kSlots = kRing<T, THREADS>;
  griddep_launch_dependents();
  griddep_wait();
  const int64_t b = blockIdx.y;
  const int v0 = static_cast<int>(blockIdx.x) * a.cols;  // V <= 2^30
  const int cols = min(a.cols, static_cast<int>(a.V) - v0);
  const T* in_row = logits + b * a.ld_logits + v0;
  O* out_row = out + b * a.ld_out + v0;
  // Windows start `shift` columns before the block's first, where both rows are
  // aligned to one; if that differs, every window goes column by column.
  const auto misaligned = [](const auto* p) {
    return static_cast<int>(reinterpret_cast<uintptr_t>(p) / sizeof(*p) % kWin);
  };
  const int shift = misaligned(in_row);
  const bool vec = shift == misaligned(out_row);
  const Windows win = windows_of(shift, cols, vec);
  const int windows = win.all, w_lo = win.lo, w_hi = win.hi;

  // What depends on nothing else is asked for at once: the row's scalars and the
  // thread's first windows.
  const int64_t len0 = a.lengths ? a.lengths[b] : a.L;
  const int prompt = a.prompt_lengths ? a.prompt_lengths[b] : 0;
  const float rep = a.repetition ? a.repetition[b] : 1.f;
  const float freq = a.frequency ? a.frequency[b] : 0.f;
  const float pres = a.presence ? a.presence[b] : 0.f;

  // Shared memory: the ring, the block's bias list, its mask words, counters,
  // bias indices (the last two one per window column).
  using Raw = decltype(load_raw(in_row));
  Raw* ring = reinterpret_cast<Raw*>(smem) + threadIdx.x;  // this thread's slots, THREADS apart
  uint32_t* listed = smem + kSlots * THREADS * sizeof(Raw) / 4;  // column << 16 | entry
  auto* before = reinterpret_cast<float*>(listed + kBiasList);      // its logit
  __shared__ int n_listed;
  uint32_t* mask = listed + (BIAS == kListedBias ? 2 * kBiasList : 0);
  const int slots = (windows * kWin + 7) / 8 * 8;
  Counts<WIDE> counts{mask + mask_words(a.cols)};
  uint32_t* bias = counts.words + (WIDE ? slots : slots / 2);
  const int words = (WIDE ? slots : slots / 2) + (BIAS == kIndexedBias ? slots / 2 : 0);
  // A thread's whole windows are k0 and every THREADS on; one group per window.
  const int k0 = w_lo + threadIdx.x;
  const int w_fetch = a.in_place ? 0 : w_hi;
  const T* src = in_row - shift + kWin * k0;
  const auto fetch = [&](const T* from, int k, Raw* slot) {
    if (k < w_fetch) copy_async<sizeof(Raw)>(slot, from);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    fetch(src + i * kWin * THREADS, k0 + i * THREADS, ring + i * THREADS);

  // mask word i holds columns 32 (v0 / 32 + i) and on
  const int first_word = v0 >> 5;
  if (a.allowed) {
    const int* m = a.allowed + b * a.ld_allowed;
    const int last = static_cast<int>((a.V - 1) >> 5);
    for (int i = threadIdx.x; i < mask_words(a.cols); i += THREADS)
      mask[i] = first_word + i <= last ? static_cast<uint32_t>(m[first_word + i]) : 0u;
  }
  for (int i = threadIdx.x; i < words / 4; i += THREADS)
    reinterpret_cast<uint4*>(counts.words)[i] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x == 0) n_listed = 0;
  __syncthreads();
  const int len = static_cast<int>(max(int64_t{0}, min(len0, a.L)));
  const auto count = [&](uint32_t c, int i) {  // entry i, c columns behind v0
    counts.add(c + shift, c < static_cast<uint32_t>(cols), i < prompt);
  };
  if (a.tokens_int64)
    each_id<THREADS>(static_cast<const int64_t*>(a.tokens) + b * a.ld_tokens, len, v0, count);
  else each_id<THREADS>(static_cast<const int*>(a.tokens) + b * a.ld_tokens, len, v0, count);
  if constexpr (BIAS != kNoBias) {
    for (int i = threadIdx.x; i < a.n_bias; i += THREADS) {
      const int64_t v = id_at(a.bias_ids, a.bias_int64, b * a.n_bias + i);
      if (v < v0 || v - v0 >= cols) continue;
      if constexpr (BIAS == kListedBias) {
        const int at = atomicAdd(&n_listed, 1), c = static_cast<int>(v - v0);
        listed[at] = static_cast<uint32_t>(c) << 16 | static_cast<uint32_t>(i);
        before[at] = load_f(in_row + c);
        continue;
      }
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

  // One column with its counter n and bias entry e (0: none).  The division is by
  // a row's one penalty: its reciprocal, unless that is near the type's ends.
  const uint32_t count_bits = WIDE || prompt > 0 ? ~Counts<WIDE>::kPrompt : ~0u;
  const float inverse = 1.f / rep;
  const bool tame = rep > 1e-30f && rep < 1e30f;
  const auto apply = [&](float l, uint32_t n, uint32_t e) {
    const uint32_t c = n & count_bits;
    const float up = tame ? l * inverse : l / rep;
    const float x = (l > 0.f ? up : l * rep) - fmaf(freq, static_cast<float>(c), c ? pres : 0.f);
    if (n) l = x;
    if (BIAS != kNoBias && e) l += a.bias_values[b * a.n_bias + e - 1];
    return l;
  };
  const int bit0 = v0 - shift - 32 * first_word;  // of a window's column 0, at k = 0
  // Columns of windows that are not whole, or all where the rows' alignments differ.
  const int edges = (windows - (w_hi - w_lo)) * kWin;
  for (int i = threadIdx.x; i < edges; i += THREADS) {
    const int k = edge_window(win, i / kWin);
    const int at = kWin * k + i % kWin, c = at - shift, bit = bit0 + at;
    if (c < 0 || c >= cols) continue;
    uint32_t e = 0;
    if constexpr (BIAS == kIndexedBias) e = bias[at >> 1] >> 16 * (at & 1) & 0xffffu;
    const bool ok = !a.allowed || (mask[bit >> 5] >> (bit & 31) & 1);
    store_f(out_row + c, ok ? apply(load_f(in_row + c), counts.at(at), e) : -INFINITY);
  }
  Raw* slot = ring;
  O* dst = out_row - shift + kWin * k0;
  for (int k = k0; k < w_hi; k += THREADS) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory");
    const auto n4 = counts.window(kWin * k);
    uint2 e4 = make_uint2(0, 0);
    if constexpr (BIAS == kIndexedBias) e4 = *reinterpret_cast<const uint2*>(bias + kWin / 2 * k);
    const bool some = any(n4) || (BIAS == kIndexedBias && any(e4));
    uint32_t ok = 0xfu;  // which of the window's columns are allowed
    if (a.allowed) {
      const int bit = bit0 + kWin * k, w = bit >> 5;
      ok = __funnelshift_r(mask[w], mask[w + 1], bit & 31) & 0xfu;
    }
    if (!(a.in_place && !some && ok == 0xfu)) {  // in place: not touched
      float l[kWin];
      floats(a.in_place ? load_raw(src) : *slot, l);
      if (some) {
        uint32_t n[kWin], e[kWin];
        unpack(n4, n);
        unpack(e4, e);
#pragma unroll
        for (int j = 0; j < kWin; ++j) l[j] = apply(l[j], n[j], e[j]);
      }
      if (ok != 0xfu) {
#pragma unroll
        for (int j = 0; j < kWin; ++j) l[j] = ok >> j & 1 ? l[j] : -INFINITY;
      }
      store_window(dst, l);
    }
    fetch(src + kSlots * kWin * THREADS, k + kSlots * THREADS, slot);
    slot = slot == ring + (kSlots - 1) * THREADS ? ring : slot + THREADS;
    src += kWin * THREADS;
    dst += kWin * THREADS;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if constexpr (BIAS == kListedBias) {
    __syncthreads();  // the block's windows are written
    for (int i = threadIdx.x; i < n_listed; i += THREADS) {
      const uint32_t mine = listed[i];
      bool last = true;  // of the entries with this column
      for (int k = 0; k < n_listed; ++k)
        last = last && !(listed[k] > mine && listed[k] >> 16 == mine >> 16);
      if (!last) continue;
      const int c = static_cast<int>(mine >> 16), bit = v0 + c - 32 * first_word;
      const bool ok = !a.allowed || (mask[bit >> 5] >> (bit & 31) & 1);
      const float l = apply(before[i], counts.at(c + shift), (mine & 0xffffu) + 1);
      store_f(out_row + c, ok ? l : -INFINITY);
    }
  }
}

// Shared memory an SM has for its blocks, and that a block may take: two an SM.
constexpr int kSmSmem = 227 * 1024, kMaxSmem = 113 * 1024;
// Columns that a block of 256 threads takes at most; more take 512.
constexpr int kSmallCols = 4096;

template <class T, class O, bool WIDE, int BIAS, int THREADS>
cudaError_t launch_process(const void* logits, void* out, int64_t B, const ProcessArgs& a,
                           int counters, cudaStream_t s) {
  // (the shift's window: 16 columns of counters more, in steps of 8)
  const int smem = kRingBytes<THREADS> * THREADS + (BIAS == kListedBias ? 8 * kBiasList : 0) +
                   4 * mask_words(a.cols) + (a.cols + 16) * counters;
  auto* k = process_kernel<T, O, WIDE, BIAS, THREADS>;
  static SmemLimit limit;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), kMaxSmem, &limit);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>((a.V + a.cols - 1) / a.cols), static_cast<unsigned>(B));
  const cudaError_t e2 = launch_overlapped(k, grid, dim3(THREADS), smem, s, 1,
                                           static_cast<const T*>(logits), static_cast<O*>(out), a);
  note_launch();
  return e2 != cudaSuccess ? e2 : cudaGetLastError();
}

template <class T, class O>
cudaError_t run_process(const void* logits, void* out, int64_t B, ProcessArgs a, int sms,
                        cudaStream_t s) {
  const bool wide = a.L > 32768;
  const int bias = a.n_bias == 0 ? kNoBias : a.n_bias <= kBiasList ? kListedBias : kIndexedBias;
  const int per_col = (wide ? 4 : 2) + (bias == kIndexedBias ? 2 : 0);
  // Blocks a row, n.  `per` of them share an SM, so that the SMs take
  // ceil(B n / (per SMs)) turns.  A turn is as long as a block's columns, three
  // tenths more for each block beside it; for each of its blocks the row's history,
  // which every block reads (an id costs about a column), and some 1024 columns of
  // setting up; and a start of some 2048.  Taken is the n with the least of that, of
  // those that fill their turns; blocks have 1024 columns at least and fit into
  // shared memory.  (Timed for 1 to 1024 rows and histories of up to 32768 this n is
  // 2% slower than the best one on average, 24% at worst.  16 x 152064 bf16,
  // histories of 32768: 1 block an SM 11.3 us, 2 14.5, 4 16.8; 8 rows without
  // histories: 4.2, 3.6, 4.2.)
  const auto smem_of = [&](int64_t cols) {  // of a block with 512 threads
    return 512 * kRingBytes<512> + 8 * kBiasList + 1024 + cols * (8 * per_col + 1) / 8;
  };
  const int64_t most = (kMaxSmem - smem_of(0)) * 8 / (8 * per_col + 1) / 64 * 64;
  const auto cols_of = [&](int64_t n) { return ((a.V + n - 1) / n + 63) / 64 * 64; };
  const int64_t least = (a.V + most - 1) / most, finest = std::max(least, (a.V + 1023) / 1024);
  int64_t blocks = least, best = INT64_MAX;
  for (int64_t fill = 1; fill <= 24; ++fill) {  // blocks an SM, all turns together
    const int64_t n = std::clamp<int64_t>(fill * sms / B, least, finest);
    const int64_t cols = cols_of(n);
    const int64_t per = cols <= kSmallCols ? kPerSm<256>
                                           : std::min<int64_t>(kPerSm<512>, kSmSmem / smem_of(cols));
    const int64_t at_once = std::min(per, (B * n + sms - 1) / sms);
    const int64_t turn = cols + cols * 3 * (at_once - 1) / 10 + at_once * (a.L + 1024) + 2048;
    const int64_t cost = (B * n + per * sms - 1) / (per * sms) * turn;
    if (cost < best) best = cost, blocks = n;
    if (n == finest) break;
  }
  a.cols = static_cast<int>(std::min(cols_of(blocks), most));
  const auto launch = [&](auto w, auto bm) {
    constexpr bool kW = decltype(w)::value;
    constexpr int kB = decltype(bm)::value;
    return a.cols <= kSmallCols ? launch_process<T, O, kW, kB, 256>(logits, out, B, a, per_col, s)
                          : launch_process<T, O, kW, kB, 512>(logits, out, B, a, per_col, s);
  };
  const auto by_bias = [&](auto w) {
    return bias == kNoBias       ? launch(w, std::integral_constant<int, kNoBias>{})
           : bias == kListedBias ? launch(w, std::integral_constant<int, kListedBias>{})
                                 : launch(w, std::integral_constant<int, kIndexedBias>{});
  };
  return wide ? by_bias(std::true_type{}) : by_bias(std::false_type{});
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
  OpRange range("flce_process_logits");
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
    err = out_dtype == FLCE_BF16
              ? run_process<__nv_bfloat16, __nv_bfloat16>(logits, out, B, a, sms, s)
              : run_process<__nv_bfloat16, float>(logits, out, B, a, sms, s);
  else
    err = out_dtype == FLCE_BF16 ? run_process<float, __nv_bfloat16>(logits, out, B, a, sms, s)
                                 : run_process<float, float>(logits, out, B, a, sms, s);
  return err == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}
