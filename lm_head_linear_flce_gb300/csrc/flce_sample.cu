// A token a row by temperature, top-k, top-p and min-p from a given random number
// (flce_sample_logits).
//
// One CTA takes a row, or a cluster of up to eight where rows are few.  It streams the row
// once, for the largest logit and, where every token counts, for their mass; what follows
// reads again, from L2, as little as the limits leave: a list of candidates for top-k, the
// tokens near the border for top-p.  What a row keeps is a prefix of its tokens in
// descending order (equal logits by id), which a logit t and a number say: all tokens
// above t, and the first so many of those equal to t.  The token is then the first, by id,
// whose cumulative mass among the kept ones exceeds u times their total.
//
// What bounds it (GB300, in a graph, inputs past L2, normal logits with forty likely ones a
// row, us at 256 x 152064 float32 / 64 x 152064 bf16 / 1 x 152064 bf16; the bytes alone would
// take 23 / 2.9 / 0.05):
//     no limits 55 / 20 / 9.9: 34 instructions a token in float32 and 31 in bf16, 57 % of the
//         issue slots (68 % on the SMs that have two of the 256 CTAs)
//     greedy 42 / 12 / 7.9: a pass for the largest (memory) and the tokens of some warps again
//     min-p 49 / 14 / 8.7: the same, and the kept ones' weights; 11 instructions a token
//     top-k of 1 to 1000, log-uniform, 67 / 25 / 11.3: a pass for the largest, the
//         candidates' list, and five to eight steps of about a microsecond each; 14
//         instructions a token, a fifth of the issue slots
//     top-p 166 to 171 / 60 / 30 to 33: three passes, 93 instructions a token in all; the
//         histogram's atomics; barriers
// One row takes its steps' latency: launch, pass, cluster barriers of 0.6 to 1 us.
//
// Masses are integers.  A token weighs 2^((l - max) / (T ln 2)) in units of 2^-42 (the
// largest 2^41 to 2^42 of them), off by 2^-29.3 of it at most (rms 2^-31.6) and by 0.55 of a
// unit.  Next to a border the cumulative mass is right to 2e-11 on a broad row, to 4e-10
// between two likely tokens, and on any row to 2^-28 + 1.1 V 2^-42 (the second where many
// tokens weigh less than a unit), where FP32 sums would be off by 1e-7 on a vocabulary with a
// border every 1e-5.  Sums of integers do not depend on their order.  What depends on how a
// row is split over lanes is the mass that is taken while the largest logit is still looked
// for (no top-k, and no min-p or top-p too): a lane's sum is rounded as that goes up, to a
// unit, and the warp's once more.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <climits>

#include "flce_device.cuh"
#include "flce_internal.h"
#include "flce_ops.h"

namespace flce {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxWarps = kWarps * kMaxCluster;  // of a row
constexpr int64_t kMaxVocab = int64_t{1} << 21;
constexpr int kMaxSlots = 1032;           // of a warp: kMaxVocab float32 logits in one CTA
constexpr float kGreedyBelow = 0x1p-64f;  // temperatures that take the largest logit
// The largest temperature (all logits up to 2^50 weigh the same there): 1 / T in two floats
// is as precise as weights need it up to about 2^117.
constexpr float kHottest = 0x1p100f;

struct SampleArgs {
  const void* logits;
  int64_t ld;
  int V;
  const float* u;
  const float* temperature;
  const int* top_k;
  const float* top_p;
  const float* min_p;
  int64_t* out;
};

// ------------------------------------------------------------------ weights
// 2^(j / 32) as a float and what that leaves of it in the exponent: 2^(j / 32) =
// first * 2^second.
__constant__ float2 kPow2[32] = {
    {0x1p0f, 0.f}, {0x1.059b0ep0f, -0x1.23c062p-24f}, {0x1.0b5586p0f, 0x1.1ecccap-24f},
    {0x1.11301ep0f, -0x1.588ac2p-24f}, {0x1.172b84p0f, -0x1.293ab8p-26f}, {0x1.1d4874p0f, -0x1.2e3b84p-24f},
    {0x1.2387a6p0f, 0x1.2512a4p-24f}, {0x1.29e9ep0f, -0x1.af7176p-25f}, {0x1.306fep0f, 0x1.8bbfd2p-25f},
    {0x1.371a74p0f, -0x1.4d327cp-25f}, {0x1.3dea64p0f, 0x1.c0bec4p-25f}, {0x1.44e086p0f, 0x1.bb86d2p-30f},
    {0x1.4bfdaep0f, -0x1.800eaep-25f}, {0x1.5342b6p0f, -0x1.46f4ap-25f}, {0x1.5ab07ep0f, -0x1.728d0ep-27f},
    {0x1.6247ecp0f, -0x1.0712d2p-24f}, {0x1.6a09e6p0f, 0x1.a82ebcp-26f}, {0x1.71f75ep0f, 0x1.1d0e32p-25f},
    {0x1.7a1148p0f, -0x1.79b05ep-25f}, {0x1.82589ap0f, -0x1.99e9aep-26f}, {0x1.8ace54p0f, 0x1.036b6ep-27f},
    {0x1.93737cp0f, -0x1.bd26f8p-25f}, {0x1.9c4918p0f, 0x1.2ec1d4p-27f}, {0x1.a5503cp0f, -0x1.81eap-25f},
    {0x1.ae89fap0f, -0x1.6cd47cp-26f}, {0x1.b7f77p0f, -0x1.5db27ep-25f}, {0x1.c199bep0f, -0x1.04ae88p-27f},
    {0x1.cb720ep0f, -0x1.3b49d2p-27f}, {0x1.d5818ep0f, -0x1.2fc81cp-27f}, {0x1.dfc974p0f, -0x1.345598p-25f},
    {0x1.ea4afap0f, 0x1.fda57cp-28f}, {0x1.f50766p0f, -0x1.af2102p-27f}};

// a + b, and what its rounding leaves.
__device__ __forceinline__ float2 two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), back = __fsub_rn(s, a);
  return make_float2(s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, back)), __fsub_rn(b, back)));
}

// What turns a row's logits into weights.  With c = 1 / (T ln 2) a weight is
// 2^(c (l - base) - shift): base is the largest logit where |c max| is very large (l - base
// is then exact for every l that weighs anything), else 0 with shift = ceil(c max), so that
// l is used as it is.  c in two floats.
constexpr float kLargestShift = 4096.f;
struct Scale {
  float base, least, c_hi, c_lo, magic;
};
constexpr float kMagic = 0x1.8p18f;   // + x rounds x to 1/32; its last bits count them
constexpr float kMagicA = 0x1.8p2f;   // the same for units of 2^-21 and of 2^-42, in
constexpr float kMagicB = 0x1.8p-19f; // which a weight is a + b
constexpr uint32_t kBitsA = 0x40c00000u, kBitsB = 0x36400000u;

// c of a temperature, in two floats.
__device__ __forceinline__ float2 inverse_of(float T) {
  constexpr float kHi = 0x1.715476p0f, kLo = 0x1.4ae0cp-26f;  // 1 / ln 2
  const float hi = __fdiv_rn(kHi, T);
  return make_float2(hi, __fdividef(fmaf(-hi, T, kHi) + kLo, T));
}
__device__ __forceinline__ Scale make_scale(float top, float2 c) {
  if (top == INFINITY) return {top, 0.f, 0.f, 0.f, kMagic};  // (only +infinities are weighed)
  Scale s;
  s.c_hi = c.x;
  s.c_lo = c.y;
  const float x = top * s.c_hi;
  const bool from_top = !(fabsf(x) <= kLargestShift);
  const float shift = from_top ? 0.f : ceilf(x);
  s.base = from_top ? top : 0.f;
  s.least = __fdividef(shift - 60.f, s.c_hi);  // below it a weight is less than 2^-59
  s.magic = kMagic - shift;
  return s;
}

// A token's weight as a * 2^-21 + b * 2^-42, each as the float that holds its bits above
// kBitsA and kBitsB.  With x = c (l - base) = k / 32 + f, |f| <= 1/64: 2^x by the table
// (Tang 1989) times 2^f by its series, whose f^4 is taken as the multiple of f^2 nearest to
// it; f carries the rounding error of the table's entry.  -infinity and NaN weigh nothing.
// Written with intrinsics so that every use rounds alike.  (Two values an instruction cost
// more registers than they save time.)
template <bool BASE = true>
__device__ __forceinline__ void weigh(float l, const Scale& s, const float2* table, uint32_t& a,
                                      uint32_t& b) {
  const float d = fmaxf(BASE ? __fsub_rn(l, s.base) : l, s.least);
  const float z = __fmaf_rn(d, s.c_hi, s.magic);
  const uint32_t k = __float_as_uint(z);
  const float2 t = table[k & 31];
  const float f = __fadd_rn(__fmaf_rn(d, s.c_hi, __fsub_rn(s.magic, z)), __fmaf_rn(d, s.c_lo, t.y));
  constexpr float kLn2 = 0.69314718055994531f;
  constexpr float kFourth = kLn2 * kLn2 * kLn2 * kLn2 / 24 * (5.f / 7) / (64 * 64);
  float p = __fmaf_rn(f, kLn2 * kLn2 * kLn2 / 6, kLn2 * kLn2 / 2 + kFourth);
  p = __fmul_rn(f, __fmaf_rn(f, p, kLn2));
  // (k's bits above the table's are the exponent; the constant's fall off the top, and the
  // table's entries are less by the others)
  const float th = __uint_as_float(__float_as_uint(t.x) + (k << 18));
  const float fa = __fadd_rn(__fmaf_rn(th, p, th), kMagicA);
  const float fb = __fadd_rn(__fmaf_rn(th, p, __fsub_rn(th, __fsub_rn(fa, kMagicA))), kMagicB);
  a = __float_as_uint(fa);
  b = __float_as_uint(fb);
}
// The mass of n weights, from the sums of their a and b modulo 2^32 (n <= 1024).
__device__ __forceinline__ uint64_t mass_of(uint32_t a, uint32_t b, uint32_t n) {
  const int64_t ia = a - n * kBitsA, ib = static_cast<int32_t>(b - n * kBitsB);
  return static_cast<uint64_t>(ia * (int64_t{1} << 21) + ib);
}
__device__ __forceinline__ uint64_t weight(float l, const Scale s, const float2* table) {
  uint32_t a, b;
  weigh(l, s, table, a, b);
  return mass_of(a, b, 1);
}

// Weights being added up.
struct Adder {
  uint64_t mass = 0;
  uint32_t a = 0, b = 0, n = 0;
  template <bool BASE = true, int PER>
  __device__ __forceinline__ void add(const float (&l)[PER], const Scale& s, const float2* table) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      uint32_t ka, kb;
      weigh<BASE>(l[j], s, table, ka, kb);
      a += ka;
      b += kb;
    }
    n += PER;
    if (n >= 512) flush();  // the sums of so many fit into 32 bits
  }
  __device__ __forceinline__ void flush() {
    mass += mass_of(a, b, n);
    a = b = n = 0;
  }
};

// ------------------------------------------------------------ a row's logits
// A row in units of 16 bytes, the first starting `shift` elements before it.  32 units
// are a slot, a lane of a warp each; a warp has consecutive slots, a lane its unit of each.
// Elements outside the row are -infinity.
template <class T>
struct Part {
  static constexpr int kPer = 16 / static_cast<int>(sizeof(T));
  const T* p;
  const uint4* aligned;
  int V, shift, slots;
  int u0, each;  // this lane's first unit, and how many
  bool inner;    // the warp's units lie in the row

  __device__ Part(const SampleArgs& a, int64_t b)
      : p(static_cast<const T*>(a.logits) + b * a.ld), V(a.V) {
    shift = static_cast<int>(reinterpret_cast<uintptr_t>(p) % 16 / sizeof(T));
    slots = ((V + shift + kPer - 1) / kPer + 31) / 32;
    aligned = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t{15});
  }
  // The first slot of warp w of `warps` (a product below 2^31).
  __device__ int first_slot(int w, int warps) const {
    return static_cast<int>(static_cast<uint32_t>(slots * w) / static_cast<uint32_t>(warps));
  }
  __device__ int warp_of(int id, int warps) const {
    const int slot = (id + shift) / (32 * kPer);  // first_slot(w) <= slot < first_slot(w + 1)
    return ((slot + 1) * warps - 1) / slots;
  }
  __device__ int first(int u) const { return u * kPer - shift; }  // column of a unit's first element
  __device__ bool whole(int u) const { return first(u) >= 0 && first(u) + kPer <= V; }
  __device__ float at(int c) const {
    if (c < 0 || c >= V) return -INFINITY;
    if constexpr (sizeof(T) == 4) return p[c];
    else return __bfloat162float(p[c]);
  }
  __device__ __noinline__ uint4 load_edge(int u) const {
    const int c = first(u);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4)
        w[i] = __float_as_uint(at(c + i));
      else  // (bf16 values: their lower halves are 0)
        w[i] = __float_as_uint(at(c + 2 * i)) >> 16 | __float_as_uint(at(c + 2 * i + 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ uint4 load(int u) const {
    return whole(u) ? aligned[u] : load_edge(u);
  }
  __device__ static __forceinline__ void floats(const uint4& r, float (&v)[kPer]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w[i]);
      else v[i] = __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
  }
  // f(a unit's column, its logits) for the units of some of the warp's lanes, spread over
  // all of them where these are few.
  static constexpr int kFlat = 4;
  template <int BATCH, class F>
  __device__ __forceinline__ void stream_of(uint32_t lanes, const F& f) const;
  // f(place in the batch, the unit's column, its logits) for the lane's units, a batch of
  // them loaded at once.
  template <int BATCH, class F>
  __device__ __forceinline__ void stream(const F& f) const {
    int s = 0;
    for (; s + BATCH <= each; s += BATCH) {
      uint4 r[BATCH];
      const int u = u0 + s * 32;
      if (inner) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) r[i] = aligned[u + i * 32];
      } else {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) r[i] = load(u + i * 32);
      }
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        float v[kPer];
        floats(r[i], v);
        f(i, first(u + i * 32), v);
      }
    }
    if (s == each) return;
    uint4 r[BATCH];
    const int u = u0 + s * 32;
#pragma unroll
    for (int i = 0; i + 1 < BATCH; ++i)
      if (s + i < each) r[i] = load(u + i * 32);
#pragma unroll
    for (int i = 0; i + 1 < BATCH; ++i) {
      if (s + i >= each) break;
      float v[kPer];
      floats(r[i], v);
      f(i, first(u + i * 32), v);
    }
  }
};
template <class T>
template <int BATCH, class F>
__device__ __forceinline__ void Part<T>::stream_of(uint32_t lanes, const F& f) const {
  constexpr int kHalf = 16;
  if (__popc(lanes) > kHalf) {
    stream<BATCH>([&](int, int c, const float (&v)[kPer]) { f(c, v); });
    return;
  }
  const int lane = threadIdx.x & 31, total = __popc(lanes) * each;
  int place = 0;  // of the lane-th one of them
  for (int r = 0; lanes; ++r, lanes &= lanes - 1)
    if (r == lane) place = __ffs(lanes) - 1;
  // this thread's unit: the slot-th of the which-th lane
  int which = lane / each, slot = lane - which * each;
#pragma unroll 1
  for (int i0 = 0; i0 < total; i0 += 32 * kFlat) {
    uint4 r[kFlat];
    int u[kFlat];
#pragma unroll
    for (int i = 0; i < kFlat; ++i) {
      u[i] = u0 - lane + __shfl_sync(0xffffffffu, place, which & 31) + slot * 32;
      // (past the last one: NaN, which is in no range)
      r[i] = i0 + i * 32 + lane < total ? load(u[i]) : make_uint4(~0u, ~0u, ~0u, ~0u);
      slot += 32;
      while (slot >= each) {
        slot -= each;
        ++which;
      }
    }
#pragma unroll
    for (int i = 0; i < kFlat; ++i) {
      if (i0 + i * 32 >= total) break;
      float v[kPer];
      floats(r[i], v);
      f(first(u[i]), v);
    }
  }
}
constexpr int kWide = 8, kFew = 4;  // batches: of passes that do little, and of those that weigh

// Logits in an order of integers (equal ones, but for the sign of a zero, alike).
// bf16 logits differ in the upper half alone.
template <class T>
__device__ __forceinline__ int key_of(float l) {
  const int i = __float_as_int(l);
  return (i < 0 ? i ^ 0x7fffffff : i) >> (sizeof(T) == 2 ? 16 : 0);
}
template <class T>
__device__ __forceinline__ float value_of(int k) {
  if constexpr (sizeof(T) == 2) k = k < 0 ? static_cast<int>(static_cast<uint32_t>(k) << 16 | 0xffffu)
                                          : static_cast<int>(static_cast<uint32_t>(k) << 16);
  return __int_as_float(k < 0 ? k ^ 0x7fffffff : k);
}

// ----------------------------------------------------- sums over the cluster
__device__ __forceinline__ uint64_t warp_sum_u64(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <class I>
__device__ __forceinline__ I warp_scan(I v) {  // of this lane and those before
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const I x = __shfl_up_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) >= o) v += x;
  }
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

constexpr int kList = 2048;        // tokens of a list
constexpr int kCompared = 64;      // of which are compared with one another
constexpr int kBins = 2048;        // of a histogram
constexpr int kGroups = 32;        // of bins, whose sums the CTAs exchange
constexpr int kGroupBins = kBins / kGroups;

// What the CTAs of a cluster read of one another, and what a CTA works in.
struct Shared {
  // one entry of every warp of the row, in every CTA; two sets, used in turn (who writes
  // one again has passed a barrier since its last readers did)
  uint64_t mass[2][kMaxWarps];
  uint32_t count[2][kMaxWarps];
  uint64_t group[kMaxCluster][kGroups];
  uint64_t list[kList];  // this CTA's tokens near a border: key << 32 | ~id
  union {
    uint32_t bins[kBins];
    uint64_t work[kList];  // every CTA's list, in order
    struct {
      uint64_t mass[kMaxSlots];
      uint32_t ties[kMaxSlots];
    } slot;  // of the warp that has the token
  };
  uint64_t weights[kList / 2];  // select_key's
  uint64_t part[kWarps];
  float2 table[32];
  float2 inverse;    // c of the temperature
  float2 log_min_p;  // T ln(min_p)
  uint64_t before, border;
  uint32_t listed, rank;
  int found[2];
};

struct Sum {
  uint64_t mass;
  uint32_t count;
};

struct Cluster {
  Shared& sh;
  int rank, ctas, phase;

  // Gives every CTA this warp's entry, and waits for all of them.
  __device__ __forceinline__ void share(uint64_t mass, uint32_t count) {
    const int lane = threadIdx.x & 31, me = rank * kWarps + (threadIdx.x >> 5);
    phase ^= 1;
    if (lane < ctas) {
      st_cluster_u64(mapa_shared(smem_u32(&sh.mass[phase][me]), lane), mass);
      st_shared_cluster_u32(mapa_shared(smem_u32(&sh.count[phase][me]), lane), count);
    }
    cluster_arrive();
    cluster_wait();
  }
  __device__ __forceinline__ Sum sum() const {
    uint64_t m = 0;
    uint32_t n = 0;
    for (int i = threadIdx.x & 31; i < ctas * kWarps; i += 32) {
      m += sh.mass[phase][i];
      n += sh.count[phase][i];
    }
    return {warp_sum_u64(m), __reduce_add_sync(0xffffffffu, n)};
  }
};

// ------------------------------------------------------- lists in shared memory
__device__ __forceinline__ uint64_t list_entry(float l, int id) {
  const uint32_t key = static_cast<uint32_t>(key_of<float>(l + 0.f)) ^ 0x80000000u;
  return static_cast<uint64_t>(key) << 32 | (static_cast<uint32_t>(id) ^ 0xffffffffu);
}
__device__ __forceinline__ float listed_logit(uint64_t e) {
  return value_of<float>(static_cast<int>(static_cast<uint32_t>(e >> 32) ^ 0x80000000u));
}
__device__ __forceinline__ int listed_id(uint64_t e) {
  return static_cast<int>(~static_cast<uint32_t>(e));
}

// The block's sum, on every thread.
__device__ __forceinline__ uint64_t block_sum(Shared& sh, uint64_t v) {
  const int lane = threadIdx.x & 31;
  v = warp_sum_u64(v);
  if (lane == 0) sh.part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = warp_sum_u64(lane < kWarps ? sh.part[lane] : 0);
  __syncthreads();
  return v;
}

// Of a list's n tokens (fewer than kList), the key at which the weights of tokens with that
// key or a larger one reach `target`, as all of them do; and the weight above that key.
// key(i): from `first` to `last`, or 0 where a token does not count; weight_of(i): at most
// 2^42.
//
// A round adds the weights up in 512 bins of the range (two halves of 21 bits each) and
// goes on with the tokens of the one that has the border; 64 tokens are compared with one
// another.  Nothing is sorted: an order by logit and then one by id took 17 us for 1200
// tokens of bf16, two of these searches take 4.
struct Border {
  uint64_t key, above;
};
template <class K, class W>
__device__ __forceinline__ Border select_key(Shared& sh, int n, const K& key, const W& weight_of,
                                               uint64_t first, uint64_t last, uint64_t target) {
  constexpr int kHalf = 21, kEach = kThreads / kCompared;
  static_assert(sizeof(sh.weights) >= 8 * kThreads + 2 * kList && kList % kThreads == 0);
  uint32_t* const upper = reinterpret_cast<uint32_t*>(sh.weights);
  uint32_t* const lower = upper + kThreads;
  uint16_t* const left = reinterpret_cast<uint16_t*>(lower + kThreads);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  bool whole = true;  // (then all are left)
  const auto at = [&](int q) { return whole ? q : static_cast<int>(left[q]); };
  uint64_t above = 0;
#pragma unroll 1
  while (n > kCompared && first < last) {
    const int shift = max(0, 64 - __clzll(static_cast<long long>(last - first)) - 9);
    upper[threadIdx.x] = lower[threadIdx.x] = 0;
    __syncthreads();
#pragma unroll 1
    for (int q = threadIdx.x; q < n; q += kThreads) {
      const int i = at(q);
      const uint64_t k = key(i);
      if (k < first || k > last) continue;
      const uint64_t w = weight_of(i);
      const uint32_t bin = static_cast<uint32_t>((k - first) >> shift);
      atomicAdd(&upper[bin], static_cast<uint32_t>(w >> kHalf));
      atomicAdd(&lower[bin], static_cast<uint32_t>(w) & ((1u << kHalf) - 1));
    }
    __syncthreads();
    if (threadIdx.x == 0) sh.listed = 0;
    const int bin = kThreads - 1 - threadIdx.x;  // larger keys first
    const uint64_t m = (static_cast<uint64_t>(upper[bin]) << kHalf) + lower[bin];
    uint64_t upto = warp_scan(m);
    if (lane == 31) sh.part[warp] = upto;
    __syncthreads();
    upto += above + warp_sum_u64(lane < warp ? sh.part[lane] : 0);
    if (upto >= target && upto - m < target) {
      sh.before = upto - m;
      sh.found[0] = bin;
    }
    __syncthreads();
    above = sh.before;
    first += static_cast<uint64_t>(sh.found[0]) << shift;
    last = min(last, first + ((uint64_t{1} << shift) - 1));
    int mine[kList / kThreads];
#pragma unroll
    for (int j = 0; j < kList / kThreads; ++j) {
      const int q = threadIdx.x + j * kThreads;
      mine[j] = q < n ? at(q) : -1;
      if (mine[j] >= 0) {
        const uint64_t k = key(mine[j]);
        if (k < first || k > last) mine[j] = -1;
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kList / kThreads; ++j)
      if (mine[j] >= 0) left[atomicAdd(&sh.listed, 1)] = static_cast<uint16_t>(mine[j]);
    __syncthreads();
    n = static_cast<int>(sh.listed);
    whole = false;
  }
  if (first == last) return {first, above};
  const int q = threadIdx.x / kEach, i = at(min(q, n - 1));
  const uint64_t k = key(i);
  uint64_t larger = 0, equal = 0;
  for (int r = threadIdx.x % kEach; r < n; r += kEach) {
    const uint64_t x = key(at(r)), w = weight_of(at(r));
    larger += x > k ? w : 0;
    equal += x == k ? w : 0;
  }
#pragma unroll
  for (int o = kEach / 2; o > 0; o >>= 1) {
    larger += __shfl_xor_sync(0xffffffffu, larger, o);
    equal += __shfl_xor_sync(0xffffffffu, equal, o);
  }
  larger += above;
  if (k != 0 && larger < target && larger + equal >= target) {  // (one key; the same above it)
    sh.border = k;
    sh.before = larger;
  }
  __syncthreads();
  return {sh.border, sh.before};
}

// ------------------------------------------------------------------- bins
// Bins of a token: of its distance from the largest logit, 1/64 of its octave each from
// 2^-12 on, for counts (a distance of any size lies in one of them); of its weight, 1/64
// of an octave each, for masses.  The last one takes what lies beyond.
constexpr int kFirstBin = (127 - 12) << 6, kBinShift = 17;
__device__ __forceinline__ int distance_bin(float l, float top) {
  const int k = static_cast<int>(__float_as_uint(top - l) >> kBinShift) - kFirstBin;
  return min(max(k, 0), kBins - 1);
}
// The least logit that may be in bin `last` or one before (or a little less).
__device__ __forceinline__ float distance_cut(int last, float top) {
  if (last == kBins - 1) return -FLT_MAX;
  const float d = __uint_as_float(static_cast<uint32_t>(last + 1 + kFirstBin) << kBinShift);
  return fmaxf(nextafterf(top - d, -INFINITY), -FLT_MAX);
}
// The logit of `step` 64ths of an octave, rounded towards `to`.
__device__ __forceinline__ float step_value(float step, float to, const Scale& s) {
  const float d = __fdiv_rn((kMagic - s.magic) - step * (1.f / 64), s.c_hi);
  return nextafterf(__fadd_rn(s.base, nextafterf(d, to)), to);
}
// A bin's mass is kept as what its tokens weigh beside the bin's middle, in units of
// 2^-bits of that: the weight there is 1 within 0.55%, and rounded to a unit, so sums are
// right to half a unit a token.  A row's tokens in one bin must stay below 2^32.
__device__ __forceinline__ int unit_bits(int V) { return min(13, __clz(V - 1) - 1); }
// For logits that weigh 2^(1 - kBins/64) at least.
struct Beside {
  float c, shift, a, b, one;
};
constexpr float kRound = 0x1.8p23f;  // + x: its last bits are x's nearest integer
__device__ __forceinline__ Beside beside(const Scale& s, float unit) {
  constexpr float kStep = 0.010830424696f;  // ln 2 / 64
  return {-64.f * s.c_hi, 64.f * (kMagic - s.magic), 0.5f * kStep * kStep * unit, -kStep * unit,
          unit + kRound};
}
__device__ __forceinline__ uint32_t beside_middle(float l, const Scale& s, const Beside& m, int& bin) {
  // -64 log2 of the weight
  const float x = __fmaf_rn(__fsub_rn(l, s.base), m.c, m.shift);
  const float k = __fadd_rn(x, kRound);
  bin = __float_as_int(k) - __float_as_int(kRound);
  const float y = __fsub_rn(x, __fsub_rn(k, kRound));
  const float n = __fmaf_rn(y, __fmaf_rn(y, m.a, m.b), m.one);
  return static_cast<uint32_t>(__float_as_int(n) - __float_as_int(kRound));
}
// What n in bin i amounts to; bits: of the unit, or -1 where tokens are counted.
__device__ __forceinline__ uint64_t bin_amount(int i, uint32_t n, int bits) {
  if (bits < 0 || n == 0) return n;
  return static_cast<uint64_t>(static_cast<float>(n) *
                               exp2f(static_cast<float>(42 - bits) - i * (1.f / 64)));
}

// The sums of this CTA's bins by groups, to every CTA (before a barrier).
__device__ __forceinline__ void share_groups(const Cluster cl, int bits) {
  const int lane = threadIdx.x & 31;
  __syncthreads();
#pragma unroll 1
  for (int g = threadIdx.x >> 5; g < kGroups; g += kWarps) {
    const int i = g * kGroupBins + 2 * lane;
    const uint2 n = *reinterpret_cast<const uint2*>(&cl.sh.bins[i]);
    const uint64_t m = warp_sum_u64(bin_amount(i, n.x, bits) + bin_amount(i + 1, n.y, bits));
    if (lane < cl.ctas) st_cluster_u64(mapa_shared(smem_u32(&cl.sh.group[cl.rank][g]), lane), m);
  }
}
// The bins at which the row's sum reaches the first `n` warps' `to` (after that barrier;
// the last one if none).  Bins keep until the next barrier.
__device__ __forceinline__ int2 find_bins(const Cluster cl, int bits, int n_warps, uint64_t to) {
  static_assert(kGroups == 32 && kGroupBins == 64);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp < n_warps) {
    uint64_t m = 0;
    for (int r = 0; r < cl.ctas; ++r) m += cl.sh.group[r][lane];
    uint64_t upto = warp_scan(m);
    uint32_t past = __ballot_sync(0xffffffffu, upto >= to);
    int found = kBins - 1;
    if (past) {
      const int g = __ffs(past) - 1;
      const uint64_t before = __shfl_sync(0xffffffffu, upto - m, g);
      // two neighbouring bins a lane, every CTA's at once
      const int i = g * kGroupBins + 2 * lane;
      const uint32_t here = smem_u32(&cl.sh.bins[i]);
      uint64_t n[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)  // (its own again, instead of those there are not)
        n[r] = ld_cluster_u64(mapa_shared(here, r < cl.ctas ? r : cl.rank));
      uint64_t m0 = 0, m1 = 0;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        if (r >= cl.ctas) break;
        m0 += bin_amount(i, static_cast<uint32_t>(n[r]), bits);
        m1 += bin_amount(i + 1, static_cast<uint32_t>(n[r] >> 32), bits);
      }
      upto = before + warp_scan(m0 + m1);
      past = __ballot_sync(0xffffffffu, upto >= to);
      const int who = past ? __ffs(past) - 1 : 31;
      found = g * kGroupBins + 2 * who +
              (__shfl_sync(0xffffffffu, static_cast<int>(upto - m1 >= to), who) ? 0 : 1);
    }
    if (lane == 0) cl.sh.found[warp] = found;
  }
  __syncthreads();
  return make_int2(cl.sh.found[0], cl.sh.found[1]);
}

// ------------------------------------------------- passes over a lane's part
// The largest logits of every fourth of its units (NaN is passed over).
template <class T>
__device__ __forceinline__ float4 largest(const Part<T> part) {
  float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  part.template stream<kWide>([&](int i, int, const float (&v)[Part<T>::kPer]) {
#pragma unroll
    for (int j = 0; j < Part<T>::kPer; ++j) top[i % 4] = fmaxf(top[i % 4], v[j]);
  });
  return make_float4(top[0], top[1], top[2], top[3]);
}
// Its largest logit and its mass, in one pass: weights are relative to 2^shift, which
// goes up with the warp's largest logit so far, and the mass with it.  For |c l| up to
// kLargestShift where anything weighs.
struct Mass {
  float top;
  uint64_t mass;
};
__device__ __forceinline__ uint64_t shifted(uint64_t mass, float by) {  // rounded
  if (!(by > 0.f)) return mass;
  if (by > 63.f) return 0;
  const int n = static_cast<int>(by);
  return (mass >> n) + (mass >> (n - 1) & 1);
}
template <class T>
__device__ __forceinline__ Mass largest_and_mass(const Part<T> part, float2 c,
                                                 const float2* table) {
  constexpr int kPer = Part<T>::kPer;
  Mass all = {-INFINITY, 0};
  Scale s = {0.f, 0.f, c.x, c.y, 0.f};
  Adder sum;
  float shift = -2.f * kLargestShift, next;  // next: the logit that weighs 1
  const auto raise = [&] {
    sum.flush();
    const float to = fmaxf(shift, fminf(ceilf(warp_max(all.top) * c.x), 2.f * kLargestShift));
    sum.mass = shifted(sum.mass, to - shift);
    shift = to;
    s.magic = kMagic - to;
    s.least = __fdividef(to - 60.f, c.x);
    next = __fdividef(to, c.x);
  };
  raise();
  part.template stream<kFew>([&](int, int, const float (&v)[kPer]) {
    float m = v[0];
#pragma unroll
    for (int j = 1; j < kPer; ++j) m = fmaxf(m, v[j]);
    all.top = fmaxf(all.top, m);
    if (__any_sync(0xffffffffu, m > next)) raise();
    sum.template add<false>(v, s, table);
  });
  raise();  // (`next` is rounded)
  all.mass = sum.mass;
  return all;
}
// How many are at or above x.
template <class T>
__device__ __forceinline__ uint32_t count_from(const Part<T> part, float x) {
  uint32_t n = 0;
  part.template stream<kWide>([&](int, int, const float (&v)[Part<T>::kPer]) {
#pragma unroll
    for (int j = 0; j < Part<T>::kPer; ++j) n += v[j] >= x;
  });
  return n;
}
// Their mass.
template <class T>
__device__ __forceinline__ uint64_t weigh_all(const Part<T> part, const Scale s, const float2* table) {
  Adder sum;
  part.template stream<kFew>(
      [&](int, int, const float (&v)[Part<T>::kPer]) { sum.add(v, s, table); });
  sum.flush();
  return sum.mass;
}
// The mass of those at or above x.
template <class T>
__device__ __forceinline__ uint64_t weigh_from(const Part<T> part, const Scale s, const float2* table,
                                            float x) {
  Adder sum;
  part.template stream<kFew>([&](int, int, const float (&v)[Part<T>::kPer]) {
    float w[Part<T>::kPer];
    bool some = false;
#pragma unroll
    for (int j = 0; j < Part<T>::kPer; ++j) {
      some = some || v[j] >= x;
      w[j] = v[j] >= x ? v[j] : -INFINITY;
    }
    if (__any_sync(0xffffffffu, some)) sum.add(w, s, table);
  });
  sum.flush();
  return sum.mass;
}
// Counts all in the CTA's bins.
template <class T>
__device__ __forceinline__ void count_bins(const Part<T> part, float top, uint32_t* bins) {
  part.template stream<kFew>([&](int, int, const float (&v)[Part<T>::kPer]) {
#pragma unroll
    for (int j = 0; j < Part<T>::kPer; ++j)
      if (v[j] > -INFINITY) atomicAdd(&bins[distance_bin(v[j], top)], 1);
  });
}
// Adds those at or above x to the CTA's bins of masses.
template <class T>
__device__ __forceinline__ void fill_bins(const Part<T> part, const Scale s, float x, float unit,
                                          uint32_t* bins) {
  const Beside m = beside(s, unit);
  part.template stream<kFew>([&](int, int, const float (&v)[Part<T>::kPer]) {
#pragma unroll
    for (int j = 0; j < Part<T>::kPer; ++j) {
      int bin;
      const uint32_t n = beside_middle(v[j], s, m, bin);
      if (v[j] >= x) atomicAdd(&bins[bin], n);
    }
  });
}
// Puts a unit's tokens from lo to hi on the CTA's list; one that is full counts on.  All
// lanes of a warp call it.
template <int PER>
__device__ __forceinline__ void list_unit(Shared& sh, int c, const float (&v)[PER], float lo,
                                          float hi) {
  uint32_t which = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) which |= v[j] >= lo && v[j] <= hi ? 1u << j : 0u;
  if (!__any_sync(0xffffffffu, which != 0)) return;
  const int lane = threadIdx.x & 31;
  const uint32_t n = __popc(which), upto = warp_scan(n);
  uint32_t at = 0;
  if (lane == 31) at = atomicAdd(&sh.listed, upto);
  at = __shfl_sync(0xffffffffu, at, 31) + upto - n;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    if (!(which >> j & 1)) continue;
    if (at < kList) sh.list[at] = list_entry(v[j], c + j);
    ++at;
  }
}
// Lists those at or above x.  `lanes`: which of the warp's lanes have one.
template <class T>
__device__ __forceinline__ void list_from(const Part<T> part, Shared& sh, float x, uint32_t lanes) {
  part.template stream_of<kWide>(lanes, [&](int c, const float (&v)[Part<T>::kPer]) {
    list_unit(sh, c, v, x, INFINITY);
  });
}
// Lists those from lo to hi; the mass of those above hi.  `lanes`: those that have some.
template <class T>
__device__ __forceinline__ uint64_t list_and_weigh(const Part<T> part, const Scale s, Shared& sh,
                                                float lo, float hi, uint32_t lanes) {
  Adder sum;
  part.template stream_of<kFew>(lanes, [&](int c, const float (&v)[Part<T>::kPer]) {
    float most = v[0];
#pragma unroll
    for (int j = 1; j < Part<T>::kPer; ++j) most = fmaxf(most, v[j]);
    if (!__any_sync(0xffffffffu, most >= lo)) return;
    list_unit(sh, c, v, lo, hi);
    if (!__any_sync(0xffffffffu, most > hi)) return;
    float w[Part<T>::kPer];
    int over = 0;
#pragma unroll
    for (int j = 0; j < Part<T>::kPer; ++j) {
      over += v[j] > hi;
      w[j] = v[j] > hi ? v[j] : -INFINITY;
    }
    if (__any_sync(0xffffffffu, over > 1)) {
      sum.add(w, s, sh.table);
    } else {  // one a lane at most
      const float one[1] = {over ? most : -INFINITY};
      sum.add(one, s, sh.table);
    }
  });
  sum.flush();
  return sum.mass;
}
// Shares the length of this CTA's list and a warp's mass.
__device__ __forceinline__ Sum share_list(Cluster& cl, uint64_t mass) {
  __syncthreads();
  cl.share(mass, threadIdx.x < 32 ? cl.sh.listed : 0);
  return cl.sum();
}
// Every CTA's list into `work`.
__device__ __forceinline__ void pull_lists(const Cluster cl) {
  Shared& sh = cl.sh;
  uint32_t most = 0;
  for (int r = 0; r < cl.ctas; ++r) most = max(most, sh.count[cl.phase][r * kWarps]);
#pragma unroll 1
  for (uint32_t i = threadIdx.x; i < most; i += kThreads) {
    const uint32_t here = smem_u32(&sh.list[i]);
    uint64_t e[kMaxCluster];
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)  // (entries past a list's end are not used)
      e[r] = ld_cluster_u64(mapa_shared(here, r < cl.ctas ? r : cl.rank));
    uint32_t at = 0;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      if (r >= cl.ctas) break;
      const uint32_t c = sh.count[cl.phase][r * kWarps];
      if (i < c) sh.work[at + i] = e[r];
      at += c;
    }
  }
}

// ------------------------------------------------------------ the kernel
template <class T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
  constexpr int kPer = Part<T>::kPer;
  __shared__ Shared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Cluster cl{sh, 0, 1, 0};
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(cl.rank));
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cl.ctas));
  // every CTA of the cluster runs before another writes to its shared memory
  cluster_arrive();
  griddep_launch_dependents();
  griddep_wait();
  const int64_t b = blockIdx.x / cl.ctas;
  const int warps = cl.ctas * kWarps, me = cl.rank * kWarps + warp;
  Part<T> part(a, b);
  const int s0 = part.first_slot(me, warps);
  part.each = part.first_slot(me + 1, warps) - s0;
  part.u0 = s0 * 32 + lane;
  part.inner = part.whole(s0 * 32) && part.whole((s0 + part.each) * 32 - 1);

  const float T_given = a.temperature ? a.temperature[b] : 1.f;
  const float T0 = T_given > kHottest ? kHottest : T_given;  // (NaN stays)
  const int k = a.top_k ? a.top_k[b] : 0;
  const float p = a.top_p ? a.top_p[b] : 1.f;
  const float min_p = a.min_p ? a.min_p[b] : 0.f;
  const float u = a.u[b];
  const bool greedy = !(T0 >= kGreedyBelow);
  for (int i = threadIdx.x; i < kBins; i += kThreads) sh.bins[i] = 0;
  if (warp == 0) {
    const float2 entry = kPow2[lane];
    sh.table[lane] = make_float2(
        __uint_as_float(__float_as_uint(entry.x) - (static_cast<uint32_t>(lane) << 18)), entry.y);
    if (lane == 0) {
      sh.listed = 0;
      sh.inverse = inverse_of(greedy ? 1.f : T0);
    }
    __syncwarp();
    if (min_p > 0.f) {
      // T ln(min_p) in two floats.  With min_p = f 2^e, e <= 0 and f from 1/2 to 1: FP32's
      // logarithm of f, corrected by what its exponential leaves of f (a weight has all its
      // bits there: of a min_p near 2^-29 it has 13), and e ln 2, whose first part is exact.
      constexpr float kLn2 = 0x1.62e4p-1f, kLn2Rest = 0x1.7f7d1cp-20f;
      const float m = fminf(min_p, 1.f);
      int e;
      frexpf(m, &e);
      e = min(e, 0);  // (1 stays 1)
      const float f = ldexpf(m, -e), y = logf(f), n = static_cast<float>(e);
      const uint64_t w = weight(y, make_scale(0.f, inverse_of(1.f)), sh.table);
      const float left = static_cast<float>(static_cast<int64_t>(__float2ull_rn(f * 0x1p42f) - w)) /
                         static_cast<float>(w);
      const float2 sum = two_sum(__fmul_rn(n, kLn2), y);
      const float rest = __fadd_rn(__fadd_rn(sum.y, left), __fmul_rn(n, kLn2Rest));
      const float hi = __fmul_rn(T0, sum.x);
      if (lane == 0)
        sh.log_min_p = make_float2(
            hi, __fadd_rn(__fmaf_rn(T0, sum.x, -hi), __fmul_rn(T0, rest)));
    }
  }

  // The largest logit, and, where all tokens' mass will be asked for, that too.
  const bool by_k = !greedy && k > 0 && k < a.V, by_p = !greedy && p < 1.f;
  bool weighed = !greedy && !by_k && (by_p || !(min_p > 0.f)) && T0 < 0x1p64f;
  float4 tops;
  float lane_top, top;
  uint64_t mass = 0;
  if (weighed) {
    __syncthreads();  // (the table)
    const Mass m = largest_and_mass(part, sh.inverse, sh.table);
    lane_top = m.top;
    tops = make_float4(m.top, m.top, m.top, m.top);  // (not used)
    top = warp_max(lane_top);
    mass = warp_sum_u64(m.mass);
  } else {
    tops = largest(part);
    lane_top = fmaxf(fmaxf(tops.x, tops.y), fmaxf(tops.z, tops.w));
    top = warp_max(lane_top);
  }
  cluster_wait();
  cl.share(mass, __float_as_uint(top));
  for (int i = lane; i < warps; i += 32) top = fmaxf(top, __uint_as_float(sh.count[cl.phase][i]));
  top = warp_max(top);
  if (top == -INFINITY) {  // nothing to pick from
    if (me == 0 && lane == 0) a.out[b] = -1;
    return;
  }
  const Scale scale = make_scale(top, sh.inverse);
  weighed = weighed && scale.base == 0.f;
  if (weighed) {  // every warp's mass relative to the row's largest logit, as share_kept leaves it
    __syncthreads();
    if (threadIdx.x < warps) {
      const float warp_top = __uint_as_float(sh.count[cl.phase][threadIdx.x]);
      uint64_t& m = sh.mass[cl.phase][threadIdx.x];
      m = warp_top > -INFINITY
              ? shifted(m, (kMagic - scale.magic) - ceilf(warp_top * scale.c_hi))
              : 0;
      sh.count[cl.phase][threadIdx.x] = 0;
    }
    __syncthreads();
  }
  // what min_p keeps: w >= min_p w_max, l >= max + T ln(min_p), rounded up
  float least = -FLT_MAX;
  if (!greedy && min_p > 0.f && top < INFINITY) {
    // (max and the logarithm may cancel: what the sum leaves is added before it is rounded)
    const float2 d = sh.log_min_p, first = two_sum(top, d.x);
    const float2 sum = two_sum(first.x, __fadd_rn(first.y, d.y));
    least = sum.y > 0.f ? nextafterf(sum.x, INFINITY) : sum.x;
    if (!(least > -FLT_MAX)) least = -FLT_MAX;
  }
  const uint64_t part_p = __float2ull_rz(fmaxf(fminf(p, 0x1.fffffep-1f), 0.f) * 0x1p64f);
  // the mass before a token that is kept is less than this
  const auto target_p = [&](uint64_t all) {  // p * all, rounded up; the first token always
    return max(static_cast<uint64_t>(__umul64hi(part_p, all)) + (part_p * all != 0), uint64_t{1});
  };
  const uint64_t part_u = __float2ull_rz(fminf(fmaxf(u, 0.f), 0x1.fffffep-1f) * 0x1p64f);

  // --- top-k: a list of everything that can be among the first k, which the cluster's
  // first CTA then has to itself.  k of the largest logits of quarters of lanes are in the
  // bins up to the one that holds the k-th, so are k tokens; other quarters have none there.
  // Where quarters are not many more than k, all tokens are counted instead.
  if (by_k && k <= kList / 2 && top < INFINITY) {
    if (2 * k > min(4 * warps, part.slots) * 32) {
      count_bins(part, top, sh.bins);
    } else {
      const float quarter[4] = {tops.x, tops.y, tops.z, tops.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (quarter[i] > -INFINITY) atomicAdd(&sh.bins[distance_bin(quarter[i], top)], 1);
    }
    share_groups(cl, -1);
    cluster_arrive();
    cluster_wait();
    const float cut = distance_cut(find_bins(cl, -1, 1, k).x, top);
    const uint32_t lanes = __ballot_sync(0xffffffffu, lane_top >= cut);
    if (lanes) list_from(part, sh, cut, lanes);
    const uint32_t N = share_list(cl, 0).count;
    if (N < kList) {
      if (cl.rank == 0) pull_lists(cl);
      cluster_arrive();  // the lists have been read
      if (cl.rank != 0) {
        cluster_wait();
        return;
      }
      __syncthreads();
      const int n = static_cast<int>(N);
      for (int i = threadIdx.x; i < n; i += kThreads)
        sh.list[i] = weight(listed_logit(sh.work[i]), scale, sh.table);
      __syncthreads();
      // Up to 128 tokens go through all limits by comparisons.  One row, top-k 100 and top-p:
      // 12.8 us, by searches 15.8; 64 rows 18.0 and 21.2, but top-k 200 alone 23.9 and 19.5.
      if (n <= 2 * kCompared) {
        const int each = n <= kCompared ? kThreads / kCompared : kThreads / (2 * kCompared);
        const int q = threadIdx.x / each, r = threadIdx.x % each;
        const uint64_t e = q < n ? sh.work[q] : 0, w = q < n && r == 0 ? sh.list[q] : 0;
        uint32_t rank = 0;
        uint64_t before = 0;
        for (int i = r; i < n; i += each)
          if (sh.work[i] > e) {
            ++rank;
            before += sh.list[i];
          }
        for (int o = each / 2; o > 0; o >>= 1) {
          rank += __shfl_xor_sync(0xffffffffu, rank, o);
          before += __shfl_xor_sync(0xffffffffu, before, o);
        }
        bool keep = q < n && rank < static_cast<uint32_t>(k);
        if (by_p) {
          const uint64_t all = block_sum(sh, keep ? w : 0);
          keep = keep && before < target_p(all);
        }
        keep = keep && (rank == 0 || listed_logit(e) >= least);
        if (r == 0) sh.weights[q] = keep ? w : 0;
        const uint64_t pick = __umul64hi(part_u, block_sum(sh, keep ? w : 0));
        uint64_t upto = 0;  // by id
        for (int i = r; i < n; i += each)
          if (static_cast<uint32_t>(sh.work[i]) >= static_cast<uint32_t>(e)) upto += sh.weights[i];
        for (int o = each / 2; o > 0; o >>= 1) upto += __shfl_xor_sync(0xffffffffu, upto, o);
        if (keep && r == 0 && upto > pick && upto - w <= pick) a.out[b] = listed_id(e);
      } else {
        const auto entry = [&](int i) { return sh.work[i]; };
        const auto mass = [&](int i) { return sh.list[i]; };
        const auto mass_kept = [&](uint64_t from) {
          uint64_t m = 0;
          for (int i = threadIdx.x; i < n; i += kThreads) m += sh.work[i] >= from ? sh.list[i] : 0;
          return block_sum(sh, m);
        };
        // the last entry that is kept
        const uint64_t last = list_entry(top, 0);
        uint64_t from = list_entry(cut, 0) >> 32 << 32;
        if (n > k)
          from = select_key(sh, n, entry, [](int) { return uint64_t{1}; }, from, last,
                            static_cast<uint64_t>(k)).key;
        if (by_p)
          from = select_key(sh, n, entry, mass, from, last, target_p(mass_kept(from))).key;
        from = max(from, list_entry(fminf(least, top), 0) >> 32 << 32);
        // of those, by id
        const uint64_t pick = __umul64hi(part_u, mass_kept(from));
        const Border inverse = select_key(
            sh, n,
            [&](int i) {
              const uint64_t e = sh.work[i];
              return e >= from ? e & 0xffffffffu : uint64_t{0};
            },
            mass, 0xffffffffu - (a.V - 1), 0xffffffffu, pick + 1);
        if (threadIdx.x == 0) a.out[b] = listed_id(inverse.key);
      }
      cluster_wait();
      return;
    }
  }

  // --- otherwise what is kept as t and ties, which the limits narrow one after another.
  float t = greedy || top == INFINITY ? top : -FLT_MAX;
  uint32_t ties = greedy ? 1 : top == INFINITY ? UINT_MAX - 1 : UINT_MAX;
  // Of the lane's tokens, as far as its warp has any (x > -infinity).
  const auto mass_from = [&](float x) {
    if (!__any_sync(0xffffffffu, lane_top >= x)) return uint64_t{0};
    return x == -FLT_MAX ? weigh_all(part, scale, sh.table)
                         : weigh_from(part, scale, sh.table, x);
  };
  const auto number_from = [&](float x) {
    return __any_sync(0xffffffffu, lane_top >= x) ? count_from(part, x) : 0u;
  };
  // Narrows t and ties to the prefix that makes `target` (tokens, or mass): halves the
  // range of logits from t to `most`, above which there is `above`, a pass over the row and
  // a barrier each; `most` (equal logits) and `likely` are tried first.  For any row; the
  // lists are faster where they are long enough.
  const auto halve = [&](uint64_t target, bool mass, float likely, float most, uint64_t above) {
    int lo = key_of<T>(t), hi = key_of<T>(most);
    int first = hi, second = key_of<T>(likely);
#pragma unroll 1
    while (lo < hi) {
      const int mid = first > lo && first <= hi
                          ? first
                          : static_cast<int>(lo + (static_cast<int64_t>(hi) - lo + 1) / 2);
      first = second;
      second = INT_MIN;
      const float x = value_of<T>(mid);
      cl.share(mass ? warp_sum_u64(mass_from(x)) : 0,
               mass ? 0 : __reduce_add_sync(0xffffffffu, number_from(x)));
      const Sum s = cl.sum();
      const uint64_t have = mass ? s.mass : s.count;
      if (have >= target) {
        lo = mid;
      } else {
        hi = mid - 1;
        above = have;
      }
    }
    const float x = value_of<T>(lo);
    uint64_t r = target - above;
    if (mass) {
      const uint64_t w = max(weight(x, scale, sh.table), uint64_t{1});
      r = (r + w - 1) / w;
    }
    r = min(r, static_cast<uint64_t>(UINT_MAX));
    if (x > t || r < ties) {
      t = x;
      ties = static_cast<uint32_t>(r);
    }
  };
  // The mass above t, or with all ties from it on, and the number of those; to every CTA.
  const auto share_kept = [&]() {
    const float next = ties == UINT_MAX ? t : nextafterf(t, INFINITY);
    const uint32_t n = ties == UINT_MAX ? 0
                       : t == INFINITY  ? number_from(t)
                                        : number_from(t) - number_from(next);
    const uint64_t m = ties != UINT_MAX && t == INFINITY ? 0 : mass_from(next);
    cl.share(warp_sum_u64(m), __reduce_add_sync(0xffffffffu, n));
  };

  bool shared = weighed;  // every CTA has what t and ties keep, by warps
  if (top == INFINITY && !greedy) {  // each +infinity weighs 1, all else nothing
    share_kept();
    shared = true;
    ties = cl.sum().count;
    if (by_k) ties = min(ties, static_cast<uint32_t>(k));
    if (by_p)
      ties = static_cast<uint32_t>((target_p(uint64_t{ties} << 42) + (uint64_t{1} << 42) - 1) >> 42);
  } else if (by_k) {
    halve(static_cast<uint64_t>(k), false, t, top, 0);
  }
  // --- top-p over many tokens: their mass, and a histogram by weight that says near which
  // one the border lies; a list of those bins' tokens then gives it.
  if (by_p && top < INFINITY) {
    if (by_k) {  // (the bins have been used)
      for (int i = threadIdx.x; i < kBins; i += kThreads) sh.bins[i] = 0;
      if (threadIdx.x == 0) sh.listed = 0;
      __syncthreads();
    }
    const int bits = unit_bits(a.V), unit = 1 << bits;
    if (!weighed) share_kept();
    const Sum s = cl.sum();
    const uint64_t all = s.mass + weight(t, scale, sh.table) * min(s.count, ties);
    const uint64_t target = target_p(all);
    // Tokens of less than 1 / V of the mass that p leaves out amount to less than that, so
    // the border is above them.  (In FP32, and where weights are many units.)
    const float small = static_cast<float>(all - target) / static_cast<float>(a.V) * 0.99f;
    const float steps = small >= 64.f ? (42.f - log2f(small)) * 64.f : 0x1p30f;
    // (a token from there on is in a bin: its step is right to 0.02)
    const float from =
        fmaxf(t, fminf(step_value(fminf(steps, kBins - 2.f), INFINITY, scale), top));
    if (__any_sync(0xffffffffu, lane_top >= from)) fill_bins(part, scale, from, unit, sh.bins);
    share_groups(cl, bits);
    cluster_arrive();
    cluster_wait();
    // the bins' sums are off by half a unit of them, and FP32's rounding
    const uint64_t slack = target / (2 * unit - unit / 16) + kBins;
    const int2 bins =
        find_bins(cl, bits, 2, warp == 0 ? target - min(slack, target - 1) : target + slack);
    shared = false;
    float likely = t, most = top;
    uint64_t above = 0;
    if (bins.y < kBins - 1) {
      // logits a little beyond the ends of these bins (|c l| up to kLargestShift, in FP32)
      const float lo = fmaxf(step_value(bins.y + 0.55f, -INFINITY, scale), t);
      const float hi = bins.x == 0 ? INFINITY : step_value(bins.x - 0.55f, INFINITY, scale);
      const uint32_t lanes = __ballot_sync(0xffffffffu, lane_top >= lo);
      const uint64_t mass = lanes ? list_and_weigh(part, scale, sh, lo, hi, lanes) : 0;
      const Sum in = share_list(cl, warp_sum_u64(mass));
      if (in.mass < target) {  // (as it should be)
        likely = lo;
        most = fminf(hi, top);
        above = in.mass;
      }
      if (in.count < kList) {
        pull_lists(cl);
        cluster_arrive();
        cluster_wait();
        const int n = static_cast<int>(in.count);
        for (int i = threadIdx.x; i < n; i += kThreads)  // (all have read the list)
          sh.list[i] = weight(listed_logit(sh.work[i]), scale, sh.table);
        if (threadIdx.x < warps) sh.count[cl.phase][threadIdx.x] = 0;
        __syncthreads();
        uint64_t m = 0;
        for (int i = threadIdx.x; i < n; i += kThreads) m += sh.list[i];
        m = block_sum(sh, m);
        shared = in.mass < target && in.mass + m >= target;
        if (shared) {
          constexpr int kShift = 32 + (sizeof(T) == 2 ? 16 : 0);
          const Border border = select_key(
              sh, n, [&](int i) { return sh.work[i] >> kShift; }, [&](int i) { return sh.list[i]; },
              list_entry(lo, 0) >> kShift, list_entry(fminf(hi, top), 0) >> kShift,
              target - in.mass);
          // every warp's mass above the border's logit and tokens equal to it, as
          // share_kept would leave them
          uint64_t at = border.key << kShift;
          if (sizeof(T) == 2 && !(at >> 63)) at |= uint64_t{0xffff} << 32;  // (a negative bf16)
          t = listed_logit(at);
          const uint64_t each = max(weight(t, scale, sh.table), uint64_t{1});
          ties = static_cast<uint32_t>((target - in.mass - border.above + each - 1) / each);
          for (int i = threadIdx.x; i < n; i += kThreads) {
            const float l = listed_logit(sh.work[i]);
            if (!(l >= t)) continue;
            const int w = part.warp_of(listed_id(sh.work[i]), warps);
            if (l > t)
              atomicAdd(reinterpret_cast<unsigned long long*>(&sh.mass[cl.phase][w]),
                        static_cast<unsigned long long>(weight(l, scale, sh.table)));
            else atomicAdd(&sh.count[cl.phase][w], 1);
          }
          __syncthreads();
        }
      }
    }
    if (!shared) halve(target, true, likely, most, above);
  }
  if (least > t) {
    t = least;
    ties = UINT_MAX;
    shared = false;
  }
  if (!shared) share_kept();

  // --- the pick: which warp has it, which of its slots, which token of that.
  const uint64_t wt = weight(t, scale, sh.table);
  if (warp == 0) {
    // four consecutive entries a lane
    constexpr int kEach = kMaxWarps / 32;
    uint64_t m[kEach], upto = 0;
    uint32_t e_at[kEach], ahead = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int w = lane * kEach + i;
      m[i] = w < warps ? sh.mass[cl.phase][w] : 0;
      e_at[i] = w < warps ? sh.count[cl.phase][w] : 0;
      ahead += e_at[i];
    }
    ahead = warp_scan(ahead) - ahead;  // ties of the lanes before
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const uint32_t e = e_at[i];
      e_at[i] = ahead;
      m[i] += wt * min(e, ties > ahead ? ties - ahead : 0u);
      upto += m[i];
      ahead += e;
    }
    const uint64_t lane_sum = upto;
    upto = warp_scan(upto);
    const uint64_t pick = __umul64hi(part_u, __shfl_sync(0xffffffffu, upto, 31));
    const int owner = __ffs(__ballot_sync(0xffffffffu, upto > pick)) - 1;
    uint64_t before = upto - lane_sum;
    int which = 0;
    uint32_t rank = e_at[0];
#pragma unroll
    for (int i = 0; i + 1 < kEach; ++i) {
      if (which == i && before + m[i] <= pick) {
        before += m[i];
        which = i + 1;
        rank = e_at[i + 1];
      }
    }
    if (lane == owner) {
      sh.before = pick - before;  // what is left to pick from there on
      sh.rank = rank;
      sh.found[0] = owner * kEach + which - cl.rank * kWarps;
    }
  }
  __syncthreads();
  const int w = sh.found[0];
  if (w < 0 || w >= kWarps) return;  // another CTA's
  // The warp's slots, a warp of this CTA each: their masses above t, and ties.
  const int first = part.first_slot(cl.rank * kWarps + w, warps);
  const int count = part.first_slot(cl.rank * kWarps + w + 1, warps) - first;
#pragma unroll 1
  for (int s = warp; s < count; s += kWarps) {
    float v[kPer];
    Part<T>::floats(part.load((first + s) * 32 + lane), v);
    uint32_t e = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const bool tie = ties != UINT_MAX && v[j] == t;
      e += tie;
      if (!(v[j] >= t) || tie) v[j] = -INFINITY;
    }
    Adder sum;
    if (t < INFINITY) {  // (where it is not, ties are all that weighs)
      sum.add(v, scale, sh.table);
      sum.flush();
    }
    sum.mass = warp_sum_u64(sum.mass);
    e = __reduce_add_sync(0xffffffffu, e);
    if (lane == 0) {
      sh.slot.mass[s] = sum.mass;
      sh.slot.ties[s] = e;
    }
  }
  __syncthreads();
  if (warp != 0) return;
  uint64_t pick = sh.before;
  uint32_t rank = sh.rank;
  if (weighed && !by_p && t == -FLT_MAX) {
    // The pass that weighed all rounded each lane's mass: should these sum to a unit less,
    // the last token is taken, and if all of them weigh nothing, the first one.
    uint64_t all = 0;
    for (int s = lane; s < count; s += 32) all += sh.slot.mass[s];
    all = warp_sum_u64(all);
    if (all > 0) {
      pick = min(pick, all - 1);
    } else {
#pragma unroll 1
      for (int s = 0; s < count; ++s) {
        const int unit = (first + s) * 32 + lane;
        float v[kPer];
        Part<T>::floats(part.load(unit), v);
        int found = -1;
#pragma unroll
        for (int j = kPer - 1; j >= 0; --j)
          if (v[j] >= t) found = j;
        const uint32_t some = __ballot_sync(0xffffffffu, found >= 0);
        if (!some) continue;
        if (lane == __ffs(some) - 1) a.out[b] = part.first(unit) + found;
        return;
      }
    }
  }
#pragma unroll 1
  for (int s = 0; s < count; s += 32) {
    const uint32_t e = s + lane < count ? sh.slot.ties[s + lane] : 0;
    const uint32_t ahead = rank + warp_scan(e) - e;
    const uint64_t m = (s + lane < count ? sh.slot.mass[s + lane] : 0) +
                       wt * min(e, ties > ahead ? ties - ahead : 0u);
    const uint64_t upto = warp_scan(m);
    const uint32_t past = __ballot_sync(0xffffffffu, upto > pick);
    if (!past) {
      pick -= __shfl_sync(0xffffffffu, upto, 31);
      rank = __shfl_sync(0xffffffffu, ahead + e, 31);
      continue;
    }
    const int who = __ffs(past) - 1;
    pick -= __shfl_sync(0xffffffffu, upto - m, who);
    rank = __shfl_sync(0xffffffffu, ahead, who);
    // the slot's tokens, a unit a lane
    const int unit = (first + s + who) * 32 + lane;
    float v[kPer];
    Part<T>::floats(part.load(unit), v);
    uint32_t equal = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) equal += ties != UINT_MAX && v[j] == t;
    rank += warp_scan(equal) - equal;
    uint64_t x[kPer], sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const bool tie = ties != UINT_MAX && v[j] == t;
      x[j] = tie ? (rank < ties ? wt : 0) : v[j] >= t ? weight(v[j], scale, sh.table) : 0;
      rank += tie;
      sum += x[j];
    }
    uint64_t at = warp_scan(sum);
    const int last = __ffs(__ballot_sync(0xffffffffu, at > pick)) - 1;
    at -= sum;
    if (lane == last) {
      int found = -1;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        at += x[j];
        if (found < 0 && at > pick) found = j;
      }
      a.out[b] = part.first(unit) + found;
    }
    return;
  }
}

// ------------------------------------------------------------- launching
// CTAs a row: as many as seven eighths of the places (two an SM) have for it, as clusters
// do not fill all of them, and fewer where a warp would have less than three slots of its
// row.  Where that is one, two take a long row all the same: with top-k or top-p, whose rows
// differ in their passes and end at different times; without, as far as an SM has no more
// than three CTAs to run; with min-p alone where rows are longer.  us in a graph over inputs
// larger than L2, without limits / top-k / top-p / min-p:
//     37 x 152064 bf16       4 CTAs 19 / 24 / 48 / 12, 7 17 / 22 / 46 / 13, 8 21 / 28 / 55 / 17
//     64 x 152064 bf16       2 CTAs 29 / 31 / 89 / 17, 4 20 / 25 / 60 / 13, 5 27 / 31 / 74 / 20
//     64 x 32003 float32     1 CTA 17 / 25 / 44 / 13, 4 11 / 18 / 28 / 10, 8 18 / 32 / 48 / 18
//     256 x 32003 float32    1 CTA 19 / 32 / 54 / 16, 2 26 / 36 / 62 / 23
//     256 x 65536 bf16       1 CTA 26 / 33 / 83 / 19, 2 33 / 36 / 86 / 23
//     256 x 65536 float32    1 CTA 29 / 43 / 84 / 24, 2 35 / 43 / 88 / 27
//     256 x 80001 float32    1 CTA - / 54 / 107 / 35, 2 - / 51 / 105 / 35
//     256 x 100352 bf16      1 CTA 38 / 46 / 122 / 26, 2 45 / 45 / 118 / 29
//     256 x 128255 bf16      1 CTA 46 / 63 / 166 / 39, 2 52 / 53 / 149 / 35
//     256 x 152064 float32   1 CTA 56 / 76 / 178 / 56, 2 63 / 73 / 166 / 51
//     200 x 100352 bf16      1 CTA 36 / 42 / 120 / 26, 2 35 / 40 / 107 / 26
//     220 x 152064 bf16      1 CTA 50 / 59 / 173 / 33, 2 45 / 49 / 147 / 34
//     240 x 152064 bf16      1 CTA 51 / 60 / 175 / 43, 2 57 / 52 / 158 / 37
//     1024 x 128255 bf16     1 CTA 143 / 192 / 617 / 101, 2 169 / 155 / 499 / 112
constexpr int kLongRow = 80000, kLongerRow = 1 << 17;  // columns
template <class T>
cudaError_t run_sample(const SampleArgs& a, int64_t B, int sms, cudaStream_t s) {
  const int64_t slots = a.V / (32 * Part<T>::kPer);
  int ctas = static_cast<int>(
      std::clamp<int64_t>(std::min<int64_t>(7 * sms / (4 * B), slots / (3 * kWarps)), 1, kMaxCluster));
  if (ctas == 1 && a.V >= kLongRow &&
      (a.top_k || a.top_p || 2 * B <= 3 * sms || (a.min_p && a.V >= kLongerRow)))
    ctas = 2;
  const cudaError_t e = launch_overlapped(sample_kernel<T>, dim3(static_cast<unsigned>(B * ctas)),
                                          dim3(kThreads), 0, s, ctas, a);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" flce_status flce_sample_logits(const void* logits, int64_t ld_logits, flce_dtype dtype,
                                          int64_t B, int64_t V, const float* u,
                                          const float* temperature, const int32_t* top_k,
                                          const float* top_p, const float* min_p, int64_t* out,
                                          flce_stream_t stream) {
  OpRange range("flce_sample_logits");
  if (B < 0 || V <= 0 || !valid_dtype(dtype)) return FLCE_ERR_INVALID_ARG;
  if (B > 65535 || V > kMaxVocab) return FLCE_ERR_UNSUPPORTED_SHAPE;
  if (B == 0) return FLCE_OK;
  if (!logits || !u || !out || ld_logits < V) return FLCE_ERR_INVALID_ARG;
  const size_t e = dtype_bytes(dtype), nb = static_cast<size_t>(B) * 4;
  if (!aligned_to(logits, e) || !aligned_to(u, 4) || !aligned_to(temperature, 4) ||
      !aligned_to(top_k, 4) || !aligned_to(top_p, 4) || !aligned_to(min_p, 4) ||
      !aligned_to(out, 8))
    return FLCE_ERR_INVALID_ARG;
  const Range o = {out, static_cast<size_t>(B) * 8};
  const Range ins[] = {{logits, span_bytes(B, V, ld_logits, e)},
                       {u, nb},
                       {temperature, nb},
                       {top_k, nb},
                       {top_p, nb},
                       {min_p, nb}};
  for (const Range& r : ins)
    if (ranges_overlap(o, r)) return FLCE_ERR_INVALID_ARG;
  int sms = 0;
  const flce_status st = check_device(&sms);
  if (st != FLCE_OK) return st;
  SampleArgs a = {};
  a.logits = logits;
  a.ld = ld_logits;
  a.V = static_cast<int>(V);
  a.u = u;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.out = out;
  const auto s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t err = dtype == FLCE_BF16 ? run_sample<__nv_bfloat16>(a, B, sms, s)
                                             : run_sample<float>(a, B, sms, s);
  return err == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}
