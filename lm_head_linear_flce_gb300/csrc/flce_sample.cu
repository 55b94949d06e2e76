// A token a row by temperature, top-k, top-p and min-p from a given random number
// (flce_sample_logits).
//
// A cluster of CTAs takes a row: each holds a part of it in shared memory, so that the
// row is read once however often its tokens are gone over.  What a row keeps is a prefix
// of its tokens in descending order (equal logits by id), which a logit t and a number r
// say: all tokens above t, and the first r of those equal to t.  The token is then the
// first, by id, whose cumulative mass among the kept ones exceeds u times their total.
//
// Masses are integers.  A token weighs 2^((l - max) / (T ln 2)) in units of 2^-42, off by
// 2^-31.6 of it (rms), and sums of integers do not depend on their order: however the
// row is split, the same tokens are kept and the same one is picked, and next to a
// border the cumulative mass is right to some 1e-12 where FP32 sums would be off by
// 1e-7, on a vocabulary with a border every 1e-5.
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
constexpr float kGreedyBelow = 0x1p-64f;         // temperatures that take the largest logit

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

// What turns a row's logits into weights.  With c = 1 / (T ln 2) a weight is
// 2^(c (l - base) - shift): base is the largest logit where |c max| is large (l - base is
// then exact for every l that weighs anything), else 0 with shift = ceil(c max), so that
// l is used as it is.  c in two floats.
struct Scale {
  float base, least, c_hi, c_lo, magic;
};
constexpr float kMagic = 0x1.8p18f;   // + x rounds x to 1/32; its last bits count them
constexpr float kMagicA = 0x1.8p2f;   // the same for units of 2^-21 and of 2^-42, in
constexpr float kMagicB = 0x1.8p-19f; // which a weight is a + b
constexpr uint32_t kBitsA = 0x40c00000u, kBitsB = 0x36400000u;

__device__ __forceinline__ Scale make_scale(float top, float T) {
  constexpr float kHi = 0x1.715476p0f, kLo = 0x1.4ae0cp-26f;  // 1 / ln 2
  Scale s;
  s.c_hi = __fdiv_rn(kHi, T);
  s.c_lo = __fdividef(fmaf(-s.c_hi, T, kHi) + kLo, T);
  if (!(s.c_hi > 0.f) || top == INFINITY) s.c_hi = s.c_lo = 0.f;  // every token alike
  const float x = top * s.c_hi;
  const bool large = fabsf(x) > 64.f;  // (an infinite top too: least is 0 then)
  s.base = large || top == INFINITY ? top : 0.f;
  const float shift = s.base == 0.f ? ceilf(x) : 0.f;
  // below it a weight is less than 2^-59
  s.least = top == INFINITY ? 0.f : s.c_hi > 0.f ? fmaxf(__fdividef(shift - 60.f, s.c_hi), -FLT_MAX)
                                                 : -FLT_MAX;
  s.magic = kMagic - shift;
  return s;
}

// A token's weight as a * 2^-21 + b * 2^-42, each as the float that holds its bits above
// kBitsA and kBitsB.  With x = c (l - base) = k / 32 + f, |f| <= 1/64: 2^x by the table
// (Tang 1989) times 2^f by its series; f carries the rounding errors of x and of the
// table's entry.  Written with intrinsics so that every use rounds alike.
__device__ __forceinline__ void weigh(float l, const Scale& s, const float2* table, uint32_t& a,
                                      uint32_t& b) {
  const float d = fmaxf(__fsub_rn(l, s.base), s.least);
  const float nq = __fmul_rn(d, -s.c_hi);
  const float e = __fmaf_rn(d, s.c_lo, __fmaf_rn(d, s.c_hi, nq));
  const float z = __fsub_rn(s.magic, nq);
  const float g = __fadd_rn(nq, __fsub_rn(z, s.magic));
  const uint32_t k = __float_as_uint(z);
  const float2 t = table[k & 31];
  const float f = __fsub_rn(__fadd_rn(e, t.y), g);
  constexpr float kLn2 = 0.69314718055994531f;
  float p = __fmaf_rn(f, kLn2 * kLn2 * kLn2 * kLn2 / 24, kLn2 * kLn2 * kLn2 / 6);
  p = __fmaf_rn(f, p, kLn2 * kLn2 / 2);
  p = __fmul_rn(f, __fmaf_rn(f, p, kLn2));
  // (k's bits above the table's are the exponent; the constant's fall off the top)
  const float th = __uint_as_float(__float_as_uint(t.x) + ((k & ~31u) << 18));
  const float y = __fmul_rn(th, p);
  const float v = __fadd_rn(th, y);
  const float rest = __fsub_rn(y, __fsub_rn(v, th));
  const float fa = __fadd_rn(v, kMagicA);
  const float fb =
      __fadd_rn(__fadd_rn(__fsub_rn(v, __fsub_rn(fa, kMagicA)), rest), kMagicB);
  a = __float_as_uint(fa);
  b = __float_as_uint(fb);
}
// The sum of n weights, from the sums of their a and b modulo 2^32.
__device__ __forceinline__ uint64_t mass_of(uint32_t a, uint32_t b, uint32_t n) {
  const int64_t ia = static_cast<int32_t>(a - n * kBitsA), ib = static_cast<int32_t>(b - n * kBitsB);
  return static_cast<uint64_t>(ia * (int64_t{1} << 21) + ib);
}
__device__ __forceinline__ uint64_t weight(float l, const Scale& s, const float2* table) {
  uint32_t a, b;
  weigh(l, s, table, a, b);
  return mass_of(a, b, 1);
}

// ------------------------------------------------------------ a row's logits
// A row in units of 16 bytes, the first starting `shift` elements before it; 32 units
// are a slot, and a warp has consecutive slots.  Elements outside the row are -infinity.
template <class T>
struct Row {
  static constexpr int kPer = 16 / static_cast<int>(sizeof(T));
  const T* p;
  int V, shift, units;

  __device__ Row(const SampleArgs& a, int64_t b)
      : p(static_cast<const T*>(a.logits) + b * a.ld), V(a.V) {
    shift = static_cast<int>(reinterpret_cast<uintptr_t>(p) % 16 / sizeof(T));
    units = (V + shift + kPer - 1) / kPer;
  }
  __device__ int first(int u) const { return u * kPer - shift; }  // column of a unit's first element
  __device__ __forceinline__ uint4 load(int u) const {
    const int c = first(u);
    if (c >= 0 && c + kPer <= V) return *reinterpret_cast<const uint4*>(p + c);
    constexpr uint32_t kNone = 0xff800000u;  // -infinity
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        w[i] = c + i >= 0 && c + i < V ? __float_as_uint(p[c + i]) : kNone;
      } else {
        const int k = c + 2 * i;
        const uint32_t lo = k >= 0 && k < V ? __bfloat16_as_ushort(p[k]) : kNone >> 16;
        const uint32_t hi = k + 1 >= 0 && k + 1 < V ? __bfloat16_as_ushort(p[k + 1]) : kNone >> 16;
        w[i] = lo | hi << 16;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ static __forceinline__ void floats(const uint4& r, float (&v)[kPer]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w[i]);
      else v[i] = __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
  }
};

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
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// One entry of every warp of the row, in every CTA of its cluster.
struct Exchange {
  uint64_t mass[2][kMaxWarps];
  uint32_t count[2][kMaxWarps];
};
struct Sum {
  uint64_t mass;
  uint32_t count;
};

struct Cluster {
  Exchange* x;
  int rank, ctas, phase;

  // Gives every CTA this warp's entry, and waits for all of them.
  __device__ __forceinline__ void share(uint64_t mass, uint32_t count) {
    const int lane = threadIdx.x & 31, me = rank * kWarps + (threadIdx.x >> 5);
    phase ^= 1;
    if (lane < ctas) {
      st_cluster_u64(mapa_shared(smem_u32(&x->mass[phase][me]), lane), mass);
      st_shared_cluster_u32(mapa_shared(smem_u32(&x->count[phase][me]), lane), count);
    }
    __syncwarp();
    cluster_sync_all();
  }
  // The sum over all warps.  (The other buffer's last readers are past this barrier's
  // predecessor, so two suffice.)
  __device__ __forceinline__ Sum total(uint64_t mass, uint32_t count) {
    share(mass, count);
    uint64_t m = 0;
    uint32_t n = 0;
    for (int i = threadIdx.x & 31; i < ctas * kWarps; i += 32) {
      m += x->mass[phase][i];
      n += x->count[phase][i];
    }
    return {warp_sum_u64(m), __reduce_add_sync(0xffffffffu, n)};
  }
};

// ------------------------------------------------------------ the kernel
template <class T, bool HELD>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
  using R = Row<T>;
  constexpr int kPer = R::kPer;
  extern __shared__ __align__(16) uint4 held[];  // HELD: this CTA's slots
  __shared__ Exchange exchange;
  __shared__ float2 table[32];
  __shared__ double log_min_p;
  // every CTA of the cluster runs before another writes to its shared memory
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Cluster cl{&exchange, 0, 1, 0};
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(cl.rank));
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cl.ctas));
  const int64_t b = blockIdx.x / cl.ctas;
  const R row(a, b);
  // this warp's slots, and the CTA's first
  const int slots = (row.units + 31) / 32, warps = cl.ctas * kWarps;
  const auto bound = [&](int w) {
    return static_cast<int>(static_cast<int64_t>(slots) * w / warps);
  };
  const int me = cl.rank * kWarps + warp, s0 = bound(me), s1 = bound(me + 1);
  const int cta0 = bound(cl.rank * kWarps);
  const auto fetch = [&](int s) {
    uint4 r = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
    if (sizeof(T) == 4) r = make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
    const int u = s * 32 + lane;
    if (u < row.units) r = row.load(u);
    return r;
  };
  const auto get = [&](int s, float (&v)[kPer]) {
    R::floats(HELD ? held[(s - cta0) * 32 + lane] : fetch(s), v);
  };

  const float T0 = a.temperature ? a.temperature[b] : 1.f;
  const int k = a.top_k ? a.top_k[b] : 0;
  const float p = a.top_p ? a.top_p[b] : 1.f;
  const float min_p = a.min_p ? a.min_p[b] : 0.f;
  const float u = a.u[b];
  if (warp == 0) {
    table[lane] = kPow2[lane];
    // one lane: 64-bit logarithms are slow
    if (lane == 0 && min_p > 0.f) log_min_p = log(static_cast<double>(fminf(min_p, 1.f)));
  }

  // The row, and its largest logit (NaN is passed over).
  float top = -INFINITY;
  constexpr int kAtOnce = 4;
  for (int s = s0; s < s1; s += kAtOnce) {
    uint4 r[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (s + i < s1) r[i] = fetch(s + i);
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (s + i >= s1) break;
      if (HELD) held[(s + i - cta0) * 32 + lane] = r[i];
      float v[kPer];
      R::floats(r[i], v);
#pragma unroll
      for (int j = 0; j < kPer; ++j) top = fmaxf(top, v[j]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  cl.share(0, __float_as_uint(top));
  for (int i = lane; i < warps; i += 32)
    top = fmaxf(top, __uint_as_float(exchange.count[cl.phase][i]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (top == -INFINITY) {  // nothing to pick from
    if (me == 0 && lane == 0) a.out[b] = -1;
    return;
  }
  const bool greedy = !(T0 >= kGreedyBelow);
  const Scale scale = make_scale(top, greedy ? 1.f : T0);

  // The tokens at or above x: how many, and (MASS) their mass.
  const auto at_least = [&](float x, bool mass) {
    uint32_t n = 0, wa = 0, wb = 0;
    for (int s = s0; s < s1; ++s) {
      float v[kPer];
      get(s, v);
      bool some = false;
#pragma unroll
      for (int j = 0; j < kPer; ++j) some = some || v[j] >= x;
      if (!__any_sync(0xffffffffu, some)) continue;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const bool in = v[j] >= x;
        if (mass) {
          uint32_t ka, kb;
          weigh(v[j], scale, table, ka, kb);
          wa += in ? ka : 0u;
          wb += in ? kb : 0u;
        }
        n += in;
      }
    }
    return cl.total(warp_sum_u64(mass ? mass_of(wa, wb, n) : 0), __reduce_add_sync(0xffffffffu, n));
  };
  // The least x above which fewer than `target` (tokens, or mass) lie, from `low` on: the
  // row's tokens above it and so many of those equal to it make the target.
  float t = -FLT_MAX;
  uint32_t ties = UINT_MAX;
  const auto prefix = [&](uint64_t target, bool mass) {
    int lo = key_of<T>(t), hi = key_of<T>(top);
    uint64_t above = 0;
    while (lo < hi) {
      const int mid = static_cast<int>(lo + (static_cast<int64_t>(hi) - lo + 1) / 2);
      const Sum s = at_least(value_of<T>(mid), mass);
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
      const uint64_t w = max(weight(x, scale, table), uint64_t{1});
      r = (r + w - 1) / w;
    }
    r = min(r, static_cast<uint64_t>(UINT_MAX));
    if (x > t || r < ties) {
      t = x;
      ties = static_cast<uint32_t>(r);
    }
  };
  // The mass of what t and ties keep, warp by warp, and those of the warps before.
  uint64_t before, mine, total;
  uint32_t ties_before, own_ties;
  const auto kept = [&]() {
    uint32_t n = 0, wa = 0, wb = 0, eq = 0;
    for (int s = s0; s < s1; ++s) {
      float v[kPer];
      get(s, v);
      bool some = false;
#pragma unroll
      for (int j = 0; j < kPer; ++j) some = some || v[j] >= t;
      if (!__any_sync(0xffffffffu, some)) continue;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const bool in = v[j] > t;
        uint32_t ka, kb;
        weigh(v[j], scale, table, ka, kb);
        wa += in ? ka : 0u;
        wb += in ? kb : 0u;
        n += in;
        eq += v[j] == t;
      }
    }
    cl.share(warp_sum_u64(mass_of(wa, wb, n)), __reduce_add_sync(0xffffffffu, eq));
    // every warp goes over all entries: four consecutive ones a lane
    const uint64_t wt = weight(t, scale, table);
    constexpr int kEach = kMaxWarps / 32;
    uint64_t m[kEach];
    uint32_t e[kEach], sum = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int w = lane * kEach + i;
      m[i] = w < warps ? exchange.mass[cl.phase][w] : 0;
      e[i] = w < warps ? exchange.count[cl.phase][w] : 0;
      sum += e[i];
    }
    uint32_t ahead = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, ahead, o);
      if (lane >= o) ahead += x;
    }
    ahead -= sum;
    uint64_t lane_mass = 0;
    uint32_t e_at[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      e_at[i] = ahead;
      const uint32_t room = ties > ahead ? ties - ahead : 0;
      m[i] += wt * min(e[i], room);
      lane_mass += m[i];
      ahead += e[i];
    }
    uint64_t upto = lane_mass;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    total = __shfl_sync(0xffffffffu, upto, 31);
    upto -= lane_mass;
    // this warp's own entry
    before = mine = 0;
    ties_before = own_ties = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const uint64_t ub = __shfl_sync(0xffffffffu, upto, me / kEach);
      const uint64_t mb = __shfl_sync(0xffffffffu, m[i], me / kEach);
      const uint32_t tb = __shfl_sync(0xffffffffu, e_at[i], me / kEach);
      if (i == me % kEach) before = ub, mine = mb, ties_before = tb;
      upto += m[i];
    }
  };

  if (greedy) {
    t = top;
    ties = 1;
  } else {
    if (k > 0 && k < a.V) prefix(static_cast<uint64_t>(k), false);
    if (p < 1.f) {
      kept();
      const uint64_t part = __float2ull_rz(fmaxf(p, 0.f) * 0x1p64f);  // p in units of 2^-64
      uint64_t target = __umul64hi(part, total) + (part * total != 0);
      prefix(max(target, uint64_t{1}), true);
    }
    if (min_p > 0.f) {
      // w >= min_p w_max: l >= max + T ln(min_p), in 64 bits
      const double least = static_cast<double>(top) + static_cast<double>(T0) * log_min_p;
      const float x = top == INFINITY ? top : __double2float_ru(least);
      if (x > t) {
        t = x;
        ties = UINT_MAX;
      }
    }
  }
  kept();
  const float uc = fminf(fmaxf(u, 0.f), 0x1.fffffep-1f);
  const uint64_t target = __umul64hi(__float2ull_rz(uc * 0x1p64f), total);
  if (target < before || target - before >= mine) return;  // another warp's
  // this warp's tokens in order
  const uint64_t wt = weight(t, scale, table);
  for (int s = s0; s < s1; ++s) {
    float v[kPer];
    get(s, v);
    uint32_t eq = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) eq += v[j] == t;
    uint32_t rank = eq;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, rank, o);
      if (lane >= o) rank += x;
    }
    const uint32_t eq_all = __shfl_sync(0xffffffffu, rank, 31);
    rank += ties_before - eq;
    uint64_t w[kPer], sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const bool tie = v[j] == t;
      w[j] = v[j] > t ? weight(v[j], scale, table) : tie && rank < ties ? wt : 0;
      rank += tie;
      sum += w[j];
    }
    uint64_t upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    const uint64_t all = __shfl_sync(0xffffffffu, upto, 31);
    if (target - before < all) {
      // the first token with before + masses up to it > target
      uint64_t at = before + upto - sum;
      if (at <= target && target < at + sum) {
        int found = -1;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          at += w[j];
          if (found < 0 && at > target) found = j;
        }
        a.out[b] = row.first(s * 32 + lane) + found;
      }
      return;
    }
    before += all;
    ties_before += eq_all;
  }
}

// ------------------------------------------------------------- launching
constexpr int kHeldMost = 96 * 1024;  // of a row in a CTA's shared memory: two CTAs an SM

template <class T, bool HELD>
cudaError_t launch_sample(const SampleArgs& a, int64_t B, int ctas, int smem, cudaStream_t s) {
  auto* k = sample_kernel<T, HELD>;
  if (HELD) {
    static SmemLimit limit;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), kHeldMost, &limit);
    if (e != cudaSuccess) return e;
  }
  const cudaError_t e = launch_overlapped(k, dim3(static_cast<unsigned>(B * ctas)), dim3(kThreads),
                                          smem, s, ctas, a);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <class T>
cudaError_t run_sample(const SampleArgs& a, int64_t B, cudaStream_t s) {
  constexpr int kPer = 16 / static_cast<int>(sizeof(T));
  const int64_t slots = ((a.V + 2 * kPer - 2) / kPer + 31) / 32;  // whatever the row's shift
  const int ctas = kMaxCluster;
  const int64_t smem = (slots / ctas + 2) * 512;
  return smem <= kHeldMost ? launch_sample<T, true>(a, B, ctas, static_cast<int>(smem), s)
                           : launch_sample<T, false>(a, B, ctas, 0, s);
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
  if (B > 65535 || V > (int64_t{1} << 21)) return FLCE_ERR_UNSUPPORTED_SHAPE;
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
  const cudaError_t err = dtype == FLCE_BF16 ? run_sample<__nv_bfloat16>(a, B, s)
                                             : run_sample<float>(a, B, s);
  return err == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}
