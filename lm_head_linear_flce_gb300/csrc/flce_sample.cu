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

// c of a temperature, in two floats.
__device__ __forceinline__ float2 inverse_of(float T) {
  constexpr float kHi = 0x1.715476p0f, kLo = 0x1.4ae0cp-26f;  // 1 / ln 2
  const float hi = __fdiv_rn(kHi, T);
  return make_float2(hi, __fdividef(fmaf(-hi, T, kHi) + kLo, T));
}
__device__ __forceinline__ Scale make_scale(float top, float2 c) {
  if (!(c.x > 0.f) || top == INFINITY) c = make_float2(0.f, 0.f);  // every token alike
  Scale s;
  s.c_hi = c.x;
  s.c_lo = c.y;
  const float x = top * s.c_hi;
  const bool from_top = fabsf(x) > 64.f || top == INFINITY;
  const float shift = from_top ? 0.f : ceilf(x);
  s.base = from_top ? top : 0.f;
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
// A row in units of 16 bytes, the first starting `shift` elements before it.  32 units
// are a slot; a warp has consecutive slots, and a lane as many consecutive units of them
// as there are slots.  Elements outside the row are -infinity.
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
  __device__ bool whole(int u) const { return first(u) >= 0 && first(u) + kPer <= V; }
  __device__ float at(int c) const {
    if (c < 0 || c >= V) return -INFINITY;
    if constexpr (sizeof(T) == 4) return p[c];
    else return __bfloat162float(p[c]);
  }
  __device__ __forceinline__ uint4 load(int u) const {
    if (whole(u)) return *reinterpret_cast<const uint4*>(p + first(u));
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
template <class I>
__device__ __forceinline__ I warp_scan(I v) {  // of this lane and those before
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const I x = __shfl_up_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) >= o) v += x;
  }
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
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
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

constexpr int kList = 1024;   // tokens of a list
constexpr int kBins = 2048;   // of a histogram of masses, 1/64 of an octave each
constexpr int kGroups = 32;   // of bins, whose sums the CTAs exchange

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
  };
  uint64_t part[kWarps];
  float2 table[32];
  float2 inverse;    // c of the temperature
  float2 log_min_p;  // T ln(min_p)
  uint32_t listed;
  int found;
  float cut;
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
  // The sum over the warps first .. last - 1.
  __device__ __forceinline__ Sum sum(int first, int last) const {
    uint64_t m = 0;
    uint32_t n = 0;
    for (int i = first + (threadIdx.x & 31); i < last; i += 32) {
      m += sh.mass[phase][i];
      n += sh.count[phase][i];
    }
    return {warp_sum_u64(m), __reduce_add_sync(0xffffffffu, n)};
  }
  __device__ __forceinline__ Sum total(uint64_t mass, uint32_t count) {
    share(mass, count);
    return sum(0, ctas * kWarps);
  }
};

// ------------------------------------------------------- lists in shared memory
// Sorts the first n (a power of two, 64 to kList) of v, the larger first, with the
// block's first n / 64 warps, which alone call it.
__device__ void sort_list(uint64_t* v, int n) {
  const int threads = n / 2;
  for (int size = 2; size <= n; size <<= 1) {
    for (int stride = size / 2; stride > 0; stride >>= 1) {
      const int t = threadIdx.x;
      const int i = 2 * t - (t & (stride - 1)), k = i + stride;
      const uint64_t a = v[i], b = v[k];
      if ((a < b) == ((i & size) == 0)) {
        v[i] = b;
        v[k] = a;
      }
      // a warp's 32 pairs lie in 64 neighbours, and stay there while strides do
      if (stride > 32 || (stride == 1 && size >= 64))
        asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
      else __syncwarp();
    }
  }
}

// Sums of w[0 .. n) up to and including each, in place, by `threads` threads (a multiple
// of 32, which alone call it); returns the total.
__device__ uint64_t scan_list(uint64_t* w, int n, int threads, uint64_t* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t carry = 0;
  for (int i0 = 0; i0 < n; i0 += threads) {
    const int i = i0 + threadIdx.x;
    const uint64_t x = warp_scan(i < n ? w[i] : uint64_t{0});
    if (lane == 31) part[warp] = x;
    asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
    const int warps = threads / 32;
    const uint64_t p = lane < warps ? part[lane] : 0;
    const uint64_t upto = warp_scan(p);
    const uint64_t before = __shfl_sync(0xffffffffu, upto - p, warp);
    if (i < n) w[i] = carry + before + x;
    carry += __shfl_sync(0xffffffffu, upto, warps - 1);
    asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
  }
  return carry;
}

__device__ __forceinline__ int list_size(uint32_t n) {  // a power of two, 64 at least
  return n <= 64 ? 64 : 2 << (31 - __clz(static_cast<int>(n) - 1));
}

// ------------------------------------------------------------ the kernel
template <class T, bool HELD>
__global__ void __launch_bounds__(kThreads, 2)
    sample_kernel(const SampleArgs a, const int stride) {
  using R = Row<T>;
  constexpr int kPer = R::kPer;
  // kList * 8 bytes at least; HELD: this CTA's part of the row, `stride` units a lane (an
  // odd number, so that lanes read their units without bank conflicts)
  extern __shared__ __align__(16) uint4 held[];
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
  const R row(a, b);
  const int slots = (row.units + 31) / 32, warps = cl.ctas * kWarps;
  const int me = cl.rank * kWarps + warp;
  const auto first_slot = [&](int w) {  // (V <= 2^21: below 2^31)
    return static_cast<int>(static_cast<uint32_t>(slots * w) / static_cast<uint32_t>(warps));
  };
  const int s0 = first_slot(me), each = first_slot(me + 1) - s0;
  const int u0 = s0 * 32;  // the warp's first unit; lane l has each of them from u0 + l * each
  uint4* mine = held + (warp * 32 + lane) * stride;
  const auto get = [&](int i, float (&v)[kPer]) {
    if constexpr (HELD) {
      R::floats(mine[i], v);
    } else {
      R::floats(row.load(u0 + lane * each + i), v);
    }
  };

  if constexpr (HELD) {
    // in the order of memory, all of it on its way at once
    int to = lane / max(each, 1), at = lane - to * each;
    const int step = 32 / max(each, 1), rest = 32 - step * each;
    for (int s = 0; s < each; ++s) {
      const int u = u0 + s * 32 + lane;
      uint4* dst = held + (warp * 32 + to) * stride + at;
      if (row.whole(u))
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)),
                     "l"(row.p + row.first(u))
                     : "memory");
      else *dst = row.load(u);
      to += step;
      at += rest;
      if (at >= each) at -= each, ++to;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  const float T0 = a.temperature ? a.temperature[b] : 1.f;
  const int k = a.top_k ? a.top_k[b] : 0;
  const float p = a.top_p ? a.top_p[b] : 1.f;
  const float min_p = a.min_p ? a.min_p[b] : 0.f;
  const float u = a.u[b];
  const bool greedy = !(T0 >= kGreedyBelow);
  if (warp == 0) {
    sh.table[lane] = kPow2[lane];
    if (lane == 0) {
      sh.listed = 0;
      sh.cut = -FLT_MAX;
      sh.inverse = inverse_of(greedy ? 1.f : T0);
      // one lane: 64-bit operations are slow
      if (min_p > 0.f) {
        const double d = static_cast<double>(T0) * log(static_cast<double>(fminf(min_p, 1.f)));
        sh.log_min_p.x = static_cast<float>(d);
        sh.log_min_p.y = static_cast<float>(d - static_cast<double>(sh.log_min_p.x));
      }
    }
  }
  for (int i = threadIdx.x; i < kBins; i += kThreads) sh.bins[i] = 0;
  if constexpr (HELD) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
  }

  // The largest logit (NaN is passed over): the lane's, the warps', the row's.
  float lane_top = -INFINITY;
  for (int i = 0; i < each; ++i) {
    float v[kPer];
    get(i, v);
#pragma unroll
    for (int j = 0; j < kPer; ++j) lane_top = fmaxf(lane_top, v[j]);
  }
  const auto warp_max = [](float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  };
  float top = warp_max(lane_top);
  cluster_wait();
  cl.share(0, __float_as_uint(top));
  const uint32_t* warp_tops = sh.count[cl.phase];
  for (int i = lane; i < warps; i += 32) top = fmaxf(top, __uint_as_float(warp_tops[i]));
  top = warp_max(top);
  if (top == -INFINITY) {  // nothing to pick from
    if (me == 0 && lane == 0) a.out[b] = -1;
    return;
  }
  const Scale scale = make_scale(top, sh.inverse);
  // what min_p keeps: w >= min_p w_max, l >= max + T ln(min_p), rounded up
  float least = -FLT_MAX;
  if (!greedy && min_p > 0.f) {
    const float2 d = sh.log_min_p;
    const float sum = __fadd_rn(top, d.x), back = __fsub_rn(sum, top);
    const float rest = __fadd_rn(
        __fadd_rn(__fsub_rn(top, __fsub_rn(sum, back)), __fsub_rn(d.x, back)), d.y);
    least = rest > 0.f ? nextafterf(sum, INFINITY) : sum;
    if (!(least > -FLT_MAX)) least = -FLT_MAX;
    if (top == INFINITY) least = top;
  }
  const bool by_k = !greedy && k > 0 && k < a.V, by_p = !greedy && p < 1.f;
  const uint64_t part_p = __float2ull_rz(fmaxf(fminf(p, 0x1.fffffep-1f), 0.f) * 0x1p64f);
  // the mass before a token that is kept is less than this
  const auto target_p = [&](uint64_t all) {  // p * all, rounded up; the first token always
    return max(static_cast<uint64_t>(__umul64hi(part_p, all)) + (part_p * all != 0), uint64_t{1});
  };
  const uint64_t part_u = __float2ull_rz(fminf(fmaxf(u, 0.f), 0x1.fffffep-1f) * 0x1p64f);

  // The tokens at or above x: how many, and (with `mass`) their mass.
  const auto at_least = [&](float x, bool mass) {
    uint32_t n = 0, wa = 0, wb = 0;
    for (int i = 0; i < each; ++i) {
      float v[kPer];
      get(i, v);
      bool some = false;
#pragma unroll
      for (int j = 0; j < kPer; ++j) some = some || v[j] >= x;
      if (!__any_sync(0xffffffffu, some)) continue;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const bool in = v[j] >= x;
        if (mass) {
          uint32_t ka, kb;
          weigh(v[j], scale, sh.table, ka, kb);
          wa += in ? ka : 0u;
          wb += in ? kb : 0u;
        }
        n += in;
      }
    }
    return cl.total(warp_sum_u64(mass ? mass_of(wa, wb, n) : 0), __reduce_add_sync(0xffffffffu, n));
  };
  float t = -FLT_MAX;
  uint32_t ties = UINT_MAX;
  // Narrows t and ties to the prefix that makes `target` (tokens, or mass): halves the
  // range of logits from t on, a pass over the row and a barrier each.  For any row; the
  // lists below are faster where they are long enough.
  const auto halve = [&](uint64_t target, bool mass) {
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
      const uint64_t w = max(weight(x, scale, sh.table), uint64_t{1});
      r = (r + w - 1) / w;
    }
    r = min(r, static_cast<uint64_t>(UINT_MAX));
    if (x > t || r < ties) {
      t = x;
      ties = static_cast<uint32_t>(r);
    }
  };

  // Puts the tokens with in(l) on the CTA's list, one that is full counts on; returns
  // the warp's number of them.
  const auto list_tokens = [&](const auto& in) {
    uint32_t n = 0;
    for (int i = 0; i < each; ++i) {
      float v[kPer];
      get(i, v);
      uint32_t which = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) which |= in(v[j]) ? 1u << j : 0u;
      if (!__any_sync(0xffffffffu, which != 0)) continue;
      const uint32_t c = __popc(which), upto = warp_scan(c);
      const uint32_t all = __shfl_sync(0xffffffffu, upto, 31);
      uint32_t at = 0;
      if (lane == 31) at = atomicAdd(&sh.listed, all);
      at = __shfl_sync(0xffffffffu, at, 31) + upto - c;
      n += all;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (!(which >> j & 1)) continue;
        const uint32_t id = static_cast<uint32_t>(row.first(u0 + lane * each + i) + j);
        const uint32_t key = static_cast<uint32_t>(key_of<float>(v[j] + 0.f)) ^ 0x80000000u;
        if (at < kList) sh.list[at] = static_cast<uint64_t>(key) << 32 | (id ^ 0xffffffffu);
        ++at;
      }
    }
    return n;
  };
  const auto listed_value = [](uint64_t e) {
    return value_of<float>(static_cast<int>(static_cast<uint32_t>(e >> 32) ^ 0x80000000u));
  };
  // Every CTA's list into `work`, n tokens in all, padded to list_size(n).
  const auto pull_lists = [&](uint32_t n) {
    uint32_t at = 0;
    for (int r = 0; r < cl.ctas; ++r) {
      const uint32_t c = cl.sum(r * kWarps, (r + 1) * kWarps).count;
      for (uint32_t i = threadIdx.x; i < c; i += kThreads)
        sh.work[at + i] = ld_cluster_u64(mapa_shared(smem_u32(&sh.list[i]), r));
      at += c;
    }
    for (uint32_t i = n + threadIdx.x; i < static_cast<uint32_t>(list_size(n)); i += kThreads)
      sh.work[i] = 0;
  };

  // --- top-k of few: a list of everything that can be among the first k, which the
  // cluster's first CTA then has to itself.
  constexpr int kFew = kMaxWarps * 7 / 8;
  if (by_k && k <= kFew && k <= warps * 7 / 8) {
    // the k-th largest of the warps' largest: k tokens are at or above it
    const int v = threadIdx.x >> 2;
    uint32_t larger = 0;
    if (v < warps) {
      const float x = __uint_as_float(warp_tops[v]);
      for (int i = threadIdx.x & 3; i < warps; i += 4) {
        const float y = __uint_as_float(warp_tops[i]);
        larger += y > x || (y == x && i < v);
      }
    }
    larger += __shfl_xor_sync(0xffffffffu, larger, 1);
    larger += __shfl_xor_sync(0xffffffffu, larger, 2);
    if (v < warps && larger == static_cast<uint32_t>(k - 1) && (threadIdx.x & 3) == 0)
      sh.cut = fmaxf(__uint_as_float(warp_tops[v]), -FLT_MAX);
    __syncthreads();
    const float cut = sh.cut;
    const uint32_t n = list_tokens([&](float l) { return l >= cut; });
    const uint32_t N = cl.total(0, n).count;
    if (N <= kList) {
      if (cl.rank == 0) pull_lists(N);
      cluster_arrive();  // the lists have been read
      if (cl.rank != 0) {
        cluster_wait();
        return;
      }
      __syncthreads();
      const int size = list_size(N), threads = size / 2;
      auto* weights = reinterpret_cast<uint64_t*>(held);  // (the row is not needed any more)
      if (threadIdx.x < threads) {
        sort_list(sh.work, size);
        uint32_t keep = min(N, static_cast<uint32_t>(k));
        for (uint32_t i = threadIdx.x; i < keep; i += threads)
          weights[i] = weight(listed_value(sh.work[i]), scale, sh.table);
        asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
        const uint64_t all = scan_list(weights, keep, threads, sh.part);
        // p and min_p keep a prefix of these
        const uint64_t target = by_p ? target_p(all) : UINT64_MAX;
        uint32_t in = 0;
        for (uint32_t i = threadIdx.x; i < keep; i += threads)
          in += i == 0 || (weights[i - 1] < target && listed_value(sh.work[i]) >= least);
        in = __reduce_add_sync(0xffffffffu, in);
        if (lane == 0) sh.part[warp] = in;
        asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
        keep = 0;
        for (int w = 0; w < threads / 32; ++w) keep += static_cast<uint32_t>(sh.part[w]);
        const uint64_t kept = weights[keep - 1];
        asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
        // by id: ~id << 32 | place, the larger first
        const int size2 = list_size(keep);
        for (int i = threadIdx.x; i < size2; i += threads) {
          const uint64_t e = i < static_cast<int>(keep) ? sh.work[i] << 32 | i : 0;
          sh.list[i] = e;
        }
        asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
        if (threadIdx.x < size2 / 2) {
          const int threads2 = size2 / 2;
          sort_list(sh.list, size2);
          uint64_t* by_id = sh.work;
          for (uint32_t i = threadIdx.x; i < keep; i += threads2) {
            const uint32_t at = static_cast<uint32_t>(sh.list[i]);
            by_id[i] = weights[at] - (at ? weights[at - 1] : 0);
          }
          asm volatile("bar.sync 1, %0;" ::"r"(threads2) : "memory");
          scan_list(by_id, keep, threads2, sh.part);
          const uint64_t pick = __umul64hi(part_u, kept);
          for (uint32_t i = threadIdx.x; i < keep; i += threads2)
            if (by_id[i] > pick && (i == 0 || by_id[i - 1] <= pick))
              a.out[b] = static_cast<int64_t>(~static_cast<uint32_t>(sh.list[i] >> 32));
        }
      }
      __syncwarp();
      cluster_wait();
      return;
    }
  }
  if (greedy) {
    t = top;
    ties = 1;
  }

  // What t and ties keep: the lane's mass above t (with `ties` all ones: from t on) and its
  // tokens equal to t, to every CTA by warps.
  uint64_t lane_mass = 0;
  uint32_t lane_ties = 0;
  const auto weigh_kept = [&]() {
    uint32_t n = 0, wa = 0, wb = 0;
    lane_ties = 0;
    const bool some_ties = ties != UINT_MAX;
    for (int i = 0; i < each; ++i) {
      float v[kPer];
      get(i, v);
      bool some = false;
#pragma unroll
      for (int j = 0; j < kPer; ++j) some = some || v[j] >= t;
      if (!__any_sync(0xffffffffu, some)) continue;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const bool tie = some_ties && v[j] == t, in = v[j] >= t && !tie;
        uint32_t ka, kb;
        weigh(v[j], scale, sh.table, ka, kb);
        wa += in ? ka : 0u;
        wb += in ? kb : 0u;
        n += in;
        lane_ties += tie;
      }
    }
    lane_mass = mass_of(wa, wb, n);
  };

  if (by_k) halve(static_cast<uint64_t>(k), false);
  if (by_p) {
    weigh_kept();
    const Sum s = cl.total(warp_sum_u64(lane_mass), __reduce_add_sync(0xffffffffu, lane_ties));
    const uint64_t wt = weight(t, scale, sh.table);
    halve(target_p(s.mass + wt * min(s.count, ties)), true);
  }
  if (least > t) {
    t = least;
    ties = UINT_MAX;
  }
  weigh_kept();
  // The lanes' parts for the warp below; the warps' to every CTA.
  uint64_t* lane_masses = sh.work;
  uint32_t* lane_tie_counts = reinterpret_cast<uint32_t*>(sh.work + kThreads);
  lane_masses[threadIdx.x] = lane_mass;
  lane_tie_counts[threadIdx.x] = lane_ties;
  cl.share(warp_sum_u64(lane_mass), __reduce_add_sync(0xffffffffu, lane_ties));
  // One warp of each CTA goes on: first, which warp has the token; four consecutive
  // entries a lane.
  if (warp != 0) return;
  const uint64_t wt = weight(t, scale, sh.table);
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
  upto -= lane_sum;
  int which = 0;
  uint64_t before = upto;
  uint32_t rank = e_at[0];
#pragma unroll
  for (int i = 0; i + 1 < kEach; ++i) {
    if (which == i && before + m[i] <= pick) {
      before += m[i];
      which = i + 1;
      rank = e_at[i + 1];
    }
  }
  before = __shfl_sync(0xffffffffu, before, owner);
  rank = __shfl_sync(0xffffffffu, rank, owner);
  const int w = owner * kEach + __shfl_sync(0xffffffffu, which, owner) - cl.rank * kWarps;
  if (w < 0 || w >= kWarps) return;  // another CTA's
  // The lane that has it, then its tokens, which are consecutive, 32 at a time.
  lane_mass = lane_masses[w * 32 + lane];
  lane_ties = lane_tie_counts[w * 32 + lane];
  rank += warp_scan(lane_ties) - lane_ties;
  lane_mass += wt * min(lane_ties, ties > rank ? ties - rank : 0u);
  upto = before + warp_scan(lane_mass);
  const int who = __ffs(__ballot_sync(0xffffffffu, upto > pick)) - 1;
  before = __shfl_sync(0xffffffffu, upto - lane_mass, who);
  rank = __shfl_sync(0xffffffffu, rank, who);
  const int first = first_slot(cl.rank * kWarps + w);
  const int count = (first_slot(cl.rank * kWarps + w + 1) - first) * kPer;
  const int c0 = row.first(first * 32) + who * count;
  const T* tokens = reinterpret_cast<const T*>(held + (w * 32 + who) * stride);
  for (int j0 = 0; j0 < count; j0 += 32) {
    const int j = j0 + lane;
    float l = -INFINITY;
    if (j < count) {
      if constexpr (!HELD) l = row.at(c0 + j);
      else if constexpr (sizeof(T) == 4) l = tokens[j];
      else l = __bfloat162float(tokens[j]);
    }
    const uint32_t equal = __ballot_sync(0xffffffffu, l == t);
    const uint32_t nth = rank + __popc(equal & ((1u << lane) - 1));
    const uint64_t x = l > t || (l == t && nth < ties) ? weight(l, scale, sh.table) : 0;
    const uint64_t sum = warp_scan(x);
    const uint32_t past = __ballot_sync(0xffffffffu, before + sum > pick);
    if (past) {
      if (lane == __ffs(past) - 1) a.out[b] = c0 + j;
      return;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
    rank += __popc(equal);
  }
}

// ------------------------------------------------------------- launching
// Of a row in a CTA's shared memory: two CTAs an SM.
static_assert(kThreads * 16 >= kList * 8);
constexpr int kHeldMost = 112 * 1024 - static_cast<int>(sizeof(Shared));

template <class T, bool HELD>
cudaError_t launch_sample(const SampleArgs& a, int64_t B, int ctas, int stride, cudaStream_t s) {
  auto* k = sample_kernel<T, HELD>;
  if (HELD) {
    static SmemLimit limit;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), kHeldMost, &limit);
    if (e != cudaSuccess) return e;
  }
  const cudaError_t e =
      launch_overlapped(k, dim3(static_cast<unsigned>(B * ctas)), dim3(kThreads),
                        HELD ? kThreads * stride * 16 : kList * 8, s, ctas, a, stride);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <class T>
cudaError_t run_sample(const SampleArgs& a, int64_t B, cudaStream_t s) {
  constexpr int kPer = 16 / static_cast<int>(sizeof(T));
  const int64_t slots = ((a.V + 2 * kPer - 2) / kPer + 31) / 32;  // whatever the row's shift
  const int ctas = kMaxCluster;
  const int each = static_cast<int>((slots + ctas * kWarps - 1) / (ctas * kWarps));
  const int stride = each | 1;
  return kThreads * stride * 16 <= kHeldMost ? launch_sample<T, true>(a, B, ctas, stride, s)
                                             : launch_sample<T, false>(a, B, ctas, stride, s);
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
