// Matrix product on 8-bit operands with block scales (flce_matmul_fp8):
//
//   y[m][v] = sum_j sa[m][j] * sb[v / 128][j] * P_j[m][v],
//   P_j     = the products of block j (128 columns of K), in FP32.
//
// The scales differ from block to block of K, so a block's sum P_j is formed by
// itself in tensor memory (four K = 32 MMAs, the first not accumulating) and the
// epilogue warps, which hold the FP32 result in registers, read it and add
// sa * sb * P_j while the tensor cores run the next block into the other
// accumulator.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "flce_fp8_device.cuh"
#include "flce_internal.h"
#include "flce_ops.h"

namespace flce {
namespace {

constexpr int kKB = 128;      // bytes (= columns of K) per pipeline stage: one scale block
constexpr int kMmaK8 = 32;    // K per MMA

// ------------------------------------------------ many rows: tiles
// A tile is 256 rows of A x 256 rows of B on a 2-CTA cluster (each CTA stages
// 128 rows of either, 32 KB a stage, and holds 128 x 256 of the result), or 128
// rows of A x 256 or 128 of B on a CTA by itself.  Eight epilogue warps per CTA:
// two per TMEM lane quarter, half of the columns each, so that the result is 128
// registers a thread at most.  Three warpgroups: the first (TMA, MMA) hands
// registers to the two of the epilogue; 384 threads launch with 168 each, 64512
// in all = 128 * 56 + 256 * 224.
//
// A block's scales change with every 128 columns of K, so its products go through
// registers (packed fma) before the next block may add to them; accumulators that
// fill TMEM, two of 256 columns or four of 128, hide that.
//
// Bound by the tensor cores, and in a loop of seconds by the board's power: pairs
// take 1.43 to 1.65 ms for 4096 x 152064 x 3584 to bf16 on one board or another (2.7
// to 3.1 PFLOP/s), 1.63 to 1.71 ms in a loop.  Up to 128 rows it is bound by reading
// B, of which a CTA by itself has 32 KB a block under way where one of a pair has 16:
// 128 x 151936 x 4096 to float32 takes 114 us (6.1 TB/s), with pairs 127.  Also measured, pairs at
// 4096 x 152064 x 3584: three accumulators of 160 columns 2.2 PFLOP/s, sixteen
// epilogue warps 1.9, accumulators in halves 1.5; a second staging buffer for the
// stores and scales fetched a tile ahead changed nothing.
constexpr int kTileThreads = 384;  // warp 0 TMA, warp 1 MMA, warps 4..11 epilogue
constexpr int kTileEpi = 8;
constexpr int kTileLeanRegs = 56;
constexpr int kTileEpiRegs = 224;
template <bool PAIR, int N>
struct TileShape {
  static constexpr int kRows = PAIR ? 256 : 128;      // rows of A, N of B
  static constexpr int kBRows = PAIR ? N / 2 : N;     // of B in this CTA's stage
  static constexpr int kBBytes = kBRows * kKB;
  static constexpr int kStageBytes = 128 * kKB + kBBytes;
  static constexpr int kStages = 192 * 1024 / kStageBytes;
  static constexpr int kAccs = kTmemCols / N;
  static constexpr int kCols = N / 2;                 // of an epilogue warp
  static constexpr int kSmem = kStages * kStageBytes + kTileEpi * kStageBufBytes + 1024 + 256;
  // a stage's barrier serves for its accumulator too, so at most kStages are ahead
  static_assert(kStages >= kAccs);
};
constexpr uint16_t kBoth = 0x3;

struct Fp8Args {
  int M, V, G;        // G: blocks of 128 columns of K
  int tiles_m, tiles_v;
  const float* a_scale;
  const float* b_scale;
  void* y;
  int64_t ldy;
  int tma_store;      // y's rows are 16-byte aligned
  unsigned long long wait_limit_ns;
  int64_t stop_after;  // self-test: blocks of K that a CTA loads before it stops; -1: all
};

struct Ring {
  uint32_t idx = 0, phase = 0;
  __device__ void advance(uint32_t n) {
    if (++idx == n) {
      idx = 0;
      phase ^= 1u;
    }
  }
};

// The four MMAs of one 128-byte K block: operands are 128-byte-swizzled, 8-row
// groups 1024 bytes apart, a K step 32 bytes along the swizzled row (2 in the
// descriptor's units of 16).  Descriptors of the first K step; their address
// field does not carry, so a step is an addition.
template <int M, int N, bool PAIR>
__device__ __forceinline__ void mma_block(uint32_t d, uint64_t ad, uint64_t bd) {
  constexpr uint32_t idesc = instr_desc_e4m3(M, N);
  constexpr uint64_t kStep = kMmaK8 / 16;
#pragma unroll
  for (int k = 0; k < kKB / kMmaK8; ++k) {
    if (PAIR) mma_e4m3_pair(d, ad + kStep * k, bd + kStep * k, idesc, k > 0);
    else mma_e4m3_single(d, ad + kStep * k, bd + kStep * k, idesc, k > 0);
  }
}

// How long a CTA that has given up waits at least for its copies and MMAs in
// flight, however short the limit is: they take microseconds.
constexpr unsigned long long kLandNs = 1000000;

// The wait that ends a role: bounded, whatever the abort flag says.
__device__ __forceinline__ WaitCtx last_wait(const WaitCtx& w, volatile uint32_t* never) {
  return {never, w.err, w.limit_ns > kLandNs ? w.limit_ns : kLandNs};
}

// Waits until the stages in `issued` have received their last loads: no CTA may
// exit with copies in flight.
template <int STAGES>
__device__ void drain_stages(uint32_t full, uint32_t issued, const Ring& pipe, const WaitCtx& w0) {
  volatile uint32_t never = 0u;
  const WaitCtx w = last_wait(w0, &never);
  for (int i = 0; i < STAGES; ++i)
    if (issued & (1u << i))
      wait_parity(full + 8 * i, static_cast<uint32_t>(i) < pipe.idx ? pipe.phase : pipe.phase ^ 1u,
                  w);
}

// The same for the CTA of a pair whose loads complete on its peer's barriers,
// which it cannot wait for: it gives them time.  Only after it has given up;
// otherwise the peer's wait covers them.
__device__ __noinline__ void let_copies_land() {
  const uint64_t t0 = global_timer_ns();
  for (int i = 0; i < 100000 && global_timer_ns() - t0 < kLandNs; ++i) __nanosleep(1000);
}

// What a result is where a wait has run out before it was complete.
constexpr uint32_t kNotComplete = 0x7fc00000u;  // NaN

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// One warp's 32 rows x 128 bytes of the result, already in its staging buffer
// (128-byte-swizzled rows), to global memory.
template <class O>
__device__ __forceinline__ void store_chunk(const Fp8Args& a, const CUtensorMap* ty, uint32_t buf,
                                            int row0, int col0, int lane) {
  constexpr int kCols = 128 / static_cast<int>(sizeof(O));
  // a TMA store writes whole 16-byte pieces, also where V ends inside one
  if (a.tma_store && (col0 + kCols <= a.V || a.V * sizeof(O) % 16 == 0)) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(ty, buf, col0, row0);
      bulk_commit();
    }
    return;
  }
  __syncwarp();
  for (int r = 0; r < 32 && row0 + r < a.M; ++r) {
#pragma unroll
    for (int c = lane; c < kCols; c += 32) {
      const uint32_t at =
          buf + r * 128 + (((c * sizeof(O) / 16) ^ (r & 7)) << 4) + (c * sizeof(O)) % 16;
      O* dst = static_cast<O*>(a.y) + static_cast<int64_t>(row0 + r) * a.ldy + col0 + c;
      if (col0 + c < a.V) {
        if (sizeof(O) == 4) {
          uint32_t v;
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
          *reinterpret_cast<uint32_t*>(dst) = v;
        } else {
          uint16_t v;
          asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
          *reinterpret_cast<uint16_t*>(dst) = v;
        }
      }
    }
  }
  __syncwarp();
}

template <class O, bool PAIR, int N>
__global__ void __launch_bounds__(kTileThreads, 1)
    flce_fp8_tile_kernel(const __grid_constant__ CUtensorMap ta,
                         const __grid_constant__ CUtensorMap tb,
                         const __grid_constant__ CUtensorMap ty, const Fp8Args a) {
  using S = TileShape<PAIR, N>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t a_base = (raw + 1023u) & ~1023u;
  const uint32_t b_base = a_base + S::kStages * 128 * kKB;
  const uint32_t staging = b_base + S::kStages * S::kBBytes;
  const uint32_t full = staging + kTileEpi * kStageBufBytes;
  const uint32_t done = full + 8 * S::kStages;
  const uint32_t tempty = done + 8 * S::kStages;
  const uint32_t drain = tempty + 8 * S::kAccs;
  auto* slot = reinterpret_cast<uint32_t*>(smem_raw + (drain + 8 - raw));
  volatile uint32_t* abort_flag = slot + 1;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(full + 8 * i, 1);  // the leader's producer, for both CTAs' bytes
      mbar_init(done + 8 * i, 1);  // the leader's multicast commit
    }
    for (int i = 0; i < S::kAccs; ++i)
      mbar_init(tempty + 8 * i, (PAIR ? 2 : 1) * kTileEpi);  // every epilogue warp
    mbar_init(drain, 1);
    *abort_flag = 0u;
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&ta);
    tma_prefetch_desc(&tb);
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(smem_u32(slot), kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc_single(smem_u32(slot), kTmemCols);
      tmem_relinquish_single();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync_all();  // no CTA signals its peer's barriers before they are set up
  tc_fence_after();
  const uint32_t tmem = *slot;
  griddep_launch_dependents();
  griddep_wait();  // set up; from here on global memory is read and written
  const WaitCtx w{abort_flag, nullptr, a.wait_limit_ns};
  const int tiles = a.tiles_m * a.tiles_v;
  const int first = blockIdx.x >> PAIR, step = gridDim.x >> PAIR;

  // The roles are branches of their own so that each is compiled for its share
  // of the registers.
  if (warp < 4) {
    regs_release<kTileLeanRegs>();
    if (warp == 0 && lane == 0) {
      Ring pipe;
      uint32_t issued = 0;
      int64_t loaded = 0;
      const uint64_t keep = l2_policy_evict_last(), once = l2_policy_evict_first();
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        const int arow = (t % a.tiles_m) * S::kRows + 128 * rank;
        const int brow = (t / a.tiles_m) * N + S::kBRows * rank;
        for (int j = 0; j < a.G; ++j) {
          ok = loaded++ != a.stop_after && wait_parity(done + 8 * pipe.idx, pipe.phase ^ 1u, w);
          if (!ok) break;
          const uint32_t bar = full + 8 * pipe.idx;
          const uint32_t as = a_base + pipe.idx * 128 * kKB, bs = b_base + pipe.idx * S::kBBytes;
          if (leader) mbar_arrive_expect_tx(bar, (PAIR ? 2 : 1) * S::kStageBytes);
          if (PAIR) {
            const uint32_t bar_c = mapa_shared(bar, 0);
            tma_load_2d_pair_hint(as, &ta, j * kKB, arow, bar_c, keep);
            tma_load_2d_pair(bs, &tb, j * kKB, brow, bar_c);
          } else {
#pragma unroll
            for (int i = 0; i < S::kBRows; i += 128)
              tma_load_2d_hint(bs + i * kKB, &tb, j * kKB, brow + i, bar, once);
            tma_load_2d_hint(as, &ta, j * kKB, arow, bar, keep);
          }
          issued |= 1u << pipe.idx;
          pipe.advance(S::kStages);
        }
      }
      if (leader) drain_stages<S::kStages>(full, issued, pipe, w);
      else if (!ok) let_copies_land();
    } else if (warp == 1 && leader) {
      // The whole warp runs the loop, so that its values stay uniform; one lane
      // issues.  A stage and an accumulator are both one block of K, so one
      // commit per block, on the stage's barrier, tells the producers that the
      // stage is free and the epilogue that the accumulator is there.
      const uint64_t ad0 = smem_desc_sw128(a_base, 0, 1024);
      const uint64_t bd0 = smem_desc_sw128(b_base, 0, 1024);
      Ring pipe, acc;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        for (int j = 0; j < a.G; ++j) {
          ok = wait_parity(full + 8 * pipe.idx, pipe.phase, w) &&
               wait_parity(tempty + 8 * acc.idx, acc.phase ^ 1u, w);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t ad = ad0 + static_cast<uint64_t>(pipe.idx) * (128 * kKB / 16);
            const uint64_t bd = bd0 + static_cast<uint64_t>(pipe.idx) * (S::kBBytes / 16);
            mma_block<S::kRows, N, PAIR>(tmem + acc.idx * N, ad, bd);
            if (PAIR) mma_commit_pair_multicast(done + 8 * pipe.idx, kBoth);
            else mma_commit_single(done + 8 * pipe.idx);
          }
          __syncwarp();
          pipe.advance(S::kStages);
          acc.advance(S::kAccs);
        }
      }
      // every issued MMA completes before tensor memory is released
      if (elect_one()) {
        if (PAIR) mma_commit_pair(drain);
        else mma_commit_single(drain);
        volatile uint32_t never = 0u;
        wait_parity(drain, 0u, last_wait(w, &never));
      }
      __syncwarp();
    }
  } else {
    regs_acquire<kTileEpiRegs>();
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t hand_back = PAIR ? mapa_shared(tempty, 0) : tempty;
    const uint32_t buf = staging + (warp - 4) * kStageBufBytes;
    Ring pipe, acc;
    bool ok = true;
    for (int t = first; t < tiles; t += step) {
      const int row0 = (t % a.tiles_m) * S::kRows + 128 * rank + q * 32;
      const int col0 = (t / a.tiles_m) * N + S::kCols * half;
      const int row = row0 + lane;
      const float* sa = a.a_scale + static_cast<int64_t>(min(row, a.M - 1)) * a.G;
      // a half past V has no scale block of its own; its columns are not stored
      const float* sb = a.b_scale + static_cast<int64_t>(min(col0, a.V - 1) / kScaleGroup) * a.G;
      uint64_t r[S::kCols / 2];
#pragma unroll
      for (int i = 0; i < S::kCols / 2; ++i) r[i] = 0;
      // scales are fetched two blocks ahead of their use
      float sa0 = sa[0], sb0 = sb[0], sa1 = sa[min(1, a.G - 1)], sb1 = sb[min(1, a.G - 1)];
      for (int j = ok ? 0 : a.G; j < a.G; ++j) {
        const float s = sa0 * sb0;
        sa0 = sa1;
        sb0 = sb1;
        const int jn = min(j + 2, a.G - 1);
        sa1 = sa[jn];
        sb1 = sb[jn];
        ok = wait_parity_warp(done + 8 * pipe.idx, pipe.phase, w);
        if (!ok) break;
        tc_fence_after();
        const uint32_t tbase = tmem + (static_cast<uint32_t>(q * 32) << 16) +
                               acc.idx * N + half * S::kCols;
        const uint32_t su = __float_as_uint(s);
        const uint64_t s2 = pack_f32x2(su, su);
#pragma unroll
        for (int c = 0; c < S::kCols / 64; ++c) {
          uint32_t x[64];
          tmem_ld(tbase + 64 * c, x);
          if (c + 1 == S::kCols / 64) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(hand_back + 8 * acc.idx);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i)
            r[32 * c + i] = fma_f32x2(s2, pack_f32x2(x[2 * i], x[2 * i + 1]), r[32 * c + i]);
        }
        pipe.advance(S::kStages);
        acc.advance(S::kAccs);
      }
      if (!ok) {  // this tile, and those after it, whose blocks are not waited for
#pragma unroll
        for (int i = 0; i < S::kCols / 2; ++i) r[i] = pack_f32x2(kNotComplete, kNotComplete);
      }
      constexpr int kWords = 32;                  // 128 bytes of one row per chunk
      constexpr int kPairs = sizeof(O) == 2 ? 32 : 16;  // register pairs per chunk
#pragma unroll
      for (int c = 0; c < S::kCols / 2 / kPairs; ++c) {
        const int x = col0 + c * 2 * kPairs;
        if (x >= a.V) break;  // warp-uniform
        uint32_t o[kWords];
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          float lo, hi;
          unpack_f32x2(r[c * kPairs + i], lo, hi);
          if (sizeof(O) == 2) {
            o[i] = pack_bf16x2(lo, hi);
          } else {
            o[2 * i] = __float_as_uint(lo);
            o[2 * i + 1] = __float_as_uint(hi);
          }
        }
        if (lane == 0) bulk_wait_read<0>();  // the buffer's last store has left it
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          st_shared_v4(buf + lane * 128 + ((i ^ (lane & 7)) << 4),
                       make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]));
        store_chunk<O>(a, &ty, buf, row0, x, lane);
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync_all();
  tc_fence_after();
  if (warp == 1) {
    if (PAIR) tmem_dealloc_pair(tmem, kTmemCols);
    else tmem_dealloc_single(tmem, kTmemCols);
  }
}

// ------------------------------------------------ few rows: B streamed
// With few rows of A the product is bound by reading B once.  The roles
// of the operands are swapped: 128 rows of B are the MMA's M, the rows of A
// (padded to NP) its N, so nothing of the tensor cores' work is wasted on
// padding to 128 rows of A.  Two CTAs per SM, whose rings keep about 190 KB in
// flight: a tile's first loads and last stores overlap the other CTA's stream,
// and 153 to 304 tiles run at once instead of in two rounds.  With fewer tiles
// of B than there is room for, a cluster of `splits` CTAs shares a tile, each
// taking a contiguous part of K; the parts are added in rank order through
// distributed shared memory.
//
// A column's scale differs from lane to lane here (it is a row of A), so each
// block costs the epilogue a scale per element from shared memory.  Of 151936 x
// 4096 bytes: 8 rows 94 to 96 us (6.6 TB/s), 32 105, 48 107, each to float32; NP = 64
// took 110 where tiles take 107, NP = 128 177 where they take 114.  NP = 48 is worth
// having where the rows of A start inside a 128-byte line and so cost two reads each:
// 37 x 32003 x 2064 18.3 to 19.7 us, padded to 64 21.8.
template <int NP>
struct RowShape {
  static constexpr int kThreads = 192;  // warp 0 TMA, warp 1 MMA, warps 2..5 epilogue
  static constexpr int kStageBytes = 128 * kKB + NP * kKB;
  static constexpr int kStages = NP <= 16 ? 6 : NP <= 32 ? 5 : 4;
  static constexpr int kAccs = 4;                     // accumulators of NP columns
  static constexpr int kTmem = NP == 48 ? 256 : NP * kAccs;  // a power of two
  // a stage's barrier serves for its accumulator too, so at most kStages are ahead
  static_assert(kStages >= kAccs);
  static constexpr int kScaleBytes = 4 * 2 * NP * 4;  // two buffers per epilogue warp
  static constexpr int kSmem = kStages * kStageBytes + kScaleBytes + 1024 + 512;
};
constexpr int kRowsPerSm = 2;  // CTAs per SM

template <int NP, class O>
__global__ void __launch_bounds__(RowShape<NP>::kThreads, kRowsPerSm)
    flce_fp8_rows_kernel(const __grid_constant__ CUtensorMap ta,
                         const __grid_constant__ CUtensorMap tb, const Fp8Args a,
                         const int splits) {
  using S = RowShape<NP>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // stage i: B rows, then A rows
  const uint32_t scales = base + S::kStages * S::kStageBytes;
  const uint32_t full = scales + S::kScaleBytes;
  const uint32_t done = full + 8 * S::kStages;
  const uint32_t tempty = done + 8 * S::kStages;
  const uint32_t drain = tempty + 8 * S::kAccs;
  auto* slot = reinterpret_cast<uint32_t*>(smem_raw + (drain + 8 - raw));
  volatile uint32_t* abort_flag = slot + 1;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(full + 8 * i, 1);  // the producer, for the stage's bytes
      mbar_init(done + 8 * i, 1);  // the MMAs' commit: stage free, accumulator there
    }
    for (int i = 0; i < S::kAccs; ++i) mbar_init(tempty + 8 * i, 4);
    mbar_init(drain, 1);
    *abort_flag = 0u;
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&ta);
    tma_prefetch_desc(&tb);
  }
  if (warp == 1) {
    tmem_alloc_single(smem_u32(slot), S::kTmem);
    tmem_relinquish_single();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  griddep_launch_dependents();
  griddep_wait();
  const WaitCtx w{abort_flag, nullptr, a.wait_limit_ns};
  const int part = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int j0 = static_cast<int>(static_cast<int64_t>(a.G) * part / splits);
  const int j1 = static_cast<int>(static_cast<int64_t>(a.G) * (part + 1) / splits);
  const int first = static_cast<int>(blockIdx.x) / splits;
  const int step = static_cast<int>(gridDim.x) / splits;
  bool ok = true;

  if (warp == 0) {
    if (lane == 0) {
      Ring pipe;
      uint32_t issued = 0;
      int64_t loaded = 0;
      const uint64_t keep = l2_policy_evict_last(), once = l2_policy_evict_first();
      for (int t = first; t < a.tiles_v && ok; t += step) {
        for (int j = j0; j < j1; ++j) {
          ok = loaded++ != a.stop_after && wait_parity(done + 8 * pipe.idx, pipe.phase ^ 1u, w);
          if (!ok) break;
          const uint32_t bar = full + 8 * pipe.idx;
          const uint32_t sb = base + pipe.idx * S::kStageBytes;
          mbar_arrive_expect_tx(bar, S::kStageBytes);
          tma_load_2d_hint(sb, &tb, j * kKB, t * 128, bar, once);
          tma_load_2d_hint(sb + 128 * kKB, &ta, j * kKB, 0, bar, keep);
          issued |= 1u << pipe.idx;
          pipe.advance(S::kStages);
        }
      }
      drain_stages<S::kStages>(full, issued, pipe, w);
    }
  } else if (warp == 1) {
    // as in the tile kernel: the whole warp in the loop, one lane issuing, one
    // commit a block
    const uint64_t bd0 = smem_desc_sw128(base, 0, 1024);
    const uint64_t ad0 = smem_desc_sw128(base + 128 * kKB, 0, 1024);
    Ring pipe, acc;
    for (int t = first; t < a.tiles_v && ok; t += step) {
      for (int j = j0; j < j1; ++j) {
        ok = wait_parity(full + 8 * pipe.idx, pipe.phase, w) &&
             wait_parity(tempty + 8 * acc.idx, acc.phase ^ 1u, w);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t at = static_cast<uint64_t>(pipe.idx) * (S::kStageBytes / 16);
          mma_block<128, NP, false>(tmem + acc.idx * NP, bd0 + at, ad0 + at);
          mma_commit_single(done + 8 * pipe.idx);
        }
        __syncwarp();
        pipe.advance(S::kStages);
        acc.advance(S::kAccs);
      }
    }
    if (elect_one()) {
      mma_commit_single(drain);
      volatile uint32_t never = 0u;
      wait_parity(drain, 0u, last_wait(w, &never));
    }
    __syncwarp();
  }

  // Epilogue warps: TMEM lane quarter q, a row of B a thread.
  const int q = warp & 3;
  constexpr int kSa = (NP + 31) / 32;  // scales of A a lane fetches per block
  float r[NP];
  if (warp >= 2) {
    auto* my_scales = reinterpret_cast<float*>(smem_raw + (scales - raw)) + (warp - 2) * 2 * NP;
    Ring pipe, acc;
    // the last tile's result stays in registers when K is split (one tile each)
    for (int t = first; t < a.tiles_v; t += step) {
      const int v = t * 128 + q * 32 + lane;
      const float* sb = a.b_scale + static_cast<int64_t>(t) * a.G;
#pragma unroll
      for (int n = 0; n < NP; ++n) r[n] = 0.f;
      // scales are fetched kAhead blocks before their use: a miss costs more than
      // a block takes
      constexpr int kAhead = 4;
      float sa[kAhead][kSa], sbj[kAhead];
      const auto fetch = [&](int slot, int j) {
        j = min(j, j1 - 1);
        sbj[slot] = sb[j];
#pragma unroll
        for (int i = 0; i < kSa; ++i) {
          const int n = i * 32 + lane;
          sa[slot][i] = n < a.M ? a.a_scale[static_cast<int64_t>(n) * a.G + j] : 0.f;
        }
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) fetch(i, j0 + i);
      for (int j = ok ? j0 : j1; j < j1; ++j) {
        // this block's scales into the warp's buffer, the queue moves up
        float* s = my_scales + (j & 1) * NP;
#pragma unroll
        for (int i = 0; i < kSa; ++i)
          if (NP % 32 == 0 || i * 32 + lane < NP) s[i * 32 + lane] = sa[0][i] * sbj[0];
        __syncwarp();
#pragma unroll
        for (int k = 0; k + 1 < kAhead; ++k) {
          sbj[k] = sbj[k + 1];
#pragma unroll
          for (int i = 0; i < kSa; ++i) sa[k][i] = sa[k + 1][i];
        }
        fetch(kAhead - 1, j + kAhead);
        ok = wait_parity_warp(done + 8 * pipe.idx, pipe.phase, w);
        if (!ok) break;
        tc_fence_after();
        const uint32_t tbase = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc.idx * NP;
        constexpr int kC = NP % 32 ? 16 : 32;
#pragma unroll
        for (int c = 0; c < NP / kC; ++c) {
          uint32_t p[kC];
          tmem_ld(tbase + kC * c, p);
#pragma unroll
          for (int i = 0; i < kC / 4; ++i) {
            const float4 f = *reinterpret_cast<const float4*>(s + kC * c + 4 * i);
            float* d = r + kC * c + 4 * i;
            d[0] = fmaf(f.x, __uint_as_float(p[4 * i]), d[0]);
            d[1] = fmaf(f.y, __uint_as_float(p[4 * i + 1]), d[1]);
            d[2] = fmaf(f.z, __uint_as_float(p[4 * i + 2]), d[2]);
            d[3] = fmaf(f.w, __uint_as_float(p[4 * i + 3]), d[3]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(tempty + 8 * acc.idx);
        pipe.advance(S::kStages);
        acc.advance(S::kAccs);
      }
      if (!ok) {  // this tile, and those after it, whose blocks are not waited for
#pragma unroll
        for (int n = 0; n < NP; ++n) r[n] = __uint_as_float(kNotComplete);
      }
      if (splits == 1 && v < a.V) {
        O* y = static_cast<O*>(a.y) + v;
#pragma unroll
        for (int n = 0; n < NP; ++n)
          if (n < a.M) {
            if constexpr (sizeof(O) == 2) y[n * a.ldy] = __float2bfloat16_rn(r[n]);
            else y[n * a.ldy] = r[n];
          }
      }
    }
  }
  if (splits > 1) {
    // Every role has finished with the stages: their memory takes this part's
    // result, [NP][128] floats, and each CTA adds a share of the columns of all
    // parts (a part that is not complete is NaN, and so are the sums).
    __syncthreads();
    const uint32_t mine = base;
    if (warp >= 2) {
#pragma unroll
      for (int n = 0; n < NP; ++n)
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(mine + 4u * (n * 128 + q * 32 + lane)),
                     "f"(r[n])
                     : "memory");
    }
    cluster_sync_all();
    const int v = first * 128 + q * 32 + lane;
    if (warp >= 2 && v < a.V && first < a.tiles_v) {
      for (int n = part; n < a.M; n += splits) {
        float sum = 0.f;
        for (int p = 0; p < splits; ++p) {
          float x;
          asm volatile("ld.shared::cluster.f32 %0, [%1];"
                       : "=f"(x)
                       : "r"(mapa_shared(mine + 4u * (n * 128 + q * 32 + lane), p))
                       : "memory");
          sum += x;
        }
        O* y = static_cast<O*>(a.y) + n * a.ldy + v;
        if constexpr (sizeof(O) == 2) *y = __float2bfloat16_rn(sum);
        else *y = sum;
      }
    }
    cluster_sync_all();  // no CTA leaves while its part is still read
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_single(tmem, S::kTmem);
}

// ------------------------------------------------------------- launching
// Rows of A up to which B is streamed past them: 48, and 64 where the tiles of B
// are so few that K is split (64 x 4000 x 4096: 10.4 us, in tiles 11.4; 64 x 32003 x
// 2064 20.0, in tiles 17.1).
constexpr int kFewRows = 48, kFewRowsSplit = 64;

template <bool PAIR, int N, class O>
cudaError_t launch_tiles(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& ty,
                         Fp8Args a, int sms, cudaStream_t s) {
  using S = TileShape<PAIR, N>;
  constexpr int kCtas = PAIR ? 2 : 1, kSmem = S::kSmem;
  a.tiles_m = (a.M + S::kRows - 1) / S::kRows;
  a.tiles_v = (a.V + N - 1) / N;
  static SmemLimit limit;
  auto* k = flce_fp8_tile_kernel<O, PAIR, N>;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), kSmem, &limit);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>(a.tiles_m) * a.tiles_v;
  const int at_once = static_cast<int>(std::min<int64_t>(tiles, sms / kCtas));
  e = launch_overlapped(k, dim3(kCtas * at_once), dim3(kTileThreads), kSmem, s, kCtas, ta, tb, ty,
                        a);
  note_launch();
  note_wait_limit(a.wait_limit_ns);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <class O>
cudaError_t launch_tiles_for(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& ty,
                             const Fp8Args& a, int sms, cudaStream_t s) {
  // Rounds of tiles, times what a round takes: a pair's tile 16, a CTA's of 256
  // columns 16.5, of 128 columns 11 (4096 x 4000 bytes: 65 rows 15.6, 15.6 and
  // 11.4 us; 256 x 151936 x 4096 137, 146 and 165; 300 x 151936 x 4096, whose last
  // pairs would be half empty, 232, 196 and 228).
  const auto rounds = [&](int64_t m, int64_t n, int64_t at_once) {
    return ((a.M + m - 1) / m * ((a.V + n - 1) / n) + at_once - 1) / at_once;
  };
  const int64_t pair = 32 * rounds(256, 256, sms / 2), single = 33 * rounds(128, 256, sms),
                narrow = 22 * rounds(128, 128, sms);
  if (narrow < std::min(pair, single)) return launch_tiles<false, 128, O>(ta, tb, ty, a, sms, s);
  return single < pair ? launch_tiles<false, 256, O>(ta, tb, ty, a, sms, s)
                       : launch_tiles<true, 256, O>(ta, tb, ty, a, sms, s);
}

template <int NP, class O>
cudaError_t launch_rows(const CUtensorMap& ta, const CUtensorMap& tb, const Fp8Args& a, int sms,
                        cudaStream_t s) {
  static SmemLimit limit;
  auto* k = flce_fp8_rows_kernel<NP, O>;
  cudaError_t e =
      allow_smem(reinterpret_cast<const void*>(k), RowShape<NP>::kSmem, &limit);
  if (e != cudaSuccess) return e;
  // As many parts of K as the device has room for, none empty.
  const int room = kRowsPerSm * sms;
  int splits = 1;
  while (splits < 8 && 2 * splits * a.tiles_v <= room && 2 * splits <= a.G) splits *= 2;
  e = launch_overlapped(k, dim3(splits > 1 ? splits * a.tiles_v : std::min(a.tiles_v, room)),
                        dim3(RowShape<NP>::kThreads), RowShape<NP>::kSmem, s, splits, ta, tb, a,
                        splits);
  note_launch();
  note_wait_limit(a.wait_limit_ns);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <class O>
cudaError_t launch_rows_for(const CUtensorMap& ta, const CUtensorMap& tb, const Fp8Args& a,
                            int np, int sms, cudaStream_t s) {
  if (np == 16) return launch_rows<16, O>(ta, tb, a, sms, s);
  if (np == 48) return launch_rows<48, O>(ta, tb, a, sms, s);
  if (np == 32) return launch_rows<32, O>(ta, tb, a, sms, s);
  return launch_rows<64, O>(ta, tb, a, sms, s);
}

flce_status matmul_fp8(const char* name, const void* A, int64_t lda, const float* a_scale,
                       const void* B, int64_t ldb, const float* b_scale, int64_t M, int64_t V,
                       int64_t K, void* y, int64_t ldy, flce_dtype out_dtype,
                       unsigned long long limit_ns, int64_t stop_after, flce_stream_t stream) {
  OpRange range(name);
  constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1024;
  if (M < 0 || V <= 0 || K <= 0 || !valid_dtype(out_dtype)) return FLCE_ERR_INVALID_ARG;
  if (K % 16 != 0 || K > kMaxRowElems || M > kMaxDim || V > kMaxDim)
    return FLCE_ERR_UNSUPPORTED_SHAPE;
  if (M == 0) return FLCE_OK;
  if (!A || !B || !a_scale || !b_scale || !y) return FLCE_ERR_INVALID_ARG;
  if (lda < K || ldb < K || ldy < V || lda % 16 != 0 || ldb % 16 != 0) return FLCE_ERR_INVALID_ARG;
  const size_t e = dtype_bytes(out_dtype);
  if (!aligned_to(A, 16) || !aligned_to(B, 16) || !aligned_to(a_scale, 4) ||
      !aligned_to(b_scale, 4) || !aligned_to(y, e))
    return FLCE_ERR_INVALID_ARG;
  const int64_t gk = (K + kScaleGroup - 1) / kScaleGroup, gv = (V + kScaleGroup - 1) / kScaleGroup;
  const Range yr = {y, span_bytes(M, V, ldy, e)};
  const Range ins[] = {{A, span_bytes(M, K, lda, 1)},
                       {B, span_bytes(V, K, ldb, 1)},
                       {a_scale, span_bytes(M, gk, gk, 4)},
                       {b_scale, span_bytes(gv, gk, gk, 4)}};
  for (const Range& r : ins)
    if (ranges_overlap(yr, r)) return FLCE_ERR_INVALID_ARG;
  if ((M + 127) / 128 * gv > kMaxDim) return FLCE_ERR_UNSUPPORTED_SHAPE;
  int sms = 0;
  const flce_status st = check_device(&sms);
  if (st != FLCE_OK) return st;
  const auto s = reinterpret_cast<cudaStream_t>(stream);
  Fp8Args a = {};
  a.M = static_cast<int>(M);
  a.V = static_cast<int>(V);
  a.G = static_cast<int>(gk);
  a.a_scale = a_scale;
  a.b_scale = b_scale;
  a.y = y;
  a.ldy = ldy;
  a.wait_limit_ns = limit_ns;
  a.stop_after = stop_after;
  constexpr CUtensorMapDataType kU8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  CUtensorMap ta, tb;
  if (!make_tmap(&tb, B, K, V, ldb, kKB, 128, kU8)) return FLCE_ERR_CUDA;
  cudaError_t err;
  if (M <= (gv <= sms ? kFewRowsSplit : kFewRows)) {
    const int np = M <= 16 ? 16 : M <= 32 ? 32 : M <= 48 ? 48 : 64;
    a.tiles_v = static_cast<int>(gv);
    if (!make_tmap(&ta, A, K, M, lda, kKB, np, kU8)) return FLCE_ERR_CUDA;
    err = out_dtype == FLCE_BF16 ? launch_rows_for<__nv_bfloat16>(ta, tb, a, np, sms, s)
                                 : launch_rows_for<float>(ta, tb, a, np, sms, s);
  } else {
    a.tma_store = aligned_to(y, 16) && ldy * e % 16 == 0;
    CUtensorMap ty = tb;  // not used without TMA stores
    if (!make_tmap(&ta, A, K, M, lda, kKB, 128, kU8)) return FLCE_ERR_CUDA;
    if (a.tma_store &&
        !make_tmap(&ty, y, V, M, ldy * e, 128 / e, 32,
                   out_dtype == FLCE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                          : CU_TENSOR_MAP_DATA_TYPE_FLOAT32))
      return FLCE_ERR_CUDA;
    err = out_dtype == FLCE_BF16 ? launch_tiles_for<__nv_bfloat16>(ta, tb, ty, a, sms, s)
                                 : launch_tiles_for<float>(ta, tb, ty, a, sms, s);
  }
  return err == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

flce_status flce_matmul_fp8(const void* A, int64_t lda, const float* a_scale, const void* B,
                            int64_t ldb, const float* b_scale, int64_t M, int64_t V, int64_t K,
                            void* y, int64_t ldy, flce_dtype out_dtype, flce_stream_t stream) {
  return matmul_fp8("flce_matmul_fp8", A, lda, a_scale, B, ldb, b_scale, M, V, K, y, ldy,
                    out_dtype, wait_limit_ns(), -1, stream);
}

flce_status flce_selftest_matmul_fp8_timeout(int64_t stop_after, int64_t limit_ns, const void* A,
                                             int64_t lda, const float* a_scale, const void* B,
                                             int64_t ldb, const float* b_scale, int64_t M,
                                             int64_t V, int64_t K, void* y, int64_t ldy,
                                             flce_dtype out_dtype, flce_stream_t stream) {
  if (stop_after < 0 || limit_ns <= 0) return FLCE_ERR_INVALID_ARG;
  return matmul_fp8("flce_selftest_matmul_fp8_timeout", A, lda, a_scale, B, ldb, b_scale, M, V, K,
                    y, ldy, out_dtype, static_cast<unsigned long long>(limit_ns), stop_after,
                    stream);
}

}  // extern "C"
