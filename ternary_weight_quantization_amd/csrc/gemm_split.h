// The MFMA GEMMs' work split over workgroups (stream-K), their kernels, and the
// host side: plans, workspace, launches. gemm_kernels.hip describes the scheme.
// Each source that includes this has its own kernels and its own count of
// waits that gave up (take_local_split_timeouts).
#pragma once

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "gemm_core.h"
#include "internal.h"

namespace bitnet {

// dX (bf16 out, scaled by bf16(gamma)) and dW (bf16 or f32 out, unscaled).
template <bool OUT_F32>
struct Bf16Epilogue {
  void* out;
  const float* gamma;  // NULL: no scale
  int64_t I, J;        // output [J][I]

  struct Pre { float g; };
  static constexpr int kEB = OUT_F32 ? 4 : 2;
  static constexpr int kWaveLds = EpStage<kEB>::kWaveBytes;
  __device__ __forceinline__ Pre prefetch(int, int) const { return Pre{gamma ? *gamma : 1.0f}; }
  __device__ __forceinline__ void store(MfmaBf16::Acc (&acc)[kFI][kFJ], const Pre& pre, int i0, int j0,
                                        int lane, char* wlds) const {
    float sc = 1.0f;
    if (gamma) sc = bf16_to_f32(f32_to_bf16_bits(pre.g));  // bf16(gamma), exact in fp32
#pragma unroll
    for (int fj = 0; fj < kFJ; ++fj) {
#pragma unroll
      for (int fi = 0; fi < kFI; ++fi)
#pragma unroll
        for (int gi = 0; gi < 4; ++gi) {
          const float v0 = acc[fi][fj][4 * gi] * sc, v1 = acc[fi][fj][4 * gi + 1] * sc;
          const float v2 = acc[fi][fj][4 * gi + 2] * sc, v3 = acc[fi][fj][4 * gi + 3] * sc;
          if constexpr (OUT_F32)
            EpStage<4>::put(wlds, lane, fi, gi, make_uint4(__float_as_uint(v0), __float_as_uint(v1),
                                                           __float_as_uint(v2), __float_as_uint(v3)));
          else
            EpStage<2>::put(wlds, lane, fi, gi, make_uint2(pack_bf16x2(v0, v1), pack_bf16x2(v2, v3)));
        }
      EpStage<kEB>::drain(wlds, static_cast<char*>(out), I, J, i0, j0 + 32 * fj, lane);
    }
  }
};

// ---------------------------------------------------------------------------
// Work split. The T output tiles of a product, each of S reduction stages,
// are T*S iterations in tile-major order (tile t = (ti, tj) with ti fastest).
// A grid of G workgroups shares them out: virtual workgroup v takes
// iterations [lo(v), lo(v+1)), lo(v) = floor(v * T * S / G). With G = T each
// workgroup gets one whole tile. With G below T (or not dividing it) a tile
// can be split between consecutive workgroups (stream-K): each piece
// accumulates its stages, and the last piece to arrive adds the partial
// tiles of the others in piece order, so the sum does not depend on the
// arrival order, and runs the epilogue.
//
// Workgroups are dispatched round-robin over the 8 XCDs (block b on XCD
// b % 8); virtual indices are numbered XCD by XCD, so an XCD owns a
// contiguous range of iterations and its blocks share operand panels in its
// L2 (and the pieces of a split tile are usually on one XCD).
// ---------------------------------------------------------------------------

struct SplitPlan {
  int64_t total;       // T * S
  int grid;            // G
  int tiles_i;
  int nstages;         // S
  uint32_t spin_limit; // polls before a wait for published partials gives up
  uint64_t gen;        // tag of this launch in the counters (0 < gen < 2^48)
  int nslots;          // partial-tile slots: min(2G, G + T - 1)
  uint64_t* counters;  // [T][2] tagged counters (pieces arrived, partials
                       // published); NULL when no tile is split
  uint4* partials;     // [nslots][64][kThreads] 16-byte chunks of partial tiles
};

__host__ __device__ __forceinline__ int64_t split_lo(const SplitPlan& p, int v) {
  return (int64_t)v * p.total / p.grid;
}

// The virtual workgroup whose range holds iteration it.
__host__ __device__ __forceinline__ int split_owner(const SplitPlan& p, int64_t it) {
  return (int)(((it + 1) * p.grid - 1) / p.total);
}

// Partial-tile slot of workgroup v's piece of tile t. Two numberings, each
// giving every piece its own slot; the plan takes the one with fewer slots:
//  - 2v for the tile v's range starts in, 2v + 1 for the tile it ends in
//    (a range holds at most two split pieces: any tile strictly inside it
//    is whole), 2G slots;
//  - v + t: along the iteration order the next piece has the next
//    workgroup, the next tile, or both, so v + t strictly increases,
//    G + T - 1 slots (fewer when G > T).
__host__ __device__ __forceinline__ int partial_slots(int64_t tiles, int grid) {
  const int64_t a = 2 * (int64_t)grid, b = (int64_t)grid + tiles - 1;
  return (int)(a < b ? a : b);
}
__host__ __device__ __forceinline__ int64_t piece_slot(const SplitPlan& p, int v, int t) {
  if (p.nslots < 2 * p.grid) return (int64_t)v + t;
  return 2 * (int64_t)v + ((int64_t)t == split_lo(p, v) / p.nstages ? 0 : 1);
}

// The piece that starts at iteration it of a range ending at hi: tile t,
// stages [s0, s1).
__host__ __device__ __forceinline__ void split_piece(const SplitPlan& p, int64_t it, int64_t hi, int* t, int* s0,
                                                     int* s1) {
  *t = (int)(it / p.nstages);
  *s0 = (int)(it - (int64_t)*t * p.nstages);
  *s1 = (int)((int64_t)p.nstages < *s0 + (hi - it) ? (int64_t)p.nstages : *s0 + (hi - it));
}

// The workgroups that hold pieces of tile t: va .. va + n - 1, in stage order.
__host__ __device__ __forceinline__ void split_tile_owners(const SplitPlan& p, int t, int* va, int* n) {
  const int64_t S = p.nstages;
  *va = split_owner(p, (int64_t)t * S);
  *n = split_owner(p, (int64_t)t * S + S - 1) - *va + 1;
}

// Waits for published partials that ran out of polls (a piece that never
// published: it cannot happen while every workgroup makes progress). The
// tile is then written as NaN (int32 accumulators: INT32_MIN) instead of a
// sum of unpublished data, and this counter is raised; the host reads and
// clears it with bitnet_split_timeouts().
static __device__ unsigned int g_split_timeouts;

__device__ __forceinline__ uint32_t tagged_count(const uint64_t* c, uint64_t gen) {
  const uint64_t v = __hip_atomic_load(c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return (v >> 16) == gen ? (uint32_t)(v & kCountMask) : 0u;
}

// Wait until `want` partials of a tile are published. Only pieces that have
// already arrived (so are running and only have their stores left) are
// waited for, so the wait ends; the bound (about a second at the default
// limit) is a safety net. Returns false when it gave up.
__device__ __forceinline__ bool wait_published(const uint64_t* c, uint64_t gen, uint32_t want, uint32_t limit) {
  for (uint32_t i = 0; i < limit; ++i) {
    if (tagged_count(c, gen) >= want) return true;
    __builtin_amdgcn_s_sleep(2);
  }
  return tagged_count(c, gen) >= want;
}

// Element e (0..3) of 16-byte chunk c (0..63) of a thread's accumulators:
// chunk c = 4 * (kFJ * fi + fj) + q holds acc[fi][fj][4q .. 4q + 3].
template <class MT>
__device__ __forceinline__ uint4 acc_chunk(const typename MT::Acc (&acc)[kFI][kFJ], int c) {
  const int fi = c / (4 * kFJ), fj = (c / 4) % kFJ, q = c % 4;
  return make_uint4(MT::to_bits(acc[fi][fj][4 * q]), MT::to_bits(acc[fi][fj][4 * q + 1]),
                    MT::to_bits(acc[fi][fj][4 * q + 2]), MT::to_bits(acc[fi][fj][4 * q + 3]));
}

template <class MT>
__device__ __forceinline__ void acc_chunk_add(typename MT::Acc (&acc)[kFI][kFJ], int c, uint4 v) {
  const int fi = c / (4 * kFJ), fj = (c / 4) % kFJ, q = c % 4;
  acc[fi][fj][4 * q] += MT::from_bits(v.x);
  acc[fi][fj][4 * q + 1] += MT::from_bits(v.y);
  acc[fi][fj][4 * q + 2] += MT::from_bits(v.z);
  acc[fi][fj][4 * q + 3] += MT::from_bits(v.w);
}

__device__ __forceinline__ uint4 chunk_add_f32(uint4 a, uint4 b) {
  return make_uint4(__float_as_uint(__uint_as_float(a.x) + __uint_as_float(b.x)),
                    __float_as_uint(__uint_as_float(a.y) + __uint_as_float(b.y)),
                    __float_as_uint(__uint_as_float(a.z) + __uint_as_float(b.z)),
                    __float_as_uint(__uint_as_float(a.w) + __uint_as_float(b.w)));
}

template <class MT>
__device__ __forceinline__ uint4 chunk_add(uint4 a, uint4 b) {
  if constexpr (std::is_same<typename MT::Elem, float>::value) {
    return chunk_add_f32(a, b);
  } else {
    return make_uint4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
  }
}

// End of a piece of a split tile. Arrive; a piece that is not the last
// issues the stores of its partial tile and returns false (the caller
// signals them published once they are complete); the last one waits for
// the others' partials, adds them in piece order into acc and returns true
// (the caller then runs the epilogue). With pieces p_0..p_{n-1} and this one at
// position me, the sum is ((p_0 + ... + p_{me-1}) + own) + p_{me+1} + ...
// evaluated left to right (own + L == L + own exactly).
template <class MT>
__device__ __forceinline__ bool finish_piece(const SplitPlan& p, typename MT::Acc (&acc)[kFI][kFJ],
                                             int v, int t, int* s_flag) {
  const int tid = threadIdx.x;
  int va, n;
  split_tile_owners(p, t, &va, &n);
  const int me = v - va;
  uint64_t* cnt = p.counters + 2 * (int64_t)t;
  if (tid == 0) *s_flag = (int)tagged_arrive(cnt, p.gen);
  __syncthreads();
  const bool last = (*s_flag == n - 1);
  __syncthreads();
  const rsrc_t pr = make_rsrc(p.partials, (uint32_t)((int64_t)p.nslots * 64 * kThreads * 16));
  if (!last) {
    const uint32_t base = (uint32_t)(piece_slot(p, v, t) * 64 * kThreads + tid) * 16;
#pragma unroll
    for (int c = 0; c < 64; ++c) buf_store16_coherent(pr, base + c * kThreads * 16, acc_chunk<MT>(acc, c));
    asm volatile("" ::: "memory");  // keep the stores ahead of the next piece's loads
    return false;
  }
  if (tid == 0) {
    const bool ok = wait_published(cnt + 1, p.gen, (uint32_t)(n - 1), p.spin_limit);
    *s_flag = ok ? 1 : 0;
    if (!ok) atomicAdd(&g_split_timeouts, 1u);
    // Every piece has arrived and published: nothing else touches this
    // tile's counters in this launch. Clearing them lets a later launch
    // with the same tag (a replay of a captured graph) count from zero.
    __hip_atomic_store(cnt, uint64_t(0), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(cnt + 1, uint64_t(0), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (*s_flag == 0) {  // gave up: write the tile as a visible sentinel
#pragma unroll
    for (int fi = 0; fi < kFI; ++fi)
#pragma unroll
      for (int fj = 0; fj < kFJ; ++fj)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[fi][fj][e] = MT::from_bits(MT::kPoisonBits);
    return true;
  }
  constexpr int kBatch = 16;
#pragma unroll
  for (int c0 = 0; c0 < 64; c0 += kBatch) {
    if (me > 0) {
      uint4 L[kBatch];
      const uint32_t b0 = (uint32_t)(piece_slot(p, va, t) * 64 * kThreads + tid) * 16;
#pragma unroll
      for (int c = 0; c < kBatch; ++c) L[c] = buf_load16_coherent(pr, b0 + (c0 + c) * kThreads * 16);
      for (int j = 1; j < me; ++j) {
        const uint32_t bj = (uint32_t)(piece_slot(p, va + j, t) * 64 * kThreads + tid) * 16;
#pragma unroll
        for (int c = 0; c < kBatch; ++c)
          L[c] = chunk_add<MT>(L[c], buf_load16_coherent(pr, bj + (c0 + c) * kThreads * 16));
      }
#pragma unroll
      for (int c = 0; c < kBatch; ++c) acc_chunk_add<MT>(acc, c0 + c, L[c]);
    }
    for (int j = me + 1; j < n; ++j) {
      const uint32_t bj = (uint32_t)(piece_slot(p, va + j, t) * 64 * kThreads + tid) * 16;
      uint4 R[kBatch];
#pragma unroll
      for (int c = 0; c < kBatch; ++c) R[c] = buf_load16_coherent(pr, bj + (c0 + c) * kThreads * 16);
#pragma unroll
      for (int c = 0; c < kBatch; ++c) acc_chunk_add<MT>(acc, c0 + c, R[c]);
    }
  }
  return true;
}

// Whether an epilogue stages per-tile data into LDS before the main loop.
template <class EP, class = void>
struct StagesBias : std::false_type {};
template <class EP>
struct StagesBias<EP, std::void_t<decltype(EP::kStagesBias)>> : std::integral_constant<bool, EP::kStagesBias> {};

// The work of virtual workgroup v of a product: one whole tile (no split),
// or its range of (tile, stage) iterations (stream-K).
template <class MT, int MAP, class PL, class QL, class EP>
__device__ __forceinline__ void gemm_body(const PL& pl, const QL& ql, const EP& ep, const SplitPlan& plan,
                                          int v, char* smem, int* s_flag_p) {
  typedef SmemLayout<PL, QL> L;
  static_assert(kThreads / 64 * EP::kWaveLds <= L::kBytes, "epilogue staging fits in the stage buffers");
  int& s_flag = *s_flag_p;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wi = wave % kWavesI, wj = wave / kWavesI;
  const int prow0 = wi * kWTI, qrow0 = wj * kWTJ;
  if (plan.counters == nullptr) {
    // whole tiles: v, v + G, v + 2G, ... (one each when G = T)
    const int T = (int)(plan.total / plan.nstages);
    for (int t = v; t < T; t += plan.grid) {
      const int i0 = (t % plan.tiles_i) * kBI, j0 = (t / plan.tiles_i) * kBJ;
      typename MT::Acc acc[kFI][kFJ];
#pragma unroll
      for (int fi = 0; fi < kFI; ++fi)
#pragma unroll
        for (int fj = 0; fj < kFJ; ++fj) zero_acc(acc[fi][fj]);
      const typename EP::Pre pre = ep.prefetch(j0 + qrow0, lane);
      if constexpr (StagesBias<EP>::value) {
        __syncthreads();
        ep.stage_bias(i0);
      }
      run_stages<MT, MAP>(pl, ql, smem, acc, i0, j0, 0, plan.nstages, prow0, qrow0, lane, nullptr, 0);
      ep.store(acc, pre, i0 + prow0, j0 + qrow0, lane, smem + wave * EP::kWaveLds);
    }
    return;
  }

  const int64_t hi = split_lo(plan, v + 1);
  uint64_t* pending = nullptr;  // published-partials counter to signal
  for (int64_t it = split_lo(plan, v); it < hi;) {
    int t, s0, s1;
    split_piece(plan, it, hi, &t, &s0, &s1);
    const int i0 = (t % plan.tiles_i) * kBI, j0 = (t / plan.tiles_i) * kBJ;

    typename MT::Acc acc[kFI][kFJ];
#pragma unroll
    for (int fi = 0; fi < kFI; ++fi)
#pragma unroll
      for (int fj = 0; fj < kFJ; ++fj) zero_acc(acc[fi][fj]);

    const typename EP::Pre pre = ep.prefetch(j0 + qrow0, lane);
    if constexpr (StagesBias<EP>::value) {
      __syncthreads();
      ep.stage_bias(i0);
    }
    run_stages<MT, MAP>(pl, ql, smem, acc, i0, j0, s0, s1, prow0, qrow0, lane, pending, plan.gen);
    pending = nullptr;
    if ((s0 == 0 && s1 == plan.nstages) || finish_piece<MT>(plan, acc, v, t, &s_flag))
      ep.store(acc, pre, i0 + prow0, j0 + qrow0, lane, smem + wave * EP::kWaveLds);
    else
      pending = plan.counters + 2 * (int64_t)t + 1;
    it += s1 - s0;
  }
  if (pending != nullptr) {
    // the last piece published: wait for its stores, then signal
    wait_vmem();
    __syncthreads();
    if (tid == 0) tagged_arrive(pending, plan.gen);
  }
}

template <class MT, int MAP, class PL, class QL, class EP>
__global__ __launch_bounds__(kThreads, 1) void gemm_kernel(PL pl, QL ql, EP ep, SplitPlan plan) {
  typedef SmemLayout<PL, QL> L;
  __shared__ __attribute__((aligned(16))) char smem[L::kBytes];
  __shared__ int s_flag;
  gemm_body<MT, MAP>(pl, ql, ep, plan, cta_order(blockIdx.x, plan.grid), smem, &s_flag);
}

// Two independent products in one launch, each on its own share of every
// XCD: of the 8 * kt workgroups (one per CU, workgroup b on XCD b % 8),
// those with b / 8 < k1 run product 1, the others product 2, each
// stream-K over the first plan.grid (at most 8 * k1, resp. 8 * (kt - k1))
// of its workgroups, numbered XCD-contiguously; the rest of a share has no
// work. Used for the two STE backward products, which otherwise would each
// pay their split tail and launch on their own.
template <class MT, int MAP1, class PL1, class QL1, class EP1, int MAP2, class PL2, class QL2, class EP2>
__global__ __launch_bounds__(kThreads, 1) void gemm_pair_kernel(PL1 pl1, QL1 ql1, EP1 ep1, SplitPlan plan1,
                                                                PL2 pl2, QL2 ql2, EP2 ep2, SplitPlan plan2,
                                                                int k1) {
  typedef SmemLayout<PL1, QL1> L1;
  typedef SmemLayout<PL2, QL2> L2;
  __shared__ __attribute__((aligned(16))) char smem[L1::kBytes > L2::kBytes ? L1::kBytes : L2::kBytes];
  __shared__ int s_flag;
  const int x = blockIdx.x % 8, k = blockIdx.x / 8;
  if (k < k1) {
    const int b = 8 * k + x;
    if (b < plan1.grid) gemm_body<MT, MAP1>(pl1, ql1, ep1, plan1, cta_order(b, plan1.grid), smem, &s_flag);
  } else {
    const int b = 8 * (k - k1) + x;
    if (b < plan2.grid) gemm_body<MT, MAP2>(pl2, ql2, ep2, plan2, cta_order(b, plan2.grid), smem, &s_flag);
  }
}

// ---------------------------------------------------------------------------
// Host side: choice of the split, workspace, launch.
// ---------------------------------------------------------------------------

// This source's waits that gave up since the last call (synchronizes the device).
static hipError_t take_local_split_timeouts(unsigned int* count) {
  unsigned int* d = nullptr;
  if (hipError_t e = hipGetSymbolAddress(reinterpret_cast<void**>(&d), HIP_SYMBOL(g_split_timeouts))) return e;
  if (hipError_t e = hipDeviceSynchronize()) return e;
  if (hipError_t e = hipMemcpy(count, d, sizeof(unsigned int), hipMemcpyDeviceToHost)) return e;
  const unsigned int zero = 0;
  return hipMemcpy(d, &zero, sizeof(unsigned int), hipMemcpyHostToDevice);
}

constexpr int kMaxGrid = 256;  // workgroups of a split launch (one per CU)
constexpr size_t kPartialBytes = (size_t)64 * kThreads * 16;  // one partial tile

struct GemmShape {
  int64_t tiles_i, tiles_j, nstages;
  int overhead;  // cost of a split piece's publish / fix-up, in stages
  int64_t tiles() const { return tiles_i * tiles_j; }
};

// Per-piece costs of a split launch, in the product's stages: the last
// piece of a split tile reads every other piece's 256 KiB partial tile on
// its own CU, and a chip with every CU busy runs at a lower clock than one
// with a few idle, so a split must save many stages to pay. Measured
// interleaved on one MI355X, whole tiles against splits over 128-256
// workgroups and the split the cost model picked:
//  - int8 forward at 512, 1024, 2048, 4096, 8192 tokens (K 6912, N 2560),
//    2048 and 4096 tokens (K 2560, N 6912) and 4096, 16384 tokens (K = N =
//    2560): whole tiles were fastest at every shape (4096 x 6912 -> 2560:
//    90.7 us against 100-114 us split; 512 tokens: 69.6 us on 20 CUs
//    against 84.6 us split over 80 workgroups);
//  - dX and dW launched alone at 1024-4096 tokens: 20 stages per piece
//    chooses the fastest or a near-fastest option at every shape (e.g. dX
//    at 4096 x 6912 -> 2560 whole, 144 us against 175 us split; at
//    4096 x 2560 -> 6912 split, 151 us against 163 us whole).
constexpr int kFwdPieceCost = 48;
constexpr int kBwdPieceCost = 20;

static GemmShape shape_of(GemmKind kind, int64_t M, int64_t N, int64_t K) {
  const int64_t Kp = k_pad(K);
  switch (kind) {
    case GemmKind::kFwd:
      return {(N + kBI - 1) / kBI, (M + kBJ - 1) / kBJ, (Kp + kStageBytes - 1) / kStageBytes, kFwdPieceCost};
    // a split piece costs the bf16 forward about 20 of its stages (measured
    // at 4096x2560->6912: whole tiles in two rounds 171 us, split over 256
    // workgroups 185 us)
    case GemmKind::kTtqFwd: return {(N + kBI - 1) / kBI, (M + kBJ - 1) / kBJ, (Kp + kRed16 - 1) / kRed16, 20};
    case GemmKind::kBwdDx:
      return {(K + kBI - 1) / kBI, (M + kBJ - 1) / kBJ, (N + kRed16 - 1) / kRed16, kBwdPieceCost};
    case GemmKind::kBwdDw: case GemmKind::kBwdPair: case GemmKind::kTtqBwd: case GemmKind::kTtqBwdPadded: break;
  }
  return {(K + kBI - 1) / kBI, (N + kBJ - 1) / kBJ, (M + kRed16 - 1) / kRed16, kBwdPieceCost};
}

// Workgroups of a split launch, or 0 for one whole tile per workgroup.
// A split pays when T tiles leave the last round of whole tiles on `cus`
// CUs partly idle; it spreads the T*S stages evenly over at most `cus`
// workgroups and about 4 pieces per tile. The split_ctas test knob
// (bitnet_set_test_knobs) forces a split over that many workgroups, or with
// a negative value whole tiles.
static int split_pays(const GemmShape& g, int cus) {
  const int64_t T = g.tiles(), S = g.nstages, W = T * S;
  if (W < 2 || cus < 1) return 0;
  const int64_t G = (int64_t)cus < 4 * T ? (int64_t)cus : 4 * T;
  const int64_t whole = (T + cus - 1) / cus * S;
  const int64_t split = (W + G - 1) / G + g.overhead;
  return split < whole ? (int)G : 0;
}
static int split_grid(const GemmShape& g, int cus) {
  const int f = test_knobs().split_ctas.load(std::memory_order_relaxed);
  if (f < 0) return 0;
  if (f > 0) {
    const int64_t W = g.tiles() * g.nstages;
    const int64_t G = f < kMaxGrid ? f : kMaxGrid;
    return (int)(G < W ? G : W);
  }
  return split_pays(g, cus);
}

// Split-launch workspace: the tile counters [T][2] (8 bytes each, rounded
// up to 256 bytes), then the partial tiles [partial_slots(T, G)].
static size_t split_control_bytes(const GemmShape& g) { return ((size_t)g.tiles() * 16 + 255) / 256 * 256; }
static size_t split_workspace(const GemmShape& g, int grid) {
  if (grid == 0) return 0;
  return split_control_bytes(g) + (size_t)partial_slots(g.tiles(), grid) * kPartialBytes;
}

// dW's x_hat buffer at the start of its workspace.
static size_t xhat_bytes(int64_t M, int64_t K) { return ((size_t)M * k_pad(K) * 2 + 255) / 256 * 256; }
static int64_t n_pad64(int64_t N) { return (N + 63) / 64 * 64; }
static size_t wt_bytes(int64_t N, int64_t K) { return ((size_t)k_pad(K) * (n_pad64(N) / 2) + 255) / 256 * 256; }


// The split grid a launch given ws_bytes of split workspace runs: the grid
// split_grid() chooses, or the largest smaller one whose workspace fits and
// whose split still beats whole tiles on `cus` CUs (a grid forced by the
// knob: the largest that fits); 0: whole tiles.
static int fit_split(const GemmShape& g, int cus, size_t ws_bytes) {
  const int want = split_grid(g, cus);
  if (want == 0 || split_workspace(g, want) <= ws_bytes) return want;
  const bool forced = test_knobs().split_ctas.load(std::memory_order_relaxed) > 0;
  const int64_t T = g.tiles(), S = g.nstages, W = T * S;
  const int64_t whole = (T + cus - 1) / cus * S;
  for (int G = want - 1; G >= 2; --G) {
    if (split_workspace(g, G) > ws_bytes) continue;
    if (forced) return G;
    return (W + G - 1) / G + g.overhead < whole ? G : 0;
  }
  return 0;
}

static int device_cus() {
  static int cached[64] = {0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return kMaxGrid;
  if (cached[dev] == 0) {
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 1) n = kMaxGrid;
    cached[dev] = n < kMaxGrid ? n : kMaxGrid;
  }
  return cached[dev];
}

// Cost model of one product on G workgroups, in dX stage times (measured
// at 4096x2560->6912): a tile's pipeline fill and epilogue cost about 5.4
// stages. Per product, the cost of a stage and of each piece of a split
// range (fill, partial exchange, epilogue): dX 1.0 and 10 stages; dW 1.07
// and 21 (dW's pieces exchange more: measured at 4096x2560->6912 and
// 4096x6912->2560, a pair launch whose dW splits over 128 CUs takes
// 325-370 us where dW in whole tiles on 136 CUs takes 260-340 us, which 10
// stages per piece did not predict). Whole tiles taken in turn cost
// ceil(T/G) tiles; a split costs W/G stages plus its pieces (about
// W/(G*S) + 1 per workgroup).
constexpr double kTileCost = 5.4;
struct ProductCosts {
  double stage, piece;
};
constexpr ProductCosts kDxCosts{1.0, 10.0}, kDwCosts{1.07, 21.0};
struct PairCost {
  double t;
  bool split;
};
static PairCost product_cost(const GemmShape& g, int64_t G, const ProductCosts& c) {
  const double T = (double)g.tiles(), S = (double)g.nstages, W = T * S;
  const double whole = std::ceil(T / (double)G) * (S * c.stage + kTileCost);
  const int64_t Gs = G < 4 * g.tiles() ? G : 4 * g.tiles();
  const double split = W / (double)Gs * c.stage + (W / ((double)Gs * S) + 1.0) * c.piece;
  return split < whole ? PairCost{split, true} : PairCost{whole, false};
}

// The 8-workgroup columns (of kt) that run dX in a pair launch: the k1 that
// minimizes the slower product's modelled cost; 0: no pair launch (the
// split_ctas knob is set, or too few CUs). The pair_cols knob overrides k1.
static int pair_columns(const GemmShape& g1, const GemmShape& g2, int cus, int* kt, const ProductCosts& c1,
                        const ProductCosts& c2) {
  if (test_knobs().split_ctas.load(std::memory_order_relaxed) != 0) return 0;
  *kt = (cus < kMaxGrid ? cus : kMaxGrid) / 8;
  if (*kt < 2) return 0;
  const int f = test_knobs().pair_cols.load(std::memory_order_relaxed);
  if (f >= 1 && f < *kt) return f;
  int best = 1;
  double best_t = 1e300;
  for (int k1 = 1; k1 < *kt; ++k1) {
    const double t = std::max(product_cost(g1, 8 * k1, c1).t, product_cost(g2, 8 * (*kt - k1), c2).t);
    if (t < best_t) {
      best_t = t;
      best = k1;
    }
  }
  return best;
}

static SplitPlan split_plan(const GemmShape& g, int grid, void* ws) {
  SplitPlan plan{};
  plan.total = g.tiles() * g.nstages;
  plan.tiles_i = (int)g.tiles_i;
  plan.nstages = (int)g.nstages;
  plan.grid = grid;
  plan.spin_limit = test_knobs().spin_limit.load(std::memory_order_relaxed);
  plan.gen = next_launch_tag();
  plan.nslots = partial_slots(g.tiles(), grid);
  plan.counters = static_cast<uint64_t*>(ws);
  plan.partials = reinterpret_cast<uint4*>(static_cast<char*>(ws) + split_control_bytes(g));
  return plan;
}

// Whole tiles taken in turn by `grid` workgroups (no split).
static SplitPlan whole_plan(const GemmShape& g, int grid) {
  SplitPlan plan{};
  plan.total = g.tiles() * g.nstages;
  plan.tiles_i = (int)g.tiles_i;
  plan.nstages = (int)g.nstages;
  plan.grid = grid;
  return plan;
}

template <class MT, int MAP, class PL, class QL, class EP>
static hipError_t run_gemm(const PL& pl, const QL& ql, const EP& ep, const GemmShape& g, void* ws,
                           size_t ws_bytes, hipStream_t stream) {
  const int grid = ws == nullptr ? 0 : fit_split(g, device_cus(), ws_bytes);
  const SplitPlan plan = grid > 0 ? split_plan(g, grid, ws) : whole_plan(g, (int)g.tiles());
  gemm_kernel<MT, MAP, PL, QL, EP><<<plan.grid, kThreads, 0, stream>>>(pl, ql, ep, plan);
  return hipGetLastError();
}

// Two products in one gemm_pair_kernel launch, each on its own share of the
// CUs (pair_columns), each splitting its tiles only when the cost model says
// that beats whole tiles taken in turn on its share (stage costs c1, c2).
// k1 == 0: no pair launch on this device. s1, s2: split workspace bytes.
struct PairPlan {
  int kt = 0, k1 = 0, G1 = 0, G2 = 0;
  bool sk1 = false, sk2 = false;
  size_t s1 = 0, s2 = 0;
};
static PairPlan plan_pair(const GemmShape& g1, const GemmShape& g2, int cus, const ProductCosts& c1,
                          const ProductCosts& c2) {
  PairPlan pp;
  pp.k1 = pair_columns(g1, g2, cus, &pp.kt, c1, c2);
  if (pp.k1 == 0) return pp;
  // every workgroup of a split needs a non-empty range, and more than about
  // 4 pieces per tile do not pay
  const auto cap = [](const GemmShape& g, int64_t G) {
    const int64_t W = g.tiles() * g.nstages, P = 4 * g.tiles();
    return (int)(G < W ? (G < P ? G : P) : (W < P ? W : P));
  };
  const int64_t share1 = 8 * pp.k1, share2 = 8 * (pp.kt - pp.k1);
  pp.sk1 = product_cost(g1, share1, c1).split;
  pp.sk2 = product_cost(g2, share2, c2).split;
  pp.G1 = pp.sk1 ? cap(g1, share1) : (int)(g1.tiles() < share1 ? g1.tiles() : share1);
  pp.G2 = pp.sk2 ? cap(g2, share2) : (int)(g2.tiles() < share2 ? g2.tiles() : share2);
  pp.s1 = pp.sk1 ? split_workspace(g1, pp.G1) : 0;
  pp.s2 = pp.sk2 ? split_workspace(g2, pp.G2) : 0;
  return pp;
}

// The pair launch of plan_pair on ws (pp.s1 + pp.s2 bytes);
// hipErrorNotSupported (nothing launched): the device or the workspace does
// not allow it.
template <int MAP1, int MAP2, class PL1, class QL1, class EP1, class PL2, class QL2, class EP2>
static hipError_t run_pair(const PL1& p1, const QL1& q1, const EP1& e1, const GemmShape& g1,
                           const ProductCosts& c1, const PL2& p2, const QL2& q2, const EP2& e2, const GemmShape& g2,
                           const ProductCosts& c2, char* ws, size_t ws_bytes, hipStream_t stream) {
  const PairPlan pp = plan_pair(g1, g2, device_cus(), c1, c2);
  if (pp.k1 == 0 || ws_bytes < pp.s1 + pp.s2) return hipErrorNotSupported;
  const SplitPlan plan1 = pp.sk1 ? split_plan(g1, pp.G1, ws) : whole_plan(g1, pp.G1);
  const SplitPlan plan2 = pp.sk2 ? split_plan(g2, pp.G2, ws + pp.s1) : whole_plan(g2, pp.G2);
  gemm_pair_kernel<MfmaBf16, MAP1, PL1, QL1, EP1, MAP2, PL2, QL2, EP2>
      <<<8 * pp.kt, kThreads, 0, stream>>>(p1, q1, e1, plan1, p2, q2, e2, plan2, pp.k1);
  return hipGetLastError();
}

}  // namespace bitnet
