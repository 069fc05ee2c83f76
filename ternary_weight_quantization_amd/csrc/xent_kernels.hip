// A linear layer with softmax cross entropy at the end of a language model,
// in pieces of the vocabulary, without keeping the logits.
//
//   z[t][v]  = sum_d h[t][d] W[v][d]
//   lse[t]   = log sum_v exp z[t][v],   loss[t] = lse[t] - z[t][target[t]]
//   G[t][v]  = c[t] (exp(z[t][v] - lse[t]) - [v == target[t]])
//   dh       = G W,   dW = G^T h
//
// (c[t]: the loss' gradient with respect to loss[t]. Under a sum or a mean it
// is one number c for all rows, and G is computed without it and the products
// are multiplied by it in fp32: the target's element is then p - 1, which
// bf16 holds to within p, where c (p - 1) would be rounded by the same 2^-9
// in every row.) The three products are
// bf16 MFMA GEMMs with fp32 sums, so the whole is MFMA bound for many tokens:
// 2TVD operations for the loss, 4TVD for the gradients and 2TVD for the
// logits computed again, because keeping them would take 4TV bytes (2 GB at
// 4096 x 128256). For few tokens the loss is bound by reading W once.
//
// With tiles and in the backward rows whose target is ignore_index are taken
// out first: the rows that count are gathered to the front (hc), so that an
// ignored row costs nothing there. The number n of rows that count stays on the
// device; tiles past it leave at once. Where all T rows count and need no
// padding, nothing is copied and h is read in place. The few-token loss gathers
// nothing: an ignored row's logits are computed and not used. Either way
// nothing an ignored row holds, NaN included, reaches a sum.
//
// Many tokens:
//   gather   rows, targets, (backward) lse and c of the rows that count
//   logits   forward: one 256 x 256 tile of z per workgroup, reduced in the
//            epilogue to a maximum and a sum of exponentials per token and
//            128 columns, and the target's logit; nothing else is written
//   combine  lse and the loss per row from those pairs; then their sum
//   logits   backward: the same tiles again, G rounded to bf16 for one piece
//            of the vocabulary at a time (small enough to stay in the last
//            level cache until it is read)
//   grads    both products of a piece in one launch: dh's tiles, split over
//            the piece's columns where they are few, accumulate in fp32
//            slabs; dW's tiles are final
//   dh       the slabs summed in a fixed order, rounded once, scattered back
//            to the rows; ignored rows get zeros
// No atomics: the same inputs give the same bits.
//
// Measured in us: 4096 tokens, 128256 columns, D = 2560: logits forward 2177
// (1235 TFLOP/s; this card's best library product alone, which writes the
// logits, takes 2024), backward logits 8 x 287, grads 8 x 537 (1252 TFLOP/s;
// the two products as library calls 377 + 393), gather 6, combine 12, dh 12.
// 1000 tokens of which 750 count, 50257 columns: 201 + 204 + 405 with 591
// tiles of logits on 256 CUs (three rounds for 2.3 of work) and dW tiles of 12
// stages. Workgroups that stay for every 256th tile and load the next one
// during the last stages of the current one were 5 % slower.

#include <algorithm>

#include "gemm_core.h"
#include "internal.h"
#include "row_io.h"

namespace bitnet {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// Control block at the start of the workspace: n, and c where it is one for
// all rows (1 otherwise).
struct XentCtl {
  int n;
  float c;
};

// ---------------------------------------------------------------------------
// Rows that count
// ---------------------------------------------------------------------------

struct XentRows {
  const uint16_t* h;       // [T][D]
  const int64_t* targets;  // [T]
  int64_t ignore;
  int T, D, Dp;            // Dp: D rounded up to 8
  int64_t V;
  XentCtl* ctl;
  uint16_t* hc;            // [T][Dp] rows that count, in order
  int* pos;                // [T] row -> index among them, -1: ignored
  int* ct;                 // [T] their targets, -1: out of range
  // backward only
  const float* lse;        // [T]
  const float* dloss;      // [1], or [T] with per_row
  int per_row, mean;
  float* lsec;             // [T] lse of the rows that count
  float* c;                // [T] what G's rows are multiplied by
};

constexpr int kGatherRows = 4;  // at a time: one for each of the block's waves

// Each block finds how many rows that count precede its own and how many
// there are by reading all targets, so that no launch or wait between blocks is
// needed: 8 T bytes out of the caches a block, 34 MB in all with 4096 tokens
// (the launch takes 6 us). `groups` of kGatherRows rows a block keep the
// blocks below 2048 and the reading linear above 8192 tokens; with the most
// that are accepted, 2^21, it is still 34 GB a launch.
template <bool BWD>
__global__ __launch_bounds__(256) void xent_gather_kernel(XentRows a, int groups) {
  __shared__ int before[4], all[4];
  const int tid = threadIdx.x;
  int t0 = blockIdx.x * groups * kGatherRows;
  int b = 0, n = 0;
#pragma unroll 8
  for (int t = tid; t < a.T; t += 256) {
    const int v = a.targets[t] != a.ignore;
    n += v;
    b += v & (t < t0);
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    b += __shfl_xor(b, off, kWave);
    n += __shfl_xor(n, off, kWave);
  }
  if ((tid & 63) == 0) {
    before[tid >> 6] = b;
    all[tid >> 6] = n;
  }
  __syncthreads();
  b = (before[0] + before[1]) + (before[2] + before[3]);
  n = (all[0] + all[1]) + (all[2] + all[3]);
  if (blockIdx.x == 0 && tid == 0) {
    a.ctl->n = n;
    if constexpr (BWD) a.ctl->c = a.per_row ? 1.0f : a.mean ? *a.dloss / (float)n : *a.dloss;
  }
  const int lane = tid & 63, wave = tid >> 6, nch = n == a.T && a.Dp == a.D ? 0 : a.Dp / 8;
  for (int end = min(a.T, t0 + groups * kGatherRows); t0 < end; t0 += kGatherRows) {
    // which of the block's rows count, in every lane of every wave
    const int tl = t0 + (lane & (kGatherRows - 1));
    const unsigned long long mask = __ballot(lane < kGatherRows && tl < a.T && a.targets[tl < a.T ? tl : 0] != a.ignore);
    const int r = wave, t = t0 + r;
    if (t < a.T && !((mask >> r) & 1)) {
      if (lane == 0) a.pos[t] = -1;
    } else if (t < a.T) {
      const int at = b + __popcll(mask & ((1ull << r) - 1));
      const int64_t target = a.targets[t];
      const bool in = target >= 0 && target < a.V;
      if (lane == 0) {
        a.pos[t] = at;
        a.ct[at] = in ? (int)target : -1;
        if constexpr (BWD) {
          const float c = a.per_row ? a.dloss[t] : 1.0f;
          a.lsec[at] = a.lse[t];
          a.c[at] = in ? c : __uint_as_float(0x7FC00000u);  // a target out of range: NaN gradients
        }
      }
      const uint16_t* src = a.h + (int64_t)t * a.D;
      uint4* dst = reinterpret_cast<uint4*>(a.hc + (int64_t)at * a.Dp);
      for (int c0 = 0; c0 < nch; c0 += 256) {
        ChunkBf16 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = a.D < 8 ? load8<true>(src, 8 * (c0 + lane + 64 * i), a.D) : load8<false>(src, 8 * (c0 + lane + 64 * i), a.D);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int ch = c0 + lane + 64 * i;
          if (a.D >= 8) settle8<false>(v[i], 8 * ch, a.D);
          if (ch < nch) dst[ch] = v[i].v;
        }
      }
    }
    b += __popcll(mask);
  }
}

// Rows of W padded to a whole number of 16-byte chunks (a width that is not a
// multiple of 8).
__global__ __launch_bounds__(256) void xent_pad_kernel(const uint16_t* __restrict__ w, int64_t rows, int D, int nch,
                                                       uint16_t* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= rows * nch) return;
  const int64_t r = i / nch;
  const int k0 = 8 * (int)(i - r * nch);
  reinterpret_cast<uint4*>(out)[i] = chunk8(w + r * D, k0, D).v;
}

// The rows that count [n][Dp]: the gathered ones, or h itself where all T
// count (`all` is hc too where h's width is padded).
struct XentHidden {
  const uint16_t* hc;
  const uint16_t* all;
  int T;
  __device__ __forceinline__ const uint16_t* rows(int n) const { return n == T ? all : hc; }
};

// ---------------------------------------------------------------------------
// Logit tiles
// ---------------------------------------------------------------------------

struct XentTiles {
  const uint16_t* w;  // [vc][ldw] rows of the piece
  int64_t ldw;
  int vc;             // valid rows
  int v0;             // the piece's first row
  int tiles_v, tiles_t, nstages;
  XentHidden h;
  int Dp;
  const XentCtl* ctl;
  const int* ct;
  // forward
  float2* part;  // [2 tiles of 128 columns][T]: maximum, sum
  int T;
  float* zt;     // [n] the target's logit
  // backward
  const float* lsec;
  const float* c;
  uint16_t* G;   // [n][ldg]
  int ldg;
};

// Tile p of tiles_v x tiles_t: groups of kGroupV rows of tiles, within a
// group v fastest, so that the workgroups that run together on an XCD share
// both their W and their h panels in its L2.
constexpr int kGroupV = 4;
__device__ __forceinline__ void xent_tile(int p, int tiles_v, int tiles_t, int& tv, int& tt) {
  const int g = p / (kGroupV * tiles_t), r = p - g * kGroupV * tiles_t;
  const int width = min(kGroupV, tiles_v - g * kGroupV);
  tt = r / width;
  tv = g * kGroupV + r - tt * width;
}

// Value e of a lane's 16 of fragment fi: row 32 fi + row_of(e, lane).
__device__ __forceinline__ int row_of(int e, int lane) { return 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3); }

typedef MfmaBf16::Acc AccTile[kFI][kFJ];

// What the epilogues need of a tile's 256 tokens, staged in LDS before the main
// loop: the target's row within the tile (out of 0..255 where it is elsewhere)
// and, backward, lse and c.
struct XentTokens {
  int target[kBJ];
  float lse[kBJ], c[kBJ];
};

// Rows past the piece count as logits of -inf: 2^-inf is 0.
__device__ __forceinline__ void xent_mask(AccTile& acc, int rows, int lane) {
  if (rows >= kWTI) return;  // uniform
#pragma unroll
  for (int fi = 0; fi < kFI; ++fi)
#pragma unroll
    for (int fj = 0; fj < kFJ; ++fj)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (32 * fi + row_of(e, lane) >= rows) acc[fi][fj][e] = -INFINITY;
}

// Forward epilogue of a wave's 128 columns (from i0 of the piece) x 128 tokens
// (from j0; the tile's token qj): the maximum m of z and the sum of e^(z - m)
// per token, over both lanes that hold a token. The difference is taken before
// it is scaled for the base 2: it is exact near the maximum and 0 there, so
// that the sum is at least 1 and its logarithm at least 0 (a rounded m log2(e)
// as the reference left its own rounding in the loss, 1e-4 at logits of 1500).
__device__ __forceinline__ void xent_stats(const XentTiles& a, const XentTokens& tok, AccTile& acc, int i0, int j0,
                                           int qj, int n, int lane) {
  xent_mask(acc, a.vc - i0, lane);
#pragma unroll
  for (int fj = 0; fj < kFJ; ++fj) {
    const int j = j0 + 32 * fj + (lane & 31);
    const int t = tok.target[qj + 32 * fj + (lane & 31)] - i0 % kBI;  // the target's row among these 128?
    float m = -INFINITY;
#pragma unroll
    for (int fi = 0; fi < kFI; ++fi)
#pragma unroll
      for (int e = 0; e < 16; ++e) m = fmaxf(m, acc[fi][fj][e]);
    m = fmaxf(m, __shfl_xor(m, 32, kWave));
    const float ref = m == -INFINITY ? 0.0f : m;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // four chains
#pragma unroll
    for (int fi = 0; fi < kFI; ++fi)
#pragma unroll
      for (int e = 0; e < 16; ++e) s[e & 3] += __builtin_amdgcn_exp2f((acc[fi][fj][e] - ref) * kLog2e);
    float sum = (s[0] + s[1]) + (s[2] + s[3]);
    sum += __shfl_xor(sum, 32, kWave);
    if (j < n && lane < 32) a.part[(int64_t)((a.v0 + i0) / kWTI) * a.T + j] = make_float2(m, sum);
    if (t >= 0 && t < kWTI && j < n && ((t >> 2) & 1) == (lane >> 5)) {  // rare
#pragma unroll
      for (int fi = 0; fi < kFI; ++fi)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (t == 32 * fi + row_of(e, lane)) a.zt[j] = acc[fi][fj][e];
    }
  }
}

// Backward epilogue: G of the tile, rounded to bf16 (the operand of both
// products; the rounding, 2^-9 of each value, is the size of the outputs'
// own), zeros in the columns past the piece. As in the forward the difference
// of z and lse is taken before it is scaled, so that p of a target that takes
// nearly all is off by lse's one rounding.
__device__ __forceinline__ void xent_g(const XentTiles& a, const XentTokens& tok, AccTile& acc, int i0, int j0, int qj,
                                       int n, int lane, char* wlds) {
  xent_mask(acc, a.vc - i0, lane);
#pragma unroll
  for (int fj = 0; fj < kFJ; ++fj) {
    const int at = qj + 32 * fj + (lane & 31);
    const int t = tok.target[at] - i0 % kBI;
    const float c = tok.c[at], l = tok.lse[at];
#pragma unroll
    for (int fi = 0; fi < kFI; ++fi)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __builtin_amdgcn_exp2f((acc[fi][fj][4 * g + e] - l) * kLog2e) * c;
        EpStage<2>::put(wlds, lane, fi, g, make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])));
      }
    if (t >= 0 && t < kWTI && ((t >> 2) & 1) == (lane >> 5)) {  // rare: the target is one of this lane's rows
      float z = 0.0f;
#pragma unroll
      for (int fi = 0; fi < kFI; ++fi)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (t == 32 * fi + row_of(e, lane)) z = acc[fi][fj][e];
      const float v = (__builtin_amdgcn_exp2f((z - l) * kLog2e) - 1.0f) * c;
      const uint16_t bits = f32_to_bf16_bits(v);
      memcpy(wlds + (lane & 31) * EpStage<2>::kPitch + 2 * t, &bits, 2);
    }
    EpStage<2>::drain(wlds, reinterpret_cast<char*>(a.G), a.ldg, n, i0, j0 + 32 * fj, lane);
  }
}

typedef CopyLoader<2, true, 1> XentW;
typedef CopyLoader<2, true, 5> XentH;

template <bool BWD>
__global__ __launch_bounds__(kThreads, 1) void xent_logits_kernel(XentTiles a) {
  typedef SmemLayout<XentW, XentH> L;
  __shared__ __attribute__((aligned(16))) char smem[L::kBytes];
  static_assert(4 * EpStage<2>::kWaveBytes <= L::kBytes, "the epilogue's staging fits the stage buffers");
  __shared__ XentTokens tok;
  const int n = a.ctl->n;
  int tv, tt;
  xent_tile(cta_order(blockIdx.x, gridDim.x), a.tiles_v, a.tiles_t, tv, tt);
  const int i0 = tv * kBI, j0 = tt * kBJ;
  if (j0 >= n) return;
  {  // read after the main loop's barriers
    const int t = threadIdx.x, j = j0 + t;
    static_assert(kThreads == kBJ, "a thread a token");
    // a target out of range (-1) or in another piece is in no tile
    const int r = j < n ? a.ct[j] : -1;
    tok.target[t] = r >= a.v0 + i0 && r < a.v0 + min(a.vc, i0 + kBI) ? r - a.v0 - i0 : -kBI;
    if constexpr (BWD) {
      tok.lse[t] = j < n ? a.lsec[j] : 0.0f;
      tok.c[t] = j < n ? a.c[j] : 0.0f;
    }
  }
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int pi = (wave % kWavesI) * kWTI, qj = (wave / kWavesI) * kWTJ;
  const XentW pl{reinterpret_cast<const char*>(a.w), 2 * a.ldw, a.vc, 2 * (int64_t)a.Dp};
  const XentH ql{reinterpret_cast<const char*>(a.h.rows(n)), 2 * (int64_t)a.Dp, n, 2 * (int64_t)a.Dp};
  AccTile acc;
#pragma unroll
  for (int fi = 0; fi < kFI; ++fi)
#pragma unroll
    for (int fj = 0; fj < kFJ; ++fj) zero_acc(acc[fi][fj]);
  run_stages<MfmaBf16, 1>(pl, ql, smem, acc, i0, j0, 0, a.nstages, pi, qj, lane, nullptr, 0);
  if constexpr (BWD) xent_g(a, tok, acc, i0 + pi, j0 + qj, qj, n, lane, smem + wave * EpStage<2>::kWaveBytes);
  else xent_stats(a, tok, acc, i0 + pi, j0 + qj, qj, n, lane);
}

// ---------------------------------------------------------------------------
// Loss from the partial statistics
// ---------------------------------------------------------------------------

// pos == NULL: the rows are the tokens themselves (none gathered).
struct XentLoss {
  const float2* part;  // [parts][T]
  int parts, T;
  const float* zt;
  const int* pos;
  const int64_t* targets;
  int64_t ignore, V;
  float* lse;
  float* loss;
  // one workgroup (up to kLossTokens tokens) also writes their sum or mean;
  // NULL: not wanted, or xent_reduce_kernel does
  float* total;
  int mean;
};

// (m, s) += (m1, s1): sums of exponentials over e^m. One that is empty, or of logits
// that are all -inf, has m = -inf and s = 0, or NaN if a logit is.
__device__ __forceinline__ void xent_join(float& m, float& s, float m1, float s1) {
  const float top = fmaxf(m, m1);
  if (top == -INFINITY) {
    s += s1;
    return;
  }
  s = s * __builtin_amdgcn_exp2f((m - top) * kLog2e) + s1 * __builtin_amdgcn_exp2f((m1 - top) * kLog2e);
  m = top;
}

// A block takes 16 tokens (a part's 16 pairs are one 128-byte line) and 64
// groups of parts: 4 groups in a wave, joined by shuffles, then 16 waves. Up to
// 16 tokens it also reduces their losses, without a launch for that.
constexpr int kLossTokens = 16;
__global__ __launch_bounds__(1024) void xent_combine_kernel(XentLoss a) {
  __shared__ float sm[16][kLossTokens], ss[16][kLossTokens];
  const int l = threadIdx.x % kLossTokens, g = threadIdx.x / kLossTokens;
  const int t = blockIdx.x * kLossTokens + l;
  const int64_t target = t < a.T ? a.targets[t] : a.ignore;
  const bool counts = target != a.ignore;
  const int at = !counts ? -1 : a.pos ? a.pos[t] : t;
  float m = -INFINITY, s = 0.0f;
  if (at >= 0) {
    const float2* src = a.part + at;
    int p = g;
    for (; p + 192 < a.parts; p += 256) {  // four loads in flight
      const float2 v0 = src[(int64_t)p * a.T], v1 = src[(int64_t)(p + 64) * a.T], v2 = src[(int64_t)(p + 128) * a.T],
                   v3 = src[(int64_t)(p + 192) * a.T];
      xent_join(m, s, v0.x, v0.y);
      xent_join(m, s, v1.x, v1.y);
      xent_join(m, s, v2.x, v2.y);
      xent_join(m, s, v3.x, v3.y);
    }
    for (; p < a.parts; p += 64) {
      const float2 v = src[(int64_t)p * a.T];
      xent_join(m, s, v.x, v.y);
    }
  }
#pragma unroll
  for (int off = 16; off <= 32; off <<= 1) {
    const float m1 = __shfl_xor(m, off, kWave), s1 = __shfl_xor(s, off, kWave);
    xent_join(m, s, m1, s1);
  }
  if ((threadIdx.x & 63) < kLossTokens) {
    sm[threadIdx.x >> 6][l] = m;
    ss[threadIdx.x >> 6][l] = s;
  }
  __syncthreads();
  if (threadIdx.x >= kLossTokens) return;
  float loss = 0.0f, lse = 0.0f;
  if (counts) {
#pragma unroll
    for (int w = 1; w < 16; ++w) xent_join(m, s, sm[w][l], ss[w][l]);
    // the loss takes the difference of the two logits, not that of the rounded
    // lse: 0 for a target that is all of the sum
    const float log_s = __builtin_amdgcn_logf(s);  // v_log_f32: base 2
    lse = fmaf(log_s, kLn2, m);
    loss = target < 0 || target >= a.V ? __uint_as_float(0x7FC00000u) : fmaf(log_s, kLn2, m - a.zt[at]);
  }
  if (t < a.T) {
    a.lse[t] = lse;
    a.loss[t] = loss;
  }
  if (a.total == nullptr) return;
  double v = (double)loss;
  int n = counts ? 1 : 0;
#pragma unroll
  for (int off = 1; off < kLossTokens; off <<= 1) {
    v += __shfl_xor(v, off, kWave);
    n += __shfl_xor(n, off, kWave);
  }
  if (l == 0) *a.total = (float)(a.mean && n > 0 ? v / (double)n : v);
}

// The rows' sum or mean over the rows that count (0 where none does), in fp64
// in a fixed order.
__global__ __launch_bounds__(1024) void xent_reduce_kernel(const float* __restrict__ loss,
                                                           const int64_t* __restrict__ targets, int64_t ignore, int T,
                                                           int mean, float* __restrict__ out) {
  __shared__ double part[16];
  __shared__ int cnt[16];
  double v = 0.0;
  int n = 0;
  for (int t = threadIdx.x; t < T; t += 1024) {
    v += (double)loss[t];
    n += targets[t] != ignore;
  }
  v = wave_sum_f64(v);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) n += __shfl_xor(n, off, kWave);
  if ((threadIdx.x & 63) == 0) {
    part[threadIdx.x >> 6] = v;
    cnt[threadIdx.x >> 6] = n;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  v = 0.0;
  n = 0;
  for (int w = 0; w < 16; ++w) {
    v += part[w];
    n += cnt[w];
  }
  *out = (float)(mean && n > 0 ? v / (double)n : v);
}

// ---------------------------------------------------------------------------
// Few tokens, or few tiles: a workgroup takes 64 tokens (or all, in groups of
// 16) and 64 or 128 rows of W, its waves every 4th stage of 64 columns; with up
// to 64 tokens that is one pass over W. Both operands go from memory straight
// to the fragments of v_mfma_f32_16x16x32_bf16, the waves' sums meet in LDS, and
// each group of 16 tokens reduces its column of the tile to one pair per
// token (forward) or writes its columns of G (backward).
//
// A fragment's lane l holds 8 values of row l % 16 at reduction chunk l / 16,
// so a load covers 64 contiguous bytes of 16 rows and the stage's second load
// the rest of those 128-byte lines. (With 32 x 32 fragments a load takes 32
// bytes of 32 rows; the other three loads of a line then often found it gone
// from L1: 36 us at 16 x 2560 against 32000 columns, where this takes 28 us,
// 5.9 TB/s of W, and slower the more loads were in flight.) Measured there for
// the whole loss: 64 rows and 4 waves a workgroup 39.0 us, 8 waves 40.1 us, 16
// waves 44.4 us, 32 rows 43.3 us; one launch in which the last workgroup joins
// the pairs 58-78 us (arrivals at one address run 25 ns apart). (These with
// rounded references in base 2; the exact differences take 1 us more in the
// join: 40.0 us.)
// ---------------------------------------------------------------------------

constexpr int kFewWaves = 4;
constexpr int kFewGroup = 64;  // tokens a workgroup takes at most

// The choice between this way and 256 x 256 tiles. At most 512 workgroups of
// 64 tokens x 64 rows (two a CU): this way, where tiles would leave most CUs
// idle. More: this way up to 64 tokens, up to 48 where the tiles of W's rows
// fill most of the CUs. The loss in us, this way / by tiles, at D = 2560: 100
// tokens 26 / 57 against 8000 columns and 67 / 61 against 20000, 256 tokens 37 /
// 58 against 8000 and 67 / 59 against 16000, 1000 tokens 26 / 60 against 1000 and
// 67 / 61 against 4000; 48 tokens 44 / 67 against 32000, 155 / 152 against 128256;
// 64 tokens 52 / 67 against 32000, 97 / 84 against 64000, 187 / 152 against
// 128256. The rule does not look at D. Repeated on one W at D = 512, 2560 and
// 8192, this way / by tiles: 16 tokens against 32000 columns 14 / 26, 33 / 58 and
// 117 / 168, 256 against 8000 15 / 27, 37 / 59 and 94 / 146, 1000 against 2000
// 15 / 29, 37 / 61 and 94 / 148; but with 48 tokens against 128256 columns 45 /
// 49, 157 / 149 and 456 / 402, and with 64 against 57300 26 / 30, 92 / 70 and
// 247 / 197: there tiles are faster from D = 2560 on and are not taken. The
// no_skinny test knob keeps to the tiles.
static int64_t few_groups(int64_t T) { return (T + kFewGroup - 1) / kFewGroup; }
static bool few_tokens(int64_t T, int64_t V) {
  if (test_knobs().no_skinny.load(std::memory_order_relaxed) != 0) return false;
  return T <= (V < 224 * kBI ? 64 : 48) || few_groups(T) * ((V + 63) / 64) <= 512;
}

struct XentFew {
  const uint16_t* w;  // [V][D] (backward: a piece's rows, D a multiple of 8)
  int64_t V;
  int D;
  XentHidden h;  // [T][D] (backward: the rows that count)
  int T, groups;  // of kFewGroup tokens
  // forward
  const int64_t* targets;
  float2* part;  // [tiles][T]
  float* zt;     // [T]
  // backward: G for the piece that starts at column v0
  const XentCtl* ctl;
  const int* ct;
  const float* lsec;
  const float* c;
  int v0;
  uint16_t* G;
  int ldg;
};

typedef float f32x4_t __attribute__((ext_vector_type(4)));

// TT groups of 16 tokens, FR fragments of 16 rows a tile. ODD: rows that are not
// whole 16-byte chunks (D >= 8), read where they are by unaligned loads: rows
// past the end repeat the last one, whose results are not used (16 x 2555
// against 32000 columns 79 us, 122 us with W copied to padded rows first; 5 x
// 403 against 7493 12.3 / 29.5).
template <bool BWD, bool ODD, int TT, int FR>
__global__ __launch_bounds__(kWave * kFewWaves) void xent_few_kernel(XentFew a) {
  constexpr int W = kFewWaves, ROWS = 16 * FR;
  __shared__ f32x4_t red[W][TT][FR][kWave];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  // the token groups of a tile of W run next to each other on an XCD
  const int b = a.groups == 1 ? blockIdx.x : cta_order(blockIdx.x, gridDim.x);
  const int tile = b / a.groups, t0 = (b - tile * a.groups) * kFewGroup;
  const int64_t v0 = (int64_t)tile * ROWS;
  const int D = a.D, q = lane >> 4;
  const int rows = (int)(a.V - v0 < ROWS ? a.V - v0 : ROWS);
  const rsrc_t rw = make_rsrc(a.w + v0 * D, (uint32_t)(rows * D * 2));
  const int n = BWD ? a.ctl->n : a.T;
  if (t0 >= n) return;
  const rsrc_t rh = make_rsrc(a.h.rows(n) + (int64_t)t0 * D, (uint32_t)(min(n - t0, kFewGroup) * D * 2));
  const uint32_t row = (uint32_t)((lane & 15) * D * 2);  // rows past the end read as zeros
  f32x4_t acc[TT][FR];
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int f = 0; f < FR; ++f) acc[t][f] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int stages = (D + 63) / 64;
  uint4 pw[FR][2], ph[TT][2];
  const auto load = [&](int s) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int k = 64 * s + 32 * c + 8 * q;
      if constexpr (ODD) {
#pragma unroll
        for (int f = 0; f < FR; ++f)
          pw[f][c] = load8<false>(a.w + v0 * D + min(16 * f + (lane & 15), rows - 1) * D, k, D).v;
#pragma unroll
        for (int t = 0; t < TT; ++t)
          ph[t][c] = load8<false>(a.h.rows(n) + ((int64_t)t0 + min(16 * t + (lane & 15), n - t0 - 1)) * D, k, D).v;
        continue;
      }
      const uint32_t off = k < D ? row + 2 * k : kOob;  // columns past D: an out-of-range offset
#pragma unroll
      for (int f = 0; f < FR; ++f) pw[f][c] = buf_load16(rw, off + (uint32_t)(32 * f * D));
#pragma unroll
      for (int t = 0; t < TT; ++t) ph[t][c] = buf_load16(rh, off + (uint32_t)(32 * t * D));
    }
  };
  load(wave);
  for (int s = wave; s < stages; s += W) {
    uint4 cw[FR][2], ch[TT][2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int f = 0; f < FR; ++f) cw[f][c] = pw[f][c];
#pragma unroll
      for (int t = 0; t < TT; ++t) ch[t][c] = ph[t][c];
      if constexpr (ODD) {
        const int k = 64 * s + 32 * c + 8 * q;
        const auto settle = [&](uint4& v) {
          ChunkBf16 x{v};
          settle8<false>(x, k, D);
          v = x.v;
        };
#pragma unroll
        for (int f = 0; f < FR; ++f) settle(cw[f][c]);
#pragma unroll
        for (int t = 0; t < TT; ++t) settle(ch[t][c]);
      }
    }
    load(s + W);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int f = 0; f < FR; ++f)
#pragma unroll
        for (int t = 0; t < TT; ++t)
          acc[t][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(MfmaBf16::Frag, cw[f][c]),
                                                              __builtin_bit_cast(MfmaBf16::Frag, ch[t][c]), acc[t][f], 0,
                                                              0, 0);
  }
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int f = 0; f < FR; ++f) red[wave][t][f][lane] = acc[t][f];
  __syncthreads();
  if (wave >= TT) return;
  // lane l: token l % 16 of the wave's group, rows 16 f + 4 (l / 16) + e
  const int t = t0 + 16 * wave + (lane & 15);
  f32x4_t z[FR];
#pragma unroll
  for (int f = 0; f < FR; ++f) {
    z[f] = red[0][wave][f][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) z[f] += red[w][wave][f][lane];
  }
  if constexpr (BWD) {  // G, zeros in the rows past the piece that G's pitch holds
    if (t >= n) return;
    const float c = a.c[t], l = a.lsec[t];
    const int r = a.ct[t] - a.v0 - (int)v0;
#pragma unroll
    for (int f = 0; f < FR; ++f) {
      float g[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 16 * f + 4 * q + e;
        const float p = __builtin_amdgcn_exp2f((z[f][e] - l) * kLog2e);
        g[e] = i < rows ? (i == r ? p - 1.0f : p) * c : 0.0f;
      }
      if (v0 + 16 * f + 4 * q < a.ldg)
        *reinterpret_cast<uint2*>(a.G + (int64_t)t * a.ldg + v0 + 16 * f + 4 * q) =
            make_uint2(pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]));
    }
    return;
  }
  float top = -INFINITY;
#pragma unroll
  for (int f = 0; f < FR; ++f)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (16 * f + 4 * q + e < rows) top = fmaxf(top, z[f][e]);
  top = fmaxf(top, __shfl_xor(top, 16, kWave));
  top = fmaxf(top, __shfl_xor(top, 32, kWave));
  const float ref = top == -INFINITY ? 0.0f : top;
  float s = 0.0f;
#pragma unroll
  for (int f = 0; f < FR; ++f)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float p = __builtin_amdgcn_exp2f((z[f][e] - ref) * kLog2e);
      if (16 * f + 4 * q + e < rows) s += p;
    }
  s += __shfl_xor(s, 16, kWave);
  s += __shfl_xor(s, 32, kWave);
  if (t >= a.T) return;
  if (q == 0) a.part[(int64_t)tile * a.T + t] = make_float2(top, s);
  const int64_t r = a.targets[t] - v0;
#pragma unroll
  for (int f = 0; f < FR; ++f)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (r == 16 * f + 4 * q + e && r < rows) a.zt[t] = z[f][e];
}

// Rows of W a workgroup takes: with more than 16 tokens h's fragments are as
// many bytes as W's, and 128 rows share them where that leaves enough
// workgroups (all groups of tokens counted). Measured at D = 2560, 128 against 64 rows: 32 tokens 41.5 / 46.0
// us against 32000 columns and 147 / 168 against 128256, but 29.7 / 20.5
// against 8000; 64 tokens 52.9 / 59.8 against 32000 and 35.4 / 25.6 against 8000;
// 256 tokens 37 / 44 against 8000.
static int few_rows(int64_t T, int64_t V) { return T > 16 && few_groups(T) * V >= 192 * 128 ? 128 : 64; }
static int64_t few_tiles(int64_t T, int64_t V) { return (V + few_rows(T, V) - 1) / few_rows(T, V); }

template <bool BWD, int TT, int FR>
static void few_at(const XentFew& f, hipStream_t st) {
  const unsigned grid = (unsigned)(few_tiles(f.T, f.V) * f.groups);
  if constexpr (!BWD) {  // the backward's rows are padded
    if (f.D % 8 != 0) {
      xent_few_kernel<false, true, TT, FR><<<grid, kWave * kFewWaves, 0, st>>>(f);
      return;
    }
  }
  xent_few_kernel<BWD, false, TT, FR><<<grid, kWave * kFewWaves, 0, st>>>(f);
}
template <bool BWD, int TT>
static void few_at(const XentFew& f, hipStream_t st) {
  if (few_rows(f.T, f.V) == 128) few_at<BWD, TT, TT == 1 ? 4 : 8>(f, st);
  else few_at<BWD, TT, 4>(f, st);
}
template <bool BWD>
static hipError_t launch_few(const XentFew& f, hipStream_t st) {
  if (f.T <= 16) few_at<BWD, 1>(f, st);
  else if (f.T <= 32) few_at<BWD, 2>(f, st);
  else if (f.T <= 48) few_at<BWD, 3>(f, st);
  else few_at<BWD, 4>(f, st);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Gradients of one piece
// ---------------------------------------------------------------------------

struct XentGrads {
  const uint16_t* G;  // [n][ldg]
  int ldg;
  const uint16_t* w;  // [vc][ldw]
  int64_t ldw;
  int vc;
  XentHidden h;
  int Dp, D, T;
  const XentCtl* ctl;
  // dh: tiles_d x tiles_t tiles, each split over `split` ranges of the
  // piece's stages, into slab[split][T][D]
  int tiles_d, tiles_t, split, stages_v;
  int first;  // the first piece: the slabs are written, else added to
  float* slab;
  int dh_units;
  // dW: tiles_d x tiles_v tiles
  void* dw;  // the piece's rows [vc][D]
};

// fp32 sums into out[j][i] (rows of I), added to what is there unless
// `first`.
struct AccumEpilogue {
  float* out;
  int64_t I, J;
  bool first;
  __device__ __forceinline__ void store(AccTile& acc, int i0, int j0, int lane, char* wlds) const {
    typedef EpStage<4> E;
    i0 = __builtin_amdgcn_readfirstlane(i0);
    j0 = __builtin_amdgcn_readfirstlane(j0);
#pragma unroll
    for (int fj = 0; fj < kFJ; ++fj) {
#pragma unroll
      for (int fi = 0; fi < kFI; ++fi)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          E::put(wlds, lane, fi, g,
                 make_uint4(__float_as_uint(acc[fi][fj][4 * g]), __float_as_uint(acc[fi][fj][4 * g + 1]),
                            __float_as_uint(acc[fi][fj][4 * g + 2]), __float_as_uint(acc[fi][fj][4 * g + 3])));
      const int c = lane % E::kChunks, rl = lane / E::kChunks;
      const int64_t i = i0 + 4 * c;
#pragma unroll
      for (int k = 0; k < E::kGets; ++k) {
        const uint4 v = *reinterpret_cast<const uint4*>(wlds + (rl + k * E::kRowsPerGet) * E::kPitch + 16 * c);
        const int64_t j = j0 + 32 * fj + k * E::kRowsPerGet + rl;
        if (j >= J || i >= I) continue;
        float* o = out + j * I + i;
        if (i + 4 <= I) {
          float4 f = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
          if (!first) {
            float4 p;
            memcpy(&p, o, 16);
            f.x += p.x; f.y += p.y; f.z += p.z; f.w += p.w;
          }
          memcpy(o, &f, 16);
        } else {
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (i + e < I) o[e] = (first ? 0.0f : o[e]) + __uint_as_float(u[e]);
        }
      }
    }
  }
};

// dW's tile times c, rounded once to its type.
template <bool F32>
struct DwEpilogue {
  void* out;
  int64_t I, J;
  float c;
  __device__ __forceinline__ void store(AccTile& acc, int i0, int j0, int lane, char* wlds) const {
    constexpr int EB = F32 ? 4 : 2;
#pragma unroll
    for (int fj = 0; fj < kFJ; ++fj) {
#pragma unroll
      for (int fi = 0; fi < kFI; ++fi)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float v0 = acc[fi][fj][4 * g] * c, v1 = acc[fi][fj][4 * g + 1] * c, v2 = acc[fi][fj][4 * g + 2] * c,
                      v3 = acc[fi][fj][4 * g + 3] * c;
          if constexpr (F32)
            EpStage<4>::put(wlds, lane, fi, g, make_uint4(__float_as_uint(v0), __float_as_uint(v1),
                                                          __float_as_uint(v2), __float_as_uint(v3)));
          else
            EpStage<2>::put(wlds, lane, fi, g, make_uint2(pack_bf16x2(v0, v1), pack_bf16x2(v2, v3)));
        }
      EpStage<EB>::drain(wlds, static_cast<char*>(out), I, J, i0, j0 + 32 * fj, lane);
    }
  }
};

typedef RowCopyBf16Loader<5> XentWt;      // dh's P: W as stored, read transposed
typedef CopyLoader<2, true, 1> XentG;     // dh's Q: G rows
typedef RowCopyBf16Loader<1> XentHt;      // dW's P: hc as stored
typedef RowCopyBf16Loader<5> XentGt;      // dW's Q: G as stored

template <bool F32>
__global__ __launch_bounds__(kThreads, 1) void xent_grads_kernel(XentGrads a) {
  typedef SmemLayout<XentWt, XentG> L1;
  typedef SmemLayout<XentHt, XentGt> L2;
  __shared__ __attribute__((aligned(16))) char smem[L1::kBytes > L2::kBytes ? L1::kBytes : L2::kBytes];
  static_assert(4 * EpStage<4>::kWaveBytes <= L1::kBytes, "the epilogue's staging fits the stage buffers");
  const int n = a.ctl->n;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int pi = (wave % kWavesI) * kWTI, qj = (wave / kWavesI) * kWTJ;
  char* wlds = smem + wave * EpStage<4>::kWaveBytes;
  AccTile acc;
#pragma unroll
  for (int fi = 0; fi < kFI; ++fi)
#pragma unroll
    for (int fj = 0; fj < kFJ; ++fj) zero_acc(acc[fi][fj]);
  int b = blockIdx.x;
  if (b < a.dh_units) {
    const int u = cta_order(b, a.dh_units);
    const int td = u % a.tiles_d, r = u / a.tiles_d, tt = r % a.tiles_t, sp = r / a.tiles_t;
    const int i0 = td * kBI, j0 = tt * kBJ;
    if (j0 >= n) return;
    const int s0 = (int)((int64_t)a.stages_v * sp / a.split), s1 = (int)((int64_t)a.stages_v * (sp + 1) / a.split);
    const XentWt pl{a.w, a.ldw, a.vc, a.Dp};
    const XentG ql{reinterpret_cast<const char*>(a.G), 2 * (int64_t)a.ldg, n, 2 * (int64_t)a.ldg};
    run_stages<MfmaBf16, 0>(pl, ql, smem, acc, i0, j0, s0, s1, pi, qj, lane, nullptr, 0);
    const AccumEpilogue ep{a.slab + (int64_t)sp * a.T * a.D, a.D, n, a.first != 0};
    ep.store(acc, i0 + pi, j0 + qj, lane, wlds);
    return;
  }
  b = cta_order(b - a.dh_units, gridDim.x - a.dh_units);
  const int i0 = (b % a.tiles_d) * kBI, j0 = (b / a.tiles_d) * kBJ;
  const XentHt pl{a.h.rows(n), a.Dp, n, a.Dp};
  const XentGt ql{a.G, a.ldg, n, a.ldg};
  run_stages<MfmaBf16, 0>(pl, ql, smem, acc, i0, j0, 0, (n + kRed16 - 1) / kRed16, pi, qj, lane, nullptr, 0);
  // no row counts: G and hc are empty and c may be anything
  const DwEpilogue<F32> ep{a.dw, a.D, a.vc, n > 0 ? a.ctl->c : 0.0f};
  ep.store(acc, i0 + pi, j0 + qj, lane, wlds);
}

// dh [T][D] from the slabs: their sum in order times c, rounded once, at the
// rows that count; zeros elsewhere.
__global__ __launch_bounds__(256) void xent_dh_kernel(const float* __restrict__ slab, int split,
                                                      const int* __restrict__ pos,
                                                      const XentCtl* __restrict__ ctl, int T, int D, int nch,
                                                      uint16_t* __restrict__ dh) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)T * nch) return;
  const int t = (int)(i / nch), k0 = 8 * (int)(i - (int64_t)t * nch);
  const int at = pos[t];
  float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (at >= 0) {
    for (int s = 0; s < split; ++s) {
      float f[8];
      chunk8(slab + ((int64_t)s * T + at) * D, k0, D).get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += f[e];
    }
    const float c = ctl->c;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= c;
  }
  store8(dh + (int64_t)t * D, k0, D, v);
}

// ---------------------------------------------------------------------------
// Plans, workspaces, launches
// ---------------------------------------------------------------------------

static int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// G's piece: at most this many bytes, so that the products that read it after
// it is written find it in the 256 MB last level cache.
constexpr int64_t kXentGBytes = int64_t(1) << 27;
// Rows of W copied with padding at a time.
constexpr int64_t kXentPadBytes = int64_t(1) << 28;

// Tiles of 256 columns per piece. Pieces are equal, so that each fills the
// CUs about as well as the others.
static int64_t piece_tiles(int64_t V, int64_t most_rows) {
  const int64_t tiles = (V + kBI - 1) / kBI, most = std::max<int64_t>(1, most_rows / kBI);
  const int64_t pieces = (tiles + most - 1) / most;
  return (tiles + pieces - 1) / pieces;
}
// The loaders' 32-bit offsets: (rows + 256) * pitch bytes <= 2^31.
constexpr int64_t kReach = int64_t(1) << 31;

struct XentPlan {
  int64_t Dp, tiles;    // tiles of columns per piece
  int64_t pos, ct, hc, part, zt, lsec, c, G, slab, pad, total;  // byte offsets
  int64_t ldg, split;
  bool padded;          // W's pieces are copied first
};

static XentPlan xent_plan(int64_t T, int64_t V, int64_t D, bool bwd) {
  XentPlan p{};
  p.Dp = up(D, 8);
  p.padded = p.Dp != D;
  int64_t rows = kReach / (2 * p.Dp) - 256;
  if (p.padded) rows = std::min(rows, kXentPadBytes / (2 * p.Dp));
  if (bwd) rows = std::min(rows, std::min(kXentGBytes / (2 * T), kReach / (2 * (T + 256))));
  const int64_t tt = (T + kBJ - 1) / kBJ;
  rows = std::min(rows, std::max<int64_t>(1, (int64_t(1) << 22) / tt) * kBI);  // a launch's tiles fit an int
  p.tiles = piece_tiles(V, rows);
  int64_t at = 256;
  const auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += up(bytes, 256);
    return o;
  };
  p.pos = take(4 * T);
  p.ct = take(4 * T);
  p.hc = take(2 * T * p.Dp);
  if (!bwd) {
    p.part = take((V + 127) / 128 * 8 * T + 8 * T);
    p.zt = take(4 * T);
  } else {
    p.lsec = take(4 * T);
    p.c = take(4 * T);
    p.ldg = std::min(p.tiles * kBI, up(V, 64));
    p.G = take(2 * T * p.ldg);
    // dh's tiles split over the piece's columns until a unit is at most
    // about 0.85 of a CU's share of the piece's work, so that units and dW's
    // tiles pack the CUs evenly
    const int64_t td = (D + kBI - 1) / kBI;
    const int64_t sv = p.tiles * kBI / kRed16, st = (T + kRed16 - 1) / kRed16;
    const double share = (double)(td * tt * sv + td * p.tiles * st) / 256.0;
    int64_t split = (int64_t)((double)sv / (0.85 * share) + 0.999);
    split = std::min<int64_t>(split, std::max<int64_t>(1, sv / 16));
    p.split = std::max<int64_t>(1, split);
    p.slab = take(4 * p.split * T * D);
  }
  if (p.padded) p.pad = take(2 * p.tiles * kBI * p.Dp);
  p.total = at;
  return p;
}

static bool xent_few(int64_t T, int64_t V, int64_t D) { return few_tokens(T, V) && D >= 8; }

size_t xent_workspace(int64_t T, int64_t V, int64_t D, bool bwd) {
  if (!bwd && xent_few(T, V, D)) return (size_t)(up(few_tiles(T, V) * 8 * T, 256) + up(4 * T, 256));
  return (size_t)xent_plan(T, V, D, bwd).total;
}

template <bool BWD>
static void launch_gather(const XentRows& r, hipStream_t st) {
  const int groups = 1 + r.T / (1 << 13), rows = groups * kGatherRows;
  xent_gather_kernel<BWD><<<(unsigned)((r.T + rows - 1) / rows), 256, 0, st>>>(r, groups);
}

static hipError_t launch_pad(const uint16_t* w, int64_t rows, int64_t D, int64_t Dp, uint16_t* out, hipStream_t st) {
  const int64_t chunks = rows * (Dp / 8);
  xent_pad_kernel<<<(unsigned)((chunks + 255) / 256), 256, 0, st>>>(w, rows, (int)D, (int)(Dp / 8), out);
  return hipGetLastError();
}

static hipError_t launch_loss(const XentLoss& l, const int64_t* targets, int64_t ignore, float* total, bool mean,
                              hipStream_t st) {
  const bool together = l.T <= kLossTokens;
  XentLoss a = l;
  a.total = together ? total : nullptr;
  a.mean = mean ? 1 : 0;
  xent_combine_kernel<<<(l.T + kLossTokens - 1) / kLossTokens, 1024, 0, st>>>(a);
  if (hipError_t e = hipGetLastError()) return e;
  if (total == nullptr || together) return hipSuccess;
  xent_reduce_kernel<<<1, 1024, 0, st>>>(l.loss, targets, ignore, l.T, mean ? 1 : 0, total);
  return hipGetLastError();
}

hipError_t launch_xent_fwd(const uint16_t* h, const uint16_t* w, const int64_t* targets, int64_t ignore, int64_t T,
                           int64_t V, int64_t D, float* loss, float* lse, float* total, bool mean, void* ws,
                           hipStream_t stream) {
  char* base = static_cast<char*>(ws);
  if (xent_few(T, V, D)) {
    XentFew f{};
    f.w = w;
    f.V = V;
    f.D = (int)D;
    f.h = XentHidden{h, h, (int)T};
    f.T = (int)T;
    f.groups = (int)few_groups(T);
    f.targets = targets;
    f.part = reinterpret_cast<float2*>(base);
    f.zt = reinterpret_cast<float*>(base + up(few_tiles(T, V) * 8 * T, 256));
    if (hipError_t e = launch_few<false>(f, stream)) return e;
    const XentLoss l{f.part, (int)few_tiles(T, V), (int)T, f.zt, nullptr, targets, ignore, V, lse, loss, nullptr, 0};
    return launch_loss(l, targets, ignore, total, mean, stream);
  }
  const XentPlan p = xent_plan(T, V, D, false);
  XentRows r{};
  r.h = h;
  r.targets = targets;
  r.ignore = ignore;
  r.T = (int)T;
  r.D = (int)D;
  r.Dp = (int)p.Dp;
  r.V = V;
  r.ctl = reinterpret_cast<XentCtl*>(base);
  r.hc = reinterpret_cast<uint16_t*>(base + p.hc);
  r.pos = reinterpret_cast<int*>(base + p.pos);
  r.ct = reinterpret_cast<int*>(base + p.ct);
  launch_gather<false>(r, stream);
  if (hipError_t e = hipGetLastError()) return e;
  XentTiles a{};
  a.h = XentHidden{r.hc, p.padded ? r.hc : h, r.T};
  a.Dp = r.Dp;
  a.ctl = r.ctl;
  a.ct = r.ct;
  a.part = reinterpret_cast<float2*>(base + p.part);
  a.T = r.T;
  a.zt = reinterpret_cast<float*>(base + p.zt);
  a.tiles_t = (int)((T + kBJ - 1) / kBJ);
  a.nstages = (int)((p.Dp + kRed16 - 1) / kRed16);
  for (int64_t v0 = 0; v0 < V; v0 += p.tiles * kBI) {
    const int64_t vc = std::min(V - v0, p.tiles * kBI);
    a.w = w + v0 * D;
    a.ldw = D;
    if (p.padded) {
      uint16_t* pad = reinterpret_cast<uint16_t*>(base + p.pad);
      if (hipError_t e = launch_pad(a.w, vc, D, p.Dp, pad, stream)) return e;
      a.w = pad;
      a.ldw = p.Dp;
    }
    a.vc = (int)vc;
    a.v0 = (int)v0;
    a.tiles_v = (int)((vc + kBI - 1) / kBI);
    xent_logits_kernel<false><<<(unsigned)(a.tiles_v * a.tiles_t), kThreads, 0, stream>>>(a);
    if (hipError_t e = hipGetLastError()) return e;
  }
  const XentLoss l{a.part, (int)((V + 127) / 128), (int)T, a.zt, r.pos, targets, ignore, V, lse, loss, nullptr, 0};
  return launch_loss(l, targets, ignore, total, mean, stream);
}

hipError_t launch_xent_bwd(const uint16_t* h, const uint16_t* w, const int64_t* targets, int64_t ignore,
                           const float* lse, const float* dloss, bool per_row, bool mean, int64_t T, int64_t V,
                           int64_t D, uint16_t* dh, void* dw, bool dw_f32, void* ws, hipStream_t stream) {
  char* base = static_cast<char*>(ws);
  const XentPlan p = xent_plan(T, V, D, true);
  XentRows r{};
  r.h = h;
  r.targets = targets;
  r.ignore = ignore;
  r.T = (int)T;
  r.D = (int)D;
  r.Dp = (int)p.Dp;
  r.V = V;
  r.ctl = reinterpret_cast<XentCtl*>(base);
  r.hc = reinterpret_cast<uint16_t*>(base + p.hc);
  r.pos = reinterpret_cast<int*>(base + p.pos);
  r.ct = reinterpret_cast<int*>(base + p.ct);
  r.lse = lse;
  r.dloss = dloss;
  r.per_row = per_row ? 1 : 0;
  r.mean = mean ? 1 : 0;
  r.lsec = reinterpret_cast<float*>(base + p.lsec);
  r.c = reinterpret_cast<float*>(base + p.c);
  launch_gather<true>(r, stream);
  if (hipError_t e = hipGetLastError()) return e;
  XentTiles a{};
  a.h = XentHidden{r.hc, p.padded ? r.hc : h, r.T};
  a.Dp = r.Dp;
  a.ctl = r.ctl;
  a.ct = r.ct;
  a.T = r.T;
  a.lsec = r.lsec;
  a.c = r.c;
  a.G = reinterpret_cast<uint16_t*>(base + p.G);
  a.ldg = (int)p.ldg;
  a.tiles_t = (int)((T + kBJ - 1) / kBJ);
  a.nstages = (int)((p.Dp + kRed16 - 1) / kRed16);
  XentGrads g{};
  g.G = a.G;
  g.ldg = a.ldg;
  g.h = a.h;
  g.Dp = a.Dp;
  g.D = (int)D;
  g.T = r.T;
  g.ctl = r.ctl;
  g.tiles_d = (int)((D + kBI - 1) / kBI);
  g.tiles_t = a.tiles_t;
  g.slab = reinterpret_cast<float*>(base + p.slab);
  g.split = (int)p.split;
  g.dh_units = dh ? g.tiles_d * g.tiles_t * g.split : 0;
  for (int64_t v0 = 0; v0 < V; v0 += p.tiles * kBI) {
    const int64_t vc = std::min(V - v0, p.tiles * kBI);
    a.w = w + v0 * D;
    a.ldw = D;
    if (p.padded) {
      uint16_t* pad = reinterpret_cast<uint16_t*>(base + p.pad);
      if (hipError_t e = launch_pad(a.w, vc, D, p.Dp, pad, stream)) return e;
      a.w = pad;
      a.ldw = p.Dp;
    }
    a.vc = (int)vc;
    a.v0 = (int)v0;
    a.tiles_v = (int)((vc + kBI - 1) / kBI);
    if (few_tokens(T, V)) {
      XentFew f{};
      f.w = a.w;
      f.V = vc;
      f.D = a.Dp;
      f.h = a.h;
      f.T = r.T;
      f.groups = (int)few_groups(T);
      f.ctl = a.ctl;
      f.ct = a.ct;
      f.lsec = a.lsec;
      f.c = a.c;
      f.v0 = a.v0;
      f.G = a.G;
      f.ldg = a.ldg;
      if (hipError_t e = launch_few<true>(f, stream)) return e;
    } else {
      xent_logits_kernel<true><<<(unsigned)(a.tiles_v * a.tiles_t), kThreads, 0, stream>>>(a);
      if (hipError_t e = hipGetLastError()) return e;
    }
    g.w = a.w;
    g.ldw = a.ldw;
    g.vc = a.vc;
    // columns [vc, up(vc, 64)) of G hold zeros
    g.stages_v = (int)((vc + kRed16 - 1) / kRed16);
    g.first = v0 == 0 ? 1 : 0;
    g.dw = dw ? static_cast<char*>(dw) + v0 * D * (dw_f32 ? 4 : 2) : nullptr;
    const unsigned grid = (unsigned)(g.dh_units + (dw ? g.tiles_d * a.tiles_v : 0));
    if (dw_f32) xent_grads_kernel<true><<<grid, kThreads, 0, stream>>>(g);
    else xent_grads_kernel<false><<<grid, kThreads, 0, stream>>>(g);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (dh == nullptr) return hipSuccess;
  const int nch = (int)(p.Dp / 8);
  xent_dh_kernel<<<(unsigned)((T * nch + 255) / 256), 256, 0, stream>>>(g.slab, g.split, r.pos, r.ctl, r.T, r.D, nch, dh);
  return hipGetLastError();
}

}  // namespace bitnet
