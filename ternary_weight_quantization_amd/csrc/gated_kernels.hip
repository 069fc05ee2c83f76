// The gated pair of ternary projections of a feed-forward block in one kernel,
//
//   g = (x_q . tg^T) s/127 gamma_g,  u = (x_q . tu^T) s/127 gamma_u,  y = act(g) u
//
// and its straight-through backward
//
//   dg = dY u act'(g),  du = dY act(g)
//   dX = gamma_g dg tg + gamma_u du tu,  dWg = dg^T x_hat,  dWu = du^T x_hat
//
// Forward: the int8 product of gemm_kernels.hip over the rows of both weights.
// A wave's 128 code rows are 64 of the gate and the same 64 of the up
// projection, so that a lane holds g and u of the same outputs in its
// accumulators and the epilogue applies the activation there: neither
// projection is written and read again. For the backward it stores y's slopes
// dy/dg = u act'(g) and dy/du = act(g) next to y, their fp32 values rounded to 24 bits
// (half a step: 2^-16 of the value; cut off they would be twice as far, and all short).
//
// Backward: one pass makes D = [gamma_g dg | gamma_u du] s/127 in bf16, then the
// two products of gemm_kernels.hip on D, the codes of both weights below each
// other and the int8 rows as bf16 (exact). The scales are all in D: dX sums over
// both halves, whose scales differ, and dW over the tokens; dX's epilogue divides
// a token's row by s/127 and dW's each half by its gamma, in fp32. So every
// gradient sees two roundings to bf16, D's and its own: 0.0024 of its norm off
// the exact one (g and u kept in bf16, D without s and x_hat rounded gave
// 0.0037, and 0.0044 for relu2). Rows of D, of the slopes and of the transposed
// codes are padded to Nd = N rounded up to 64 in each half, so that every width
// runs the aligned loaders and no 32 rows of dW belong to both halves.
//
// Measured, 4096 x 2560 -> 2 x 6912: forward 195 to 208 us (290 G operations; the 227 MB
// of y and slopes in its epilogue are 44 of it at a copy's rate), D and the operands 65
// (400 MB, 6.1 TB/s, half of it left in the last-level cache), both products 445 to 489 (580 GFLOP, 1.19
// to 1.30 PFLOP/s by the card's clock; the largest library product reaches 1.32). Up to
// 256 tokens few8.h's kernels and up to about 1000 mid.h's tiles run instead.

#include <algorithm>

#include "activation.h"
#include "bwd_prep.h"
#include "few8.h"
#include "gemm_split.h"
#include "mid.h"
#include "row_io.h"

namespace bitnet {

hipError_t take_gated_split_timeouts(unsigned int* count) { return take_local_split_timeouts(count); }

static int64_t n_half(int64_t N) { return (N + 63) / 64 * 64; }
size_t gated_slopes_bytes(int64_t M, int64_t N) { return (size_t)M * 2 * n_half(N) * 3; }

// P: the codes [2N][Kp/4], gate rows first. Row r of tile ti (row0 = 256 ti): wave
// half r / 128, then 64 gate rows and 64 up rows of outputs
// 128 ti + 64 (r / 128) + r % 64.
struct GatedCodesLoader : RowCodesLoader<CodesI8Frags> {
  int64_t N;
  __device__ __forceinline__ void load(Regs& r, int row0, int s) const {
    const int t = threadIdx.x;
    const int64_t n = row0 / 2 + 64 * (t >> 7) + (t & 63);
    const rsrc_t rs = make_rsrc(packed, (uint32_t)(rows * pitch));
    r.lane_off = n < N ? (uint32_t)(((t & 64) ? N + n : n) * pitch) : kOob;
#pragma unroll
    for (int h = 0; h < 2; ++h) r.v[h] = buf_load16(rs, offset(r, s, h));
  }
};

// A slope, rounded to the nearest multiple of 2^8 in its bits, is kept as the upper 16
// and the 8 below them, in two planes: [M][2 Nd] of 16 bits, then [M][2 Nd] bytes. The
// carry takes no NaN away: all that reach here stem from g's and u's factors
// (quiet_nan) or from the operations, whose own has no low bits.
__device__ __forceinline__ uint32_t slope24(float v) { return __float_as_uint(v) + 0x80u; }
__device__ __forceinline__ uint2 slopes_hi(const float (&v)[4]) {
  return make_uint2(perm(slope24(v[1]), slope24(v[0]), 0x07060302u), perm(slope24(v[3]), slope24(v[2]), 0x07060302u));
}
__device__ __forceinline__ uint32_t slopes_lo(const float (&v)[4]) {
  return perm(perm(slope24(v[3]), slope24(v[2]), 0x0C0C0501u), perm(slope24(v[1]), slope24(v[0]), 0x0C0C0501u),
              0x05040100u);
}
__device__ __forceinline__ float quiet_nan(float c) {
  const uint32_t b = __float_as_uint(c);
  return __uint_as_float((b & 0x7FFFFFFFu) > 0x7F800000u ? 0x7FC00000u : b);
}
__device__ __forceinline__ void slopes8(uint4 hi, uint2 lo, float (&f)[8]) {
  const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[2] = {lo.x, lo.y};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    f[e] = __uint_as_float(((e & 1) ? h[e >> 1] & 0xFFFF0000u : h[e >> 1] << 16) | ((l[e >> 2] >> (8 * (e & 3))) & 0xFFu) << 8);
}

// y = act(g) u and, with SLOPES, dy/dg and dy/du.
template <class ACT, bool SLOPES>
__device__ __forceinline__ void gated_value(float g, float u, float& y, float& dg, float& du) {
  if constexpr (SLOPES) {
    float da;
    ACT::fd(g, du, da);
    dg = da * u;
    y = du * u;
  } else {
    y = ACT::f(g) * u;
  }
}

// acc: fragments fi 0, 1 hold the gate, 2, 3 the up projection of the same
// outputs. SAVE: the slopes are stored too, [M][2 Nd].
template <class ACT, bool SAVE>
struct GatedEpilogue {
  uint16_t* y;    // [M][N]
  uint16_t* slopes;
  const float* s;
  const float* gamma;  // [2]
  int64_t N, Nd, M;

  struct Pre { float gg, gu; float sj[kFJ]; };
  static constexpr int kDg = HalfStage::kBytes, kDu = 2 * HalfStage::kBytes;  // LDS offsets
  static constexpr int kDgLo = 3 * HalfStage::kBytes, kDuLo = kDgLo + RowStage<1>::kBytes;
  static constexpr int kWaveLds = kDuLo + RowStage<1>::kBytes;
  __device__ __forceinline__ Pre prefetch(int j0, int lane) const {
    Pre pre;
    pre.gg = gamma[0];
    pre.gu = gamma[1];
#pragma unroll
    for (int fj = 0; fj < kFJ; ++fj) {
      const int64_t j = j0 + 32 * fj + (lane & 31);
      pre.sj[fj] = j < M ? s[j] : 0.0f;
    }
    return pre;
  }
  __device__ __forceinline__ void store(MfmaI8::Acc (&acc)[kFI][kFJ], const Pre& pre, int i0, int j0, int lane,
                                        char* wlds) const {
    const int n0 = i0 / 2;
    // The tile of a wait that gave up, whose accumulators are INT32_MIN throughout (no sum
    // of codes is): y would be 0 there, act's value far below 0, so the factors are NaN.
    const bool lost = (uint32_t)acc[0][0][0] == MfmaI8::kPoisonBits;
#pragma unroll
    for (int fj = 0; fj < kFJ; ++fj) {
      const float sj = lost ? __uint_as_float(0x7FC00000u) : pre.sj[fj];
      const float cg = quiet_nan(sj * pre.gg / 127.0f), cu = quiet_nan(sj * pre.gu / 127.0f);
#pragma unroll
      for (int fi = 0; fi < 2; ++fi)
#pragma unroll
        for (int gi = 0; gi < 4; ++gi) {
          float dg[4], du[4], y4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            gated_value<ACT, SAVE>((float)acc[fi][fj][4 * gi + e] * cg, (float)acc[fi + 2][fj][4 * gi + e] * cu, y4[e],
                                   dg[e], du[e]);
          HalfStage::put(wlds, lane, fi, gi, make_uint2(pack_bf16x2(y4[0], y4[1]), pack_bf16x2(y4[2], y4[3])));
          if constexpr (SAVE) {
            HalfStage::put(wlds + kDg, lane, fi, gi, slopes_hi(dg));
            HalfStage::put(wlds + kDu, lane, fi, gi, slopes_hi(du));
            RowStage<1>::put(wlds + kDgLo, lane, fi, gi, slopes_lo(dg));
            RowStage<1>::put(wlds + kDuLo, lane, fi, gi, slopes_lo(du));
          }
        }
      HalfStage::drain(wlds, y, N, N, M, n0, j0 + 32 * fj, lane);
      if constexpr (SAVE) {
        uint8_t* lo = reinterpret_cast<uint8_t*>(slopes + M * 2 * Nd);
        HalfStage::drain(wlds + kDg, slopes, 2 * Nd, Nd, M, n0, j0 + 32 * fj, lane);
        HalfStage::drain(wlds + kDu, slopes + Nd, 2 * Nd, Nd, M, n0, j0 + 32 * fj, lane);
        RowStage<1>::drain(wlds + kDgLo, lo, 2 * Nd, Nd, M, n0, j0 + 32 * fj, lane);
        RowStage<1>::drain(wlds + kDuLo, lo + Nd, 2 * Nd, Nd, M, n0, j0 + 32 * fj, lane);
      }
    }
  }
};

// ---------------------------------------------------------------------------
// Few tokens (few8.h; up to 4 groups of kFewM, gated_form): a workgroup's pairs of tiles
// are 16 rows of the gate and the same 16 of the up projection.
// ---------------------------------------------------------------------------

// RP: pairs of tiles.
template <class ACT, int RP, int MT, int W, int P, bool TX, int NX>
__global__ __launch_bounds__(kWave * W) void gated_few_kernel(FewArgs a, const float* __restrict__ s,
                                                              const float* __restrict__ gamma, int64_t N, int64_t Nd,
                                                              uint16_t* __restrict__ y, uint16_t* __restrict__ slopes) {
  __shared__ __attribute__((aligned(16))) char smem[few_lds<true, 2 * RP, MT, W, TX, false>()];
  __shared__ FewRows<NX, W> rows;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int64_t M = a.M;
  int tile, m0;
  few_place(a, tile, m0);
  const int64_t n0 = (int64_t)tile * (16 * RP);
  int64_t row[2 * RP];
#pragma unroll
  for (int p = 0; p < RP; ++p) {
    const int64_t n = n0 + 16 * p + (lane & 15);
    row[2 * p] = n < N ? n : -1;
    row[2 * p + 1] = n < N ? N + n : -1;
  }
  few_tokens_product<true, 2 * RP, MT, W, P, TX, false>(a, row, smem, rows);
  for (int i = wave; i < RP * MT; i += W) {
    const int p = i % RP, mt = i / RP;
    const int64_t ml = 16 * mt + (lane & 15), m = m0 + ml;
    if (ml >= a.M) continue;
    int vg[4], vu[4];
    few_tokens_sum<2 * RP, MT, W>(smem, 2 * p, mt, vg);
    few_tokens_sum<2 * RP, MT, W>(smem, 2 * p + 1, mt, vu);
    float sm;
    if constexpr (NX > 0) sm = rows.s[m];
    else sm = s[m];
    // the large-M epilogue's expressions
    const float cg = quiet_nan(sm * gamma[0] / 127.0f), cu = quiet_nan(sm * gamma[1] / 127.0f);
    const int64_t nb = n0 + 16 * p + 4 * (lane >> 4);
    float dg[4], du[4], o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) gated_value<ACT, true>((float)vg[e] * cg, (float)vu[e] * cu, o[e], dg[e], du[e]);
    store4(y + m * N, nb, N, o);
    if (slopes != nullptr && nb < Nd) {  // the padding's columns past the last workgroup's stay unwritten and are not read
      uint16_t* r = slopes + m * 2 * Nd + nb;
      uint8_t* lo = reinterpret_cast<uint8_t*>(slopes + M * 2 * Nd) + m * 2 * Nd + nb;
      *reinterpret_cast<uint2*>(r) = slopes_hi(dg);
      *reinterpret_cast<uint2*>(r + Nd) = slopes_hi(du);
      *reinterpret_cast<uint32_t*>(lo) = slopes_lo(dg);
      *reinterpret_cast<uint32_t*>(lo + Nd) = slopes_lo(du);
    }
  }
}

// ---------------------------------------------------------------------------
// Middling M (mid.h): the 64 rows of a wave are 32 of the gate and the same 32 of the up
// projection.
// ---------------------------------------------------------------------------

struct GatedRow {
  int n0;
  int64_t N;
  __device__ __forceinline__ int64_t operator()(int r) const {
    const int64_t n = n0 + 32 * (r >> 6) + (r & 31);
    return n < N ? ((r & 32) ? N + n : n) : -1;
  }
};

template <class ACT, int FJ, int P>
__global__ __launch_bounds__(256) void gated_mid_kernel(const uint8_t* __restrict__ packed, const int8_t* __restrict__ xq,
                                                        const float* __restrict__ s, const float* __restrict__ gamma,
                                                        int64_t M, int64_t N, int64_t Nd, int64_t Kp, int tiles_j,
                                                        uint16_t* __restrict__ y, uint16_t* __restrict__ slopes) {
  typedef MidShape<2, FJ, 2, 2> S;
  typedef MidCodes<GatedRow> LP;
  typedef MidRows<TileRow> LQ;
  __shared__ __attribute__((aligned(16))) char lds[S::template kLds<LP, LQ>];
  const int v = xcd_major(blockIdx.x, gridDim.x), lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int n0 = v / tiles_j * (S::kI / 2), j0 = v % tiles_j * S::kJ;
  const int nw = n0 + 32 * (wave % 2), jw = j0 + 32 * FJ * (wave / 2);
  float sj[FJ];
#pragma unroll
  for (int fj = 0; fj < FJ; ++fj) {
    const int64_t m = jw + 32 * fj + (lane & 31);
    sj[fj] = m < M ? s[m] : 0.0f;
  }
  const float gg = gamma[0], gu = gamma[1];
  const LP lp{{}, packed, 2 * N, Kp / 4, {n0, N}};
  const LQ lq{{}, xq, M, Kp, {j0, M}};
  MfmaI8::Acc acc[2][FJ] = {};
  mid_tile<MfmaI8, 2, FJ, 2, 2, P>(lp, lq, (int)((Kp + kStageBytes - 1) / kStageBytes), lds, acc);
  // y and the slopes go through LDS, as whole rows of the wave's 32 columns (stored from
  // the accumulators, 8 bytes a lane: 1024 x 640 -> 2 x 1728 with slopes 14.6 us, 10.2 so)
  typedef RowStage<2, 32> Half;
  typedef RowStage<1, 32> Byte;
  constexpr int kDg = Half::kBytes, kDu = 2 * Half::kBytes, kDgLo = 3 * Half::kBytes, kDuLo = kDgLo + Byte::kBytes;
  constexpr int kWave1 = kDuLo + Byte::kBytes;
  static_assert(4 * kWave1 <= sizeof(lds), "the epilogue's staging");
  char* w = lds + wave * kWave1;
  const bool save = slopes != nullptr;
  uint8_t* lo = save ? reinterpret_cast<uint8_t*>(slopes + M * 2 * Nd) : nullptr;
#pragma unroll
  for (int fj = 0; fj < FJ; ++fj) {
    // the large tiles' expressions
    const float cg = quiet_nan(sj[fj] * gg / 127.0f), cu = quiet_nan(sj[fj] * gu / 127.0f);
#pragma unroll
    for (int gi = 0; gi < 4; ++gi) {
      float dg[4], du[4], o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        gated_value<ACT, true>((float)acc[0][fj][4 * gi + e] * cg, (float)acc[1][fj][4 * gi + e] * cu, o[e], dg[e], du[e]);
      Half::put(w, lane, 0, gi, make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])));
      if (save) {
        Half::put(w + kDg, lane, 0, gi, slopes_hi(dg));
        Half::put(w + kDu, lane, 0, gi, slopes_hi(du));
        Byte::put(w + kDgLo, lane, 0, gi, slopes_lo(dg));
        Byte::put(w + kDuLo, lane, 0, gi, slopes_lo(du));
      }
    }
    const int j = jw + 32 * fj;
    Half::drain(w, y, N, N, M, nw, j, lane);
    if (save) {
      Half::drain(w + kDg, slopes, 2 * Nd, Nd, M, nw, j, lane);
      Half::drain(w + kDu, slopes + Nd, 2 * Nd, Nd, M, nw, j, lane);
      Byte::drain(w + kDgLo, lo, 2 * Nd, Nd, M, nw, j, lane);
      Byte::drain(w + kDuLo, lo + Nd, 2 * Nd, Nd, M, nw, j, lane);
    }
  }
}

// ---------------------------------------------------------------------------
// Backward, what the products read, in one launch: D, the codes of both weights
// transposed to fp4 [Kp][2 Nd / 2] and the int8 rows as bf16 [M][Kp]. (D in a launch of
// its own: 51.5 + 15.6 us for 64.8 at 4096 x 2560 -> 2 x 6912.)
// ---------------------------------------------------------------------------

// D [M][2 Nd] from dY [M][N] and the slopes, times the half's gamma and (sx not
// NULL) the token's sx/127. A thread takes 8 columns of both halves; columns past N
// are zeros.
struct GatedD {
  const uint16_t* dY;
  const uint16_t* slopes;
  const float* gamma;
  const float* sx;
  int64_t total;  // M Nd / 8
  int N, Nd;
  uint16_t* D;
};

__device__ __forceinline__ void gated_d_block(const GatedD& a, int64_t b) {
  const int64_t i = b * 256 + threadIdx.x;
  if (i >= a.total) return;
  const int nch = a.Nd / 8, N = a.N, Nd = a.Nd;
  const int64_t row = i / nch;
  const int k0 = 8 * (int)(i - row * nch);
  const int64_t at = row * 2 * Nd + k0;
  const int64_t src = k0 < N ? at : at - k0;  // past N: any written columns, not used
  const uint8_t* lo = reinterpret_cast<const uint8_t*>(a.slopes + a.total * 16);  // total / nch rows of 2 Nd = 16 nch
  const uint4 hg = *reinterpret_cast<const uint4*>(a.slopes + src);
  const uint4 hu = *reinterpret_cast<const uint4*>(a.slopes + src + Nd);
  const uint2 lg = *reinterpret_cast<const uint2*>(lo + src), lu = *reinterpret_cast<const uint2*>(lo + src + Nd);
  float d[8], g[8], u[8];
  chunk8(a.dY + row * N, k0, N).get(d);
  slopes8(hg, lg, g);
  slopes8(hu, lu, u);
  const float sc = a.sx != nullptr ? a.sx[row] / 127.0f : 1.0f, gg = a.gamma[0] * sc, gu = a.gamma[1] * sc;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const bool in_row = k0 + e < N;  // a slope of the padding may be anything
    g[e] = in_row ? d[e] * g[e] * gg : 0.0f;
    u[e] = in_row ? d[e] * u[e] * gu : 0.0f;
  }
  store8_in(a.D + at, g);
  store8_in(a.D + at + Nd, u);
}

// Blocks: wt_bx * wt_by of the transposed codes, xhat_nb of the rows, then D's.
__global__ __launch_bounds__(256) void gated_prep_kernel(const uint8_t* __restrict__ packed, int64_t N, int64_t Kp,
                                                         int64_t Nd, uint8_t* __restrict__ wt, int wt_bx, int wt_by,
                                                         const int8_t* __restrict__ xq, int64_t M,
                                                         uint16_t* __restrict__ xhat, int xhat_nb, GatedD d) {
  const int64_t b = blockIdx.x;
  const int nwt = wt_bx * wt_by;
  if (b >= nwt + xhat_nb) {
    gated_d_block(d, b - (nwt + xhat_nb));
  } else if (b < nwt) {
    const int v = xcd_major((int)b, nwt);
    const auto row = [N, Nd](int64_t n) {
      const int64_t c = n < Nd ? n : n - Nd;
      return c < N ? (n < Nd ? c : N + c) : int64_t(-1);
    };
    wt_fp4_block(packed, row, Kp, 2 * Nd, wt, v % wt_bx, v / wt_bx);
  } else {
    xhat_blocks(xq, nullptr, M, Kp, xhat, (int)b - nwt, xhat_nb);
  }
}

// dX: a token's row is divided by the s/127 in D (s NULL: none is).
struct TokenEpilogue {
  uint16_t* out;  // [J][I]
  const float* s;
  int64_t I, J;   // K, M

  struct Pre { float c[kFJ]; };
  static constexpr int kWaveLds = EpStage<2>::kWaveBytes;
  __device__ __forceinline__ Pre prefetch(int j0, int lane) const {
    Pre pre;
#pragma unroll
    for (int fj = 0; fj < kFJ; ++fj) {
      const int64_t j = j0 + 32 * fj + (lane & 31);
      pre.c[fj] = s != nullptr && j < J ? per_scale(s[j]) : 1.0f;
    }
    return pre;
  }
  __device__ __forceinline__ void store(MfmaBf16::Acc (&acc)[kFI][kFJ], const Pre& pre, int i0, int j0, int lane,
                                        char* wlds) const {
#pragma unroll
    for (int fj = 0; fj < kFJ; ++fj) {
      const float c = pre.c[fj];
#pragma unroll
      for (int fi = 0; fi < kFI; ++fi)
#pragma unroll
        for (int gi = 0; gi < 4; ++gi)
          EpStage<2>::put(wlds, lane, fi, gi,
                          make_uint2(pack_bf16x2(acc[fi][fj][4 * gi] * c, acc[fi][fj][4 * gi + 1] * c),
                                     pack_bf16x2(acc[fi][fj][4 * gi + 2] * c, acc[fi][fj][4 * gi + 3] * c)));
      EpStage<2>::drain(wlds, reinterpret_cast<char*>(out), I, J, i0, j0 + 32 * fj, lane);
    }
  }
};

// dW of both halves: rows j < Nd go to out[0], the others to out[1], divided by
// the half's scale (in D).
template <bool OUT_F32>
struct HalvesEpilogue {
  void* out[2];
  const float* gamma;  // [2]
  int64_t I, N, Nd;    // outputs [N][I]

  struct Pre { float g[2]; };
  static constexpr int kEB = OUT_F32 ? 4 : 2;
  static constexpr int kWaveLds = EpStage<kEB>::kWaveBytes;
  __device__ __forceinline__ Pre prefetch(int, int) const { return Pre{{gamma[0], gamma[1]}}; }
  __device__ __forceinline__ void store(MfmaBf16::Acc (&acc)[kFI][kFJ], const Pre& pre, int i0, int j0, int lane,
                                        char* wlds) const {
#pragma unroll
    for (int fj = 0; fj < kFJ; ++fj) {
      const int j = __builtin_amdgcn_readfirstlane(j0 + 32 * fj);
      const bool up = j >= Nd;  // of all 32 rows: Nd is a multiple of 64
      const int jh = up ? (int)(j - Nd) : j;
      if (jh >= N) continue;
      const float sc = 1.0f / (up ? pre.g[1] : pre.g[0]);
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
      EpStage<kEB>::drain(wlds, static_cast<char*>(out[up]), I, N, i0, jh, lane);
    }
  }
};

// The same for mid.h's tiles.
template <int EB>
struct MidHalves {
  static constexpr int kEB = EB;
  void* out[2];
  const float* gamma;
  int64_t I, N, Nd;
  __device__ __forceinline__ float scale(int64_t j) const { return 1.0f / gamma[j >= Nd ? 1 : 0]; }
  __device__ __forceinline__ void* part(int& j, int64_t& rows) const {
    const bool up = j >= Nd;  // of all 32 rows: Nd is a multiple of 64
    if (up) j -= (int)Nd;
    rows = N;
    return up ? out[1] : out[0];
  }
};

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------

static bool few(int64_t M) {
  return M <= kSkinnyMaxM && test_knobs().no_skinny.load(std::memory_order_relaxed) == 0;
}

static GemmShape fwd_shape(int64_t M, int64_t N, int64_t K) {
  return {(N + 127) / 128, (M + kBJ - 1) / kBJ, (k_pad(K) + kStageBytes - 1) / kStageBytes, kFwdPieceCost};
}

// The forward's kernel: kFew up to 32 tokens, and up to 256 while the workgroups of 32
// outputs and 64 tokens fit the device at once (2560 -> 2 x 1728, 256 tokens: 9.4 us, 13.2
// with mid.h's tiles; 2560 -> 2 x 6912, 128: 16.6 and 14.3; 2560 -> 2 x 13824, 64: 16.8 and
// 14.2). Up to 64 tokens a long reduction is better off in it too, whose waves share it
// (6912 -> 2 x 9000, 64 tokens: 23.7 and 29.0).
enum GatedForm { kFew, kMid1, kMid2, kTiles };
static bool deep(int64_t K) { return k_pad(K) > 12 * FewStep<true>::kK; }
static GatedForm gated_form(int64_t M, int64_t N, int64_t K) {
  const int64_t groups = (M + kFewM - 1) / kFewM;
  if (few(1) && (M <= 32 || (M <= kFewM && deep(K)) ||
                 (M <= 4 * kFewM && (N + 31) / 32 * groups <= device_cus())))
    return kFew;
  const int fj = mid_blocks(M, (N + 63) / 64);
  return fj == 1 || (fj == 0 && few(M)) ? kMid1 : fj == 2 ? kMid2 : kTiles;
}

size_t gated_fwd_workspace(int64_t M, int64_t N, int64_t K) {
  if (gated_form(M, N, K) != kTiles) return 0;
  const GemmShape g = fwd_shape(M, N, K);
  return split_workspace(g, split_grid(g, device_cus()));
}

template <class ACT, int RP, int MT, int W, int P, bool TX, int NX = 0>
static void gated_few(const FewArgs& a, const float* s, const float* gamma, int64_t N, int64_t Nd, uint16_t* y,
                      uint16_t* slopes, hipStream_t st) {
  gated_few_kernel<ACT, RP, MT, W, P, TX, NX>
      <<<(unsigned)((N + 16 * RP - 1) / (16 * RP) * ((a.M + kFewM - 1) / kFewM)), kWave * W, 0, st>>>(a, s, gamma, N, Nd, y,
                                                                                                   slopes);
}

template <class ACT, int FJ, int P>
static hipError_t gated_mid(const uint8_t* w_packed, const int8_t* x_q, const float* s_x, const float* gamma, int64_t M,
                            int64_t N, int64_t Kp, uint16_t* y, uint16_t* slopes, hipStream_t st) {
  const int64_t tj = (M + 64 * FJ - 1) / (64 * FJ), ti = (N + 63) / 64;
  gated_mid_kernel<ACT, FJ, P><<<(unsigned)(ti * tj), 256, 0, st>>>(w_packed, x_q, s_x, gamma, M, N, n_half(N), Kp,
                                                                     (int)tj, y, slopes);
  return hipGetLastError();
}

template <class ACT>
static hipError_t gated_fwd(const uint16_t* x, const int8_t* x_q, const float* s_x, const uint8_t* w_packed,
                            const float* gamma, int64_t M, int64_t N, int64_t K, uint16_t* y, uint16_t* slopes, void* ws,
                            size_t ws_bytes, hipStream_t stream) {
  const int64_t Kp = k_pad(K), Nd = n_half(N);
  const GatedForm form = gated_form(M, N, K);
  if (form == kFew) {
    const FewArgs a{w_packed, 2 * N, Kp / 4, x_q, Kp, (int)M, x, (int)K};
    // Up to 32 tokens 16 outputs a workgroup of 4 waves, or 8 where each would have more
    // than 3 steps (1 token, 6912 -> 2 x 2560: 6.0 us with 8, 7.1 with 4; 2560 -> 2 x 6912
    // 8.1 and 5.7). Above, x_q's traffic counts: 32 outputs share it (64 tokens, 2560 -> 2 x
    // 6912: 8.7 us against 15.3 with 16, 6912 -> 2 x 2560 12.4 against 13.5).
    const bool deep = bitnet::deep(K);
    if (x != nullptr) {  // M <= rows_direct(K)
      if (M > 2 && deep) gated_few<ACT, 1, 1, 8, 3, false, 4>(a, s_x, gamma, N, Nd, y, slopes, stream);
      else if (M > 2) gated_few<ACT, 1, 1, 4, 3, false, 4>(a, s_x, gamma, N, Nd, y, slopes, stream);
      else if (M > 1 && deep) gated_few<ACT, 1, 1, 8, 3, false, 2>(a, s_x, gamma, N, Nd, y, slopes, stream);
      else if (M > 1) gated_few<ACT, 1, 1, 4, 3, false, 2>(a, s_x, gamma, N, Nd, y, slopes, stream);
      else if (deep) gated_few<ACT, 1, 1, 8, 3, false, 1>(a, s_x, gamma, N, Nd, y, slopes, stream);
      else gated_few<ACT, 1, 1, 4, 3, false, 1>(a, s_x, gamma, N, Nd, y, slopes, stream);
      return hipGetLastError();
    }
    if (M > 32) gated_few<ACT, 2, 4, 8, 1, true>(a, s_x, gamma, N, Nd, y, slopes, stream);
    else if (M > 16 && deep) gated_few<ACT, 1, 2, 8, 2, true>(a, s_x, gamma, N, Nd, y, slopes, stream);
    else if (M > 16) gated_few<ACT, 1, 2, 4, 2, true>(a, s_x, gamma, N, Nd, y, slopes, stream);
    else if (M > 2 && deep) gated_few<ACT, 1, 1, 8, 3, true>(a, s_x, gamma, N, Nd, y, slopes, stream);
    else if (M > 2) gated_few<ACT, 1, 1, 4, 3, true>(a, s_x, gamma, N, Nd, y, slopes, stream);
    else if (deep) gated_few<ACT, 1, 1, 8, 3, false>(a, s_x, gamma, N, Nd, y, slopes, stream);
    else gated_few<ACT, 1, 1, 4, 3, false>(a, s_x, gamma, N, Nd, y, slopes, stream);
    return hipGetLastError();
  }
  if (form == kMid1) return gated_mid<ACT, 1, 4>(w_packed, x_q, s_x, gamma, M, N, Kp, y, slopes, stream);
  if (form == kMid2) return gated_mid<ACT, 2, 2>(w_packed, x_q, s_x, gamma, M, N, Kp, y, slopes, stream);
  GatedCodesLoader pl;
  pl.packed = w_packed;
  pl.pitch = Kp / 4;
  pl.rows = 2 * N;
  pl.N = N;
  const CopyLoader<1, true> ql{reinterpret_cast<const char*>(x_q), Kp, M, Kp};
  const GemmShape g = fwd_shape(M, N, K);
  if (slopes != nullptr)
    return run_gemm<MfmaI8, 1>(pl, ql, GatedEpilogue<ACT, true>{y, slopes, s_x, gamma, N, Nd, M}, g, ws, ws_bytes, stream);
  return run_gemm<MfmaI8, 1>(pl, ql, GatedEpilogue<ACT, false>{y, nullptr, s_x, gamma, N, Nd, M}, g, ws, ws_bytes, stream);
}

hipError_t launch_gated_fwd(bool relu2, const uint16_t* x, const int8_t* x_q, const float* s_x, const uint8_t* w_packed,
                            const float* gamma, int64_t M, int64_t N, int64_t K, uint16_t* y, uint16_t* slopes, void* ws,
                            size_t ws_bytes, hipStream_t stream) {
  return relu2 ? gated_fwd<ActRelu2>(x, x_q, s_x, w_packed, gamma, M, N, K, y, slopes, ws, ws_bytes, stream)
               : gated_fwd<ActSilu>(x, x_q, s_x, w_packed, gamma, M, N, K, y, slopes, ws, ws_bytes, stream);
}

// The backward's workspace: D, the transposed codes, x_hat, then the products'
// split tiles.
struct GatedWs {
  size_t d, wt, xhat, split;
};
static size_t up256(size_t n) { return (n + 255) / 256 * 256; }
static GatedWs gated_ws(int64_t M, int64_t N, int64_t K) {
  const int64_t Kp = k_pad(K), Nd = n_half(N);
  const GemmShape g1 = shape_of(GemmKind::kBwdDx, M, 2 * Nd, K), g2 = shape_of(GemmKind::kBwdDw, M, 2 * Nd, K);
  const int cus = device_cus();
  const PairPlan pp = plan_pair(g1, g2, cus, kDxCosts, kDwCosts);
  return {up256((size_t)M * 4 * Nd), up256((size_t)Kp * Nd), up256((size_t)M * Kp * 2),
          std::max(pp.k1 == 0 ? 0 : pp.s1 + pp.s2,
                   std::max(split_workspace(g1, split_grid(g1, cus)), split_workspace(g2, split_grid(g2, cus))))};
}
size_t gated_bwd_workspace(int64_t M, int64_t N, int64_t K) {
  const GatedWs w = gated_ws(M, N, K);
  return w.d + w.wt + w.xhat + w.split;
}

template <bool OUT_F32>
static hipError_t gated_products(const uint16_t* D, const uint8_t* wt, const uint16_t* xhat, const float* gamma,
                                 const float* s_x, int64_t M, int64_t N, int64_t K, uint16_t* dX, void* dWg, void* dWu, char* ws,
                                 size_t ws_bytes, hipStream_t stream) {
  const int64_t Kp = k_pad(K), Nd = n_half(N), J = 2 * Nd;
  const GemmShape g1 = shape_of(GemmKind::kBwdDx, M, J, K), g2 = shape_of(GemmKind::kBwdDw, M, J, K);
  const RowCodesLoader<CodesFp4Frags> p1{wt, J / 2, Kp};
  const CopyLoader<2, true> q1{reinterpret_cast<const char*>(D), 2 * J, M, 2 * J};
  const TokenEpilogue e1{dX, s_x, K, M};
  const RowCopyBf16Loader<1> p2{xhat, Kp, M, Kp};
  const RowCopyBf16Loader<5> q2{D, J, M, J};
  const HalvesEpilogue<OUT_F32> e2{{dWg, dWu}, gamma, K, N, Nd};
  const bool dx = dX != nullptr && !few(M), dw = dWg != nullptr;  // few tokens' dX has a kernel of its own
  if (dX != nullptr && !dx)
    if (hipError_t e = launch_dx_skinny(wt, D, nullptr, s_x, M, J, K, dX, stream)) return e;
  if (!dx && !dw) return hipSuccess;
  if (const int fj = mid_bwd_blocks(g1, g2, dx, dw, pair_pays(g1, g2), M, K, J)) {
    const MidFp4<TileRow> lp1{{}, wt, Kp, J / 2, {0, Kp}};
    const MidRows<TileRow> lq1{{}, D, M, 2 * J, {0, M}};
    const MidOut<2> m1{dX, K, M, s_x};
    const MidCols lp2{xhat, M, Kp, Kp, 0}, lq2{D, M, J, J, 0};
    const MidHalves<OUT_F32 ? 4 : 2> m2{{dWg, dWu}, gamma, K, N, Nd};
    return fj == 1 ? mid_products_at<1, 4>(lp1, lq1, m1, lp2, lq2, m2, dx, dw, M, K, J, J, stream)
                   : mid_products_at<2, 2>(lp1, lq1, m1, lp2, lq2, m2, dx, dw, M, K, J, J, stream);
  }
  if (dx && dw && pair_pays(g1, g2)) {
    const hipError_t e = run_pair<1, 0>(p1, q1, e1, g1, kDxCosts, p2, q2, e2, g2, kDwCosts, ws, ws_bytes, stream);
    if (e != hipErrorNotSupported) return e;
  }
  if (dx)
    if (hipError_t e = run_gemm<MfmaBf16, 1>(p1, q1, e1, g1, ws, ws_bytes, stream)) return e;
  return dw ? run_gemm<MfmaBf16, 0>(p2, q2, e2, g2, ws, ws_bytes, stream) : hipSuccess;
}

hipError_t launch_gated_bwd(const uint16_t* dY, const uint16_t* slopes, const int8_t* x_q, const float* s_x,
                            const uint8_t* w_packed, const float* gamma, int64_t M, int64_t N, int64_t K, uint16_t* dX,
                            void* dWg, void* dWu, bool dw_f32, void* ws, size_t ws_bytes, hipStream_t stream) {
  const int64_t Kp = k_pad(K), Nd = n_half(N);
  const GatedWs w = gated_ws(M, N, K);
  char* base = static_cast<char*>(ws);
  uint16_t* D = reinterpret_cast<uint16_t*>(base);
  uint8_t* wt = reinterpret_cast<uint8_t*>(base + w.d);
  uint16_t* xhat = reinterpret_cast<uint16_t*>(base + w.d + w.wt);
  char* split = base + w.d + w.wt + w.xhat;
  const size_t split_bytes = ws_bytes - (w.d + w.wt + w.xhat);

  const GatedD d{dY, slopes, gamma, s_x, M * (Nd / 8), (int)N, (int)Nd, D};
  const int wt_bx = dX != nullptr ? (int)(Kp / 64) : 0, wt_by = (int)((2 * Nd + 255) / 256);
  const int64_t want = (M * (Kp / 16) + 255) / 256;
  const int xhat_nb = dWg != nullptr ? (int)std::min<int64_t>(want, 4096) : 0;
  const int64_t grid = wt_bx * wt_by + xhat_nb + (d.total + 255) / 256;
  gated_prep_kernel<<<(unsigned)grid, 256, 0, stream>>>(w_packed, N, Kp, Nd, wt, wt_bx, wt_by, x_q, M, xhat, xhat_nb, d);
  if (hipError_t e = hipGetLastError()) return e;
  return dw_f32 ? gated_products<true>(D, wt, xhat, gamma, s_x, M, N, K, dX, dWg, dWu, split, split_bytes, stream)
                : gated_products<false>(D, wt, xhat, gamma, s_x, M, N, K, dX, dWg, dWu, split, split_bytes, stream);
}

}  // namespace bitnet
