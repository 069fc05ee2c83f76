// MFMA GEMMs of the BitLinear layer for gfx950 (CDNA4, wave64).
//
// All three products are computed by one kernel template
//
//     C[i][j] = sum_r P[i][r] * Q[j][r],      output O[j][i] (i contiguous)
//
// with both operand tiles staged in LDS, 64 bf16 or 128 int8 reduction
// values per row per stage:
//
//   forward  y[m][n]  = sum_k x_q[m][k] q[n][k]        i = n, j = m, r = k
//            P = the 2-bit codes as stored (expanded to int8 after the
//            fragment read), Q = x_q copied; v_mfma_i32_32x32x32_i8, exact
//            int32 accumulation
//   dX       dX[m][k] = sum_n dY[m][n] W_hat[n][k]     i = k, j = m, r = n
//            P = the codes transposed to fp4 [k][n] by a pre-pass (expanded
//            to bf16 +-1, 0 after the fragment read), Q = dY copied;
//            v_mfma_f32_32x32x16_bf16; bf16(gamma) applied in the epilogue
//            (exact: q * bf16(gamma) is exact in bf16)
//   dW       dW[n][k] = sum_m dY[m][n] x_hat[m][k]     i = k, j = n, r = m
//            P = bf16 x_hat built by a pre-pass, Q = dY, both staged in
//            their [m][.] orientation and read transposed from LDS
//            (ds_read_b64_tr_b16); v_mfma_f32_32x32x16_bf16
//
// ("bitnet-qat-train": opening bullets - INT8 forward, backward operands
// rebuilt transiently from the 2-bit / INT8 state; Semantics - forward
// formula and STE backward dX = dY W_hat, dW = dY^T x_hat.)
//
// The LDS traffic, not the MFMA rate, bounds these kernels on gfx950 (about
// 128 B/clk/CU of 16-byte reads and 64 B/clk/CU of 16-byte writes), so the
// ternary operand stays 2-bit in LDS and is expanded in registers.
//
// Block tile 256 x 256, 4 waves (one per SIMD) in a 2 x 2 grid, wave tile
// 128 x 128 = 4 x 4 fragments of 32 x 32 (256 accumulator registers per
// lane, held in AGPRs). Two LDS stages (one barrier per stage); while the
// MFMAs of stage s run, the registers holding stage s+1 are converted and
// stored into the other LDS buffer and stage s+2 is fetched into them, one
// quarter per k-step.
//
// MFMA 32x32 output layout (both instructions): lane l, accumulator element
// v holds row i = 8*(v/4) + 4*(l/32) + (v%4), column j = l%32. Operand
// fragments: lane l supplies 16 bytes of row (l%32) of its operand for lane
// half h = l/32 of the k-step; which reduction values those are (red_chunk)
// is the same for P and Q of a GEMM, so the hardware's internal order of the
// reduction index within a step does not matter.

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdlib>
#include <mutex>
#include <random>
#include <type_traits>

#include "bwd_prep.h"
#include "gemm_split.h"

namespace bitnet {

__global__ __launch_bounds__(256) void xhat_kernel(const int8_t* __restrict__ xq, const float* __restrict__ s,
                                                   int64_t M, int64_t Kp, uint16_t* __restrict__ xhat) {
  xhat_blocks(xq, s, M, Kp, xhat, blockIdx.x, gridDim.x);
}

__device__ __forceinline__ void wt_fp4_xcd(const uint8_t* __restrict__ packed, int64_t N, int64_t Kp, int64_t Np,
                                           uint8_t* __restrict__ wt, int b, int wt_bx, int wt_by) {
  const int v = xcd_major(b, wt_bx * wt_by);
  wt_fp4_block(packed, [N](int64_t n) { return n < N ? n : int64_t(-1); }, Kp, Np, wt, v % wt_bx, v / wt_bx);
}

__global__ __launch_bounds__(256) void wt_fp4_kernel(const uint8_t* __restrict__ packed, int64_t N, int64_t Kp,
                                                     int64_t Np, uint8_t* __restrict__ wt, int wt_bx, int wt_by) {
  wt_fp4_xcd(packed, N, Kp, Np, wt, blockIdx.x, wt_bx, wt_by);
}

// Both backward pre-passes in one launch: the first wt_bx * wt_by blocks
// transpose the codes, the other xhat_nb blocks build x_hat (the two are
// independent, and the transpose is ALU-heavy while x_hat is HBM-heavy).
__global__ __launch_bounds__(256) void bwd_prep_kernel(const uint8_t* __restrict__ packed, int64_t N, int64_t Kp,
                                                       int64_t Np, uint8_t* __restrict__ wt, int wt_bx, int wt_by,
                                                       const int8_t* __restrict__ xq, const float* __restrict__ s,
                                                       int64_t M, uint16_t* __restrict__ xhat, int xhat_nb) {
  const int b = blockIdx.x, nwt = wt_bx * wt_by;
  if (b < nwt)
    wt_fp4_xcd(packed, N, Kp, Np, wt, b, wt_bx, wt_by);
  else
    xhat_blocks(xq, s, M, Kp, xhat, b - nwt, xhat_nb);
}

// The bias values of the output tile being computed (FwdEpilogue<true>),
// staged once per tile before its main loop so that the epilogue reads
// them from LDS: each lane needs 16 groups of 4 per tile and reads each of
// them in all four column passes.
__shared__ __attribute__((aligned(16))) uint16_t s_tile_bias[kBI];

// BIAS: a bf16 bias [N] is added before the rounding (a separate
// instantiation, so that the plain epilogue keeps its registers).
template <bool BIAS>
struct FwdEpilogue {
  uint16_t* y;
  int32_t* acc_out;  // NULL: not written
  const float* s;
  const float* gamma;
  int64_t I, J;          // N, M
  const uint16_t* bias;  // [N] bf16 (BIAS only)

  // The scales this lane's columns need, loaded before the main loop so
  // that their latency is hidden (raw values; combined in store()).
  struct Pre { float g; float sj[kFJ]; };
  __device__ __forceinline__ Pre prefetch(int j0, int lane) const {
    Pre pre;
    pre.g = *gamma;
#pragma unroll
    for (int fj = 0; fj < kFJ; ++fj) {
      const int64_t j = j0 + 32 * fj + (lane & 31);
      pre.sj[fj] = j < J ? s[j] : 0.0f;
    }
    return pre;
  }
  static constexpr int kWaveLds = EpStage<4>::kWaveBytes;  // the int32 pass needs the larger buffer
  static constexpr bool kStagesBias = BIAS;
  // bias[ti0 .. ti0 + kBI) into s_tile_bias (zeros past I); called by every
  // thread of the block, after a barrier that ends the previous tile's
  // epilogue and before the main loop's barriers that order it before this
  // tile's epilogue
  __device__ __forceinline__ void stage_bias(int ti0) const {
    const int t = threadIdx.x;
    if (t < kBI / 8) {
      const int64_t n = (int64_t)ti0 + 8 * t;
      uint4 v;
      if (n + 8 <= I) {
        v = *reinterpret_cast<const uint4*>(bias + n);
      } else {
        uint32_t d[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t lo = n + 2 * e < I ? bias[n + 2 * e] : 0u;
          const uint32_t hi = n + 2 * e + 1 < I ? bias[n + 2 * e + 1] : 0u;
          d[e] = lo | (hi << 16);
        }
        v = make_uint4(d[0], d[1], d[2], d[3]);
      }
      *reinterpret_cast<uint4*>(s_tile_bias + 8 * t) = v;
    }
  }
  __device__ __forceinline__ void store(MfmaI8::Acc (&acc)[kFI][kFJ], const Pre& pre, int i0, int j0,
                                        int lane, char* wlds) const {
    const float g = pre.g;
#pragma unroll
    for (int fj = 0; fj < kFJ; ++fj) {
      const float c = pre.sj[fj] * g / 127.0f;
#pragma unroll
      for (int fi = 0; fi < kFI; ++fi)
#pragma unroll
        for (int gi = 0; gi < 4; ++gi) {
          float v0 = (float)acc[fi][fj][4 * gi] * c, v1 = (float)acc[fi][fj][4 * gi + 1] * c;
          float v2 = (float)acc[fi][fj][4 * gi + 2] * c, v3 = (float)acc[fi][fj][4 * gi + 3] * c;
          if constexpr (BIAS) {  // n = i0 + 32fi + 8gi + 4h + 0..3 (EpStage::put); tiles start at multiples of kBI
            const uint2 b = *reinterpret_cast<const uint2*>(s_tile_bias + (i0 % kBI) + 32 * fi + 8 * gi +
                                                           4 * (lane >> 5));
            v0 += bf16_lo(b.x); v1 += bf16_hi(b.x); v2 += bf16_lo(b.y); v3 += bf16_hi(b.y);
          }
          EpStage<2>::put(wlds, lane, fi, gi, make_uint2(pack_bf16x2(v0, v1), pack_bf16x2(v2, v3)));
        }
      EpStage<2>::drain(wlds, reinterpret_cast<char*>(y), I, J, i0, j0 + 32 * fj, lane);
      if (acc_out != nullptr) {
#pragma unroll
        for (int fi = 0; fi < kFI; ++fi)
#pragma unroll
          for (int gi = 0; gi < 4; ++gi)
            EpStage<4>::put(wlds, lane, fi, gi,
                            make_uint4((uint32_t)acc[fi][fj][4 * gi], (uint32_t)acc[fi][fj][4 * gi + 1],
                                       (uint32_t)acc[fi][fj][4 * gi + 2], (uint32_t)acc[fi][fj][4 * gi + 3]));
        EpStage<4>::drain(wlds, reinterpret_cast<char*>(acc_out), I, J, i0, j0 + 32 * fj, lane);
      }
    }
  }
};

// dW as 1-bit signs for sign-based optimisers ("1BitTraining.md", closing
// paragraphs: the identity-STE gradient has the sign of the gradient with
// respect to the quantised weight, so a sign optimiser needs only 1 bit per
// weight). out [J][Ip/8] bytes (Ip = Kp): bit b of byte c of row j is set
// iff the fp32 sum for element (j, 8c + b) is negative (zero sums, and the
// zero sums of the padding columns, give 0). Nothing is staged: the lane of
// row j = l % 32 holds, per fragment fi and group g, the sums of
// i = 32fi + 8g + 4h + 0..3 (h = l / 32). Their flags form a nibble, and the
// nibbles of lanes l and l ^ 32 make the bytes of i = 32fi + 8g .. +7; lane
// half h then stores the 8 bytes of i = 64h .. 64h + 63 of the wave tile.
struct Sign1Epilogue {
  uint8_t* out;
  int64_t Ip, J;  // Kp, N

  struct Pre {};
  static constexpr int kWaveLds = 0;
  __device__ __forceinline__ Pre prefetch(int, int) const { return Pre{}; }
  __device__ __forceinline__ void store(MfmaBf16::Acc (&acc)[kFI][kFJ], const Pre&, int i0, int j0, int lane,
                                        char*) const {
    const int h = lane >> 5;
#pragma unroll
    for (int fj = 0; fj < kFJ; ++fj) {
      uint32_t word[kFI];
#pragma unroll
      for (int fi = 0; fi < kFI; ++fi) {
        uint32_t mine = 0;  // flag of i = 32fi + 8g + 4h + e at bit 4g + e
#pragma unroll
        for (int r = 0; r < 16; ++r) mine |= (acc[fi][fj][r] < 0.0f ? 1u : 0u) << r;
        const uint32_t other = (uint32_t)__shfl_xor((int)mine, 32, kWave);
        const uint32_t lo = h ? other : mine, hi = h ? mine : other;
        uint32_t w = 0;
#pragma unroll
        for (int g = 0; g < 4; ++g) w |= (((lo >> (4 * g)) & 0xFu) | (((hi >> (4 * g)) & 0xFu) << 4)) << (8 * g);
        word[fi] = w;
      }
      const int64_t j = j0 + 32 * fj + (lane & 31);
      const int64_t i = i0 + 64 * h;
      if (j < J && i < Ip)
        *reinterpret_cast<uint2*>(out + j * (Ip / 8) + i / 8) =
            h ? make_uint2(word[2], word[3]) : make_uint2(word[0], word[1]);
    }
  }
};

// TTQ dW ("TTQ_VERIFICATION.md": Backward Pass, a straight-through
// estimator, and Bugs Fixed item 5, the gradient of Wp as a masked sum).
// dW = dY^T x is written as Bf16Epilogue writes it (the latent weight gets
// the quantized weight's gradient unchanged). With partials set, each wave
// also adds up its fp32 sums, before any rounding, over the positions whose
// code is +1 and over those whose code is -1, and writes the two totals to
// partials[wave tile] (one float2 per 128 x 128 wave tile, row-major over
// the wave-tile grid; every entry is written once per call, so nothing
// needs clearing). ttq_grads_kernel adds them up in a fixed order.
//
// Lane l holds k = i0 + 32fi + 8g + 4h + e (h = l/32, e < 4) of row
// n = j0 + 32fj + l%32. i0 + 32fi is a multiple of 32, so the codes of those
// 32 k are the two 32-bit words at byte (i0 + 32fi)/4 of row n (8 bytes,
// one load), and code k sits in word g/2 at bit 8e + 2(2(g%2) + h) (code j
// of a word at bit 8(j%4) + 2(j/4), j = k % 16).
template <bool OUT_F32>
struct TtqDwEpilogue {
  Bf16Epilogue<OUT_F32> out;  // dW [J][I], unscaled
  const uint8_t* codes;       // [J][code_pitch]
  uint32_t code_pitch;        // Kp / 4 bytes
  float2* partials;           // NULL: no sums
  int wtiles_i;               // wave tiles along i

  typedef typename Bf16Epilogue<OUT_F32>::Pre Pre;
  static constexpr int kWaveLds = Bf16Epilogue<OUT_F32>::kWaveLds;
  __device__ __forceinline__ Pre prefetch(int j0, int lane) const { return out.prefetch(j0, lane); }
  __device__ __forceinline__ void store(MfmaBf16::Acc (&acc)[kFI][kFJ], const Pre& pre, int i0, int j0, int lane,
                                        char* wlds) const {
    if (partials == nullptr) {
      out.store(acc, pre, i0, j0, lane, wlds);
      return;
    }
    const int h = lane >> 5;
    // rows past J fall outside the resource; words past the row's end get an
    // out-of-range offset (zeros: no code)
    const rsrc_t rs = make_rsrc(codes, (uint32_t)out.J * code_pitch);
    uint2 c[kFI][kFJ];
#pragma unroll
    for (int fj = 0; fj < kFJ; ++fj) {
      const uint32_t n = (uint32_t)(j0 + 32 * fj + (lane & 31));
#pragma unroll
      for (int fi = 0; fi < kFI; ++fi) {
        const uint32_t col = (uint32_t)(i0 + 32 * fi) / 4;
        c[fi][fj] = buf_load8(rs, col < code_pitch ? n * code_pitch + col : kOob);
      }
    }
    out.store(acc, pre, i0, j0, lane, wlds);
    float sp = 0.0f, sn = 0.0f;
#pragma unroll
    for (int fi = 0; fi < kFI; ++fi)
#pragma unroll
      for (int fj = 0; fj < kFJ; ++fj)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint32_t w = (g < 2 ? c[fi][fj].x : c[fi][fj].y) >> (4 * (g & 1) + 2 * h);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t code = (w >> (8 * e)) & 3u;
            const float v = acc[fi][fj][4 * g + e];
            sp += code == 1u ? v : 0.0f;
            sn += code == 3u ? v : 0.0f;
          }
        }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      sp += __shfl_xor(sp, off, kWave);
      sn += __shfl_xor(sn, off, kWave);
    }
    if (lane == 0) partials[(j0 / kWTJ) * wtiles_i + i0 / kWTI] = make_float2(sp, sn);
  }
};

// The two scale gradients from the wave-tile partials: grads[0] = sum of the
// +1 sums (dL/dWp), grads[1] = -(sum of the -1 sums) (dL/dWn: the weight
// there is -Wn). Thread t adds partials t, t + 256, ... in fp64, then the
// block adds the thread sums in a fixed order; rounded once to fp32.
__global__ __launch_bounds__(256) void ttq_grads_kernel(const float2* __restrict__ partials, int count,
                                                        float* __restrict__ grads) {
  double p = 0.0, n = 0.0;
  for (int i = threadIdx.x; i < count; i += 256) {
    const float2 v = partials[i];
    p += (double)v.x;
    n += (double)v.y;
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    p += __shfl_xor(p, off, kWave);
    n += __shfl_xor(n, off, kWave);
  }
  __shared__ double sp[4], sn[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (lane == 0) {
    sp[wave] = p;
    sn[wave] = n;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    grads[0] = (float)((sp[0] + sp[1]) + (sp[2] + sp[3]));
    grads[1] = (float)(-((sn[0] + sn[1]) + (sn[2] + sn[3])));
  }
}

// dW for few tokens (M <= 64, N % 8 == 0): dW[n][k] = sum_{m < M} dY[m][n] *
// x_hat[m][k] ("bitnet-qat-train", Semantics). The reduction is at most 4
// MFMA steps of 16 tokens, so the cost is writing dW: small output tiles
// (64 n x 256 k per workgroup) keep every CU busy with several tiles whose
// loads and stores overlap. The tile's slice of x_hat is converted from
// x_q and s on the way into LDS (xhat16, the pre-pass's arithmetic), so no
// pre-pass runs and the tiles can share a launch with the code transpose
// that the few-token dX needs. Both operands are staged as stored, rows m
// in LDS (rows m >= M as zeros), and read transposed with
// ds_read_b64_tr_b16 (TrFrags): A = x_hat columns k (wave k half 128wk +
// 32f, f < 4), B = dY columns n (wave n half 32wn). D[k][n] goes back
// through LDS as rows n and is written as 16-byte row pieces (element by
// element when K does not keep them aligned). Products are exact in fp32
// and each sum runs in token order. Tile b of ktiles x ceil(N / 64), 256
// threads.
template <bool OUT_F32>
__device__ __forceinline__ void dw_skinny_tile(const int8_t* __restrict__ xq, const float* __restrict__ sx,
                                               const uint16_t* __restrict__ dY, int M, int64_t N, int64_t Kp,
                                               int64_t K, int ktiles, void* __restrict__ dW, int b) {
  constexpr int kEB = OUT_F32 ? 4 : 2;
  constexpr int kOutPitch = 256 * kEB + 16;
  constexpr int kYPitch = 64 * 2 + 16;     // dY rows: 64 n, padded
  constexpr int kXB = 64 * kTrPitch;       // 64 token rows of x_hat
  constexpr int kInB = kXB + 64 * kYPitch;
  constexpr int kOutB = 64 * kOutPitch;
  __shared__ __attribute__((aligned(16))) char smem[kInB > kOutB ? kInB : kOutB];
  char* xs = smem;        // x_hat [m][256 k]
  char* ys = smem + kXB;  // dY [m][64 n]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t k0 = (int64_t)(b % ktiles) * 256, n0 = (int64_t)(b / ktiles) * 64;
  const int ms = (M + 15) / 16;  // MFMA steps of 16 tokens

  const rsrc_t rxq = make_rsrc(xq, (uint32_t)(M * Kp));
  const rsrc_t rdy = make_rsrc(dY, (uint32_t)(M * N * 2));
  uint4 vq[4], vy[2];
  float rq[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // x_q: rows m < 64, 16 pieces of 16 bytes per row
    const int e = tid + 256 * i, m = e >> 4;
    const int64_t k = k0 + 16 * (e & 15);
    vq[i] = buf_load16(rxq, m < M && k < Kp ? (uint32_t)(m * Kp + k) : kOob);
    rq[i] = m < M ? sx[m] / 127.0f : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // dY: rows m < 64, 8 pieces per row
    const int e = tid + 256 * i, m = e >> 3;
    const int64_t n = n0 + 8 * (e & 7);
    vy[i] = buf_load16(rdy, m < M && n < N ? (uint32_t)((m * N + n) * 2) : kOob);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // zeros past M (and past Kp) convert to 0
    const int e = tid + 256 * i;
    if ((e >> 4) < 16 * ms) {
      uint4 lo, hi;
      xhat16(vq[i], rq[i], lo, hi);
      char* dst = xs + (e >> 4) * kTrPitch + 32 * (e & 15);
      *reinterpret_cast<uint4*>(dst) = lo;
      *reinterpret_cast<uint4*>(dst + 16) = hi;
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = tid + 256 * i;
    if ((e >> 3) < 16 * ms) *reinterpret_cast<uint4*>(ys + (e >> 3) * kYPitch + 16 * (e & 7)) = vy[i];
  }
  __syncthreads();

  const int wn = wave & 1, wk = wave >> 1;
  TrFrags fa;
  TrFragsP<kYPitch> fb;
  fa.init(xs, 128 * wk, lane);
  fb.init(ys, 32 * wn, lane);
  MfmaBf16::Acc acc[4];
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[f][e] = 0.0f;
  const auto step = [&](auto ks) {
    constexpr int KS = decltype(ks)::value;
    fb.template read<KS>(0);
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      fa.template read<KS>(f);
      acc[f] = MfmaBf16::mma(fa.template frag<KS>(f), fb.template frag<KS>(0), acc[f]);
    }
  };
  step(std::integral_constant<int, 0>());
  if (ms > 1) step(std::integral_constant<int, 1>());
  if (ms > 2) step(std::integral_constant<int, 2>());
  if (ms > 3) step(std::integral_constant<int, 3>());
  __syncthreads();

  // D[k][n]: lane column n = 32wn + l % 32, rows k = 128wk + 32f + 8g + 4h + 0..3
  const int nl = 32 * wn + (lane & 31), h = lane >> 5;
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      char* dst = smem + nl * kOutPitch + (128 * wk + 32 * f + 8 * g + 4 * h) * kEB;
      const float v0 = acc[f][4 * g], v1 = acc[f][4 * g + 1], v2 = acc[f][4 * g + 2], v3 = acc[f][4 * g + 3];
      if constexpr (OUT_F32)
        *reinterpret_cast<uint4*>(dst) = make_uint4(__float_as_uint(v0), __float_as_uint(v1), __float_as_uint(v2),
                                                    __float_as_uint(v3));
      else
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(v0, v1), pack_bf16x2(v2, v3));
    }
  __syncthreads();
  constexpr int kPieces = 256 * kEB / 16;  // 16-byte pieces per output row of the tile
  constexpr int kPer = 16 / kEB;           // elements per piece
  char* out = static_cast<char*>(dW);
#pragma unroll
  for (int i = 0; i < 64 * kPieces / 256; ++i) {
    const int e = tid + 256 * i, r = e / kPieces, c = e % kPieces;
    const int64_t n = n0 + r, k = k0 + kPer * c;
    if (n >= N || k >= K) continue;
    const char* src = smem + r * kOutPitch + 16 * c;
    if (K % kPer == 0) {
      *reinterpret_cast<uint4*>(out + (n * K + k) * kEB) = *reinterpret_cast<const uint4*>(src);
    } else {
      for (int j = 0; j < kPer && k + j < K; ++j) {
        if constexpr (OUT_F32)
          reinterpret_cast<uint32_t*>(out)[n * K + k + j] = reinterpret_cast<const uint32_t*>(src)[j];
        else
          reinterpret_cast<uint16_t*>(out)[n * K + k + j] = reinterpret_cast<const uint16_t*>(src)[j];
      }
    }
  }
}

template <bool OUT_F32>
__global__ __launch_bounds__(256) void dw_skinny_kernel(const int8_t* __restrict__ xq, const float* __restrict__ sx,
                                                        const uint16_t* __restrict__ dY, int M, int64_t N,
                                                        int64_t Kp, int64_t K, int ktiles, void* __restrict__ dW) {
  dw_skinny_tile<OUT_F32>(xq, sx, dY, M, N, Kp, K, ktiles, dW, blockIdx.x);
}

// Few tokens with both outputs, first launch: the first wt_bx * wt_by blocks
// transpose the codes to fp4 for the few-token dX (which runs next), the
// others compute dW tiles (independent of the transpose: ALU- and
// latency-bound work next to the HBM writes of dW).
template <bool OUT_F32>
__global__ __launch_bounds__(256) void bwd_skinny_front_kernel(const uint8_t* __restrict__ packed, int64_t Np,
                                                               uint8_t* __restrict__ wt, int wt_bx, int wt_by,
                                                               const int8_t* __restrict__ xq,
                                                               const float* __restrict__ sx,
                                                               const uint16_t* __restrict__ dY, int M, int64_t N,
                                                               int64_t Kp, int64_t K, int ktiles,
                                                               void* __restrict__ dW) {
  const int b = blockIdx.x, nwt = wt_bx * wt_by;
  if (b < nwt)
    wt_fp4_xcd(packed, N, Kp, Np, wt, b, wt_bx, wt_by);
  else
    dw_skinny_tile<OUT_F32>(xq, sx, dY, M, N, Kp, K, ktiles, dW, b - nwt);
}

// ---------------------------------------------------------------------------
// Host side: choice of the split, workspace, launch.
// ---------------------------------------------------------------------------

TestKnobs& test_knobs() {
  static TestKnobs knobs;
  return knobs;
}

hipError_t take_split_timeouts(unsigned int* count) {
  unsigned int gated = 0, int8 = 0;
  if (hipError_t e = take_local_split_timeouts(count)) return e;
  if (hipError_t e = take_gated_split_timeouts(&gated)) return e;
  if (hipError_t e = take_int8_split_timeouts(&int8)) return e;
  *count += gated + int8;
  return hipSuccess;
}

int64_t debug_split_pieces(int64_t T, int S, int G, int32_t* v, int32_t* t, int32_t* s0, int32_t* s1,
                           int64_t* slot, int32_t* va, int32_t* n, int64_t cap) {
  SplitPlan p{};
  p.total = T * S;
  p.grid = G;
  p.nstages = S;
  p.nslots = partial_slots(T, G);
  int64_t k = 0;
  for (int w = 0; w < G; ++w) {
    const int64_t hi = split_lo(p, w + 1);
    for (int64_t it = split_lo(p, w); it < hi;) {
      int tt, a, b, o, c;
      split_piece(p, it, hi, &tt, &a, &b);
      split_tile_owners(p, tt, &o, &c);
      if (k < cap) {
        v[k] = w;
        t[k] = tt;
        s0[k] = a;
        s1[k] = b;
        slot[k] = piece_slot(p, w, tt);
        va[k] = o;
        n[k] = c;
      }
      ++k;
      it += b - a;
    }
  }
  return k;
}

void debug_cta_order(int G, int32_t* out) {
  for (int b = 0; b < G; ++b) out[b] = cta_order(b, G);
}

// TTQ backward: the wave-tile partials of the scale gradients come first.
static int64_t ttq_wave_tiles(int64_t N, int64_t K) {
  const GemmShape g = shape_of(GemmKind::kBwdDw, 1, N, K);
  return 4 * g.tiles();
}
static size_t ttq_partials_bytes(int64_t N, int64_t K) {
  return ((size_t)ttq_wave_tiles(N, K) * sizeof(float2) + 255) / 256 * 256;
}

// Launch tags: a 48-bit counter started at a random value, so tags of
// different launches (and processes) differ.
static uint64_t next_gen() {
  static std::atomic<uint64_t> gen{0};
  static std::once_flag once;
  std::call_once(once, [] {
    std::random_device rd;
    gen.store(((uint64_t)rd() << 20) ^ (uint64_t)rd());
  });
  uint64_t g;
  do {
    g = gen.fetch_add(1) & ((uint64_t(1) << 48) - 1);
  } while (g == 0);
  return g;
}

uint64_t next_launch_tag() { return next_gen(); }

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------

// Few tokens run the decode-shaped kernels (the no_skinny test knob keeps
// the large-M GEMMs at any M).
static bool skinny(int64_t M) {
  return M <= kSkinnyMaxM && test_knobs().no_skinny.load(std::memory_order_relaxed) == 0;
}

hipError_t launch_fwd(const int8_t* x_q, const float* s_x, const uint8_t* w_packed,
                      const float* gamma, const uint16_t* bias, int64_t M, int64_t N, int64_t K, uint16_t* y,
                      int32_t* acc_out, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (skinny(M))
    return launch_fwd_skinny(x_q, s_x, w_packed, gamma, bias, M, N, K, y, acc_out, stream);
  const int64_t Kp = k_pad(K);
  PackedCodesLoader pl{w_packed, Kp / 4, N};
  CopyLoader<1, true> ql{reinterpret_cast<const char*>(x_q), Kp, M, Kp};
  if (bias != nullptr)
    return run_gemm<MfmaI8, 1>(pl, ql, FwdEpilogue<true>{y, acc_out, s_x, gamma, N, M, bias},
                               shape_of(GemmKind::kFwd, M, N, K), ws, ws_bytes, stream);
  return run_gemm<MfmaI8, 1>(pl, ql, FwdEpilogue<false>{y, acc_out, s_x, gamma, N, M, nullptr},
                             shape_of(GemmKind::kFwd, M, N, K), ws, ws_bytes, stream);
}

static hipError_t launch_wt(const uint8_t* w_packed, int64_t N, int64_t K, uint8_t* wt, hipStream_t stream) {
  const int64_t Kp = k_pad(K), Np = n_pad64(N);
  const int wt_bx = (int)(Kp / 64), wt_by = (int)((Np + 255) / 256);
  wt_fp4_kernel<<<wt_bx * wt_by, 256, 0, stream>>>(w_packed, N, Kp, Np, wt, wt_bx, wt_by);
  return hipGetLastError();
}

static hipError_t launch_xhat(const int8_t* x_q, const float* s_x, int64_t M, int64_t K, uint16_t* xhat,
                              hipStream_t stream) {
  const int64_t Kp = k_pad(K);
  const int64_t want = (M * (Kp / 16) + 255) / 256;
  xhat_kernel<<<(int)(want < 4096 ? want : 4096), 256, 0, stream>>>(x_q, s_x, M, Kp, xhat);
  return hipGetLastError();
}

hipError_t launch_bwd_dx(const uint16_t* dY, const uint8_t* w_packed, const float* gamma,
                         int64_t M, int64_t N, int64_t K, uint16_t* dX, void* ws, size_t ws_bytes,
                         hipStream_t stream) {
  const int64_t Kp = k_pad(K), Np = n_pad64(N);
  const size_t wb = wt_bytes(N, K);
  if (ws == nullptr || ws_bytes < wb) return hipErrorInvalidValue;  // the C ABI sized it
  uint8_t* wt = static_cast<uint8_t*>(ws);
  void* split_ws = static_cast<char*>(ws) + wb;
  const size_t split_bytes = ws_bytes - wb;
  if (hipError_t e = launch_wt(w_packed, N, K, wt, stream)) return e;
  if (skinny(M) && N % 8 == 0) return launch_dx_skinny(wt, dY, gamma, nullptr, M, N, K, dX, stream);

  const RowCodesLoader<CodesFp4Frags> pl{wt, Np / 2, Kp};
  Bf16Epilogue<false> ep{dX, gamma, K, M};
  const GemmShape g = shape_of(GemmKind::kBwdDx, M, N, K);
  if (N % 8 == 0) {
    CopyLoader<2, true> ql{reinterpret_cast<const char*>(dY), 2 * N, M, 2 * N};
    return run_gemm<MfmaBf16, 1>(pl, ql, ep, g, split_ws, split_bytes, stream);
  }
  CopyLoader<2, false> ql{reinterpret_cast<const char*>(dY), 2 * N, M, 2 * N};
  return run_gemm<MfmaBf16, 1>(pl, ql, ep, g, split_ws, split_bytes, stream);
}

// The dW product on x_hat (already built) with epilogue ep.
template <class EP>
static hipError_t run_dw(const uint16_t* dY, const uint16_t* xhat, int64_t M, int64_t N, int64_t K, const EP& ep,
                         void* split_ws, size_t split_bytes, hipStream_t stream) {
  const int64_t Kp = k_pad(K);
  const GemmShape g = shape_of(GemmKind::kBwdDw, M, N, K);
  if (N % 8 == 0) {
    // both operands copied in their memory orientation, fragments read transposed
    const RowCopyBf16Loader<1> pc{xhat, Kp, M, Kp};
    const RowCopyBf16Loader<5> qc{dY, N, M, N};
    return run_gemm<MfmaBf16, 0>(pc, qc, ep, g, split_ws, split_bytes, stream);
  }
  const RowTransposeBf16Loader<true, 3> pl{xhat, Kp, M, Kp};
  if (N % 4 == 0) return run_gemm<MfmaBf16, 0>(pl, RowTransposeBf16Loader<true, 5>{dY, N, M, N}, ep, g, split_ws, split_bytes, stream);
  return run_gemm<MfmaBf16, 0>(pl, RowTransposeBf16Loader<false, 5>{dY, N, M, N}, ep, g, split_ws, split_bytes, stream);
}

// The few-token dW (dw_skinny_kernel, x_hat converted in the kernel from x_q
// and s): N % 8 == 0, a bf16 or f32 output (the 1-bit output runs the
// large-M GEMM's epilogue).
static bool dw_skinny_ok(int64_t M, int64_t N, int64_t K, DwOut dw_out) {
  const int64_t dw_tiles = (k_pad(K) + 255) / 256 * ((N + 63) / 64);
  return skinny(M) && N % 8 == 0 && dw_out != DwOut::kSign1 && dw_tiles < (int64_t(1) << 31);
}
static hipError_t launch_dw_skinny(const int8_t* x_q, const float* s_x, const uint16_t* dY, int64_t M, int64_t N,
                                   int64_t K, void* dW, DwOut dw_out, hipStream_t stream) {
  const int64_t Kp = k_pad(K);
  const int ktiles = (int)((Kp + 255) / 256);
  const unsigned grid = (unsigned)((Kp + 255) / 256 * ((N + 63) / 64));
  if (dw_out == DwOut::kF32)
    dw_skinny_kernel<true><<<grid, 256, 0, stream>>>(x_q, s_x, dY, (int)M, N, Kp, K, ktiles, dW);
  else
    dw_skinny_kernel<false><<<grid, 256, 0, stream>>>(x_q, s_x, dY, (int)M, N, Kp, K, ktiles, dW);
  return hipGetLastError();
}

// Few tokens with both outputs: one bwd_skinny_front_kernel launch (the fp4
// transposed codes and every dW tile), then the few-token dX.
static bool skinny_both_ok(int64_t M, int64_t N, int64_t K, DwOut dw_out) {
  return dw_skinny_ok(M, N, K, dw_out);  // dx_skinny needs N % 8 == 0 as well
}
static hipError_t launch_skinny_front(const uint8_t* w_packed, const int8_t* x_q, const float* s_x,
                                      const uint16_t* dY, int64_t M, int64_t N, int64_t K, uint8_t* wt, void* dW,
                                      DwOut dw_out, hipStream_t stream) {
  const int64_t Kp = k_pad(K), Np = n_pad64(N);
  const int wt_bx = (int)(Kp / 64), wt_by = (int)((Np + 255) / 256);
  const int ktiles = (int)((Kp + 255) / 256);
  const unsigned grid = (unsigned)(wt_bx * wt_by + (Kp + 255) / 256 * ((N + 63) / 64));
  if (dw_out == DwOut::kF32)
    bwd_skinny_front_kernel<true><<<grid, 256, 0, stream>>>(w_packed, Np, wt, wt_bx, wt_by, x_q, s_x, dY, (int)M, N,
                                                            Kp, K, ktiles, dW);
  else
    bwd_skinny_front_kernel<false><<<grid, 256, 0, stream>>>(w_packed, Np, wt, wt_bx, wt_by, x_q, s_x, dY, (int)M, N,
                                                             Kp, K, ktiles, dW);
  return hipGetLastError();
}
static void launch_prep(const uint8_t* w_packed, const int8_t* x_q, const float* s_x, int64_t M, int64_t N,
                        int64_t K, uint8_t* wt, uint16_t* xhat, hipStream_t stream) {
  const int64_t Kp = k_pad(K), Np = n_pad64(N);
  const int wt_bx = (int)(Kp / 64), wt_by = (int)((Np + 255) / 256);
  const int64_t want = (M * (Kp / 16) + 255) / 256;
  const int xhat_nb = (int)(want < 4096 ? want : 4096);
  bwd_prep_kernel<<<wt_bx * wt_by + xhat_nb, 256, 0, stream>>>(w_packed, N, Kp, Np, wt, wt_bx, wt_by, x_q, s_x, M,
                                                               xhat, xhat_nb);
}

hipError_t launch_bwd_dw(const uint16_t* dY, const int8_t* x_q, const float* s_x, int64_t M,
                         int64_t N, int64_t K, void* dW, DwOut dw_out, void* ws, size_t ws_bytes,
                         hipStream_t stream) {
  if (dw_skinny_ok(M, N, K, dw_out)) return launch_dw_skinny(x_q, s_x, dY, M, N, K, dW, dw_out, stream);
  const size_t xb = xhat_bytes(M, K);
  if (ws == nullptr || ws_bytes < xb) return hipErrorInvalidValue;  // the C ABI sized it
  uint16_t* xhat = static_cast<uint16_t*>(ws);
  void* split_ws = static_cast<char*>(ws) + xb;
  const size_t split_bytes = ws_bytes - xb;
  if (hipError_t e = launch_xhat(x_q, s_x, M, K, xhat, stream)) return e;
  switch (dw_out) {
    case DwOut::kF32: return run_dw(dY, xhat, M, N, K, Bf16Epilogue<true>{dW, nullptr, K, N}, split_ws, split_bytes, stream);
    case DwOut::kSign1:
      return run_dw(dY, xhat, M, N, K, Sign1Epilogue{static_cast<uint8_t*>(dW), k_pad(K), N}, split_ws, split_bytes, stream);
    default: return run_dw(dY, xhat, M, N, K, Bf16Epilogue<false>{dW, nullptr, K, N}, split_ws, split_bytes, stream);
  }
}

static bool skinny(int64_t M);

// The STE backward products run in one launch when N % 8 == 0, there are
// more than a few tokens and each product would split its tiles on the full
// device anyway.
// The paired launch runs when both products are large enough that their
// split tails and fills are worth sharing: each would split when launched
// alone under a 3-stage piece cost (the gate under which the pair's own
// cost model, plan_pair, was measured; at 4096 x 6912 -> 2560 the pair
// takes 287 us where dX whole and dW split alone take 144 + 190 us).
static bool pair_gate(int64_t M, int64_t N, int64_t K) {
  const int cus = device_cus();
  GemmShape dx = shape_of(GemmKind::kBwdDx, M, N, K), dw = shape_of(GemmKind::kBwdDw, M, N, K);
  dx.overhead = dw.overhead = 3;
  return split_pays(dx, cus) > 0 && split_pays(dw, cus) > 0;
}
static bool pair_eligible(int64_t M, int64_t N, int64_t K) {
  return N % 8 == 0 && !skinny(M) && pair_gate(M, N, K);
}
// TTQ's pair: both operands copied as stored (row pitches multiples of 8).
static bool ttq_pair_eligible(int64_t M, int64_t N, int64_t K, int64_t ldy, int64_t ldx) {
  return ldy % 8 == 0 && ldx % 8 == 0 && pair_gate(M, N, K);
}
static size_t pair_split_bytes(int64_t M, int64_t N, int64_t K) {
  const PairPlan pp = plan_pair(shape_of(GemmKind::kBwdDx, M, N, K), shape_of(GemmKind::kBwdDw, M, N, K),
                                device_cus(), kDxCosts, kDwCosts);
  return pp.k1 == 0 ? 0 : pp.s1 + pp.s2;
}

// Workspace of each entry point, from the plan its launch runs on this
// device (the split grids, the pair's shares and modes). A backward call
// with one output reuses the paired call's workspace: its pre-pass buffer
// comes first and its split grid fits into the rest (fit_split).
size_t gemm_workspace_bytes(GemmKind kind, int64_t M, int64_t N, int64_t K) {
  const int cus = device_cus();
  const auto alone = [&](GemmKind k) {
    const GemmShape g = shape_of(k, M, N, K);
    return split_workspace(g, split_grid(g, cus));
  };
  switch (kind) {
    case GemmKind::kFwd:
      return skinny(M) ? 0 : alone(kind);  // the few-token forward needs none
    case GemmKind::kTtqFwd: return alone(kind);
    case GemmKind::kBwdDx: return wt_bytes(N, K) + (skinny(M) && N % 8 == 0 ? 0 : alone(kind));
    case GemmKind::kBwdDw: return xhat_bytes(M, K) + alone(kind);
    case GemmKind::kBwdPair: {
      // (any dW output: the sign output of few tokens takes the separate route)
      if (skinny_both_ok(M, N, K, DwOut::kBf16))  // the 1-bit dW output runs the two products separately
        return std::max(wt_bytes(N, K), std::max(gemm_workspace_bytes(GemmKind::kBwdDx, M, N, K),
                                                 gemm_workspace_bytes(GemmKind::kBwdDw, M, N, K)));
      if (pair_eligible(M, N, K) && pair_split_bytes(M, N, K) > 0)
        return std::max(wt_bytes(N, K) + xhat_bytes(M, K) + pair_split_bytes(M, N, K),
                        std::max(wt_bytes(N, K), xhat_bytes(M, K)));
      return std::max(gemm_workspace_bytes(GemmKind::kBwdDx, M, N, K),
                      gemm_workspace_bytes(GemmKind::kBwdDw, M, N, K));
    }
    case GemmKind::kTtqBwd: {
      if (ttq_pair_eligible(M, N, K, N, K) && pair_split_bytes(M, N, K) > 0)
        return ttq_partials_bytes(N, K) + pair_split_bytes(M, N, K);
      return ttq_partials_bytes(N, K) + std::max(alone(GemmKind::kBwdDx), alone(GemmKind::kBwdDw));
    }
    case GemmKind::kTtqBwdPadded:
      return ttq_partials_bytes(N, K) + std::max(pair_gate(M, N, K) ? pair_split_bytes(M, N, K) : 0,
                                                 std::max(alone(GemmKind::kBwdDx), alone(GemmKind::kBwdDw)));
  }
  return 0;
}

hipError_t launch_bwd_pair(const uint16_t* dY, const uint8_t* w_packed, const float* gamma, const int8_t* x_q,
                           const float* s_x, int64_t M, int64_t N, int64_t K, uint16_t* dX, void* dW,
                           DwOut dw_out, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (ws != nullptr && skinny_both_ok(M, N, K, dw_out) && ws_bytes >= wt_bytes(N, K)) {
    uint8_t* wt = static_cast<uint8_t*>(ws);
    if (hipError_t e = launch_skinny_front(w_packed, x_q, s_x, dY, M, N, K, wt, dW, dw_out, stream)) return e;
    return launch_dx_skinny(wt, dY, gamma, nullptr, M, N, K, dX, stream);
  }
  if (!pair_eligible(M, N, K) || ws == nullptr) return hipErrorNotSupported;
  const GemmShape g1 = shape_of(GemmKind::kBwdDx, M, N, K), g2 = shape_of(GemmKind::kBwdDw, M, N, K);
  const size_t wb = wt_bytes(N, K), xb = xhat_bytes(M, K);
  const PairPlan pp = plan_pair(g1, g2, device_cus(), kDxCosts, kDwCosts);
  if (pp.k1 == 0 || ws_bytes < wb + xb + pp.s1 + pp.s2) return hipErrorNotSupported;
  char* base = static_cast<char*>(ws);
  uint8_t* wt = reinterpret_cast<uint8_t*>(base);
  uint16_t* xhat = reinterpret_cast<uint16_t*>(base + wb);
  const int64_t Kp = k_pad(K), Np = n_pad64(N);
  launch_prep(w_packed, x_q, s_x, M, N, K, wt, xhat, stream);
  if (hipError_t e = hipGetLastError()) return e;
  const RowCodesLoader<CodesFp4Frags> p1{wt, Np / 2, Kp};
  const CopyLoader<2, true> q1{reinterpret_cast<const char*>(dY), 2 * N, M, 2 * N};
  const Bf16Epilogue<false> e1{dX, gamma, K, M};
  const RowCopyBf16Loader<1> p2{xhat, Kp, M, Kp};
  const RowCopyBf16Loader<5> q2{dY, N, M, N};
  char* sws = base + wb + xb;
  const size_t sbytes = ws_bytes - wb - xb;
  hipError_t e;
  switch (dw_out) {
    case DwOut::kF32:
      e = run_pair<1, 0>(p1, q1, e1, g1, kDxCosts, p2, q2, Bf16Epilogue<true>{dW, nullptr, K, N}, g2, kDwCosts, sws,
                         sbytes, stream);
      break;
    case DwOut::kSign1:
      e = run_pair<1, 0>(p1, q1, e1, g1, kDxCosts, p2, q2, Sign1Epilogue{static_cast<uint8_t*>(dW), Kp, N}, g2,
                         kDwCosts, sws, sbytes, stream);
      break;
    default:
      e = run_pair<1, 0>(p1, q1, e1, g1, kDxCosts, p2, q2, Bf16Epilogue<false>{dW, nullptr, K, N}, g2, kDwCosts, sws,
                         sbytes, stream);
      break;
  }
  // (the C ABI's workspace covers the pair and pair_columns was checked
  // above, so this is not NotSupported; if it were, the separate launches
  // the caller falls back to rebuild both operands)
  return e;
}

// ---------------------------------------------------------------------------
// TTQ products ("TTQ_VERIFICATION.md": pure TTQ, unquantized bf16
// activations; the quantized weight wt [N][Kp] holds bf16(Wp), -bf16(Wn) or
// 0). All three are bf16 MFMA GEMMs with fp32 accumulation.
// ---------------------------------------------------------------------------

// y [M][N] = x [M][K] . wt^T: both operands copied as stored (reduction k
// contiguous).
hipError_t launch_ttq_fwd(const uint16_t* x, const uint16_t* wt, int64_t M, int64_t N, int64_t K, uint16_t* y,
                          void* ws, size_t ws_bytes, hipStream_t stream) {
  const int64_t Kp = k_pad(K);
  const CopyLoader<2, true, 1> pl{reinterpret_cast<const char*>(wt), 2 * Kp, N, 2 * Kp};
  const Bf16Epilogue<false> ep{y, nullptr, N, M};
  const GemmShape g = shape_of(GemmKind::kTtqFwd, M, N, K);
  const char* xb = reinterpret_cast<const char*>(x);
  if (K % 8 == 0) return run_gemm<MfmaBf16, 1>(pl, CopyLoader<2, true, 5>{xb, 2 * K, M, 2 * K}, ep, g, ws, ws_bytes, stream);
  return run_gemm<MfmaBf16, 1>(pl, CopyLoader<2, false, 5>{xb, 2 * K, M, 2 * K}, ep, g, ws, ws_bytes, stream);
}

// The forward from the stored codes: few tokens read the 2-bit codes once
// (launch_ttq_fwd_skinny); otherwise the codes become wt at the start of the
// workspace and the GEMM above runs on it. The no_skinny test knob keeps
// the second route at any M.
static bool ttq_codes_skinny(int64_t M, int64_t K) { return skinny(M) && K % 8 == 0; }
static size_t ttq_wt_bytes(int64_t N, int64_t K) { return ((size_t)N * k_pad(K) * 2 + 255) / 256 * 256; }

size_t ttq_codes_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  // none for the few-token route (a decode caller needs no 2*N*Kp buffer);
  // the no_skinny knob is read here too, so a size queried under it covers
  // the GEMM route
  if (ttq_codes_skinny(M, K)) return 0;
  return ttq_wt_bytes(N, K) + gemm_workspace_bytes(GemmKind::kTtqFwd, M, N, K);
}

hipError_t launch_ttq_fwd_codes(const uint16_t* x, const uint8_t* w_packed, const float* params, int64_t M,
                                int64_t N, int64_t K, uint16_t* y, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (ttq_codes_skinny(M, K)) return launch_ttq_fwd_skinny(x, w_packed, params, M, N, K, y, stream);
  const size_t wb = ttq_wt_bytes(N, K);
  if (ws == nullptr || ws_bytes < wb) return hipErrorInvalidValue;  // the C ABI sized it
  uint16_t* wt = static_cast<uint16_t*>(ws);
  if (hipError_t e = launch_ttq_expand(w_packed, N, K, params, wt, stream)) return e;
  return launch_ttq_fwd(x, wt, M, N, K, y, static_cast<char*>(ws) + wb, ws_bytes - wb, stream);
}

// dX [M][K] = dY [M][N] . wt: wt staged as stored (rows n) and read
// transposed (TrFrags), dY copied as stored. dY's rows are ldy apart; where
// ldy > N the columns past N hold zeros.
static hipError_t launch_ttq_dx(const uint16_t* dY, int64_t ldy, const uint16_t* wt, int64_t M, int64_t N, int64_t K,
                                uint16_t* dX, void* ws, size_t ws_bytes, hipStream_t stream) {
  const int64_t Kp = k_pad(K);
  const RowCopyBf16Loader<5> pl{wt, Kp, N, K};
  const Bf16Epilogue<false> ep{dX, nullptr, K, M};
  const GemmShape g = shape_of(GemmKind::kBwdDx, M, N, K);
  const char* db = reinterpret_cast<const char*>(dY);
  if (ldy % 8 == 0)
    return run_gemm<MfmaBf16, 0>(pl, CopyLoader<2, true, 1>{db, 2 * ldy, M, 2 * ldy}, ep, g, ws, ws_bytes, stream);
  return run_gemm<MfmaBf16, 0>(pl, CopyLoader<2, false, 1>{db, 2 * N, M, 2 * N}, ep, g, ws, ws_bytes, stream);
}

// dW [N][K] = dY^T x with the masked sums (TtqDwEpilogue); rows of dY and x
// ldy and ldx apart (zeros past N and K).
template <bool OUT_F32>
static hipError_t launch_ttq_dw(const uint16_t* dY, int64_t ldy, const uint16_t* x, int64_t ldx,
                                const uint8_t* w_packed, int64_t M, int64_t N, int64_t K, void* dW, float2* partials,
                                void* ws, size_t ws_bytes, hipStream_t stream) {
  const GemmShape g = shape_of(GemmKind::kBwdDw, M, N, K);
  const TtqDwEpilogue<OUT_F32> ep{Bf16Epilogue<OUT_F32>{dW, nullptr, K, N}, w_packed, (uint32_t)(k_pad(K) / 4),
                                  partials, (int)(2 * g.tiles_i)};
  if (ldx % 8 == 0 && ldy % 8 == 0)
    return run_gemm<MfmaBf16, 0>(RowCopyBf16Loader<1>{x, ldx, M, K}, RowCopyBf16Loader<5>{dY, ldy, M, N}, ep, g, ws,
                                 ws_bytes, stream);
  if (ldx == K && ldy == N && K % 4 == 0 && N % 4 == 0)
    return run_gemm<MfmaBf16, 0>(RowTransposeBf16Loader<true, 3>{x, K, M, K},
                                 RowTransposeBf16Loader<true, 5>{dY, N, M, N}, ep, g, ws, ws_bytes, stream);
  return run_gemm<MfmaBf16, 0>(RowTransposeBf16Loader<false, 3>{x, ldx, M, K},
                               RowTransposeBf16Loader<false, 5>{dY, ldy, M, N}, ep, g, ws, ws_bytes, stream);
}

// dX and dW in one gemm_pair_kernel launch (as the BitNet backward):
// hipErrorNotSupported when the shape or the device does not allow it.
template <bool OUT_F32>
static hipError_t launch_ttq_pair(const uint16_t* dY, int64_t ldy, const uint16_t* x, int64_t ldx, const uint16_t* wt,
                                  const uint8_t* w_packed, int64_t M, int64_t N, int64_t K, uint16_t* dX, void* dW,
                                  float2* partials, char* ws, size_t ws_bytes, hipStream_t stream) {
  if (!ttq_pair_eligible(M, N, K, ldy, ldx)) return hipErrorNotSupported;
  const int64_t Kp = k_pad(K);
  const GemmShape g1 = shape_of(GemmKind::kBwdDx, M, N, K), g2 = shape_of(GemmKind::kBwdDw, M, N, K);
  const RowCopyBf16Loader<5> p1{wt, Kp, N, K};
  const CopyLoader<2, true, 1> q1{reinterpret_cast<const char*>(dY), 2 * ldy, M, 2 * ldy};
  const Bf16Epilogue<false> e1{dX, nullptr, K, M};
  const RowCopyBf16Loader<1> p2{x, ldx, M, K};
  const RowCopyBf16Loader<5> q2{dY, ldy, M, N};
  const TtqDwEpilogue<OUT_F32> e2{Bf16Epilogue<OUT_F32>{dW, nullptr, K, N}, w_packed, (uint32_t)(Kp / 4), partials,
                                  (int)(2 * g2.tiles_i)};
  // stage costs as for the BitNet pair: measured alone at 4096x2560->6912,
  // this dX (bf16 weight) takes 158-166 us and dW 176-189 us, about the
  // BitNet products' ratio; 15 of 32 columns for dX then give 260 us, 16
  // give 325 us (equal costs chose 16)
  return run_pair<0, 0>(p1, q1, e1, g1, kDxCosts, p2, q2, e2, g2, kDwCosts, ws, ws_bytes, stream);
}

hipError_t launch_ttq_bwd(const uint16_t* dY, int64_t ldy, const uint16_t* x, int64_t ldx, const uint16_t* wt,
                          const uint8_t* w_packed, int64_t M, int64_t N, int64_t K, uint16_t* dX, void* dW, bool dw_f32,
                          float* grads, void* ws, size_t ws_bytes, hipStream_t stream) {
  const size_t pb = ttq_partials_bytes(N, K);
  if (ws == nullptr || ws_bytes < pb) return hipErrorInvalidValue;  // the C ABI sized it
  float2* partials = static_cast<float2*>(ws);
  char* split_ws = static_cast<char*>(ws) + pb;
  const size_t split_bytes = ws_bytes - pb;
  float2* p = grads != nullptr ? partials : nullptr;
  if (dX != nullptr && dW != nullptr) {
    const hipError_t e =
        dw_f32 ? launch_ttq_pair<true>(dY, ldy, x, ldx, wt, w_packed, M, N, K, dX, dW, p, split_ws, split_bytes, stream)
               : launch_ttq_pair<false>(dY, ldy, x, ldx, wt, w_packed, M, N, K, dX, dW, p, split_ws, split_bytes, stream);
    if (e != hipErrorNotSupported) {
      if (e != hipSuccess || grads == nullptr) return e;
      ttq_grads_kernel<<<1, 256, 0, stream>>>(partials, (int)ttq_wave_tiles(N, K), grads);
      return hipGetLastError();
    }
  }
  if (dX != nullptr)
    if (hipError_t e = launch_ttq_dx(dY, ldy, wt, M, N, K, dX, split_ws, split_bytes, stream)) return e;
  if (dW != nullptr) {
    const hipError_t e =
        dw_f32 ? launch_ttq_dw<true>(dY, ldy, x, ldx, w_packed, M, N, K, dW, p, split_ws, split_bytes, stream)
               : launch_ttq_dw<false>(dY, ldy, x, ldx, w_packed, M, N, K, dW, p, split_ws, split_bytes, stream);
    if (e != hipSuccess) return e;
    if (grads != nullptr) {
      ttq_grads_kernel<<<1, 256, 0, stream>>>(partials, (int)ttq_wave_tiles(N, K), grads);
      return hipGetLastError();
    }
  }
  return hipSuccess;
}

}  // namespace bitnet
