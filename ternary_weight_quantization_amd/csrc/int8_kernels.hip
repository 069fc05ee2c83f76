// Linear layer in 8-bit integers with a scale per token and per channel:
//
//   y  = (x_q . w_q^T) sx/127 sw/127 (+ bias)        int32 sums, exact
//   dX = dY w_hat,  dW = dY^T x_hat                  (straight through both quantizations)
//
// with x_hat = bf16(x_q sx/127), w_hat = bf16(w_q sw/127). The forward is the
// scheme of gemm_kernels.hip with both operands int8 copied as stored, or few8.h's or
// mid.h's for fewer tokens; the backward rebuilds both bf16 operands in one launch,
// which also takes dY's column sums for the bias, and runs on them the bf16 products of
// the TTQ layer (launch_ttq_bwd), which take any widths once dY's rows are a multiple
// of 8, or mid.h's.
//
// Measured, 4096 x 2560 -> 6912: forward 84 us (145 G operations, 1.73 P/s; a library
// product of these sizes 83.9), operands 18, products 255 (290 GFLOP, 1.14 PFLOP/s).
// 1000 x 2555 -> 2561: 19, 13 and 54.

#include <algorithm>

#include "bwd_prep.h"
#include "few8.h"
#include "gemm_split.h"
#include "mid.h"
#include "row_io.h"

namespace bitnet {

hipError_t take_int8_split_timeouts(unsigned int* count) { return take_local_split_timeouts(count); }

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------

// The tile's channel scales (over 127) and biases, staged before its main loop.
__shared__ __attribute__((aligned(16))) float s_tile_sw[kBI];
__shared__ __attribute__((aligned(16))) float s_tile_b[kBI];

struct Int8Epilogue {
  uint16_t* y;  // [J][I]
  const float* s;
  const float* sw;
  const uint16_t* bias;  // [I] or NULL
  int64_t I, J;          // N, M

  struct Pre { float sj[kFJ]; };
  __device__ __forceinline__ Pre prefetch(int j0, int lane) const {
    Pre pre;
#pragma unroll
    for (int fj = 0; fj < kFJ; ++fj) {
      const int64_t j = j0 + 32 * fj + (lane & 31);
      pre.sj[fj] = j < J ? s[j] : 0.0f;
    }
    return pre;
  }
  static constexpr int kWaveLds = EpStage<2>::kWaveBytes;
  static constexpr bool kStagesBias = true;
  __device__ __forceinline__ void stage_bias(int ti0) const {
    const int64_t n = (int64_t)ti0 + threadIdx.x;  // kThreads = kBI
    s_tile_sw[threadIdx.x] = n < I ? sw[n] / 127.0f : 0.0f;
    s_tile_b[threadIdx.x] = bias != nullptr && n < I ? bf16_to_f32(bias[n]) : 0.0f;
  }
  __device__ __forceinline__ void store(MfmaI8::Acc (&acc)[kFI][kFJ], const Pre& pre, int i0, int j0, int lane,
                                        char* wlds) const {
#pragma unroll
    for (int fj = 0; fj < kFJ; ++fj) {
      const float c = pre.sj[fj] / 127.0f;
#pragma unroll
      for (int fi = 0; fi < kFI; ++fi)
#pragma unroll
        for (int gi = 0; gi < 4; ++gi) {
          const int at = (i0 % kBI) + 32 * fi + 8 * gi + 4 * (lane >> 5);
          const float4 w = *reinterpret_cast<const float4*>(s_tile_sw + at);
          const float4 b = *reinterpret_cast<const float4*>(s_tile_b + at);
          const float v0 = fmaf((float)acc[fi][fj][4 * gi] * c, w.x, b.x);
          const float v1 = fmaf((float)acc[fi][fj][4 * gi + 1] * c, w.y, b.y);
          const float v2 = fmaf((float)acc[fi][fj][4 * gi + 2] * c, w.z, b.z);
          const float v3 = fmaf((float)acc[fi][fj][4 * gi + 3] * c, w.w, b.w);
          EpStage<2>::put(wlds, lane, fi, gi, make_uint2(pack_bf16x2(v0, v1), pack_bf16x2(v2, v3)));
        }
      EpStage<2>::drain(wlds, reinterpret_cast<char*>(y), I, J, i0, j0 + 32 * fj, lane);
    }
  }
};

// Few tokens (few8.h).
template <int RT, int MT, int W, int P, bool TX, int NX>
__global__ __launch_bounds__(kWave * W) void int8_few_kernel(FewArgs a, const float* __restrict__ s,
                                                             const float* __restrict__ sw,
                                                             const uint16_t* __restrict__ bias,
                                                             uint16_t* __restrict__ y) {
  __shared__ __attribute__((aligned(16))) char smem[few_lds<false, RT, MT, W, TX, true>()];
  __shared__ FewRows<NX, W> rows;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  int tile, m0;
  few_place(a, tile, m0);
  const int64_t n0 = (int64_t)tile * (16 * RT), N = a.rows;
  int64_t row[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) row[t] = n0;
  few_tokens_product<false, RT, MT, W, P, TX, true>(a, row, smem, rows);
  for (int i = wave; i < RT * MT; i += W) {
    const int t = i % RT, mt = i / RT;
    const int64_t ml = 16 * mt + (lane & 15), m = m0 + ml;
    if (ml >= a.M) continue;
    int v[4];
    few_tokens_sum<RT, MT, W>(smem, t, mt, v);
    float sm;
    if constexpr (NX > 0) sm = rows.s[m];
    else sm = s[m];
    const float c = sm / 127.0f;  // the large-M epilogue's expressions
    const int64_t nb = n0 + 16 * t + 4 * (lane >> 4);
    float f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      f[e] = nb + e < N ? fmaf((float)v[e] * c, sw[nb + e] / 127.0f, bias != nullptr ? bf16_to_f32(bias[nb + e]) : 0.0f)
                        : 0.0f;
    store4(y + m * N, nb, N, f);
  }
}

template <int RT, int MT, int W, int P, bool TX, int NX = 0>
static void int8_few_at(const FewArgs& a, const float* s, const float* sw, const uint16_t* bias, uint16_t* y,
                        hipStream_t st) {
  const int64_t grid = (a.rows + 16 * RT - 1) / (16 * RT) * ((a.M + kFewM - 1) / kFewM);
  int8_few_kernel<RT, MT, W, P, TX, NX><<<(unsigned)grid, kWave * W, 0, st>>>(a, s, sw, bias, y);
}

// Middling M (mid.h).
template <int FJ, int P>
__global__ __launch_bounds__(256) void int8_mid_kernel(const int8_t* __restrict__ wq, const int8_t* __restrict__ xq,
                                                       const float* __restrict__ s, const float* __restrict__ sw,
                                                       const uint16_t* __restrict__ bias, int64_t M, int64_t N,
                                                       int64_t Kp, int tiles_j, uint16_t* __restrict__ y) {
  typedef MidShape<2, FJ, 2, 2> S;
  typedef MidRows<TileRow> LP, LQ;
  __shared__ __attribute__((aligned(16))) char lds[S::template kLds<LP, LQ>];
  const int v = xcd_major(blockIdx.x, gridDim.x), lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int i0 = v / tiles_j * S::kI, j0 = v % tiles_j * S::kJ;
  if (threadIdx.x < S::kI) {
    const int64_t n = i0 + threadIdx.x;
    s_tile_sw[threadIdx.x] = n < N ? sw[n] / 127.0f : 0.0f;
    s_tile_b[threadIdx.x] = bias != nullptr && n < N ? bf16_to_f32(bias[n]) : 0.0f;
  }
  const int jw = j0 + 32 * FJ * (wave / 2), iw = 64 * (wave % 2);
  float sj[FJ];
#pragma unroll
  for (int fj = 0; fj < FJ; ++fj) {
    const int64_t m = jw + 32 * fj + (lane & 31);
    sj[fj] = m < M ? s[m] : 0.0f;
  }
  const LP lp{{}, wq, N, Kp, {i0, N}}, lq{{}, xq, M, Kp, {j0, M}};
  MfmaI8::Acc acc[2][FJ] = {};
  mid_tile<MfmaI8, 2, FJ, 2, 2, P>(lp, lq, (int)((Kp + kStageBytes - 1) / kStageBytes), lds, acc);
  char* wlds = lds + wave * HalfStage::kBytes;
#pragma unroll
  for (int fj = 0; fj < FJ; ++fj) {
    const float c = sj[fj] / 127.0f;  // the large tiles' expressions
#pragma unroll
    for (int fi = 0; fi < 2; ++fi)
#pragma unroll
      for (int gi = 0; gi < 4; ++gi) {
        const int at = iw + 32 * fi + 8 * gi + 4 * (lane >> 5);
        const float4 w = *reinterpret_cast<const float4*>(s_tile_sw + at);
        const float4 b = *reinterpret_cast<const float4*>(s_tile_b + at);
        const float v0 = fmaf((float)acc[fi][fj][4 * gi] * c, w.x, b.x);
        const float v1 = fmaf((float)acc[fi][fj][4 * gi + 1] * c, w.y, b.y);
        const float v2 = fmaf((float)acc[fi][fj][4 * gi + 2] * c, w.z, b.z);
        const float v3 = fmaf((float)acc[fi][fj][4 * gi + 3] * c, w.w, b.w);
        HalfStage::put(wlds, lane, fi, gi, make_uint2(pack_bf16x2(v0, v1), pack_bf16x2(v2, v3)));
      }
    HalfStage::drain(wlds, y, N, N, M, i0 + iw, jw + 32 * fj, lane);
  }
}

static bool few(int64_t M) {
  return M <= kSkinnyMaxM && test_knobs().no_skinny.load(std::memory_order_relaxed) == 0;
}

// Tiles of 16 rows a workgroup of the few-token kernel takes, 0: the kernel is not used.
// Up to 16 tokens one at every N (16 tokens 2560 -> 32000: 15.5 us, with two 16.5). Above,
// x_q's traffic counts and more rows share it as long as the workgroups fill the CUs (32
// tokens 6912 -> 2560 8.7 us with 16, 11.0 with 32; 64 tokens 2560 -> 6912 8.9 with 32, 10.4
// with 16, 9.7 with 64) and fit the device at once, up to 256 tokens in groups of 64;
// mid.h's tiles take over there (6912 -> 2560, 256 tokens: 17.9 us here with 64 rows, 25.5
// there; 2560 -> 6912, 192: 18.2 and 12.6; 2560 -> 32000, 64: 24.1 and 17.2, 32: 19.3 and
// 17.3).
static int few_tiles(int64_t M, int64_t N) {
  if (!few(1) || M > 4 * kFewM) return 0;
  if (M <= 16) return 1;
  const int64_t groups = (M + kFewM - 1) / kFewM;
  for (int rt = 1; rt <= 4; rt *= 2)
    if ((N + 16 * rt - 1) / (16 * rt) * groups <= device_cus()) return rt;
  return 0;
}

// The token blocks of mid.h's tiles where the few-token kernel is not used, 0: 256 x 256
// tiles. Up to 64 tokens any number of 128 x 64 tiles, in rounds (64 tokens 2560 -> 128256:
// 66 us for 63 of bytes, 106 in the few-token kernel).
static int mid_form(int64_t M, int64_t N) {
  const int fj = mid_blocks(M, (N + 127) / 128);
  return fj == 0 && few(M) ? 1 : fj;
}

static void int8_few(const FewArgs& a, const float* s, const float* sw, const uint16_t* bias, uint16_t* y,
                     hipStream_t st) {
  const int rt = few_tiles(a.M, a.rows);
  if (a.x != nullptr) {  // M <= rows_direct(K)
    const bool deep = a.Kp > FewRows<1, 4>::kMaxK;
    if (a.M > 2 && deep) int8_few_at<1, 1, 8, 5, false, 4>(a, s, sw, bias, y, st);
    else if (a.M > 2) int8_few_at<1, 1, 4, 5, false, 4>(a, s, sw, bias, y, st);
    else if (a.M > 1 && deep) int8_few_at<1, 1, 8, 5, false, 2>(a, s, sw, bias, y, st);
    else if (a.M > 1) int8_few_at<1, 1, 4, 5, false, 2>(a, s, sw, bias, y, st);
    else if (deep) int8_few_at<1, 1, 8, 5, false, 1>(a, s, sw, bias, y, st);
    else int8_few_at<1, 1, 4, 5, false, 1>(a, s, sw, bias, y, st);
  } else if (a.M <= 2) int8_few_at<1, 1, 4, 5, false>(a, s, sw, bias, y, st);
  else if (a.M <= 16) int8_few_at<1, 1, 4, 5, true>(a, s, sw, bias, y, st);
  else if (a.M <= 32 && rt == 1) int8_few_at<1, 2, 4, 5, true>(a, s, sw, bias, y, st);
  else if (a.M <= 32 && rt == 2) int8_few_at<2, 2, 4, 4, true>(a, s, sw, bias, y, st);
  else if (a.M <= 32) int8_few_at<4, 2, 4, 2, true>(a, s, sw, bias, y, st);
  else if (rt == 1) int8_few_at<1, 4, 8, 3, true>(a, s, sw, bias, y, st);
  else if (rt == 2) int8_few_at<2, 4, 8, 2, true>(a, s, sw, bias, y, st);
  else int8_few_at<4, 4, 8, 1, true>(a, s, sw, bias, y, st);
}

template <int FJ, int P>
static hipError_t int8_mid(const int8_t* w_q, const int8_t* x_q, const float* s_x, const float* s_w,
                           const uint16_t* bias, int64_t M, int64_t N, int64_t Kp, uint16_t* y, hipStream_t st) {
  const int64_t tj = (M + 64 * FJ - 1) / (64 * FJ), ti = (N + 127) / 128;
  int8_mid_kernel<FJ, P><<<(unsigned)(ti * tj), 256, 0, st>>>(w_q, x_q, s_x, s_w, bias, M, N, Kp, (int)tj, y);
  return hipGetLastError();
}

size_t int8_fwd_workspace(int64_t M, int64_t N, int64_t K) {
  if (few_tiles(M, N) || mid_form(M, N)) return 0;
  const GemmShape g = shape_of(GemmKind::kFwd, M, N, K);
  return split_workspace(g, split_grid(g, device_cus()));
}

int rows_direct(int64_t K) { return few(1) && K >= 8 && K <= FewRows<1, 8>::kMaxK ? 4 : 0; }

hipError_t launch_int8_fwd(const uint16_t* x, const int8_t* x_q, const float* s_x, const int8_t* w_q, const float* s_w,
                           const uint16_t* bias, int64_t M, int64_t N, int64_t K, uint16_t* y, void* ws,
                           size_t ws_bytes, hipStream_t stream) {
  const int64_t Kp = k_pad(K);
  if (few_tiles(M, N)) {
    const FewArgs a{reinterpret_cast<const uint8_t*>(w_q), N, Kp, x_q, Kp, (int)M, x, (int)K};
    int8_few(a, s_x, s_w, bias, y, stream);
    return hipGetLastError();
  }
  const int fj = mid_form(M, N);
  if (fj == 1) return int8_mid<1, 4>(w_q, x_q, s_x, s_w, bias, M, N, Kp, y, stream);
  if (fj == 2) return int8_mid<2, 2>(w_q, x_q, s_x, s_w, bias, M, N, Kp, y, stream);
  const CopyLoader<1, true, 1> pl{reinterpret_cast<const char*>(w_q), Kp, N, Kp};
  const CopyLoader<1, true, 5> ql{reinterpret_cast<const char*>(x_q), Kp, M, Kp};
  return run_gemm<MfmaI8, 1>(pl, ql, Int8Epilogue{y, s_x, s_w, bias, N, M}, shape_of(GemmKind::kFwd, M, N, K), ws,
                             ws_bytes, stream);
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------

// What the products read, in one launch: x_hat [M][Kp] (xb blocks), w_hat [N][Kp] (wb
// blocks) and, where dY's rows are not a multiple of 8 or their sum is wanted, one pass
// over dY (the first yb blocks, which take longest): rows copied to `padded` [M][ld] (zeros past N), and
// partial column sums, a row [N] for each of the `groups` groups of rows. A block takes
// 2048 columns of a group's rows in turn, a thread 8 of them.
struct Int8Dy {
  const uint16_t* dY;
  int64_t M;
  int N;
  uint16_t* padded;  // NULL: not wanted
  int ld;
  float* sums;       // NULL: not wanted
  int groups, cols;  // blocks: groups * cols
};
constexpr int kDyCols = 2048;

__device__ __forceinline__ void dy_block(const Int8Dy& a, int b) {
  const int g = b / a.cols, k0 = (b % a.cols) * kDyCols + 8 * threadIdx.x;
  const int64_t lo = a.M * g / a.groups, hi = a.M * (g + 1) / a.groups;
  const int end = a.padded ? a.ld : a.N;
  if (k0 >= end) return;
  float sum[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int64_t m = lo; m < hi; ++m) {
    const ChunkBf16 c = chunk8(a.dY + m * a.N, k0, a.N);
    if (a.padded) *reinterpret_cast<uint4*>(a.padded + m * a.ld + k0) = c.v;
    float f[8];
    c.get(f);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] += f[e];
  }
  if (a.sums) store8(a.sums + (int64_t)g * a.N, k0, a.N, sum);
}

__global__ __launch_bounds__(256) void int8_prep_kernel(const int8_t* __restrict__ xq, const float* __restrict__ sx,
                                                        int64_t M, uint16_t* __restrict__ xhat, int xb,
                                                        const int8_t* __restrict__ wq, const float* __restrict__ sw,
                                                        int64_t N, uint16_t* __restrict__ what, int wb, int64_t Kp,
                                                        Int8Dy dy, int yb) {
  const int b = (int)blockIdx.x - yb;
  if (b < 0) dy_block(dy, b + yb);
  else if (b < xb) xhat_blocks(xq, sx, M, Kp, xhat, b, xb);
  else xhat_blocks(wq, sw, N, Kp, what, b - xb, wb);
}

static size_t up256(size_t n) { return (n + 255) / 256 * 256; }
// Groups of rows of the pass over dY: 16 rows or more each, at most 256 groups (4096 x
// 6912: the launch takes 25 us with the sums and 18 without; with 64 groups 42).
static int dy_groups(int64_t M) { return (int)std::max<int64_t>(1, std::min<int64_t>(256, M / 16)); }
struct Int8Ws {
  size_t xhat, what, dy, sums;
  size_t before() const { return xhat + what + dy + sums; }
};
static Int8Ws int8_ws(int64_t M, int64_t N, int64_t K) {
  const int64_t Kp = k_pad(K);
  return {up256((size_t)M * Kp * 2), up256((size_t)N * Kp * 2), N % 8 == 0 ? 0 : up256((size_t)M * k_pad(N) * 2),
          up256((size_t)dy_groups(M) * N * 4)};
}
size_t int8_bwd_workspace(int64_t M, int64_t N, int64_t K) {
  return int8_ws(M, N, K).before() + gemm_workspace_bytes(GemmKind::kTtqBwdPadded, M, N, K);
}

hipError_t launch_int8_bwd(const uint16_t* dY, const int8_t* x_q, const float* s_x, const int8_t* w_q,
                           const float* s_w, int64_t M, int64_t N, int64_t K, uint16_t* dX, void* dW, bool dw_f32,
                           void* db, bool db_f32, void* ws, size_t ws_bytes, hipStream_t stream) {
  const int64_t Kp = k_pad(K);
  const Int8Ws w = int8_ws(M, N, K);
  char* base = static_cast<char*>(ws);
  uint16_t* xhat = reinterpret_cast<uint16_t*>(base);
  uint16_t* what = reinterpret_cast<uint16_t*>(base + w.xhat);
  const bool products = dX != nullptr || dW != nullptr, pad = products && N % 8 != 0;
  const int64_t ldy = pad ? k_pad(N) : N;
  Int8Dy dy{dY, M, (int)N, pad ? reinterpret_cast<uint16_t*>(base + w.xhat + w.what) : nullptr, (int)ldy,
            db != nullptr ? reinterpret_cast<float*>(base + w.xhat + w.what + w.dy) : nullptr, dy_groups(M),
            (int)((ldy + kDyCols - 1) / kDyCols)};
  const auto blocks = [&](int64_t rows) { return (int)std::min<int64_t>((rows * (Kp / 16) + 255) / 256, 4096); };
  const int xb = dW != nullptr ? blocks(M) : 0, wb = dX != nullptr ? blocks(N) : 0;
  const int yb = pad || db != nullptr ? dy.groups * dy.cols : 0;
  int8_prep_kernel<<<xb + wb + yb, 256, 0, stream>>>(x_q, s_x, M, xhat, xb, w_q, s_w, N, what, wb, Kp, dy, yb);
  if (hipError_t e = hipGetLastError()) return e;
  if (db != nullptr)
    if (hipError_t e = launch_norm_cols(dy.sums, dy.groups, 1, N, db, nullptr, db_f32, stream)) return e;
  if (!products) return hipSuccess;
  const uint16_t* y = pad ? dy.padded : dY;
  const GemmShape g1 = shape_of(GemmKind::kBwdDx, M, N, K), g2 = shape_of(GemmKind::kBwdDw, M, N, K);
  if (const int fj = mid_bwd_blocks(g1, g2, dX != nullptr, dW != nullptr, pair_pays(g1, g2), M, K, N)) {
    const MidCols lp1{what, N, Kp, Kp, 0}, lp2{xhat, M, Kp, Kp, 0}, lq2{y, M, ldy, ldy, 0};
    const MidRows<TileRow> lq1{{}, y, M, 2 * ldy, {0, M}};
    const MidOut<2> e1{dX, K, M, nullptr};
    const auto run = [&](auto e2) {
      return fj == 1 ? mid_products_at<1, 4>(lp1, lq1, e1, lp2, lq2, e2, dX != nullptr, dW != nullptr, M, K, N, N, stream)
                     : mid_products_at<2, 2>(lp1, lq1, e1, lp2, lq2, e2, dX != nullptr, dW != nullptr, M, K, N, N, stream);
    };
    return dw_f32 ? run(MidOut<4>{dW, K, N, nullptr}) : run(MidOut<2>{dW, K, N, nullptr});
  }
  return launch_ttq_bwd(y, ldy, xhat, Kp, what, nullptr, M, N, K, dX, dW, dw_f32, nullptr,
                        base + w.before(), ws_bytes - w.before(), stream);
}

}  // namespace bitnet
