// Layer norm over rows of K values, forward and backward.
//
//   mu = sum x / K,  r = (sum (x - mu)^2 / K + eps)^(-1/2),  xh = (x - mu) r
//   y  = xh w + b
//   g  = dY w,  c1 = sum g / K,  c2 = sum g xh / K
//   dX = r (g - c1 - xh c2),  dw = sum over rows dY xh,  db = sum over rows dY
//
// A row of up to 16384 values lives in the registers of TPR threads (CPT chunks
// of 8 values each), so x is read once forward and once backward and the
// variance is the sum of centered squares. Wider rows do too, but with 5 to 8
// chunks in each of 512 threads the backward no longer fits the registers
// beside its column sums (6 to 310 spilled, at most 936 bytes of scratch a
// thread), nor does the forward from 7 chunks on (f32: 6; up to 223 spilled). Statistics and sums are fp32. With 8-bit codes the
// forward also writes the row's codes and block scales (row_io.h), and the
// backward takes x from them; mu and r are those of the uncoded row.
//
// The weight's and bias' gradients are column sums over all rows. Each
// thread of the backward keeps its columns' sums in registers over the rows
// its block takes, the block adds its rows' sums through LDS and writes one
// partial row [2][K]; a second launch adds the partial rows in block order.
// No atomics: the same inputs give the same bits.
//
// About 10 operations a value, so HBM bounds both directions of long
// problems. Measured, forward / backward / column sums in us, traced back to
// back: 16384 x 6912 bf16 with codes 130 / 133 / 6.0 (4.4 and 4.3 TB/s, a copy
// reaches 5.2; 244 for all three among other work), 2048 x 6912 f32 17.9 /
// 31.2 / 5.3 (4.7 and 4.5 TB/s), 4096 x 16384 bf16 61 / 91 / 6.7, one row of
// 2560 3.7. Short problems pay for each block's start and end, the weight to
// LDS, its rows' sums and a partial row, whatever the width: 4096 x 2560 bf16
// 11.0 / 18.0 / 4.3 (a copy of its bytes: 8 and 12), 1537 x 2560 with codes
// 10.1 / 13.9 / 3.9 and 1537 x 2555 11.0 / 14.3 / 3.9. Where registers spill
// the scratch traffic bounds the backward: 4096 x 24576 bf16 67 / 434 / 9.0, f32
// 144 / 821 / 9.2, 2048 x 32768 bf16 110 / 516 / 11.

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "row_io.h"

namespace bitnet {

__device__ __forceinline__ float wave_sum_f32(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, kWave);
  return v;
}

// Sum over the TPR threads of a row (whole waves), in every one of them.
// `slot`: an LDS array of one float per wave of the block, free on entry.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* slot) {
  v = wave_sum_f32(v);
  if constexpr (TPR > kWave) {
    constexpr int W = TPR / kWave;
    const int w0 = threadIdx.x / TPR * W;
    if (threadIdx.x % kWave == 0) slot[threadIdx.x / kWave] = v;
    __syncthreads();
    v = slot[w0];
#pragma unroll
    for (int j = 1; j < W; ++j) v += slot[w0 + j];
  }
  return v;
}

struct NormParams {
  const void* w;  // [K] or NULL
  const void* b;
  bool f32;       // their type
};

// Keeps a loaded chunk as it is across a row's reduction: the values derived
// from it are computed again after it instead of being held in registers.
__device__ __forceinline__ void hold(ChunkBf16& c) { asm volatile("" : "+v"(c.v.x), "+v"(c.v.y), "+v"(c.v.z), "+v"(c.v.w)); }
__device__ __forceinline__ void hold(ChunkF32& c) {
  asm volatile("" : "+v"(c.a.x), "+v"(c.a.y), "+v"(c.a.z), "+v"(c.a.w), "+v"(c.b.x), "+v"(c.b.y), "+v"(c.b.z), "+v"(c.b.w));
}

struct NormFwd {
  const void* x;
  NormParams p;
  int64_t M;
  int K, nch;
  float eps;
  void* y;
  bool y_f32;
  float* mean;    // each NULL if not wanted
  float* rstd;
  int8_t* codes;
  float* scales;
};

// Waves a SIMD holds: what the chunks held per thread leave registers for. The
// launch takes as many blocks as run together, so that each block's weight and
// bias are read once and no block starts late.
template <class T, int CPT>
constexpr int norm_fwd_waves() {
  return CPT <= 2 ? 4 : CPT == 3 ? (sizeof(T) == 2 ? 4 : 3) : CPT == 4 && sizeof(T) == 2 ? 3 : 2;
}

// A block takes rows (TPR threads each) in turn; the weight and bias stay in
// its registers as loaded, and the next row is requested before the current
// one is reduced. P: the parameters' type. SHORT: K < 8 (one chunk a row).
template <class T, class P, int BLOCK, int TPR, int CPT, bool SHORT>
__global__ __launch_bounds__(BLOCK, (norm_fwd_waves<T, CPT>())) void layernorm_fwd_kernel(NormFwd a) {
  constexpr int RPB = BLOCK / TPR;
  __shared__ float slot[4][BLOCK / kWave];
  const int t = threadIdx.x % TPR;
  const int rl = __builtin_amdgcn_readfirstlane((int)threadIdx.x / TPR);  // whole waves share a row
  const int K = a.K;
  const int ch_last = t + (CPT - 1) * TPR, k_last = 8 * ch_last;
  typename ChunkOf<P>::type cw[CPT] = {}, cb[CPT] = {};
  typename ChunkOf<T>::type c[CPT], nx[CPT];
  // only a thread's last chunk can reach past K (row_split)
  const auto load = [&](auto* row, auto (&v)[CPT]) {
#pragma unroll
    for (int i = 0; i < CPT - 1; ++i) v[i] = load8_in(row + 8 * (t + i * TPR));
    v[CPT - 1] = load8<SHORT>(row, k_last, K);
  };
  const T* x = static_cast<const T*>(a.x);
  // Every thread passes every barrier: past the last row a wave (rows are
  // uniform in a wave) repeats it and writes nothing.
  const int64_t stride = (int64_t)gridDim.x * RPB, last = a.M - 1;
  int64_t base = (int64_t)blockIdx.x * RPB, row = base + rl < last ? base + rl : last;
  load(x + row * K, c);
  if (a.p.w) load(static_cast<const P*>(a.p.w), cw);
  if (a.p.b) load(static_cast<const P*>(a.p.b), cb);
  settle8<SHORT>(cw[CPT - 1], k_last, K);
  settle8<SHORT>(cb[CPT - 1], k_last, K);
  int flip = 0;
  for (; base < a.M; base += stride, flip ^= 2) {
    const bool ok = base + rl < a.M;
    const int64_t want = base + stride + rl, next = want < last ? want : last;
    const bool more = base + stride < a.M;  // uniform
    if (more) load(x + next * K, nx);
    settle8<SHORT>(c[CPT - 1], k_last, K);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      float f[8];
      c[i].get(f);
      sum += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
      hold(c[i]);
    }
    // two slot pairs in turn: a row's readers are done with one pair before
    // the barrier of the next row, after which it may be written again
    const float mu = row_sum<TPR>(sum, slot[flip]) / (float)K;
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int left = K - 8 * (t + i * TPR);
      float f[8];
      c[i].get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] -= mu;
      if (i == CPT - 1 && left < 8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = e < left ? f[e] : 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sq = fmaf(f[e], f[e], sq);
      hold(c[i]);
    }
    const float r = 1.0f / sqrtf(row_sum<TPR>(sq, slot[flip + 1]) / (float)K + a.eps);
    if (ok) {
      if (t == 0) {
        if (a.mean) a.mean[row] = mu;
        if (a.rstd) a.rstd[row] = r;
      }
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        const int ch = t + i * TPR, k0 = 8 * ch;
        if (i == CPT - 1 && ch >= a.nch) continue;
        float f[8], w[8], b[8];
        c[i].get(f);
        if (a.codes) {  // uniform; the 16 lanes of a block are all here
          const float s = block_scale(c[i]);
          reinterpret_cast<uint2*>(a.codes)[row * a.nch + ch] = codes8(f, s);
          if ((t & 15) == 0) a.scales[(row * a.nch + ch) >> 4] = s;
        }
        cw[i].get(w);
        cb[i].get(b);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = (f[e] - mu) * r;
        if (a.p.w) {
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = fmaf(f[e], w[e], b[e]);  // b: zeros where there is none
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] += b[e];
        }
        if (a.y_f32) {
          float* yr = static_cast<float*>(a.y) + row * K;
          if (i < CPT - 1) store8_in(yr + k0, f);
          else store8(yr, k0, K, f);
        } else {
          uint16_t* yr = static_cast<uint16_t*>(a.y) + row * K;
          if (i < CPT - 1) store8_in(yr + k0, f);
          else store8(yr, k0, K, f);
        }
      }
    }
    if (more) {
#pragma unroll
      for (int i = 0; i < CPT; ++i) c[i] = nx[i];
    }
    row = next;
  }
}

// Where the backward's x comes from: bf16 or f32 rows, or codes.
struct FromBf16 { typedef ChunkBf16 Chunk; };
struct FromF32 { typedef ChunkF32 Chunk; };
struct ChunkCodes {
  uint2 q;
  float s;
};
struct FromCodes { typedef ChunkCodes Chunk; };

// xh = x r + (-mu r), one operation a value; of a code, (q s / 127) r with
// the scale's factors taken together.
template <class C>
__device__ __forceinline__ void normalized8(const C& c, float r, float nmr, float (&xh)[8]) {
  float k = r;
  if constexpr (std::is_same<C, ChunkCodes>::value) {
    k = c.s / 127.0f * r;
    values8(c.q, 1.0f, xh);
  } else {
    c.get(xh);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) xh[e] = fmaf(xh[e], k, nmr);
}

struct NormBwd {
  const void* dY;
  const void* x;        // rows (FromBf16, FromF32)
  const int8_t* codes;  // FromCodes
  const float* scales;
  NormParams p;
  const float* mean;
  const float* rstd;
  int64_t M;
  int K, nch;
  void* dX;
  float* partials;  // [blocks][2][K], NULL: no column sums
};

// Chunk ch of a row; IN: it lies inside the row.
template <class X, bool IN, bool SHORT>
__device__ __forceinline__ typename X::Chunk norm_x(const NormBwd& a, int64_t row, int ch) {
  if constexpr (std::is_same<X, FromCodes>::value) {
    ChunkCodes c;
    const int at = IN || ch < a.nch ? ch : 0;
    c.q = reinterpret_cast<const uint2*>(a.codes)[row * a.nch + at];
    c.s = a.scales[(row * a.nch + at) >> 4];
    return c;
  } else if constexpr (std::is_same<X, FromF32>::value) {
    const float* p = static_cast<const float*>(a.x) + row * a.K;
    if constexpr (IN) return load8_in(p + 8 * ch);
    else return load8<SHORT>(p, 8 * ch, a.K);
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(a.x) + row * a.K;
    if constexpr (IN) return load8_in(p + 8 * ch);
    else return load8<SHORT>(p, 8 * ch, a.K);
  }
}

// The weight as fp32 in LDS: every row of the block reads it twice.
extern __shared__ __attribute__((aligned(16))) float norm_lds[];

__device__ __forceinline__ void hold(ChunkCodes& c) { asm volatile("" : "+v"(c.q.x), "+v"(c.q.y), "+v"(c.s)); }

template <class X, class DX, class DY, int BLOCK, int TPR, int CPT, bool SHORT>
__global__ __launch_bounds__(BLOCK, BLOCK == 512 ? 1 : 2) void layernorm_bwd_kernel(NormBwd a) {
  constexpr int RPB = BLOCK / TPR;
  __shared__ float slot[4][BLOCK / kWave];
  const int t = threadIdx.x % TPR;
  const int rl = __builtin_amdgcn_readfirstlane((int)threadIdx.x / TPR);  // whole waves share a row
  const int K = a.K;
  for (int k = threadIdx.x; k < a.nch; k += BLOCK) {
    float w[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
    if (a.p.w) param8(a.p.w, a.p.f32, 8 * k, K, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) norm_lds[8 * k + e] = w[e];
  }
  __syncthreads();
  float dw[CPT][8], db[CPT][8];
#pragma unroll
  for (int i = 0; i < CPT; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = db[i][e] = 0.0f;

  // the chunks of a row; only a thread's last can reach past K (row_split):
  // dY is zero there, so nothing is added
  const auto load = [&](int64_t row, typename ChunkOf<DY>::type (&cd)[CPT], typename X::Chunk (&cx)[CPT]) {
    const DY* dr = static_cast<const DY*>(a.dY) + row * K;
#pragma unroll
    for (int i = 0; i < CPT - 1; ++i) {
      cd[i] = load8_in(dr + 8 * (t + i * TPR));
      cx[i] = norm_x<X, true, SHORT>(a, row, t + i * TPR);
    }
    cd[CPT - 1] = load8<SHORT>(dr, 8 * (t + (CPT - 1) * TPR), K);
    cx[CPT - 1] = norm_x<X, false, SHORT>(a, row, t + (CPT - 1) * TPR);
  };
  // what a chunk past the row's end reads of the weight (chunk 0) does not matter
  const int k_last = t + (CPT - 1) * TPR < a.nch ? 8 * (t + (CPT - 1) * TPR) : 0;
  // The next row is loaded while this one is reduced where both fit the
  // registers next to the column sums (measured at 2048 x 6912, f32 x: 55 us
  // with it and spilled, 33 us without; at 16384 x 2560 bf16 113 us for both
  // directions with it, 84 us without; at 16384 x 6912 from codes 118 us with
  // it, 147 us without).
  constexpr bool AHEAD = (sizeof(typename ChunkOf<DY>::type) + sizeof(typename X::Chunk)) / 4 * CPT <= 36;
  typename ChunkOf<DY>::type cd[CPT], nd[CPT];
  typename X::Chunk cx[CPT], nx[CPT];
  // The block's row groups; every thread passes every barrier. Past the last
  // row a wave (rows are uniform in a wave) repeats it with dY = 0.
  const int64_t stride = (int64_t)gridDim.x * RPB, last = a.M - 1;
  int64_t base = (int64_t)blockIdx.x * RPB, row = base + rl < last ? base + rl : last;
  if constexpr (AHEAD) load(row, cd, cx);
  float mu = a.mean[row], r = a.rstd[row];
  int flip = 0;
  for (; base < a.M; base += stride, flip ^= 2) {
    const bool ok = base + rl < a.M;
    const int64_t want = base + stride + rl, next = want < last ? want : last;
    if constexpr (AHEAD) load(next, nd, nx);
    else load(row, cd, cx);
    const float nmu = a.mean[next], nr = a.rstd[next], nmr = -mu * r;
    if (!ok) {
#pragma unroll
      for (int i = 0; i < CPT; ++i) cd[i] = typename ChunkOf<DY>::type{};
    }
    settle8<SHORT>(cd[CPT - 1], 8 * (t + (CPT - 1) * TPR), K);
    if constexpr (!std::is_same<X, FromCodes>::value) settle8<SHORT>(cx[CPT - 1], 8 * (t + (CPT - 1) * TPR), K);
    float sg = 0.0f, sgx = 0.0f;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const float* w = norm_lds + (i < CPT - 1 ? 8 * (t + i * TPR) : k_last);
      float d[8], xh[8];
      cd[i].get(d);
      normalized8(cx[i], r, nmr, xh);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float g = d[e] * w[e];
        sg += g;
        sgx = fmaf(g, xh[e], sgx);
        dw[i][e] = fmaf(d[e], xh[e], dw[i][e]);
        db[i][e] += d[e];
      }
      hold(cd[i]);
      hold(cx[i]);
      __builtin_amdgcn_sched_barrier(0);  // one chunk's values at a time
    }
    // two slot pairs in turn: a row's readers are done with one pair before
    // the barrier of the next row, after which it may be written again
    const float c1 = row_sum<TPR>(sg, slot[flip]) / (float)K * r;
    const float c2 = row_sum<TPR>(sgx, slot[flip + 1]) / (float)K * r;
    if (a.dX != nullptr && ok) {
      DX* xr = static_cast<DX*>(a.dX) + row * K;
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        const float* w = norm_lds + (i < CPT - 1 ? 8 * (t + i * TPR) : k_last);
        float d[8], xh[8], o[8];
        cd[i].get(d);
        normalized8(cx[i], r, nmr, xh);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fmaf(-c2, xh[e], fmaf(d[e] * w[e], r, -c1));
        if (i < CPT - 1) store8_in(xr + 8 * (t + i * TPR), o);
        else store8(xr, 8 * (t + i * TPR), K, o);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (AHEAD) {
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        cd[i] = nd[i];
        cx[i] = nx[i];
      }
    }
    mu = nmu;
    r = nr;
    row = next;
  }

  if (a.partials == nullptr) return;
  float* out = a.partials + (int64_t)blockIdx.x * 2 * K;
  if constexpr (RPB > 1) {
    // the block's rows in turn, one chunk column at a time
    __shared__ float acc[RPB][TPR][9];
#pragma unroll
    for (int q = 0; q < 2 * CPT; ++q) {
      const int i = q >> 1;
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[rl][t][e] = (q & 1) ? db[i][e] : dw[i][e];
      __syncthreads();
      // 8 * TPR sums over RPB rows by the block
      for (int j = threadIdx.x; j < 8 * TPR; j += BLOCK) {
        float v = acc[0][j >> 3][j & 7];
#pragma unroll
        for (int w = 1; w < RPB; ++w) v += acc[w][j >> 3][j & 7];
        const int k = 8 * TPR * i + j;
        if (k < K) out[(q & 1) * (int64_t)K + k] = v;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int k0 = 8 * (t + i * TPR);
      if (k0 >= K) continue;
      store8(out, k0, K, dw[i]);
      store8(out + K, k0, K, db[i]);
    }
  }
}

// The column sums of the partial rows [blocks][cols], columns [0, K) to dw
// and [K, 2K) to db: a block takes 64 columns, its 16 waves every 16th
// partial row each, then the wave sums are added in order.
__global__ __launch_bounds__(1024) void layernorm_cols_kernel(const float* __restrict__ partials, int blocks, int K,
                                                              void* __restrict__ dw, void* __restrict__ db,
                                                              bool p_f32) {
  __shared__ float part[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + lane, cols = 2 * (int64_t)K;
  float v = 0.0f;
  if (col < cols) {
    const float* src = partials + col;
    int r = wave;
    for (; r + 48 < blocks; r += 64) {  // four loads in flight
      const float a = src[(int64_t)r * cols], b = src[(int64_t)(r + 16) * cols], c = src[(int64_t)(r + 32) * cols],
                  d = src[(int64_t)(r + 48) * cols];
      v += (a + b) + (c + d);
    }
    for (; r < blocks; r += 16) v += src[(int64_t)r * cols];
  }
  part[wave][lane] = v;
  __syncthreads();
  if (wave != 0 || col >= cols) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) v += part[w][lane];
  void* out = col < K ? dw : db;
  const int64_t k = col < K ? col : col - K;
  if (out == nullptr) return;
  if (p_f32) static_cast<float*>(out)[k] = v;
  else static_cast<uint16_t*>(out)[k] = f32_to_bf16_bits(v);
}

// ---------------------------------------------------------------------------
// Launches. Threads per row and chunks per thread from the row length alone:
// one wave (no barriers) up to five chunks a thread, two waves for three, four
// up to four chunks, eight above, up to the eight chunks of kNormMaxK (no other
// split was tried above 8192). Measured, forward and backward in
// us, without / with codes: 32768 x 1536 one wave 102 / 102, two 121 / 136;
// 16384 x 2560 one wave 84 / 93, two 86 / 96, four 112 / 130; 16384 x 2900 one
// wave (six chunks) 138 / 155, two 104 / 108; 8192 x 4096 four waves 72 / 81,
// two 74 / 89; 8192 x 6912 four waves 121 / 125, eight 119 / 158.
// ---------------------------------------------------------------------------

struct RowSplit {
  int tpr, cpt;
};
// nch and tpr are multiples of 16, so every chunk before a thread's last is a
// whole chunk of the row (it lies before the row's last block of 128).
static RowSplit row_split(int64_t K) {
  const int nch = (int)(ckpt_pad(K) / 8);
  const int tpr = nch <= 320 ? 64 : nch <= 384 ? 128 : nch <= 1024 ? 256 : 512;
  return {tpr, (nch + tpr - 1) / tpr};
}

// Every pair that row_split gives, and rows of fewer than 8 values.
#define BITNET_NORM_SHAPES(F)                                                                                  \
  F(64, 1, true) F(64, 1, false) F(64, 2, false) F(64, 3, false) F(64, 4, false) F(64, 5, false)               \
  F(128, 3, false) F(256, 2, false) F(256, 3, false) F(256, 4, false) F(512, 3, false) F(512, 4, false)        \
  F(512, 5, false) F(512, 6, false) F(512, 7, false) F(512, 8, false)

// Row groups of a launch.
static int64_t row_groups(int64_t M, const RowSplit& s) {
  const int64_t rpb = s.tpr < 256 ? 256 / s.tpr : 1;
  return (M + rpb - 1) / rpb;
}

template <class T, class P, int TPR, int CPT, bool SHORT>
static hipError_t norm_fwd_at(const NormFwd& a, int64_t groups, hipStream_t st) {
  constexpr int BLOCK = TPR < 256 ? 256 : TPR;
  constexpr int64_t kMost = 256 * (norm_fwd_waves<T, CPT>() * 256 / BLOCK);  // on 256 CUs
  layernorm_fwd_kernel<T, P, BLOCK, TPR, CPT, SHORT><<<(unsigned)std::min(groups, kMost), BLOCK, 0, st>>>(a);
  return hipGetLastError();
}

template <class T, class P>
static hipError_t norm_fwd(const NormFwd& a, hipStream_t st) {
  const RowSplit s = row_split(a.K);
#define BITNET_CASE(TPR, CPT, SHORT)                        \
  if (s.tpr == TPR && s.cpt == CPT && SHORT == (a.K < 8))   \
    return norm_fwd_at<T, P, TPR, CPT, SHORT>(a, row_groups(a.M, s), st);
  BITNET_NORM_SHAPES(BITNET_CASE)
#undef BITNET_CASE
  return hipErrorInvalidValue;
}

hipError_t launch_layernorm_fwd(const void* x, bool x_f32, const void* w, const void* b, bool p_f32, int64_t M,
                                int64_t K, float eps, void* y, bool y_f32, float* mean, float* rstd, int8_t* codes,
                                float* scales, hipStream_t stream) {
  const NormFwd a{x, NormParams{w, b, p_f32}, M, (int)K, (int)(ckpt_pad(K) / 8), eps, y, y_f32, mean, rstd, codes, scales};
  if (x_f32) return p_f32 ? norm_fwd<float, float>(a, stream) : norm_fwd<float, uint16_t>(a, stream);
  return p_f32 ? norm_fwd<uint16_t, float>(a, stream) : norm_fwd<uint16_t, uint16_t>(a, stream);
}

// Blocks of the backward: enough for two of 256 threads on each of 256 CUs,
// no more than there are row groups.
constexpr int kNormBwdBlocks = 512;
static int norm_bwd_blocks(int64_t M, int64_t K) {
  const RowSplit s = row_split(K);
  return (int)std::min<int64_t>(row_groups(M, s), s.tpr == 512 ? kNormBwdBlocks / 2 : kNormBwdBlocks);
}

size_t layernorm_bwd_workspace(int64_t M, int64_t K) { return (size_t)norm_bwd_blocks(M, K) * 2 * (size_t)K * 4; }

template <class X, class DX, class DY>
static hipError_t norm_bwd(const NormBwd& a, hipStream_t st) {
  const RowSplit s = row_split(a.K);
  const int blocks = norm_bwd_blocks(a.M, a.K);
#define BITNET_CASE(TPR, CPT, SHORT)                                                               \
  if (s.tpr == TPR && s.cpt == CPT && SHORT == (a.K < 8)) {                                        \
    constexpr int BLOCK = TPR < 256 ? 256 : TPR;                                                   \
    layernorm_bwd_kernel<X, DX, DY, BLOCK, TPR, CPT, SHORT><<<blocks, BLOCK, (size_t)a.nch * 32, st>>>(a); \
    return hipGetLastError();                                                                      \
  }
  BITNET_NORM_SHAPES(BITNET_CASE)
#undef BITNET_CASE
  return hipErrorInvalidValue;
}

hipError_t launch_layernorm_bwd(const void* dY, bool dy_f32, const void* x, bool x_f32, const int8_t* codes,
                                const float* scales, const void* w, bool p_f32, const float* mean, const float* rstd,
                                int64_t M, int64_t K, void* dX, void* dw, void* db, void* ws, hipStream_t stream) {
  NormBwd a{};
  a.dY = dY;
  a.x = x;
  a.codes = codes;
  a.scales = scales;
  a.p = NormParams{w, nullptr, p_f32};
  a.mean = mean;
  a.rstd = rstd;
  a.M = M;
  a.K = (int)K;
  a.nch = (int)(ckpt_pad(K) / 8);
  a.dX = dX;
  a.partials = dw || db ? static_cast<float*>(ws) : nullptr;
  hipError_t e;
  if (codes && x_f32) e = dy_f32 ? norm_bwd<FromCodes, float, float>(a, stream) : norm_bwd<FromCodes, float, uint16_t>(a, stream);
  else if (codes) e = dy_f32 ? norm_bwd<FromCodes, uint16_t, float>(a, stream) : norm_bwd<FromCodes, uint16_t, uint16_t>(a, stream);
  else if (x_f32) e = dy_f32 ? norm_bwd<FromF32, float, float>(a, stream) : norm_bwd<FromF32, float, uint16_t>(a, stream);
  else e = dy_f32 ? norm_bwd<FromBf16, uint16_t, float>(a, stream) : norm_bwd<FromBf16, uint16_t, uint16_t>(a, stream);
  if (e != hipSuccess || a.partials == nullptr) return e;
  layernorm_cols_kernel<<<(unsigned)((2 * K + 63) / 64), 1024, 0, stream>>>(a.partials, norm_bwd_blocks(M, K), (int)K,
                                                                            dw, db, p_f32);
  return hipGetLastError();
}

}  // namespace bitnet
