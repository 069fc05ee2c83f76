// Root-mean-square norm over rows of K values, forward, with the residual's
// addition before it and an output in 8 bits with a scale a row:
//
//   h = round(res + x)  (or x alone),  r = (sum h^2 / K + eps)^(-1/2),  v = h r w
//   y = round(v), or s = max(max |v|, 1e-8), q = round_half_even(127 v / s)
//
// Backward: rms_bwd_kernels.hip. A row lives in the registers of TPR threads
// in chunks of 8 values, as in the layer norm (norm_kernels.hip): every input
// is read once, the stream and the rows are written once. Two row reductions,
// the sum of squares and, for 8-bit rows, the largest magnitude; v is computed
// again after each rather than held. Statistics are fp32, v is quantized from
// fp32 without a rounding to bf16 between.

#include <algorithm>

#include "internal.h"
#include "row_norm.h"

namespace bitnet {

struct RmsFwd {
  const void* x;
  const void* res;
  const void* w;  // [K] or NULL
  bool p_f32;     // its type
  int64_t M;
  int K, nch, nq;  // chunks of a row, of its 8-bit codes
  float eps;
  void* h;
  void* y;  // NULL: 8-bit rows
  bool y_f32;
  int8_t* xq;
  float* sx;
  float* rstd;  // NULL: not wanted
};

__device__ __forceinline__ void from8(ChunkBf16& c, const float (&f)[8]) {
  c.v = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void from8(ChunkF32& c, const float (&f)[8]) {
  c.a = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  c.b = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
}

// Waves a SIMD holds: what a thread's chunks (this row's, the next row's, the
// weight in fp32) leave registers for.
template <class T, int CPT>
constexpr int rms_fwd_waves() {
  return CPT <= 2 ? 4 : CPT == 3 ? 3 : 2;
}

// T: the stream's type. X: the branch's type where ADD (else T). SHORT: K < 8.
// A block takes rows (TPR threads each) in turn; the weight stays in its
// registers and the next row is requested before the current one is reduced.
template <class T, class X, bool ADD, int BLOCK, int TPR, int CPT, bool SHORT>
__global__ __launch_bounds__(BLOCK, (rms_fwd_waves<T, CPT>())) void rmsnorm_fwd_kernel(RmsFwd a) {
  constexpr int RPB = BLOCK / TPR;
  __shared__ float slot[4][BLOCK / kWave];
  const int t = threadIdx.x % TPR;
  const int rl = __builtin_amdgcn_readfirstlane((int)threadIdx.x / TPR);  // whole waves share a row
  const int K = a.K;
  const int k_last = 8 * (t + (CPT - 1) * TPR);
  float w[CPT][8];
  typename ChunkOf<T>::type c[CPT], nc[CPT];
  typename ChunkOf<X>::type cx[CPT], nx[CPT];  // ADD only
  // only a thread's last chunk can reach past K (rms_split)
  const auto load = [&](auto* row, auto (&v)[CPT]) {
#pragma unroll
    for (int i = 0; i < CPT - 1; ++i) v[i] = load8_in(row + 8 * (t + i * TPR));
    v[CPT - 1] = load8<SHORT>(row, k_last, K);
  };
  const X* x = static_cast<const X*>(a.x);
  const T* res = static_cast<const T*>(ADD ? a.res : a.x);
  // Every thread passes every barrier: past the last row a wave (rows are
  // uniform in a wave) repeats it and writes nothing.
  const int64_t stride = (int64_t)gridDim.x * RPB, last = a.M - 1;
  int64_t base = (int64_t)blockIdx.x * RPB, row = base + rl < last ? base + rl : last;
  load(res + row * K, c);
  if constexpr (ADD) load(x + row * K, cx);
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    if (a.w) {
      param8(a.w, a.p_f32, 8 * (t + i * TPR), K, w[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[i][e] = 1.0f;
    }
  }
  const float inv_k = 1.0f / (float)K;
  int flip = 0;
  for (; base < a.M; base += stride, flip ^= 2) {
    const bool ok = base + rl < a.M;
    const int64_t want = base + stride + rl, next = want < last ? want : last;
    const bool more = base + stride < a.M;  // uniform
    if (more) {
      load(res + next * K, nc);
      if constexpr (ADD) load(x + next * K, nx);
    }
    settle8<SHORT>(c[CPT - 1], k_last, K);
    if constexpr (ADD) settle8<SHORT>(cx[CPT - 1], k_last, K);
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      float f[8];
      c[i].get(f);
      if constexpr (ADD) {
        float g[8];
        cx[i].get(g);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] += g[e];
        from8(c[i], f);
        c[i].get(f);  // the norm is of the stream as stored
        if (ok) {
          T* hr = static_cast<T*>(a.h) + row * K;
          if (i < CPT - 1) store8_in(hr + 8 * (t + i * TPR), f);
          else store8(hr, k_last, K, f);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sq = fmaf(f[e], f[e], sq);
      hold(c[i]);
    }
    // two slot pairs in turn: a row's readers are done with one pair before
    // the barrier of the next row, after which it may be written again
    const float r = 1.0f / sqrtf(row_sum<TPR>(sq, slot[flip]) * inv_k + a.eps);
    if (ok && t == 0 && a.rstd) a.rstd[row] = r;
    const auto value8 = [&](int i, float (&f)[8]) {
      c[i].get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = f[e] * r * w[i][e];
      if (i == CPT - 1) {  // a row with a NaN has NaNs past its end too
        const int left = K - k_last;
        if (left < 8) {
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = e < left ? f[e] : 0.0f;
        }
      }
    };
    if (a.y == nullptr) {  // uniform: 8-bit rows
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        float f[8];
        value8(i, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t b = __float_as_uint(f[e]) & 0x7FFFFFFFu;
          m = b > m ? b : m;
        }
        hold(c[i]);
      }
      m = row_max_bits<TPR>(m, slot[flip + 1]);
      // a row that holds an infinity or a NaN stands for NaN throughout
      const float s = m >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : fmaxf(__uint_as_float(m), 1e-8f);
      if (ok) {
        if (t == 0) a.sx[row] = s;
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
          const int ch = t + i * TPR;
          if (i == CPT - 1 && ch >= a.nq) continue;
          float f[8];
          value8(i, f);
          reinterpret_cast<uint2*>(a.xq)[row * a.nq + ch] = codes8(f, s);
        }
      }
    } else if (ok) {
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        const int k0 = 8 * (t + i * TPR);
        float f[8];
        value8(i, f);
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
      for (int i = 0; i < CPT; ++i) {
        c[i] = nc[i];
        if constexpr (ADD) cx[i] = nx[i];
      }
    }
    row = next;
  }
}

template <class T, class X, bool ADD, int TPR, int CPT, bool SHORT>
static hipError_t rms_fwd_at(const RmsFwd& a, int64_t groups, hipStream_t st) {
  constexpr int BLOCK = TPR < 256 ? 256 : TPR;
  constexpr int64_t kMost = 256 * (rms_fwd_waves<T, CPT>() * 256 / BLOCK);  // on 256 CUs
  rmsnorm_fwd_kernel<T, X, ADD, BLOCK, TPR, CPT, SHORT><<<(unsigned)std::min(groups, kMost), BLOCK, 0, st>>>(a);
  return hipGetLastError();
}

template <class T, class X, bool ADD>
static hipError_t rms_fwd(const RmsFwd& a, hipStream_t st) {
  const RmsSplit s = rms_split(a.K);
#define BITNET_CASE(TPR, CPT, SHORT)                      \
  if (s.tpr == TPR && s.cpt == CPT && SHORT == (a.K < 8)) \
    return rms_fwd_at<T, X, ADD, TPR, CPT, SHORT>(a, rms_groups(a.M, s), st);
  BITNET_RMS_SHAPES(BITNET_CASE)
#undef BITNET_CASE
  return hipErrorInvalidValue;
}

hipError_t launch_rmsnorm_fwd(const void* x, bool x_f32, const void* res, bool h_f32, const void* w, bool p_f32,
                              int64_t M, int64_t K, float eps, void* h, void* y, bool y_f32, int8_t* x_q, float* s_x,
                              float* rstd, hipStream_t stream) {
  const RmsFwd a{x, res, w, p_f32, M, (int)K, (int)(ckpt_pad(K) / 8), (int)(k_pad(K) / 8), eps, h, y, y_f32, x_q, s_x,
                 rstd};
  if (res == nullptr) return h_f32 ? rms_fwd<float, float, false>(a, stream) : rms_fwd<uint16_t, uint16_t, false>(a, stream);
  if (!h_f32) return rms_fwd<uint16_t, uint16_t, true>(a, stream);
  return x_f32 ? rms_fwd<float, float, true>(a, stream) : rms_fwd<float, uint16_t, true>(a, stream);
}

// ---------------------------------------------------------------------------
// What 8-bit rows stand for: x[m,k] = fp32(q * fp32(s / 127)), rounded to bf16.
// A thread takes 8 codes.
// ---------------------------------------------------------------------------

__global__ __launch_bounds__(256) void rows_unpack_kernel(const int8_t* __restrict__ xq, const float* __restrict__ s,
                                                          int64_t total, int K, int nq, uint16_t* __restrict__ x) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / nq;
    const int ch = (int)(i - row * nq);
    float f[8];
    values8(reinterpret_cast<const uint2*>(xq)[i], s[row] / 127.0f, f);
    store8(x + row * K, 8 * ch, K, f);
  }
}

hipError_t launch_rows_unpack(const int8_t* x_q, const float* s_x, int64_t M, int64_t K, uint16_t* x,
                              hipStream_t stream) {
  const int nq = (int)(k_pad(K) / 8);
  const int64_t total = M * nq, blocks = (total + 255) / 256;
  rows_unpack_kernel<<<(unsigned)std::min<int64_t>(blocks, 1 << 20), 256, 0, stream>>>(x_q, s_x, total, (int)K, nq, x);
  return hipGetLastError();
}

}  // namespace bitnet
