// Root-mean-square norm over rows of K values, forward, with the residual's
// addition before it and an output in 8 bits with a scale a row:
//
//   h = round(res + x)  (or x alone),  r = (sum h^2 / K + eps)^(-1/2),  v = h r w
//   y = round(v), or s = max(max |v|, 1e-8), q = round_half_even(127 v / s)
//
// Backward: rms_bwd_kernels.hip. A row lives in the registers of TPR threads
// in chunks of 8 values, as in the layer norm (norm_kernels.hip): every input
// is read once, the stream and the rows are written once. For 8-bit rows the
// largest |h w| is taken along with the sum of squares, before r is known: then
// s = r max |h w|, q = round(h w (127 / max |h w|)), one reduction and one pass over the
// row's registers. Statistics are fp32, and no rounding to bf16 comes between h
// and q. Bound by HBM once there are rows enough: 16384 x 6912 bf16 to 8-bit rows 69
// us (340 MB, 4.9 TB/s), 4096 x 2560 with a residual 15.0 (73 MB, 4.9 TB/s), 1537 x 6905
// bf16 onto an f32 stream 24 (127 MB, 5.3 TB/s). One row of 2560 takes 4.6, where a launch
// of little work is 1.9 and a row's 8-bit codes alone are 2.9: its threads are chosen for
// many rows, one wave that loads five chunks of three operands, after a vote of the
// block on the weight.

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
  void* y;  // (not QUANT)
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
// weight and h w in fp32) leave registers for. The launch takes as many blocks as
// run together. B: bytes read a value.
template <int B, int CPT>
constexpr int rms_fwd_waves() {
  if (B == 2) return CPT <= 4 ? 4 : 3;
  if (B == 8) return CPT <= 2 ? 3 : CPT <= 4 ? 2 : 1;
  return CPT <= 2 ? 4 : CPT == 3 ? 3 : 2;
}
template <class T, class X, bool ADD>
constexpr int rms_fwd_bytes() { return (int)(sizeof(T) + (ADD ? sizeof(X) : 0)); }

// round_half_even(f k) of 8 values as int8, |f k| <= 127.
__device__ __forceinline__ uint2 codes8_scaled(const float (&f)[8], float k) {
  uint32_t t[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) t[e] = __float_as_uint(fmaf(f[e], k, kCodeMagic));  // the low byte
  const auto pack = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return perm(perm(d, c, 0x0C0C0400u), perm(b, a, 0x0C0C0400u), 0x05040100u);
  };
  return make_uint2(pack(t[0], t[1], t[2], t[3]), pack(t[4], t[5], t[6], t[7]));
}

// a / b in fp32, rounded up (a, b > 0).
__device__ __forceinline__ float div_up(float a, float b) {
  const float k = a / b;
  return fmaf(k, b, -a) < 0.0f ? __uint_as_float(__float_as_uint(k) + 1u) : k;
}

// Sum of v and maximum of m over the TPR threads of a row, in every one of them.
template <int TPR>
__device__ __forceinline__ void row_sum_max(float& v, float& m, float* vs, float* ms) {
  v = wave_sum_f32(v);
  m = wave_max_f32(m);
  if constexpr (TPR > kWave) {
    constexpr int W = TPR / kWave;
    const int w0 = threadIdx.x / TPR * W;
    if (threadIdx.x % kWave == 0) {
      vs[threadIdx.x / kWave] = v;
      ms[threadIdx.x / kWave] = m;
    }
    __syncthreads();
    v = vs[w0];
    m = ms[w0];
#pragma unroll
    for (int j = 1; j < W; ++j) {
      v += vs[w0 + j];
      m = fmaxf(m, ms[w0 + j]);
    }
  }
}

// T: the stream's type. X: the branch's type where ADD (else T). QUANT: 8-bit rows.
// SHORT: K < 8.
// A block takes rows (TPR threads each) in turn; the weight stays in its
// registers and the next row is requested before the current one is reduced.
template <class T, class X, bool ADD, bool QUANT, int BLOCK, int TPR, int CPT, bool SHORT>
__global__ __launch_bounds__(BLOCK, (rms_fwd_waves<rms_fwd_bytes<T, X, ADD>(), CPT>())) void rmsnorm_fwd_kernel(RmsFwd a) {
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
  bool w_bad = false;  // a weight that is not finite: every row stands for NaN
  if constexpr (QUANT) {
    int bad = 0;
#pragma unroll
    for (int i = 0; i < CPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) bad |= (__float_as_uint(w[i][e]) & 0x7F800000u) == 0x7F800000u;
    w_bad = __syncthreads_or(bad) != 0;
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
    float sq = 0.0f, mx = 0.0f, hw[CPT][8];  // hw, mx: QUANT
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
      if constexpr (QUANT) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          hw[i][e] = f[e] * w[i][e];
          mx = fmaxf(mx, fabsf(hw[i][e]));
        }
      } else {
        hold(c[i]);
      }
    }
    // two slot pairs in turn: a row's readers are done with one pair before
    // the barrier of the next row, after which it may be written again
    if constexpr (QUANT) row_sum_max<TPR>(sq, mx, slot[flip], slot[flip + 1]);
    else sq = row_sum<TPR>(sq, slot[flip]);
    const float r = 1.0f / sqrtf(sq * inv_k + a.eps);
    if (ok && t == 0 && a.rstd) a.rstd[row] = r;
    if constexpr (QUANT) {
      // a row that holds an infinity or a NaN, or whose r is one (no positive sum under
      // the root), stands for NaN throughout
      const float inf = __uint_as_float(0x7F800000u);
      const bool fine = sq < inf && r < inf && mx < inf && !w_bad;
      const float top = r * mx;
      const float s = fine ? fmaxf(top, 1e-8f) : __uint_as_float(0x7FC00000u);
      // 127 r / s without r where it cancels, rounded up: half of the largest |h w| then
      // gives 63.5 or more, to 64 as half-even wants it, and where the largest is 127 2^j
      // the factor and every tie are exact. (Each quotient decided exactly, as codes8
      // does: 16384 x 6912 81 us, 64.6 so.)
      const float k = top > 1e-8f ? div_up(127.0f, mx) : 127.0f * r / 1e-8f;
      if (ok) {
        if (t == 0) a.sx[row] = s;
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
          const int ch = t + i * TPR;
          if (i == CPT - 1) {
            if (ch >= a.nq) continue;
            const int left = K - k_last;
            if (left < 8) {  // in a row with a NaN the padding would be NaN too
#pragma unroll
              for (int e = 0; e < 8; ++e) hw[i][e] = e < left ? hw[i][e] : 0.0f;
            }
          }
          const uint2 q = codes8_scaled(hw[i], fine ? k : 0.0f);
          reinterpret_cast<uint2*>(a.xq)[row * a.nq + ch] = q;
        }
      }
    } else if (ok) {
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        const int k0 = 8 * (t + i * TPR);
        float f[8];
        c[i].get(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = f[e] * r * w[i][e];
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

template <class T, class X, bool ADD, bool QUANT, int TPR, int CPT, bool SHORT>
static hipError_t rms_fwd_at(const RmsFwd& a, int64_t groups, hipStream_t st) {
  constexpr int BLOCK = TPR < 256 ? 256 : TPR;
  constexpr int64_t kMost = 256 * (rms_fwd_waves<rms_fwd_bytes<T, X, ADD>(), CPT>() * 256 / BLOCK);  // on 256 CUs
  rmsnorm_fwd_kernel<T, X, ADD, QUANT, BLOCK, TPR, CPT, SHORT><<<(unsigned)std::min(groups, kMost), BLOCK, 0, st>>>(a);
  return hipGetLastError();
}

template <class T, class X, bool ADD, bool QUANT>
static hipError_t rms_fwd(const RmsFwd& a, hipStream_t st) {
  const RmsSplit s = rms_split(a.K);
#define BITNET_CASE(TPR, CPT, SHORT)                      \
  if (s.tpr == TPR && s.cpt == CPT && SHORT == (a.K < 8)) \
    return rms_fwd_at<T, X, ADD, QUANT, TPR, CPT, SHORT>(a, rms_groups(a.M, s), st);
  BITNET_RMS_SHAPES(BITNET_CASE)
#undef BITNET_CASE
  return hipErrorInvalidValue;
}

template <class T, class X, bool ADD>
static hipError_t rms_fwd(const RmsFwd& a, hipStream_t st) {
  return a.y == nullptr ? rms_fwd<T, X, ADD, true>(a, st) : rms_fwd<T, X, ADD, false>(a, st);
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

}  // namespace bitnet
