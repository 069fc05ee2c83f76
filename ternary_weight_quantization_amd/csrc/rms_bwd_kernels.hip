// Backward of the root-mean-square norm (rms_kernels.hip):
//
//   g  = dY w,  hn = h r,  c = sum g hn / K
//   dh = r (g - hn c) + dH,  dw = sum over rows dY hn
//
// dH is the gradient of the stream h itself (what later layers read), dY that
// of the norm's output, straight through its quantization. dY, h and dH are
// read once. The weight's gradient is a column sum over all rows: registers
// over the rows of a block, LDS over its row groups, one partial row a block,
// added in block order by a second launch (launch_norm_cols). No atomics: the
// same inputs give the same bits. Measured with the second launch: 16384 x 6912 bf16
// 152 us (680 MB, 4.5 TB/s), 1537 x 6905 f32 with dH 39 (170 MB, 4.3), 4096 x 2560 bf16
// with dH 22.8 (84 MB, 3.7): the smaller ones end with the blocks' partial rows and the
// second launch, 4 to 5 us of it.

#include <algorithm>

#include "internal.h"
#include "row_norm.h"

namespace bitnet {

struct RmsBwd {
  const void* dY;
  const void* h;
  const void* dH;
  const void* w;
  bool p_f32;
  const float* rstd;
  int64_t M;
  int K, nch;
  void* dh;         // T, NULL: not written
  uint16_t* dx;     // bf16 copy of an f32 stream's gradient, NULL: not written
  float* partials;  // [blocks][K], NULL: no column sums
};

// The weight as fp32 in LDS: every row of the block reads it twice.
extern __shared__ __attribute__((aligned(16))) float rms_lds[];

template <class T, class DY, bool DH, int BLOCK, int TPR, int CPT, bool SHORT>
__global__ __launch_bounds__(BLOCK, BLOCK == 512 ? 1 : 2) void rmsnorm_bwd_kernel(RmsBwd a) {
  constexpr int RPB = BLOCK / TPR;
  typedef typename ChunkOf<DY>::type CD;
  typedef typename ChunkOf<T>::type CT;
  __shared__ float slot[2][BLOCK / kWave];
  const int t = threadIdx.x % TPR;
  const int rl = __builtin_amdgcn_readfirstlane((int)threadIdx.x / TPR);  // whole waves share a row
  const int K = a.K;
  for (int k = threadIdx.x; k < a.nch; k += BLOCK) {
    float w[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
    if (a.w) param8(a.w, a.p_f32, 8 * k, K, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) rms_lds[8 * k + e] = w[e];
  }
  __syncthreads();
  float dw[CPT][8];
#pragma unroll
  for (int i = 0; i < CPT; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.0f;

  // only a thread's last chunk can reach past K (rms_split): dY and h are zero
  // there, so nothing is added
  const int k_end = 8 * (t + (CPT - 1) * TPR);
  const auto load1 = [&](auto* row, auto (&v)[CPT]) {
#pragma unroll
    for (int i = 0; i < CPT - 1; ++i) v[i] = load8_in(row + 8 * (t + i * TPR));
    v[CPT - 1] = load8<SHORT>(row, k_end, K);
  };
  const auto load = [&](int64_t row, CD (&cd)[CPT], CT (&ch)[CPT], CT (&cg)[CPT]) {
    load1(static_cast<const DY*>(a.dY) + row * K, cd);
    load1(static_cast<const T*>(a.h) + row * K, ch);
    if constexpr (DH) load1(static_cast<const T*>(a.dH) + row * K, cg);
  };
  // what a chunk past the row's end reads of the weight (chunk 0) does not matter
  const int k_last = t + (CPT - 1) * TPR < a.nch ? k_end : 0;
  // The next row is loaded while this one is reduced where both fit the
  // registers next to the column sums (4096 x 2560 bf16 with dH, 60 dwords a row and
  // thread: 18.9 us without it, 23.8 with it and 18 registers spilled).
  constexpr bool AHEAD = (sizeof(CD) + sizeof(CT) * (DH ? 2 : 1)) / 4 * CPT <= 40;
  CD cd[CPT], nd[CPT];
  CT ch[CPT], nh[CPT], cg[CPT], ng[CPT];
  // The block's row groups; every thread passes every barrier. Past the last
  // row a wave (rows are uniform in a wave) repeats it with dY = 0.
  const int64_t stride = (int64_t)gridDim.x * RPB, last = a.M - 1;
  int64_t base = (int64_t)blockIdx.x * RPB, row = base + rl < last ? base + rl : last;
  if constexpr (AHEAD) load(row, cd, ch, cg);
  float r = a.rstd[row];
  int flip = 0;
  for (; base < a.M; base += stride, flip ^= 1) {
    const bool ok = base + rl < a.M;
    const int64_t want = base + stride + rl, next = want < last ? want : last;
    if constexpr (AHEAD) load(next, nd, nh, ng);
    else load(row, cd, ch, cg);
    const float nr = a.rstd[next];
    if (!ok) {
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        cd[i] = CD{};
        ch[i] = CT{};
      }
    }
    settle8<SHORT>(cd[CPT - 1], k_end, K);
    settle8<SHORT>(ch[CPT - 1], k_end, K);
    if constexpr (DH) settle8<SHORT>(cg[CPT - 1], k_end, K);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const float* w = rms_lds + (i < CPT - 1 ? 8 * (t + i * TPR) : k_last);
      float d[8], f[8];
      cd[i].get(d);
      ch[i].get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float hn = f[e] * r;
        sum = fmaf(d[e] * w[e], hn, sum);
        dw[i][e] = fmaf(d[e], hn, dw[i][e]);
      }
      hold(cd[i]);
      hold(ch[i]);
      __builtin_amdgcn_sched_barrier(0);  // one chunk's values at a time
    }
    // two slots in turn: a row's readers are done with one before the barrier
    // of the next row, after which it may be written again
    const float c = row_sum<TPR>(sum, slot[flip]) / (float)K * r;
    if (ok && (a.dh != nullptr || a.dx != nullptr)) {
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        const float* w = rms_lds + (i < CPT - 1 ? 8 * (t + i * TPR) : k_last);
        float d[8], f[8], o[8];
        cd[i].get(d);
        ch[i].get(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fmaf(-c, f[e] * r, d[e] * w[e] * r);
        if constexpr (DH) {
          float g[8];
          cg[i].get(g);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] += g[e];
        }
        const int k0 = 8 * (t + i * TPR);
        if (a.dh != nullptr) {
          T* out = static_cast<T*>(a.dh) + row * K;
          if (i < CPT - 1) store8_in(out + k0, o);
          else store8(out, k0, K, o);
        }
        if constexpr (sizeof(T) == 4) {
          if (a.dx != nullptr) {
            uint16_t* out = a.dx + row * K;
            if (i < CPT - 1) store8_in(out + k0, o);
            else store8(out, k0, K, o);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (AHEAD) {
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        cd[i] = nd[i];
        ch[i] = nh[i];
        if constexpr (DH) cg[i] = ng[i];
      }
    }
    r = nr;
    row = next;
  }

  if (a.partials == nullptr) return;
  float* out = a.partials + (int64_t)blockIdx.x * K;
  if constexpr (RPB > 1) {
    // the block's rows in turn, one chunk column at a time
    __shared__ float acc[RPB][TPR][9];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[rl][t][e] = dw[i][e];
      __syncthreads();
      // 8 * TPR sums over RPB rows by the block
      for (int j = threadIdx.x; j < 8 * TPR; j += BLOCK) {
        float v = acc[0][j >> 3][j & 7];
#pragma unroll
        for (int q = 1; q < RPB; ++q) v += acc[q][j >> 3][j & 7];
        const int k = 8 * TPR * i + j;
        if (k < K) out[k] = v;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int k0 = 8 * (t + i * TPR);
      if (k0 < K) store8(out, k0, K, dw[i]);
    }
  }
}

// Blocks: enough for two of 256 threads on each of 256 CUs, no more than there
// are row groups.
constexpr int kRmsBwdBlocks = 512;
static int rms_bwd_blocks(int64_t M, int64_t K) {
  const RmsSplit s = rms_split(K);
  return (int)std::min<int64_t>(rms_groups(M, s), s.tpr == 512 ? kRmsBwdBlocks / 2 : kRmsBwdBlocks);
}

size_t rmsnorm_bwd_workspace(int64_t M, int64_t K) { return (size_t)rms_bwd_blocks(M, K) * (size_t)K * 4; }

template <class T, class DY, bool DH>
static hipError_t rms_bwd(const RmsBwd& a, hipStream_t st) {
  const RmsSplit s = rms_split(a.K);
  const int blocks = rms_bwd_blocks(a.M, a.K);
#define BITNET_CASE(TPR, CPT, SHORT)                                                                            \
  if (s.tpr == TPR && s.cpt == CPT && SHORT == (a.K < 8)) {                                                     \
    constexpr int BLOCK = TPR < 256 ? 256 : TPR;                                                                \
    rmsnorm_bwd_kernel<T, DY, DH, BLOCK, TPR, CPT, SHORT><<<blocks, BLOCK, (size_t)a.nch * 32, st>>>(a);        \
    return hipGetLastError();                                                                                   \
  }
  BITNET_RMS_SHAPES(BITNET_CASE)
#undef BITNET_CASE
  return hipErrorInvalidValue;
}

template <class T, class DY>
static hipError_t rms_bwd(const RmsBwd& a, hipStream_t st) {
  return a.dH != nullptr ? rms_bwd<T, DY, true>(a, st) : rms_bwd<T, DY, false>(a, st);
}

hipError_t launch_rmsnorm_bwd(const void* dY, bool y_f32, const void* dH, const void* h, bool h_f32, const void* w,
                              bool p_f32, const float* rstd, int64_t M, int64_t K, void* dh, uint16_t* dx, void* dw,
                              void* ws, hipStream_t stream) {
  const RmsBwd a{dY, h, dH, w, p_f32, rstd, M, (int)K, (int)(ckpt_pad(K) / 8), dh, dx,
                 dw ? static_cast<float*>(ws) : nullptr};
  hipError_t e;
  if (h_f32) e = y_f32 ? rms_bwd<float, float>(a, stream) : rms_bwd<float, uint16_t>(a, stream);
  else e = y_f32 ? rms_bwd<uint16_t, float>(a, stream) : rms_bwd<uint16_t, uint16_t>(a, stream);
  if (e != hipSuccess || dw == nullptr) return e;
  return launch_norm_cols(a.partials, rms_bwd_blocks(M, K), 1, K, dw, nullptr, p_f32, stream);
}

}  // namespace bitnet
