// 8-bit rows with a scale a row: made of bf16 or f32 rows,
//
//   s = max(max |x|, 1e-8),  q = round_half_even(127 x / s), exactly,
//
// and the bf16 values they stand for. A layer in 8 bits quantizes its
// activations and its weight's channels alike, so both share a launch: one pass
// over HBM, each row in the registers of TPR threads (64 to 256; rows of more than
// 16384 values are read twice, the second time from L2). Rows may start at any
// element. Measured: 4096 x 2560 and 6912 x 2560 bf16 together 20-22 us (85 MB, 4.0
// TB/s; in two launches 24.2), 1000 x 2555 and 2561 x 2555 9.0 (18.4).

#include <algorithm>

#include "rows_quant.h"

namespace bitnet {

constexpr int kQuantBlock = 256;
constexpr int64_t kQuantMaxChunks = 256 * 8;  // of a row in registers

// The rows of a (the first ab blocks) and of b.
template <class TB, int TPR, int CPT, bool SHORT>
__global__ __launch_bounds__(kQuantBlock) void rows_quant_kernel(QuantRows<uint16_t> a, int ab, QuantRows<TB> b, int K,
                                                                 int nq) {
  __shared__ float slot[kQuantBlock / kWave];
  constexpr int RPB = kQuantBlock / TPR;
  const int blk = blockIdx.x, rl = __builtin_amdgcn_readfirstlane((int)threadIdx.x / TPR);
  if (blk < ab) quant_row<uint16_t, TPR, CPT, SHORT>(a, (int64_t)blk * RPB + rl, K, nq, slot);
  else quant_row<TB, TPR, CPT, SHORT>(b, (int64_t)(blk - ab) * RPB + rl, K, nq, slot);
}

template <class T>
__global__ __launch_bounds__(kQuantBlock) void rows_quant_long_kernel(QuantRows<T> a, int K, int nq) {
  __shared__ float slot[kQuantBlock / kWave];
  const int64_t row = blockIdx.x;
  const T* xr = a.x + row * K;
  uint32_t m = 0;
  for (int ch = threadIdx.x; ch < nq; ch += kQuantBlock) {
    const uint32_t o = magnitude8(chunk8(xr, 8 * ch, K));
    m = o > m ? o : m;
  }
  const float s = row_scale(row_max_bits<kQuantBlock>(m, slot));
  if (threadIdx.x == 0) a.s[row] = s;
  for (int ch = threadIdx.x; ch < nq; ch += kQuantBlock) {
    float f[8];
    chunk8(xr, 8 * ch, K).get(f);
    reinterpret_cast<uint2*>(a.q)[row * nq + ch] = codes8(f, s);
  }
}

template <class TB>
static hipError_t rows_quant(const QuantRows<uint16_t>& a, const QuantRows<TB>& b, int64_t K, hipStream_t st) {
  const int nq = (int)(k_pad(K) / 8);
  if (nq > kQuantMaxChunks) {
    if (a.rows > 0) rows_quant_long_kernel<uint16_t><<<(unsigned)a.rows, kQuantBlock, 0, st>>>(a, (int)K, nq);
    if (b.rows > 0) rows_quant_long_kernel<TB><<<(unsigned)b.rows, kQuantBlock, 0, st>>>(b, (int)K, nq);
    return hipGetLastError();
  }
  // as many threads a row as have a chunk: the more rows' loads are in flight on a CU
  const int tpr = nq >= 256 ? 256 : nq >= 128 ? 128 : 64, cpt = (nq + tpr - 1) / tpr;
  const int64_t rpb = kQuantBlock / tpr;
  const int64_t ab = (a.rows + rpb - 1) / rpb, bb = (b.rows + rpb - 1) / rpb;
#define BITNET_CASE(TPR, CPT, SHORT)                                                                                \
  if (tpr == TPR && cpt == CPT && SHORT == (K < 8)) {                                                               \
    rows_quant_kernel<TB, TPR, CPT, SHORT><<<(unsigned)(ab + bb), kQuantBlock, 0, st>>>(a, (int)ab, b, (int)K, nq); \
    return hipGetLastError();                                                                                       \
  }
  BITNET_CASE(64, 1, true) BITNET_CASE(64, 1, false) BITNET_CASE(64, 2, false) BITNET_CASE(128, 1, false)
  BITNET_CASE(128, 2, false) BITNET_CASE(256, 1, false) BITNET_CASE(256, 2, false) BITNET_CASE(256, 3, false)
  BITNET_CASE(256, 4, false) BITNET_CASE(256, 5, false) BITNET_CASE(256, 6, false) BITNET_CASE(256, 7, false)
  BITNET_CASE(256, 8, false)
#undef BITNET_CASE
  return hipErrorInvalidValue;
}

hipError_t launch_rows_quant(const uint16_t* x, int64_t M, int8_t* x_q, float* s_x, const void* w, bool w_f32, int64_t N,
                             int8_t* w_q, float* s_w, int64_t K, hipStream_t stream) {
  const QuantRows<uint16_t> a{x, M, x_q, s_x};
  if (w_f32) return rows_quant(a, QuantRows<float>{static_cast<const float*>(w), N, w_q, s_w}, K, stream);
  return rows_quant(a, QuantRows<uint16_t>{static_cast<const uint16_t*>(w), N, w_q, s_w}, K, stream);
}

// ---------------------------------------------------------------------------
// What 8-bit rows stand for: x[m,k] = fp32(q * fp32(s / 127)), rounded to bf16.
// A thread takes 8 codes (16384 x 6912: 59 us, 340 MB at 5.8 TB/s, the codes partly from
// the last-level cache).
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
