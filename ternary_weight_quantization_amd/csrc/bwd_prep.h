// The operands that the backward products rebuild from the saved state: bf16
// x_hat from int8 rows, and the ternary codes transposed to fp4.
#pragma once

#include "device_common.h"

namespace bitnet {

// dW P: x_hat = bf16(fl32(x_q * fl32(s/127))) is built once per backward
// call into the workspace ([M][Kp] bf16; for the scales act-quant produces
// it equals the exactly rounded bf16(x_q * s / 127)) and then staged like dY
// (RowTransposeBf16Loader). Each element is converted once instead of once
// per output tile column. Thread t converts 16 int8 of row m: each byte is
// biased to [1, 255] so that u*r - 128r = x_q*r exactly before the single
// rounding of the fma.
// 16 int8 of a row with scale factor r = s / 127 -> 16 bf16 (lo: values
// 0..7, hi: 8..15). The one definition of x_hat's arithmetic: the pre-pass
// and the few-token dW kernel, which converts its own slice, both call it.
__device__ __forceinline__ void xhat16(uint4 v, float r, uint4& lo, uint4& hi) {
  const float bias = -128.0f * r;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[8];
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const uint32_t u = w[d] ^ 0x80808080u;
    o[2 * d] = pack_bf16x2(fmaf((float)(u & 0xFFu), r, bias), fmaf((float)((u >> 8) & 0xFFu), r, bias));
    o[2 * d + 1] = pack_bf16x2(fmaf((float)((u >> 16) & 0xFFu), r, bias), fmaf((float)(u >> 24), r, bias));
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// s NULL: the codes themselves (exact).
__device__ __forceinline__ void xhat_blocks(const int8_t* __restrict__ xq, const float* __restrict__ s, int64_t M,
                                            int64_t Kp, uint16_t* __restrict__ xhat, int b, int nb) {
  const int64_t cpr = Kp / 16;  // 16-byte chunks per row
  const int64_t total = M * cpr;
  for (int64_t c = (int64_t)b * 256 + threadIdx.x; c < total; c += (int64_t)nb * 256) {
    const int64_t m = c / cpr;
    uint4* dst = reinterpret_cast<uint4*>(xhat) + 2 * c;
    xhat16(reinterpret_cast<const uint4*>(xq)[c], s != nullptr ? s[m] / 127.0f : 1.0f, dst[0], dst[1]);
  }
}

// dX P: the ternary codes transposed to [k][n] as fp4 nibbles (the layout
// CodesFp4Frags reads: n even in the low nibble, +1 = 0x2, -1 = 0xA, 0 =
// 0x0), rows of Np/2 bytes with Np = N rounded up to 64 (zero nibbles past
// N), built once per backward call into the workspace and then copied stage
// by stage like the forward's codes (RowCodesLoader). A block covers 64 k x
// 256 n: thread t loads the 64 codes k0..k0+63 of row n0 + t (16 bytes, 4
// planar words; code j of a word sits at bit 8(j%4) + 2(j/4)), then writes
// the 64 nibbles n0 + 64(t%4) + 0..63 of row k0 + t/4 (32 bytes). row(n): the
// row of packed that n stands for, negative for none (zeros).
template <class ROW>
__device__ __forceinline__ void wt_fp4_block(const uint8_t* __restrict__ packed, const ROW& row, int64_t Kp, int64_t Np,
                                             uint8_t* __restrict__ wt, int bx, int by) {
  // tile[word][n]: the 4 words of each row, word-major so that the words
  // of 4 consecutive rows are one 16-byte read
  __shared__ __attribute__((aligned(16))) uint32_t tile[4][256 + 4];
  const int t = threadIdx.x;
  const int64_t k0 = (int64_t)bx * 64, n0 = (int64_t)by * 256;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  const int64_t at = row(n0 + t);
  if (at >= 0) v = *reinterpret_cast<const uint4*>(packed + at * (Kp / 4) + k0 / 4);
  tile[0][t] = v.x;
  tile[1][t] = v.y;
  tile[2][t] = v.z;
  tile[3][t] = v.w;
  __syncthreads();
  // code j of a word: byte j % 4, bits 2(j / 4)
  const int kl = t >> 2, w = kl >> 4, j = kl & 15;
  const uint32_t byte = j & 3, sh = 2 * (j >> 2);
  const uint32_t gsel = byte | ((byte + 4) << 8);
  const int nb = 64 * (t & 3);
  if (n0 + nb >= Np) return;
  // nibbles of rows n..n+3 (4 words) -> bytes 0 and 2 of the result
  const auto quad = [&](uint4 a) {
    const uint32_t g = perm(perm(a.w, a.z, gsel), perm(a.y, a.x, gsel), 0x05040100u);  // byte e: row n+e
    const uint32_t f = perm(0u, 0x0A000200u, (g >> sh) & 0x03030303u);                 // code 0, 1, 3 -> fp4 0, 2, A
    return f | (f >> 4);
  };
  const uint4* src = reinterpret_cast<const uint4*>(&tile[w][nb]);
  uint32_t o[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) o[q] = perm(quad(src[2 * q + 1]), quad(src[2 * q]), 0x06040200u);
  uint4* dst = reinterpret_cast<uint4*>(wt + (k0 + kl) * (Np / 2) + (n0 + nb) / 2);
  dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
  dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

// Transpose blocks in XCD-major order. Blocks are dispatched round-robin
// over the 8 XCDs (block b on XCD b % 8), and the 8 k-blocks that read one
// 128-byte line of a code row are neighbours; numbered as they come, each
// line was fetched once per XCD into 8 private L2s. Here the blocks of one
// XCD take consecutive indices (k fastest), so the line's readers share one
// L2. The first 8 * floor(nb / 8) indices are permuted; the rest keep
// theirs.
__device__ __forceinline__ int xcd_major(int b, int nb) {
  const int per = nb / 8;
  return b < per * 8 ? (b % 8) * per + b / 8 : b;
}

}  // namespace bitnet
