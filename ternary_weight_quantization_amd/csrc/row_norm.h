// Row reductions of the norms: a row lives in the registers of TPR threads
// (whole waves) in chunks of 8 values.
#pragma once

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

// The largest bit pattern over the threads of a row, likewise.
template <int TPR>
__device__ __forceinline__ uint32_t row_max_bits(uint32_t v, float* slot) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)v, off, kWave);
    v = o > v ? o : v;
  }
  if constexpr (TPR > kWave) {
    constexpr int W = TPR / kWave;
    const int w0 = threadIdx.x / TPR * W;
    if (threadIdx.x % kWave == 0) slot[threadIdx.x / kWave] = __uint_as_float(v);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const uint32_t o = __float_as_uint(slot[w0 + j]);
      v = o > v ? o : v;
    }
  }
  return v;
}

// Keeps a loaded chunk as it is across a row's reduction: the values derived
// from it are computed again after it instead of being held in registers.
__device__ __forceinline__ void hold(ChunkBf16& c) { asm volatile("" : "+v"(c.v.x), "+v"(c.v.y), "+v"(c.v.z), "+v"(c.v.w)); }
__device__ __forceinline__ void hold(ChunkF32& c) {
  asm volatile("" : "+v"(c.a.x), "+v"(c.a.y), "+v"(c.a.z), "+v"(c.a.w), "+v"(c.b.x), "+v"(c.b.y), "+v"(c.b.z), "+v"(c.b.w));
}

// Threads a row and chunks a thread of the RMS norm (K <= kRmsMaxK), from the
// row length alone, as the layer norm's (measured there): one wave up to five
// chunks a thread, two waves for three, four up to four chunks, eight above.
// Both chunk counts and tpr are multiples of 16, so every chunk before a
// thread's last lies inside the row.
struct RmsSplit {
  int tpr, cpt;
};
inline RmsSplit rms_split(int64_t K) {
  const int nch = (int)(ckpt_pad(K) / 8);
  const int tpr = nch <= 320 ? 64 : nch <= 384 ? 128 : nch <= 1024 ? 256 : 512;
  return {tpr, (nch + tpr - 1) / tpr};
}
inline int64_t rms_groups(int64_t M, const RmsSplit& s) {
  const int64_t rpb = s.tpr < 256 ? 256 / s.tpr : 1;
  return (M + rpb - 1) / rpb;
}
// Every pair that rms_split gives, and rows of fewer than 8 values.
#define BITNET_RMS_SHAPES(F)                                                                                   \
  F(64, 1, true) F(64, 1, false) F(64, 2, false) F(64, 3, false) F(64, 4, false) F(64, 5, false)               \
  F(128, 3, false) F(256, 2, false) F(256, 3, false) F(256, 4, false) F(512, 3, false) F(512, 4, false)

}  // namespace bitnet
