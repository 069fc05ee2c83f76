// One row of bf16 or f32 values to 8-bit codes with a scale, in the registers of
// TPR threads.

#pragma once

#include "row_norm.h"

namespace bitnet {

// s from the largest magnitude's bits: a row that holds an infinity or a NaN stands
// for NaN throughout.
__device__ __forceinline__ float row_scale(uint32_t m) {
  return m >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : fmaxf(__uint_as_float(m), 1e-8f);
}

template <class T>
struct QuantRows {
  const T* x;  // [rows][K]
  int64_t rows;
  int8_t* q;   // [rows][8 nq]
  float* s;
};

// Row `row` (uniform in a wave; at or past the end: nothing is written). `slot`: a float
// per wave of the block.
template <class T, int TPR, int CPT, bool SHORT>
__device__ __forceinline__ void quant_row(const QuantRows<T>& a, int64_t row, int K, int nq, float* slot) {
  const int t = threadIdx.x % TPR, k_last = 8 * (t + (CPT - 1) * TPR);
  const bool ok = row < a.rows;
  const T* xr = a.x + (ok ? row : a.rows - 1) * K;
  typename ChunkOf<T>::type c[CPT];
  // nq and TPR are multiples of 8, so only a thread's last chunk can reach past K
#pragma unroll
  for (int i = 0; i < CPT - 1; ++i) c[i] = load8_in(xr + 8 * (t + i * TPR));
  c[CPT - 1] = load8<SHORT>(xr, k_last, K);
  settle8<SHORT>(c[CPT - 1], k_last, K);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const uint32_t o = magnitude8(c[i]);
    m = o > m ? o : m;
  }
  const float s = row_scale(row_max_bits<TPR>(m, slot));
  if (!ok) return;
  if (t == 0) a.s[row] = s;
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int ch = t + i * TPR;
    if (i == CPT - 1 && ch >= nq) continue;
    float f[8];
    c[i].get(f);
    reinterpret_cast<uint2*>(a.q)[row * nq + ch] = codes8(f, s);
  }
}

}  // namespace bitnet
