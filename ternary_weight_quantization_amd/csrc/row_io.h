// Rows of bf16 or f32 values in chunks of 8, and the 8-bit codes of blocks
// of 128 values: the device helpers shared by the normalization, activation
// and checkpoint kernels.
#pragma once

#include <string.h>

#include "device_common.h"

namespace bitnet {

// 8 consecutive values of a row as loaded.
struct ChunkBf16 {
  uint4 v;
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
  }
};
struct ChunkF32 {
  uint4 a, b;
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y); f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
    f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y); f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
  }
};
template <class T> struct ChunkOf;
template <> struct ChunkOf<uint16_t> { typedef ChunkBf16 type; };
template <> struct ChunkOf<float> { typedef ChunkF32 type; };

// The 8 values k0 .. k0 + 7 of a row of K, zeros at or past K, in two steps:
// load8 and, once it is needed, settle8. The load is unconditional, so that
// all chunks of a row are in flight together (a load under a condition is
// waited for where the branches join): a chunk that crosses or lies past the
// row's end loads the row's last 8 values, which settle8 moves down. Rows may
// start at any element (unaligned 16-byte loads). SHORT: rows of fewer than 8
// values, read one by one.
template <bool SHORT>
__device__ __forceinline__ ChunkBf16 load8(const uint16_t* row, int k0, int K) {
  ChunkBf16 c;
  if constexpr (SHORT) {
    uint32_t d[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = k0 + 2 * j < K ? row[k0 + 2 * j] : 0u;
      const uint32_t hi = k0 + 2 * j + 1 < K ? row[k0 + 2 * j + 1] : 0u;
      d[j] = lo | (hi << 16);
    }
    c.v = make_uint4(d[0], d[1], d[2], d[3]);
    return c;
  }
  memcpy(&c.v, row + (k0 + 8 <= K ? k0 : K - 8), 16);
  return c;
}
template <bool SHORT>
__device__ __forceinline__ void settle8(ChunkBf16& c, int k0, int K) {
  const int d = k0 + 8 - K;  // values to drop
  if (SHORT || d <= 0) return;
  if (d >= 8) {
    c.v = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  uint32_t w[5] = {c.v.x, c.v.y, c.v.z, c.v.w, 0u};
  if (d & 4) { w[0] = w[2]; w[1] = w[3]; w[2] = 0u; w[3] = 0u; }
  if (d & 2) { w[0] = w[1]; w[1] = w[2]; w[2] = w[3]; w[3] = 0u; }
  if (d & 1) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = (w[j] >> 16) | (w[j + 1] << 16);
  }
  c.v = make_uint4(w[0], w[1], w[2], w[3]);
}
template <bool SHORT>
__device__ __forceinline__ ChunkF32 load8(const float* row, int k0, int K) {
  ChunkF32 c;
  if constexpr (SHORT) {
    uint32_t d[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) d[j] = k0 + j < K ? __float_as_uint(row[k0 + j]) : 0u;
    c.a = make_uint4(d[0], d[1], d[2], d[3]);
    c.b = make_uint4(d[4], d[5], d[6], d[7]);
    return c;
  }
  const float* p = row + (k0 + 8 <= K ? k0 : K - 8);
  memcpy(&c.a, p, 16);
  memcpy(&c.b, p + 4, 16);
  return c;
}
template <bool SHORT>
__device__ __forceinline__ void settle8(ChunkF32& c, int k0, int K) {
  const int d = k0 + 8 - K;
  if (SHORT || d <= 0) return;
  uint32_t w[8] = {c.a.x, c.a.y, c.a.z, c.a.w, c.b.x, c.b.y, c.b.z, c.b.w};
#pragma unroll
  for (int s = 4; s >= 1; s >>= 1)
    if (d & s) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = j + s < 8 ? w[j + s] : 0u;
    }
  if (d >= 8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 0u;
  }
  c.a = make_uint4(w[0], w[1], w[2], w[3]);
  c.b = make_uint4(w[4], w[5], w[6], w[7]);
}

// The same where the chunk lies inside the row.
__device__ __forceinline__ ChunkBf16 load8_in(const uint16_t* p) {
  ChunkBf16 c;
  memcpy(&c.v, p, 16);
  return c;
}
__device__ __forceinline__ ChunkF32 load8_in(const float* p) {
  ChunkF32 c;
  memcpy(&c.a, p, 16);
  memcpy(&c.b, p + 4, 16);
  return c;
}

// Both steps, rows of any length.
template <class T>
__device__ __forceinline__ typename ChunkOf<T>::type chunk8(const T* row, int k0, int K) {
  if (K < 8) return load8<true>(row, k0, K);
  typename ChunkOf<T>::type c = load8<false>(row, k0, K);
  settle8<false>(c, k0, K);
  return c;
}

// 8 values of a parameter vector [K] of either type (f32: is_f32), zeros at
// or past K.
__device__ __forceinline__ void param8(const void* p, bool is_f32, int k0, int K, float (&f)[8]) {
  if (is_f32) chunk8(static_cast<const float*>(p), k0, K).get(f);
  else chunk8(static_cast<const uint16_t*>(p), k0, K).get(f);
}

// 8 values, all inside the row.
__device__ __forceinline__ void store8_in(uint16_t* p, const float (&f)[8]) {
  const uint4 v = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                             pack_bf16x2(f[6], f[7]));
  memcpy(p, &v, 16);
}
__device__ __forceinline__ void store8_in(float* p, const float (&f)[8]) { memcpy(p, f, 32); }

// Values k0 .. k0 + 7 of a row, those below K: a broken chunk in pieces of 4,
// 2 and 1.
__device__ __forceinline__ void store8(uint16_t* row, int k0, int K, const float (&f)[8]) {
  const int n = K - k0;
  uint16_t* p = row + k0;
  if (n >= 8) {
    store8_in(p, f);
  } else if (n > 0) {
    uint2 a = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
    const uint2 b = make_uint2(pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    if (n & 4) {
      memcpy(p, &a, 8);
      p += 4;
      a = b;
    }
    if (n & 2) {
      memcpy(p, &a.x, 4);
      p += 2;
      a.x = a.y;
    }
    if (n & 1) *p = (uint16_t)a.x;
  }
}
__device__ __forceinline__ void store8(float* row, int k0, int K, const float (&f)[8]) {
  const int n = K - k0;
  float* p = row + k0;
  if (n >= 8) {
    store8_in(p, f);
  } else if (n > 0) {
    float4 a = make_float4(f[0], f[1], f[2], f[3]);
    if (n & 4) {
      memcpy(p, &a, 16);
      p += 4;
      a = make_float4(f[4], f[5], f[6], f[7]);
    }
    if (n & 2) {
      const float2 v = make_float2(a.x, a.y);
      memcpy(p, &v, 8);
      p += 2;
      a.x = a.z;
    }
    if (n & 1) *p = a.x;
  }
}

// ---------------------------------------------------------------------------
// 8-bit codes: 128 consecutive values of a row (16 lanes of 8) share the
// scale s = their largest magnitude, and each is kept as
// q = clip(round_half_even(127 x / s), -127, 127), exactly; it stands for
// q s / 127. A block of zeros has s = 0. A block that holds an infinity or a
// NaN stands for NaN throughout: the magnitudes are compared as bit patterns,
// so that s is then infinite or NaN, and 0 times infinity is NaN.
// ---------------------------------------------------------------------------

// Rotation within the 16 lanes of a DPP row.
template <int N>
__device__ __forceinline__ uint32_t row_ror(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xF, 0xF, true);
}

// The largest magnitude of a lane's 8 values as a bit pattern.
__device__ __forceinline__ uint32_t magnitude8(const ChunkF32& c) {
  const uint32_t w[8] = {c.a.x, c.a.y, c.a.z, c.a.w, c.b.x, c.b.y, c.b.z, c.b.w};
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t a = w[e] & 0x7FFFFFFFu;
    m = a > m ? a : m;
  }
  return m;
}
__device__ __forceinline__ uint32_t magnitude8(const ChunkBf16& c) {  // two values an instruction
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  const auto mag = [](uint32_t w) { return __builtin_bit_cast(u16x2, w & 0x7FFF7FFFu); };
  const u16x2 m = __builtin_elementwise_max(__builtin_elementwise_max(mag(c.v.x), mag(c.v.y)),
                                            __builtin_elementwise_max(mag(c.v.z), mag(c.v.w)));
  const uint32_t lo = m.x, hi = m.y;
  return (lo > hi ? lo : hi) << 16;
}

// The scale of a block, in each of its 16 lanes.
template <class C>
__device__ __forceinline__ float block_scale(const C& c) {
  uint32_t m = magnitude8(c);
  uint32_t o;
  o = row_ror<8>(m); m = o > m ? o : m;
  o = row_ror<4>(m); m = o > m ? o : m;
  o = row_ror<2>(m); m = o > m ? o : m;
  o = row_ror<1>(m); m = o > m ? o : m;
  return __uint_as_float(m);
}

// round_half_even(127 x / s) for |x| <= s as the fp32 value 1.5 * 2^23 + q,
// whose low byte is q. t = fl(x fl(127/s) + 1.5 * 2^23) holds the integer
// nearest to x fl(127/s), which is within 1.6e-5 of the quotient; where their
// distance is less than 1/2 - 2^-15 that integer is the quotient's too.
// Otherwise the quotient is taken in fp64, whose rounding error (below 2^-46)
// is far below the least distance (2^-33) of a quotient of fp32 values from a
// half integer that it is not.
constexpr float kCodeMagic = 12582912.0f;  // 1.5 * 2^23
constexpr float kCodeSure = 0.49996948f;   // 1/2 - 2^-15
__device__ __forceinline__ float code_exact(float x, float s) {
  return (float)__builtin_rint(127.0 * (double)x / (double)s) + kCodeMagic;
}

// The codes of 8 values of a block with scale s. Scales so small that 127 / s
// would not be a finite fp32 number, and zero, take the exact route. The
// largest of the 8 distances decides once for all (four operations a value:
// the code, its integer, the distance, its maximum).
__device__ __forceinline__ uint2 codes8(const float (&f)[8], float s) {
  const bool tiny = s < 1e-30f;
  const float r127 = tiny ? 0.0f : 127.0f / s;
  float t[8], far = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    t[e] = fmaf(f[e], r127, kCodeMagic);
    far = fmaxf(far, fabsf(fmaf(f[e], r127, -(t[e] - kCodeMagic))));
  }
  if (far > kCodeSure || (tiny && s > 0.0f)) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (tiny || fabsf(fmaf(f[e], r127, -(t[e] - kCodeMagic))) > kCodeSure) t[e] = code_exact(f[e], s);
  }
  const auto pack = [](float a, float b, float c, float d) {
    const uint32_t lo = perm(__float_as_uint(b), __float_as_uint(a), 0x0C0C0400u);
    const uint32_t hi = perm(__float_as_uint(d), __float_as_uint(c), 0x0C0C0400u);
    return perm(hi, lo, 0x05040100u);
  };
  return make_uint2(pack(t[0], t[1], t[2], t[3]), pack(t[4], t[5], t[6], t[7]));
}

// The values of 8 codes, r = s / 127.
__device__ __forceinline__ void values8(uint2 q, float r, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[e] = (float)((int)(q.x << (24 - 8 * e)) >> 24) * r;
    f[4 + e] = (float)((int)(q.y << (24 - 8 * e)) >> 24) * r;
  }
}

}  // namespace bitnet
