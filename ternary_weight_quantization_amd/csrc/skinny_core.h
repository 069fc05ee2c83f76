// The loop of the products for few tokens (skinny_kernels.hip describes it).
#pragma once

#include "device_common.h"
#include "internal.h"

namespace bitnet {

// Forward: A = 2-bit codes [N][Kp/4] (rows i = n), B = x_q [M][Kp].
struct SkFwd {
  typedef i32x16_t Acc;
  typedef int Elem;
  static constexpr int kCodeB = 32;  // code bytes per row per super-step
  static __device__ __forceinline__ Acc mma(uint32_t code_word, uint4 b, Acc acc) {
    i32x4_t a;
#pragma unroll
    for (int t = 0; t < 4; ++t) a[t] = (int)codes4_to_i8((code_word >> (2 * t)) & 0x03030303u);
    const i32x4_t bx = {(int)b.x, (int)b.y, (int)b.z, (int)b.w};
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, bx, acc, 0, 0, 0);
  }
};

// The code operand: `rows` rows of `pitch` bytes, the first `bytes` of
// each in use; the token operand: M rows of `tpitch` bytes, the first
// `tbytes` of each valid (both multiples of 16). tlo, thi: SkTtq's value
// table (unused by the other policies).
struct SkArgs {
  const uint8_t* codes;
  int64_t rows, pitch, bytes;
  const void* tok;
  int64_t tpitch, tbytes;
  int M;
  uint32_t tlo, thi;
};

template <int MT>  // token tiles of 32: 1 for M <= 32, 2 for M <= 64
struct SkChunk {
  uint4 x[4 * MT];  // this thread's 16-byte pieces of the chunk's token columns (32 MT rows x 128 W bytes)
  uint4 codes;      // this lane's code bytes for its wave's super-step
};

// The partial tiles of the W waves of a workgroup, in LDS (skinny_sum). crow:
// the code row of this lane (r32 = lane % 32), negative for none (zeros).
template <class SK, int MT, int W, int P>
__device__ __forceinline__ void skinny_partials(const SkArgs& a, int64_t crow, char* smem) {
  typedef typename SK::Elem E;
  constexpr int kThreads = kWave * W;
  constexpr int kChunkB = 128 * W;           // token-operand bytes per row per chunk
  constexpr int kPitch = kChunkB + 16;       // LDS bytes per token row
  constexpr int kRowPieces = kChunkB / 16;   // 16-byte pieces per token row of a chunk
  static_assert(32 * MT * kRowPieces / kThreads == 4 * MT, "32 MT rows x 128 W bytes over 64 W threads");
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int h = lane >> 5, r32 = lane & 31;
  constexpr int kCB = SK::kCodeB;
  const int nchunks = (int)((a.bytes + kCB * W - 1) / (kCB * W));

  const rsrc_t rc = make_rsrc(a.codes, (uint32_t)(a.rows * a.pitch));
  const uint32_t coff = crow >= 0 ? (uint32_t)(crow * a.pitch) : kOob;
  const rsrc_t rx = make_rsrc(a.tok, (uint32_t)(a.M * a.tpitch));
  // piece p of a chunk: token row (p * kThreads + tid) / kRowPieces, 16-byte
  // column (p * kThreads + tid) % kRowPieces of the chunk
  const auto load = [&](SkChunk<MT>& b, int c) {
#pragma unroll
    for (int p = 0; p < 4 * MT; ++p) {
      const int e = p * kThreads + tid, row = e / kRowPieces, col = 16 * (e % kRowPieces);
      const int64_t x = (int64_t)c * kChunkB + col;
      b.x[p] = buf_load16(rx, row < a.M && x < a.tbytes ? (uint32_t)(row * a.tpitch + x) : kOob);
    }
    const int64_t cb = (int64_t)c * (kCB * W) + kCB * wave + (kCB / 2) * h;
    const uint32_t off = cb < a.bytes ? coff + (uint32_t)cb : kOob;
    if constexpr (kCB == 32) {
      b.codes = buf_load16(rc, off);
    } else {
      const uint2 c8 = buf_load8(rc, off);
      b.codes = make_uint4(c8.x, c8.y, 0u, 0u);
    }
  };
  const auto stage = [&](const SkChunk<MT>& b) {
#pragma unroll
    for (int p = 0; p < 4 * MT; ++p) {
      const int e = p * kThreads + tid;
      *reinterpret_cast<uint4*>(smem + (e / kRowPieces) * kPitch + 16 * (e % kRowPieces)) = b.x[p];
    }
  };

  typename SK::Acc acc[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[mt][e] = 0;
  const auto compute = [&](const SkChunk<MT>& b) {
    const uint32_t w4[4] = {b.codes.x, b.codes.y, b.codes.z, b.codes.w};
    const char* xr = smem + r32 * kPitch + 128 * wave + 64 * h;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const uint4 tok = *reinterpret_cast<const uint4*>(xr + 32 * mt * kPitch + 16 * j);
        if constexpr (kCB == 32)
          acc[mt] = SK::mma(w4[j], tok, acc[mt]);
        else
          acc[mt] = SK::mma(w4[j >> 1] >> (4 * (j & 1)), tok, acc[mt], a.tlo, a.thi);
      }
  };

  SkChunk<MT> buf[P];
#pragma unroll
  for (int d = 0; d < P; ++d) load(buf[d], d);
  for (int i = 0; i < nchunks; i += P) {
#pragma unroll
    for (int d = 0; d < P; ++d) {
      if (i + d < nchunks) {
        __syncthreads();  // the previous chunk's fragment reads are done
        stage(buf[d]);
        __syncthreads();
        compute(buf[d]);
        load(buf[d], i + d + P);  // past the last chunk: zeros, never staged
      }
    }
  }

  __syncthreads();
  E* red = reinterpret_cast<E*>(smem);  // [wave][mt][16][lane]
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int e = 0; e < 16; ++e) red[((wave * MT + mt) * 16 + e) * kWave + lane] = acc[mt][e];
  __syncthreads();
}

// Those, summed in wave order for the 4 values of rows 8g + 4h + 0..3 and token
// 32mt + l % 32 of the workgroup's tile (h = l / 32).
template <class SK, int MT, int W>
__device__ __forceinline__ void skinny_sum(const char* smem, int g, int mt, typename SK::Elem (&out)[4]) {
  typedef typename SK::Elem E;
  const E* red = reinterpret_cast<const E*>(smem);
  const int lane = threadIdx.x % kWave;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    E sum = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) sum += red[((w * MT + mt) * 16 + 4 * g + e) * kWave + lane];
    out[e] = sum;
  }
}

// Both for code rows 32 * blockIdx.x + 0..31: the lane's values in out, g =
// wave % 4, mt = wave / 4 (nothing when mt >= MT).
template <class SK, int MT, int W, int P>
__device__ __forceinline__ void skinny_body(const SkArgs& a, char* smem, typename SK::Elem (&out)[4], int& mt_out,
                                            int& g_out) {
  const int64_t i = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
  skinny_partials<SK, MT, W, P>(a, i < a.rows ? i : -1, smem);
  const int wave = threadIdx.x / kWave;
  g_out = wave % 4;
  mt_out = wave / 4;
  if (mt_out < MT) skinny_sum<SK, MT, W>(smem, g_out, mt_out, out);
}

// LDS bytes: the token tile of a chunk, reused for the partial tiles.
template <int MT, int W>
constexpr int skinny_lds() {
  return 32 * MT * (128 * W + 16) > W * MT * 16 * kWave * 4 ? 32 * MT * (128 * W + 16) : W * MT * 16 * kWave * 4;
}

}  // namespace bitnet
