// Products of 8-bit rows for few tokens, groups of up to kFewM: acc[m][n] = sum_k
// x_q[m][k] * w[n][k] in int32 for weights in 8 bits or as 2-bit codes. At these sizes
// the cost is reading the weights once, so that as many bytes as possible have to be
// in flight from the first cycle on.
//
// A workgroup of W waves takes RT tiles of 16 weight rows and the tokens of a group. The
// waves share the reduction: wave w takes steps w, w + W, ... of 256 (codes) or 128
// (int8) k, so that a step is 64 or 128 consecutive bytes of each row, and requests P
// steps ahead. v_mfma_i32_16x16x64_i8 takes 16 bytes of weight row l % 16 and of
// token l % 16 from lane l: those of k = 64j + 16q .. + 15 of the step in instruction
// j (q = l / 16). Of codes a lane loads the 16 bytes of k = 64q .. 64q + 63, and the four
// lanes of a row exchange their words (transpose4).
//
// Loaded as the instruction takes them, consecutive lanes lie in different rows, and
// the address unit takes those one at a time: 16 bytes a clock and CU. Where that is
// too slow the wave loads 8 (int8) or 16 lanes a row instead, 64 bytes a clock, and
// turns the block in its own part of LDS, with no barrier: TW the weights, TX x_q.
// Measured, us, with neither / TX / TW / both, int8: 1 token 2560 -> 32000 20.3 / 19.7 /
// 15.6 / 16.2 (82 MB at the rate of a copy: 15.8), 16 tokens 26.0 / 20.4 / 20.2 / 15.5,
// 1 token 6912 -> 2560 7.4 / 7.4 / 5.8 / 6.4, 64 tokens 19.7 / 12.6 / 17.4 / 12.3; codes, 16
// tokens 2560 -> 2 x 6912 7.8 / 6.4.
//
// The weights are read once; x_q is read by every workgroup, from the caches. The
// waves' partial tiles, 1 KiB for 16 rows x 16 tokens, meet in LDS. Rows, tokens and k
// past the operands read as zeros through the buffer range checks.
#pragma once

#include "device_common.h"
#include "bwd_prep.h"
#include "gemm_core.h"
#include "rows_quant.h"

namespace bitnet {

typedef int i32x4acc_t __attribute__((ext_vector_type(4)));

struct FewArgs {
  const uint8_t* w;  // rows of `pitch` bytes
  int64_t rows, pitch;
  const int8_t* xq;  // [M][Kp]
  int64_t Kp;
  int M;
  const uint16_t* x;  // [M][K] (FewRows)
  int K;
};

// More than kFewM tokens are groups of kFewM. A workgroup's tile of weight rows and
// first token; a becomes the group's. The groups of a tile are neighbours on one XCD, so
// that the weights come to it once.
constexpr int kFewM = 64;
__device__ __forceinline__ void few_place(FewArgs& a, int& tile, int& m0) {
  const int groups = (a.M + kFewM - 1) / kFewM;
  const int v = groups > 1 ? xcd_major(blockIdx.x, gridDim.x) : (int)blockIdx.x;
  tile = v / groups;
  m0 = v % groups * kFewM;
  a.xq += (int64_t)m0 * a.Kp;
  a.M = a.M - m0 < kFewM ? a.M - m0 : kFewM;
}

template <bool CODES>
struct FewStep {
  static constexpr int kJ = CODES ? 4 : 2;       // instructions of a step
  static constexpr int kLoads = CODES ? 1 : kJ;  // 16-byte weight loads a tile
  static constexpr int kK = 64 * kJ;             // k of a step
};

// Word j of lane quarter q becomes word q of quarter j.
__device__ __forceinline__ void transpose4(uint4& v) {
  // halves of the wave, then quarters within each half
  auto a = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
  auto b = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
  auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  v = make_uint4(c[0], c[1], d[0], d[1]);
}

// Bytes of LDS: the waves' turned blocks, then their partial tiles.
template <bool CODES, int RT, int MT, int W, bool TX, bool TW>
constexpr int few_lds() {
  constexpr int x = W * 16 * ((TX ? MT : 0) + (TW ? RT : 0)) * (FewStep<CODES>::kK + 16), red = W * RT * MT * kWave * 16;
  return x > red ? x : red;
}

// The codes of up to NX tokens of at most kMaxK values, which every workgroup makes
// of the bf16 rows for itself while its first weights are on the way: no launch before
// this one, and no codes in memory. The work is a row's reduction and codes for each
// token in every workgroup, so it pays at 1 and 2 tokens and less with each more.
// Measured, us a call among others, 1 / 2 / 3 / 4 tokens, and 5 with the rows' launch and
// the product: codes, 2560 -> 2 x 6912 6.0 / 7.0 / 8.1 / 8.4, 9.0; 6912 -> 2 x 2560 7.0 / 7.9 /
// 9.8 / 10.1, 9.9; int8, 6912 -> 2560 6.7 / 7.8 / 9.1 / 10.3, 9.9; 2560 -> 32000 (2000
// workgroups) 15.0 / 17.0 / 20.6 / 22.0, 18.5: there 3 and 4 tokens lose.
template <int NX, int W>
struct FewRows {
  static constexpr int kThreads = kWave * W, kChunks = 2, kMaxK = 8 * kChunks * kThreads;
  __attribute__((aligned(16))) int8_t codes[NX][kMaxK];
  float s[NX], slot[NX][W];
};
template <int W>
struct FewRows<0, W> {};

template <int NX, int W>
struct FewChunks {
  ChunkBf16 c[NX][FewRows<NX, W>::kChunks];
};
template <int W>
struct FewChunks<0, W> {};

// 8 <= K <= kMaxK
template <int NX, int W>
__device__ __forceinline__ void few_rows_load(const FewArgs& a, FewChunks<NX, W>& v) {
  typedef FewRows<NX, W> R;
#pragma unroll
  for (int m = 0; m < NX; ++m)
#pragma unroll
    for (int i = 0; i < R::kChunks; ++i)
      v.c[m][i] = load8<false>(a.x + (int64_t)(m < a.M ? m : 0) * a.K, 8 * ((int)threadIdx.x + i * R::kThreads), a.K);
}

// Ends with a barrier.
template <int NX, int W>
__device__ __forceinline__ void few_rows_quantize(const FewArgs& a, FewChunks<NX, W>& v, FewRows<NX, W>& r) {
  typedef FewRows<NX, W> R;
  const int t = threadIdx.x, lane = t % kWave, wave = t / kWave, nq = (int)(a.Kp / 8);
#pragma unroll
  for (int m = 0; m < NX; ++m) {
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < R::kChunks; ++i) {
      settle8<false>(v.c[m][i], 8 * (t + i * R::kThreads), a.K);
      const uint32_t o = magnitude8(v.c[m][i]);
      mx = o > mx ? o : mx;
    }
    mx = row_max_bits<kWave>(mx, nullptr);
    if (lane == 0) r.slot[m][wave] = __uint_as_float(mx);
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < NX; ++m) {
    if (m >= a.M) break;
    uint32_t mx = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const uint32_t o = __float_as_uint(r.slot[m][w]);
      mx = o > mx ? o : mx;
    }
    const float s = row_scale(mx);
    if (t == 0) r.s[m] = s;
#pragma unroll
    for (int i = 0; i < R::kChunks; ++i) {
      const int ch = t + i * R::kThreads;
      if (ch >= nq) continue;
      float f[8];
      v.c[m][i].get(f);
      *reinterpret_cast<uint2*>(&r.codes[m][8 * ch]) = codes8(f, s);
    }
  }
  __syncthreads();
}

// The waves' partial tiles in smem (few_lds bytes), after a barrier. row[t]: this
// lane's weight row of tile t (of lane % 16), negative for none; TW: row[0] the first of
// 16 RT consecutive rows. NX (MT 1, not TX): the tokens are a.x's, not a.xq's.
template <bool CODES, int RT, int MT, int W, int P, bool TX, bool TW, int NX>
__device__ __forceinline__ void few_tokens_product(const FewArgs& a, const int64_t (&row)[RT], char* smem,
                                                   FewRows<NX, W>& rows) {
  static_assert(NX == 0 || (MT == 1 && !TX), "codes made here are read where they lie");
  typedef FewStep<CODES> S;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, q = lane >> 4, r16 = lane & 15;
  const rsrc_t rw = make_rsrc(a.w, (uint32_t)(a.rows * a.pitch)), rx = make_rsrc(a.xq, NX > 0 ? 0u : (uint32_t)(a.M * a.Kp));
  constexpr int kLanes = S::kK / 16, kRows = kWave / kLanes;  // of a row, of a load (kTurn)
  constexpr int kPitch = S::kK + 16;
  char* xl = smem + wave * (16 * ((TX ? MT : 0) + (TW ? RT : 0)) * kPitch);
  char* wl = xl + (TX ? 16 * MT * kPitch : 0);
  const int xr = lane / kLanes, xc = 16 * (lane % kLanes);
  uint32_t woff[RT], xoff[MT];
#pragma unroll
  for (int t = 0; t < RT; ++t) woff[t] = row[t] >= 0 ? (uint32_t)(row[t] * a.pitch) : kOob;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) xoff[mt] = 16 * mt + r16 < a.M ? (uint32_t)((16 * mt + r16) * a.Kp) : kOob;

  struct Step {
    uint4 w[RT][S::kLoads], x[MT][S::kJ];
  };
  const auto load = [&](Step& b, int64_t s) {
    const int64_t k0 = s * S::kK;  // Kp is a multiple of 64: an instruction's k are all inside or all outside
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int j = 0; j < S::kLoads; ++j) {
        if constexpr (TW) {  // rows row0 .. row0 + 16 RT - 1
          const int64_t r = row[0] + 16 * t + j * kRows + xr;
          b.w[t][j] = buf_load16(rw, r < a.rows && k0 + xc < a.Kp ? (uint32_t)(r * a.pitch + k0 + xc) : kOob);
          continue;
        }
        const int64_t k = k0 + 64 * (CODES ? q : j);
        b.w[t][j] = buf_load16(rw, k < a.Kp ? woff[t] + (uint32_t)(CODES ? k / 4 : k + 16 * q) : kOob);
      }
    if constexpr (NX > 0) {
    } else if constexpr (TX) {
#pragma unroll
      for (int i = 0; i < MT * S::kJ; ++i) {
        const int r = i * kRows + xr;
        b.x[i / S::kJ][i % S::kJ] = buf_load16(rx, r < a.M && k0 + xc < a.Kp ? (uint32_t)(r * a.Kp + k0 + xc) : kOob);
      }
    } else {
#pragma unroll
      for (int j = 0; j < S::kJ; ++j) {
        const int64_t k = k0 + 64 * j;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) b.x[mt][j] = buf_load16(rx, k < a.Kp ? xoff[mt] + (uint32_t)(k + 16 * q) : kOob);
      }
    }
  };
  i32x4acc_t acc[RT][MT];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[t][mt] = i32x4acc_t{0, 0, 0, 0};
  const auto compute = [&](Step& b, int64_t s) {
    if constexpr (NX > 0) {
#pragma unroll
      for (int j = 0; j < S::kJ; ++j) {
        const int64_t k = s * S::kK + 64 * j;
        b.x[0][j] = make_uint4(0u, 0u, 0u, 0u);
        if (r16 < a.M && k < a.Kp) b.x[0][j] = *reinterpret_cast<const uint4*>(&rows.codes[r16][k + 16 * q]);
      }
    }
    if constexpr (CODES) {
#pragma unroll
      for (int t = 0; t < RT; ++t) transpose4(b.w[t][0]);
    }
    if constexpr (TW) {
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int j = 0; j < S::kJ; ++j)
          *reinterpret_cast<uint4*>(wl + (16 * t + j * kRows + xr) * kPitch + xc) = b.w[t][j];
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int j = 0; j < S::kJ; ++j)
          b.w[t][j] = *reinterpret_cast<const uint4*>(wl + (16 * t + r16) * kPitch + 64 * j + 16 * q);
    }
    if constexpr (TX) {
#pragma unroll
      for (int i = 0; i < MT * S::kJ; ++i)
        *reinterpret_cast<uint4*>(xl + (i * kRows + xr) * kPitch + xc) = b.x[i / S::kJ][i % S::kJ];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < S::kJ; ++j)
          b.x[mt][j] = *reinterpret_cast<const uint4*>(xl + (16 * mt + r16) * kPitch + 64 * j + 16 * q);
    }
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int j = 0; j < S::kJ; ++j) {
        i32x4_t wv;
        if constexpr (CODES) {
          const uint32_t c = j == 0 ? b.w[t][0].x : j == 1 ? b.w[t][0].y : j == 2 ? b.w[t][0].z : b.w[t][0].w;
#pragma unroll
          for (int e = 0; e < 4; ++e) wv[e] = (int)codes4_to_i8((c >> (2 * e)) & 0x03030303u);
        } else {
          wv = __builtin_bit_cast(i32x4_t, b.w[t][j]);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          acc[t][mt] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv, __builtin_bit_cast(i32x4_t, b.x[mt][j]), acc[t][mt], 0, 0, 0);
      }
  };

  const int64_t steps = (a.Kp + S::kK - 1) / S::kK;
  Step buf[P];
  FewChunks<NX, W> chunks;
  if constexpr (NX > 0) few_rows_load<NX, W>(a, chunks);
#pragma unroll
  for (int d = 0; d < P; ++d) load(buf[d], wave + d * W);
  if constexpr (NX > 0) few_rows_quantize<NX, W>(a, chunks, rows);
  for (int64_t s = wave; s < steps; s += P * W) {
#pragma unroll
    for (int d = 0; d < P; ++d) {
      compute(buf[d], s + d * W);  // past the last step: zeros
      load(buf[d], s + (P + d) * W);
    }
  }

  int* red = reinterpret_cast<int*>(smem);  // [wave][tile][token tile][lane][4]
  if constexpr (TX || TW) __syncthreads();  // the last reads of turned blocks are done
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
      *reinterpret_cast<i32x4acc_t*>(red + (((wave * RT + t) * MT + mt) * kWave + lane) * 4) = acc[t][mt];
  __syncthreads();
}

// Their sums: out[e] for row 4 (lane / 16) + e of tile t and token 16 mt + lane % 16.
template <int RT, int MT, int W>
__device__ __forceinline__ void few_tokens_sum(const char* smem, int t, int mt, int (&out)[4]) {
  const int lane = threadIdx.x % kWave;
  const int* red = reinterpret_cast<const int*>(smem);
  i32x4acc_t sum = i32x4acc_t{0, 0, 0, 0};
#pragma unroll
  for (int v = 0; v < W; ++v)
    sum += *reinterpret_cast<const i32x4acc_t*>(red + (((v * RT + t) * MT + mt) * kWave + lane) * 4);
#pragma unroll
  for (int e = 0; e < 4; ++e) out[e] = sum[e];
}

// 4 consecutive values n .. n + 3 of a row of N, those below N.
__device__ __forceinline__ void store4(uint16_t* row, int64_t n, int64_t N, const float (&f)[4]) {
  if (N % 4 == 0 && n + 4 <= N) {
    *reinterpret_cast<uint2*>(row + n) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < N) row[n + e] = f32_to_bf16_bits(f[e]);
  }
}

}  // namespace bitnet
