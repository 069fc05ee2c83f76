// Products for a middling number of tokens, out[j][i] = sum_k p[i][k] q[j][k]: too many
// for the few-token kernels, too few for the 256 x 256 tiles of gemm_core.h to fill the
// CUs. There a workgroup has a CU for itself and a tile's time is its chain of stages,
// 1.3 us each; here tiles are 128 x 64 or 128 x 128, two workgroups share a CU, and the
// loads of P stages are in flight from the first cycle on.
//
// A stage is 128 bytes of every row (128 int8 or 64 bf16). Loaded into registers P stages
// ahead, it is stored to one of two LDS buffers, expanded there if it is codes, while the
// other is multiplied: one barrier a stage. Waves lie WI x WJ, each with FI x FJ blocks of
// 32 x 32. LDS rows are 144 bytes apart: 9 chunks of 16, so the 32 rows a wave reads at
// once start in different banks.
#pragma once

#include "bwd_prep.h"
#include "gemm_split.h"

namespace bitnet {

// Rows r0 + r.
struct TileRow {
  int r0;
  int64_t rows;
  __device__ __forceinline__ int64_t operator()(int r) const { return r0 + r < rows ? r0 + r : -1; }
};

// 128 bytes of each of ROWS rows for T threads: 16-byte chunks as stored. ROW: the
// operand's row of tile row r, negative for none.
template <class ROW>
struct MidRows {
  const void* p;
  int64_t rows, pitch;  // bytes
  ROW row;
  template <int ROWS, int T>
  struct Stage {
    static constexpr int kN = ROWS * 8 / T;
    uint4 v[kN];
  };
  template <int ROWS, int T>
  __device__ __forceinline__ void load(Stage<ROWS, T>& g, int s) const {
    const rsrc_t rs = make_rsrc(p, (uint32_t)(rows * pitch));
#pragma unroll
    for (int i = 0; i < Stage<ROWS, T>::kN; ++i) {
      const int at = i * T + threadIdx.x;
      const int64_t r = row(at / 8);
      const uint32_t k = (uint32_t)s * kStageBytes + 16 * (at % 8);
      g.v[i] = buf_load16(rs, r >= 0 && k < pitch ? (uint32_t)(r * pitch) + k : kOob);
    }
  }
  template <int ROWS, int T>
  __device__ __forceinline__ void store(const Stage<ROWS, T>& g, char* lds) const {
#pragma unroll
    for (int i = 0; i < Stage<ROWS, T>::kN; ++i) {
      const int at = i * T + threadIdx.x;
      *reinterpret_cast<uint4*>(lds + at / 8 * kPitch + 16 * (at % 8)) = g.v[i];
    }
  }
};

// The same of 2-bit codes (32 bytes a row and stage), expanded to int8 on the way to LDS.
template <class ROW>
struct MidCodes {
  const void* p;
  int64_t rows, pitch;
  ROW row;
  template <int ROWS, int T>
  struct Stage {
    static constexpr int kN = ROWS * 2 / T;
    uint4 v[kN];
  };
  template <int ROWS, int T>
  __device__ __forceinline__ void load(Stage<ROWS, T>& g, int s) const {
    const rsrc_t rs = make_rsrc(p, (uint32_t)(rows * pitch));
#pragma unroll
    for (int i = 0; i < Stage<ROWS, T>::kN; ++i) {
      const int at = i * T + threadIdx.x;
      const int64_t r = row(at / 2);
      const uint32_t k = (uint32_t)s * (kStageBytes / 4) + 16 * (at % 2);
      g.v[i] = buf_load16(rs, r >= 0 && k < pitch ? (uint32_t)(r * pitch) + k : kOob);
    }
  }
  template <int ROWS, int T>
  __device__ __forceinline__ void store(const Stage<ROWS, T>& g, char* lds) const {
#pragma unroll
    for (int i = 0; i < Stage<ROWS, T>::kN; ++i) {
      const int at = i * T + threadIdx.x;
      const uint32_t w[4] = {g.v[i].x, g.v[i].y, g.v[i].z, g.v[i].w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = codes4_to_i8((w[c] >> (2 * e)) & 0x03030303u);
        *reinterpret_cast<uint4*>(lds + at / 2 * kPitch + 64 * (at % 2) + 16 * c) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
};

// LDS staging of 32 output rows x 64 columns of bf16 (EpStage's scheme): a lane
// puts 4 values of row l % 32 at column 32fi + 8g + 4(l / 32), and every wave
// store is 8 rows of 128 bytes.
struct HalfStage {
  static constexpr int kPitch = 128 + 16;
  static constexpr int kBytes = 32 * kPitch;
  static __device__ __forceinline__ void put(char* w, int lane, int fi, int g, uint2 v) {
    *reinterpret_cast<uint2*>(w + (lane & 31) * kPitch + 8 * (lane >> 5) + (32 * fi + 8 * g) * 2) = v;
  }
  // Rows j0 .. j0 + 31 (those below J), columns i0 .. i0 + 63 (those below I) of
  // out [J][ld]. i0, j0 are uniform in the wave; 32 * ld * 2 < 2^31.
  static __device__ __forceinline__ void drain(const char* w, uint16_t* out, int64_t ld, int64_t I, int64_t J, int i0,
                                               int j0, int lane) {
    i0 = __builtin_amdgcn_readfirstlane(i0);
    j0 = __builtin_amdgcn_readfirstlane(j0);
    int c = lane & 7, rl = lane >> 3;
    asm volatile("" : "+v"(c), "+v"(rl));  // as EpStage::drain
    const char* src = w + rl * kPitch + 16 * c;
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = *reinterpret_cast<const uint4*>(src + 8 * k * kPitch);
    const int rows_in = J - j0 < 32 ? (int)(J - j0) : 32;
    if (((ld | I) & 7) == 0) {
      const uint32_t row_b = (uint32_t)ld * 2;
      const rsrc_t rs = make_rsrc(out + (int64_t)j0 * ld + i0, 32u * row_b);
      const uint32_t lane_off = i0 + 8 * c < I ? rl * row_b + 16 * c : kOob;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        buf_store16_stream(rs, rl < rows_in - 8 * k ? lane_off : kOob, (uint32_t)(8 * k) * row_b, v[k]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (8 * k + rl >= rows_in) continue;
        uint16_t* row = out + (int64_t)(j0 + 8 * k + rl) * ld + i0 + 8 * c;
        const int64_t n = I - (i0 + 8 * c);  // values of this chunk inside the row
        if (n >= 8) {
          memcpy(row, &v[k], 16);
        } else {
          const uint32_t wv[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e < n) row[e] = (uint16_t)(wv[e >> 1] >> (16 * (e & 1)));
        }
      }
    }
  }
};

template <int FI, int FJ, int WI, int WJ>
struct MidShape {
  static constexpr int kI = 32 * FI * WI, kJ = 32 * FJ * WJ, kT = kWave * WI * WJ;
  static constexpr int kLds = 2 * (kI + kJ) * kPitch;
};

// acc[fi][fj] of this wave: rows 32 (FI (wave % WI) + fi) of the tile, columns
// 32 (FJ (wave / WI) + fj). lds: kLds bytes.
template <class MT, int FI, int FJ, int WI, int WJ, int P, class LP, class LQ>
__device__ __forceinline__ void mid_tile(const LP& lp, const LQ& lq, int nstages, char* lds,
                                         typename MT::Acc (&acc)[FI][FJ]) {
  typedef MidShape<FI, FJ, WI, WJ> S;
  static_assert(P % 2 == 0, "a stage's LDS buffer is known when compiled");
  struct Ring {
    typename LP::template Stage<S::kI, S::kT> p;
    typename LQ::template Stage<S::kJ, S::kT> q;
  } ring[P];
  constexpr int kBuf = (S::kI + S::kJ) * kPitch, kQ = S::kI * kPitch;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int frag = (lane & 31) * kPitch + 16 * (lane >> 5);
  const int pi = wave % WI * (32 * FI) * kPitch + frag, qj = kQ + wave / WI * (32 * FJ) * kPitch + frag;
  const auto load = [&](Ring& r, int s) {
    lp.template load<S::kI, S::kT>(r.p, s);
    lq.template load<S::kJ, S::kT>(r.q, s);
  };
  const auto store = [&](const Ring& r, char* buf) {
    lp.template store<S::kI, S::kT>(r.p, buf);
    lq.template store<S::kJ, S::kT>(r.q, buf + kQ);
  };
#pragma unroll
  for (int d = 0; d < P; ++d) load(ring[d], d);
  store(ring[0], lds);
  load(ring[0], P);
  __syncthreads();
  for (int s0 = 0; s0 < nstages; s0 += P) {
#pragma unroll
    for (int d = 0; d < P; ++d) {
      const int s = s0 + d;
      if (s >= nstages) break;  // the same in every thread
      Ring& next = ring[(d + 1) % P];
      store(next, lds + ((d + 1) & 1) * kBuf);  // past the last stage: zeros, not read
      load(next, s + 1 + P);
      const char* buf = lds + (d & 1) * kBuf;
#pragma unroll
      for (int ks = 0; ks < kKSteps; ++ks) {
        typename MT::Frag a[FI], b[FJ];
#pragma unroll
        for (int f = 0; f < FI; ++f)
          a[f] = *reinterpret_cast<const typename MT::Frag*>(buf + pi + f * 32 * kPitch + 32 * ks);
#pragma unroll
        for (int f = 0; f < FJ; ++f)
          b[f] = *reinterpret_cast<const typename MT::Frag*>(buf + qj + f * 32 * kPitch + 32 * ks);
#pragma unroll
        for (int fi = 0; fi < FI; ++fi)
#pragma unroll
          for (int fj = 0; fj < FJ; ++fj) acc[fi][fj] = MT::mma(a[fi], b[fj], acc[fi][fj]);
      }
      __syncthreads();
    }
  }
}

// The token blocks (FJ, with 2 x 2 waves) for M tokens and `tiles_i` tiles of 128 rows, 0:
// the 256 x 256 tiles. Up to two workgroups a CU the smaller tile, then the larger, then
// neither fits at once. Measured, us, 128 x 64 / 128 x 128 / 256 x 256: 8 bits, 2560 -> 2560, 512
// tokens 13.0 / 18.3 / 30.0, 1024 19.2 / 19.9 / 31.5, 2048 29.9 / 28.2 / 33.6; 2560 -> 6912, 512
// 20.1 / 19.4 / 30.9, 1024 36.5 / 29.2 / 33.9, 2048 66 / 56 / 39.5; gated, 2560 -> 2 x 6912, 128
// 14.3 / 19.1 / 30.4, 512 33.9 / 27.8 / 32.6, 1024 57.8 / 51.1 / 36.9.
static int mid_blocks(int64_t M, int64_t tiles_i) {
  if (test_knobs().no_skinny.load(std::memory_order_relaxed) != 0 ||
      test_knobs().split_ctas.load(std::memory_order_relaxed) != 0)
    return 0;  // tests that ask for the large tiles
  const int64_t at_once = 2 * (int64_t)device_cus();
  for (int fj = 1; fj <= 2; ++fj)
    if ((M + 64 * fj - 1) / (64 * fj) * tiles_i <= at_once) return fj;
  return 0;
}

}  // namespace bitnet
