// Products for a middling number of tokens, out[j][i] = sum_k p[i][k] q[j][k]: too many
// for the few-token kernels, too few for the 256 x 256 tiles of gemm_core.h to fill the
// CUs. There a tile's time is its chain of stages, 1.2 to 1.6 us each whatever the other
// CUs do; here tiles are 128 x 64 or 128 x 128 and take 0.4 to 0.8 us a stage, two
// workgroups share a CU, and the loads of P stages are in flight from the first cycle on.
// What bounds a stage is its LDS traffic (24 to 32 KB stored and 48 to 64 KB read for 8 or 16
// instructions a wave) and the barrier: twice the stages in flight, or reading each step's
// fragments while the one before is multiplied, changed nothing.
//
// A stage is 128 bytes of every row (128 int8 or 64 bf16). Loaded into registers P stages
// ahead, it is stored to one of two LDS buffers, expanded there if it is codes, while the
// other is multiplied: one barrier a stage. Waves lie WI x WJ, each with FI x FJ blocks of
// 32 x 32. LDS rows are 144 bytes apart: 9 chunks of 16, so the 32 rows a wave reads at
// once start in different banks.
#pragma once

#include <algorithm>

#include "bwd_prep.h"
#include "gemm_split.h"

namespace bitnet {

// How a K-major operand's stage lies in LDS: rows of 128 bytes.
struct RowLds {
  template <int ROWS>
  static constexpr int kBytes = ROWS * kPitch;
  // a wave's fragments: rows row0 + 32 f + l % 32
  template <int ROWS>
  static __device__ __forceinline__ int first(int row0, int lane) {
    return (row0 + (lane & 31)) * kPitch + 16 * (lane >> 5);
  }
  template <class MT, int ROWS>
  static __device__ __forceinline__ typename MT::Frag frag(const char* p, int f, int ks) {
    return *reinterpret_cast<const typename MT::Frag*>(p + f * 32 * kPitch + 32 * ks);
  }
};

// Rows r0 + r.
struct TileRow {
  int r0;
  int64_t rows;
  __device__ __forceinline__ void set(int r) { r0 = r; }
  __device__ __forceinline__ int64_t operator()(int r) const { return r0 + r < rows ? r0 + r : -1; }
};

// 128 bytes of each of ROWS rows for T threads: 16-byte chunks as stored. ROW: the
// operand's row of tile row r, negative for none.
template <class ROW>
struct MidRows : RowLds {
  const void* p;
  int64_t rows, pitch;  // bytes
  ROW row;
  __device__ __forceinline__ void set(int r) { row.set(r); }
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
struct MidCodes : RowLds {
  const void* p;
  int64_t rows, pitch;
  ROW row;
  __device__ __forceinline__ void set(int r) { row.set(r); }
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

// Transposed fp4 codes (bwd_prep.h; 32 bytes a row and stage), expanded to bf16.
template <class ROW>
struct MidFp4 : RowLds {
  const void* p;
  int64_t rows, pitch;
  ROW row;
  __device__ __forceinline__ void set(int r) { row.set(r); }
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
        o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[c], 1.0f, 0));
        o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[c], 1.0f, 1));
        o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[c], 1.0f, 2));
        o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[c], 1.0f, 3));
        *reinterpret_cast<uint4*>(lds + at / 2 * kPitch + 64 * (at % 2) + 16 * c) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
};

// A bf16 operand [red][ld] whose columns are the tile's rows: a stage is 64 rows of it, as
// stored, and ds_read_b64_tr_b16 turns the fragments (TrFragsP's scheme; the 64 bytes
// between rows keep its reads free of bank conflicts).
struct MidCols {
  const uint16_t* p;
  int64_t red, ld, cols;  // cols, ld: multiples of 8
  int c0;
  __device__ __forceinline__ void set(int c) { c0 = c; }
  template <int ROWS>
  static constexpr int kColPitch = 2 * ROWS + 64;
  template <int ROWS>
  static constexpr int kBytes = kRed16 * kColPitch<ROWS>;
  template <int ROWS, int T>
  struct Stage {
    static constexpr int kLanes = ROWS / 8, kRows = T / kLanes, kN = kRed16 / kRows;
    uint4 v[kN];
  };
  template <int ROWS, int T>
  __device__ __forceinline__ void load(Stage<ROWS, T>& g, int s) const {
    typedef Stage<ROWS, T> S;
    const rsrc_t rs = make_rsrc(p, (uint32_t)(red * ld * 2));
    const int64_t c = c0 + 8 * (threadIdx.x % S::kLanes);
#pragma unroll
    for (int i = 0; i < S::kN; ++i) {
      const int64_t r = (int64_t)s * kRed16 + i * S::kRows + threadIdx.x / S::kLanes;
      g.v[i] = buf_load16(rs, r < red && c < cols ? (uint32_t)((r * ld + c) * 2) : kOob);
    }
  }
  template <int ROWS, int T>
  __device__ __forceinline__ void store(const Stage<ROWS, T>& g, char* lds) const {
    typedef Stage<ROWS, T> S;
#pragma unroll
    for (int i = 0; i < S::kN; ++i)
      *reinterpret_cast<uint4*>(lds + (i * S::kRows + threadIdx.x / S::kLanes) * kColPitch<ROWS> +
                                16 * (threadIdx.x % S::kLanes)) = g.v[i];
  }
  template <int ROWS>
  static __device__ __forceinline__ int first(int row0, int lane) {
    const int g = lane >> 4, e = (lane >> 2) & 3, q = lane & 3;
    return (8 * (g >> 1) + e) * kColPitch<ROWS> + 2 * (row0 + 16 * (g & 1) + 4 * q);
  }
  template <class MT, int ROWS>
  static __device__ __forceinline__ typename MT::Frag frag(const char* p, int f, int ks) {
    typedef TrFragsP<kColPitch<ROWS>> F;
    typedef short v8i16_t __attribute__((ext_vector_type(8)));
    const char* a = p + 16 * ks * kColPitch<ROWS> + 64 * f;
    const v8i16_t v = __builtin_shufflevector(F::tr(a), F::tr(a + 4 * kColPitch<ROWS>), 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(typename MT::Frag, v);
  }
};

// LDS staging of 32 output rows x COLS columns of EB bytes each (EpStage's scheme): a lane
// puts 4 values of row l % 32 at column 32fi + 8g + 4(l / 32), and every wave store is
// whole rows of COLS values.
template <int EB, int COLS = 64>
struct RowStage {
  static constexpr int kRow = COLS * EB, kPitch = kRow + 16;
  static constexpr int kBytes = 32 * kPitch;
  static constexpr int kLanes = kRow / 16, kRows = kWave / kLanes, kPer = 16 / EB;  // of a row, of a store, values a lane
  template <class V>
  static __device__ __forceinline__ void put(char* w, int lane, int fi, int g, V v) {
    static_assert(sizeof(V) == 4 * EB, "");
    *reinterpret_cast<V*>(w + (lane & 31) * kPitch + 4 * EB * (lane >> 5) + (32 * fi + 8 * g) * EB) = v;
  }
  // Rows j0 .. j0 + 31 (those below J), columns i0 .. i0 + COLS - 1 (those below I) of
  // out [J][ld]. i0, j0 are uniform in the wave; 32 * ld * EB < 2^31. EB 1: ld and I
  // multiples of 16.
  static __device__ __forceinline__ void drain(const char* w, void* out, int64_t ld, int64_t I, int64_t J, int i0,
                                               int j0, int lane) {
    i0 = __builtin_amdgcn_readfirstlane(i0);
    j0 = __builtin_amdgcn_readfirstlane(j0);
    int c = lane % kLanes, rl = lane / kLanes;
    asm volatile("" : "+v"(c), "+v"(rl));  // as EpStage::drain
    const char* src = w + rl * kPitch + 16 * c;
    constexpr int kStores = 32 / kRows;
    uint4 v[kStores];
#pragma unroll
    for (int k = 0; k < kStores; ++k) v[k] = *reinterpret_cast<const uint4*>(src + kRows * k * kPitch);
    const int rows_in = J - j0 < 32 ? (int)(J - j0) : 32;
    char* base = static_cast<char*>(out) + ((int64_t)j0 * ld + i0) * EB;
    if (EB == 1 || ((ld | I) % kPer) == 0) {
      const uint32_t row_b = (uint32_t)ld * EB;
      const rsrc_t rs = make_rsrc(base, 32u * row_b);
      const uint32_t lane_off = i0 + kPer * c < I ? rl * row_b + 16 * c : kOob;
#pragma unroll
      for (int k = 0; k < kStores; ++k)
        buf_store16_stream(rs, rl < rows_in - kRows * k ? lane_off : kOob, (uint32_t)(kRows * k) * row_b, v[k]);
    } else if constexpr (EB > 1) {
#pragma unroll
      for (int k = 0; k < kStores; ++k) {
        if (kRows * k + rl >= rows_in) continue;
        char* row = base + ((int64_t)(kRows * k + rl) * ld + kPer * c) * EB;
        const int64_t n = I - (i0 + kPer * c);  // values of this chunk inside the row
        if (n >= kPer) {
          memcpy(row, &v[k], 16);
        } else {
          const uint32_t wv[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
          for (int e = 0; e < kPer; ++e) {
            if (e >= n) continue;
            if constexpr (EB == 4) *reinterpret_cast<uint32_t*>(row + 4 * e) = wv[e];
            else *reinterpret_cast<uint16_t*>(row + 2 * e) = (uint16_t)(wv[e >> 1] >> (16 * (e & 1)));
          }
        }
      }
    }
  }
};
using HalfStage = RowStage<2>;

template <int FI, int FJ, int WI, int WJ>
struct MidShape {
  static constexpr int kI = 32 * FI * WI, kJ = 32 * FJ * WJ, kT = kWave * WI * WJ;
  template <class LP, class LQ>
  static constexpr int kLds = 2 * (LP::template kBytes<kI> + LQ::template kBytes<kJ>);
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
  constexpr int kQ = LP::template kBytes<S::kI>, kBuf = kQ + LQ::template kBytes<S::kJ>;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int pi = LP::template first<S::kI>(wave % WI * (32 * FI), lane);
  const int qj = kQ + LQ::template first<S::kJ>(wave / WI * (32 * FJ), lane);
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
        for (int f = 0; f < FI; ++f) a[f] = LP::template frag<MT, S::kI>(buf + pi, f, ks);
#pragma unroll
        for (int f = 0; f < FJ; ++f) b[f] = LQ::template frag<MT, S::kJ>(buf + qj, f, ks);
#pragma unroll
        for (int fi = 0; fi < FI; ++fi)
#pragma unroll
          for (int fj = 0; fj < FJ; ++fj) acc[fi][fj] = MT::mma(a[fi], b[fj], acc[fi][fj]);
      }
      __syncthreads();
    }
  }
}

// A bf16 product on such tiles: LP and LQ for the tile at 0 (their row0 or c0 is set here).
// EP: scale(j), the factor of row j of the output, and part(j): the output that 32 rows from
// j on belong to, its rows and width, j counted within it.
template <class LP_, class LQ_, class EP_, int FJ, int P>
struct MidProduct {
  typedef LP_ LP;
  typedef LQ_ LQ;
  typedef EP_ EP;
  typedef MidShape<2, FJ, 2, 2> S;
  typedef RowStage<EP::kEB> Out;
  static constexpr int kLds = S::template kLds<LP, LQ>;
  static_assert(4 * Out::kBytes <= kLds, "the epilogue's staging");
  LP lp;
  LQ lq;
  EP ep;
  int nstages, tiles_j, tiles;

  MidProduct(const LP& p, const LQ& q, const EP& e, int64_t I, int64_t J, int64_t red)
      : lp(p), lq(q), ep(e), nstages((int)((red + kRed16 - 1) / kRed16)), tiles_j((int)((J + S::kJ - 1) / S::kJ)),
        tiles((int)((I + S::kI - 1) / S::kI) * tiles_j) {}

  __device__ __forceinline__ void run(int v, char* lds) {
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int i0 = v / tiles_j * S::kI, j0 = v % tiles_j * S::kJ;
    lp.set(i0);
    lq.set(j0);
    const int jw = j0 + 32 * FJ * (wave / 2);
    float sc[FJ];
#pragma unroll
    for (int fj = 0; fj < FJ; ++fj) sc[fj] = ep.scale(jw + 32 * fj + (lane & 31));
    MfmaBf16::Acc acc[2][FJ] = {};
    mid_tile<MfmaBf16, 2, FJ, 2, 2, P>(lp, lq, nstages, lds, acc);
    char* w = lds + wave * Out::kBytes;
#pragma unroll
    for (int fj = 0; fj < FJ; ++fj) {
#pragma unroll
      for (int fi = 0; fi < 2; ++fi)
#pragma unroll
        for (int gi = 0; gi < 4; ++gi) {
          const float v0 = acc[fi][fj][4 * gi] * sc[fj], v1 = acc[fi][fj][4 * gi + 1] * sc[fj];
          const float v2 = acc[fi][fj][4 * gi + 2] * sc[fj], v3 = acc[fi][fj][4 * gi + 3] * sc[fj];
          if constexpr (EP::kEB == 4) Out::put(w, lane, fi, gi, make_float4(v0, v1, v2, v3));
          else Out::put(w, lane, fi, gi, make_uint2(pack_bf16x2(v0, v1), pack_bf16x2(v2, v3)));
        }
      int j = __builtin_amdgcn_readfirstlane(jw + 32 * fj);
      int64_t J;
      void* out = ep.part(j, J);
      if (j < J) Out::drain(w, out, ep.I, ep.I, J, i0 + 64 * (wave % 2), j, lane);
    }
  }
};

template <class A>
__global__ __launch_bounds__(256) void mid_kernel(A a) {
  __shared__ __attribute__((aligned(16))) char lds[A::kLds];
  a.run(xcd_major(blockIdx.x, a.tiles), lds);
}

// Two products in one launch, a's tiles (the longer ones) first.
template <class A, class B>
__global__ __launch_bounds__(256) void mid_pair_kernel(A a, B b) {
  __shared__ __attribute__((aligned(16))) char lds[A::kLds > B::kLds ? A::kLds : B::kLds];
  const int at = blockIdx.x;
  if (at < a.tiles) a.run(xcd_major(at, a.tiles), lds);
  else b.run(xcd_major(at - a.tiles, b.tiles), lds);
}

// out [J][I], rows times 127 / s (s NULL: 1).
template <int EB>
struct MidOut {
  static constexpr int kEB = EB;
  void* out;
  int64_t I, J;
  const float* s;
  __device__ __forceinline__ float scale(int64_t j) const { return s != nullptr && j < J ? per_scale(s[j]) : 1.0f; }
  __device__ __forceinline__ void* part(int&, int64_t& rows) const {
    rows = J;
    return out;
  }
};

// The products of a backward pass: dX [M][K] over `nx` columns of dY (LP1, LQ1) on 128 x 64
// tiles, dW [nw][K] over the M tokens on 128 x 64 or 128 x 128.
template <int FJ, int P, class LP1, class LQ1, class EP1, class LP2, class LQ2, class EP2>
static hipError_t mid_products_at(const LP1& lp1, const LQ1& lq1, const EP1& ep1, const LP2& lp2, const LQ2& lq2,
                                  const EP2& ep2, bool dx, bool dw, int64_t M, int64_t K, int64_t nx, int64_t nw,
                                  hipStream_t st) {
  typedef MidProduct<LP1, LQ1, EP1, 1, 4> X;
  typedef MidProduct<LP2, LQ2, EP2, FJ, P> W;
  const X x(lp1, lq1, ep1, K, M, nx);
  const W w(lp2, lq2, ep2, K, nw, M);
  if (dx && dw) mid_pair_kernel<X, W><<<(unsigned)(x.tiles + w.tiles), 256, 0, st>>>(x, w);
  else if (dx) mid_kernel<X><<<(unsigned)x.tiles, 256, 0, st>>>(x);
  else mid_kernel<W><<<(unsigned)w.tiles, 256, 0, st>>>(w);
  return hipGetLastError();
}

// As gemm_kernels.hip's rule for its own pair: both products split on the whole
// device under a 3-stage piece cost.
static bool pair_pays(GemmShape dx, GemmShape dw) {
  dx.overhead = dw.overhead = 3;
  return split_pays(dx, device_cus()) > 0 && split_pays(dw, device_cus()) > 0;
}

// What a launch of these tiles takes, in us: a tile of FJ 1 / 2 takes 0.52 / 0.82 us a stage
// with a CU for itself, 0.80 / 1.25 with another beside it. Fitted, like the times of the
// 256 x 256 tiles below, to 16 to 2048 tokens of layers of 640 to 6912 columns.
struct MidTime {
  double tile = 0, all = 0;  // the longest tile, and all of them on a device whose CUs are shared by two
  void add(int64_t I, int64_t J, int64_t stages, int fj) {
    const double tiles = (double)((I + 127) / 128 * ((J + 64 * fj - 1) / (64 * fj)));
    tile = std::max(tile, (fj == 1 ? 0.52 : 0.82) * stages);
    all += tiles * ((fj == 1 ? 0.80 : 1.25) * stages + 2.5) / (2 * device_cus());
  }
  double us() const { return std::max(tile + 4.5, 1.15 * (all + 5)); }
};

// The token blocks of dW's tiles where the products of a backward pass (those wanted) are
// faster here than on 256 x 256 tiles, 0 where they are not. g1, g2: their shapes there;
// both: they would share a launch there, split over its workgroups, whose pieces cost it
// 45 us (95 for one product). Measured, us, here / there, 8 bits 2560 -> 2560: 16 tokens 23.4 /
// 82, 512 26.4 / 72, 1024 47 / 61; 2560 -> 6912, 128: 55 / 109, 512 66 / 94; gated, 640 -> 2 x
// 1728, 512: 27.7 / 73.
static int mid_bwd_blocks(const GemmShape& g1, const GemmShape& g2, bool dx, bool dw, bool both, int64_t M, int64_t K,
                          int64_t nw) {
  if (test_knobs().no_skinny.load(std::memory_order_relaxed) != 0 ||
      test_knobs().split_ctas.load(std::memory_order_relaxed) != 0)
    return 0;  // tests that ask for the large tiles
  const auto split_us = [](const GemmShape& g, double base) {
    return base + 1.45 * (double)(g.tiles() * g.nstages) / device_cus();
  };
  const auto one_us = [&](const GemmShape& g) {
    const double whole = (double)((g.tiles() + device_cus() - 1) / device_cus()) * (1.65 * g.nstages + 8);
    return split_pays(g, device_cus()) ? std::min(whole, split_us(g, 95)) : whole;
  };
  const double there = dx && dw && both ? split_us(g1, 45) + split_us(g2, 0)
                                        : (dx ? one_us(g1) : 0) + (dw ? one_us(g2) : 0);
  double best = there;
  int blocks = 0;
  for (int fj = 2; fj >= 1; --fj) {
    MidTime t;
    if (dx) t.add(K, M, g1.nstages, 1);
    if (dw) t.add(K, nw, g2.nstages, fj);
    if (t.us() < best) {
      best = t.us();
      blocks = fj;
    }
  }
  return blocks;
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
