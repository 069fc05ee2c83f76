// Building blocks of the MFMA GEMMs for gfx950: tile constants, MFMA flavours,
// fragment readers, operand loaders, the staged main loop of one output tile
// and the LDS staging of its epilogue. gemm_kernels.hip describes the scheme
// and the LDS layouts.
#pragma once

#include "device_common.h"

namespace bitnet {

constexpr int kBI = 256, kBJ = 256;
constexpr int kThreads = 256;        // 4 waves, one per SIMD
constexpr int kWavesI = 2, kWavesJ = 2;
constexpr int kWTI = kBI / kWavesI;  // 128
constexpr int kWTJ = kBJ / kWavesJ;  // 128
constexpr int kFI = kWTI / 32;       // 4
constexpr int kFJ = kWTJ / 32;       // 4
constexpr int kStageBytes = 128;     // operand bytes per row per stage (bf16 or int8)
constexpr int kKSteps = kStageBytes / 32;
constexpr int kPitch = kStageBytes + 16;  // plain tiles: 9 chunks of 16 bytes
constexpr int kRed16 = kStageBytes / 2;   // bf16 reduction elements per stage

// Byte offset of 16-byte chunk c (0..7) of a plain LDS tile row r. Tiles
// written by the transposing loaders (one chunk of many rows at a time)
// XOR-swizzle the chunk index with bits 4..6 of the row so those stores
// spread over the banks; the other tiles are stored plainly.
template <bool SWZ>
__device__ __forceinline__ int lds_off(int r, int c) {
  return r * kPitch + ((SWZ ? (c ^ ((r >> 4) & 7)) : c) << 4);
}

// 16-byte reduction chunk (8 bf16 or 16 int8 values) that lane half h
// supplies at k-step ks. MAP 0: chunk 2ks + h; MAP 1: chunk 4h + ks.
template <int MAP>
__device__ __forceinline__ constexpr int red_chunk(int ks, int h) {
  return MAP == 0 ? 2 * ks + h : 4 * h + ks;
}

// ---------------------------------------------------------------------------
// MFMA flavours
// ---------------------------------------------------------------------------

struct MfmaI8 {
  typedef i32x4_t Frag;
  typedef i32x16_t Acc;
  typedef int Elem;
  static constexpr uint32_t kPoisonBits = 0x80000000u;  // INT32_MIN
  static __device__ __forceinline__ Elem from_bits(uint32_t b) { return (int)b; }
  static __device__ __forceinline__ uint32_t to_bits(Elem e) { return (uint32_t)e; }
  static __device__ __forceinline__ Acc mma(Frag a, Frag b, Acc c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
  }
};

struct MfmaBf16 {
  typedef bf16x8_t Frag;
  typedef f32x16_t Acc;
  typedef float Elem;
  static constexpr uint32_t kPoisonBits = 0x7FC00000u;  // quiet NaN
  static __device__ __forceinline__ Elem from_bits(uint32_t b) { return __uint_as_float(b); }
  static __device__ __forceinline__ uint32_t to_bits(Elem e) { return __float_as_uint(e); }
  static __device__ __forceinline__ Acc mma(Frag a, Frag b, Acc c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};

typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// Fragment readers: the kFI (or kFJ) fragments of a wave for each k-step.
// A k-step is 16 MFMA slots (see gemm_slot); slot<KS, U>() runs after the
// MFMA of slot U and issues this reader's share of the work for later
// slots: the LDS reads of the next k-step's fragments and, for code
// operands, the expansion of fragment f + 1 during the slots of fragment f
// (and of the next k-step's fragment 0 during the last four). k-step 0 of a
// stage is prepared during the last k-step of the previous stage, by the
// reader of the other LDS buffer: ahead<U>() is the share of slot U (after
// the stage's barrier) of the LDS reads and expansion k-step 0 needs.
// frag<KS>(f) is fragment f of k-step KS, ready by the first slot that uses
// it. init() points the reader at the tile of one LDS buffer.
// ---------------------------------------------------------------------------

// The end-of-stage barrier sits in slot kBarrierSlot of the last k-step:
// by then every LDS store of the staged next stage has been issued (each
// loader's kLastStoreSlot is earlier) and the last k-step reads no LDS, so
// the next stage's k-step 0 reads can start right after it and overlap the
// remaining MFMAs of this stage.
constexpr int kBarrierSlot = 8;
static_assert(kBarrierSlot + 7 == 15, "ahead<U> covers the slots after the barrier");

// When the plain (LDS-read) fragments are read. Slot U of k-step KS uses P
// fragment U/4 and Q fragment U%4, so the Q fragments of a k-step are all
// needed in its first four slots and the P fragments in slots 0, 4, 8, 12.
// The next k-step's fragments are read in the first half of the current
// one, Q first, so that each is requested at least 9 slots before its use:
// P fragment f in slot next_read_slot<false>(f), Q fragment f in
// next_read_slot<true>(f); the next stage's k-step 0 fragments are read
// after the stage barrier in the same order (ahead_slot).
template <bool Q>
__device__ __forceinline__ constexpr int next_read_slot(int f) { return Q ? f : (f == 0 ? 0 : 3 + f); }
template <bool Q>
__device__ __forceinline__ constexpr int ahead_slot(int f) {
  return kBarrierSlot + 1 + (Q ? f / 2 : (f == 0 ? 0 : 1 + f));
}
static_assert(ahead_slot<false>(3) < 16, "");

// 16-byte fragments read directly from a plain tile (pitch kPitch).
template <class MT, bool SWZ, int MAP>
struct PlainFrags {
  typename MT::Frag buf[2][4];
  const char* base;
  __device__ __forceinline__ void init(const char* tile, int row0, int lane) {
    // row0 is a multiple of 128, so the swizzle of row row0 + 32f + (l%32)
    // is 2f + bit 4 of l (fragment offsets below)
    const int h = lane >> 5;
    if constexpr (SWZ) {
      static_assert(MAP == 0, "swizzled tiles use chunk map 0");
      base = tile + (row0 + (lane & 31)) * kPitch + 16 * (h ^ ((lane >> 4) & 1));
    } else {
      base = tile + (row0 + (lane & 31)) * kPitch + 16 * red_chunk<MAP>(0, h);
    }
  }
  template <int KS>
  static __device__ __forceinline__ constexpr int off(int f) {
    return SWZ ? f * 32 * kPitch + 32 * (KS ^ f) : f * 32 * kPitch + 16 * (MAP == 0 ? 2 * KS : KS);
  }
  template <int KS>
  __device__ __forceinline__ void read(int f) {
    buf[KS & 1][f] = *reinterpret_cast<const typename MT::Frag*>(base + off<KS>(f));
  }
  template <int U, bool Q>
  __device__ __forceinline__ void ahead() {
    if constexpr (U == ahead_slot<Q>(0)) read<0>(0);
    if constexpr (U == ahead_slot<Q>(1)) read<0>(1);
    if constexpr (U == ahead_slot<Q>(2)) read<0>(2);
    if constexpr (U == ahead_slot<Q>(3)) read<0>(3);
  }
  template <int KS, int U, bool Q>
  __device__ __forceinline__ void slot() {
    if constexpr (KS + 1 < kKSteps) {
      if constexpr (U == next_read_slot<Q>(0)) read<KS + 1>(0);
      if constexpr (U == next_read_slot<Q>(1)) read<KS + 1>(1);
      if constexpr (U == next_read_slot<Q>(2)) read<KS + 1>(2);
      if constexpr (U == next_read_slot<Q>(3)) read<KS + 1>(3);
    }
  }
  template <int KS>
  __device__ __forceinline__ typename MT::Frag frag(int f) const { return buf[KS & 1][f]; }
};

// Forward P: rows of 2-bit codes in the stored layout (tile pitch 48 bytes,
// 32 bytes = 8 words = 128 codes per row per stage). Lane half h of k-step
// ks takes word 4h + ks (codes k = 16(4h+ks)..+15, chunk map 1); one 16-byte
// read per fragment per stage, expanded word by word with
// (w >> 2t) & 0x03030303.
struct CodesI8Frags {
  static constexpr int kPitchB = 48;
  uint4 raw[4];
  MfmaI8::Frag cur[2][4];
  const char* base;
  __device__ __forceinline__ void init(const char* tile, int row0, int lane) {
    base = tile + (row0 + (lane & 31)) * kPitchB + 16 * (lane >> 5);
  }
  template <int KS, int F, int T>
  __device__ __forceinline__ void expand() {
    const uint32_t w = KS == 0 ? raw[F].x : KS == 1 ? raw[F].y : KS == 2 ? raw[F].z : raw[F].w;
    cur[KS & 1][F][T] = (int)codes4_to_i8((w >> (2 * T)) & 0x03030303u);
  }
  template <int U, bool Q>
  __device__ __forceinline__ void ahead() {
    static_assert(kBarrierSlot + 2 < 12, "raw words must be read before slot 12");
    if constexpr (U == kBarrierSlot + 1 || U == kBarrierSlot + 2) {
      constexpr int f0 = 2 * (U - kBarrierSlot - 1);
      raw[f0] = *reinterpret_cast<const uint4*>(base + f0 * 32 * kPitchB);
      raw[f0 + 1] = *reinterpret_cast<const uint4*>(base + (f0 + 1) * 32 * kPitchB);
    }
    if constexpr (U >= 12) expand<0, 0, U - 12>();
  }
  template <int KS, int U, bool Q>
  __device__ __forceinline__ void slot() {
    if constexpr (U / 4 < 3) expand<KS, U / 4 + 1, U % 4>();
    else if constexpr (KS + 1 < kKSteps) expand<KS + 1, 0, U % 4>();
  }
  template <int KS>
  __device__ __forceinline__ MfmaI8::Frag frag(int f) const { return cur[KS & 1][f]; }
};

// dX P: the ternary codes transposed to [k][n] as fp4 (E2M1) nibbles in n
// order (tile pitch 48 bytes, 32 bytes = 64 n per row per stage): +1 = 0x2,
// -1 = 0xA, 0 = 0x0, n even in the low nibble. Lane half h of k-step ks
// takes n = 32h + 8ks..+7 (chunk map 1), dword ks of the 16 bytes at 16h:
// one 16-byte read per fragment per stage. A fragment is expanded by four
// v_cvt_scalef32_pk_bf16_fp4 (scale 1: exact +-1, 0), one per slot.
struct CodesFp4Frags {
  static constexpr int kPitchB = 48;
  uint4 raw[4];
  u32x4_t cur[2][4];
  const char* base;
  __device__ __forceinline__ void init(const char* tile, int row0, int lane) {
    base = tile + (row0 + (lane & 31)) * kPitchB + 16 * (lane >> 5);
  }
  template <int KS, int F, int T>
  __device__ __forceinline__ void expand() {
    const uint32_t w = KS == 0 ? raw[F].x : KS == 1 ? raw[F].y : KS == 2 ? raw[F].z : raw[F].w;
    cur[KS & 1][F][T] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, T));
  }
  template <int U, bool Q>
  __device__ __forceinline__ void ahead() {
    static_assert(kBarrierSlot + 2 < 12, "raw words must be read before slot 12");
    if constexpr (U == kBarrierSlot + 1 || U == kBarrierSlot + 2) {
      constexpr int f0 = 2 * (U - kBarrierSlot - 1);
      raw[f0] = *reinterpret_cast<const uint4*>(base + f0 * 32 * kPitchB);
      raw[f0 + 1] = *reinterpret_cast<const uint4*>(base + (f0 + 1) * 32 * kPitchB);
    }
    if constexpr (U >= 12) expand<0, 0, U - 12>();
  }
  template <int KS, int U, bool Q>
  __device__ __forceinline__ void slot() {
    if constexpr (U / 4 < 3) expand<KS, U / 4 + 1, U % 4>();
    else if constexpr (KS + 1 < kKSteps) expand<KS + 1, 0, U % 4>();
  }
  template <int KS>
  __device__ __forceinline__ MfmaBf16::Frag frag(int f) const {
    return __builtin_bit_cast(MfmaBf16::Frag, cur[KS & 1][f]);
  }
};

// ---------------------------------------------------------------------------
// Operand loaders. load(): global -> registers for one stage (rows row0..+255
// of the operand, reduction stage s); store(): registers -> LDS tile (used
// for the first stage); slot<KS, U>(): the share of MFMA slot U of k-step KS
// in staging the next stage from registers into LDS and fetching the stage
// after it.
// Out-of-range data (rows past the operand, reduction past its end, stages
// past the last) reads as zeros through the buffer resource range check or
// an out-of-range offset, so the loads of a stage are issued without
// branches. Each thread's addresses are a per-thread base plus offsets that
// are uniform or compile-time.
// ---------------------------------------------------------------------------

// Row-major source already in MFMA element form with the reduction axis
// contiguous (x_q for the forward, dY for dX). Thread t handles chunk t%8 of
// rows 8(t/8)+h, h < 8; a wave instruction covers 8 rows x 128 bytes.
// FULL: the valid reduction extent is a multiple of 16 bytes. S0: first
// staging slot (1, or 5 when the other operand is a CopyLoader too).
template <int kElem, bool FULL, int S0 = 1>
struct CopyLoader {
  static constexpr bool kSwz = false;
  static constexpr int kTileB = 256 * kPitch;
  template <class MT, int MAP>
  using Frags = PlainFrags<MT, false, MAP>;
  const char* base;
  int64_t pitch;      // bytes between rows
  int64_t rows;       // valid rows
  int64_t red_bytes;  // valid reduction bytes per row
  // lane_off: byte offset of the thread's chunk of its first row in stage 0
  // (below 2^31: every operand read this way satisfies
  // (rows + 256) * pitch <= 2^31)
  struct Regs { uint4 v[8]; uint32_t lane_off; };

  // Offset of row h of the thread's 8 in stage s, or an out-of-range offset
  // for a chunk past the reduction (and every chunk of a stage past the
  // last): 32-bit arithmetic on a per-lane base and uniform terms, so that
  // the main loop keeps no 64-bit per-lane values.
  __device__ __forceinline__ uint32_t stage_off(const Regs& r, int s, int h) const {
    const int lim = (int)red_bytes - s * kStageBytes;
    return (int)(threadIdx.x & 7) * 16 < lim ? r.lane_off + (uint32_t)(s * kStageBytes) + (uint32_t)(h * pitch) : kOob;
  }

  __device__ __forceinline__ void load(Regs& r, int row0, int s) const {
    const int tid = threadIdx.x;
    const int64_t rowb = row0 + 8 * (tid >> 3);
    if constexpr (FULL) {
      // rows past the end fall outside the resource; chunks past the
      // reduction (and stages past the last) get an out-of-range offset
      const rsrc_t rs = make_rsrc(base, (uint32_t)(rows * pitch));
      r.lane_off = (uint32_t)(rowb * pitch) + (uint32_t)((tid & 7) * 16);
#pragma unroll
      for (int h = 0; h < 8; ++h) r.v[h] = buf_load16(rs, stage_off(r, s, h));
    } else {
      const int64_t kb = (int64_t)s * kStageBytes + (tid & 7) * 16;
      const char* p = base + rowb * pitch + kb;
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        uint32_t d[4] = {0, 0, 0, 0};
        if (kb < red_bytes && rowb + h < rows) {
          const char* src = p + h * pitch;
          if constexpr (kElem == 1) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (kb + e < red_bytes) d[e >> 2] |= uint32_t(uint8_t(src[e])) << (8 * (e & 3));
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (kb + 2 * e < red_bytes)
                d[e >> 1] |= uint32_t(*reinterpret_cast<const uint16_t*>(src + 2 * e)) << (16 * (e & 1));
          }
        }
        r.v[h] = make_uint4(d[0], d[1], d[2], d[3]);
      }
    }
  }
  __device__ __forceinline__ void store(const Regs& r, char* lds) const {
    const int tid = threadIdx.x;
    char* dst = lds + lds_off<kSwz>(8 * (tid >> 3), tid & 7);
#pragma unroll
    for (int h = 0; h < 8; ++h) *reinterpret_cast<uint4*>(dst + h * kPitch) = r.v[h];
  }

  // Staging of the next stage, spread over the slots of k-step KS: rows
  // 2KS, 2KS+1 of the thread's block are stored (slots S0, S0+2), then
  // refilled with stage s+2 (slots S0+8, S0+10).
  struct Tmp {};
  static constexpr int kLastStoreSlot = S0 + 2;
  static_assert(S0 + 10 < 16, "the refills fit the k-step");
  template <int KS, int U>
  __device__ __forceinline__ void slot(Regs& r, Tmp&, char* lds, int row0, int s2) const {
    const int tid = threadIdx.x;
    if constexpr (U == S0 || U == S0 + 2) {
      constexpr int h = 2 * KS + (U == S0 + 2);
      *reinterpret_cast<uint4*>(lds + lds_off<kSwz>(8 * (tid >> 3), tid & 7) + h * kPitch) = r.v[h];
    }
    if constexpr (FULL && (U == S0 + 8 || U == S0 + 10)) {
      constexpr int h = 2 * KS + (U == S0 + 10);
      const rsrc_t rs = make_rsrc(base, (uint32_t)(rows * pitch));
      r.v[h] = buf_load16(rs, stage_off(r, s2, h));
    }
    if constexpr (!FULL && KS == kKSteps - 1 && U == S0 + 8) load(r, row0, s2);
  }
};

// A narrow code operand copied as stored, 32 bytes per row per stage: the
// forward's 2-bit codes [N][Kp/4] (rows n; F = CodesI8Frags) or dX's fp4
// transposed codes [Kp][Np/2] (rows k; F = CodesFp4Frags). Thread t handles
// row t: two 16-byte loads.
template <class F>
struct RowCodesLoader {
  static constexpr bool kSwz = false;
  static constexpr int kTileB = 256 * F::kPitchB;
  template <class MT, int MAP>
  using Frags = F;
  const uint8_t* packed;
  int64_t pitch;  // bytes per row (a multiple of 16)
  int64_t rows;   // valid rows
  // lane_off: byte offset of the thread's row (below 2^31, as every operand
  // read through a buffer resource)
  struct Regs { uint4 v[2]; uint32_t lane_off; };
  struct Tmp {};

  // Half h of the thread's row in stage s; a column past the row (a stage
  // past the last) gets an out-of-range offset. The column test is uniform.
  __device__ __forceinline__ uint32_t offset(const Regs& r, int s, int h) const {
    const int col = s * (kStageBytes / 4) + 16 * h;
    return col < (int)pitch ? r.lane_off + (uint32_t)col : kOob;
  }
  __device__ __forceinline__ void load(Regs& r, int row0, int s) const {
    const rsrc_t rs = make_rsrc(packed, (uint32_t)(rows * pitch));
    r.lane_off = (uint32_t)((row0 + threadIdx.x) * pitch);
#pragma unroll
    for (int h = 0; h < 2; ++h) r.v[h] = buf_load16(rs, offset(r, s, h));
  }
  __device__ __forceinline__ void store(const Regs& r, char* lds) const {
    char* dst = lds + threadIdx.x * F::kPitchB;
    *reinterpret_cast<uint4*>(dst) = r.v[0];
    *reinterpret_cast<uint4*>(dst + 16) = r.v[1];
  }
  // K-steps 0 and 1 store one half of the row (slot 5) and refill it with
  // stage s+2 (slot 13).
  static constexpr int kLastStoreSlot = -1;
  template <int KS, int U>
  __device__ __forceinline__ void slot(Regs& r, Tmp&, char* lds, int row0, int s2) const {
    if constexpr (KS < 2 && U == 5)
      *reinterpret_cast<uint4*>(lds + threadIdx.x * F::kPitchB + 16 * KS) = r.v[KS];
    if constexpr (KS < 2 && U == 13) {
      const rsrc_t rs = make_rsrc(packed, (uint32_t)(rows * pitch));
      r.v[KS] = buf_load16(rs, offset(r, s2, KS));
    }
  }
};
using PackedCodesLoader = RowCodesLoader<CodesI8Frags>;

// dW operands from a bf16 [rows m][ld] matrix read transposed: rows j
// (n of dY for Q, k of x_hat for P), reduction m (strided). Thread
// (mg = wave, nq = lane) reads 4 bf16 (columns 4nq..4nq+3) from each of the
// rows m = 16mg..16mg+15 and writes the 16 x 4 transpose as 4 rows of 16 m
// values.
template <bool VEC, int W0>
struct RowTransposeBf16Loader {
  static constexpr bool kSwz = true;
  static constexpr int kTileB = 256 * kPitch;
  template <class MT, int MAP>
  using Frags = PlainFrags<MT, true, MAP>;
  const uint16_t* dy;
  int64_t ld;    // elements per source row (N, or Kp for x_hat)
  int64_t mred;  // M (valid reduction rows)
  int64_t rows;  // valid operand rows (N, or Kp)
  // lane_off: byte offset of the thread's first element in stage 0, or an
  // out-of-range offset for columns past the operand (adding a stage's
  // offset, below 2^31, keeps it out of range)
  struct Regs { uint2 v[16]; uint32_t lane_off; };

  // Byte offset of row e of the thread's 16 in stage s (uniform part).
  __device__ __forceinline__ uint32_t stage_off(int s, int e) const {
    return (uint32_t)(((int64_t)s * kRed16 + e) * ld * 2);
  }
  __device__ __forceinline__ void load(Regs& r, int row0, int s) const {
    const int tid = threadIdx.x;
    const int64_t m = (int64_t)s * kRed16 + 16 * (tid >> 6);
    const int64_t n = row0 + 4 * (tid & 63);
    if constexpr (VEC) {
      const rsrc_t rs = make_rsrc(dy, (uint32_t)(mred * ld * 2));
      r.lane_off = n < rows ? (uint32_t)((16 * (tid >> 6) * ld + n) * 2) : kOob;
#pragma unroll
      for (int e = 0; e < 16; ++e) r.v[e] = buf_load8(rs, r.lane_off + stage_off(s, e));
    } else {
      const uint16_t* p = dy + m * ld + n;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        uint32_t q[4] = {0, 0, 0, 0};
        if (m + e < mred) {
          const uint16_t* src = p + e * ld;
#pragma unroll
          for (int j = 0; j < 4; ++j) q[j] = (n + j < rows) ? src[j] : 0u;
        }
        r.v[e] = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
      }
    }
  }
  __device__ __forceinline__ void store(const Regs& r, char* lds) const {
    const int tid = threadIdx.x;
    const int nq = tid & 63, mg = tid >> 6;
    // element (m = e, n = q) is half (q & 1) of word (q >> 1) of v[e]
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      char* dst = lds + lds_off<kSwz>(4 * nq, 2 * mg + hh);  // rows 4nq..4nq+3 share the swizzle
      const uint2* v = r.v + 8 * hh;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t sel = (q & 1) ? 0x07060302u : 0x05040100u;
        uint4 o;
        o.x = perm((q >> 1) ? v[1].y : v[1].x, (q >> 1) ? v[0].y : v[0].x, sel);
        o.y = perm((q >> 1) ? v[3].y : v[3].x, (q >> 1) ? v[2].y : v[2].x, sel);
        o.z = perm((q >> 1) ? v[5].y : v[5].x, (q >> 1) ? v[4].y : v[4].x, sel);
        o.w = perm((q >> 1) ? v[7].y : v[7].x, (q >> 1) ? v[6].y : v[6].x, sel);
        *reinterpret_cast<uint4*>(dst + q * kPitch) = o;
      }
    }
  }

  // Staging in the slots of k-step KS: half hh = KS/2 (m rows 8hh..8hh+7 of
  // the thread's 16), n columns q = 2(KS&1), +1 (slots W0, W0+1; each uses
  // all 8 rows); odd k-steps then refill that half's 8 rows with stage s+2,
  // one row per slot (slots W0+2 .. W0+9) so that the loads of the two
  // operands do not arrive at the memory pipeline in bursts. W0 = 3 for the
  // P operand and 5 for Q.
  struct Tmp {};
  static constexpr int kLastStoreSlot = W0 + 1;
  __device__ __forceinline__ void write_q(const Regs& r, char* lds, int hh, int q) const {
    const int tid = threadIdx.x;
    const int nq = tid & 63, mg = tid >> 6;
    char* dst = lds + lds_off<kSwz>(4 * nq, 2 * mg + hh);
    const uint2* v = r.v + 8 * hh;
    const uint32_t sel = (q & 1) ? 0x07060302u : 0x05040100u;
    uint4 o;
    o.x = perm((q >> 1) ? v[1].y : v[1].x, (q >> 1) ? v[0].y : v[0].x, sel);
    o.y = perm((q >> 1) ? v[3].y : v[3].x, (q >> 1) ? v[2].y : v[2].x, sel);
    o.z = perm((q >> 1) ? v[5].y : v[5].x, (q >> 1) ? v[4].y : v[4].x, sel);
    o.w = perm((q >> 1) ? v[7].y : v[7].x, (q >> 1) ? v[6].y : v[6].x, sel);
    *reinterpret_cast<uint4*>(dst + q * kPitch) = o;
  }
  template <int KS, int U>
  __device__ __forceinline__ void slot(Regs& r, Tmp&, char* lds, int row0, int s2) const {
    constexpr int hh = KS >> 1;
    if constexpr (U == W0 || U == W0 + 1) write_q(r, lds, hh, 2 * (KS & 1) + (U == W0 + 1));
    if constexpr ((KS & 1) && U >= W0 + 2 && U < W0 + 10) {
      if constexpr (VEC) {
        const rsrc_t rs = make_rsrc(dy, (uint32_t)(mred * ld * 2));
        constexpr int e = 8 * hh + (U - W0 - 2);
        r.v[e] = buf_load8(rs, r.lane_off + stage_off(s2, e));
      } else if constexpr (KS == kKSteps - 1 && U == W0 + 9) {
        load(r, row0, s2);
      }
    }
  }
};

// dW operands kept in their memory orientation. The tile of a stage is 64
// reduction rows m x 256 operand rows (columns of the source), copied as
// stored into LDS rows of kTrPitch bytes, and the fragments are read with
// ds_read_b64_tr_b16, which transposes 4 x 16 blocks of 16-bit values on
// the way out: in each 16-lane group, lane 4e + q addresses LDS row e,
// columns 4q..4q+3, and lane 4q + p receives column 4q + p of rows 0..3.
// A 32 x 16 MFMA fragment is two such reads per lane (reduction rows
// 16KS + 8h + 0..3 and + 4..7 for lane half h). The 64-byte row padding puts
// the 4 rows a 32-lane half reads 16 banks apart, so a read is free of bank
// conflicts, and a staging store (one 512-byte row per half-wave) is too.
constexpr int kTrPitch = 512 + 64;

typedef short v4i16_t __attribute__((ext_vector_type(4)));

template <int PITCH>
struct TrFragsP {
  MfmaBf16::Frag buf[2][4];
  const char* base;
  __device__ __forceinline__ void init(const char* tile, int row0, int lane) {
    const int g = lane >> 4, e = (lane >> 2) & 3, q = lane & 3;
    base = tile + (8 * (g >> 1) + e) * PITCH + 2 * (row0 + 16 * (g & 1) + 4 * q);
  }
  static __device__ __forceinline__ v4i16_t tr(const char* p) {
    typedef __attribute__((address_space(3))) v4i16_t lds_v4i16_t;
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_t*)(__attribute__((address_space(3))) char*)p);
  }
  template <int KS>
  __device__ __forceinline__ void read(int f) {
    const char* a = base + 16 * KS * PITCH + 64 * f;
    const v4i16_t lo = tr(a), hi = tr(a + 4 * PITCH);
    typedef short v8i16_t __attribute__((ext_vector_type(8)));
    const v8i16_t v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    buf[KS & 1][f] = __builtin_bit_cast(MfmaBf16::Frag, v);
  }
  template <int U, bool Q>
  __device__ __forceinline__ void ahead() {
    if constexpr (U == ahead_slot<Q>(0)) read<0>(0);
    if constexpr (U == ahead_slot<Q>(1)) read<0>(1);
    if constexpr (U == ahead_slot<Q>(2)) read<0>(2);
    if constexpr (U == ahead_slot<Q>(3)) read<0>(3);
  }
  template <int KS, int U, bool Q>
  __device__ __forceinline__ void slot() {
    if constexpr (KS + 1 < kKSteps) {
      if constexpr (U == next_read_slot<Q>(0)) read<KS + 1>(0);
      if constexpr (U == next_read_slot<Q>(1)) read<KS + 1>(1);
      if constexpr (U == next_read_slot<Q>(2)) read<KS + 1>(2);
      if constexpr (U == next_read_slot<Q>(3)) read<KS + 1>(3);
    }
  }
  template <int KS>
  __device__ __forceinline__ MfmaBf16::Frag frag(int f) const { return buf[KS & 1][f]; }
};

using TrFrags = TrFragsP<kTrPitch>;

// Copy loader for TrFrags tiles from a bf16 [m][ld] matrix whose first
// `cols` columns are the operand rows (x_hat: ld = cols = Kp; dY: ld = cols
// = N), ld a multiple of 8 so that 16-byte pieces never straddle a row end.
// Thread t handles 16-byte chunk t % 32 of reduction rows t / 32 + 8h,
// h < 8 (a wave instruction covers 2 rows x 512 bytes). Staging in k-step
// KS: rows h = 2KS, 2KS + 1 are stored (slots S0, S0 + 2) and refilled with
// stage s+2 (slots S0 + 8, S0 + 10). S0 = 1 for P and 5 for Q.
template <int S0>
struct RowCopyBf16Loader {
  static constexpr bool kSwz = false;
  static constexpr int kTileB = 64 * kTrPitch;
  static constexpr int kLastStoreSlot = S0 + 2;
  template <class MT, int MAP>
  using Frags = TrFrags;
  const uint16_t* src;
  int64_t ld;    // elements per source row
  int64_t mred;  // valid reduction rows (M)
  int64_t cols;  // valid operand rows (columns of the source)
  // lane_off: byte offset of the thread's chunk in stage 0, row t/32, or an
  // out-of-range offset for chunks past `cols`
  struct Regs { uint4 v[8]; uint32_t lane_off; };
  struct Tmp {};

  __device__ __forceinline__ uint32_t stage_off(int s, int h) const {
    return (uint32_t)(((int64_t)s * kRed16 + 8 * h) * ld * 2);
  }
  __device__ __forceinline__ void load(Regs& r, int row0, int s) const {
    const int tid = threadIdx.x;
    const int64_t col = row0 + 8 * (tid & 31);
    r.lane_off = col < cols ? (uint32_t)(((tid >> 5) * ld + col) * 2) : kOob;
    const rsrc_t rs = make_rsrc(src, (uint32_t)(mred * ld * 2));
#pragma unroll
    for (int h = 0; h < 8; ++h) r.v[h] = buf_load16(rs, r.lane_off + stage_off(s, h));
  }
  __device__ __forceinline__ void store(const Regs& r, char* lds) const {
    const int tid = threadIdx.x;
    char* dst = lds + (tid >> 5) * kTrPitch + 16 * (tid & 31);
#pragma unroll
    for (int h = 0; h < 8; ++h) *reinterpret_cast<uint4*>(dst + 8 * h * kTrPitch) = r.v[h];
  }
  template <int KS, int U>
  __device__ __forceinline__ void slot(Regs& r, Tmp&, char* lds, int, int s2) const {
    const int tid = threadIdx.x;
    if constexpr (U == S0 || U == S0 + 2) {
      constexpr int h = 2 * KS + (U == S0 + 2);
      *reinterpret_cast<uint4*>(lds + ((tid >> 5) + 8 * h) * kTrPitch + 16 * (tid & 31)) = r.v[h];
    }
    if constexpr (U == S0 + 8 || U == S0 + 10) {
      constexpr int h = 2 * KS + (U == S0 + 10);
      const rsrc_t rs = make_rsrc(src, (uint32_t)(mred * ld * 2));
      r.v[h] = buf_load16(rs, r.lane_off + stage_off(s2, h));
    }
  }
};

// Workgroup b of G, dispatched round-robin over the 8 XCDs, to a virtual
// index numbered XCD by XCD: an XCD owns a contiguous range of indices.
__host__ __device__ __forceinline__ int cta_order(int b, int G) {
  const int q = G / 8, r = G % 8;
  const int x = b % 8, k = b / 8;
  return (x < r) ? x * (q + 1) + k : r * (q + 1) + (x - r) * q + k;
}

// Tagged counters: a 64-bit word gen << 16 | count. A word written by
// another launch (another tag) counts as zero, so the counters never need
// clearing before a launch; the last piece of a tile clears its two words
// once they are no longer used, so that a launch repeated with the same tag
// (a captured graph replayed) also starts from zero. The counters only
// order the exchange of partial tiles, whose stores and loads are
// device-coherent and complete (wait_vmem) before the counter moves, so
// relaxed device-scope atomics suffice and no cache-wide fence is needed.
constexpr uint64_t kCountMask = 0xFFFF;

__device__ __forceinline__ uint32_t tagged_arrive(uint64_t* c, uint64_t gen) {
  uint64_t old = __hip_atomic_load(c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (;;) {
    const bool same = (old >> 16) == gen;
    const uint64_t nw = same ? old + 1 : ((gen << 16) | 1u);
    if (__hip_atomic_compare_exchange_strong(c, &old, nw, __ATOMIC_RELAXED, __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT))
      return same ? (uint32_t)(old & kCountMask) : 0u;
  }
}

template <class Acc>
__device__ __forceinline__ void zero_acc(Acc& a) {
#pragma unroll
  for (int e = 0; e < 16; ++e) a[e] = 0;
}

// All of ahead<U>() of a reader at once (the first stage of a run).
template <bool Q, class F>
__device__ __forceinline__ void prime(F& f) {
  f.template ahead<kBarrierSlot + 1, Q>(); f.template ahead<kBarrierSlot + 2, Q>();
  f.template ahead<kBarrierSlot + 3, Q>(); f.template ahead<kBarrierSlot + 4, Q>();
  f.template ahead<kBarrierSlot + 5, Q>(); f.template ahead<kBarrierSlot + 6, Q>();
  f.template ahead<kBarrierSlot + 7, Q>();
}

// One MFMA slot of a k-step: MFMA (U / 4, U % 4), then each reader's and
// loader's share of the work for U (issued behind the MFMA so that it
// overlaps its 32 cycles), fenced from the next slot so that the compiler
// keeps this interleave. fpn/fqn read the other LDS buffer (the next
// stage); `more` says whether there is a next stage.
template <int KS, int U, class MT, class PL, class QL, class FP, class FQ>
__device__ __forceinline__ void gemm_slot(const PL& pl, const QL& ql, typename PL::Regs& pr,
                                          typename QL::Regs& qr, typename PL::Tmp& pt,
                                          typename QL::Tmp& qt, FP& fp, FQ& fq, FP& fpn, FQ& fqn,
                                          char* Pn, char* Qn, typename MT::Acc (&acc)[kFI][kFJ],
                                          int i0, int j0, int s2, bool more) {
  acc[U / 4][U % 4] = MT::mma(fp.template frag<KS>(U / 4), fq.template frag<KS>(U % 4), acc[U / 4][U % 4]);
  fp.template slot<KS, U, false>();
  fq.template slot<KS, U, true>();
  pl.template slot<KS, U>(pr, pt, Pn, i0, s2);
  ql.template slot<KS, U>(qr, qt, Qn, j0, s2);
  if constexpr (KS == kKSteps - 1) {
    if constexpr (U == kBarrierSlot) __syncthreads();
    if constexpr (U > kBarrierSlot) {
      if (more) {
        fpn.template ahead<U, false>();
        fqn.template ahead<U, true>();
      }
    }
  }
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (U + 1 < kFI * kFJ)
    gemm_slot<KS, U + 1, MT>(pl, ql, pr, qr, pt, qt, fp, fq, fpn, fqn, Pn, Qn, acc, i0, j0, s2, more);
}

// LDS: two stages, each a P tile followed by a Q tile.
template <class PL, class QL>
struct SmemLayout {
  static constexpr int kStage = PL::kTileB + QL::kTileB;
  static constexpr int kBytes = 2 * kStage;
};

// One pipeline stage: MFMAs on LDS buffer CUR (readers fp, fq) for
// reduction stage s, while staging stage s+1 from registers into buffer
// CUR^1 and fetching stage s+2 into those registers, one quarter per
// k-step, and, when `more`, preparing k-step 0 of stage s+1 (readers fpn,
// fqn of buffer CUR^1). Past the last stage the staging runs on zeros and
// is never read.
template <int CUR, class MT, class PL, class QL, class FP, class FQ>
__device__ __forceinline__ void gemm_stage(const PL& pl, const QL& ql, typename PL::Regs& pr,
                                           typename QL::Regs& qr, char* smem, FP& fp, FQ& fq,
                                           FP& fpn, FQ& fqn, typename MT::Acc (&acc)[kFI][kFJ],
                                           int i0, int j0, int s, bool more) {
  typedef SmemLayout<PL, QL> L;
  char* Pn = smem + (CUR ^ 1) * L::kStage;
  char* Qn = Pn + PL::kTileB;
  typename PL::Tmp pt;
  typename QL::Tmp qt;
  gemm_slot<0, 0, MT>(pl, ql, pr, qr, pt, qt, fp, fq, fpn, fqn, Pn, Qn, acc, i0, j0, s + 2, more);
  gemm_slot<1, 0, MT>(pl, ql, pr, qr, pt, qt, fp, fq, fpn, fqn, Pn, Qn, acc, i0, j0, s + 2, more);
  gemm_slot<2, 0, MT>(pl, ql, pr, qr, pt, qt, fp, fq, fpn, fqn, Pn, Qn, acc, i0, j0, s + 2, more);
  gemm_slot<3, 0, MT>(pl, ql, pr, qr, pt, qt, fp, fq, fpn, fqn, Pn, Qn, acc, i0, j0, s + 2, more);
}

// The stages [s0, s1) of tile (i0, j0), accumulated into acc. LDS is free
// on entry and on return. `arrive`, when not NULL, is the published-partials
// counter of this workgroup's previous piece, whose partial stores were
// issued but not waited for: it is incremented (tag gen) once every wave
// has waited for its first stage's loads, which were issued after those
// stores, so the stores are complete by then.
template <class MT, int MAP, class PL, class QL>
__device__ __forceinline__ void run_stages(const PL& pl, const QL& ql, char* smem,
                                           typename MT::Acc (&acc)[kFI][kFJ], int i0, int j0, int s0,
                                           int s1, int prow0, int qrow0, int lane, uint64_t* arrive,
                                           uint64_t gen) {
  static_assert(PL::kLastStoreSlot < kBarrierSlot && QL::kLastStoreSlot < kBarrierSlot,
                "staging stores must precede the end-of-stage barrier");
  typedef SmemLayout<PL, QL> L;
  typename PL::Regs pr;
  typename QL::Regs qr;
  pl.load(pr, i0, s0);
  ql.load(qr, j0, s0);
  __syncthreads();
  pl.store(pr, smem);
  ql.store(qr, smem + PL::kTileB);
  pl.load(pr, i0, s0 + 1);
  ql.load(qr, j0, s0 + 1);
  __syncthreads();
  if (arrive != nullptr && threadIdx.x == 0) tagged_arrive(arrive, gen);
  typename PL::template Frags<MT, MAP> fp0, fp1;
  typename QL::template Frags<MT, MAP> fq0, fq1;
  fp0.init(smem, prow0, lane);
  fq0.init(smem + PL::kTileB, qrow0, lane);
  fp1.init(smem + L::kStage, prow0, lane);
  fq1.init(smem + L::kStage + PL::kTileB, qrow0, lane);
  prime<false>(fp0);
  prime<true>(fq0);
  __builtin_amdgcn_sched_barrier(0);
  int s = s0;
  for (; s + 1 < s1; s += 2) {
    gemm_stage<0, MT>(pl, ql, pr, qr, smem, fp0, fq0, fp1, fq1, acc, i0, j0, s, true);
    gemm_stage<1, MT>(pl, ql, pr, qr, smem, fp1, fq1, fp0, fq0, acc, i0, j0, s + 1, s + 2 < s1);
  }
  if (s < s1) gemm_stage<0, MT>(pl, ql, pr, qr, smem, fp0, fq0, fp1, fq1, acc, i0, j0, s, false);
}

// ---------------------------------------------------------------------------
// Epilogues: acc (wave tile origin i0, j0) -> memory. Lane l holds, for each
// fragment (fi, fj) and group g, the 4 consecutive i = i0 + 32fi + 8g +
// 4(l/32) + 0..3 at j = j0 + 32fj + l%32.
//
// Stored from the accumulator layout, one instruction would write 16-byte
// pieces of 32 output rows, which runs at about half the HBM write rate of
// whole-row stores. The block goes through LDS instead (EpStage): in four
// passes of 32 rows j (one fragment column fj), each lane puts its 4-value
// pieces into a per-wave LDS buffer of 32 rows, and every store instruction
// then writes whole 128-value row segments (4 rows of bf16 or 2 of 32-bit
// values). LDS rows are padded by 16 bytes: the 16 rows a half-wave puts to
// start 4 banks apart, and a row read by 16 or 32 lanes covers every bank
// once; all LDS offsets are a per-lane base plus a constant. LDS is free
// when the epilogue runs: the last stage's reads and staging stores all
// precede its barrier.
// ---------------------------------------------------------------------------

template <int EB>  // bytes per output element: 2 (bf16) or 4 (f32, int32)
struct EpStage {
  static constexpr int kRowB = 128 * EB;
  static constexpr int kPitch = kRowB + 16;
  static constexpr int kChunks = kRowB / 16;
  static constexpr int kWaveBytes = 32 * kPitch;
  static constexpr int kRowsPerGet = 1024 / kRowB;  // rows per wave instruction
  static constexpr int kGets = 32 / kRowsPerGet;
  // The lane's piece of (fi, g): 4 values of row l%32 at i = 32fi + 8g + 4(l/32).
  template <class V>
  static __device__ __forceinline__ void put(char* w, int lane, int fi, int g, V v) {
    char* base = w + (lane & 31) * kPitch + 4 * EB * (lane >> 5);
    *reinterpret_cast<V*>(base + (32 * fi + 8 * g) * EB) = v;
  }
  // Row-wise read-out of the 32 rows into out[j][i] (rows of I elements):
  // get k is the 16 bytes of row k * kRowsPerGet + lane / kChunks, chunk
  // lane % kChunks, i.e. out[j0 + row][i0 + chunk * 16 / EB ..]. All gets
  // are issued first. When I is a multiple of 16 / EB (a chunk then lies
  // all inside or all outside a row), each get is one 16-byte store through
  // a buffer resource based at the pass's first row (a streaming store: the
  // output is not read again by the launch), with the row offset as the
  // uniform soffset and an out-of-range voffset for rows at or past J
  // and chunks at or past I (32 * I * EB < 2^31, checked by the C ABI);
  // otherwise rows are not 16-byte aligned and the valid elements are
  // stored one by one. i0, j0 are uniform in the wave.
  static __device__ __forceinline__ void drain(const char* w, char* out, int64_t I, int64_t J, int i0, int j0,
                                               int lane) {
    i0 = __builtin_amdgcn_readfirstlane(i0);
    j0 = __builtin_amdgcn_readfirstlane(j0);
    int c = lane % kChunks, rl = lane / kChunks;
    // opaque to the optimizer: keeps the per-get row terms from being
    // computed once per kernel and spilled across the main loop
    asm volatile("" : "+v"(c), "+v"(rl));
    const char* src = w + rl * kPitch + 16 * c;
    uint4 v[kGets];
#pragma unroll
    for (int k = 0; k < kGets; ++k) v[k] = *reinterpret_cast<const uint4*>(src + k * kRowsPerGet * kPitch);
    const int rows_in = J - j0 < 32 ? (int)(J - j0) : 32;
    if ((I & (16 / EB - 1)) == 0) {
      const uint32_t row_b = (uint32_t)I * EB;
      const rsrc_t rs = make_rsrc(out + ((int64_t)j0 * I + i0) * EB, 32u * row_b);
      const uint32_t lane_off = i0 + c * (16 / EB) < I ? rl * row_b + 16 * c : kOob;
#pragma unroll
      for (int k = 0; k < kGets; ++k)
        buf_store16_stream(rs, rl < rows_in - k * kRowsPerGet ? lane_off : kOob,
                           (uint32_t)(k * kRowsPerGet) * row_b, v[k]);
    } else {
      const int64_t i = i0 + c * (16 / EB);
#pragma unroll
      for (int k = 0; k < kGets; ++k) {
        if (k * kRowsPerGet + rl >= rows_in) continue;
        char* row = out + (int64_t)(j0 + k * kRowsPerGet + rl) * I * EB;
        const uint32_t wv[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int e = 0; e < 16 / EB; ++e) {
          if (i + e >= I) continue;
          if constexpr (EB == 2)
            reinterpret_cast<uint16_t*>(row)[i + e] = (uint16_t)(wv[e >> 1] >> (16 * (e & 1)));
          else
            reinterpret_cast<uint32_t*>(row)[i + e] = wv[e];
        }
      }
    }
  }
};

}  // namespace bitnet
