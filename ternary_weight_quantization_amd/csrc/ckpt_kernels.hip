// Activations kept in 8 bits between the forward and the backward pass:
// codes and block scales (row_io.h), packed from bf16 or f32 rows and
// unpacked again, and the gated activation of a feed-forward block, whose
// backward reads the codes of its two inputs.
//
// Everything here is one pass over HBM: a block of 128 values is 16 lanes of
// 8, its scale is a rotation maximum within a DPP row, and a lane's 8 codes
// are one 8-byte store. Measured at 4096 x 6912 with gate, up and both codes:
// forward 46.5 us (228 MB, 4.9 TB/s), backward 37.8 us (228 MB, some of it from
// the last level cache); 2048 x 2560 packed in 6.2 us and unpacked in 6.8.

#include "activation.h"
#include "internal.h"
#include "row_io.h"

namespace bitnet {

constexpr int kRowThreads = 256;

// A thread per chunk, `total` of them (below 2^32: the most threads a launch
// may have): chunk index -> row and chunk within the row. nch is a multiple of
// 16, so the 16 lanes of a block share a row.
struct ChunkAt {
  int64_t row;
  int ch;
};
__device__ __forceinline__ uint32_t chunk_index() { return blockIdx.x * (uint32_t)kRowThreads + threadIdx.x; }
__device__ __forceinline__ ChunkAt chunk_at(uint32_t i, int nch) {
  const uint32_t r = i / (uint32_t)nch;
  return {(int64_t)r, (int)(i - r * (uint32_t)nch)};
}

template <class T>
__global__ __launch_bounds__(kRowThreads) void ckpt_pack_kernel(const T* __restrict__ x, uint32_t total, int K, int nch,
                                                                int8_t* __restrict__ codes,
                                                                float* __restrict__ scales) {
  const uint32_t i = chunk_index();
  if (i >= total) return;  // total is a multiple of 16: whole blocks leave
  const ChunkAt at = chunk_at(i, nch);
  const typename ChunkOf<T>::type c = chunk8(x + at.row * K, 8 * at.ch, K);
  float f[8];
  c.get(f);
  const float s = block_scale(c);
  reinterpret_cast<uint2*>(codes)[i] = codes8(f, s);
  if ((threadIdx.x & 15) == 0) scales[i >> 4] = s;
}

// Rows of ld values: the codes past K stand for zeros.
template <class T>
__global__ __launch_bounds__(kRowThreads) void ckpt_unpack_kernel(const int8_t* __restrict__ codes,
                                                                  const float* __restrict__ scales, uint32_t total,
                                                                  int ld, int nch, T* __restrict__ x) {
  const uint32_t i = chunk_index();
  if (i >= total) return;
  const ChunkAt at = chunk_at(i, nch);
  float f[8];
  values8(reinterpret_cast<const uint2*>(codes)[i], scales[i >> 4] / 127.0f, f);
  store8(x + at.row * ld, 8 * at.ch, ld, f);
}

// Rows of K bf16 values copied to rows of ld (zeros past K), and with codes
// their checkpoint from the same registers.
__global__ __launch_bounds__(kRowThreads) void pad_rows_kernel(const uint16_t* __restrict__ x, uint32_t total, int K,
                                                               int nch, uint16_t* __restrict__ padded, int ld,
                                                               int8_t* __restrict__ codes, float* __restrict__ scales) {
  const uint32_t i = chunk_index();
  if (i >= total) return;
  const ChunkAt at = chunk_at(i, nch);
  const ChunkBf16 c = chunk8(x + at.row * K, 8 * at.ch, K);
  if (8 * at.ch < ld) *reinterpret_cast<uint4*>(padded + at.row * ld + 8 * at.ch) = c.v;
  if (codes == nullptr) return;
  float f[8];
  c.get(f);
  const float s = block_scale(c);
  reinterpret_cast<uint2*>(codes)[i] = codes8(f, s);
  if ((threadIdx.x & 15) == 0) scales[i >> 4] = s;
}

static unsigned row_grid(uint32_t total) { return (total + kRowThreads - 1) / kRowThreads; }

hipError_t launch_ckpt_pack(const void* x, bool x_f32, int64_t M, int64_t K, int8_t* codes, float* scales,
                            hipStream_t stream) {
  const int nch = (int)(ckpt_pad(K) / 8);
  const uint32_t total = (uint32_t)(M * nch);
  if (x_f32)
    ckpt_pack_kernel<<<row_grid(total), kRowThreads, 0, stream>>>(static_cast<const float*>(x), total, (int)K, nch,
                                                                  codes, scales);
  else
    ckpt_pack_kernel<<<row_grid(total), kRowThreads, 0, stream>>>(static_cast<const uint16_t*>(x), total, (int)K, nch,
                                                                  codes, scales);
  return hipGetLastError();
}

hipError_t launch_pad_rows(const uint16_t* x, int64_t M, int64_t K, uint16_t* padded, int64_t ld, int8_t* codes,
                           float* scales, hipStream_t stream) {
  const int nch = (int)(ckpt_pad(K) / 8);
  const uint32_t total = (uint32_t)(M * nch);
  pad_rows_kernel<<<row_grid(total), kRowThreads, 0, stream>>>(x, total, (int)K, nch, padded, (int)ld, codes, scales);
  return hipGetLastError();
}

hipError_t launch_ckpt_unpack(const int8_t* codes, const float* scales, int64_t M, int64_t K, void* x, int64_t ld,
                              bool x_f32, hipStream_t stream) {
  const int nch = (int)(ckpt_pad(K) / 8);
  const uint32_t total = (uint32_t)(M * nch);
  if (x_f32)
    ckpt_unpack_kernel<<<row_grid(total), kRowThreads, 0, stream>>>(codes, scales, total, (int)ld, nch,
                                                                    static_cast<float*>(x));
  else
    ckpt_unpack_kernel<<<row_grid(total), kRowThreads, 0, stream>>>(codes, scales, total, (int)ld, nch,
                                                                    static_cast<uint16_t*>(x));
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Gated activation y = act(gate) * up (up absent: y = act(gate)).
// ---------------------------------------------------------------------------

// CK: the codes of gate and up are written too.
template <class A, bool CK, bool UP>
__global__ __launch_bounds__(kRowThreads) void gate_fwd_kernel(const uint16_t* __restrict__ gate, int64_t ldg,
                                                               const uint16_t* __restrict__ up, int64_t ldu,
                                                               uint32_t total, int K, int nch, uint16_t* __restrict__ y,
                                                               int8_t* __restrict__ gq, float* __restrict__ gs,
                                                               int8_t* __restrict__ uq, float* __restrict__ us) {
  const uint32_t i = chunk_index();
  if (i >= total) return;
  const ChunkAt at = chunk_at(i, nch);
  const int k0 = 8 * at.ch;
  // every load before the first use
  ChunkBf16 cg, cu;
  if (K < 8) {
    cg = load8<true>(gate + at.row * ldg, k0, K);
    if constexpr (UP) cu = load8<true>(up + at.row * ldu, k0, K);
  } else {
    cg = load8<false>(gate + at.row * ldg, k0, K);
    if constexpr (UP) cu = load8<false>(up + at.row * ldu, k0, K);
    settle8<false>(cg, k0, K);
    if constexpr (UP) settle8<false>(cu, k0, K);
  }
  float g[8], u[8], o[8];
  cg.get(g);
  if constexpr (UP) cu.get(u);
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = UP ? A::f(g[e]) * u[e] : A::f(g[e]);
  store8(y + at.row * K, k0, K, o);
  if constexpr (CK) {
    const float s = block_scale(cg);
    reinterpret_cast<uint2*>(gq)[i] = codes8(g, s);
    if ((threadIdx.x & 15) == 0) gs[i >> 4] = s;
    if constexpr (UP) {
      const float t = block_scale(cu);
      reinterpret_cast<uint2*>(uq)[i] = codes8(u, t);
      if ((threadIdx.x & 15) == 0) us[i >> 4] = t;
    }
  }
}

// CK: gate and up come from their codes, else from the bf16 rows.
template <class A, bool CK, bool UP>
__global__ __launch_bounds__(kRowThreads) void gate_bwd_kernel(const uint16_t* __restrict__ dY,
                                                               const uint16_t* __restrict__ gate, int64_t ldg,
                                                               const uint16_t* __restrict__ up, int64_t ldu,
                                                               const int8_t* __restrict__ gq,
                                                               const float* __restrict__ gs,
                                                               const int8_t* __restrict__ uq,
                                                               const float* __restrict__ us, uint32_t total, int K,
                                                               int nch, uint16_t* __restrict__ dgate, int64_t lddg,
                                                               uint16_t* __restrict__ dup, int64_t lddu) {
  const uint32_t i = chunk_index();
  if (i >= total) return;
  const ChunkAt at = chunk_at(i, nch);
  const int k0 = 8 * at.ch;
  float g[8], u[8], d[8];
  if constexpr (CK) {
    const uint2 qg = reinterpret_cast<const uint2*>(gq)[i];
    const float sg = gs[i >> 4];
    uint2 qu = make_uint2(0u, 0u);
    float su = 0.0f;
    if constexpr (UP) {
      qu = reinterpret_cast<const uint2*>(uq)[i];
      su = us[i >> 4];
    }
    chunk8(dY + at.row * K, k0, K).get(d);
    values8(qg, sg / 127.0f, g);
    if constexpr (UP) values8(qu, su / 127.0f, u);
  } else {
    chunk8(gate + at.row * ldg, k0, K).get(g);
    if constexpr (UP) chunk8(up + at.row * ldu, k0, K).get(u);
    chunk8(dY + at.row * K, k0, K).get(d);
  }
  float dg[8], du[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float a, da;
    A::fd(g[e], a, da);
    dg[e] = UP ? d[e] * u[e] * da : d[e] * da;
    du[e] = d[e] * a;
  }
  store8(dgate + at.row * lddg, k0, K, dg);
  if constexpr (UP) store8(dup + at.row * lddu, k0, K, du);
}

template <class A>
static void gate_fwd(const uint16_t* gate, int64_t ldg, const uint16_t* up, int64_t ldu, int64_t M, int64_t K,
                     uint16_t* y, int8_t* gq, float* gs, int8_t* uq, float* us, hipStream_t st) {
  const int nch = (int)(ckpt_pad(K) / 8);
  const uint32_t total = (uint32_t)(M * nch);
  const unsigned grid = row_grid(total);
  const int k = (int)K;
  if (up && gq) gate_fwd_kernel<A, true, true><<<grid, kRowThreads, 0, st>>>(gate, ldg, up, ldu, total, k, nch, y, gq, gs, uq, us);
  else if (up) gate_fwd_kernel<A, false, true><<<grid, kRowThreads, 0, st>>>(gate, ldg, up, ldu, total, k, nch, y, gq, gs, uq, us);
  else if (gq) gate_fwd_kernel<A, true, false><<<grid, kRowThreads, 0, st>>>(gate, ldg, up, ldu, total, k, nch, y, gq, gs, uq, us);
  else gate_fwd_kernel<A, false, false><<<grid, kRowThreads, 0, st>>>(gate, ldg, up, ldu, total, k, nch, y, gq, gs, uq, us);
}

hipError_t launch_gate_fwd(bool relu2, const uint16_t* gate, int64_t ldg, const uint16_t* up, int64_t ldu, int64_t M,
                           int64_t K, uint16_t* y, int8_t* gq, float* gs, int8_t* uq, float* us, hipStream_t stream) {
  if (relu2) gate_fwd<ActRelu2>(gate, ldg, up, ldu, M, K, y, gq, gs, uq, us, stream);
  else gate_fwd<ActSilu>(gate, ldg, up, ldu, M, K, y, gq, gs, uq, us, stream);
  return hipGetLastError();
}

template <class A>
static void gate_bwd(const uint16_t* dY, const uint16_t* gate, int64_t ldg, const uint16_t* up, int64_t ldu,
                     const int8_t* gq, const float* gs, const int8_t* uq, const float* us, int64_t M, int64_t K,
                     uint16_t* dgate, int64_t lddg, uint16_t* dup, int64_t lddu, hipStream_t st) {
  const int nch = (int)(ckpt_pad(K) / 8);
  const uint32_t total = (uint32_t)(M * nch);
  const unsigned grid = row_grid(total);
  const int k = (int)K;
  if (dup && gq) gate_bwd_kernel<A, true, true><<<grid, kRowThreads, 0, st>>>(dY, gate, ldg, up, ldu, gq, gs, uq, us, total, k, nch, dgate, lddg, dup, lddu);
  else if (dup) gate_bwd_kernel<A, false, true><<<grid, kRowThreads, 0, st>>>(dY, gate, ldg, up, ldu, gq, gs, uq, us, total, k, nch, dgate, lddg, dup, lddu);
  else if (gq) gate_bwd_kernel<A, true, false><<<grid, kRowThreads, 0, st>>>(dY, gate, ldg, up, ldu, gq, gs, uq, us, total, k, nch, dgate, lddg, dup, lddu);
  else gate_bwd_kernel<A, false, false><<<grid, kRowThreads, 0, st>>>(dY, gate, ldg, up, ldu, gq, gs, uq, us, total, k, nch, dgate, lddg, dup, lddu);
}

hipError_t launch_gate_bwd(bool relu2, const uint16_t* dY, const uint16_t* gate, int64_t ldg, const uint16_t* up,
                           int64_t ldu, const int8_t* gq, const float* gs, const int8_t* uq, const float* us,
                           int64_t M, int64_t K, uint16_t* dgate, int64_t lddg, uint16_t* dup, int64_t lddu,
                           hipStream_t stream) {
  if (relu2) gate_bwd<ActRelu2>(dY, gate, ldg, up, ldu, gq, gs, uq, us, M, K, dgate, lddg, dup, lddu, stream);
  else gate_bwd<ActSilu>(dY, gate, ldg, up, ldu, gq, gs, uq, us, M, K, dgate, lddg, dup, lddu, stream);
  return hipGetLastError();
}

}  // namespace bitnet
