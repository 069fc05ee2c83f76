/*
 * bitnet.h - C ABI of the MI355X (gfx950) BitLinear library, libbitnet.so.
 *
 * One BitNet b1.58 linear layer with ternary weights and int8 activations
 * (W1.58 / A8), for quantization-aware training: the weight ternarization
 * and 2-bit packing, the per-token int8 activation quantization, the INT8
 * forward GEMM and the straight-through-estimator (STE) backward GEMMs.
 * A TTQ variant (learned threshold and asymmetric scales, bf16 activations)
 * is declared at the end. The BitNet operations are those of the
 * "bitnet-qat-train" page (Hugging Face
 * kernels, phanerozoic): its opening bullets and its "Semantics" section,
 * with the quantizers of "bitlinear.py" (h4-polytopic-attention:
 * ternary_quantize, activation_quant_int8) and "1BitTraining.md" (Codys12
 * gist: weight_quant, activation_quant).
 *
 * Conventions for every entry point:
 *  - Tensors are dense and row-major. bf16 data is passed as its raw 16-bit
 *    patterns (uint16_t). Every array pointer is a DEVICE pointer and must be
 *    16-byte aligned, except `gamma` (4-byte aligned).
 *  - `stream` is a hipStream_t passed as void* (NULL = the default stream).
 *    Work is enqueued on it asynchronously; nothing synchronizes the host.
 *  - The caller owns every buffer (inputs, outputs, workspace) and keeps it
 *    alive until the stream work completes. The library allocates no device
 *    memory and keeps no pointer after it returns.
 *  - Arguments are validated before any launch; a validation failure returns
 *    its code and enqueues nothing. A failed launch returns BITNET_ERR_HIP.
 *  - Sizes are int64_t and must be >= 1 (M, N, K). Any K is accepted: the
 *    reduction axis of the int8 and 2-bit state is padded to
 *    Kp = bitnet_k_pad(K) (a multiple of 64) with zero codes and values;
 *    reductions and scales use the true K only.
 *  - Non-finite inputs (inf, NaN) give unspecified results.
 *  - Size limits (BITNET_ERR_SHAPE beyond them): M, N <= 2^30, K <= 2^24;
 *    for the GEMM entry points every operand the call reads among x_q,
 *    w_packed and dY satisfies (rows + 256) * row_bytes <= 2^31, i.e.
 *    (M + 256) * Kp, (N + 256) * Kp/4 and (M + 256) * 2N bytes, and with dW
 *    also (M + 256) * 2Kp for its bf16 x_hat, with dX also (Kp + 256) * Np/2
 *    for its fp4 transposed codes (Np = N rounded up to 64) (the kernels
 *    address them with 32-bit offsets); the forward also needs N <= 2^24
 *    (its epilogue addresses 32 output rows of up to 4-byte elements the
 *    same way).
 */
#ifndef BITNET_H
#define BITNET_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    BITNET_OK = 0,
    BITNET_ERR_NULL = 1,      /* a required pointer is NULL */
    BITNET_ERR_SHAPE = 2,     /* a size is < 1 or too large */
    BITNET_ERR_DTYPE = 3,     /* unsupported dtype enum */
    BITNET_ERR_ALIGN = 4,     /* a pointer is not aligned as required */
    BITNET_ERR_WORKSPACE = 5, /* workspace NULL or smaller than required */
    BITNET_ERR_HIP = 6        /* the HIP runtime reported an error */
} bitnet_status;

typedef enum {
    BITNET_BF16 = 0,
    BITNET_F32 = 1,
    BITNET_SIGN1 = 2  /* bitlinear_bwd's dW only: 1-bit signs (see there) */
} bitnet_dtype;

/* Human-readable name of a status code (static storage). */
const char* bitnet_status_string(bitnet_status status);

/* Padded reduction length: K rounded up to a multiple of 64 (K >= 1). */
int64_t bitnet_k_pad(int64_t K);

/* Bytes of workspace bitnet_ternarize_pack needs (fixed, a few KiB). */
size_t bitnet_ternarize_workspace_bytes(int64_t N, int64_t K);

/* Bytes of workspace bitlinear_fwd / bitlinear_bwd need for these sizes
 * (0 for sizes the call rejects). 0 means the call takes no workspace (the
 * pointer may then be NULL). The size is that of the plan the call runs on
 * the current device: a GEMM needs workspace when it splits output tiles
 * over several workgroups so that all CUs stay busy (16 bytes of tagged
 * counters per 256 x 256 output tile and 256 KiB per partial tile, at most
 * min(2G, G + T - 1) of them for G workgroups and T tiles); few tokens
 * (M <= 64) need none for the forward. The contents need no
 * initialization, and the calls leave the counters cleared, so a call
 * captured into a HIP graph may be replayed any number of times; a
 * workspace must not be shared by calls that may run at the same time
 * (calls on one stream may share it). bitlinear_bwd's size is that of its
 * call with both outputs; a call with one output uses the same size (its
 * split then uses fewer workgroups if it must). Each product first builds a
 * transient operand at the start of the workspace: dX the ternary codes
 * transposed to fp4 [Kp][Np/2] (Kp*Np/2 bytes, Np = N rounded up to 64), dW
 * a bf16 x_hat = bf16(x_q * s/127) [M][Kp] (2*M*Kp bytes); a call with
 * both outputs builds both, one after the other, in one launch. For at most
 * 64 tokens a bf16 or f32 dW converts its slices of x_hat itself and needs
 * no workspace, and a call with both outputs builds only the fp4 codes, in
 * the launch that also computes dW. */
size_t bitlinear_fwd_workspace_bytes(int64_t M, int64_t N, int64_t K);
size_t bitlinear_bwd_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * bitnet_ternarize_pack - per-tensor absmean scale, RoundClip ternarization
 * and 2-bit packing of the master weight ("bitnet-qat-train", opening
 * bullets: one fused ternarize, scale and pack pass; "bitlinear.py",
 * ternary_quantize; "1BitTraining.md", weight_quant). For bf16 W with K a
 * multiple of 64 and N*K up to about 25 M, W is read once: one launch holds
 * it in registers while its workgroups exchange their partial sums through
 * the workspace, then writes the codes. Otherwise a reduction pass over W
 * and a fused ternarize + pack pass. Both give the same bits.
 *
 *   gamma = max(fp32(S / (N*K)), 1e-8f), S = sum |W| accumulated in fp64 in
 *           a fixed order (bitwise deterministic across calls);
 *   q[n,k] = clip(round_half_even(W[n,k] / gamma), -1, 1), evaluated exactly
 *           (equivalently q = sign(w) if |w| > gamma/2, else 0).
 *
 * W         [N][K] master weights, bf16 bits (w_dtype BITNET_BF16) or float
 *           (BITNET_F32).
 * w_packed  [N][Kp/4] output bytes: row n holds Kp/16 little-endian 32-bit
 *           words of 16 codes; word w holds k = 16w..16w+15, the code of
 *           k = 16w + j at bit 8*(j%4) + 2*(j/4), as a 2-bit two's complement
 *           value: +1 = 0b01, 0 = 0b00, -1 = 0b11 (0b10 is never written).
 *           Padding codes (k >= K) are 0. (Byte b of a word holds the codes
 *           j = b, b+4, b+8, b+12, so (word >> 2t) & 0x03030303 gives the
 *           codes of k = 16w+4t..16w+4t+3 in its four bytes.)
 * gamma     [1] output float (device).
 * workspace device scratch of at least bitnet_ternarize_workspace_bytes();
 *           no initialization needed (the words that publish partial sums
 *           between workgroups carry a per-launch tag and sequence, so
 *           whatever the memory held never matches); clobbered. Calls that
 *           may run at the same time must not share a workspace.
 */
bitnet_status bitnet_ternarize_pack(const void* W, bitnet_dtype w_dtype,
                                    int64_t N, int64_t K,
                                    uint8_t* w_packed, float* gamma,
                                    void* workspace, size_t workspace_bytes,
                                    void* stream);

/*
 * bitnet_quantize - bitnet_ternarize_pack and bitnet_act_quant of one layer
 * step in one call, with the same results bit for bit (gamma, w_packed,
 * x_q, s_x). The activation rows are quantized in the weight's launch: in
 * the one-pass case each workgroup quantizes its share of the rows while
 * the others' partial sums arrive; otherwise the absmean pass and the rows
 * share one launch (two independent streams over W and x) and the codes are
 * packed after it. The two inputs share the reduction length K: W [N][K], x
 * [M][K]. Arguments, layouts and errors are those of the two calls;
 * workspace as bitnet_ternarize_pack's.
 */
bitnet_status bitnet_quantize(const void* W, bitnet_dtype w_dtype, int64_t N, int64_t K,
                              const uint16_t* x, int64_t M,
                              uint8_t* w_packed, float* gamma, int8_t* x_q, float* s_x,
                              void* workspace, size_t workspace_bytes, void* stream);

/*
 * bitnet_quantize_static - bitnet_quantize for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation): no workspace argument; the scratch
 * (the weight absmean's fp64 partial sums, and the one-pass launch's
 * per-workgroup records of partial and publication word) lives in a device
 * array of the library, 8192 bytes per GPU the library runs on, held until
 * the process ends. Results are bit for bit those of bitnet_quantize. The
 * array keeps the last call's contents; no call needs it cleared (partials
 * are written before they are read; publication words are tagged per launch
 * and never match a later launch's), but calls that may run at the same
 * time on one GPU race on it. Returns BITNET_ERR_WORKSPACE if a call would need more scratch
 * than the array holds (not the case for any size: the need is fixed at
 * bitnet_ternarize_workspace_bytes()), BITNET_ERR_HIP if the array's device
 * address cannot be obtained; otherwise the arguments and errors of
 * bitnet_quantize. Calls no allocating routine.
 */
bitnet_status bitnet_quantize_static(const void* W, bitnet_dtype w_dtype, int64_t N, int64_t K,
                                     const uint16_t* x, int64_t M,
                                     uint8_t* w_packed, float* gamma, int8_t* x_q, float* s_x,
                                     void* stream);

/*
 * bitnet_quantize2 - bitnet_ternarize_pack of two weights of one size and
 * type, for a layer that puts both to one input: the codes [2 N][Kp/4] of W0
 * and below them those of W1, gamma[0] and gamma[1], each bit for bit what
 * that call alone gives. x may be NULL (M, x_q and s_x are not used then);
 * otherwise its M rows become x_q and s_x as bitnet_rows_quant makes them, in
 * the weights' launch. Errors and limits as those calls' (with x M <= 2^23 and
 * K <= 2^24); workspace as bitnet_ternarize_pack's.
 */
bitnet_status bitnet_quantize2(const void* W0, const void* W1, bitnet_dtype w_dtype, int64_t N, int64_t K,
                               const uint16_t* x, int64_t M, uint8_t* w_packed, float* gamma,
                               int8_t* x_q, float* s_x, void* workspace, size_t workspace_bytes, void* stream);

/*
 * bitnet_code_counts - how many weights each ternary value takes, for the
 * share of -1, 0 and +1 ("bitlinear.py", BitLinear.ternary_stats):
 *
 *   counts[0] = #{(n, k) : q[n,k] = -1},  counts[1] = #{(n, k) : q[n,k] = +1}
 *
 * over the true N x K weights (padding codes are 0 and count for neither;
 * the zeros are N*K - counts[0] - counts[1]).
 *
 * w_packed  [N][Kp/4] codes as written by bitnet_ternarize_pack (16-byte
 *           aligned).
 * counts    [2] uint64 output (device, 8-byte aligned).
 * No workspace. Exact and repeatable (a fixed summation order).
 */
bitnet_status bitnet_code_counts(const uint8_t* w_packed, int64_t N, int64_t K,
                                 uint64_t* counts, void* stream);

/*
 * bitnet_act_quant - per-token absmax int8 quantization ("bitlinear.py",
 * activation_quant_int8; "1BitTraining.md", activation_quant;
 * "bitnet-qat-train", opening paragraph).
 *
 *   s[m]      = max(max_k |x[m,k]|, 1e-8f)             (the row absmax)
 *   x_q[m,k]  = clip(round_half_even(127 * x[m,k] / s[m]), -127, 127),
 *               evaluated exactly.
 *
 * x    [M][K] bf16 bits.
 * x_q  [M][Kp] int8 output; columns K..Kp-1 are written as 0.
 * s_x  [M] float output: the floored absmax. The dequantization scale is
 *      s_x/127; it is applied where the int8 values are used.
 */
bitnet_status bitnet_act_quant(const uint16_t* x, int64_t M, int64_t K,
                               int8_t* x_q, float* s_x, void* stream);

/*
 * bitlinear_fwd - INT8 forward GEMM with exact INT32 accumulation and a
 * fused rescale ("bitnet-qat-train", Semantics):
 *
 *   acc[m,n] = sum_{k<Kp} x_q[m,k] * q[n,k]        (int32, exact)
 *   y[m,n]   = bf16_rne(acc[m,n] * (s_x[m]/127) * gamma)   (fp32 rescale)
 *
 * x_q, s_x  as written by bitnet_act_quant (x_q [M][Kp]).
 * w_packed, gamma as written by bitnet_ternarize_pack (w_packed [N][Kp/4]).
 * y        [M][N] bf16 bits output.
 * acc_out  [M][N] int32 output of the raw accumulators, or NULL (the
 *          production setting; it exists for bit-exact checks).
 * K        the true reduction length (Kp = bitnet_k_pad(K)).
 * workspace device scratch of bitlinear_fwd_workspace_bytes(M, N, K) bytes
 *          (NULL allowed when that is 0); clobbered.
 */
bitnet_status bitlinear_fwd(const int8_t* x_q, const float* s_x,
                            const uint8_t* w_packed, const float* gamma,
                            int64_t M, int64_t N, int64_t K,
                            uint16_t* y, int32_t* acc_out,
                            void* workspace, size_t workspace_bytes,
                            void* stream);

/*
 * bitlinear_fwd_bias - bitlinear_fwd with a bias added before the rounding
 * ("bitlinear.py", BitLinear: an optional bias, zero-initialised, added after
 * the product):
 *
 *   y[m,n] = bf16_rne(fp32(acc[m,n] * (s_x[m]/127) * gamma) + bias[n])
 *
 * (the product as in bitlinear_fwd, one fp32 add, one rounding). bias is
 * [N] bf16 bits, 16-byte aligned, or NULL (then identical to
 * bitlinear_fwd). Other arguments, the workspace and the errors are those
 * of bitlinear_fwd.
 */
bitnet_status bitlinear_fwd_bias(const int8_t* x_q, const float* s_x,
                                 const uint8_t* w_packed, const float* gamma,
                                 const uint16_t* bias,
                                 int64_t M, int64_t N, int64_t K,
                                 uint16_t* y, int32_t* acc_out,
                                 void* workspace, size_t workspace_bytes,
                                 void* stream);

/*
 * bitlinear_bias_grad - gradient of that bias: db[n] = sum_m dY[m,n], the
 * products of nothing but the bf16 values, summed in fp32 in a fixed order
 * (bitwise deterministic across calls) and rounded once to db_dtype.
 *
 * dY  [M][N] bf16 bits (16-byte aligned).
 * db  [N] output, BITNET_F32 or BITNET_BF16 bits (16-byte aligned).
 * No workspace.
 */
bitnet_status bitlinear_bias_grad(const uint16_t* dY, int64_t M, int64_t N,
                                  void* db, bitnet_dtype db_dtype, void* stream);

/*
 * bitlinear_bwd - straight-through-estimator backward with the operands
 * rebuilt from the saved 2-bit and int8 state ("bitnet-qat-train",
 * Semantics and opening bullets; gamma is treated as a constant):
 *
 *   dX[m,k] = sum_n dY[m,n] * W_hat[n,k],  W_hat = q * bf16_rne(gamma)
 *   dW[n,k] = sum_m dY[m,n] * x_hat[m,k],  x_hat = bf16_rne(x_q * s_x/127)
 *
 * Products are exact in fp32 (bf16 x bf16); sums accumulate in fp32; the
 * results are rounded once to the output dtype.
 *
 * dY        [M][N] bf16 bits.
 * x_q, s_x  saved activation state (x_q [M][Kp]); may be NULL if dW is NULL.
 * w_packed, gamma saved weight state; may be NULL if dX is NULL.
 * dX        [M][K] bf16 bits output, or NULL to skip the dX GEMM.
 * dW        [N][K] output in dW_dtype (BITNET_BF16 bits or BITNET_F32), or
 *           NULL to skip the dW GEMM. At least one of dX, dW is non-NULL.
 *           With BITNET_SIGN1, dW is [N][Kp/8] bytes of 1-bit signs for a
 *           sign-based optimiser ("1BitTraining.md", closing paragraphs: the
 *           identity-STE gradient has the sign of the gradient with respect
 *           to the quantised weight, so only 1 bit per weight is needed):
 *           bit j of byte b of row n is 1 iff the fp32 sum for dW[n, 8b + j]
 *           is negative, 0 otherwise (zero sums included); bits of k >= K
 *           are 0. No bf16 or f32 dW is written.
 * workspace device scratch of bitlinear_bwd_workspace_bytes(M, N, K) bytes
 *           (NULL allowed when that is 0); clobbered.
 */
bitnet_status bitlinear_bwd(const uint16_t* dY,
                            const int8_t* x_q, const float* s_x,
                            const uint8_t* w_packed, const float* gamma,
                            int64_t M, int64_t N, int64_t K,
                            uint16_t* dX, void* dW, bitnet_dtype dW_dtype,
                            void* workspace, size_t workspace_bytes,
                            void* stream);

/*
 * TTQ: trained ternary quantization ("TTQ_VERIFICATION.md", LabStrangeLoop
 * bitnet, summarising Zhu et al.), the variant with a learned threshold and
 * two learned scales per layer. params is a device float[3] =
 * {delta, Wp, Wn} (positive values; a caller that learns them through a
 * positivity transform passes the transformed values). Activations are the
 * layer's bf16 inputs, unquantized ("Bugs Fixed", item 4); the products run
 * on bf16 operands with fp32 accumulation. The quantized weight is kept as
 * its 2-bit codes (the w_packed format above) and as bf16 values
 * wt [N][Kp] = bf16(Wp), -bf16(Wn) or 0 (round half to even; padding 0).
 */

/* Bytes of workspace ttq_fwd and ttq_bwd need for these sizes (0 for sizes
 * they reject): the split-tile workspace of their GEMMs, as for
 * bitlinear_fwd, and for ttq_bwd 8 bytes per 128 x 128 tile of dW for the
 * scale-gradient partial sums. No initialization needed; graph replays are
 * safe; not shared by calls that may run at the same time. */
size_t ttq_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * ttq_init - the initial parameters (Algorithm Summary, Initialization,
 * Eq. 2): E = mean |W| computed exactly as bitnet_ternarize_pack's gamma
 * (the same bits, floor 1e-8 included), delta = fl32(0.7f * E) (one fp32
 * multiplication), Wp = Wn = E.
 *
 * W       [N][K] bf16 bits or float (w_dtype), 16-byte aligned.
 * params  [3] output float (device, 4-byte aligned).
 * workspace at least bitnet_ternarize_workspace_bytes(N, K); clobbered.
 */
bitnet_status ttq_init(const void* W, bitnet_dtype w_dtype, int64_t N, int64_t K,
                       float* params, void* workspace, size_t workspace_bytes,
                       void* stream);

/*
 * ttq_quantize - Eq. 1 in one pass over W: code +1 where W > delta, -1
 * where W < -delta, 0 elsewhere (strict, exact comparisons).
 *
 * W         [N][K] bf16 bits or float (w_dtype).
 * params    [3] float (device): delta, Wp, Wn.
 * w_packed  [N][Kp/4] output codes (the bitnet_ternarize_pack format).
 * wt        [N][Kp] output bf16 bits: bf16(Wp), -bf16(Wn) or 0.
 * No workspace.
 */
bitnet_status ttq_quantize(const void* W, bitnet_dtype w_dtype, int64_t N, int64_t K,
                           const float* params, uint8_t* w_packed, uint16_t* wt,
                           void* stream);

/*
 * ttq_fwd - y[m,n] = sum_k x[m,k] * wt[n,k] (Eq. 1's weight applied to the
 * unquantized activations), fp32 sums rounded once to bf16.
 *
 * x   [M][K] bf16 bits.  wt [N][Kp] from ttq_quantize.  y [M][N] bf16 bits.
 * workspace ttq_workspace_bytes(M, N, K) bytes (NULL when that is 0).
 * Limits as for the GEMMs above, with (M + 256) * 2K and (N + 256) * 2Kp
 * bytes for x and wt.
 */
bitnet_status ttq_fwd(const uint16_t* x, const uint16_t* wt, int64_t M, int64_t N, int64_t K,
                      uint16_t* y, void* workspace, size_t workspace_bytes, void* stream);

/*
 * ttq_fwd_codes - the same forward from the stored state (the codes and
 * params, e.g. an exported layer): y[m,n] = sum_k x[m,k] * v(q[n,k]), with
 * v(+1) = bf16(Wp), v(-1) = -bf16(Wn), v(0) = 0, fp32 sums rounded once to
 * bf16. For few tokens (M <= 64, K % 8 == 0) one kernel reads the 2-bit
 * codes once and expands them in registers; otherwise the codes are
 * expanded to wt in the workspace and ttq_fwd's GEMM runs on it (the same
 * bits as ttq_fwd on ttq_quantize's wt).
 *
 * x         [M][K] bf16 bits.  w_packed [N][Kp/4] codes.  params [3] float
 *           (device, 4-byte aligned): delta (unused here), Wp, Wn.
 * y         [M][N] bf16 bits.
 * workspace ttq_fwd_codes_workspace_bytes(M, N, K) bytes: 0 (NULL allowed)
 *           when the few-token kernel applies, else 2*N*Kp for the expanded
 *           weight plus the GEMM's share; clobbered.
 * Limits as for ttq_fwd, and (N + 256) * Kp/4 bytes of codes.
 */
size_t ttq_fwd_codes_workspace_bytes(int64_t M, int64_t N, int64_t K);
bitnet_status ttq_fwd_codes(const uint16_t* x, const uint8_t* w_packed, const float* params,
                            int64_t M, int64_t N, int64_t K, uint16_t* y,
                            void* workspace, size_t workspace_bytes, void* stream);

/*
 * ttq_bwd - the straight-through backward (Algorithm Summary, Backward
 * Pass; "Bugs Fixed", item 5):
 *
 *   dX[m,k] = sum_n dY[m,n] * wt[n,k]
 *   dW[n,k] = sum_m dY[m,n] * x[m,k]   (the latent weight's gradient is
 *                                       the quantized weight's, unchanged)
 *   grads[0] = dL/dWp =   sum of dW[n,k] over the codes +1
 *   grads[1] = dL/dWn = - sum of dW[n,k] over the codes -1
 *
 * The masked sums take the fp32 dW values before rounding, add them per
 * 128 x 128 tile in fp32 and across tiles in fp64, in a fixed order
 * (bitwise deterministic across calls), rounded once to fp32. delta gets no
 * gradient (the hard threshold has none).
 *
 * dY  [M][N] bf16 bits.  x [M][K] bf16 bits (needed for dW).
 * wt  from ttq_quantize (needed for dX); w_packed its codes (needed for
 *     grads).
 * dX  [M][K] bf16 bits output, or NULL.
 * dW  [N][K] output in dW_dtype (BITNET_BF16 or BITNET_F32), or NULL.
 * grads [2] float output (device, 4-byte aligned), or NULL; needs dW.
 * At least one of dX, dW is non-NULL.
 * workspace ttq_workspace_bytes(M, N, K) bytes; clobbered.
 */
bitnet_status ttq_bwd(const uint16_t* dY, const uint16_t* x, const uint16_t* wt,
                      const uint8_t* w_packed, int64_t M, int64_t N, int64_t K,
                      uint16_t* dX, void* dW, bitnet_dtype dW_dtype, float* grads,
                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * Layer norm over rows of K values (the norm that stands before a BitLinear),
 * forward and backward:
 *
 *   mu[m]   = sum_k x[m,k] / K
 *   r[m]    = (sum_k (x[m,k] - mu[m])^2 / K + eps)^(-1/2)
 *   xh[m,k] = (x[m,k] - mu[m]) * r[m]
 *   y[m,k]  = xh[m,k] * w[k] + b[k]
 *
 *   g[m,k]  = dY[m,k] * w[k]
 *   dX[m,k] = r[m] * (g[m,k] - sum_j g[m,j] / K - xh[m,k] * sum_j g[m,j] xh[m,j] / K)
 *   dw[k]   = sum_m dY[m,k] * xh[m,k],   db[k] = sum_m dY[m,k]
 *
 * Statistics and sums are fp32, each output is rounded once. Sums run in a
 * fixed order (bitwise deterministic across calls). NaN and infinities
 * propagate within their row (and into dw, db). K <= 32768.
 *
 * x, dX     [M][K] in x_dtype (BITNET_BF16 bits or BITNET_F32).
 * w, b      [K] in p_dtype (BITNET_BF16 or BITNET_F32), or NULL (1 and 0).
 * y, dY     [M][K] in y_dtype (BITNET_BF16 or BITNET_F32).
 * mean, rstd [M] float: mu and r, written by the forward (NULL: not
 *           written) and read by the backward.
 * codes, scales  the 8-bit checkpoint of x (bitnet_ckpt_pack's layout; x is
 *           the input, not xh). The forward writes both if codes is not NULL;
 *           the backward given codes reads them instead of x (x may then be
 *           NULL; x_dtype still names dX's type), with mu and r of the
 *           uncoded row.
 * dX, dw, db  each NULL if not wanted, at least one not (dw, db in p_dtype).
 * Data pointers need only their element's alignment; codes and the workspace
 * 16 bytes.
 * workspace of the backward: bitnet_layernorm_workspace_bytes(M, K) bytes
 * (0 for sizes it rejects; NULL allowed when neither dw nor db is wanted);
 * no initialization, not shared by calls that may run at the same time.
 */
size_t bitnet_layernorm_workspace_bytes(int64_t M, int64_t K);
bitnet_status bitnet_layernorm_fwd(const void* x, bitnet_dtype x_dtype, const void* w, const void* b,
                                   bitnet_dtype p_dtype, int64_t M, int64_t K, float eps, void* y,
                                   bitnet_dtype y_dtype, float* mean, float* rstd, int8_t* codes, float* scales,
                                   void* stream);
bitnet_status bitnet_layernorm_bwd(const void* dY, bitnet_dtype y_dtype, const void* x, bitnet_dtype x_dtype,
                                   const int8_t* codes, const float* scales, const void* w, bitnet_dtype p_dtype,
                                   const float* mean, const float* rstd, int64_t M, int64_t K, void* dX, void* dw,
                                   void* db, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Activations kept in 8 bits between the forward and the backward pass
 * (1.03 bytes a value instead of 2 or 4). Each 128 consecutive values of a
 * row share a scale:
 *
 *   s[m,j] = max |x[m,k]| over k = 128j .. 128j + 127 (k < K)
 *   q[m,k] = clip(round_half_even(127 * x[m,k] / s[m,j]), -127, 127),
 *            evaluated exactly (0 where s = 0)
 *
 * and q stands for fp32(q * fp32(s / 127)). A block that holds an infinity or
 * a NaN stands for NaN throughout.
 *
 * x       [M][K] in x_dtype (BITNET_BF16 bits or BITNET_F32), element
 *         aligned; unpack rounds once to x_dtype.
 * codes   [M][Kc] int8, Kc = bitnet_ckpt_pad(K) (K rounded up to 128), 16-byte
 *         aligned; columns K..Kc-1 are written as 0 and not read back.
 * scales  [M][Kc/128] float, 4-byte aligned.
 * M * Kc <= 2^34, K <= 2^24. No workspace.
 */
int64_t bitnet_ckpt_pad(int64_t K);
bitnet_status bitnet_ckpt_pack(const void* x, bitnet_dtype x_dtype, int64_t M, int64_t K, int8_t* codes,
                               float* scales, void* stream);
bitnet_status bitnet_ckpt_unpack(const int8_t* codes, const float* scales, int64_t M, int64_t K, void* x,
                                 bitnet_dtype x_dtype, void* stream);

/*
 * The gated activation of a feed-forward block, y = act(gate) * up, or
 * y = act(gate) without up, and its gradients
 *
 *   dgate = dY * up * act'(gate),   dup = dY * act(gate)
 *
 * BITNET_ACT_SILU: act(g) = g / (1 + e^-g).
 * BITNET_ACT_RELU2: act(g) = max(g, 0)^2.
 * fp32 arithmetic, each output rounded once to bf16.
 *
 * gate, up    [M] rows of K bf16, ldg and ldu elements apart (>= K), 2-byte
 *             aligned: they may be the halves of one [M][2K] tensor. up NULL:
 *             no gate (then dup, up_codes, up_scales are NULL too).
 * y, dY       [M][K] bf16.
 * gate_codes, gate_scales, up_codes, up_scales  8-bit checkpoints
 *             (bitnet_ckpt_pack's layout). The forward writes them if
 *             gate_codes is not NULL; the backward given gate_codes reads
 *             them instead of gate and up.
 * dgate, dup  [M] rows of K bf16, lddg and lddu elements apart (>= K).
 * Sizes as for bitnet_ckpt_pack. No workspace.
 */
typedef enum { BITNET_ACT_SILU = 0, BITNET_ACT_RELU2 = 1 } bitnet_act;
bitnet_status bitnet_gate_fwd(bitnet_act act, const uint16_t* gate, int64_t ldg, const uint16_t* up, int64_t ldu,
                              int64_t M, int64_t K, uint16_t* y, int8_t* gate_codes, float* gate_scales,
                              int8_t* up_codes, float* up_scales, void* stream);
bitnet_status bitnet_gate_bwd(bitnet_act act, const uint16_t* dY, const uint16_t* gate, int64_t ldg,
                              const uint16_t* up, int64_t ldu, const int8_t* gate_codes, const float* gate_scales,
                              const int8_t* up_codes, const float* up_scales, int64_t M, int64_t K,
                              uint16_t* dgate, int64_t lddg, uint16_t* dup, int64_t lddu, void* stream);

/*
 * TTQ with x kept as its 8-bit checkpoint: ttq_fwd that also writes the codes
 * and scales of x [M][K] (bitnet_ckpt_pack's; codes NULL: not written), and
 * ttq_bwd that reads them: the values, rounded to bf16, take x's place in
 * dW = dY^T x. With dW NULL, codes and scales may be NULL. Widths that are not
 * multiples of 8 are copied to padded rows in the workspace (x forward, dY
 * backward), with the same results. workspace:
 * ttq_fwd_ckpt_workspace_bytes / ttq_bwd_ckpt_workspace_bytes; the other
 * arguments and the errors are ttq_fwd's and ttq_bwd's, the limits too, with K
 * and N rounded up to 64.
 */
size_t ttq_fwd_ckpt_workspace_bytes(int64_t M, int64_t N, int64_t K);
bitnet_status ttq_fwd_ckpt(const uint16_t* x, const uint16_t* wt, int64_t M, int64_t N, int64_t K, uint16_t* y,
                           int8_t* codes, float* scales, void* workspace, size_t workspace_bytes, void* stream);
size_t ttq_bwd_ckpt_workspace_bytes(int64_t M, int64_t N, int64_t K);
bitnet_status ttq_bwd_ckpt(const uint16_t* dY, const int8_t* codes, const float* scales, const uint16_t* wt,
                           const uint8_t* w_packed, int64_t M, int64_t N, int64_t K, uint16_t* dX, void* dW,
                           bitnet_dtype dW_dtype, float* grads, void* workspace, size_t workspace_bytes,
                           void* stream);

/*
 * A linear layer with softmax cross entropy over a large vocabulary (the head
 * and the loss of a language model), in pieces of the vocabulary, without
 * keeping the logits:
 *
 *   z[t,v]  = sum_d h[t,d] * w[v,d]
 *   lse[t]  = log sum_v exp z[t,v]
 *   loss[t] = lse[t] - z[t,target[t]]    (0 where target[t] == ignore_index),
 *             taken as (m - z[t,target[t]]) + log sum_v exp(z[t,v] - m) with m the
 *             largest logit: 0 for a target that is all of the sum
 *   total   = sum_t loss[t], or the mean over the rows that count (0 if none)
 *
 *   G[t,v]  = c[t] * (exp(z[t,v] - lse[t]) - [v == target[t]])
 *   dh[t,d] = sum_v G[t,v] * w[v,d],     dw[v,d] = sum_t G[t,v] * h[t,d]
 *
 * with c[t] the gradient of whatever is minimised with respect to loss[t]:
 * dloss[t] (BITNET_REDUCE_NONE), *dloss (SUM), or *dloss divided by the
 * number of rows that count (MEAN); 0 for ignored rows. Products are exact in
 * fp32 and sums are fp32; G is rounded to bf16 between the products (a
 * rounding of 2^-9 of each value, as the outputs'); the logits are never
 * written. All sums run in a fixed order (bitwise deterministic). What an
 * ignored row of h holds reaches nothing. A target outside 0..V-1 that is not
 * ignore_index makes its row's loss, and gradients that it takes part in, NaN.
 *
 * h, dh    [T][D] bf16 bits.   w [V][D] bf16 bits.   targets [T] int64.
 * loss, lse [T] float, written by the forward; lse is read by the backward.
 * total    [1] float, or NULL.
 * dw       [V][D] in dw_dtype (BITNET_BF16 or BITNET_F32). dh or dw may be
 *          NULL (not computed), not both.
 * Alignment: h, w, dh, dw and the workspace 16 bytes, targets 8, the rest 4.
 * workspace: bitnet_xent_fwd_workspace_bytes / bitnet_xent_bwd_workspace_bytes
 * (0 for sizes the call rejects); no initialization, not shared by calls that
 * may run at the same time. The backward's holds G for one piece of the
 * vocabulary (128 MiB at most, or 256 columns) and fp32 sums of dh.
 * Limits: T <= 2^21, V <= 2^28, D <= 65536, (T + 256) * 2 * (D rounded up to
 * 8) <= 2^31. Widths D that are multiples of 8 are fastest (others copy h,
 * and w a piece at a time, to padded rows first, but for the loss of few
 * tokens).
 */
typedef enum { BITNET_REDUCE_NONE = 0, BITNET_REDUCE_SUM = 1, BITNET_REDUCE_MEAN = 2 } bitnet_reduce;
size_t bitnet_xent_fwd_workspace_bytes(int64_t T, int64_t V, int64_t D);
size_t bitnet_xent_bwd_workspace_bytes(int64_t T, int64_t V, int64_t D);
bitnet_status bitnet_xent_fwd(const uint16_t* h, const uint16_t* w, const int64_t* targets, int64_t ignore_index,
                              int64_t T, int64_t V, int64_t D, float* loss, float* lse, float* total,
                              bitnet_reduce reduce, void* workspace, size_t workspace_bytes, void* stream);
bitnet_status bitnet_xent_bwd(const uint16_t* h, const uint16_t* w, const int64_t* targets, int64_t ignore_index,
                              const float* lse, const float* dloss, bitnet_reduce reduce, int64_t T, int64_t V,
                              int64_t D, uint16_t* dh, void* dw, bitnet_dtype dw_dtype, void* workspace,
                              size_t workspace_bytes, void* stream);

/*
 * Root-mean-square norm over rows of K values, with the residual's addition
 * before it and an output in 8 bits with a scale a row (what bitnet_act_quant
 * makes of bf16 rows, here from the norm's fp32 values):
 *
 *   h[m,k] = round(res[m,k] + x[m,k]) in the stream's type, or x without res
 *   r[m]   = (sum_k h[m,k]^2 / K + eps)^(-1/2),  v[m,k] = h[m,k] * r[m] * w[k]
 *   y[m,k] = round(v[m,k]),  or
 *   s[m]   = max(max_k |v[m,k]|, 1e-8f),
 *   x_q[m,k] = round_half_even(127 * v[m,k] / s[m]), the quotient taken in fp32 as
 *              h w (127 / max|h w|), the factor rounded up: off by less than 2^-22 of
 *              its value, and right at the exact ties of values of up to 8 bits (half
 *              of the row's largest; half integers where that is 127 * 2^j)
 *
 *   g[m,k]  = dY[m,k] * w[k],  hn[m,k] = h[m,k] * r[m]
 *   dh[m,k] = r[m] * (g[m,k] - hn[m,k] * sum_j g[m,j] hn[m,j] / K) + dH[m,k]
 *   dw[k]   = sum_m dY[m,k] * hn[m,k]
 *
 * dh is the gradient of x and of res alike (straight through the
 * quantization). Statistics and sums are fp32, in a fixed order; squares are
 * summed in fp32, so magnitudes have to stay below about 1e19 / sqrt(K). Each
 * output is rounded once. NaN and infinities propagate within their row (and
 * into dw), and so does a root of no positive number (eps 0 over a row of zeros, eps
 * below 0): a row of 8-bit codes that holds one has s = NaN. K <= 16384.
 *
 * x       [M][K] in x_dtype: with res BITNET_BF16 or the stream's type, without
 *         res the stream's type h_dtype.
 * res, h  [M][K] in h_dtype (BITNET_BF16 or BITNET_F32); both or neither.
 * w       [K] in p_dtype, or NULL (1).
 * y       [M][K] in y_dtype (BITNET_BF16 or BITNET_F32), or NULL: then
 * x_q     [M][Kp] int8 (Kp = bitnet_k_pad(K), columns K..Kp-1 are written as 0)
 * s_x     [M] float.
 * rstd    [M] float: r, written by the forward (NULL: not written), read by the
 *         backward.
 * dY      [M][K] in y_dtype.  dH [M][K] in h_dtype, the gradient of h itself,
 *         or NULL (0).
 * dh      [M][K] in h_dtype, or NULL.  dx [M][K] bf16, the same gradient for a
 *         bf16 x beside a float stream (h_dtype BITNET_F32), or NULL.
 * dw      [K] in p_dtype, or NULL. At least one of dh, dx, dw.
 * Data pointers need only their element's alignment; x_q, s_x and the workspace
 * 16 bytes.
 * workspace of the backward: bitnet_rmsnorm_workspace_bytes(M, K) bytes (0 for
 * sizes it rejects; NULL allowed without dw); no initialization, not shared by
 * calls that may run at the same time.
 */
size_t bitnet_rmsnorm_workspace_bytes(int64_t M, int64_t K);
bitnet_status bitnet_rmsnorm_fwd(const void* x, bitnet_dtype x_dtype, const void* res, bitnet_dtype h_dtype,
                                 const void* w, bitnet_dtype p_dtype, int64_t M, int64_t K, float eps, void* h,
                                 void* y, bitnet_dtype y_dtype, int8_t* x_q, float* s_x, float* rstd, void* stream);
bitnet_status bitnet_rmsnorm_bwd(const void* dY, bitnet_dtype y_dtype, const void* dH, const void* h,
                                 bitnet_dtype h_dtype, const void* w, bitnet_dtype p_dtype, const float* rstd,
                                 int64_t M, int64_t K, void* dh, uint16_t* dx, void* dw, void* workspace,
                                 size_t workspace_bytes, void* stream);

/*
 * 8-bit rows with a scale a row (bitnet_act_quant's layout): made of bf16 or
 * float rows by bitnet_act_quant's arithmetic, and the values they stand for,
 * x[m,k] = bf16_rne(fp32(x_q[m,k] * fp32(s_x[m] / 127))).
 *
 * rows_quant: x [M][K] in x_dtype, element aligned (M <= 2^23, K <= 2^24); x_q [M][Kp],
 *             s_x [M], both 16-byte aligned. A row that holds an infinity or a NaN has
 *             s_x = NaN.
 * rows_quant2: the rows of bf16 x [M][K] and of w [N][K] in w_dtype (a layer's activations
 *             and channels) in one launch; M or N may be 0, M + N < 2^24.
 * rows_unpack: x [M][K] bf16 bits, 2-byte aligned. M * Kp <= 2^34.
 * rows_direct: how many tokens of K values the forwards of the layers below take as
 *             they are, each workgroup making the codes for itself (0: none).
 */
int bitnet_rows_direct(int64_t K);
bitnet_status bitnet_rows_quant(const void* x, bitnet_dtype x_dtype, int64_t M, int64_t K, int8_t* x_q, float* s_x,
                                void* stream);
bitnet_status bitnet_rows_quant2(const uint16_t* x, int64_t M, int8_t* x_q, float* s_x, const void* w,
                                 bitnet_dtype w_dtype, int64_t N, int8_t* w_q, float* s_w, int64_t K, void* stream);
bitnet_status bitnet_rows_unpack(const int8_t* x_q, const float* s_x, int64_t M, int64_t K, uint16_t* x, void* stream);

/*
 * The gated pair of ternary projections of a feed-forward block:
 *
 *   g[m,n] = acc_g * (s_x[m]/127) * gamma[0],  u[m,n] = acc_u * (s_x[m]/127) * gamma[1]
 *   y[m,n] = bf16_rne(act(g[m,n]) * u[m,n])
 *
 * with acc_g and acc_u the exact int32 products of x_q with the codes of the
 * gate (rows 0..N-1 of w_packed) and of the up projection (rows N..2N-1), fp32
 * after them; and its straight-through backward (gamma treated as constants)
 *
 *   Dg = bf16(dY p gamma[0] c),  Du = bf16(dY a gamma[1] c),  c[m] = s_x[m]/127
 *   dX[m,k] = sum_n (Dg[m,n] q_g[n,k] + Du[m,n] q_u[n,k]) / c[m], 0 where |s_x[m]| < 2^-100
 *   dW_gate[n,k] = sum_m Dg[m,n] x_q[m,k] / gamma[0],  dW_up likewise with Du, gamma[1]
 *
 * (dg = dY u act'(g) and du = dY act(g) with the scales of what they are multiplied
 * by, rounded once; fp32 sums, divided in fp32.)
 *
 * x          NULL, or the rows [M][K] as bf16 bits (2-byte aligned, M <=
 *            bitnet_rows_direct(K)): they are quantized on the way as
 *            bitnet_rows_quant does, and x_q and s_x are not used.
 * x_q, s_x   8-bit rows (bitnet_rows_quant, bitnet_rmsnorm_fwd).
 * w_packed   [2N][Kp/4] codes and gamma [2] as bitnet_ternarize_pack writes them
 *            for each weight [N][K].
 * y, dY      [M][N] bf16 bits.
 * slopes     bitnet_gated_slopes_bytes(M, N) bytes: y's derivatives p = u act'(g) and
 *            a = act(g), written by the forward (NULL: not written) and read by the
 *            backward, their fp32 values rounded to 24 bits.
 * dX         [M][K] bf16 bits, or NULL.
 * dW_gate, dW_up [N][K] in dW_dtype (BITNET_BF16 or BITNET_F32), both or neither.
 * The backward without dW takes x_q NULL, and s_x NULL too (c is then 1); without dX
 * w_packed NULL.
 * workspace  bitnet_gated_fwd_workspace_bytes / bitnet_gated_bwd_workspace_bytes
 *            (0 for sizes the call rejects); as for bitlinear_fwd.
 * Pointers 16-byte aligned but gamma, the backward's s_x (4) and dY (2). Limits: those
 * of the GEMM entry points for a weight of 2 Nd rows, (M + 256) * 4 Nd <= 2^31.
 */
size_t bitnet_gated_slopes_bytes(int64_t M, int64_t N);
size_t bitnet_gated_fwd_workspace_bytes(int64_t M, int64_t N, int64_t K);
bitnet_status bitnet_gated_fwd(bitnet_act act, const uint16_t* x, const int8_t* x_q, const float* s_x, const uint8_t* w_packed,
                               const float* gamma, int64_t M, int64_t N, int64_t K, uint16_t* y, void* slopes,
                               void* workspace, size_t workspace_bytes, void* stream);
size_t bitnet_gated_bwd_workspace_bytes(int64_t M, int64_t N, int64_t K);
bitnet_status bitnet_gated_bwd(const uint16_t* dY, const void* slopes, const int8_t* x_q,
                               const float* s_x, const uint8_t* w_packed, const float* gamma, int64_t M, int64_t N,
                               int64_t K, uint16_t* dX, void* dW_gate, void* dW_up, bitnet_dtype dW_dtype,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * A linear layer in 8-bit integers with a scale per token and per channel (what a
 * model keeps out of its ternary layers, such as its head):
 *
 *   y[m,n]  = bf16_rne(acc[m,n] * (s_x[m]/127) * (s_w[n]/127) + bias[n]), acc exact int32
 *   dX[m,k] = sum_n dY[m,n] * w_hat[n,k],  w_hat = bf16_rne(w_q * s_w/127)
 *   dW[n,k] = sum_m dY[m,n] * x_hat[m,k],  x_hat = bf16_rne(x_q * s_x/127)
 *   db[n]   = sum_m dY[m,n]
 *
 * (fp32 rescale and sums, in a fixed order; the gradients are straight through both
 * quantizations).
 *
 * x_q [M][Kp], s_x [M]; w_q [N][Kp], s_w [N]: 8-bit rows (bitnet_rows_quant), columns
 *            K..Kp-1 zero.  x: as for bitnet_gated_fwd.
 * bias       [N] bf16 bits, or NULL.   y, dY [M][N] bf16 bits.
 * dX         [M][K] bf16 bits, or NULL.  dW [N][K] in dW_dtype, or NULL.  db [N] in
 *            db_dtype, or NULL; not all NULL.
 * workspace  bitnet_int8_fwd_workspace_bytes / bitnet_int8_bwd_workspace_bytes (0 for
 *            sizes the call rejects); as for bitlinear_fwd. The backward's holds both
 *            bf16 operands.
 * Pointers 16-byte aligned but db (its element). K <= 131072 (the int32 sums); (M + 256) * 2 Kp,
 * (N + 256) * 2 Kp and (M + 256) * 2 Nd bytes <= 2^31 (Nd = bitnet_k_pad(N); the forward
 * needs (M + 256) * Kp and (N + 256) * Kp only), N <= 2^24.
 */
size_t bitnet_int8_fwd_workspace_bytes(int64_t M, int64_t N, int64_t K);
bitnet_status bitnet_int8_fwd(const uint16_t* x, const int8_t* x_q, const float* s_x, const int8_t* w_q, const float* s_w,
                              const uint16_t* bias, int64_t M, int64_t N, int64_t K, uint16_t* y, void* workspace,
                              size_t workspace_bytes, void* stream);
size_t bitnet_int8_bwd_workspace_bytes(int64_t M, int64_t N, int64_t K);
bitnet_status bitnet_int8_bwd(const uint16_t* dY, const int8_t* x_q, const float* s_x, const int8_t* w_q,
                              const float* s_w, int64_t M, int64_t N, int64_t K, uint16_t* dX, void* dW,
                              bitnet_dtype dW_dtype, void* db, bitnet_dtype db_dtype, void* workspace,
                              size_t workspace_bytes, void* stream);

/*
 * Test hooks (for the library's own tests and tuning; not needed to use it).
 *
 * bitnet_set_test_knobs - process-wide knobs read by every later launch:
 *   split_ctas  0: the cost model chooses how output tiles are shared out;
 *               > 0: every large-M GEMM splits its tiles over that many
 *               workgroups (at most 256; no paired backward launch);
 *               < 0: whole tiles only.
 *   pair_cols   0: the cost model; k >= 1: a paired backward launch gives
 *               dX k of its 8-workgroup columns.
 *   no_skinny   nonzero: the cross entropy by tiles for every size, and the
 *               large-M GEMMs also for M <= 64 (workspace
 *               sizes queried while it is set cover that route).
 *   spin_limit  polls (each a short sleep) before a workgroup waiting for
 *               another's partial tile gives up; the default,
 *               bitnet_default_spin_limit(), is about a second. A wait
 *               that gives up writes its output tile as NaN (outputs of
 *               int32 accumulators, but the gated pair's: as of INT32_MIN)
 *               and is counted.
 *               The one-pass weight quantization waits at most the same
 *               number of polls, and at most 200 us, for the other
 *               workgroups' partial sums; when it gives up, a workgroup
 *               computes the missing sums itself (same results, more reads
 *               of W) and counts each.
 * bitnet_split_timeouts - the number of such waits that gave up on the
 *   current device since the last call (then reset to 0). Synchronizes the
 *   device. BITNET_ERR_HIP if the runtime fails.
 * bitnet_quantize_recomputes - the number of partial sums one-pass
 *   launches computed themselves on the current device since the last call
 *   (then reset to 0). Synchronizes the device.
 * bitnet_debug_split_pieces - the pieces a split launch of `tiles` tiles of
 *   `stages` reduction stages over `grid` workgroups (grid <= tiles*stages)
 *   runs, computed on the host by the functions the kernels use: for each
 *   piece in workgroup order, its virtual workgroup v, tile t, stages
 *   [s0, s1), partial-tile slot, and the first workgroup va and piece count
 *   n of its tile. Writes at most cap entries per array; returns the number
 *   of pieces, or -1 for invalid arguments. bitnet_debug_partial_slots: the
 *   slot count the plan reserves. bitnet_debug_cta_order: the virtual index
 *   of each of `grid` workgroups (workgroup b runs on XCD b % 8; each XCD
 *   gets a contiguous range).
 * bitnet_debug_mfma_probe - enqueues one launch of register-only MFMA chains
 *   on every SIMD (int8 != 0: v_mfma_i32_32x32x32_i8, else
 *   v_mfma_f32_32x32x16_bf16), `iters` rounds (1 .. 2^24), and stores in
 *   *ops (host) the operations it performs; timing it gives the MFMA rate
 *   the chip sustains under a full load. sink: device float[2048] (not
 *   written in practice).
 */
void bitnet_set_test_knobs(int split_ctas, int pair_cols, int no_skinny, uint32_t spin_limit);
uint32_t bitnet_default_spin_limit(void);
bitnet_status bitnet_split_timeouts(uint32_t* count);
bitnet_status bitnet_quantize_recomputes(uint32_t* count);
int64_t bitnet_debug_split_pieces(int64_t tiles, int32_t stages, int32_t grid, int32_t* v, int32_t* t,
                                  int32_t* s0, int32_t* s1, int64_t* slot, int32_t* va, int32_t* n,
                                  int64_t cap);
int32_t bitnet_debug_partial_slots(int64_t tiles, int32_t grid);
void bitnet_debug_cta_order(int32_t grid, int32_t* out);
bitnet_status bitnet_debug_mfma_probe(int32_t int8, int32_t iters, float* sink, double* ops, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BITNET_H */
