/*
 * jet_fp8.h - C ABI of the GB300 (sm_103a) unified-precision FP8 linear layer.
 *
 * The layer is the one Jet-RL runs for both rollout and training ("Jet-RL:
 * Enabling On-Policy FP8 Reinforcement Learning with Unified Training and
 * Rollout Precision Flow", gist.science summary, sections "Kernarchitektur"
 * and "Quantisierungsschema"): activations and output gradients quantized to
 * E4M3 in 1x128 groups, weights in 128x128 blocks, each group with an FP32
 * scale ("NVIDIA强化学习加速实操：10分钟提升2倍训练效率", nmedialink.com,
 * section "为什么FP8适配线性层？", quantization table); forward, DGrad and WGrad
 * GEMMs in FP8, WGrad fed by 1x128 and 128x1 groups.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - All tensor pointers are DEVICE pointers owned by the caller.  The library
 *    allocates and frees nothing and keeps no pointer after a call returns.
 *  - Tensors are dense and row-major (last index contiguous).  BF16 values are
 *    passed as their uint16_t bit patterns; E4M3 codes as uint8_t (OCP E4M3FN:
 *    bias 7, max 448, NaN 0x7F/0xFF).  Scales are IEEE binary32.
 *  - Naming follows nn.Linear: X [M,K] (M tokens, K in-features), W [N,K]
 *    (N out-features), Y = X W^T [M,N], dY [M,N], dX = dY W [M,K],
 *    dW = dY^T X [N,K].  Kb = K/128, Nb = N/128, Mb = M/128.
 *  - The quantization rule for every group G: amax = max |v| over G (binary32),
 *    s = amax / 448 (IEEE binary32 division; s = 1 when amax == 0), and each
 *    code q = E4M3(fl32(v / s)) rounded to nearest, ties to even, saturating
 *    at +-448, sign of zero kept.  The stored scale dequantizes: v ~ q * s.
 *  - Every call validates its arguments on the host, in this order, and returns
 *    the first violation without launching anything: JET_ERR_NULL,
 *    JET_ERR_SHAPE, JET_ERR_ALIGN (every pointer must be 16-byte aligned, but
 *    for the arrays of one value per token, row, request or head of
 *    jet_add_rmsnorm_*, jet_rope*, jet_kv_slot_map, jet_sample*,
 *    jet_kv_attention and jet_head_logp*, and the logits of jet_sample_unaligned, which need their type's alignment),
 *    JET_ERR_WORKSPACE, JET_ERR_DEVICE (current device must be sm_103).
 *    A pointer may be NULL only when its tensor is empty.
 *  - Work is enqueued asynchronously on `stream` (a cudaStream_t; NULL is the
 *    legacy default stream).  Launch failures return JET_ERR_CUDA.  Device-side
 *    bounded waits that give up are reported by jet_device_status().
 *  - Kernels are launched with programmatic dependent launch allowed: their
 *    blocks may start while earlier work on the stream finishes, but each
 *    waits for that work to complete before it reads or writes memory, so
 *    stream order holds (also inside captured CUDA graphs).
 *  - Non-finite inputs are outside the contract (their codes are unspecified).
 *  - Calls are reentrant; concurrent calls must not share output buffers.
 */
#ifndef JET_FP8_H
#define JET_FP8_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define JET_API __attribute__((visibility("default")))
#else
#define JET_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    JET_OK = 0,
    JET_ERR_NULL = 1,      /* a required pointer is NULL                       */
    JET_ERR_SHAPE = 2,     /* a size is negative or not a required multiple    */
    JET_ERR_ALIGN = 3,     /* a pointer is not 16-byte aligned                 */
    JET_ERR_CUDA = 4,      /* a CUDA runtime call or a kernel launch failed    */
    JET_ERR_DEVICE = 5,    /* no current device, or it is not sm_103           */
    JET_ERR_WORKSPACE = 6, /* workspace missing or smaller than required       */
    JET_ERR_TIMEOUT = 7    /* a device-side bounded wait gave up (see status)  */
} jet_status;

/* Operation ids for jet_workspace_bytes(). */
typedef enum {
    JET_OP_QUANT_ACT_1X128 = 0,
    JET_OP_QUANT_W_128X128 = 1,
    JET_OP_REQUANT_128X1 = 2,
    JET_OP_GEMM_FWD = 3,
    JET_OP_GEMM_DGRAD = 4,
    JET_OP_GEMM_WGRAD = 5,
    JET_OP_TOKEN_MULT_PROB_ERROR = 6,
    JET_OP_QUANT_DUAL_1X128_128X1 = 7,
    JET_OP_TOKEN_MISMATCH_MASKED = 8,
    JET_OP_SWIGLU_QUANT_1X128 = 9,
    JET_OP_KV_CALIBRATE = 10,
    JET_OP_KV_CACHE_WRITE = 11,
    JET_OP_TOKEN_MISMATCH_PER_SEQUENCE = 12,
    JET_OP_RMSNORM_QUANT_1X128 = 13,
    JET_OP_ADD_RMSNORM_QUANT_1X128 = 14,
    JET_OP_ADD_RMSNORM_BWD = 15,
    JET_OP_ROPE = 16,
    JET_OP_ROPE_KV_CACHE_WRITE = 17,
    JET_OP_KV_SLOT_MAP = 18,
    JET_OP_SAMPLE = 19,
    JET_OP_KV_ATTENTION = 20, /* its workspace: jet_kv_attention_workspace() */
    JET_OP_SWIGLU_BWD_QUANT_1X128 = 21,
    JET_OP_HEAD_LOGP = 22,
    JET_OP_HEAD_LOGP_BWD = 23
} jet_op;

/* Pair layouts of jet_rope: (i, i + R/2) or (2 i, 2 i + 1). */
typedef enum { JET_ROPE_HALF = 0, JET_ROPE_INTERLEAVED = 1 } jet_rope_layout;

/* Frequency scalings of jet_rope_inv_freq. */
typedef enum {
    JET_ROPE_SCALE_NONE = 0,
    JET_ROPE_SCALE_LINEAR = 1,
    JET_ROPE_SCALE_WAVELENGTH = 2,
    JET_ROPE_SCALE_RAMP = 3
} jet_rope_scaling;

/* Types of the logits of jet_sample. */
typedef enum { JET_BF16 = 0, JET_FP32 = 1 } jet_dtype;

/* A cudaStream_t handle passed as an opaque pointer. */
typedef void *jet_stream_t;

/* Static, NUL-terminated name of a status code ("JET_OK", ...). */
JET_API const char *jet_status_str(int status);

/* ABI version (major * 10000 + minor * 100 + patch). */
JET_API int jet_version(void);

/*
 * 1x128 quantization of activations or output gradients.
 * Source: nmedialink.com page, section "为什么FP8适配线性层？" (input activations
 * and output gradients: E4M3, [1,128], FP32 scales); gist.science summary,
 * "Quantisierungsschema" (activations 1x128).  Used for X before the forward
 * GEMM and for dY (with K := N) before the DGrad GEMM.
 *   x  [M][K] BF16 bits (in).       M >= 0, K >= 0 and K % 128 == 0.
 *   q  [M][K] E4M3 codes (out).
 *   s  [Kb][M] FP32 scales (out): s[kb*M + m] belongs to row m, columns
 *      128*kb .. 128*kb+127 (K-block-major so a GEMM tile's row scales are
 *      contiguous).
 */
JET_API jet_status jet_quant_act_1x128(const uint16_t *x, int64_t M, int64_t K,
                               uint8_t *q, float *s, jet_stream_t stream);

/*
 * 128x128 block quantization of weights (run once per weight sync).
 * Source: nmedialink.com page, quantization table (weights: E4M3, [128,128],
 * FP32); gist.science summary, "Quantisierungsschema" (weights 128x128).
 *   w  [N][K] BF16 bits (in).       N, K >= 0, both multiples of 128.
 *   q  [N][K] E4M3 codes (out).
 *   s  [Nb][Kb] FP32 scales (out), s[nb*Kb + kb].
 */
JET_API jet_status jet_quant_w_128x128(const uint16_t *w, int64_t N, int64_t K,
                               uint8_t *q, float *s, jet_stream_t stream);

/*
 * 128x1 re-quantization along the token axis, fused with the transpose that
 * the WGrad GEMM needs.  Source: 163.com article, section 五 (1x128 forward
 * groups re-quantized as 128x1 in backward); gist.science summary,
 * "Quantisierungsschema" (WGrad with 1x128 and 128x1 groups).  The input is
 * the saved FP8 form: v[m][k] = fl32(D4(q[m][k]) * s[k/128][m]); each group is
 * tokens 128*mb .. 128*mb+127 of one column k.
 *   q   [M][K] E4M3 codes, s [Kb][M] scales (in; the jet_quant_act_1x128 form).
 *   qT  [K][M] E4M3 codes (out), transposed.   M, K >= 0, multiples of 128.
 *   sT  [Mb][K] FP32 scales (out), sT[mb*K + k].
 */
JET_API jet_status jet_requant_128x1(const uint8_t *q, const float *s, int64_t M,
                             int64_t K, uint8_t *qT, float *sT,
                             jet_stream_t stream);

/*
 * SwiGLU with the 1x128 quantization of its output fused: the input of an
 * MLP's down projection, h = silu(gate) * up, written directly as the
 * jet_quant_act_1x128 form (no BF16 copy of h).  Source: 163.com article,
 * section 三, and gist.science summary, "Quantisierungsschema" (the quantizer
 * fused into the operator that produces a linear layer's input).  h is
 * evaluated in binary32 by a fixed sequence of IEEE operations (Cody-Waite
 * e^x with a degree-7 Taylor polynomial; 1/(1 + e^-g) by a bit-pattern seed
 * and three Newton-Raphson steps; g < -80 gives a signed zero), within 3 ulps
 * of silu(g) * up; its 128-wide groups then follow the 1x128 group rule.
 *   gate, up  BF16 bits, row m at gate + m*ld and up + m*ld (in).  For the
 *       concatenated [M][2F] output of a gate_up product pass gate = base,
 *       up = base + F, ld = 2F.  ld >= F, a multiple of 8.
 *   q   [M][F] E4M3 codes, s [F/128][M] FP32 scales (out).  M, F >= 0, F a
 *       multiple of 128.  Non-finite h (overflowing products) is a
 *       precondition violation with unspecified codes.
 */
JET_API jet_status jet_swiglu_quant_1x128(const uint16_t *gate, const uint16_t *up, int64_t ld,
                                          int64_t M, int64_t F, uint8_t *q, float *s,
                                          jet_stream_t stream);

/*
 * RMSNorm with the 1x128 quantization of its output fused: the input of the
 * q/k/v and gate/up projections written as E4M3 codes and FP32 scales
 * straight from the residual stream, with no BF16 normalised activation.
 * Source: gist.science summary, "Implementierung" (fused activation/RMSNorm
 * operators in custom kernels), and 163.com article, section 五 (a linear
 * layer's input quantized in the operator that produces it).  The pages give
 * no arithmetic; y = x * g / sqrt(mean(x^2) + eps) is evaluated in binary32
 * in one fixed order: lane partial sums of squares (lane l adds the elements
 * 8 (32 j + l) + t in order of j, then t = 0 .. 7), a five-level butterfly,
 * ms = ss / K, v = ms + eps, r = 1 / sqrt(v) (IEEE operations; r = 0 when
 * v == 0), y = (x * r) * g; its 128-wide groups then follow the 1x128 group
 * rule.  Within a few ulps of binary64 RMSNorm (at most (K/64 + 8.5) 2^-24
 * relative).
 *   x   [M][K] BF16 bits (in; the residual stream), g [K] BF16 bits (in; the
 *       norm's gain).  M, K >= 0, K a multiple of 128 and below 2^24.
 *   eps >= 0 (finite); the model's value, e.g. 1e-5.
 *   q   [M][K] E4M3 codes, s [K/128][M] FP32 scales (out).
 * Rows whose sum of squares overflows binary32 are a precondition violation
 * with unspecified codes.
 */
JET_API jet_status jet_rmsnorm_quant_1x128(const uint16_t *x, const uint16_t *g, int64_t M,
                                           int64_t K, float eps, uint8_t *q, float *s,
                                           jet_stream_t stream);

/*
 * FP8 KV cache, scales recalibrated after each model update.  Source: FP8-RL
 * article (m.66260.cn), KV-cache paragraph (scale factors calibrated again
 * after every model update); nmedialink page, section "FP8探索新维度：KV缓存与
 * 注意力机制赋能" (FP8 KV cache).  The pages give no granularity; here one
 * FP32 scale per KV head, for K and for V separately.
 *
 * jet_kv_calibrate: scale[h] = amax_h / 448 (IEEE division; 1 when the head
 * is all zero), amax_h over all T tokens and D channels of head h of the
 * calibration batch x [T][H][D] (BF16 bits).  Writes scale [H] FP32 (device;
 * also used as scratch during the call).
 *
 * jet_kv_cache_write: cache[slots[t]][h][d] = E4(fl32(x[t][h][d] / scale[h]))
 * for the T new entries x [T][H][D] (BF16 bits); entries beyond the
 * calibrated range saturate to +-448.  slots [T] int64 DEVICE array of
 * distinct cache rows; a slot outside [0, S) is skipped.  cache [S][H][D]
 * E4M3 codes (in/out; other rows untouched).
 *
 * T, S >= 0; 0 <= H <= 1024; D a multiple of 16.
 */
JET_API jet_status jet_kv_calibrate(const uint16_t *x, int64_t T, int64_t H, int64_t D,
                                    float *scale, jet_stream_t stream);
JET_API jet_status jet_kv_cache_write(const uint16_t *x, const float *scale,
                                      const int64_t *slots, int64_t T, int64_t H, int64_t D,
                                      uint8_t *cache, int64_t S, jet_stream_t stream);

/*
 * Both quantizations of one tensor from a single read: the 1x128 form of
 * jet_quant_act_1x128 and the transposed 128x1 form that jet_requant_128x1
 * derives from it (re-quantized from the FP8 1x128 values).  Used for the
 * output gradient dY, whose two forms feed DGrad and WGrad in the same
 * backward step.  Source: 163.com article, section 五 (1x128 groups
 * re-quantized as 128x1 for backward; quantization fused into the operator
 * that produces the tensor); gist.science summary, "Quantisierungsschema"
 * (DGrad with 1x128, WGrad with 1x128 and 128x1).  Codes and scales equal
 * those of jet_quant_act_1x128 followed by jet_requant_128x1, bit for bit.
 *   x   [M][K] BF16 bits (in).      M, K >= 0, both multiples of 128.
 *   q   [M][K] E4M3 codes, s [Kb][M] FP32 scales (out; the 1x128 form).
 *   qT  [K][M] E4M3 codes, sT [Mb][K] FP32 scales (out; the 128x1 form).
 */
JET_API jet_status jet_quant_dual_1x128_128x1(const uint16_t *x, int64_t M, int64_t K,
                                              uint8_t *q, float *s, uint8_t *qT, float *sT,
                                              jet_stream_t stream);

/*
 * Forward GEMM  Y = X W^T  with per-128-K-block scale promotion:
 *   Y[m][n] = sum_kb sx[kb][m] * sw[n/128][kb] * sum_{k in kb} qx[m][k] qw[n][k]
 * accumulated in FP32 and written as BF16 (round to nearest even).
 * Source: gist.science summary, "Quantisierungsschema" (FP8 GEMMs of linear
 * layers); 163.com article, section 五 (1x128 inputs times 128x128 weights).
 *   qx [M][K], sx [Kb][M] (jet_quant_act_1x128 of X);  M >= 0.
 *   qw [N][K], sw [Nb][Kb] (jet_quant_w_128x128 of W); N, K multiples of 128.
 *   y  [M][N] BF16 bits (out).  K == 0 writes zeros.
 *   ws / ws_bytes: device workspace of at least
 *   jet_workspace_bytes(JET_OP_GEMM_FWD, M, N, K) bytes, else JET_ERR_WORKSPACE
 *   (NULL/0 allowed when that is 0).  It can be non-zero only for M <= 512,
 *   where the contraction may be split into ranges whose FP32 partial tiles
 *   [splits][M][N] go to ws and are then summed in a fixed order and rounded
 *   once to BF16; the split depends only on (M, N, K), so results are the same
 *   on every call and every device.  Its contents need no initialisation and
 *   are scratch after the call; concurrent calls need separate workspaces.
 *   M == 1, and 2 <= M <= 4 with M * N * K <= 2^25 (decode), run a weight-streaming kernel
 *   on CUDA cores with the same arithmetic (exact code products, FP32 sums
 *   per scale group, scaled and summed in a fixed order) and needs no
 *   workspace.
 */
JET_API jet_status jet_gemm_fp8_fwd(const uint8_t *qx, const float *sx,
                            const uint8_t *qw, const float *sw, int64_t M,
                            int64_t N, int64_t K, uint16_t *y, void *ws,
                            size_t ws_bytes, jet_stream_t stream);

/*
 * Grouped forward GEMM of expert linears (mixture-of-experts layers), one
 * launch for all experts:  for every expert e and its tokens
 * m in [offsets[e], offsets[e+1]),
 *   Y[m][n] = sum_kb sx[kb][m] * sw[e][n/128][kb] * sum_{k in kb} qx[m][k] qw[e][n][k]
 * with the arithmetic of jet_gemm_fp8_fwd (FP32 accumulation, BF16 out).
 * Source: 163.com article / nmedialink.com page (FP8 for the Qwen3-30B MoE
 * model, section "在专家混合模型中的突破"); m.66260.cn FP8-RL article (expert
 * layers in the compressed format).  The pages give no grouped kernel; this
 * layout is this library's choice.
 *   qx [M][K], sx [Kb][M]: the tokens of all experts, in expert order (the
 *     jet_quant_act_1x128 form of the concatenated activations).
 *   qw [E][N][K], sw [E][Nb][Kb]: the experts' weights and scales, stacked.
 *   offsets [E+1] int64, DEVICE array: offsets[0] = 0, non-decreasing,
 *     offsets[E] = M (e.g. written by the routing kernel).  Offsets outside
 *     [0, M] are clamped and a decreasing pair is an empty expert, so no
 *     write ever leaves y; results are then unspecified.
 *   y [M][N] BF16 bits (out).  1 <= E <= 384; N, K multiples of 128.
 */
JET_API jet_status jet_gemm_fp8_fwd_grouped(const uint8_t *qx, const float *sx,
                                            const uint8_t *qw, const float *sw,
                                            const int64_t *offsets, int64_t E, int64_t M,
                                            int64_t N, int64_t K, uint16_t *y,
                                            jet_stream_t stream);

/*
 * Grouped DGrad of expert linears, one launch: for every expert e and its
 * tokens m in [offsets[e], offsets[e+1]),
 *   dX[m][k] = sum_nb sdy[nb][m] * sw[e][nb][k/128] * sum_{n in nb} qdy[m][n] qw[e][n][k]
 * with the arithmetic of jet_gemm_fp8_dgrad.  Source and layout as
 * jet_gemm_fp8_fwd_grouped (the backward of the same expert linears).
 *   qdy [M][N], sdy [Nb][M]: the output gradients of all experts' tokens in
 *     expert order.  qw [E][N][K], sw [E][Nb][Kb] as in the forward.
 *   offsets [E+1] int64 DEVICE array, as in jet_gemm_fp8_fwd_grouped.
 *   dx [M][K] BF16 bits (out).  1 <= E <= 384; N, K multiples of 128.
 */
JET_API jet_status jet_gemm_fp8_dgrad_grouped(const uint8_t *qdy, const float *sdy,
                                              const uint8_t *qw, const float *sw,
                                              const int64_t *offsets, int64_t E, int64_t M,
                                              int64_t N, int64_t K, uint16_t *dx,
                                              jet_stream_t stream);

/*
 * Grouped WGrad of expert linears, one launch: every expert's weight
 * gradient over its own tokens,
 *   dW[e][n][k] = sum_{mb in expert e} sdyT[mb][n] * sxT[mb][k]
 *                 * sum_{m in mb} qdyT[n][m] qxT[k][m]
 * with the arithmetic of jet_gemm_fp8_wgrad.  Source as
 * jet_gemm_fp8_fwd_grouped; 128x1 groups as jet_gemm_fp8_wgrad.
 *   qdyT [N][M], sdyT [Mb][N] and qxT [K][M], sxT [Mb][K]: the 128x1 forms
 *     (jet_requant_128x1 / jet_quant_dual_1x128_128x1) of the expert-ordered
 *     output gradients and inputs.
 *   offsets [E+1] int64 DEVICE array: offsets[0] = 0, non-decreasing,
 *     offsets[E] = M, every offset a multiple of 128 (a 128-token group never
 *     straddles two experts: experts are padded to whole groups, with zero
 *     rows).  Offsets are clamped to [0, M]; other violations give
 *     unspecified results, never a write outside dw.
 *   dw [E][N][K] BF16 bits (out); an expert without tokens gets zeros.
 *   M, N, K multiples of 128; 1 <= E <= 384.
 */
JET_API jet_status jet_gemm_fp8_wgrad_grouped(const uint8_t *qdyT, const float *sdyT,
                                              const uint8_t *qxT, const float *sxT,
                                              const int64_t *offsets, int64_t E, int64_t M,
                                              int64_t N, int64_t K, uint16_t *dw,
                                              jet_stream_t stream);

/*
 * DGrad GEMM  dX = dY W :
 *   dX[m][k] = sum_nb sdy[nb][m] * sw[nb][k/128] * sum_{n in nb} qdy[m][n] qw[n][k]
 * FP32 accumulation, BF16 out.  Source: gist.science summary,
 * "Quantisierungsschema", "Backward-Pass" (DGrad in FP8).
 *   qdy [M][N], sdy [Nb][M] (jet_quant_act_1x128 of dY with K := N).
 *   qw  [N][K], sw [Nb][Kb] (the forward weight codes, read transposed).
 *   dx  [M][K] BF16 bits (out).  N == 0 writes zeros.
 *   ws / ws_bytes: as for the forward GEMM, with
 *   jet_workspace_bytes(JET_OP_GEMM_DGRAD, M, N, K) (partials [splits][M][K]).
 */
JET_API jet_status jet_gemm_fp8_dgrad(const uint8_t *qdy, const float *sdy,
                              const uint8_t *qw, const float *sw, int64_t M,
                              int64_t N, int64_t K, uint16_t *dx, void *ws,
                              size_t ws_bytes, jet_stream_t stream);

/*
 * WGrad GEMM  dW = dY^T X  on the 128x1 (token-axis) groups:
 *   dW[n][k] = sum_mb sdyT[mb][n] * sxT[mb][k] * sum_{m in mb} qdyT[n][m] qxT[k][m]
 * FP32 accumulation, BF16 out.  Source: gist.science summary,
 * "Quantisierungsschema", "Backward-Pass" (WGrad in FP8 with 1x128 and 128x1).
 *   qdyT [N][M], sdyT [Mb][N]  (jet_requant_128x1 of dY's 1x128 form).
 *   qxT  [K][M], sxT  [Mb][K]  (jet_requant_128x1 of X's 1x128 form).
 *   dw   [N][K] BF16 bits (out).  M % 128 == 0; M == 0 writes zeros.
 *   ws / ws_bytes: unused (jet_workspace_bytes(JET_OP_GEMM_WGRAD, ...) is 0).
 */
JET_API jet_status jet_gemm_fp8_wgrad(const uint8_t *qdyT, const float *sdyT,
                              const uint8_t *qxT, const float *sxT, int64_t M,
                              int64_t N, int64_t K, uint16_t *dw, void *ws,
                              size_t ws_bytes, jet_stream_t stream);

/*
 * Train/rollout mismatch metric
 *   token-mult-prob-error = (1/n) * sum_i exp(|logp_train[i] - logp_rollout[i]|)
 * Source: nmedialink.com page, section "FP8面临的关键挑战：数值分歧".  No mask:
 * every one of the n tokens counts.  Per-thread sums in FP32, across threads
 * and blocks in FP64 (fixed order, deterministic); result written as FP32.
 *   logp_train, logp_rollout [n] FP32 (in), n >= 1.
 *   out: one FP32 in device memory (out).
 *   ws / ws_bytes: at least jet_workspace_bytes(JET_OP_TOKEN_MULT_PROB_ERROR,
 *   n, 0, 0) bytes of device memory (per-block FP64 partial sums).
 */
JET_API jet_status jet_token_mult_prob_error(const float *logp_train,
                                     const float *logp_rollout, int64_t n,
                                     float *out, void *ws, size_t ws_bytes,
                                     jet_stream_t stream);

/*
 * token-mult-prob-error without a workspace argument, for callers that cannot
 * allocate device memory: a plain C host that only receives device pointers
 * from another runtime and has no allocator of its own, or a latency-bound
 * loop that must not call cudaMalloc (it can synchronize the whole device and
 * is not ordered on a stream).  The pages have no counterpart; this is a
 * convenience of this library.  Same arithmetic, grid and result as
 * jet_token_mult_prob_error.
 *   logp_train, logp_rollout [n] FP32 (in), out: one FP32 (out); device
 *   pointers owned by the caller, as everywhere else.
 *   1 <= n <= 2,097,152; larger n returns JET_ERR_SHAPE before any launch.
 * The per-block partial sums go to a static 8 KB device array inside the
 * library (1024 FP64 slots; every device that loads the library keeps it until
 * the process exits).  The library allocates and frees nothing here.  The first
 * call on a device looks up that array's device address (with the device
 * current) and caches it for the device's current context (after a device
 * reset the next call looks it up again); make that first call before any
 * stream capture.
 * All calls share the one array: calls whose kernels overlap on the GPU (e.g.
 * on two streams at once) race on it and may return wrong values - order them
 * on one stream or use jet_token_mult_prob_error with separate workspaces.
 * Nothing needs clearing between calls: every slot a call reads is written
 * earlier in the same call.
 */
JET_API jet_status jet_token_mult_prob_error_noalloc(const float *logp_train,
                                                     const float *logp_rollout,
                                                     int64_t n, float *out,
                                                     jet_stream_t stream);

/*
 * The mismatch metric over a subset of the tokens, fused with the per-token
 * importance weights of the training loss, in one pass over the tokens.
 * Source: nmedialink.com page, sections "FP8面临的关键挑战：数值分歧" (the
 * metric) and "重要抽样技术：提升RL精度的尖兵" (importance sampling with FP8);
 * m.66260.cn FP8-RL article (the weight is the ratio of the original to the
 * compressed model's token probability).  With a = logp_train, b =
 * logp_rollout and mask m (the tokens that count, e.g. a response mask):
 *   w_i = m_i ? min(exp(a_i - b_i), cap) : 0        (no cap when cap <= 0;
 *                                                    the pages give none)
 *   out = sum_{m_i} exp(|a_i - b_i|) / count,  count = #{i : m_i != 0}
 * exp in FP32 per token, sums in FP32 per thread and FP64 across threads and
 * blocks in a fixed order; out is NaN when no token counts.
 *   logp_train, logp_rollout [n] FP32 (in), n >= 1.
 *   mask [n] uint8 (in; nonzero = the token counts), or NULL: every token.
 *   w [n] FP32 (out), or NULL: the weights are not written.
 *   out: one FP32 (out); count: one int64 (out), or NULL.  Device pointers.
 *   ws / ws_bytes: at least jet_workspace_bytes(JET_OP_TOKEN_MISMATCH_MASKED,
 *   n, 0, 0) bytes of device memory.
 */
JET_API jet_status jet_token_mismatch_masked(const float *logp_train, const float *logp_rollout,
                                             const uint8_t *mask, int64_t n, float cap, float *w,
                                             float *out, int64_t *count, void *ws,
                                             size_t ws_bytes, jet_stream_t stream);

/*
 * Per-sequence form of jet_token_mismatch_masked, one pass: for every
 * sequence s (tokens seq_offsets[s] .. seq_offsets[s+1]) the mean of
 * exp|logp_train_i - logp_rollout_i| over its masked tokens, and the same
 * per-token importance weights.  Source: nmedialink page, "FP8面临的关键挑战：
 * 数值分歧" (the metric) and its importance-sampling paragraph; FP8-RL article
 * (the probability ratio).  Computed as jet_token_mismatch_masked: exp in
 * FP32 per token, sums in FP64, result FP32; deterministic.
 *   logp_train, logp_rollout [n] FP32; mask [n] uint8 or NULL (every token).
 *   seq_offsets [S+1] int64 DEVICE array: 0, non-decreasing, n (offsets are
 *     clamped to [0, n]; a decreasing pair is an empty sequence).
 *   cap: importance weights min(w, cap) when cap > 0.
 *   w [n] FP32 or NULL (out); out [S] FP32 (out; NaN for a sequence without
 *   masked tokens); count [S] int64 or NULL (out).  S >= 1, n >= 0.
 */
JET_API jet_status jet_token_mismatch_per_sequence(const float *logp_train,
                                                   const float *logp_rollout,
                                                   const uint8_t *mask,
                                                   const int64_t *seq_offsets, int64_t S,
                                                   int64_t n, float cap, float *w, float *out,
                                                   int64_t *count, jet_stream_t stream);

/*
 * The residual addition, RMSNorm and the 1x128 quantization in one pass: the
 * step between two projections of a layer.  The pages have no counterpart
 * beyond the fused RMSNorm of jet_rmsnorm_quant_1x128, whose arithmetic this
 * call follows:
 *   h = BF16(x + d) (binary32 sum, one rounding), then
 *   q, s = jet_rmsnorm_quant_1x128(h, g, eps), bit for bit, at any M.
 *   x   [M][K] BF16 bits (in; the residual stream), d [M][K] BF16 bits (in;
 *       the preceding projection's output), g [K] BF16 bits (in; the gain).
 *   h   [M][K] BF16 bits (out; the new residual stream).  May be x or d
 *       itself (in place); no other overlap is allowed.
 *   q   [M][K] E4M3 codes, s [K/128][M] FP32 scales (out).
 *   rstd [M] FP32 (out; 1 / sqrt(mean(h^2) + eps) of each row, 0 where that
 *       sum is 0; what jet_add_rmsnorm_bwd needs), or NULL.
 * M, K >= 0, K a multiple of 128 and below 2^24; eps >= 0 (finite).
 */
JET_API jet_status jet_add_rmsnorm_quant_1x128(const uint16_t *x, const uint16_t *d,
                                               const uint16_t *g, int64_t M, int64_t K, float eps,
                                               uint16_t *h, uint8_t *q, float *s, float *rstd,
                                               jet_stream_t stream);

/*
 * Backward of the addition and the norm (the quantization passes gradients
 * straight through).  With dy = dy0 + dy1 + dy2 (the DGrads of the products
 * that read the normalised activation: q, k, v or gate, up) and r = rstd:
 *   dx = dres + r (g dy - h r^2 sum_k(g dy h) / K)      (of x and of d alike)
 *   dg = sum_m dy h r
 * in binary32; dx rounded once to BF16, dg kept in FP32, its sum over the
 * rows in one fixed order (deterministic).
 *   h [M][K], g [K] BF16 bits, rstd [M] FP32: as written by the forward.
 *   dy0, dy1, dy2 [M][K] BF16 bits (in); dy1 and dy2 may be NULL.
 *   dres [M][K] BF16 bits (in; the gradient arriving on the residual stream),
 *       or NULL for none.
 *   dx [M][K] BF16 bits (out; may be dres itself), dg [K] FP32 (out; zeros
 *       when M == 0).
 *   ws / ws_bytes: at least jet_workspace_bytes(JET_OP_ADD_RMSNORM_BWD, M, 0,
 *       K) bytes of device memory; scratch, not initialised.
 * M >= 0; K a multiple of 128, 0 <= K <= 32768.
 */
JET_API jet_status jet_add_rmsnorm_bwd(const uint16_t *h, const uint16_t *g, const float *rstd,
                                       const uint16_t *dy0, const uint16_t *dy1,
                                       const uint16_t *dy2, const uint16_t *dres, int64_t M,
                                       int64_t K, uint16_t *dx, float *dg, void *ws,
                                       size_t ws_bytes, jet_stream_t stream);

/*
 * Rotary position frequencies, a HOST function (no device, no stream): the
 * angle per position of channel pair i, 0 <= i < R/2, in binary64,
 *   f_i = base^(-2 i / R),
 * scaled for contexts longer than the `context` positions of training:
 *   NONE        f_i
 *   LINEAR      f_i / factor
 *   WAVELENGTH  with n_i = context f_i / (2 pi) turns over that context:
 *               f_i (1 - s + s / factor), s = 0 for n_i >= high, 1 for
 *               n_i <= low, (high - n_i) / (high - low) between.
 *   RAMP        the same blend with s linear in i between the pairs that turn
 *               `high` and `low` times over that context: i_n = R ln(context /
 *               (2 pi n)) / (2 ln base), from floor(i_high) to ceil(i_low),
 *               both kept within [0, R - 1]; and mscale = 1 + 0.1 ln(factor)
 *               for factor > 1 (published as YaRN, Peng et al., 2023).
 *   inv_freq [R/2] (out, host memory), mscale (out, host; 1 except for RAMP).
 * R even, 2 <= R <= 1024; base > 1; factor, context > 0; WAVELENGTH and RAMP:
 * 0 < low < high.  Unused parameters are ignored.
 */
JET_API jet_status jet_rope_inv_freq(int64_t R, double base, int scaling, double factor,
                                     double context, double low, double high, double *inv_freq,
                                     float *mscale);

/*
 * Rotary positions of q and k in one launch, forward and backward.  Channel
 * pair (a, b) number i of the first R channels of every head is turned by the
 * angle pos[t] f_i and scaled:
 *   a' = mscale (a cos - b sin),  b' = mscale (b cos + a sin),
 * pairs (i, i + R/2) in JET_ROPE_HALF, (2 i, 2 i + 1) in
 * JET_ROPE_INTERLEAVED; channels R .. D-1 are copied.  backward != 0 turns by
 * the negative angle: the gradients of the inputs from those of the outputs.
 * Angles are reduced modulo a turn in 64-bit integer arithmetic, so positions
 * may be any int64; products in binary32, one rounding to BF16.
 *   q: token t, head h at q + t*ldq + h*D (BF16 bits), h < Hq; k likewise
 *       with ldk, Hk.  qo, ko: outputs, strides ldqo, ldko; they may be q and
 *       k themselves with the same strides (in place; with others of more than
 *       one token JET_ERR_SHAPE).  A tensor with no head may be NULL.
 *   inv_freq [R/2] FP64, pos [T] int64: DEVICE arrays.
 * T, Hq, Hk >= 0, at most 1024 heads each; D a multiple of 8, at most 1024;
 * R even, 0 <= R <= D; strides >= H*D and multiples of 8.
 */
JET_API jet_status jet_rope(const uint16_t *q, int64_t ldq, int64_t Hq, const uint16_t *k,
                            int64_t ldk, int64_t Hk, int64_t T, int64_t D, int64_t R,
                            const double *inv_freq, const int64_t *pos, int layout, float mscale,
                            int backward, uint16_t *qo, int64_t ldqo, uint16_t *ko, int64_t ldko,
                            jet_stream_t stream);

/*
 * Rotary positions fused with the FP8 KV-cache write, for serving: q is
 * rotated into qo, k is rotated and written with v as E4M3 codes into their
 * cache slots.  Equal bit for bit to jet_rope of q and k followed by
 * jet_kv_cache_write of the rotated k (k_scale, k_cache) and of v (v_scale,
 * v_cache).  Arguments as in those calls; a slot outside [0, S) is skipped
 * (its q is still rotated); D a multiple of 16.  With Hk = 0 k, v, the scales,
 * the slots and the caches may be NULL.
 */
JET_API jet_status jet_rope_kv_cache_write(const uint16_t *q, int64_t ldq, int64_t Hq,
                                           const uint16_t *k, int64_t ldk, const uint16_t *v,
                                           int64_t ldv, int64_t Hk, int64_t T, int64_t D,
                                           int64_t R, const double *inv_freq, const int64_t *pos,
                                           int layout, float mscale, const float *k_scale,
                                           const float *v_scale, const int64_t *slots,
                                           uint16_t *qo, int64_t ldqo, uint8_t *k_cache,
                                           uint8_t *v_cache, int64_t S, jet_stream_t stream);

/*
 * Block tables and slot maps of a paged KV cache from the requests' lengths,
 * on the GPU.  The cache's slots come in blocks of block_size; request b holds
 * cached[b] tokens in the blocks table[b][0 ..] and adds added[b] tokens in
 * this step.  The blocks it lacks are taken from the free list in request
 * order, starting at free_blocks[*free_next], and entered in the table; then
 * for every new token t, in request order,
 *   positions[t] = its position in its request,
 *   slots[t] = table[b][pos / block_size] * block_size + pos % block_size,
 *   rows[t] = b.
 * A token without a block gets slot -1 (which the cache writes skip): past the
 * table's width, past the free list's end (its table entry becomes -1), or
 * behind a negative table entry.  Negative lengths count as 0.
 *   cached, added [B] int32; table [B][width] int32 (in/out); free_blocks
 *   [n_free] int32; free_next [1] int64: the number of free blocks already
 *   taken (in).  All DEVICE arrays.
 *   N: capacity of the token outputs.  Tokens past N are not written;
 *   positions, slots, rows of [total, N) get 0, -1, -1.
 *   offsets [B+1] int64 (out): first token of each request, then the total.
 *   positions, slots [N] int64, rows [N] int32 (out).
 *   counts [2] int64 (out): the next free_next (at most n_free), and the
 *   number of blocks that were lacking.  counts must not hold free_next
 *   (JET_ERR_SHAPE); a loop alternates two of them, counts being the next
 *   call's free_next.
 * 0 <= B <= 8192; 1 <= block_size < 2^30; width, n_free < 2^31; N >= 0.
 */
JET_API jet_status jet_kv_slot_map(const int32_t *cached, const int32_t *added, int64_t B,
                                   int64_t block_size, int32_t *table, int64_t width,
                                   const int32_t *free_blocks, int64_t n_free,
                                   const int64_t *free_next, int64_t N, int64_t *offsets,
                                   int64_t *positions, int64_t *slots, int32_t *rows,
                                   int64_t *counts, jet_stream_t stream);

/*
 * One token per row of logits, drawn with temperature, top-k, top-p and min-p
 * from given uniform numbers, and its log-probabilities (the logp_rollout of
 * the mismatch metric).  Per row, with m the largest logit and r =
 * fl32(1 / temperature), brought into binary32's normal range:
 *   z_i = fl32(fl32(x_i - m) * r), w_i = fl32(e^z_i) (CUDA's expf);
 * in the order of falling logit, ties by rising index, kept are the tokens of
 * rank < top_k, of those the ones before which less than top_p of their mass
 * lies, and of those the ones with w_i >= min_p (the largest w is 1).  Drawn
 * is the first kept token, in index order, at which the running sum of the
 * kept weights exceeds u times their sum.  The sums are exact, in 64-bit
 * integers of w_i 2^45 (rounded to nearest), so the token does not depend on
 * the batch or the launch.
 *   logits: row b at logits + b*ld elements, BF16 or FP32 by `dtype`
 *       (jet_dtype).  -inf and NaN are never drawn; +inf counts as the type's
 *       largest finite number.  ld >= V; rows after the first need no
 *       alignment.
 *   u [B] FP32 in [0, 1) (others are brought to the nearest end).
 *   temperature, top_p, min_p [B] FP32, top_k [B] int32: one per row, or NULL:
 *       1, 1, 0, off.  temperature <= 0: the largest logit (lowest index);
 *       top_k <= 0, top_p >= 1, min_p <= 0 turn their filter off; top_p <= 0
 *       keeps the first token alone; min_p > 1 counts as 1.
 *   token [B] int64 (out): -1 for a row with nothing to draw.
 *   logp [B] FP32 (out): log-probability under the kept, renormalised weights;
 *   logp_all [B] FP32 (out): under all of them (a greedy row's at temperature
 *       1); NaN for a row with nothing to draw.
 *   kept [B] int32 (out): the number of kept tokens.
 * 0 <= B < 2^28; 1 <= V <= 262144.
 */
JET_API jet_status jet_sample(const void *logits, int dtype, int64_t B, int64_t V, int64_t ld,
                              const float *u, const float *temperature, const int32_t *top_k,
                              const float *top_p, const float *min_p, int64_t *token, float *logp,
                              float *logp_all, int32_t *kept, jet_stream_t stream);

/*
 * The same for logits that start at any element of their type, as the later
 * rows of a batch with an odd vocabulary do.  The results are the same bits; a
 * row's first and last elements up to a 16-byte boundary are read one by one,
 * in either call.
 */
JET_API jet_status jet_sample_unaligned(const void *logits, int dtype, int64_t B, int64_t V,
                                        int64_t ld, const float *u, const float *temperature,
                                        const int32_t *top_k, const float *top_p,
                                        const float *min_p, int64_t *token, float *logp,
                                        float *logp_all, int32_t *kept, jet_stream_t stream);

/*
 * Attention of a step's new tokens over the paged FP8 cache, grouped-query and
 * causal; for decoding (one token a request), chunks of a prompt (any number),
 * and groups of requests that share a prefix, whose keys are then read once for
 * all of them.  Request b holds lengths[b] keys behind its row of the block
 * table, its own new ones among them (jet_rope_kv_cache_write comes first); its
 * new tokens are rows offsets[b] .. offsets[b+1]-1 of q, the last of them at
 * position lengths[b]-1.  For the query at position pos, head hq of KV head
 * h = hq / (Hq / Hk), over the keys p <= pos:
 *   x_p = scale k_scale[h] (q . k_p),  lse = ln sum_p e^x_p,
 *   out = v_scale[h] sum_p e^(x_p - lse) v_p,
 * k_p, v_p the codes in slot table[b][p / block_size] * block_size +
 * p % block_size.  A key without a slot (a negative table entry, a slot >= S, a
 * position past the table's width) is left out; a query that sees no key gets
 * out 0 and lse -inf.  What a key that a query does not see holds does not matter
 * to it, NaN codes included; a NaN among the values of one that it sees makes that
 * channel of its output NaN, and can make the head's others NaN too.  Products of the queries with the codes are exact to 2^-38
 * of the query's largest channel, sums in binary32, weights rounded to 11 bits
 * (those below 2^-21 of the row's largest to within 2^-32 of it), one rounding to BF16; the result is the same for the same call, whatever ran
 * before.
 * Groups: group i is the requests prefix_offsets[i] .. prefix_offsets[i+1]-1,
 * whose first prefix_lengths[i] keys are the same; they are read through the
 * table row of the group's first request (a longer prefix than that one's
 * length counts as that length), whatever the other rows hold there.  Requests
 * before prefix_offsets[0] or from prefix_offsets[n_prefix] on are in no group.
 *   q: token t, head hq at q + t*ldq + hq*D (BF16 bits); out likewise with ldo.
 *       Tokens outside [offsets[0], offsets[B]) are not written.
 *   k_cache, v_cache [S][Hk][D] E4M3 codes; k_scale, v_scale [Hk] FP32.
 *   table [B][width] int32, offsets [B+1] int64 (non-decreasing), lengths [B]
 *       int32 (jet_kv_slot_map's cached + added): DEVICE arrays.
 *   prefix_offsets [n_prefix+1] int64 (non-decreasing), prefix_lengths
 *       [n_prefix] int32: DEVICE arrays, or NULL with n_prefix = 0.
 *   lse [T][Hq] FP32 (out), or NULL.
 *   ws / ws_bytes: at least jet_kv_attention_workspace() bytes of device
 *       memory; scratch, not initialised.
 * 0 <= T < 2^24, T*Hq < 2^31; Hq <= 1024, a multiple of Hk; D = 64, 128 or 256; B <= 8192;
 * n_prefix <= B; S, width < 2^31; 1 <= block_size < 2^30; scale > 0; strides
 * >= Hq*D and multiples of 8.
 */
JET_API jet_status jet_kv_attention(const uint16_t *q, int64_t ldq, int64_t T, int64_t Hq,
                                    int64_t Hk, int64_t D, const uint8_t *k_cache,
                                    const uint8_t *v_cache, int64_t S, const float *k_scale,
                                    const float *v_scale, const int32_t *table, int64_t width,
                                    int64_t block_size, const int64_t *offsets,
                                    const int32_t *lengths, int64_t B,
                                    const int64_t *prefix_offsets, const int32_t *prefix_lengths,
                                    int64_t n_prefix, float scale, uint16_t *out, int64_t ldo,
                                    float *lse, void *ws, size_t ws_bytes, jet_stream_t stream);

/* Workspace bytes of jet_kv_attention (0 for sizes it refuses).  Host function. */
JET_API size_t jet_kv_attention_workspace(int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t B,
                                          int64_t n_prefix);

/*
 * Backward of the SwiGLU of jet_swiglu_quant_1x128 (the quantization passes
 * gradients straight through), its two gradients quantized for the DGrads of the
 * gate and up projections.  With s = 1 / (1 + e^-gate) in binary32:
 *   dup = dh gate s,  dgate = dh up s (1 + gate (1 - s)),
 * within a few 2^-22 relative (s below 2^-126 counts as 0); the 1x128 group rule applies to the binary32
 * values.  The 128x1 forms for the WGrads come from jet_requant_128x1, as for
 * every other operand.
 *   gate, up [M][F] BF16 bits (in) with row stride ld (two halves of a gate_up
 *       product, or two dense tensors with ld = F).
 *   dh [M][F] BF16 bits (in; the down projection's DGrad), dense.
 *   qg, qu [M][F] E4M3 codes, sg, su [F/128][M] FP32 scales (out) of dgate, dup.
 * M, F >= 0, F a multiple of 128, ld >= F a multiple of 8.
 */
JET_API jet_status jet_swiglu_bwd_quant_1x128(const uint16_t *gate, const uint16_t *up, int64_t ld,
                                              const uint16_t *dh, int64_t M, int64_t F, uint8_t *qg,
                                              float *sg, uint8_t *qu, float *su,
                                              jet_stream_t stream);

/*
 * Log-probabilities of given tokens under the head, without its logits: the
 * logp_train of the mismatch metric and of a policy or cross-entropy loss.
 *   z_tv = scale (x_t . w_v),  lse_t = ln sum_v e^z_tv,
 *   logp_t = z_t,target[t] - lse_t,
 * products of BF16 values with binary32 sums, exponentials and sums in binary32;
 * the vocabulary is walked in tiles, each row's maxima and sums joined in a fixed
 * order.  A target outside [0, V) is ignored: logp 0 (lse is still that row's).
 *   x [T][K] BF16 bits (in; the final norm's output), w [V][K] BF16 bits (in;
 *       the head), target [T] int64 (in).
 *   scale: 1, or 1 / temperature.
 *   logp, lse [T] FP32 (out).
 *   ws / ws_bytes: at least jet_workspace_bytes(JET_OP_HEAD_LOGP, T, V, K) bytes
 *       of device memory; scratch, not initialised.
 * 0 <= T < 2^22; 1 <= V < 2^24; 8 <= K <= 65536, a multiple of 8; scale > 0.
 */
JET_API jet_status jet_head_logp(const uint16_t *x, const uint16_t *w, int64_t T, int64_t K,
                                 int64_t V, const int64_t *target, float scale, float *logp,
                                 float *lse, void *ws, size_t ws_bytes, jet_stream_t stream);

/*
 * Gradients of sum_t dlogp_t logp_t (any loss of the logp is written so by its
 * dlogp: -1/T for the mean cross entropy):
 *   d_tv = scale dlogp_t ([v = target[t]] - e^(z_tv - lse_t)), 0 for ignored rows,
 *   dx = d w,  dw = d^T x.
 * The logits are computed again, by the same sums as in jet_head_logp and a piece
 * of the vocabulary at a time (at most 512 MB of d, 4096 entries at least); d is rounded to BF16 (2^-8 of each
 * value; in two parts, 2^-16, for up to 128 tokens), sums are binary32 (the tensor
 * core's, which cuts off up to 2^-23 of a sum every 16 terms: dw over T tokens, dx
 * over a range of the vocabulary), dx and dw rounded once to BF16.
 *   x, w, target, scale, lse: as in and from jet_head_logp.  dlogp [T] FP32 (in;
 *       not read for ignored rows).
 *   dx [T][K], dw [V][K] BF16 bits (out); either may be NULL.  dw is zeros for
 *       T = 0.
 *   ws / ws_bytes: at least jet_workspace_bytes(JET_OP_HEAD_LOGP_BWD, T, V, K)
 *       bytes of device memory; scratch, not initialised.
 */
JET_API jet_status jet_head_logp_bwd(const uint16_t *x, const uint16_t *w, int64_t T, int64_t K,
                                     int64_t V, const int64_t *target, const float *lse,
                                     const float *dlogp, float scale, uint16_t *dx, uint16_t *dw,
                                     void *ws, size_t ws_bytes, jet_stream_t stream);

/*
 * Workspace bytes an operation needs for the given sizes (0 if none).
 * For JET_OP_TOKEN_MULT_PROB_ERROR and JET_OP_TOKEN_MISMATCH_MASKED pass n as M.  Returns 0 for negative sizes
 * or an unknown op.  Pure host function; needs no device.
 */
JET_API size_t jet_workspace_bytes(int op, int64_t M, int64_t N, int64_t K);

/*
 * Synchronizes `stream`, then reads and clears the device-side status word of
 * the current device.  Returns JET_OK, JET_ERR_TIMEOUT (a bounded wait inside
 * a kernel gave up; the kernel skipped its remaining work and released its
 * resources, so the context stays usable) or JET_ERR_CUDA (the synchronize
 * itself failed).  If `detail` is not NULL it receives the raw status word
 * (0 when clean; otherwise the code in the low byte and the wait site above).
 */
JET_API jet_status jet_device_status(jet_stream_t stream, uint32_t *detail);

/*
 * Self-test of the failure path every pipelined kernel uses: launches one
 * block that waits on a barrier nothing completes, with a limit of
 * `limit_us` microseconds at the maximum SM clock (1 .. 1,000,000; the wait
 * is counted in SM cycles, so it lasts longer at lower clocks).  The wait gives up, records
 * JET_ERR_TIMEOUT in the device status word and the kernel returns, so a
 * following jet_device_status() reports JET_ERR_TIMEOUT and the context stays
 * usable.  The pages have no counterpart; it exists to test the bounded waits.
 */
JET_API jet_status jet_selftest_bounded_wait(uint32_t limit_us, jet_stream_t stream);

/*
 * Self-test of the GEMM's own failure path: runs the forward product
 * Y = X W^T (same operands and layouts as jet_gemm_fp8_fwd, M <= 128 tokens,
 * on the single-CTA tensor-core kernel, contraction not split) with every
 * pipeline wait limited to `limit_cycles` SM cycles (1 .. 4e9; the library's
 * GEMMs use 4e9, about 2 s).  With a limit shorter than the first operand
 * load, a role of the kernel gives up: it records JET_ERR_TIMEOUT and its wait
 * site (1 producer, 2 MMA issuer waiting for operands, 3 MMA issuer waiting
 * for an accumulator, 4 promotion warps) in the device status word and sets
 * the CTA's abort flag; the other roles stop at their next wait, the producer
 * waits for its loads in flight, the MMA issuer for its MMAs, TMEM is freed
 * and the kernel returns, so jet_device_status() reports JET_ERR_TIMEOUT and
 * the context stays usable.  Y is then unspecified.  Same argument checks as
 * jet_gemm_fp8_fwd, plus M <= 128 and the limit's range (JET_ERR_SHAPE).
 * The pages have no counterpart; it exists to test the bounded waits.
 */
JET_API jet_status jet_selftest_gemm_timeout(const uint8_t *qx, const float *sx,
                                             const uint8_t *qw, const float *sw, int64_t M,
                                             int64_t N, int64_t K, uint16_t *y,
                                             uint64_t limit_cycles, jet_stream_t stream);

/*
 * Self-test of the division the quantizers use: q[i] = x[i] / s[i] computed
 * exactly as a quantizer divides a value x by its group scale s (a
 * reciprocal of s shared by the group and Markstein's correction steps).  It
 * equals the IEEE binary32 quotient whenever s >= 2^-90 and |x/s| >= 2^-11,
 * and for every pair when s < 2^-90; smaller quotients agree in sign and lie
 * below 2^-10, so their E4M3 codes are the same.  x, s, q: [n] FP32 device
 * arrays.  The pages have no counterpart; it exists to test that division.
 */
JET_API jet_status jet_selftest_quotient(const float *x, const float *s, int64_t n, float *q,
                                         jet_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* JET_FP8_H */
