/*
 * nvfp4_w4a16.h -- C ABI of the NVFP4 W4A16 lm_head library for MI355X (gfx950).
 *
 * Three calls: quantize a bf16 lm_head weight to NVFP4, re-quantize it in
 * place into the same buffers, and compute logits from the quantized weight
 * with bf16 activations.  Two more adopt a pre-quantized NVFP4 checkpoint
 * (ModelOpt or compressed-tensors) for the same GEMM.  Everything runs in
 * hand-written HIP kernels.
 *
 * The method is the one the vLLM API docs describe for
 * vllm.model_executor.layers.quantization.online.lm_head (function
 * _quantize_nvfp4, class _LMHeadNvfp4Method, refresh_quantized_lm_heads).
 *
 * Conventions shared by every call
 * --------------------------------
 *  - Every pointer is a DEVICE pointer on the current HIP device, except where
 *    stated.  bf16 tensors are passed as raw 16-bit words (bfloat16 bits).
 *  - All matrices are row-major and dense (row pitch = number of columns).
 *  - The caller owns every buffer; the library allocates nothing and keeps no
 *    state between calls, so calls are reentrant and can be captured into a
 *    HIP graph.
 *  - `stream` is a hipStream_t passed as void* (NULL = the null stream).  Each
 *    call only enqueues work on it: no host<->device synchronisation.
 *  - Arguments are validated on the host before any HIP API call.  A non-zero
 *    status means nothing was enqueued, except NVFP4_ERR_LAUNCH, which reports
 *    a HIP error raised while enqueueing (see nvfp4_last_hip_error()).
 *  - Device faults surface as HIP errors at the caller's next synchronisation.
 *  - Alignment: W, x and y must be 16-byte aligned; packed 16-byte aligned;
 *    scales 4-byte aligned (16-byte for the two checkpoint calls);
 *    global_scale, flags and partition scales 4-byte aligned; bias 2-byte
 *    aligned.
 *  - Outputs may not overlap inputs or each other (NVFP4_ERR_ALIAS).
 *  - Non-finite weights are outside the contract (results unspecified).
 */
#ifndef NVFP4_W4A16_H_
#define NVFP4_W4A16_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  NVFP4_OK = 0,
  NVFP4_ERR_NULL = 1,   /* a required pointer is NULL                                   */
  NVFP4_ERR_SHAPE = 2,  /* N < 1, K < 16, K % 16 != 0, M < 0, or a size too large       */
  NVFP4_ERR_ALIGN = 3,  /* a pointer breaks the alignment rules above                   */
  NVFP4_ERR_ALIAS = 4,  /* an output byte range overlaps an input or another output     */
  NVFP4_ERR_LAUNCH = 5, /* HIP reported an error while enqueueing                        */
  NVFP4_ERR_ARG = 6,    /* an enumerated argument (e.g. a scale convention) is out of range */
  NVFP4_ERR_SCRATCH = 7 /* the call needs more scratch than the library's static array holds */
} nvfp4_status;

/* Group size along K: one E4M3 scale per 16 consecutive weights of a row
 * (vLLM modelopt.py, ModelOptNvFp4Config default group size; vLLM API docs,
 * compressed_tensors.schemes, CompressedTensorsW4A16Fp4). */
#define NVFP4_GROUP 16

/*
 * nvfp4_quantize -- online NVFP4 quantization of a bf16 weight.
 * (vLLM API docs, quantization.online.lm_head, _quantize_nvfp4.)
 *
 *   W            in   bf16 [N, K]                the weight (e.g. a vocab shard of lm_head)
 *   N, K         in   N >= 1 rows, K >= 16 columns, K % 16 == 0 (vLLM modelopt.py,
 *                     KNvfp4Static rejects other K)
 *   packed       out  uint8 [N, K/2]            E2M1 codes, two per byte, the even-k code
 *                                               in the low nibble; bit 3 of a code = sign
 *   scales       out  float8_e4m3fn bytes [N, K/16]   block scale of W[n, 16j : 16j+16]
 *   global_scale out  1 float                   max(amax(|W|) / (6 * 448), 1e-12): the
 *                                               dequantization-direction global scale
 *                                               (ModelOpt's amax/2688, per modelopt.py
 *                                               KNvfp4Static.process)
 *
 * Dequantization: w[n,k] ~= E2M1(code[n,k]) * e4m3(scales[n,k/16]) * global_scale.
 * Per block: u = min((max|w| / 6) * (1/global_scale), 448) rounded to E4M3
 * (nearest-even); each weight is multiplied by (1/global_scale)/scale and
 * rounded to the E2M1 grid {0,.5,1,1.5,2,3,4,6} (nearest, ties to the even
 * code, saturating at 6).  A zero block has scale 0 and codes 0; zero never
 * carries a sign.  The global_scale word also serves as the amax accumulator
 * while the call runs, so the outputs are only valid once the stream reaches
 * the end of the call.
 */
nvfp4_status nvfp4_quantize(const void* W, int64_t N, int64_t K,
                            uint8_t* packed, uint8_t* scales, float* global_scale,
                            void* stream);

/*
 * nvfp4_refresh_inplace -- re-derive the quantized copy from an updated weight.
 * (vLLM API docs, quantization.online.lm_head, refresh_quantized_lm_heads: the
 * copy is rewritten in place so that captured graphs keep valid pointers.)
 *
 * Same arguments, computation and result as nvfp4_quantize, into buffers that
 * already hold a quantization of a weight of the same (N, K).  It writes only
 * the bytes of packed, scales and global_scale, allocates nothing and uses no
 * memset nodes, so a HIP graph that captured nvfp4_w4a16_gemm on these
 * pointers reads the new values on its next replay.  A refresh that overlaps
 * a GEMM reading the same buffers on another stream is the caller's race.
 */
nvfp4_status nvfp4_refresh_inplace(const void* W, int64_t N, int64_t K,
                                   uint8_t* packed, uint8_t* scales, float* global_scale,
                                   void* stream);

/*
 * nvfp4_w4a16_gemm -- logits from bf16 activations and the NVFP4 weight.
 * (vLLM API docs, quantization.online.lm_head, _LMHeadNvfp4Method.apply:
 * weight-only NVFP4, activations stay in the model dtype.)
 *
 *   x            in   bf16 [M, K]     activations; M >= 0 (M == 0 enqueues nothing, and
 *                                    x and y may then be NULL)
 *   packed, scales, global_scale in  as produced by nvfp4_quantize for [N, K]
 *   N            in   N >= 1
 *   bias         in   bf16 [N] or NULL
 *   y            out  bf16 [M, N]
 *
 *   y[m, n] = bf16_rne( global_scale * sum_k x[m,k] * E2M1(code[n,k]) * e4m3(scale[n,k/16])
 *                       + bias[n] )
 * with fp32 accumulation; summation order is unspecified but deterministic.
 * The dequantized weight E2M1 * e4m3 is exact (at most 6 significant bits).
 * M <= 64 runs the streaming decode kernels, larger M the MFMA prefill kernel.
 *
 * Products: the prefill kernel and most decode kernels multiply the bf16
 * activations as given, so every product is exact in fp32.  The decode
 * kernels for 3 <= M <= 16 that hold the activation in LDS, whole (K a
 * multiple of 256 and M * (2K + 16) bytes small enough) or one range of K/2,
 * K/4 or K/8 columns (a multiple of 1024) at a time, stage each activation
 * row m in f16 as x * 2^-p_m, with the power of two chosen from the whole
 * row's largest magnitude so that it lands in [2^14, 2^15), and multiply the
 * f16 results by 2^p_m in fp32.  An activation with |x| >= 2^-28 * max_k |x[m,k]| converts
 * exactly (bf16's 8 significant bits fit f16's 11); a smaller one may move by
 * at most max(2^-39 * max_k |x[m,k]|, 2^-151), half the f16 subnormal spacing
 * at that scale.  Each y[m, n] may therefore differ from the exact-product
 * sum by at most that bound times sum_k |w[n,k]| before the fp32 summation
 * and bf16 rounding errors; no other rounding enters.
 */
nvfp4_status nvfp4_w4a16_gemm(const void* x, int64_t M, int64_t K,
                              const uint8_t* packed, const uint8_t* scales,
                              const float* global_scale, int64_t N,
                              const void* bias, void* y, void* stream);

/*
 * Pre-quantized checkpoints.
 * (vLLM modelopt.py, class KNvfp4Static, create_weights and process; vLLM API
 * docs, compressed_tensors.schemes, class CompressedTensorsW4A16Fp4,
 * create_weights and process_weights_after_loading.)
 *
 * Both formats store the packed codes as uint8 [N, K/2] and the block scales
 * as float8_e4m3fn [N, K/16] exactly as nvfp4_quantize writes them, so
 * nvfp4_w4a16_gemm reads them as loaded.  They differ in the per-partition
 * global scale (one float per fused output partition, e.g. 1 for lm_head):
 */
typedef enum {
  /* weight_scale_2 = amax / 2688 (the dequantization direction); the global
   * scale is the largest of them, used as is */
  NVFP4_SCALE2_MODELOPT = 0,
  /* weight_global_scale = 2688 / amax, stored inverted; the global scale is
   * 1 / (the largest of them), one IEEE float32 division */
  NVFP4_SCALE2_COMPRESSED_TENSORS = 1
} nvfp4_scale2_convention;

/* Bits of the flags word nvfp4_import_checkpoint writes. */
#define NVFP4_IMPORT_SCALES_NOT_LOADED 1u   /* a block scale is an e4m3fn NaN (0x7F or 0xFF)      */
#define NVFP4_IMPORT_PARTITIONS_DIFFER 2u   /* the partition scales are not all equal (IEEE ==),   */
                                            /* which costs accuracy: one global scale serves all   */
#define NVFP4_IMPORT_BAD_GLOBAL_SCALE  4u   /* the global scale is not a finite number > 0         */

/*
 * nvfp4_fill_scale_sentinel -- mark a block-scale buffer as not loaded.
 *
 *   scales  out  float8_e4m3fn bytes [N, K/16], 16-byte aligned; every byte is
 *                set to 0x7F (an e4m3fn NaN), the sentinel KNvfp4Static
 *                creates its weight_scale with
 *   N, K    in   the weight's shape (rules of nvfp4_quantize)
 *
 * Call it on a freshly allocated buffer before the checkpoint loader fills
 * it, so that nvfp4_import_checkpoint can tell which scales were never loaded.
 */
nvfp4_status nvfp4_fill_scale_sentinel(uint8_t* scales, int64_t N, int64_t K, void* stream);

/*
 * nvfp4_import_checkpoint -- the GEMM's global scale from a checkpoint, and a
 * check of its block scales.
 *
 *   partition_scales in  float [num_partitions], 4-byte aligned: the stored
 *                        per-partition global scales, in `convention`
 *   num_partitions   in  1 .. 2^20
 *   convention       in  an nvfp4_scale2_convention (else NVFP4_ERR_ARG)
 *   scales           in  float8_e4m3fn bytes [N, K/16] as loaded, 16-byte aligned
 *   N, K             in  the weight's shape (rules of nvfp4_quantize)
 *   global_scale     out 1 float: what nvfp4_w4a16_gemm takes as global_scale
 *                        (a NaN result is written as the quiet NaN 0x7FC00000)
 *   flags            out 1 uint32: NVFP4_IMPORT_* bits
 *
 * The library only reports: a caller that follows KNvfp4Static rejects the
 * tensor when NVFP4_IMPORT_SCALES_NOT_LOADED is set and warns on
 * NVFP4_IMPORT_PARTITIONS_DIFFER.  Both outputs are valid once the stream
 * reaches the end of the call; no output may overlap an input or the other
 * output.  The partition scales are read once, the block scales once
 * (N*K/16 bytes).
 */
nvfp4_status nvfp4_import_checkpoint(const float* partition_scales, int64_t num_partitions, int convention,
                                     const uint8_t* scales, int64_t N, int64_t K, float* global_scale,
                                     uint32_t* flags, void* stream);

/*
 * The FP8 lm_head copy.
 * (vLLM API docs, quantization.online.lm_head, quantized_lm_head_copy: the
 * "fp8" copy uses per-row weight scales and per-token activation scales on
 * an FP8 linear kernel; vLLM modelopt.py, KFp8StaticChannel and the
 * FP8_PER_CHANNEL_PER_TOKEN recipe; vLLM API docs, compressed_tensors.schemes,
 * the W8A8 FP8 apply_weights path.)
 *
 * nvfp4_fp8_quantize_rows -- row-wise E4M3 quantization of a bf16 matrix;
 * quantizes the weight once (one scale per output row) and the activations
 * at every call (one scale per token).
 *
 *   A           in   bf16 [R, K], 16-byte aligned (R >= 1, K >= 16, K % 16 == 0)
 *   q           out  float8_e4m3fn bytes [R, K], 16-byte aligned
 *   row_scales  out  float [R]
 *
 *   s[r] = max(max_k |A[r,k]| / 448, 1e-12)     (float32, one IEEE division)
 *   q[r,k] = e4m3_rne(clamp(A[r,k] * (1 / s[r]), -448, 448)), sign kept
 *
 * The pages do not show the quantizer's arithmetic; this is the plainest
 * reading (the clamp mirrors the NVFP4 global scale's).
 */
nvfp4_status nvfp4_fp8_quantize_rows(const void* A, int64_t R, int64_t K, uint8_t* q, float* row_scales,
                                     void* stream);

/*
 * nvfp4_fp8_gemm -- logits from the FP8 copy.
 *
 *   xq, x_scales in  float8_e4m3fn [M, K] and float [M] from nvfp4_fp8_quantize_rows (M >= 0;
 *                    M == 0 enqueues nothing, and xq, x_scales and y may then be NULL)
 *   wq, w_scales in  float8_e4m3fn [N, K] and float [N], likewise
 *   bias         in  bf16 [N] or NULL
 *   y            out bf16 [M, N], 16-byte aligned
 *
 *   y[m, n] = bf16_rne(x_scales[m] * w_scales[n] * sum_k e4m3(xq[m,k]) * e4m3(wq[n,k]) + bias[n])
 * with float32 accumulation of exact float32 products.
 */
nvfp4_status nvfp4_fp8_gemm(const uint8_t* xq, const float* x_scales, int64_t M, int64_t K, const uint8_t* wq,
                            const float* w_scales, int64_t N, const void* bias, void* y, void* stream);

/*
 * NVFP4 W4A4: activations quantized to NVFP4 at run time with a static global
 * input scale, and the GEMM of the two NVFP4 operands.
 * (vLLM modelopt.py, KNvfp4Dynamic, maybe_fuse_global_scales and the NVFP4
 * recipe: static FP4 weight, dynamic FP4 activation, alpha =
 * input_global_scale * weight_global_scale.)
 *
 * nvfp4_quantize_activations -- x bf16 [M, K] (16-byte aligned) -> packed
 * uint8 [M, K/2] and float8_e4m3fn scales [M, K/16], with the rules of
 * nvfp4_quantize but the given input_global_scale (1 float on the device, the
 * dequantization direction, e.g. the max of a checkpoint's input_scale; it
 * must be a finite number > 0) in place of amax/2688.  Nothing is written to
 * input_global_scale.
 */
nvfp4_status nvfp4_quantize_activations(const void* x, int64_t M, int64_t K, const float* input_global_scale,
                                        uint8_t* packed, uint8_t* scales, void* stream);

/*
 * nvfp4_w4a4_workspace_bytes -- size of nvfp4_w4a4_gemm's workspace: 2*M*K + 16
 * (host helper, no device work; 0 for negative sizes).
 */
int64_t nvfp4_w4a4_workspace_bytes(int64_t M, int64_t K);

/*
 * nvfp4_w4a4_gemm -- logits from NVFP4 activations and the NVFP4 weight.
 *
 *   x_packed, x_scales   in  from nvfp4_quantize_activations, [M, K/2] / [M, K/16]
 *   input_global_scale   in  the global scale they were quantized with (1 float)
 *   packed, scales, global_scale, N, bias   in  as for nvfp4_w4a16_gemm
 *   workspace            tmp device buffer of nvfp4_w4a4_workspace_bytes(M, K) bytes,
 *                            16-byte aligned, overlapping nothing else; it holds the
 *                            activations' exact bf16 values code * block scale, then
 *                            alpha, and may be reused once the stream is past the call
 *   y                    out bf16 [M, N]
 *
 *   y[m, n] = bf16_rne( alpha * sum_k (E2M1(cx) * e4m3(sx)) * (E2M1(cw) * e4m3(sw)) + bias[n] ),
 *   alpha = fl32(input_global_scale * global_scale), float32 accumulation of exact products.
 * M == 0 enqueues nothing (the activation pointers, workspace and y may then be NULL).
 */
nvfp4_status nvfp4_w4a4_gemm(const uint8_t* x_packed, const uint8_t* x_scales, const float* input_global_scale,
                             int64_t M, int64_t K, const uint8_t* packed, const uint8_t* scales,
                             const float* global_scale, int64_t N, const void* bias, void* workspace, void* y,
                             void* stream);

/*
 * nvfp4_w4a4_gemm_noalloc -- nvfp4_w4a4_gemm without a workspace argument and
 * without any allocation, for callers that cannot allocate device memory
 * (code being captured into a HIP graph, tight serving loops, harnesses that
 * forbid hipMalloc).
 *
 * Same arguments (minus `workspace`), computation, result and errors as
 * nvfp4_w4a4_gemm.  The workspace lives in a static device array of
 * NVFP4_W4A4_SCRATCH_BYTES bytes that the library holds on each GPU it runs
 * on until the process ends; calls whose workspace
 * (nvfp4_w4a4_workspace_bytes(M, K) = 2*M*K + 16 bytes, i.e. M*K <= 2097144)
 * would not fit return NVFP4_ERR_SCRATCH and enqueue nothing.  All calls on
 * one GPU share that array: calls that may overlap on one GPU (other streams,
 * other host threads) race and must be serialised by the caller.  The first
 * call on a device looks up the array's address on that device (no
 * allocation); every call writes the whole region it reads before reading it.
 */
#define NVFP4_W4A4_SCRATCH_BYTES (4 << 20)
nvfp4_status nvfp4_w4a4_gemm_noalloc(const uint8_t* x_packed, const uint8_t* x_scales,
                                     const float* input_global_scale, int64_t M, int64_t K,
                                     const uint8_t* packed, const uint8_t* scales, const float* global_scale,
                                     int64_t N, const void* bias, void* y, void* stream);

/*
 * Mixture of experts, W4A16 NVFP4 (vLLM modelopt.py, ModelOptNvFp4FusedMoE with
 * use_a16: per-expert NVFP4 weights w13 [E, 2I, H/2] / scales [E, 2I, H/16] and
 * w2 [E, H, I/2] / scales [E, H, I/16], one float32 global scale per expert and
 * matrix -- for w13 the w1 column of w13_weight_scale_2 -- and routing by
 * topk_ids / topk_weights as apply() receives them).
 *
 * Pair p = t * topk + j is token t's j-th routed expert topk_ids[t * topk + j].
 * A pair whose id lies outside [0, E) is outside the contract: it is counted
 * into *invalid_pairs (when non-NULL) and its GEMM output row is zero.
 *
 * nvfp4_moe_gemm_workspace_bytes -- workspace of nvfp4_moe_w4a16_gemm: the
 * routing table, 4 * (round_up(E + 2, 4) + round_up(P, 4)) bytes (host helper;
 * 0 for P < 0 or E < 1).
 */
int64_t nvfp4_moe_gemm_workspace_bytes(int64_t P, int64_t E);

/*
 * nvfp4_moe_w4a16_gemm -- the grouped expert GEMM:
 *   y[p, n] = bf16_rne( gs[e] * sum_k x[p / row_div, k] * E2M1(code_e[n, k]) * e4m3(scale_e[n, k/16]) ),
 *   e = topk_ids[p], float32 accumulation of exact products.
 *
 *   x              in  bf16 [x_rows, K]; row_div = topk reads token rows (the first
 *                      GEMM), row_div = 1 reads one row per pair (the second);
 *                      x_rows >= ceil(P / row_div)
 *   topk_ids       in  int32 [P]
 *   packed, scales in  [E, N, K/2] uint8 / [E, N, K/16] e4m3fn, the per-expert layout
 *                      of the pages (packed 16-byte aligned)
 *   global_scales  in  float32 [E]
 *   workspace      tmp nvfp4_moe_gemm_workspace_bytes(P, E) bytes, 16-byte aligned
 *   y              out bf16 [P, N]
 *   invalid_pairs  out optional uint32 (NULL = not reported)
 * An expert with no pair reads none of its weights.  P == 0 enqueues nothing.
 */
nvfp4_status nvfp4_moe_w4a16_gemm(const void* x, int64_t x_rows, int64_t K, const int32_t* topk_ids, int64_t P,
                                  int64_t row_div, const uint8_t* packed, const uint8_t* scales,
                                  const float* global_scales, int64_t E, int64_t N, void* workspace, void* y,
                                  uint32_t* invalid_pairs, void* stream);

/*
 * nvfp4_moe_silu_and_mul -- a[p, i] = bf16_rne( silu(h[p, i]) * h[p, I + i] ),
 * silu(g) = g / (1 + exp(-g)) in float32: the act-and-mul layout [w1; w3] of
 * w13.  h bf16 [P, 2I], a bf16 [P, I], I % 8 == 0, both 16-byte aligned.
 */
nvfp4_status nvfp4_moe_silu_and_mul(const void* h, int64_t P, int64_t I, void* a, void* stream);

/*
 * nvfp4_moe_combine -- out[t, n] = bf16_rne( sum_j topk_weights[t, j] * o[t * topk + j, n] ),
 * float32 in slot order j = 0, 1, ...  o bf16 [T * topk, H], topk_weights float32
 * [T, topk], out bf16 [T, H], H % 8 == 0, o and out 16-byte aligned.
 */
nvfp4_status nvfp4_moe_combine(const void* o, const float* topk_weights, int64_t T, int64_t topk, int64_t H,
                               void* out, void* stream);

/*
 * nvfp4_moe_workspace_bytes -- workspace of nvfp4_moe_w4a16_forward: the routing
 * table, then h [P, 2I], a [P, I] and o [P, H] in bf16, each rounded up to 256 bytes
 * (host helper; 0 for invalid sizes).
 *
 * nvfp4_moe_w4a16_forward -- the whole W4A16 expert layer on bf16 x [T, H]:
 * routing, h = grouped GEMM with w13, a = silu_and_mul(h), o = grouped GEMM
 * with w2, out = combine(o, topk_weights); each stage as the calls above, h, a
 * and o rounded to bf16.  out bf16 [T, H].  T == 0 enqueues nothing.
 */
int64_t nvfp4_moe_workspace_bytes(int64_t T, int64_t topk, int64_t E, int64_t H, int64_t I);
nvfp4_status nvfp4_moe_w4a16_forward(const void* x, int64_t T, int64_t H, const int32_t* topk_ids,
                                     const float* topk_weights, int64_t topk, const uint8_t* w13_packed,
                                     const uint8_t* w13_scales, const float* w13_global_scales,
                                     const uint8_t* w2_packed, const uint8_t* w2_scales,
                                     const float* w2_global_scales, int64_t E, int64_t I, void* workspace,
                                     void* out, uint32_t* invalid_pairs, void* stream);

/*
 * The whole W4A16 expert layer for a few tokens, from the router's logits.
 *
 * nvfp4_moe_decode_workspace_bytes -- workspace of nvfp4_moe_w4a16_decode
 * (host helper; 0 for sizes the call rejects).
 *
 * nvfp4_moe_w4a16_decode -- routing, both expert products, SiLU-and-mul and the
 * weighted sum in two kernels, for 0 <= T <= 16 tokens (T == 0 enqueues nothing):
 *   score[t, e] = softmax over e or sigmoid of router_logits[t, e]
 *   topk_ids[t] = the topk experts of largest logit -- of largest score + correction_bias
 *                 where a bias is given -- equal ones by the lower index
 *   topk_weights[t, j] = score[t, e_j] (/ their sum over j, with renormalize) * weight_scale
 *   a[t, j] = silu(g) * u,  g = w1_e x[t],  u = w3_e x[t]        (w13 rows 0..I, I..2I)
 *   out[t] = bf16_rne( sum_j topk_weights[t, j] * w2_e a[t, j] )
 * float32 sums of exact products.  Where H and I are multiples of 32 from 64 on, the
 * activations enter the products as 11-bit floats scaled by powers of two: x
 * unchanged, a as a pair of them that keeps 20 bits (of either, what is below 2^-28
 * of the largest value near it loses bits); with other sizes x is unchanged and a is
 * kept to 16 bits (a bf16 pair).  The only other rounding is out's to bf16.  A chosen expert's weights are read once, the others' not
 * at all.  An expert whose logit is -inf or NaN is never chosen; a slot left
 * without an expert has id -1, weight 0 and adds nothing.
 *
 *   x               in  bf16 [T, H], 16-byte aligned
 *   router_logits   in  router_dtype (NVFP4_F32 or NVFP4_BF16) [T, E], 1 <= E <= 1024
 *   topk            in  1 .. min(E, 32)
 *   scoring         in  an nvfp4_moe_scoring
 *   renormalize     in  0 or 1
 *   correction_bias in  float [E] or NULL (it moves the choice, not the weights)
 *   weight_scale    in  factor of every weight (1 = none)
 *   w13_*, w2_*     in  as for nvfp4_moe_w4a16_forward (w2_packed and w13_packed 16-byte aligned)
 *   workspace       tmp nvfp4_moe_decode_workspace_bytes(T, topk, E, H, I) bytes, 16-byte aligned;
 *                       its contents need no preparation
 *   out             out bf16 [T, H], 16-byte aligned
 *   topk_ids, topk_weights   out  int32 / float [T, topk], each optional (NULL)
 */
typedef enum {
  NVFP4_MOE_SOFTMAX = 0,
  NVFP4_MOE_SIGMOID = 1
} nvfp4_moe_scoring;
int64_t nvfp4_moe_decode_workspace_bytes(int64_t T, int64_t topk, int64_t E, int64_t H, int64_t I);
nvfp4_status nvfp4_moe_w4a16_decode(const void* x, int64_t T, int64_t H, const void* router_logits,
                                    int router_dtype, int64_t E, int64_t topk, int scoring, int renormalize,
                                    const float* correction_bias, float weight_scale, const uint8_t* w13_packed,
                                    const uint8_t* w13_scales, const float* w13_global_scales,
                                    const uint8_t* w2_packed, const uint8_t* w2_scales,
                                    const float* w2_global_scales, int64_t I, void* workspace, void* out,
                                    int32_t* topk_ids, float* topk_weights, void* stream);

/*
 * int4 weights with group scales.
 * (vLLM API docs, compressed_tensors.schemes, class CompressedTensorsWNA16,
 * 4 bits without activation reordering.)
 *
 * nvfp4_int4_gemm -- logits from bf16 activations and an int4 weight, for few
 * activation rows:
 *   y[m, n] = bf16_rne( sum_j scale[n, j] * sum_{k in group j} x[m, k] * (code[n, k] - zero[n, j]) + bias[n] )
 * The sums are float32 over exact products (a group's sum holds
 * sum x * (16 + code) and -(16 + zero) * sum x, so a non-finite activation makes
 * its row non-finite, and so may finite ones whose sum passes float32 / 31); summation order is unspecified but deterministic.
 *
 *   x            in  bf16 [M, K], 16-byte aligned; M >= 0 (M == 0 enqueues nothing, x and y may
 *                    then be NULL).  Beyond 64 rows the weight is read once per 64 rows.
 *   packed       in  int32 [N, K / 8], 16-byte aligned: code k of a row is bits 4 (k % 8) .. + 3 of word
 *                    k / 8, in 0 .. 15
 *   scales       in  scale_dtype (NVFP4_BF16 or NVFP4_F16) [N, K / group]
 *   zero_points  in  int32 [ceil(N / 8), K / group] or NULL (zero = 8): row n's is bits
 *                    4 (n % 8) .. + 3 of word [n / 8, j]
 *   group        in  32, 64, a multiple of 128, or K (one scale per row); K % group == 0 and
 *                    K % 32 == 0
 *   bias         in  bf16 [N] or NULL
 *   y            out bf16 [M, N], 16-byte aligned
 */
nvfp4_status nvfp4_int4_gemm(const void* x, int64_t M, int64_t K, const int32_t* packed, const void* scales,
                             int scale_dtype, const int32_t* zero_points, int64_t group, int64_t N,
                             const void* bias, void* y, void* stream);

/*
 * Log probabilities of given tokens, from the logits a GEMM above wrote (or
 * any other logits).
 *
 * Row i holds V logits of type `dtype` at logits + i * row_stride elements
 * (row_stride >= V; rows need only the element's own alignment).  With
 * z[i, j] = logits[i, j] / temperature[i] over the allowed tokens of the row:
 *   lse[i]            = log sum_j exp(z[i, j])
 *   token_logprobs[i] = z[i, id] - lse[i],  id = token_ids[i]
 *   token_ranks[i]    = 1 + (how many allowed logits of the row are larger than the token's)
 *   entropy[i]        = -sum_j p[i, j] log p[i, j],  p = exp(z - lse)
 *   top_ids[i, 0..topk), top_logprobs: the largest allowed logits in falling
 *                       order, equal ones in the order of their index
 * All sums are float32 (per lane, then joined pairwise); selection and ranks
 * compare the logits themselves, exactly (-0 equals 0).  The outputs do not
 * depend on timing: the same call gives the same bits.
 */
typedef enum {
  NVFP4_BF16 = 0,
  NVFP4_F16 = 1,
  NVFP4_F32 = 2
} nvfp4_dtype;

/*
 * nvfp4_logprobs_workspace_bytes -- workspace of nvfp4_logprobs (host helper;
 * at least 16; 0 for sizes the call rejects).
 *
 * nvfp4_logprobs
 *   logits         in  dtype [M, V] rows of row_stride elements, aligned to the element
 *   M, V           in  0 <= M <= 2^23 (M == 0 enqueues nothing), 1 <= V <= 2^30
 *   token_ids      in  optional int32 [M] (NULL = none); a row whose id is outside [0, V)
 *                      has no given token: logprob 0, rank 0
 *   temperatures   in  optional float [M] (NULL = 1); 1 / temperature must be finite; one that
 *                      is not > 0 (a greedy row) counts as 1; at +inf every allowed finite
 *                      logit has z = 0
 *   allowed        in  optional uint32 [M, ceil(V / 32)]: token j is allowed if bit j % 32 of
 *                      word j / 32 is set; logits of the others are not looked at, whatever
 *                      they hold (NULL = all allowed)
 *   topk           in  0 .. 64 alternatives
 *   workspace      tmp nvfp4_logprobs_workspace_bytes(M, V, topk) bytes, 16-byte aligned; the size never falls
 *                      as M grows, so that one workspace serves every batch up to its own
 *   token_logprobs, token_ranks, lse, entropy   out  float / int32 [M], each optional (NULL)
 *   top_logprobs, top_ids   out  float / int32 [M, topk] (NULL only if topk == 0)
 *
 * A logit of -inf has probability 0: a given token there has logprob -inf, and
 * it is never an alternative.  Where fewer than topk alternatives exist the
 * rest are id -1, logprob -inf.  A row with nothing allowed, or only -inf, has
 * lse -inf, entropy 0, logprob -inf and no alternatives.  An allowed NaN or
 * +inf makes the row's lse, entropy and logprobs NaN; a NaN is never an
 * alternative.
 */
int64_t nvfp4_logprobs_workspace_bytes(int64_t M, int64_t V, int64_t topk);
nvfp4_status nvfp4_logprobs(const void* logits, int dtype, int64_t M, int64_t V, int64_t row_stride,
                            const int32_t* token_ids, const float* temperatures, const uint32_t* allowed,
                            int64_t topk, void* workspace, float* token_logprobs, int32_t* token_ranks, float* lse,
                            float* entropy, float* top_logprobs, int32_t* top_ids, void* stream);

/*
 * nvfp4_logprobs_backward -- the gradient of a loss through token_logprobs,
 * entropy and lse to the logits:
 *   dlogits[i, j] = (1 / T) * ( dlogprob[i] * 1[j = id] + p * (dlse[i] - dlogprob[i]
 *                               - dentropy[i] * (log p + entropy[i])) ),   log p = z[i, j] - lse[i]
 * in float32, rounded once to dtype.  Tokens that are not allowed, logits of
 * -inf and rows with lse -inf get 0.  Where |lse| is 1024 or more (8192 for bf16),
 * its rounding would show in p: there log p is taken from the row's logits again, relative to
 * their maximum (slower, a row at a time).
 *
 *   logits, token_ids, temperatures, allowed   in  as given to nvfp4_logprobs
 *   lse, entropy   in  float [M] as nvfp4_logprobs wrote them (entropy only with dentropy)
 *   dlogprob, dentropy, dlse   in  float [M], each optional (NULL = 0); a row without a given
 *                                  token takes dlogprob as 0
 *   dlogits        out dtype [M, V] rows of dlogits_stride elements; it may be logits itself
 *                      (same pointer and stride: the gradient replaces the logits) and
 *                      otherwise its span, first row's start to last row's end, overlaps no
 *                      input's
 */
nvfp4_status nvfp4_logprobs_backward(const void* logits, int dtype, int64_t M, int64_t V, int64_t row_stride,
                                     const int32_t* token_ids, const float* temperatures, const uint32_t* allowed,
                                     const float* lse, const float* entropy, const float* dlogprob,
                                     const float* dentropy, const float* dlse, void* dlogits,
                                     int64_t dlogits_stride, void* stream);

/*
 * int8 weights and activations, one scale per token and per channel.
 * (vLLM API docs, compressed_tensors.schemes, class CompressedTensorsW8A8Int8,
 * dynamic symmetric per-token activations and per-channel weights.)
 *
 * nvfp4_int8_quantize_rows -- row-wise int8 quantization of a bf16 [R, K] matrix:
 *   scales[r] = max(fl32(amax_r / 127), 1e-12),  q = rne(127 a / amax_r) in [-127, 127]
 * The codes are those of the exact ratio (nearest, ties to even); in a row whose scale is 1e-12 they
 * are rne(fl32(a / scale)).  A row that holds a NaN or an infinity has the scale NaN and codes 0: each of its
 * products is NaN.  0 <= R <= 2^23 (0 enqueues nothing).
 * K as below; a and q 16-byte aligned.
 *
 * nvfp4_int8_gemm
 *   y[m, n] = bf16_rne( x_scales[m] * w_scales[n] * sum_k xq[m, k] * wq[n, k] + bias[n] )
 * The sum is exact (any int8 codes, -128 among them), scaling and bias are float32.
 *   xq       in  int8 [M, K], 16-byte aligned; 0 <= M <= 2^22 (M == 0 enqueues nothing)
 *   wq       in  int8 [N, K], 16-byte aligned; K % 16 == 0, 16 <= K < 2^17; M * N <= 2^37
 *   x_scales, w_scales  in  float [M], [N]
 *   bias     in  bf16 [N] or NULL
 *   y        out bf16 [M, N], 16-byte aligned
 */
nvfp4_status nvfp4_int8_quantize_rows(const void* a, int64_t R, int64_t K, int8_t* q, float* scales, void* stream);
nvfp4_status nvfp4_int8_gemm(const int8_t* xq, const float* x_scales, int64_t M, int64_t K, const int8_t* wq,
                             const float* w_scales, int64_t N, const void* bias, void* y, void* stream);

/*
 * Softmax cross entropy straight from hidden states and the bf16 lm_head weight (the
 * weight that nvfp4_quantize takes; after a training step
 * nvfp4_refresh_inplace re-derives the quantized copy), and its gradients.  The
 * logits are never in memory.  With z[i, j] = sum_k x[i, k] weight[j, k] + bias[j]
 * (float32 sums, not rounded):
 *   stats[i] = (m, s),  m = max_j z[i, j],  s = sum_j exp(z[i, j] - m)
 *   lse[i]   = m + log s
 *   loss[i]  = (m - z[i, t]) + log s,  t = targets[i]
 * A row whose target is outside [0, V) does not count: loss and lse 0, stats (0, 1),
 * gradient 0, and neither its x nor its dloss is looked at.  The others are
 * gathered first, so rows that do not count cost nothing.  A logit of -inf (a bias
 * of -inf masks a token) has probability 0 and no gradient; a target there has
 * loss +inf, and in a row with nothing else lse is -inf.  A NaN or +inf logit makes its
 * row's loss and lse NaN.
 *
 * nvfp4_linear_ce_backward: with p = exp(z - m) / s, z computed again,
 *   dz[i, j]    = bf16_rne( (dloss[i] + dlse[i]) * p[i, j] - dloss[i] * 1[j = t] )
 *   dx[i, k]    = bf16_rne( sum_j dz[i, j] * weight[j, k] )
 *   dweight[j, k] = bf16_rne( sum_i dz[i, j] * x[i, k] ),  dbias[j] = bf16_rne( sum_i dz[i, j] )
 * float32 sums.  dz is rounded to bf16 because it is an operand of the two products; what that takes from
 * the targets' dz, the large ones, is added to all three sums (to dweight's rounded to bf16 itself).
 *
 *   x          in  bf16 [M, K], 16-byte aligned; 0 <= M <= 2^22 (M == 0 enqueues nothing: a
 *                  caller's dweight and dbias stay as they are)
 *   weight     in  bf16 [V, K], 16-byte aligned; K % 16 == 0, 16 <= K <= 2^20; M * K, V * K and M * V
 *                  at most 2^37
 *   bias       in  bf16 [V] or NULL
 *   targets    in  int32 [M]
 *   workspace  tmp nvfp4_linear_ce_workspace_bytes(M, V, K, backward) bytes, 16-byte aligned; its
 *                  contents need no preparation.  The size never falls as M grows, and the backward
 *                  pass's is the larger one, so that one workspace serves both calls and every batch
 *                  up to its own.  The backward pass keeps dz of a piece of the vocabulary in it: 128 MiB
 *                  at most up to 65536 rows, 2 KiB a row beyond
 *   loss       out float [M];  lse out float [M] or NULL;  stats out float [M, 2], 8-byte aligned
 *   dloss      in  float [M];  dlse in float [M] or NULL (0)
 *   dx, dweight, dbias  out  bf16, each optional (NULL), dx and dweight 16-byte aligned
 */
int64_t nvfp4_linear_ce_workspace_bytes(int64_t M, int64_t V, int64_t K, int backward);
nvfp4_status nvfp4_linear_ce(const void* x, int64_t M, int64_t K, const void* weight, int64_t V, const void* bias,
                             const int32_t* targets, void* workspace, float* loss, float* lse, float* stats,
                             void* stream);
nvfp4_status nvfp4_linear_ce_backward(const void* x, int64_t M, int64_t K, const void* weight, int64_t V,
                                      const void* bias, const int32_t* targets, const float* stats,
                                      const float* dloss, const float* dlse, void* workspace, void* dx,
                                      void* dweight, void* dbias, void* stream);

/*
 * Gated feed-forward block on bf16 weights: the dense block beside the expert
 * layer, with the experts' layout of w13 (rows [w1; w3]).
 *   [g, u] = x w13^T,  a = silu(g) * u,  y = bf16_rne(a w2^T)
 * float32 sums; a enters its product rounded to bf16, for up to 16 tokens as a pair of bf16
 * that keeps 16 bits of it.  h and act, where given, receive [g, u] in float32 and the
 * a rounded to bf16 for the backward pass:
 *   da = dy w2,  dg = da * u * silu'(g),  du = da * silu(g)
 *   dx = [dg, du] w13,  dw13 = [dg, du]^T x,  dw2 = dy^T a
 * with g and u from h and a from act, and dg and du rounded to bf16 as operands of the products.
 *
 *   x          in  bf16 [T, H]; 0 <= T <= 2^22 (T == 0 enqueues nothing: dw13 and dw2 stay as they
 *                  are)
 *   w13, w2    in  bf16 [2 I, H], [H, I]; H and I multiples of 16, H <= 2^20, I <= 2^19, I * H <= 0x38000000;
 *                  T * H and 2 T * I at most 2^37
 *   h, act     out (forward, both or neither NULL) / in (backward)  float [T, 2 I], bf16 [T, I]
 *   dy         in  bf16 [T, H]
 *   workspace  tmp nvfp4_gated_ffn_workspace_bytes(T, H, I, backward) bytes; its contents need no
 *                  preparation.  The size never falls as T grows, and the backward pass's is the larger
 *                  one, so that one workspace serves both calls and every batch up to its own
 *   y          out bf16 [T, H]
 *   dx, dw13, dw2  out  bf16 as x, w13 and w2, each optional (NULL)
 * Every pointer is 16-byte aligned.
 */
int64_t nvfp4_gated_ffn_workspace_bytes(int64_t T, int64_t H, int64_t I, int backward);
nvfp4_status nvfp4_gated_ffn(const void* x, int64_t T, int64_t H, const void* w13, const void* w2, int64_t I,
                             float* h, void* act, void* workspace, void* y, void* stream);
nvfp4_status nvfp4_gated_ffn_backward(const void* x, int64_t T, int64_t H, const float* h, const void* act,
                                      const void* w13, const void* w2, int64_t I, const void* dy, void* workspace,
                                      void* dx, void* dw13, void* dw2, void* stream);

/* Host-side helpers (no device work). */
const char* nvfp4_status_string(int status);   /* static string for a status code        */
const char* nvfp4_last_hip_error(void);        /* last HIP error text of this thread, or "" */
int nvfp4_abi_version(void);                   /* bumps when a signature above changes   */

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_W4A16_H_ */
