/*
 * nvfp4rac -- NVFP4 W4A4 MoE GEMMs with Residual Activation Compensation,
 * native on AMD Instinct MI355X (gfx950).  C ABI.
 *
 * What the calls compute (cited by page title and section):
 *  - QUADS arXiv abstract (mlsanity paper page, "Abstract (arXiv)"): NVFP4
 *    pairs per-block scale factors with 4-bit E2M1 values and multiplies
 *    4-bit weights by 4-bit activations; rollout activations are new at
 *    every step and are quantized at run time; Residual Activation
 *    Compensation (RAC) repairs the activation channels with the worst
 *    quantization error and keeps the 4-bit GEMMs.
 *  - Blog post "Why 4-bit RL rollout collapses - and it isn't the weights",
 *    section "The failure mode": E2M1 can represent eight magnitudes for
 *    each sign; every engine quantizes the synchronized weights the same way.
 *  - Same post, section "Two fixes, on two different sides": about half of
 *    the activation channels, those with the largest error, also go through
 *    a second 4-bit GEMM on their quantized residual, in the same kernels;
 *    the ordinary 4-bit pass is unchanged.
 *
 * Number formats (the pages name no block size or scale encoding; this library
 * implements the standard NVFP4 layout):
 *  - element: E2M1 code, 4 bits, sign in bit 3, magnitude index in bits 0-2
 *    over {0, 0.5, 1, 1.5, 2, 3, 4, 6}; -0 is never produced.
 *  - block scale: one OCP E4M3 byte (bias 7, max 448, never NaN, sign 0) per
 *    16 consecutive elements along K, blocks starting at k = 0.
 *  - tensor scale: FP32 s_t = RN32(amax / 2688), 2688 = 6 * 448.
 *  - layout: codes[rows, K/2] bytes, element 2j in the low nibble of byte j;
 *    scales[rows, K/16] bytes.  Weights are [N, K] (out x in), y = x W^T.
 *  - rounding: round-to-nearest-even with saturation for both encodings.
 *    rho_b = RN32(amax_b / (6 s_t)), s_b = E4M3(rho_b), S_b = RN32(s_b s_t),
 *    r_b = RN32(1 / S_b), code = E2M1(RN32(x r_b)).
 *
 * Conventions for every call:
 *  - Pointers are device pointers unless stated; the caller owns all memory.
 *    Calls allocate nothing; scratch comes from the caller's workspace `ws`
 *    of at least the size the matching *_workspace_size call returns.
 *  - Calls are asynchronous and ordered on `stream` (a hipStream_t; NULL is
 *    the default stream).  Arguments are validated on the host before
 *    anything is enqueued; a failed check returns its status and enqueues no
 *    work.  Launch failures return NVFP4_ERR_HIP.  Device faults surface at
 *    the caller's next synchronization.
 *  - Not checked on the device (preconditions): finite inputs; group offsets
 *    non-decreasing with the last equal to total_rows; gather indices in
 *    range; an `amax_in` not smaller than the true max|x|.  The group and
 *    gather rules can be checked on host copies with nvfp4_check_groups.
 *  - Re-entrant on distinct buffers; results are bit-reproducible (integer
 *    and max reductions only; no floating-point atomics).
 */
#ifndef NVFP4RAC_H
#define NVFP4RAC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  NVFP4_OK = 0,
  NVFP4_ERR_NULL = 1,      /* a required pointer is NULL */
  NVFP4_ERR_SHAPE = 2,     /* a size is negative or violates a divisibility rule */
  NVFP4_ERR_DTYPE = 3,     /* unknown dtype or epilogue enum */
  NVFP4_ERR_ALIGN = 4,     /* a pointer or leading dimension is misaligned */
  NVFP4_ERR_WORKSPACE = 5, /* workspace missing or too small */
  NVFP4_ERR_HIP = 6        /* a kernel launch failed */
} nvfp4_status_t;

typedef enum { NVFP4_IN_F32 = 0, NVFP4_IN_BF16 = 1 } nvfp4_in_dtype_t;

typedef enum {
  NVFP4_EPI_F32 = 0,           /* out: float [total_rows, N] */
  NVFP4_EPI_SILU_MUL_BF16 = 1, /* out: bf16 [total_rows, N/2], h = silu(gate) * up */
  NVFP4_EPI_BF16 = 2           /* out: bf16 [total_rows, N], y rounded to nearest even
                                  (fp8_ and int8_grouped_gemm only) */
} nvfp4_epilogue_t;

/* Text for a status code (static storage). */
const char* nvfp4_status_string(int status);

/* ------------------------------------------------------------------------
 * nvfp4_quantize -- run-time NVFP4 quantization of one tensor (abstract:
 * activations are quantized at every step; blog, "The failure mode": the
 * weights go through the same quantizer once per synchronization).
 *
 * x        [rows, K] row-major, row stride ldx elements, dtype F32 or BF16.
 *          Requires K % 16 == 0, ldx % 16 == 0, ldx >= K, x 16-byte aligned.
 * amax_in  nullable device float: the tensor amax to use instead of max|x|
 *          (a producer that already knows it, e.g. the SiLU*mul epilogue).
 * codes    out [rows, K/2];  scales out [rows, K/16];  tensor_scale out [1].
 * channel_score  nullable.  When given, the RAC per-channel error statistics
 *          are computed in the same pass over x:  e = x - deq(q(x)) in FP32;
 *          with Es the exponent of s_t (s_t = f 2^Es, f in [0.5, 1)) and
 *          q = min(floor(|e| 2^(8-Es)), 2^17 - 1):  channel_score[k] = sum
 *          over rows of q^2 (int64, exact).  It feeds rac_select_residual.
 *          (Blog, "Two fixes": channels ranked by quantization error; the
 *          metric is this library's reading: the sum of squared errors, in
 *          fixed point so that it is exact.)
 * channel_max  nullable; requires channel_score.  When given, also
 *          channel_max[k] = max over rows of |e| (float), a diagnostic the
 *          selection does not read; leaving it NULL saves its arithmetic and
 *          atomics (about a tenth of the call).
 * rows == 0 is allowed (writes s_t = RN32(amax_in/2688) or 0, and zero stats).
 * ------------------------------------------------------------------------ */
size_t nvfp4_quantize_workspace_size(int64_t rows, int64_t K);
int nvfp4_quantize(const void* x, int dtype, int64_t rows, int64_t K, int64_t ldx,
                   const float* amax_in, uint8_t* codes, uint8_t* scales,
                   float* tensor_scale, int64_t* channel_score, float* channel_max,
                   void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * rac_select_residual -- RAC channel selection and residual re-quantization
 * (blog, "Two fixes, on two different sides": the activation channels with
 * the largest errors, about half of them, get a second 4-bit GEMM pass on
 * their quantized residual).
 *
 * Inputs: the same x, scales, tensor_scale that nvfp4_quantize used and
 * wrote, and its channel_score.  codes is not read and may be NULL: the main
 * codes are a function of x, scales and tensor_scale, and the residual pass
 * recomputes them, which costs less than reading them back.  channel_max is
 * not read either (the selection ranks the scores) and may be NULL.
 * n_select (0 <= n_select <= K; K/2 in the workloads): the channels with the
 *          largest channel_score are selected, ties toward the lower channel
 *          index.
 * selected out [n_select] int32, ascending channel indices.
 * kblock_active out [K/16]: 1 where the 16-block holds a selected channel.
 * res_codes/res_scales out, same layout as codes/scales; res_tensor_scale out:
 *          r = e on selected channels and 0 elsewhere, quantized to NVFP4 in
 *          the same 16-element blocks with the activation's own tensor scale
 *          s_t (the residual pass shares the main pass's tensor scale, so the
 *          GEMM adds both passes in one accumulator): block scale
 *          E4M3(RN32(max|r_b| / (6 s_t))), codes as nvfp4_quantize.
 *          *res_tensor_scale receives s_t.
 * Requires K <= 16384 and the layout rules of nvfp4_quantize; ws 4-byte
 * aligned.  The result is deterministic (integer ranks, max reductions).
 * ------------------------------------------------------------------------ */
size_t rac_select_residual_workspace_size(int64_t rows, int64_t K);
int rac_select_residual(const void* x, int dtype, int64_t rows, int64_t K, int64_t ldx,
                        const uint8_t* codes, const uint8_t* scales,
                        const float* tensor_scale, const int64_t* channel_score,
                        const float* channel_max, int64_t n_select,
                        int32_t* selected, uint8_t* kblock_active,
                        uint8_t* res_codes, uint8_t* res_scales,
                        float* res_tensor_scale, void* ws, size_t ws_bytes,
                        void* stream);

/* ------------------------------------------------------------------------
 * nvfp4_quantize_rac_static -- nvfp4_quantize (with statistics) followed by
 * rac_select_residual, in one call that allocates nothing and takes no
 * workspace: for callers that cannot allocate (code under HIP graph capture,
 * tight serving loops, harnesses that forbid allocation).  Arguments and
 * results are those of the two calls (channel_score is required,
 * channel_max may be NULL).  Scratch (6 KiB: amax partials and block masks) lives in a
 * device array of the library, one per GPU, held until the process ends; its
 * address is looked up on the first call on each device (which must be the
 * current device, the stream's device).  Every call on a GPU shares that
 * GPU's array: calls that overlap on one GPU race (serialize them on one
 * stream).  Nothing in it needs to start at zero.  Limit: K <= 16384
 * (NVFP4_ERR_SHAPE beyond); otherwise the rules of nvfp4_quantize and
 * rac_select_residual.  NVFP4_ERR_HIP if the array's address cannot be found.
 * ------------------------------------------------------------------------ */
int nvfp4_quantize_rac_static(const void* x, int dtype, int64_t rows, int64_t K, int64_t ldx,
                              const float* amax_in, uint8_t* codes, uint8_t* scales,
                              float* tensor_scale, int64_t* channel_score, float* channel_max,
                              int64_t n_select, int32_t* selected, uint8_t* kblock_active,
                              uint8_t* res_codes, uint8_t* res_scales, float* res_tensor_scale,
                              void* stream);

/* ------------------------------------------------------------------------
 * moe_route -- top-k routing of T tokens over E experts and the gather map
 * for the grouped GEMM (the MoE layer of the rollout model; the pages give no
 * routing details, so this is the plain reading).
 *
 * logits   [T, E] float.  Per token, the k experts with the largest logit,
 *          ties toward the lower expert index, in (logit desc, index asc)
 *          order -> topk_ids [T, k].
 * topk_weights nullable [T, k]: softmax(logits) of the chosen experts (not
 *          renormalized; FP32, not bit-defined).
 * expert_offsets [E+1]: exclusive prefix sum of per-expert counts.
 * gather_rows [T*k]: source token of each grouped row, expert-major, tokens
 *          ascending within an expert.  row_of [T, k]: grouped row of
 *          (token, slot).
 * Requires 1 <= k <= min(E, 16), E <= 1024.  With T == 0 the per-token
 * pointers may be NULL and expert_offsets is all zero.
 * ------------------------------------------------------------------------ */
size_t moe_route_workspace_size(int64_t T, int64_t E, int64_t k);
int moe_route(const float* logits, int64_t T, int64_t E, int64_t k,
              int32_t* topk_ids, float* topk_weights, int32_t* expert_offsets,
              int32_t* gather_rows, int32_t* row_of, void* ws, size_t ws_bytes,
              void* stream);

/* ------------------------------------------------------------------------
 * Per-expert RAC.  The pages leave open over which rows RAC's tensor scale and
 * channel selection are taken (blog post, section "Two fixes, on two
 * different sides").  The calls above take one GEMM-input tensor; these take
 * each expert group on its own: the grouped rows j of group g,
 * group_offsets[g] <= j < group_offsets[g+1], read from x row gather_rows[j]
 * (or row j when gather_rows is NULL), form a tensor with its own amax and
 * tensor scale, channel statistics, selection of n_select channels and
 * residual tensor scale.  Every step is the per-tensor definition applied to
 * that tensor.  Outputs are in grouped row order: codes / res_codes
 * [total_rows, K/2], scales / res_scales [total_rows, K/16]; per group:
 * tensor_scales / res_tensor_scales [G], channel_score [G, K] (int64),
 * channel_max [G, K] (nullable, requires channel_score), selected
 * [G, n_select] (ascending per group), kblock_active [G, K/16].  The GEMM then runs without a gather, with
 * NVFP4_GEMM_PER_GROUP_SCALES.  Requires 1 <= G <= 65535, K % 16 == 0,
 * total_rows * K / 16 < 2^31, x 16-byte aligned, ldx % 16 == 0; the
 * selection needs K <= 16384.  Empty groups get zero tensor scales and the
 * n_select lowest channels.
 * ------------------------------------------------------------------------ */
size_t nvfp4_quantize_grouped_workspace_size(int64_t G, int64_t K);
int nvfp4_quantize_grouped(const void* x, int in_dtype, int64_t K, int64_t ldx,
                           const int32_t* group_offsets, int64_t G, int64_t total_rows,
                           const int32_t* gather_rows, uint8_t* codes, uint8_t* scales,
                           float* tensor_scales, int64_t* channel_score, float* channel_max,
                           void* ws, size_t ws_bytes, void* stream);
size_t rac_select_residual_grouped_workspace_size(int64_t G, int64_t K);
int rac_select_residual_grouped(const void* x, int in_dtype, int64_t K, int64_t ldx,
                                const int32_t* group_offsets, int64_t G, int64_t total_rows,
                                const int32_t* gather_rows, const uint8_t* scales,
                                const float* tensor_scales, const int64_t* channel_score,
                                const float* channel_max, int64_t n_select, int32_t* selected,
                                uint8_t* kblock_active, uint8_t* res_codes, uint8_t* res_scales,
                                float* res_tensor_scales, void* ws, size_t ws_bytes,
                                void* stream);

/* ------------------------------------------------------------------------
 * moe_combine -- weighted combine of the expert outputs back to token order
 * (the end of the MoE layer whose expert GEMMs the pages quantize).  For each
 * token t, in slot order s = 0 .. k-1 (the order moe_route writes):
 *   acc = RN32(acc + RN32(topk_weights[t, s] * y[row_of[t, s], :])), acc from 0
 * then out[t, :] = acc (FP32, out_dtype NVFP4_IN_F32) or bf16(acc) (nearest
 * even, NVFP4_IN_BF16).  A gather, not an atomic scatter-add, so the result
 * is deterministic.  y is float [rows, H] in grouped order; row_of and
 * topk_weights are [T, k] from moe_route; out is [T, H].  Requires 1 <= k <=
 * 16, H % 8 == 0, y and out 16-byte aligned.  No workspace.
 * ------------------------------------------------------------------------ */
int moe_combine(const float* y, const int32_t* row_of, const float* topk_weights, int64_t T,
                int64_t k, int64_t H, int out_dtype, void* out, void* stream);

/* ------------------------------------------------------------------------
 * w4a4_grouped_gemm_rac -- grouped (per-expert) W4A4 GEMM with the RAC
 * residual pass fused into the same kernel (abstract: 4-bit by 4-bit GEMMs;
 * blog, "Two fixes": the selected channels' residual pass adds to the
 * unchanged main pass).
 *
 * For grouped row j of group g (offsets[g] <= j < offsets[g+1]) and src =
 * gather_rows[j] (or j when gather_rows is NULL):
 *   y[j, n] = s_tw[g] * s_ta * ( sum_k A[src,k] W_g[n,k]
 *                              + sum_{k in active blocks} R[src,k] W_g[n,k] )
 * with A, R, W the exact dequantized values g * s_b, both passes accumulated
 * in one FP32 accumulator.  The residual shares the activation's tensor
 * scale (rac_select_residual writes *r_tscale = s_ta): the call requires
 * *r_tscale == *a_tscale (per group with NVFP4_GEMM_PER_GROUP_SCALES) and
 * writes NaN outputs for a group where they differ.
 * r_codes == NULL turns RAC off (naive W4A4).  kblock_active == NULL means
 * every block is active.  With NVFP4_GEMM_SKIP_INACTIVE_BLOCKS in `flags`, the
 * residual MFMAs of each 32-k step run only if one of its two 16-blocks is
 * active; without it the residual pass runs over every block.  Both are exact
 * (an inactive block's residual codes are zero); the flag pays off when the
 * selection leaves many blocks inactive, and costs a few percent otherwise.
 * Epilogue F32 writes y.  Epilogue SILU_MUL_BF16 treats W as the fused
 * gate/up weight [N = 2I, K] with the gate in rows [0, I) and writes
 * h[j, i] = bf16(silu(y[j, i]) * y[j, I + i]) to out [total_rows, I] and, if
 * out_amax is given, max-combines max|h| into *out_amax (an atomic max on the
 * float bits; the caller initializes *out_amax, normally to 0, so that the
 * call launches the GEMM kernel alone).  With SILU_MUL, a non-NULL out_y
 * (float [total_rows, N], 4-byte aligned) also receives the FP32 values y
 * that enter the SiLU*mul, gate columns then up columns as in W: the same
 * kernel and accumulation, plus these stores (for verification).
 * Requires K % 128 == 0, N % 128 == 0, all tensors 16-byte aligned.
 * ------------------------------------------------------------------------ */
typedef struct {
  int64_t num_groups;           /* G >= 1 */
  int64_t N;                    /* output columns (2I for SILU_MUL) */
  int64_t K;                    /* contraction length */
  int64_t total_rows;           /* rows of the grouped output */
  const int32_t* group_offsets; /* [G+1], ascending, [0] = 0, [G] = total_rows */
  const int32_t* gather_rows;   /* [total_rows] or NULL (identity) */
  const uint8_t* a_codes;       /* [src_rows, K/2] */
  const uint8_t* a_scales;      /* [src_rows, K/16] */
  const float* a_tscale;        /* [1] */
  const uint8_t* r_codes;       /* residual, or NULL for RAC off */
  const uint8_t* r_scales;
  const float* r_tscale;
  const uint8_t* kblock_active; /* [K/16] or NULL */
  const uint8_t* w_codes;       /* [G, N, K/2] */
  const uint8_t* w_scales;      /* [G, N, K/16] */
  const float* w_tscale;        /* [G] */
  int64_t epilogue;             /* nvfp4_epilogue_t */
  void* out;                    /* float [total_rows, N] or bf16 [total_rows, N/2] */
  float* out_amax;              /* SILU_MUL only, nullable, caller-initialized */
  int64_t flags;                /* NVFP4_GEMM_* bits */
  float* out_y;                 /* SILU_MUL only, nullable: FP32 y [total_rows, N] */
} w4a4_gemm_args_t;

/* nvfp4_check_groups -- host-side check of the grouped GEMM's preconditions
 * that the device does not check (a violation would read out of bounds).
 * All pointers are HOST pointers (copies of the device arrays).
 * offsets [G+1]: offsets[0] == 0, non-decreasing, offsets[G] == total_rows.
 * gather [total_rows] (nullable): every index in [0, src_rows).
 * Returns NVFP4_OK, NVFP4_ERR_NULL (offsets NULL) or NVFP4_ERR_SHAPE (the
 * first violated rule).  Reads only; no device work. */
int nvfp4_check_groups(const int32_t* offsets, int64_t G, int64_t total_rows,
                       const int32_t* gather, int64_t src_rows);

#define NVFP4_GEMM_SKIP_INACTIVE_BLOCKS 1
/* Per-expert RAC: a_tscale and r_tscale are [G] (group g's tensor scales) and
 * kblock_active is [G, K/16], as nvfp4_quantize_grouped and
 * rac_select_residual_grouped write them. */
#define NVFP4_GEMM_PER_GROUP_SCALES 2

size_t w4a4_grouped_gemm_rac_workspace_size(const w4a4_gemm_args_t* args);
int w4a4_grouped_gemm_rac(const w4a4_gemm_args_t* args, void* ws, size_t ws_bytes,
                          void* stream);

/* ------------------------------------------------------------------------
 * Trainer-side weight fake-quantization (Asymmetric QAT).  The trainer
 * fake-quantizes its weights, and only its weights, with the rollout's own
 * NVFP4 quantize-dequantize path, so the two sides see the same weight error
 * (blog post, section "Two fixes, on two different sides"; arXiv abstract:
 * weights align through a shared quantization-dequantization path).
 *
 * nvfp4_qdq: runs the quantizer of nvfp4_quantize (same kernel, same
 * arithmetic, tensor scale from max|x| or from amax_in) and stores, instead of
 * codes and scales, the dequantized values v = RN32(RN32(g s_b) s_t) -- the
 * exact product g s_b s_t rounded once -- to out [rows, K] (row stride K):
 * FP32 for out_dtype NVFP4_IN_F32, bf16 (nearest even of v) for
 * NVFP4_IN_BF16.  *tensor_scale receives s_t.  Workspace as
 * nvfp4_quantize (none with amax_in).  Requires K % 16 == 0, x and out
 * 16-byte aligned, ldx % 16 == 0 (elements), as nvfp4_quantize.
 *
 * nvfp4_dequantize: the same values from stored codes [rows, K/2], scales
 * [rows, K/16] and tensor scale; nvfp4_qdq(x) equals
 * nvfp4_dequantize(nvfp4_quantize(x)) bit for bit.  Requires K % 16 == 0,
 * codes 8-byte aligned, out 16-byte aligned.  No workspace.
 * ------------------------------------------------------------------------ */
size_t nvfp4_qdq_workspace_size(int64_t rows, int64_t K);
int nvfp4_qdq(const void* x, int in_dtype, int64_t rows, int64_t K, int64_t ldx,
              const float* amax_in, int out_dtype, void* out, float* tensor_scale, void* ws,
              size_t ws_bytes, void* stream);
int nvfp4_dequantize(const uint8_t* codes, const uint8_t* scales, const float* tensor_scale,
                     int64_t rows, int64_t K, int out_dtype, void* out, void* stream);

/* ------------------------------------------------------------------------
 * FP8 (E4M3) W8A8 comparator.  The pages measure QUADS against FP8 rollout
 * (arXiv abstract on the mlsanity page; blog post, section "What it buys")
 * without saying how the FP8 engine scales its tensors; these calls
 * implement one FP32 scale per activation row (token) and per weight output
 * channel, so that a QUADS step can be timed beside an FP8 step on the same
 * workload.
 *
 * fp8_quantize_rows: for each row of x [rows, K] (FP32 or bf16, row-major):
 *   s = RN32(amax_row / 448)   (double quotient rounded once; 0 for a zero row)
 *   r = RN32(1 / s)            (0 when s == 0)
 *   codes[row, k] = E4M3(RN32(x r)): OCP E4M3 (bias 7, max 448), nearest
 *   even, saturating at +-448, sign bit from the product (so -0 may occur).
 * codes is uint8 [rows, K]; row_scales is float [rows].  Requires K % 16 == 0,
 * x 16-byte aligned, codes 8-byte aligned.
 * ------------------------------------------------------------------------ */
int fp8_quantize_rows(const void* x, int in_dtype, int64_t rows, int64_t K, uint8_t* codes,
                      float* row_scales, void* stream);

/* fp8_grouped_gemm: grouped (per-expert) FP8 GEMM with the grouping, gather
 * and epilogues of w4a4_grouped_gemm_rac:
 *   y[j, n] = a_scales[src] * w_scales[g*N + n] * sum_k A[src,k] W_g[n,k]
 * with A, W the E4M3 values (products exact, FP32 accumulation).  Epilogue
 * SILU_MUL_BF16 writes h[j, i] = bf16(silu(y[j, i]) * y[j, I + i]) to out
 * [total_rows, I] (no amax: the FP8 quantizer scales per row); epilogue
 * BF16 writes bf16(y) to out [total_rows, N] (the output type of the vendor
 * FP8 GEMM it is compared with).  Requires
 * K % 128 == 0, N % 128 == 0, codes 16-byte aligned, scales 4-byte aligned.
 * No workspace. */
typedef struct {
  int64_t num_groups;           /* G >= 1 */
  int64_t N;                    /* output columns (2I for SILU_MUL) */
  int64_t K;                    /* contraction length */
  int64_t total_rows;           /* rows of the grouped output */
  const int32_t* group_offsets; /* [G+1], ascending, [0] = 0, [G] = total_rows */
  const int32_t* gather_rows;   /* [total_rows] or NULL (identity) */
  const uint8_t* a_codes;       /* [src_rows, K] E4M3 */
  const float* a_scales;        /* [src_rows] */
  const uint8_t* w_codes;       /* [G, N, K] E4M3 */
  const float* w_scales;        /* [G, N] */
  int64_t epilogue;             /* nvfp4_epilogue_t */
  void* out;                    /* float or bf16 [total_rows, N], or bf16 [total_rows, N/2] */
} fp8_gemm_args_t;

int fp8_grouped_gemm(const fp8_gemm_args_t* args, void* stream);

/* ------------------------------------------------------------------------
 * nvfp4_moe_decode -- a whole MoE FFN layer for a few tokens (a decode step)
 * on the NVFP4 expert weights: routing, gate/up product, SiLU*mul, down
 * product and weighted combine.  At this size the layer costs the bytes of
 * the routed experts' weights, so the activations are not quantized at all:
 * the layer computes with the values that the trainer's forward has (blog,
 * "Two fixes": fake-quantized weights, activations left alone), which the
 * W4A4 + RAC calls approximate for large batches.
 *
 * For token t with logits row l = logits[t, :] (a NaN counts as -inf):
 *   topk_ids[t, :]     the k experts with the largest logit, ties toward the
 *                      lower expert index, in (logit desc, index asc) order;
 *   topk_weights[t, s] softmax(l) at that expert (not renormalized), 0 where
 *                      the logit is -inf;
 *   out[t, :] = sum over slots s with weight > 0 of
 *      topk_weights[t, s] * s_d[e] * W_d[e] h,
 *      h = silu(g) * u,  [g; u] = s_gu[e] * W_gu[e] x[t, :]
 * with W the exact dequantized values g * s_b.  A slot of weight 0 costs
 * nothing and adds nothing, so rows that pad a batch to a captured size are
 * given logits of -inf: their out row is 0 and their x row is not read.
 * Products are exact and sums are FP32; x and h enter the matrix cores as
 * fp16 pieces scaled per row and K range by a power of two: one piece (11
 * bits, which holds a bf16 x exactly and h to an eighth of bf16's step) for
 * bf16, two (22 bits) for FP32.  SiLU and the routing weights take the
 * hardware's exponential (a weight is within 2^-20 of its value).
 *
 * x [T, H] (row stride ldx) and out [T, H] (row stride ldo) have x_dtype;
 * logits is float [T, E] (row stride ld_logits).  gu_* hold [E, 2I, H] with
 * the gate in rows [0, I), d_* hold [E, H, I], in the layout of
 * nvfp4_quantize, tensor scales [E].  topk_ids / topk_weights [T, k] are
 * nullable.  Requires 0 <= T <= 64, 1 <= k <= min(E, 16), E <= 1024, H and I
 * multiples of 32 up to 65536, ldx and ldo multiples of 8, x, out, codes and
 * scales 16-byte aligned, ws 16-byte aligned.  Inputs and out may not
 * overlap.  Finite x is a precondition for the row it is in only; logits of
 * +inf give their row NaN weights, and such slots are left out of the sum.
 * An h beyond FP32's range enters the down product as its infinity.
 * The result is deterministic (sums in a fixed order).  Calls that may
 * overlap (on two streams, in two graphs) need workspaces and outputs of their
 * own.  With T == 0 nothing is enqueued.
 * ------------------------------------------------------------------------ */
typedef struct {
  int64_t T, E, k, H, I;
  const void* x;              /* [T, H] */
  int64_t x_dtype, ldx;       /* nvfp4_in_dtype_t; elements */
  const float* logits;        /* [T, E] */
  int64_t ld_logits;
  const uint8_t* gu_codes;    /* [E, 2I, H/2] */
  const uint8_t* gu_scales;   /* [E, 2I, H/16] */
  const float* gu_tscale;     /* [E] */
  const uint8_t* d_codes;     /* [E, H, I/2] */
  const uint8_t* d_scales;    /* [E, H, I/16] */
  const float* d_tscale;      /* [E] */
  void* out;                  /* [T, H], x_dtype */
  int64_t ldo;
  int32_t* topk_ids;          /* [T, k], nullable */
  float* topk_weights;        /* [T, k], nullable */
} nvfp4_moe_decode_args_t;

size_t nvfp4_moe_decode_workspace_size(const nvfp4_moe_decode_args_t* args);
int nvfp4_moe_decode(const nvfp4_moe_decode_args_t* args, void* ws, size_t ws_bytes,
                     void* stream);

/* ------------------------------------------------------------------------
 * token_logprobs -- what a rollout records of each sampled token and a
 * trainer scores again (the pages measure the rollout-trainer log-prob gap:
 * blog post, section "What it buys"): the token's log-probability, the
 * entropy of its distribution and the largest alternatives, in one pass over
 * the logits.
 *
 * Per row t, with z_j = logits[t, j] * inv_temperature[t] (1 where NULL):
 *   lse = log sum_j exp(z_j),  log p_j = z_j - lse
 *   logprobs[t]  = log p_y, y = targets[t]; 0 where y < 0 (ignored
 *                  position), NaN where y >= V
 *   entropy[t]   = -sum_j p_j log p_j (a term with p_j = 0 is 0)
 *   norm[t]      = {m, L}: m = max_j logits[t, j] (0 if all are -inf) and
 *                  lse = m * inv_temperature[t] + L ln 2; what
 *                  token_logprobs_backward reads
 *   top_ids[t, :], top_logprobs[t, :]  the top_k largest logits in (logit
 *                  desc, index asc) order and their log p; a NaN ranks as -inf
 * Logits of -inf are masked tokens (probability 0).  A row of nothing else
 * has logprobs -inf (0 where ignored), entropy 0, top_ids 0, 1, .. and
 * top_logprobs -inf.  A NaN or +inf logit makes its row's statistics NaN.
 *
 * logits [T, V] float or bf16, row stride ld elements (any ld >= V, no
 * alignment beyond the element's).  targets and logprobs are given together
 * or both NULL; entropy, norm and inv_temperature are nullable; top_ids and
 * top_logprobs are required if top_k > 0.  inv_temperature must be positive
 * and finite.  Requires 1 <= V <= 2^30, 0 <= top_k <= min(V, 32), T < 2^24,
 * arrays aligned to their elements.  ws may be NULL where its size is 0; calls
 * that may overlap need workspaces of their own.  Sums are FP32, and
 * exponentials and logarithms the hardware's in base 2: results are off by some
 * 2^-23 of the sizes that meet in them (1, |log p|, and the logit's distance from
 * the row's maximum), and by the rounding of sums of V terms, V / 64 or fewer in
 * a chain.  The result is deterministic.  Rows in which more
 * than 512 16-byte pieces hold a logit that could be among the top_k (ties,
 * rising rows) take top_k further passes over the row.
 *
 * token_logprobs_backward -- the gradient of the logits:
 *   grad[t, j] = inv_temperature[t] * ( a ([j = y] - p_j)
 *                                       - b p_j (log p_j + entropy[t]) )
 * with a = grad_logprobs[t] (0 where NULL, where y < 0, or where the whole
 * row is masked) and b = grad_entropy[t] (0 where NULL), rounded once to the
 * logits' dtype; 0 for masked tokens, NaN for a row with y >= V.  A row with
 * a = b = 0 (an ignored position without an entropy gradient) gets 0 and its
 * logits are not read, whatever they are.  targets is required with
 * grad_logprobs, entropy with grad_entropy.  grad_logits has row stride ldg
 * >= V and may be the logits themselves (same ld), but not overlap them in
 * another way.  Where row t of both starts at the same offset from a 16-byte
 * boundary (the same ld and base alignment, say) memory is accessed in 16-byte
 * pieces, else by elements, several times slower.  The forward call's limits
 * hold.  No workspace.
 * ------------------------------------------------------------------------ */
size_t token_logprobs_workspace_size(int64_t T, int64_t V, int64_t top_k);
int token_logprobs(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld,
                   const int64_t* targets, const float* inv_temperature, int64_t top_k,
                   float* logprobs, float* entropy, float* norm, int32_t* top_ids,
                   float* top_logprobs, void* ws, size_t ws_bytes, void* stream);
int token_logprobs_backward(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld,
                            const int64_t* targets, const float* inv_temperature,
                            const float* norm, const float* entropy,
                            const float* grad_logprobs, const float* grad_entropy,
                            void* grad_logits, int64_t ldg, void* stream);

/* ------------------------------------------------------------------------
 * INT8 (W8A8) comparator: matrix products in 8-bit integers with one FP32
 * scale per activation row (token, at run time) and per weight output channel,
 * the other 8-bit form that a rollout can take where the pages take NVFP4
 * (arXiv abstract on the mlsanity page; blog post, section "What it buys",
 * compares with FP8).  Every product and sum is exact, so the only errors are
 * the two roundings to 8 bits and the one to the output's type.
 *
 * int8_quantize_rows: for each row of x [rows, K] (FP32 or bf16, row stride
 * ldx elements):
 *   s = RN32(amax_row / 127)   (double quotient rounded once), at least 2^-126;
 *                              0 for a zero row
 *   r = RN32(1 / s)            (0 when s == 0)
 *   codes[row, k] = nearest integer to RN32(x r), ties to even, in [-127, 127]
 * A row that holds an infinity or a NaN gets the scale NaN and codes 0, which
 * makes its outputs NaN and no other row's.  codes is int8 [rows, K];
 * row_scales is float [rows].  Requires K % 16 == 0, K <= 2^24, ldx >= K, ldx %
 * 8 == 0, x and codes 16-byte aligned.
 * ------------------------------------------------------------------------ */
int int8_quantize_rows(const void* x, int in_dtype, int64_t rows, int64_t K, int64_t ldx,
                       int8_t* codes, float* row_scales, void* stream);

/* int8_grouped_gemm: grouped (per-expert) INT8 GEMM with the grouping, gather
 * and epilogues of w4a4_grouped_gemm_rac and fp8_grouped_gemm:
 *   y[j, n] = RN32(RN32(a_scales[src] w_scales[g*N + n]) float(sum_k A[src,k] W_g[n,k]))
 * with the sum exact in 32 bits.  Epilogue F32 writes y, BF16 writes bf16(y),
 * SILU_MUL_BF16 h[j, i] = bf16(silu(y[j, i]) * y[j, I + i]) to [total_rows, I].
 * The activations come either quantized (a_codes, a_scales) or as x, whose
 * src_rows rows the call quantizes into the workspace first, as int8_quantize_rows
 * does.  group_offsets may be NULL with one group.  group_offsets[G] may be less
 * than total_rows; rows of out behind it are left alone.  Requires 1 <= N <= 2^24 (even for SiLU), K % 16 == 0,
 * 16 <= K <= 131056 (no sum of 8-bit products can leave 32 bits), num_groups <=
 * 2^20, total_rows <= 2^30; codes and x 16-byte aligned, out aligned to its
 * elements, ws 16-byte aligned.  Without a gather, src_rows >= total_rows;
 * src_rows < 2^31 and src_rows K <= 2^36, with a gather (src_rows - 1) K / 16 + 7 <
 * 2^32 too (the copies count 16-byte units in 32 bits).  A call that needs a grid of 2^32 threads (some 2^23 tiles
 * of 64 x 128 or larger) is refused.  Calls that may overlap need workspaces of their own. */
typedef struct {
  int64_t num_groups;           /* G >= 1 */
  int64_t N;                    /* output columns (2I for SILU_MUL) */
  int64_t K;                    /* contraction length */
  int64_t total_rows;           /* rows of the grouped output */
  const int32_t* group_offsets; /* [G+1], ascending, [0] = 0, [G] <= total_rows */
  const int32_t* gather_rows;   /* [total_rows] or NULL (identity) */
  const int8_t* a_codes;        /* [src_rows, K], or NULL where x is given */
  const float* a_scales;        /* [src_rows] */
  const void* x;                /* [src_rows, K], or NULL where a_codes is given */
  int64_t x_dtype, ldx;         /* nvfp4_in_dtype_t; row stride in elements */
  int64_t src_rows;             /* rows of a_codes or of x */
  const int8_t* w_codes;        /* [G, N, K] */
  const float* w_scales;        /* [G, N] */
  int64_t epilogue;             /* nvfp4_epilogue_t */
  void* out;                    /* float or bf16 [total_rows, N], or bf16 [total_rows, N/2] */
} int8_gemm_args_t;

size_t int8_grouped_gemm_workspace_size(const int8_gemm_args_t* args);
int int8_grouped_gemm(const int8_gemm_args_t* args, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * moe_balance_loss -- what a trainer adds for the router of the MoE layers
 * (the pages train an MoE policy and describe no router): the slots that each
 * expert got, each expert's mean probability, the balance loss and the z-loss.
 *
 * Row t counts if mask[t] != 0 (or mask is NULL) and not all of its logits are
 * -inf; n = number of such rows, p_t = softmax(logits[t, :]), lse_t = its log-sum
 * of exponentials (an expert of logit -inf has probability 0).
 *   counts[e]     = slots s of counted rows with topk_ids[t, s] == e
 *   tokens[0]     = n
 *   mean_probs[e] = P_e = (1/n) sum_t p_te
 *   losses[0]     = E / (k n) sum_e counts[e] P_e   (1 where both are even)
 *   losses[1]     = (1/n) sum_t lse_t^2
 * all 0 for n == 0.  An id outside [0, E) is a dropped slot: it is not counted,
 * and k n stays the divisor.  Rows that do not count are not read where the
 * mask says so.  A NaN or +inf logit of a counted row makes the losses (and,
 * backward, its own row's gradient) NaN.
 *
 * moe_balance_loss_backward -- the gradient of the logits from that of the two
 * losses (grad_losses, float [2], device), with counts held constant:
 *   grad[t, j] = p_tj (a (counts[j] - sum_e counts[e] p_te) + b lse_t),
 *   a = grad_losses[0] E / (k n^2),  b = grad_losses[1] 2 / n,
 * rounded once to the logits' dtype; 0 in rows that do not count.
 *
 * logits [T, E] float or bf16, row stride ld elements (any ld >= E, no
 * alignment beyond the element's; rows that start on 16 bytes are read in
 * 16-byte pieces).  topk_ids int32 [T, k] (moe_route's), mask uint8 [T] or
 * NULL.  mean_probs is nullable.  grad_logits has row stride ldg >= E and may
 * be the logits themselves (same ld).  Requires 1 <= E <= 1024, 1 <= k <= E, T k <
 * 2^31.  Sums of probabilities over rows are FP32 over at most 64 rows of a lane and
 * then over the lanes of a workgroup (chains of at most 84 roundings), FP64 above
 * that, and the sum of lse^2 is FP64 throughout; exponentials and logarithms are the
 * hardware's.  The results are
 * deterministic.  Calls that may overlap need workspaces of their own.
 * ------------------------------------------------------------------------ */
size_t moe_balance_loss_workspace_size(int64_t T, int64_t E);
int moe_balance_loss(const void* logits, int dtype, int64_t T, int64_t E, int64_t ld,
                     const int32_t* topk_ids, int64_t k, const uint8_t* mask, int32_t* counts,
                     int32_t* tokens, float* mean_probs, float* losses, void* ws,
                     size_t ws_bytes, void* stream);
int moe_balance_loss_backward(const void* logits, int dtype, int64_t T, int64_t E, int64_t ld,
                              int64_t k, const uint8_t* mask, const int32_t* counts,
                              const int32_t* tokens, const float* grad_losses,
                              void* grad_logits, int64_t ldg, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* NVFP4RAC_H */
