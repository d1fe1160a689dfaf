/*
 * fp8q_fp4.h -- the part of libfp8q's C ABI for 4-bit microscaled operands
 * (nvfp4, mxfp4) and for experts: quantization, the block-scaled GEMM, routing
 * and the experts' products on B200 (sm_100a).
 *
 * The conventions are those of fp8q.h: device pointers owned by the caller,
 * bf16 bit patterns, leading dimensions in elements unless said otherwise,
 * asynchronous calls on `stream` that can be captured into CUDA graphs,
 * argument errors found on the host before anything is launched, bounded
 * device-side waits.  Matrices and codes are 16-byte aligned, fp32 and int32
 * arrays 4-byte aligned.  With no rows (M, T or n = 0) a call validates its
 * sizes and returns FP8Q_OK; data pointers may then be NULL.
 */
#ifndef FP8Q_FP4_H
#define FP8Q_FP4_H

#include "fp8q.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------ */
/* 4-bit microscaled operands (nvfp4, mxfp4)                                 */
/* ------------------------------------------------------------------------ */

/*
 * The FP8 path one format further down: e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6
 * and their negatives) with a scale per group of consecutive values of a row.
 * The pages name the two formats and their kernels (the MXFP4 CUTLASS MoE
 * page, vllm PR #37463); this library fixes their arithmetic as follows.
 *   nvfp4   groups of 16, value = code * sf * g: sf e4m3, g one fp32 scale of
 *           the whole tensor (`gscale`, a device pointer; NULL = 1):
 *             u = fl32(fl32(amax / 6) / g), sf = e4m3_rn(min(u, 448)),
 *             d = fl32(sf g), code = e2m1_rn(fl32(y / d)); d = 0 gives code 0
 *           g must be positive, between 2^-64 and 2^64.
 *   mxfp4   groups of 32, value = code * sf: sf = fl32(max(amax, 1e-10) / 6)
 *           rounded up to a power of two, stored as its E8M0 byte (254 at
 *           most); no tensor scale (`gscale` must be NULL).  The OCP MX rule,
 *           2^(floor(log2 amax) - 2), lets the largest values saturate: for an
 *           amax above 1.5 times the power of two below it, its byte is one less
 *           than this one, else (from 1e-10 on) the same.  Both are mxfp4
 *           tensors, and the products take either.
 * Codes go to the nearest, ties to the even code, saturating at +-6; every
 * code keeps its value's sign.  A y that is NaN (a NaN input, 0 times
 * infinity, a gate of -infinity, a row of zeros under eps = 0) leaves the codes
 * and the scale of its group unspecified.
 *   codes   two to a byte, the lower index in the low half; K must be a
 *           multiple of 32
 *   scales  bytes in blocks of 128 rows x 4 groups, the layout the tensor core
 *           reads: block (r / 128, j / 4) of row r and group j is 512 bytes,
 *           blocks of a row consecutive, and inside a block the byte lies at
 *           (r % 32) * 16 + (r % 128) / 32 * 4 + j % 4.  A buffer holds
 *           fp8q_fp4_sf_bytes(rows, K, format) bytes, 16-byte aligned.  Groups
 *           that only fill the last block of a row must be 0 (the quant entry
 *           points write them so); the bytes of rows that only fill the last
 *           block row are not written and have no effect.
 */
#define FP8Q_FP4_NV 0
#define FP8Q_FP4_MX 1

/* Bytes of the scale buffer of a [rows, K] matrix (0 for a bad argument). */
FP8Q_API size_t fp8q_fp4_sf_bytes(int64_t rows, int64_t K, int format);

/*
 * fp8q_fp4_quant, fp8q_rmsnorm_fp4_quant, fp8q_silu_mul_fp4_quant -- the quant
 * ops of this header with 4-bit codes: the same y (x itself; bf16(bf16(x r) w);
 * bf16(silu(gate) up)), always exactly rounded.  Weights are quantized with
 * fp8q_fp4_quant (a row is an output channel).
 *   x       as in fp8q_group_quant (K), fp8q_rmsnorm_quant (H) and
 *           fp8q_silu_mul_quant (2I); ldx a multiple of 8
 *   q       codes, ldq BYTES a row (>= K / 2, a multiple of 8)
 *   sf      scale blocks
 */
FP8Q_API fp8q_status fp8q_fp4_quant(const void* x, int64_t M, int64_t K, int64_t ldx, int format,
                                    const float* gscale, void* q, int64_t ldq, uint8_t* sf, void* stream);
FP8Q_API fp8q_status fp8q_rmsnorm_fp4_quant(const void* x, const void* w, float eps, int64_t M, int64_t H,
                                            int64_t ldx, int format, const float* gscale, void* q,
                                            int64_t ldq, uint8_t* sf, void* stream);
FP8Q_API fp8q_status fp8q_silu_mul_fp4_quant(const void* x, int64_t M, int64_t I, int64_t ldx, int format,
                                             const float* gscale, void* q, int64_t ldq, uint8_t* sf,
                                             void* stream);

/*
 * fp8q_fp4_dequant -- the values that codes and scales stand for:
 *   y = bf16_rn(fl32(fl32(code * sf) * g))        bf16 [M, K], ldy (>= K, multiple of 8)
 */
FP8Q_API fp8q_status fp8q_fp4_dequant(const void* q, int64_t ldq, const uint8_t* sf, int format,
                                      const float* gscale, int64_t M, int64_t K, void* y, int64_t ldy,
                                      void* stream);

/*
 * fp8q_scaled_mm_fp4 -- the block-scaled GEMM on 4-bit operands:
 *   y[m, n] = bf16_rn( ga gb sum_k (qa[m, k] sfa[m, k/g]) (qb[n, k] sfb[n, k/g]) )
 * with an fp32 accumulator; both operands in one format.
 *   a_q, b_q    codes [M, K] and [N, K], rows contiguous (K / 2 bytes)
 *   a_sf, b_sf  scale blocks of the M and N rows
 *   a_gscale, b_gscale  fp32 [1] or NULL (1)
 *   N a multiple of 16; y bf16 [M, N] (ldy >= N, multiple of 8).  No workspace.
 */
FP8Q_API fp8q_status fp8q_scaled_mm_fp4(const void* a_q, const void* b_q, const uint8_t* a_sf,
                                        const uint8_t* b_sf, int format, const float* a_gscale,
                                        const float* b_gscale, int64_t M, int64_t N, int64_t K, void* y,
                                        int64_t ldy, void* stream);

/* ------------------------------------------------------------------------ */
/* Experts: routing, and their products on 4-bit operands                    */
/* ------------------------------------------------------------------------ */

#define FP8Q_ROUTE_SOFTMAX 0
#define FP8Q_ROUTE_SIGMOID 1

/*
 * fp8q_moe_route -- each token's experts and their weights, from the router's
 * logits [T, E] (fp32, or bf16 with logits_bf16 = 1; leading dimension ldl).
 *   score    softmax over the E logits, or sigmoid of each
 *   key      score + bias[e] (bias fp32 [E] or NULL); only the selection uses
 *            the bias
 *   groups   with topk_groups < num_groups, the E experts are num_groups
 *            equal groups of neighbours; a group counts with its largest key,
 *            or, with a bias, the sum of its two largest; experts outside the
 *            best topk_groups groups are not selected
 *   ids      the topk largest keys, descending; equal keys (and equal groups)
 *            go to the lowest index.  With a bias keys are as fp64 tells them
 *            apart; without one the logits decide, with which both scores grow
 *            (scores that fp64 rounds to the same value are not equal then)
 *   weights  the scores of the selected experts, divided by their sum if
 *            renormalize is set (0 where that sum is 0), times scale
 * Scores are those of fp64 (smaller ones count as 0), each good to 2^-19 of
 * itself; an fp32 weight below 2^-126 may be 0.
 * A logit of -inf (or NaN) masks its expert: score 0, key -inf, selected only
 * after all unmasked ones of the groups that are left; a token whose experts are
 * all masked has weights 0.  A sum with a masked key is -inf, too: with a bias
 * a group with one unmasked expert counts no more than one with none.
 *   E <= 512, topk <= 32, num_groups <= 32 (else FP8Q_ERR_UNSUPPORTED);
 *   topk <= E / num_groups * topk_groups
 *   weights fp32 [T, topk], ids int32 [T, topk], both contiguous
 */
FP8Q_API fp8q_status fp8q_moe_route(const void* logits, int logits_bf16, int64_t T, int64_t E, int64_t ldl,
                                    int topk, int scoring, const float* bias, int num_groups,
                                    int topk_groups, int renormalize, float scale, float* weights,
                                    int* ids, void* stream);

/*
 * fp8q_moe_plan -- order n = T topk (token, slot) entries by expert, in entry
 * order within an expert.
 *   ids         int32 [n]; any id outside [0, E), negative ones of every size
 *               among them, gets no row (an expert that another GPU holds; the
 *               ids may be given less the first expert that is here)
 *   offsets     int32 [E + 1]: expert e's rows are [offsets[e], offsets[e+1])
 *   sf_offsets  int32 [E + 1]: its scales begin at block row sf_offsets[e]
 *               (every expert begins a block row of its own; n rows of E
 *               experts take at most n / 128 + min(n, E) block rows)
 *   pos         int32 [n]: the entry's row, or -1
 *   sf_row      int32 [n]: the row whose place its scales take, or -1
 *   workspace   fp8q_moe_plan_workspace_bytes(n, E) bytes (NULL if 0), of any
 *               content; calls that share one must not overlap in time
 * E <= 512, n <= 2^25 (else FP8Q_ERR_UNSUPPORTED).  The order never depends on
 * timing.
 */
FP8Q_API size_t fp8q_moe_plan_workspace_bytes(int64_t n, int64_t E);
FP8Q_API fp8q_status fp8q_moe_plan(const int* ids, int64_t n, int64_t E, int* offsets, int* sf_offsets,
                                   int* pos, int* sf_row, void* workspace, size_t ws_bytes, void* stream);

/*
 * fp8q_moe_fp4_quant -- fp8q_fp4_quant of T tokens, each written to the rows
 * of its topk experts: row pos[t, j] of q and the scales of row sf_row[t, j].
 * Negative entries are skipped.
 */
FP8Q_API fp8q_status fp8q_moe_fp4_quant(const void* x, int64_t T, int64_t K, int64_t ldx, int topk,
                                        const int* pos, const int* sf_row, int format,
                                        const float* gscale, void* q, int64_t ldq, uint8_t* sf,
                                        void* stream);

/*
 * fp8q_grouped_mm_fp4 -- each expert's rows times its own weights: the GEMM of
 * fp8q_scaled_mm_fp4 for rows [offsets[e], offsets[e+1]) and weights b_q[e].
 *   a_q [M, K], a_sf  rows and scales as fp8q_moe_plan orders them; M is at
 *               least offsets[E] (rows from offsets[E] on are neither used nor
 *               written)
 *   b_q [E, N, K], b_sf  E matrices, their scales each in a buffer of
 *               fp8q_fp4_sf_bytes(N, K, format) bytes, one after the other
 *   b_gscale    fp32 [E] or NULL
 *   y           bf16 [M, N]
 */
FP8Q_API fp8q_status fp8q_grouped_mm_fp4(const void* a_q, const void* b_q, const uint8_t* a_sf,
                                         const uint8_t* b_sf, int format, const float* a_gscale,
                                         const float* b_gscale, const int* offsets,
                                         const int* sf_offsets, int64_t E, int64_t M, int64_t N,
                                         int64_t K, void* y, int64_t ldy, void* stream);

/*
 * fp8q_grouped_mm_fp4_silu_quant -- the experts' gate_up product with SiLU*mul
 * and the next quantization in its epilogue.  b_q [E, 2I, K] = [gate | up];
 * h = ga gb a b^T stays fp32, y = silu(h_gate) h_up (fp32, not rounded to
 * bf16; silu good to 2^-20 of itself for gates of at least -85, below to 2^-119),
 * then codes q [M, I] (I / 2 bytes a row) and scales sf at the same rows and
 * scale rows as the input, with tensor scale gscale.
 * I must be a multiple of 128 (else FP8Q_ERR_UNSUPPORTED; pad with zero rows).
 */
FP8Q_API fp8q_status fp8q_grouped_mm_fp4_silu_quant(const void* a_q, const void* b_q, const uint8_t* a_sf,
                                                    const uint8_t* b_sf, int format,
                                                    const float* a_gscale, const float* b_gscale,
                                                    const int* offsets, const int* sf_offsets, int64_t E,
                                                    int64_t M, int64_t I, int64_t K, const float* gscale,
                                                    void* q, uint8_t* sf, void* stream);

/*
 * fp8q_moe_combine -- y[t] = bf16_rn( sum_j weights[t, j] o[pos[t, j]] ), fp32,
 * j in order; negative positions add nothing.  o bf16 rows (ldo), y bf16
 * [T, H] (ldy), H a multiple of 8.
 */
FP8Q_API fp8q_status fp8q_moe_combine(const void* o, int64_t ldo, const int* pos, const float* weights,
                                      int64_t T, int topk, int64_t H, void* y, int64_t ldy, void* stream);

/*
 * fp8q_moe_experts_fp4 -- the experts' pass over T tokens: plan, quantization
 * into the experts' rows, gate_up product with SiLU*mul and quantization, down
 * product (its rows rounded to bf16), weighted sum.
 *   x bf16 [T, H] (ldx), ids int32 and weights fp32 [T, topk], contiguous
 *   w13 codes [E, 2I, H] = [gate | up], w2 codes [E, H, I], with their scales
 *   x_gscale, h_gscale   fp32 [1] or NULL: tensor scales of x and of the
 *               hidden activations; w13_gscale, w2_gscale  fp32 [E] or NULL
 *   y bf16 [T, H] (ldy; may not overlap x)
 *   workspace   fp8q_moe_experts_fp4_workspace_bytes(...) bytes, 256-byte
 *               aligned, of any content; calls that share one must not overlap
 *               in time
 *   E <= 512, topk <= 32, T topk <= 2^25, H a multiple of 32, I of 128
 */
FP8Q_API size_t fp8q_moe_experts_fp4_workspace_bytes(int64_t T, int topk, int64_t E, int64_t H, int64_t I,
                                                     int format);
FP8Q_API fp8q_status fp8q_moe_experts_fp4(const void* x, int64_t T, int64_t ldx, const int* ids,
                                          const float* weights, int topk, int64_t E, int64_t H, int64_t I,
                                          int format, const void* w13, const uint8_t* w13_sf,
                                          const void* w2, const uint8_t* w2_sf, const float* x_gscale,
                                          const float* w13_gscale, const float* h_gscale,
                                          const float* w2_gscale, void* y, int64_t ldy, void* workspace,
                                          size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8Q_FP4_H */
