/*
 * moe_experts.h -- C ABI of the experts' products between dispatch and
 * combine, in the same library (libmoe_route.so) and under the conventions
 * of moe_route.h: caller-owned buffers, no allocation, no host
 * synchronisation, device-resident counts, errors found on the host, bad
 * data never an access outside the buffers passed.
 *
 *   moe_dispatch_i8        token rows into the expert-contiguous buffer as
 *                          8-bit integers with one scale per row
 *   moe_quantize_i8        rows to 8-bit integers with one scale per row
 *   moe_expert_matmul_i8   every expert's product in 8-bit integers over the
 *                          expert-contiguous buffer, optionally with SwiGLU
 *   moe_layer_few          the whole layer (grouping, both products, SwiGLU,
 *                          weighted sum) for a few tokens, in two kernels
 *
 * A prefill runs moe_create_indices, moe_dispatch_i8, moe_expert_matmul_i8
 * with MOE_MATMUL_SWIGLU, moe_quantize_i8, moe_expert_matmul_i8 and
 * moe_combine; a decode step runs moe_layer_few on the same weights.
 */
#ifndef MOE_EXPERTS_H
#define MOE_EXPERTS_H

#include "moe_route.h"

#ifdef __cplusplus
extern "C" {
#endif

/* moe_expert_matmul_i8 flags */
#define MOE_MATMUL_SWIGLU 1u /* weights hold gate rows then up rows; out = silu(gate) * up */

#define MOE_MATMUL_MAX_DEPTH 131056 /* 128 * 128 * depth stays below 2^31 */
#define MOE_FEW_MAX_SLOTS 2048

/*
 * Dispatch in 8-bit integers.  As moe_dispatch, with each token row quantised
 * once and its payload and scale written to every position the row's slots
 * map to.  For a row x:
 *   a     = max(max |x|, 2^-118)
 *   scale = fl(a / 127), inv = fl(127 / a)           (fp32, each rounded once)
 *   q     = fl(x * inv) rounded to the nearest integer, ties to even; |q| <= 127.
 * A row that holds an infinity or a NaN gets scale NaN and an unspecified
 * payload, so that every product made of it is NaN; other rows are not
 * touched by it.
 *
 *   input_tokens, n_rows, top_k, restore_token_order  as moe_dispatch.
 *   hidden        > 0, a multiple of 16, at most 1048576.
 *   out_q         [device] int8 [out_rows, hidden], 16-byte aligned.
 *   out_scales    [device] fp32 [out_rows].  Neither of the outputs may overlap
 *                 an input or the other.
 * Rows no slot points to are left untouched; positions >= out_rows are
 * skipped.  Rows with nothing routed are not read.
 */
int moe_dispatch_i8(const uint16_t* input_tokens, int64_t n_rows, int32_t hidden, int32_t top_k,
                    const uint32_t* restore_token_order, int8_t* out_q, float* out_scales,
                    int64_t out_rows, void* stream);

/*
 * Rows to 8-bit integers, one scale per row, by the formula of
 * moe_dispatch_i8: the activations between two products, or weights laid out
 * once (a weight's output channels are its rows).
 *
 *   x             [device] bf16 [n_rows, hidden], 16-byte aligned.
 *   n_rows        0 <= n_rows <= 0xFFFFFFFE; hidden > 0, a multiple of 16,
 *                 at most 1048576.
 *   row_count     [device] uint32[1] or NULL: rows [0, min(n_rows, *row_count))
 *                 are quantised (expert_start_indices + n_experts holds the
 *                 number of routed slots); the others are neither read nor
 *                 written.  NULL: all n_rows.
 *   out_q         [device] int8 [n_rows, hidden], 16-byte aligned.
 *   out_scales    [device] fp32 [n_rows].  Neither of the outputs may overlap
 *                 an input or the other.
 */
int moe_quantize_i8(const uint16_t* x, int64_t n_rows, int32_t hidden, const uint32_t* row_count,
                    int8_t* out_q, float* out_scales, void* stream);

/*
 * The experts' products in 8-bit integers, with a scale for each row and each
 * output channel.  Row p of the expert-contiguous buffer belongs to the
 * active expert j with expert_start_indices[j] <= p < expert_start_indices[j+1],
 * whose weights are those of e = expert_ids[j]:
 *   c[p, n] = sum_k a_q[p, k] * w_q[e, n, k]                  (exact, int32)
 *   v[p, n] = fl(fl(fl(c) * a_scales[p]) * w_scales[e, n])    (fp32)
 *   out[p, n] = bf16(v[p, n])
 * With MOE_MATMUL_SWIGLU the weights of an expert are 2*n_out rows, the gate
 * rows first and the up rows after them, and
 *   out[p, n] = bf16(silu(v[p, n]) * v[p, n_out + n]),  silu(v) = v / (1 + exp(-v)).
 * Below v = -88.72 exp(-v) is infinite in fp32 and silu(v), less than 2^-121 in
 * magnitude, becomes -0.
 *
 *   a_q           [device] int8 [a_rows, depth], 16-byte aligned.
 *   a_scales      [device] fp32 [a_rows].
 *   a_rows        0 <= a_rows <= 0xFFFFFFFE: rows of a_q and out.  Rows at or
 *                 past expert_start_indices[n_experts] are neither read nor
 *                 written; starts beyond a_rows count as a_rows.
 *   expert_start_indices, expert_ids  from moe_create_indices, as it writes
 *                 them (device; the counts are never read on the host).  An
 *                 active expert with an id outside [0, n_experts) is skipped.
 *   n_experts     1 <= n_experts <= MOE_MAX_EXPERTS.
 *   w_q           [device] int8 [n_experts, n_out (2*n_out with SwiGLU), depth],
 *                 16-byte aligned.
 *   w_scales      [device] fp32 [n_experts, n_out (2*n_out with SwiGLU)], 16-byte aligned.
 *   n_out, depth  > 0, multiples of 16; depth <= MOE_MATMUL_MAX_DEPTH,
 *                 n_out <= 1048576.
 *   flags         0 or MOE_MATMUL_SWIGLU.
 *   out           [device] bf16 [a_rows, n_out], 16-byte aligned; must not
 *                 overlap the inputs.
 */
int moe_expert_matmul_i8(const int8_t* a_q, const float* a_scales, int64_t a_rows,
                         const uint32_t* expert_start_indices, const int32_t* expert_ids,
                         int32_t n_experts, const int8_t* w_q, const float* w_scales,
                         int32_t n_out, int32_t depth, uint32_t flags, uint16_t* out,
                         void* stream);

/*
 * Size in bytes of the scratch workspace of moe_layer_few (0 if the sizes
 * are out of range).  Never above 4*n_rows*top_k*inter + 256. [host]
 */
size_t moe_layer_few_workspace_bytes(int64_t n_rows, int32_t top_k, int32_t inter);

/*
 * The whole layer for a few tokens: from the routing map to the layer's
 * output in two kernels, with no index stage, dispatch or combine beside it.
 * For every token t and every routed choice j of it, with e = topk_ids[t, j]:
 *   g = w_gate_up[e][0:inter] x[t],  u = w_gate_up[e][inter:2*inter] x[t]
 *   h = silu(g) * u,                 y_j = w_down[e] h
 *   out[t] = bf16( sum_{j routed, ascending} router_weights[t, j] * y_j )
 * with fp32 sums, and silu as in moe_expert_matmul_i8.  Between the kernels h is
 * held as two bf16 values, 16 bits of mantissa.  Made for few slots on an expert:
 * its time grows with them.  From about two on each active expert the grouped
 * calls (moe_create_indices to moe_combine), whose activations have 8 bits then,
 * take less time on the GPU with 8-bit weights, and from about eight with bf16
 * ones.  Tokens without a routed choice are written as +0.
 * Infinities and NaNs in a token stay in its own output; an infinite weight
 * may give NaN where the formula gives an infinity.
 *
 *   x              [device] bf16 [n_rows, hidden], 16-byte aligned.
 *   n_rows, top_k  n_rows*top_k <= MOE_FEW_MAX_SLOTS, 1 <= top_k <= MOE_MAX_TOP_K.
 *   hidden, inter  > 0, multiples of 16, at most 131072.
 *   topk_ids       [device] int32 [n_rows, top_k]; ids outside [0, n_experts)
 *                  are unrouted.  Not modified.
 *   router_weights [device] fp32 [n_rows, top_k].
 *   real_token_count, tp_rank  as moe_mask_padding, or NULL and 0: rows at or
 *                  past the boundary are unrouted, whatever their ids are.
 *   n_experts      1 <= n_experts <= MOE_MAX_EXPERTS.
 *   w_gate_up      [device] [n_experts, 2*inter, hidden], 16-byte aligned:
 *                  bf16 where gate_up_scales is NULL, int8 otherwise.
 *   gate_up_scales [device] fp32 [n_experts, 2*inter], 16-byte aligned, or NULL.
 *   w_down         [device] [n_experts, hidden, inter], of the same type.
 *   down_scales    [device] fp32 [n_experts, hidden], 16-byte aligned; NULL
 *                  exactly where gate_up_scales is.
 *   output_tokens  [device] bf16 [n_rows, hidden], 16-byte aligned.  Neither it
 *                  nor the workspace may overlap the inputs or the other.
 *   workspace      [device] scratch of at least
 *                  moe_layer_few_workspace_bytes(n_rows, top_k, inter) bytes,
 *                  256-byte aligned; needs no initialisation.  Calls (and
 *                  captured graphs) that share one must not overlap.
 */
int moe_layer_few(const uint16_t* x, int64_t n_rows, int32_t hidden, int32_t top_k,
                  const int32_t* topk_ids, const float* router_weights,
                  const int32_t* real_token_count, int32_t tp_rank, int32_t n_experts,
                  const void* w_gate_up, const float* gate_up_scales, const void* w_down,
                  const float* down_scales, int32_t inter, uint16_t* output_tokens,
                  void* workspace, size_t workspace_bytes, void* stream);

/* As moe_layer_few for an int64 routing map. */
int moe_layer_few_i64(const uint16_t* x, int64_t n_rows, int32_t hidden, int32_t top_k,
                      const int64_t* topk_ids, const float* router_weights,
                      const int32_t* real_token_count, int32_t tp_rank, int32_t n_experts,
                      const void* w_gate_up, const float* gate_up_scales, const void* w_down,
                      const float* down_scales, int32_t inter, uint16_t* output_tokens,
                      void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERTS_H */
