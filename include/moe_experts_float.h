/*
 * moe_experts_float.h -- C ABI of the experts' products in floating point, in
 * the same library (libmoe_route.so) and under the conventions of moe_route.h:
 * caller-owned buffers, no allocation, no host synchronisation, device-resident
 * counts, errors found on the host, bad data never an access outside the
 * buffers passed.
 *
 *   moe_expert_matmul      every expert's product in bf16 over the
 *                          expert-contiguous buffer, optionally with SwiGLU
 *   moe_dispatch_f8        token rows into the expert-contiguous buffer as e4m3
 *                          with one scale for each 128 values
 *   moe_quantize_f8        rows to e4m3 with one scale for each 128 values
 *   moe_expert_matmul_f8   every expert's product in e4m3, with a scale for each
 *                          128 values of a row and each 128 x 128 block of the
 *                          weights, optionally with SwiGLU
 *   moe_layer_few_f8       the whole layer for a few tokens on such weights
 *
 * e4m3 is the 8-bit format with four exponent and three mantissa bits, no
 * infinity, one NaN and 448 as its largest value; its values are passed as
 * their bytes (uint8_t).  A prefill in bf16 runs moe_create_indices,
 * moe_dispatch, moe_expert_matmul with MOE_MATMUL_SWIGLU, moe_expert_matmul and
 * moe_combine; one in e4m3 moe_create_indices, moe_dispatch_f8,
 * moe_expert_matmul_f8 with MOE_MATMUL_SWIGLU, moe_quantize_f8,
 * moe_expert_matmul_f8 and moe_combine.  A decode step runs moe_layer_few or
 * moe_layer_few_f8 on the same weights.
 */
#ifndef MOE_EXPERTS_FLOAT_H
#define MOE_EXPERTS_FLOAT_H

#include "moe_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_F8_BLOCK 128 /* values, and weight rows, that share a scale */

/*
 * Every expert's product in bf16.  Row p of the expert-contiguous buffer belongs
 * to the active expert j with expert_start_indices[j] <= p <
 * expert_start_indices[j+1], whose weights are those of e = expert_ids[j]:
 *   v[p, n] = sum_k a[p, k] * w[e, n, k]       (fp32)
 *   out[p, n] = bf16(v[p, n])
 * With MOE_MATMUL_SWIGLU the weights of an expert are 2*n_out rows, the gate
 * rows first and the up rows after them, and
 *   out[p, n] = bf16(silu(v[p, n]) * v[p, n_out + n]),  silu(v) = v / (1 + exp(-v)).
 * Below v = -88.72 exp(-v) is infinite in fp32 and silu(v), less than 2^-121 in
 * magnitude, becomes -0.
 * The order of a sum depends on the sizes, the other rows and the row's place among
 * them, but not on time: the same call gives the same bits.  Infinities and
 * NaNs in a row stay in its own output.
 *
 *   a             [device] bf16 [a_rows, depth], 16-byte aligned.
 *   a_rows        0 <= a_rows <= 0xFFFFFFFE: rows of a and out.  Rows at or
 *                 past expert_start_indices[n_experts] are neither read nor
 *                 written; starts beyond a_rows count as a_rows.
 *   expert_start_indices, expert_ids  from moe_create_indices, as it writes
 *                 them (device; the counts are never read on the host).  An
 *                 active expert with an id outside [0, n_experts) is skipped.
 *   n_experts     1 <= n_experts <= MOE_MAX_EXPERTS.
 *   w             [device] bf16 [n_experts, n_out (2*n_out with SwiGLU), depth],
 *                 16-byte aligned.
 *   n_out, depth  > 0, multiples of 16; depth <= MOE_MATMUL_MAX_DEPTH,
 *                 n_out <= 1048576.
 *   flags         0 or MOE_MATMUL_SWIGLU.
 *   out           [device] bf16 [a_rows, n_out], 16-byte aligned; must not
 *                 overlap the inputs.
 */
int moe_expert_matmul(const uint16_t* a, int64_t a_rows, const uint32_t* expert_start_indices,
                      const int32_t* expert_ids, int32_t n_experts, const uint16_t* w, int32_t n_out,
                      int32_t depth, uint32_t flags, uint16_t* out, void* stream);

/*
 * Dispatch in e4m3.  As moe_dispatch, with each token row quantised once and its
 * payload and scales written to every position the row's slots map to.  For
 * each block of 128 consecutive values x of a row (the last one may be shorter):
 *   a     = max(max |x|, 2^-116)
 *   scale = fl(a / 448), inv = fl(448 / a)           (fp32, each rounded once)
 *   q     = fl(x * inv) rounded to e4m3, ties to even; |q| <= 448.
 * A block that holds an infinity or a NaN gets scale NaN and an unspecified
 * payload, so that every product made of its row is NaN; other rows are not
 * touched by it.
 *
 *   input_tokens, n_rows, top_k, restore_token_order  as moe_dispatch.
 *   hidden        > 0, a multiple of 16, at most 1048576.
 *   out_q         [device] e4m3 [out_rows, hidden], 16-byte aligned.
 *   out_scales    [device] fp32 [out_rows, ceil(hidden / 128)].  Neither of the
 *                 outputs may overlap an input or the other.
 * Rows no slot points to are left untouched; positions >= out_rows are
 * skipped.  Rows with nothing routed are not read.
 */
int moe_dispatch_f8(const uint16_t* input_tokens, int64_t n_rows, int32_t hidden, int32_t top_k,
                    const uint32_t* restore_token_order, uint8_t* out_q, float* out_scales,
                    int64_t out_rows, void* stream);

/*
 * Rows to e4m3, one scale for each 128 values, by the formula of
 * moe_dispatch_f8: the activations between two products.
 *
 *   x             [device] bf16 [n_rows, hidden], 16-byte aligned.
 *   n_rows        0 <= n_rows <= 0xFFFFFFFE; hidden > 0, a multiple of 16,
 *                 at most 1048576.
 *   row_count     [device] uint32[1] or NULL: rows [0, min(n_rows, *row_count))
 *                 are quantised (expert_start_indices + n_experts holds the
 *                 number of routed slots); the others are neither read nor
 *                 written.  NULL: all n_rows.
 *   out_q         [device] e4m3 [n_rows, hidden], 16-byte aligned.
 *   out_scales    [device] fp32 [n_rows, ceil(hidden / 128)].  Neither of the
 *                 outputs may overlap an input or the other.
 */
int moe_quantize_f8(const uint16_t* x, int64_t n_rows, int32_t hidden, const uint32_t* row_count,
                    uint8_t* out_q, float* out_scales, void* stream);

/*
 * Every expert's product in e4m3.  As moe_expert_matmul, with
 *   v[p, n] = sum_b fl(a_scales[p, b] * w_scales[e, n / 128, b])
 *                   * sum_{k in block b} a_q[p, k] * w_q[e, n, k]     (fp32)
 * where block b is the values 128*b .. of k.  The last block of a row, and the
 * last block of weight rows, may be shorter.  The matrix unit adds the products
 * of a block eight at a time (values 8*i .. 8*i+7 of k), and of these eight it
 * cuts off what lies below 2^-13 of the largest one; all other sums are fp32.
 * A scale that is infinite or NaN makes every output that it enters infinite or
 * NaN, and no other.
 *
 *   a_q           [device] e4m3 [a_rows, depth], 16-byte aligned.
 *   a_scales      [device] fp32 [a_rows, ceil(depth / 128)].
 *   w_q           [device] e4m3 [n_experts, n_out (2*n_out with SwiGLU), depth],
 *                 16-byte aligned.
 *   w_scales      [device] fp32 [n_experts, ceil(n_out / 128), ceil(depth / 128)];
 *                 with SwiGLU [n_experts, 2 * ceil(n_out / 128), ceil(depth / 128)],
 *                 the blocks of the gate rows and then those of the up rows, each
 *                 counted from the first of its rows.
 *   The others as moe_expert_matmul.
 */
int moe_expert_matmul_f8(const uint8_t* a_q, const float* a_scales, int64_t a_rows,
                         const uint32_t* expert_start_indices, const int32_t* expert_ids,
                         int32_t n_experts, const uint8_t* w_q, const float* w_scales, int32_t n_out,
                         int32_t depth, uint32_t flags, uint16_t* out, void* stream);

/*
 * The whole layer for a few tokens, as moe_layer_few, on e4m3 weights with a
 * scale for each 128 x 128 block; the activations stay bf16.
 *
 *   w_gate_up      [device] e4m3 [n_experts, 2*inter, hidden], 16-byte aligned.
 *   gate_up_scales [device] fp32 [n_experts, 2 * ceil(inter / 128), ceil(hidden / 128)],
 *                  laid out as w_scales of moe_expert_matmul_f8 with SwiGLU.
 *   w_down         [device] e4m3 [n_experts, hidden, inter], 16-byte aligned.
 *   down_scales    [device] fp32 [n_experts, ceil(hidden / 128), ceil(inter / 128)].
 *   The others as moe_layer_few, the workspace's size among them.
 * A scale that is infinite or NaN makes what it enters infinite or NaN, as in
 * moe_expert_matmul_f8.
 */
int moe_layer_few_f8(const uint16_t* x, int64_t n_rows, int32_t hidden, int32_t top_k,
                     const int32_t* topk_ids, const float* router_weights,
                     const int32_t* real_token_count, int32_t tp_rank, int32_t n_experts,
                     const uint8_t* w_gate_up, const float* gate_up_scales, const uint8_t* w_down,
                     const float* down_scales, int32_t inter, uint16_t* output_tokens,
                     void* workspace, size_t workspace_bytes, void* stream);

/* As moe_layer_few_f8 for an int64 routing map. */
int moe_layer_few_f8_i64(const uint16_t* x, int64_t n_rows, int32_t hidden, int32_t top_k,
                         const int64_t* topk_ids, const float* router_weights,
                         const int32_t* real_token_count, int32_t tp_rank, int32_t n_experts,
                         const uint8_t* w_gate_up, const float* gate_up_scales,
                         const uint8_t* w_down, const float* down_scales, int32_t inter,
                         uint16_t* output_tokens, void* workspace, size_t workspace_bytes,
                         void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERTS_FLOAT_H */
