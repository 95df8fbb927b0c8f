// C entry points of the experts' products in floating point: argument checks,
// the gfx950 device check, then the launch.  Nothing here allocates,
// synchronises or reads device memory.
#include "moe_experts_float.h"

#include "entry_experts.h"
#include "experts.h"

namespace {

using namespace moe;

static_assert(MOE_F8_BLOCK == kBlock);

// Both grouped products; bf16 has no scales.
int expert_matmul(bool f8, const void* a, const float* a_scales, int64_t a_rows, const uint32_t* starts,
                  const int32_t* expert_ids, int32_t n_experts, const void* w, const float* w_scales, int32_t n_out,
                  int32_t depth, uint32_t flags, uint16_t* out, void* stream) {
  if (a_rows < 0 || a_rows > kMaxRows || n_experts < 1 || n_experts > MOE_MAX_EXPERTS || !width_ok(n_out) ||
      !width_ok(depth) || depth > MOE_MATMUL_MAX_DEPTH || (flags & ~MOE_MATMUL_SWIGLU) != 0)
    return MOE_ERR_INVALID_ARGUMENT;
  if (starts == nullptr || expert_ids == nullptr || w == nullptr || (f8 && w_scales == nullptr))
    return MOE_ERR_INVALID_ARGUMENT;
  if (a_rows > 0 && (a == nullptr || (f8 && a_scales == nullptr) || out == nullptr)) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(a, 16) || !aligned(a_scales, 4) || !aligned(starts, 4) || !aligned(expert_ids, 4) ||
      !aligned(w, 16) || !aligned(w_scales, 4) || !aligned(out, 16))
    return MOE_ERR_INVALID_ARGUMENT;
  const bool swiglu = (flags & MOE_MATMUL_SWIGLU) != 0;
  const uint64_t rows = uint64_t(a_rows), halves = swiglu ? 2 : 1, row_bytes = uint64_t(depth) * (f8 ? 1 : 2);
  if (clash({{a, rows * row_bytes},
             {a_scales, rows * blocks_of(depth) * 4},
             {starts, uint64_t(n_experts + 1) * 4},
             {expert_ids, uint64_t(n_experts) * 4},
             {w, uint64_t(n_experts) * halves * uint64_t(n_out) * row_bytes},
             {w_scales, uint64_t(n_experts) * halves * blocks_of(n_out) * blocks_of(depth) * 4}},
            {{out, rows * uint64_t(n_out) * 2}}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (const int d = check_device()) return d;
  const ExpertMatmul p{a, a_scales, uint32_t(a_rows), starts, expert_ids, n_experts, w, w_scales, n_out, depth, out};
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return launched(f8 ? launch_expert_matmul_f8(p, swiglu, s) : launch_expert_matmul_bf16(p, swiglu, s));
}

}  // namespace

extern "C" {

int moe_expert_matmul(const uint16_t* a, int64_t a_rows, const uint32_t* expert_start_indices,
                      const int32_t* expert_ids, int32_t n_experts, const uint16_t* w, int32_t n_out,
                      int32_t depth, uint32_t flags, uint16_t* out, void* stream) {
  return expert_matmul(false, a, nullptr, a_rows, expert_start_indices, expert_ids, n_experts, w, nullptr, n_out,
                       depth, flags, out, stream);
}

int moe_dispatch_f8(const uint16_t* input_tokens, int64_t n_rows, int32_t hidden, int32_t top_k,
                    const uint32_t* restore_token_order, uint8_t* out_q, float* out_scales,
                    int64_t out_rows, void* stream) {
  if (!slots_ok(n_rows, top_k) || !width_ok(hidden) || out_rows < 0) return MOE_ERR_INVALID_ARGUMENT;
  if (n_rows > 0 && (input_tokens == nullptr || restore_token_order == nullptr))
    return MOE_ERR_INVALID_ARGUMENT;
  if (out_rows > 0 && (out_q == nullptr || out_scales == nullptr)) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(input_tokens, 16) || !aligned(out_q, 16) || !aligned(out_scales, 4) ||
      !aligned(restore_token_order, 4))
    return MOE_ERR_INVALID_ARGUMENT;
  if (clash({{input_tokens, uint64_t(n_rows) * uint64_t(hidden) * 2},
             {restore_token_order, uint64_t(n_rows) * uint64_t(top_k) * 4}},
            {{out_q, uint64_t(out_rows) * uint64_t(hidden)},
             {out_scales, uint64_t(out_rows) * blocks_of(hidden) * 4}}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (const int d = check_device()) return d;
  return launched(launch_dispatch_f8(input_tokens, n_rows, hidden, top_k, restore_token_order, out_q, out_scales,
                                     out_rows, static_cast<hipStream_t>(stream)));
}

int moe_quantize_f8(const uint16_t* x, int64_t n_rows, int32_t hidden, const uint32_t* row_count,
                    uint8_t* out_q, float* out_scales, void* stream) {
  if (n_rows < 0 || n_rows > kMaxRows || !width_ok(hidden)) return MOE_ERR_INVALID_ARGUMENT;
  if (n_rows > 0 && (x == nullptr || out_q == nullptr || out_scales == nullptr))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(x, 16) || !aligned(out_q, 16) || !aligned(out_scales, 4) || !aligned(row_count, 4))
    return MOE_ERR_INVALID_ARGUMENT;
  const uint64_t n = uint64_t(n_rows) * uint64_t(hidden);
  if (clash({{x, 2 * n}, {row_count, 4}}, {{out_q, n}, {out_scales, uint64_t(n_rows) * blocks_of(hidden) * 4}}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (const int d = check_device()) return d;
  return launched(launch_quantize_f8(x, n_rows, hidden, row_count, out_q, out_scales,
                                     static_cast<hipStream_t>(stream)));
}

int moe_expert_matmul_f8(const uint8_t* a_q, const float* a_scales, int64_t a_rows,
                         const uint32_t* expert_start_indices, const int32_t* expert_ids,
                         int32_t n_experts, const uint8_t* w_q, const float* w_scales, int32_t n_out,
                         int32_t depth, uint32_t flags, uint16_t* out, void* stream) {
  return expert_matmul(true, a_q, a_scales, a_rows, expert_start_indices, expert_ids, n_experts, w_q, w_scales, n_out,
                       depth, flags, out, stream);
}

int moe_layer_few_f8(const uint16_t* x, int64_t n_rows, int32_t hidden, int32_t top_k,
                     const int32_t* topk_ids, const float* router_weights,
                     const int32_t* real_token_count, int32_t tp_rank, int32_t n_experts,
                     const uint8_t* w_gate_up, const float* gate_up_scales, const uint8_t* w_down,
                     const float* down_scales, int32_t inter, uint16_t* output_tokens,
                     void* workspace, size_t workspace_bytes, void* stream) {
  return layer_few_entry(true, x, n_rows, hidden, top_k, topk_ids, router_weights, real_token_count, tp_rank, n_experts,
                         w_gate_up, gate_up_scales, w_down, down_scales, inter, output_tokens, workspace,
                         workspace_bytes, stream);
}

int moe_layer_few_f8_i64(const uint16_t* x, int64_t n_rows, int32_t hidden, int32_t top_k,
                     const int64_t* topk_ids, const float* router_weights,
                     const int32_t* real_token_count, int32_t tp_rank, int32_t n_experts,
                     const uint8_t* w_gate_up, const float* gate_up_scales, const uint8_t* w_down,
                     const float* down_scales, int32_t inter, uint16_t* output_tokens,
                     void* workspace, size_t workspace_bytes, void* stream) {
  return layer_few_entry(true, x, n_rows, hidden, top_k, topk_ids, router_weights, real_token_count, tp_rank, n_experts,
                         w_gate_up, gate_up_scales, w_down, down_scales, inter, output_tokens, workspace,
                         workspace_bytes, stream);
}

}  // extern "C"
