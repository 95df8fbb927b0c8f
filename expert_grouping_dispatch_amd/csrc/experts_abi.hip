// C entry points of the experts' products: argument checks, the gfx950 device
// check, then the launch.  Nothing here allocates, synchronises or reads
// device memory.
#include "moe_experts.h"

#include <initializer_list>

#include "entry.h"
#include "experts.h"

namespace {

using moe::aligned;
using moe::check_device;
using moe::launched;
using moe::slots_ok;

constexpr int64_t kMaxRows = 0xFFFFFFFEll;
constexpr int32_t kMaxWidth = 1 << 20;
constexpr int32_t kMaxFewWidth = 1 << 17;  // 4 bytes each of MOE_FEW_MAX_SLOTS rows stay below 2^31

bool width_ok(int32_t n) { return n > 0 && n <= kMaxWidth && n % 16 == 0; }

struct Span {
  const void* at;
  uint64_t bytes;
};

bool overlap(const Span& a, const Span& b) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.at), q = reinterpret_cast<uintptr_t>(b.at);
  return a.at != nullptr && b.at != nullptr && a.bytes > 0 && b.bytes > 0 && p < q + b.bytes && q < p + a.bytes;
}

// Whether something written lies on something read or on something else written.
bool clash(std::initializer_list<Span> reads, std::initializer_list<Span> writes) {
  for (const Span* w = writes.begin(); w != writes.end(); ++w) {
    for (const Span& r : reads)
      if (overlap(r, *w)) return true;
    for (const Span* v = writes.begin(); v != w; ++v)
      if (overlap(*v, *w)) return true;
  }
  return false;
}

template <typename IdT>
int layer_few(const uint16_t* x, int64_t n_rows, int32_t hidden, int32_t top_k, const IdT* topk_ids,
              const float* router_weights, const int32_t* real_token_count, int32_t tp_rank,
              int32_t n_experts, const void* w_gate_up, const float* gate_up_scales,
              const void* w_down, const float* down_scales, int32_t inter, uint16_t* output_tokens,
              void* workspace, size_t workspace_bytes, void* stream) {
  const size_t need = moe_layer_few_workspace_bytes(n_rows, top_k, inter);
  if (need == 0 || !width_ok(hidden) || hidden > kMaxFewWidth || n_experts < 1 || n_experts > MOE_MAX_EXPERTS ||
      tp_rank < 0)
    return MOE_ERR_INVALID_ARGUMENT;
  if (w_gate_up == nullptr || w_down == nullptr || (gate_up_scales == nullptr) != (down_scales == nullptr))
    return MOE_ERR_INVALID_ARGUMENT;
  if (n_rows > 0 && (x == nullptr || topk_ids == nullptr || router_weights == nullptr ||
                     output_tokens == nullptr || workspace == nullptr))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(x, 16) || !aligned(topk_ids, sizeof(IdT)) || !aligned(router_weights, 4) ||
      !aligned(real_token_count, 4) || !aligned(w_gate_up, 16) || !aligned(gate_up_scales, 16) ||
      !aligned(w_down, 16) || !aligned(down_scales, 16) || !aligned(output_tokens, 16) ||
      !aligned(workspace, 256))
    return MOE_ERR_INVALID_ARGUMENT;
  if (n_rows > 0 && workspace_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const uint64_t row_bytes = uint64_t(n_rows) * uint64_t(hidden) * 2, slots = uint64_t(n_rows) * uint64_t(top_k);
  const uint64_t w_bytes = uint64_t(n_experts) * uint64_t(hidden) * uint64_t(inter) * (gate_up_scales == nullptr ? 2 : 1);
  const uint64_t channels = uint64_t(n_experts) * 4;
  if (clash({{x, row_bytes},
             {topk_ids, slots * sizeof(IdT)},
             {router_weights, slots * 4},
             {real_token_count, 4},
             {w_gate_up, 2 * w_bytes},
             {w_down, w_bytes},
             {gate_up_scales, channels * 2 * uint64_t(inter)},
             {down_scales, channels * uint64_t(hidden)}},
            {{output_tokens, row_bytes}, {workspace, n_rows > 0 ? need : 0}}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (const int d = check_device()) return d;
  const moe::FewLayer<IdT> p{x, int(n_rows), hidden, top_k, topk_ids, router_weights,
                             moe::PadMask{real_token_count, top_k, tp_rank}, n_experts, w_gate_up,
                             gate_up_scales, w_down, down_scales, inter, output_tokens,
                             static_cast<uint16_t*>(workspace)};
  return launched(moe::launch_layer_few(p, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int moe_dispatch_i8(const uint16_t* input_tokens, int64_t n_rows, int32_t hidden, int32_t top_k,
                    const uint32_t* restore_token_order, int8_t* out_q, float* out_scales,
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
            {{out_q, uint64_t(out_rows) * uint64_t(hidden)}, {out_scales, uint64_t(out_rows) * 4}}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (const int d = check_device()) return d;
  return launched(moe::launch_dispatch_i8(input_tokens, n_rows, hidden, top_k, restore_token_order,
                                          out_q, out_scales, out_rows,
                                          static_cast<hipStream_t>(stream)));
}

int moe_quantize_i8(const uint16_t* x, int64_t n_rows, int32_t hidden, const uint32_t* row_count,
                    int8_t* out_q, float* out_scales, void* stream) {
  if (n_rows < 0 || n_rows > kMaxRows || !width_ok(hidden)) return MOE_ERR_INVALID_ARGUMENT;
  if (n_rows > 0 && (x == nullptr || out_q == nullptr || out_scales == nullptr))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(x, 16) || !aligned(out_q, 16) || !aligned(out_scales, 4) || !aligned(row_count, 4))
    return MOE_ERR_INVALID_ARGUMENT;
  const uint64_t n = uint64_t(n_rows) * uint64_t(hidden);
  if (clash({{x, 2 * n}, {row_count, 4}}, {{out_q, n}, {out_scales, uint64_t(n_rows) * 4}}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (const int d = check_device()) return d;
  return launched(moe::launch_quantize_i8(x, n_rows, hidden, row_count, out_q, out_scales,
                                          static_cast<hipStream_t>(stream)));
}

int moe_expert_matmul_i8(const int8_t* a_q, const float* a_scales, int64_t a_rows,
                         const uint32_t* expert_start_indices, const int32_t* expert_ids,
                         int32_t n_experts, const int8_t* w_q, const float* w_scales,
                         int32_t n_out, int32_t depth, uint32_t flags, uint16_t* out,
                         void* stream) {
  if (a_rows < 0 || a_rows > kMaxRows || n_experts < 1 || n_experts > MOE_MAX_EXPERTS ||
      !width_ok(n_out) || !width_ok(depth) || depth > MOE_MATMUL_MAX_DEPTH ||
      (flags & ~MOE_MATMUL_SWIGLU) != 0)
    return MOE_ERR_INVALID_ARGUMENT;
  if (expert_start_indices == nullptr || expert_ids == nullptr || w_q == nullptr || w_scales == nullptr)
    return MOE_ERR_INVALID_ARGUMENT;
  if (a_rows > 0 && (a_q == nullptr || a_scales == nullptr || out == nullptr))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(a_q, 16) || !aligned(a_scales, 4) || !aligned(expert_start_indices, 4) ||
      !aligned(expert_ids, 4) || !aligned(w_q, 16) || !aligned(w_scales, 16) || !aligned(out, 16))
    return MOE_ERR_INVALID_ARGUMENT;
  const bool swiglu = (flags & MOE_MATMUL_SWIGLU) != 0;
  const uint64_t rows = uint64_t(a_rows), wide = uint64_t(n_experts) * uint64_t(n_out) * (swiglu ? 2 : 1);
  if (clash({{a_q, rows * uint64_t(depth)},
             {a_scales, rows * 4},
             {expert_start_indices, uint64_t(n_experts + 1) * 4},
             {expert_ids, uint64_t(n_experts) * 4},
             {w_q, wide * uint64_t(depth)},
             {w_scales, wide * 4}},
            {{out, rows * uint64_t(n_out) * 2}}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (const int d = check_device()) return d;
  const moe::ExpertMatmul p{a_q, a_scales, uint32_t(a_rows), expert_start_indices, expert_ids,
                            n_experts, w_q, w_scales, n_out, depth, out};
  return launched(moe::launch_expert_matmul_i8(p, swiglu, static_cast<hipStream_t>(stream)));
}

size_t moe_layer_few_workspace_bytes(int64_t n_rows, int32_t top_k, int32_t inter) {
  if (n_rows < 0 || top_k < 1 || top_k > MOE_MAX_TOP_K || n_rows > MOE_FEW_MAX_SLOTS / top_k ||
      !width_ok(inter) || inter > kMaxFewWidth)
    return 0;
  const size_t bytes = size_t(n_rows) * size_t(top_k) * size_t(inter) * 4;
  return bytes == 0 ? 256 : (bytes + 255) & ~size_t(255);
}

int moe_layer_few(const uint16_t* x, int64_t n_rows, int32_t hidden, int32_t top_k,
                  const int32_t* topk_ids, const float* router_weights,
                  const int32_t* real_token_count, int32_t tp_rank, int32_t n_experts,
                  const void* w_gate_up, const float* gate_up_scales, const void* w_down,
                  const float* down_scales, int32_t inter, uint16_t* output_tokens,
                  void* workspace, size_t workspace_bytes, void* stream) {
  return layer_few(x, n_rows, hidden, top_k, topk_ids, router_weights, real_token_count, tp_rank,
                   n_experts, w_gate_up, gate_up_scales, w_down, down_scales, inter, output_tokens,
                   workspace, workspace_bytes, stream);
}

int moe_layer_few_i64(const uint16_t* x, int64_t n_rows, int32_t hidden, int32_t top_k,
                      const int64_t* topk_ids, const float* router_weights,
                      const int32_t* real_token_count, int32_t tp_rank, int32_t n_experts,
                      const void* w_gate_up, const float* gate_up_scales, const void* w_down,
                      const float* down_scales, int32_t inter, uint16_t* output_tokens,
                      void* workspace, size_t workspace_bytes, void* stream) {
  return layer_few(x, n_rows, hidden, top_k, topk_ids, router_weights, real_token_count, tp_rank,
                   n_experts, w_gate_up, gate_up_scales, w_down, down_scales, inter, output_tokens,
                   workspace, workspace_bytes, stream);
}

}  // extern "C"
