// What the entry points of the experts' products share: the checks of sizes and
// of buffers that lie on one another, and the layer for a few tokens.
#pragma once

#include <initializer_list>

#include "entry.h"
#include "experts.h"
#include "moe_experts.h"

namespace moe {

constexpr int64_t kMaxRows = 0xFFFFFFFEll;
constexpr int32_t kMaxWidth = 1 << 20;
constexpr int32_t kMaxFewWidth = 1 << 17;  // 4 bytes each of MOE_FEW_MAX_SLOTS rows stay below 2^31

inline bool width_ok(int32_t n) { return n > 0 && n <= kMaxWidth && n % 16 == 0; }

struct Span {
  const void* at;
  uint64_t bytes;
};

inline bool overlap(const Span& a, const Span& b) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.at), q = reinterpret_cast<uintptr_t>(b.at);
  return a.at != nullptr && b.at != nullptr && a.bytes > 0 && b.bytes > 0 && p < q + b.bytes && q < p + a.bytes;
}

// Whether something written lies on something read or on something else written.
inline bool clash(std::initializer_list<Span> reads, std::initializer_list<Span> writes) {
  for (const Span* w = writes.begin(); w != writes.end(); ++w) {
    for (const Span& r : reads)
      if (overlap(r, *w)) return true;
    for (const Span* v = writes.begin(); v != w; ++v)
      if (overlap(*v, *w)) return true;
  }
  return false;
}

inline uint64_t blocks_of(int32_t n) { return (uint64_t(n) + kBlock - 1) / kBlock; }

// f8: e4m3 weights and scales of their blocks; without, bf16 ones or int8 ones with scales of their rows.
template <typename IdT>
int layer_few_entry(bool f8, const uint16_t* x, int64_t n_rows, int32_t hidden, int32_t top_k, const IdT* topk_ids,
                    const float* router_weights, const int32_t* real_token_count, int32_t tp_rank, int32_t n_experts,
                    const void* w_gate_up, const float* gate_up_scales, const void* w_down, const float* down_scales,
                    int32_t inter, uint16_t* output_tokens, void* workspace, size_t workspace_bytes, void* stream) {
  const size_t need = moe_layer_few_workspace_bytes(n_rows, top_k, inter);
  if (need == 0 || !width_ok(hidden) || hidden > kMaxFewWidth || n_experts < 1 || n_experts > MOE_MAX_EXPERTS ||
      tp_rank < 0)
    return MOE_ERR_INVALID_ARGUMENT;
  if (w_gate_up == nullptr || w_down == nullptr || (gate_up_scales == nullptr) != (down_scales == nullptr) ||
      (f8 && gate_up_scales == nullptr))
    return MOE_ERR_INVALID_ARGUMENT;
  if (n_rows > 0 && (x == nullptr || topk_ids == nullptr || router_weights == nullptr ||
                     output_tokens == nullptr || workspace == nullptr))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(x, 16) || !aligned(topk_ids, sizeof(IdT)) || !aligned(router_weights, 4) ||
      !aligned(real_token_count, 4) || !aligned(w_gate_up, 16) || !aligned(gate_up_scales, f8 ? 4 : 16) ||
      !aligned(w_down, 16) || !aligned(down_scales, f8 ? 4 : 16) || !aligned(output_tokens, 16) ||
      !aligned(workspace, 256))
    return MOE_ERR_INVALID_ARGUMENT;
  if (n_rows > 0 && workspace_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const uint64_t row_bytes = uint64_t(n_rows) * uint64_t(hidden) * 2, slots = uint64_t(n_rows) * uint64_t(top_k);
  const uint64_t w_bytes = uint64_t(n_experts) * uint64_t(hidden) * uint64_t(inter) * (gate_up_scales == nullptr ? 2 : 1);
  const uint64_t each = uint64_t(n_experts) * 4;
  const uint64_t up_bytes = 2 * each * (f8 ? blocks_of(inter) * blocks_of(hidden) : uint64_t(inter));
  const uint64_t down_bytes = each * (f8 ? blocks_of(inter) * blocks_of(hidden) : uint64_t(hidden));
  if (clash({{x, row_bytes},
             {topk_ids, slots * sizeof(IdT)},
             {router_weights, slots * 4},
             {real_token_count, 4},
             {w_gate_up, 2 * w_bytes},
             {w_down, w_bytes},
             {gate_up_scales, up_bytes},
             {down_scales, down_bytes}},
            {{output_tokens, row_bytes}, {workspace, n_rows > 0 ? need : 0}}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (const int d = check_device()) return d;
  const FewLayer<IdT> p{x, int(n_rows), hidden, top_k, topk_ids, router_weights,
                        PadMask{real_token_count, top_k, tp_rank}, n_experts, w_gate_up, gate_up_scales, w_down,
                        down_scales, inter, output_tokens, static_cast<uint16_t*>(workspace), f8};
  return launched(launch_layer_few(p, static_cast<hipStream_t>(stream)));
}

}  // namespace moe
