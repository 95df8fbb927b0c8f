// Host-side launchers and device-side pieces of the experts' products.
// Arguments are validated by the C entry points before a launcher is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"
#include "internal.h"

namespace moe {

hipError_t launch_dispatch_i8(const uint16_t* x, int64_t n_rows, int hidden, int top_k,
                              const uint32_t* restore, int8_t* q, float* scales, int64_t out_rows,
                              hipStream_t s);

hipError_t launch_quantize_i8(const uint16_t* x, int64_t n_rows, int hidden,
                              const uint32_t* row_count, int8_t* q, float* scales, hipStream_t s);

// The grouped int8 product.  `wide` rows of weights per expert: n_out, or
// 2*n_out with swiglu.
struct ExpertMatmul {
  const int8_t* a;
  const float* a_scales;
  uint32_t a_rows;
  const uint32_t* starts;
  const int32_t* expert_ids;
  int n_experts;
  const int8_t* w;
  const float* w_scales;
  int n_out;
  int depth;
  uint16_t* out;
};
hipError_t launch_expert_matmul_i8(const ExpertMatmul& p, bool swiglu, hipStream_t s);

// The whole layer for a few tokens; pad.count == nullptr masks nothing.
template <typename IdT>
struct FewLayer {
  const uint16_t* x;
  int n_rows;
  int hidden;
  int top_k;
  const IdT* ids;
  const float* router_weights;
  PadMask pad;
  int n_experts;
  const void* w_gate_up;
  const float* gate_up_scales;
  const void* w_down;
  const float* down_scales;
  int inter;
  uint16_t* out;
  uint16_t* h;  // [n_rows*top_k, inter], the workspace
};
template <typename IdT>
hipError_t launch_layer_few(const FewLayer<IdT>& p, hipStream_t s);

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// fp32 to bf16, round to nearest even; NaN stays NaN.
__device__ __forceinline__ uint32_t bf16_bits(float v) {
  const uint32_t u = __float_as_uint(v);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0x7FC0u;
  return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  return bf16_bits(lo) | (bf16_bits(hi) << 16);
}

// silu(g) * u = g / (1 + exp(-g)) * u in fp32.  exp(-g) overflows to
// infinity for g < -88.7, where silu(g) is below 2^-120: the quotient is -0.
__device__ __forceinline__ float silu_times(float g, float u) {
  return g / (1.0f + __expf(-g)) * u;
}

}  // namespace moe
