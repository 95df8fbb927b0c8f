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
  uint16_t* h;  // two [n_rows*top_k, inter], the workspace
};
template <typename IdT>
hipError_t launch_layer_few(const FewLayer<IdT>& p, hipStream_t s);

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two fp32 values to bf16, round to nearest even; NaN stays NaN.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

// A value that is the same in all lanes, in a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return uint32_t(__builtin_amdgcn_readfirstlane(int(v))); }

__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  return reinterpret_cast<const uint8_t*>(uint64_t(uniform(uint32_t(v >> 32))) << 32 | uniform(uint32_t(v)));
}

// The upper half of `a`'s lanes changes places with the lower half of `b`'s.
__device__ __forceinline__ u32x2 permlane32_swap(uint32_t a, uint32_t b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  return u32x2{r[0], r[1]};
}

// The odd rows of 16 of `a`'s lanes change places with the even rows of `b`'s.
__device__ __forceinline__ u32x2 permlane16_swap(uint32_t a, uint32_t b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  return u32x2{r[0], r[1]};
}

// silu(g) * u = g / (1 + exp(-g)) * u in fp32.  exp(-g) overflows to
// infinity for g < -88.7, where silu(g) is below 2^-120: the quotient is -0.
__device__ __forceinline__ float silu_times(float g, float u) {
  return g / (1.0f + __expf(-g)) * u;
}

}  // namespace moe
