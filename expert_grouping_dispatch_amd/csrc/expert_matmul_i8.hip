// The experts' products in 8-bit integers over the expert-contiguous buffer.
//
//   c[p, n] = sum_k a[p, k] * w[e(p), n, k]  (int32, exact in any order)
//   out = bf16(fl(fl(fl(c) * sa[p]) * sw[e, n])), or silu(gate) * up of two of them
//
// Strips: 776 rows on 247 experts, 7168 -> 2048 with SwiGLU: 1025 us, 7.0 TB/s.
// Tiles: 14000 rows on 8 experts, 4096 -> 14336 with SwiGLU: 1.50 ms, 2.2e15
// operations/s, as many as the library's product of 8192 x 8192 x 8192 reaches.
// The clock falls with what the operands switch (zeros take 10% less time).
#include "expert_matmul.h"

namespace moe {

namespace {

struct MatI8 {
  static constexpr int kSize = 1;
  static constexpr bool kFloat = false, kChannels = true, kBlocks = false;
  static constexpr int kFewPerSimd = 4;
  static constexpr uint32_t kStripsMin = 256;
  typedef i32x16 Acc;
  typedef CoreI8 Few;
  typedef i32x4 FewAcc;
  static __device__ __forceinline__ Acc mac(const u32x4& w, const u32x4& a, const Acc& c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, w), __builtin_bit_cast(i32x4, a), c, 0, 0, 0);
  }
  static __device__ __forceinline__ float value(int32_t c, float sa, float sw) { return scaled(c, sa, sw); }
  template <bool kSwiglu>
  static void tiles(const ExpertMatmul& p, hipStream_t s) {
    hipLaunchKernelGGL((k_matmul_tile<MatI8, kSwiglu>), dim3(256), dim3(kTileThreads), 0, s, p);
  }
};

}  // namespace

hipError_t launch_expert_matmul_i8(const ExpertMatmul& p, bool swiglu, hipStream_t s) {
  if (p.a_rows == 0) return hipSuccess;
  return swiglu ? go_matmul<MatI8, true>(p, s) : go_matmul<MatI8, false>(p, s);
}

}  // namespace moe
