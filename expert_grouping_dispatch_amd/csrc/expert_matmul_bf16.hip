// The experts' products in bf16 over the expert-contiguous buffer.
//
//   v[p, n] = sum_k a[p, k] * w[e(p), n, k]  (fp32)
//   out = bf16(v), or bf16(silu(gate) * up) of two of them
//
// The kernels are those of the 8-bit integers: a step is 128 bytes of a row, so
// 64 values of k, and a matrix instruction takes the same 16 bytes a lane.
//
// Tiles are bound by the matrix units and the clock that random operands leave
// them (14000 rows on 8 experts, 4096 -> 2 x 14336: 2690 to 2770 us, 1.2e15
// operations/s, 69% busy at 1.6 GHz; the instructions alone would take 2260), strips
// by reading the weights (6.2 TB/s), few rows by a few rounds of loads (24 experts,
// 2 rows each, 1040 -> 528: 6.7 us a call).
#include "expert_matmul.h"

namespace moe {

namespace {

struct MatBf16 {
  static constexpr int kSize = 2;
  static constexpr bool kFloat = true, kChannels = false, kBlocks = false;
  static constexpr int kFewPerSimd = 3;
  static constexpr uint32_t kStripsMin = 160;
  typedef f32x16 Acc;
  typedef CoreBf16 Few;
  typedef f32x4 FewAcc;
  static __device__ __forceinline__ Acc mac(const u32x4& w, const u32x4& a, const Acc& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, a), c, 0, 0,
                                                   0);
  }
  static __device__ __forceinline__ float value(float c, float, float) { return c; }
  template <bool kSwiglu>
  static void tiles(const ExpertMatmul& p, hipStream_t s) {
    hipLaunchKernelGGL((k_matmul_tile<MatBf16, kSwiglu>), dim3(256), dim3(kTileThreads), 0, s, p);
  }
};

}  // namespace

hipError_t launch_expert_matmul_bf16(const ExpertMatmul& p, bool swiglu, hipStream_t s) {
  if (p.a_rows == 0) return hipSuccess;
  return swiglu ? go_matmul<MatBf16, true>(p, s) : go_matmul<MatBf16, false>(p, s);
}

}  // namespace moe
