// Products of a few activation rows with many weight rows, at the rate the
// weights arrive: each weight is read once from HBM straight into the
// registers that feed the matrix instruction, with no LDS between.
//
// The weights are the A operand (16 channels), the activation rows the B
// operand (16 columns) of a 16x16 product.  Lane l supplies 16 consecutive
// values of k, k0 + (l/16)*16 .., of weight row l%16 and of activation row
// l%16; since both operands use the same assignment of k to lanes, the sum
// over k is complete and only its order differs from the ascending one.
// Lane l gets channels (l/16)*4 + i, i < 4, of activation row l%16.
//
// Columns without a row of their own repeat another row's pointer: columns do
// not mix, so what they hold is dropped by the caller.
#pragma once

#include "experts.h"

namespace moe {

constexpr int kStreamStep = 64;  // values of k per step: 16 per lane, four lane groups

struct CoreBf16 {  // bf16 weights, bf16 activations
  typedef f32x4 Acc;
  static constexpr int kWBytes = 32, kXBytes = 32;  // per lane and step
  struct W { u32x4 v[2]; };
  struct X { u32x4 v[2]; };
  static __device__ __forceinline__ Acc mac(const W& w, const X& x, Acc c) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w.v[i]),
                                                  __builtin_bit_cast(bf16x8, x.v[i]), c, 0, 0, 0);
    return c;
  }
};

// Four 8-bit integers to bf16: every one of them is a bf16 value, so the
// conversion is exact and the high half of the fp32 form holds it.
__device__ __forceinline__ u32x2 bf16_of_i8(uint32_t w) {
  const float f0 = float(int8_t(w)), f1 = float(int8_t(w >> 8)), f2 = float(int8_t(w >> 16)),
              f3 = float(int32_t(w) >> 24);
  return u32x2{__builtin_amdgcn_perm(__float_as_uint(f1), __float_as_uint(f0), 0x07060302u),
               __builtin_amdgcn_perm(__float_as_uint(f3), __float_as_uint(f2), 0x07060302u)};
}

struct CoreI8Bf16 {  // int8 weights, bf16 activations
  typedef f32x4 Acc;
  static constexpr int kWBytes = 16, kXBytes = 32;
  struct W { u32x4 v[1]; };
  struct X { u32x4 v[2]; };
  static __device__ __forceinline__ Acc mac(const W& w, const X& x, Acc c) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const u32x2 a = bf16_of_i8(w.v[0][2 * i]), b = bf16_of_i8(w.v[0][2 * i + 1]);
      const u32x4 wb{a.x, a.y, b.x, b.y};
      c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wb),
                                                  __builtin_bit_cast(bf16x8, x.v[i]), c, 0, 0, 0);
    }
    return c;
  }
};

// Four e4m3 values to bf16, exact: four bits of mantissa, exponents from -9 to 8.
__device__ __forceinline__ u32x2 bf16_of_f8(uint32_t w) {
  return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true))};
}

struct CoreF8Bf16 {  // e4m3 weights, bf16 activations; block scales are the caller's
  typedef f32x4 Acc;
  static constexpr int kWBytes = 16, kXBytes = 32;
  struct W { u32x4 v[1]; };
  struct X { u32x4 v[2]; };
  static __device__ __forceinline__ Acc mac(const W& w, const X& x, Acc c) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const u32x2 a = bf16_of_f8(w.v[0][2 * i]), b = bf16_of_f8(w.v[0][2 * i + 1]);
      const u32x4 wb{a.x, a.y, b.x, b.y};
      c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wb),
                                                  __builtin_bit_cast(bf16x8, x.v[i]), c, 0, 0, 0);
    }
    return c;
  }
};

struct CoreI8 {  // int8 weights, int8 activations
  typedef i32x4 Acc;
  static constexpr int kWBytes = 16, kXBytes = 16;
  struct W { u32x4 v[1]; };
  struct X { u32x4 v[1]; };
  static __device__ __forceinline__ Acc mac(const W& w, const X& x, Acc c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w.v[0]),
                                                 __builtin_bit_cast(i32x4, x.v[0]), c, 0, 0, 0);
  }
};

// 16 bytes of a weight row.  A lane group's 16 bytes are an eighth of a cache
// line, whose rest the next step reads: plain loads, which keep the line,
// reached 6.3 TB/s over 7.5 GB, non-temporal ones 5.4 to 5.7.
__device__ __forceinline__ u32x4 load_weight(const uint8_t* p) {
  return *reinterpret_cast<const u32x4*>(p);
}

// acc[r][g] += the products of the weight rows w[r] and the activation rows
// x[g] over steps [begin, end) of kStreamStep values of k.  w and x point at
// this lane's row; `depth` values (a multiple of 16) are in a row, so in the
// last step a lane group may have nothing: both operands are zero then and
// nothing is read.  U steps are requested together, all of them before the
// first product: 50 rows on each of 4 experts, 4096 -> 2048 in int8: 18 us
// against 23 us where the compiler places the loads.
template <class C, int RT, int NG, int U>
__device__ __forceinline__ void stream_products(const uint8_t* const (&w)[RT], const uint8_t* const (&x)[NG],
                                                int begin, int end, int depth,
                                                typename C::Acc (&acc)[RT][NG]) {
  constexpr int WV = C::kWBytes / 16, XV = C::kXBytes / 16;
  const int group = __lane_id() / 16;
  const int whole = min(end, depth / kStreamStep);
  int s = begin;
  for (; s + U <= whole; s += U) {
    typename C::W wv[U][RT];
    typename C::X xv[U][NG];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < WV; ++i)
          wv[u][r].v[i] = load_weight(w[r] + (int64_t(s + u) * 4 + group) * C::kWBytes + 16 * i);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int i = 0; i < XV; ++i)
          xv[u][g].v[i] =
              *reinterpret_cast<const u32x4*>(x[g] + (int64_t(s + u) * 4 + group) * C::kXBytes + 16 * i);
    }
    __builtin_amdgcn_sched_barrier(0);  // or the loads are put between the products, to spare registers
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int g = 0; g < NG; ++g) acc[r][g] = C::mac(wv[u][r], xv[u][g], acc[r][g]);
  }
  for (; s < end; ++s) {
    const bool some = s * kStreamStep + group * 16 < depth;
    typename C::W wv[RT];
    typename C::X xv[NG];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int i = 0; i < WV; ++i)
        wv[r].v[i] = some ? load_weight(w[r] + (int64_t(s) * 4 + group) * C::kWBytes + 16 * i)
                          : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int i = 0; i < XV; ++i)
        xv[g].v[i] = some ? *reinterpret_cast<const u32x4*>(x[g] + (int64_t(s) * 4 + group) * C::kXBytes + 16 * i)
                          : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int g = 0; g < NG; ++g) acc[r][g] = C::mac(wv[r], xv[g], acc[r][g]);
  }
}

// The same for weights with a scale for each 128 values of k, two steps:
// scales[r][s / 2] is that of step s for the weight rows of this lane's sums.
template <class C, int RT, int NG, int U>
__device__ __forceinline__ void stream_scaled(const uint8_t* const (&w)[RT], const uint8_t* const (&x)[NG],
                                              const float* const (&scales)[RT], int begin, int end, int depth,
                                              typename C::Acc (&acc)[RT][NG]) {
  constexpr int WV = C::kWBytes / 16, XV = C::kXBytes / 16;
  const int group = __lane_id() / 16;
  for (int s = begin; s < end; s += U) {
    typename C::W wv[U][RT];
    typename C::X xv[U][NG];
    float sv[U][RT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool some = s + u < end && (s + u) * kStreamStep + group * 16 < depth;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        sv[u][r] = s + u < end ? scales[r][(s + u) / 2] : 0.0f;  // the sums are of all lane groups
#pragma unroll
        for (int i = 0; i < WV; ++i)
          wv[u][r].v[i] = some ? load_weight(w[r] + (int64_t(s + u) * 4 + group) * C::kWBytes + 16 * i)
                               : u32x4{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int i = 0; i < XV; ++i)
          xv[u][g].v[i] =
              some ? *reinterpret_cast<const u32x4*>(x[g] + (int64_t(s + u) * 4 + group) * C::kXBytes + 16 * i)
                   : u32x4{0u, 0u, 0u, 0u};
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const typename C::Acc part = C::mac(wv[u][r], xv[u][g], typename C::Acc{});
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][g][i] = __builtin_fmaf(part[i], sv[u][r], acc[r][g][i]);
        }
  }
}

// The same for e4m3 operands with a scale for each 128 values of k: a step is
// such a block, 32 values a lane and lane group, and its sums are multiplied
// with both scales in fp32 before they are added.  w_scales[r][s] and
// x_scales[g][s] are those of step s, for this lane's activation row.
template <int RT, int NG, int U>
__device__ __forceinline__ void stream_blocks(const uint8_t* const (&w)[RT], const uint8_t* const (&x)[NG],
                                              const float* const (&w_scales)[RT], const float* const (&x_scales)[NG],
                                              int begin, int end, int depth, f32x4 (&acc)[RT][NG]) {
  const int group = __lane_id() / 16;
  const u32x4 zero{0u, 0u, 0u, 0u};
  struct Bytes {
    u32x4 v[2];
  };
  for (int s = begin; s < end; s += U) {
    Bytes wv[U][RT], xv[U][NG];
    float sx[U][NG];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = (s + u) * kBlock + group * 32 + 16 * i;
        const bool some = s + u < end && at < depth;
#pragma unroll
        for (int r = 0; r < RT; ++r) wv[u][r].v[i] = some ? load_weight(w[r] + at) : zero;
#pragma unroll
        for (int g = 0; g < NG; ++g) xv[u][g].v[i] = some ? *reinterpret_cast<const u32x4*>(x[g] + at) : zero;
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int g = 0; g < NG; ++g) sx[u][g] = x_scales[g][min(s + u, end - 1)];
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        if (s + u >= end) continue;  // a scale that is NaN would make NaN of the zeros
        const float sw = w_scales[r][s + u];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const f32x4 part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              __builtin_bit_cast(i32x8, wv[u][r]), __builtin_bit_cast(i32x8, xv[u][g]), f32x4{}, 0, 0, 0, 0, 0, 0);
          const float scale = sx[u][g] * sw;
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][g][i] = __builtin_fmaf(part[i], scale, acc[r][g][i]);
        }
      }
  }
}

// Steps [begin, end) of part p of n over a row of `depth` values.
__device__ __forceinline__ void step_range(int depth, int p, int n, int& begin, int& end) {
  const int steps = (depth + kStreamStep - 1) / kStreamStep;
  begin = steps * p / n;  // steps <= 2^15
  end = steps * (p + 1) / n;
}

}  // namespace moe
