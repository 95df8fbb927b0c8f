// Rows to 8-bit integers with one scale per row, in place order
// (moe_quantize_i8) or fanned out to the expert-contiguous buffer
// (moe_dispatch_i8).
//
//   a = max(max |x|, 2^-118), scale = fl(a/127), inv = fl(127/a),
//   q = fl(x * inv) rounded to nearest, ties to even.
//
// The floor 2^-118 keeps inv finite and scale a normal number for rows of
// zeros and of subnormals.  |x| <= a gives |x*inv| <= 127*(1 + 2^-24), which
// rounds to at most 127.
//
// Bound by memory: 2 bytes read and top_k (or 1) written per element, a dozen
// vector operations between them.  One workgroup per row holds the row in
// registers across the two passes (largest value, then the payload), so x is
// read once; longer rows (above 32768 elements) are read again, from cache.
#include "experts.h"
#include "rows.h"

namespace moe {

namespace {

constexpr int kMaxI8Threads = 512;

// Largest 15-bit magnitude of the sixteen bf16 values of a unit.
__device__ __forceinline__ uint32_t unit_amax(const u32x4& v0, const u32x4& v1) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m = max(m, max(v0[i] & 0x7FFFu, (v0[i] >> 16) & 0x7FFFu));
    m = max(m, max(v1[i] & 0x7FFFu, (v1[i] >> 16) & 0x7FFFu));
  }
  return m;
}

// Two bf16 values of a 32-bit word to 8-bit integers in the low bytes of two
// words.  Adding 1.5 * 2^23 rounds to the nearest integer, ties to even, and
// leaves its two's complement in the low bits.
__device__ __forceinline__ void word_i8(uint32_t w, float inv, uint32_t& lo, uint32_t& hi) {
  const float a = __uint_as_float(w << 16) * inv;
  const float b = __uint_as_float(w & 0xFFFF0000u) * inv;
  lo = __float_as_uint(a + 12582912.0f);
  hi = __float_as_uint(b + 12582912.0f);
}

__device__ __forceinline__ uint32_t pack_i8(uint32_t w0, uint32_t w1, float inv) {
  uint32_t b0, b1, b2, b3;
  word_i8(w0, inv, b0, b1);
  word_i8(w1, inv, b2, b3);
  const uint32_t l = __builtin_amdgcn_perm(b1, b0, 0x0C0C0400u);  // byte 0 of b0, byte 0 of b1
  const uint32_t h = __builtin_amdgcn_perm(b3, b2, 0x04000C0Cu);
  return l | h;
}

__device__ __forceinline__ u32x4 unit_i8(const u32x4& v0, const u32x4& v1, float inv) {
  return u32x4{pack_i8(v0.x, v0.y, inv), pack_i8(v0.z, v0.w, inv), pack_i8(v1.x, v1.y, inv),
               pack_i8(v1.z, v1.w, inv)};
}

// scale and inverse of a row whose largest 15-bit magnitude is `amax`.
__device__ __forceinline__ void row_scale(uint32_t amax, float& scale, float& inv) {
  const uint32_t bits = max(amax << 16, 0x04800000u);  // 2^-118; also orders infinities and NaNs above
  const float a = __uint_as_float(bits);
  scale = bits >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : a / 127.0f;
  inv = 127.0f / a;
}

// Largest `v` over the workgroup, returned to every lane.
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* s_part) {
  v = wave_max(v);
  const int waves = blockDim.x / kWave;
  if (waves == 1) return v;
  if ((threadIdx.x & (kWave - 1)) == 0) s_part[threadIdx.x / kWave] = v;
  __syncthreads();
  v = s_part[0];
  for (int i = 1; i < waves; ++i) v = max(v, s_part[i]);
  return v;
}

// One workgroup per row t; lane u owns the units (16 elements: 32 bytes in,
// 16 out) u, u + lanes, ...  U > 0: at most U units per lane, held in
// registers; U == 0: any number, read twice.  `store(unit, bytes)` writes one
// unit of the payload, `scale_out(scale)` runs on lane 0.
template <int U, class Store, class ScaleOut>
__device__ __forceinline__ void quantize_row(const u32x4* __restrict__ src, int units, uint32_t* s_part,
                                             Store store, ScaleOut scale_out) {
  const int tid = threadIdx.x, lanes = blockDim.x;
  uint32_t amax = 0;
  float scale, inv;
  if constexpr (U > 0) {
    u32x4 v[U][2];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = tid + i * lanes;
      if (u < units) {
        v[i][0] = src[2 * u];
        v[i][1] = src[2 * u + 1];
        amax = max(amax, unit_amax(v[i][0], v[i][1]));
      }
    }
    row_scale(block_max(amax, s_part), scale, inv);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = tid + i * lanes;
      if (u < units) store(u, unit_i8(v[i][0], v[i][1], inv));
    }
  } else {
    for (int u = tid; u < units; u += lanes) amax = max(amax, unit_amax(src[2 * u], src[2 * u + 1]));
    row_scale(block_max(amax, s_part), scale, inv);
    for (int u = tid; u < units; u += lanes) store(u, unit_i8(src[2 * u], src[2 * u + 1], inv));
  }
  if (tid == 0) scale_out(scale);
}

}  // namespace

template <int U>
__global__ __launch_bounds__(kMaxI8Threads) void k_quantize_i8(
    const u32x4* __restrict__ x, int64_t n_rows, int units, const uint32_t* __restrict__ row_count,
    u32x4* __restrict__ q, float* __restrict__ scales) {
  __shared__ uint32_t s_part[kMaxI8Threads / kWave];
  const int64_t rows = row_count == nullptr ? n_rows : min(n_rows, int64_t(*row_count));
  for (int64_t t = blockIdx.x; t < rows; t += gridDim.x) {
    u32x4* dst = q + t * units;
    quantize_row<U>(
        x + t * units * 2, units, s_part, [&](int u, const u32x4& b) { dst[u] = b; },
        [&](float s) { scales[t] = s; });
    __syncthreads();  // s_part is rewritten for the next row
  }
}

// K > 0: top_k == K, positions in scalar registers; K == 0: any top_k,
// positions compacted into LDS by wave 0.
template <int K, int U>
__global__ __launch_bounds__(kMaxI8Threads) void k_dispatch_i8(
    const u32x4* __restrict__ x, int64_t n_rows, int units, int top_k,
    const uint32_t* __restrict__ restore, u32x4* __restrict__ q, float* __restrict__ scales,
    uint32_t limit) {
  __shared__ uint32_t s_part[kMaxI8Threads / kWave];
  __shared__ uint32_t s_pos[K > 0 ? 1 : kMaxTopK];
  __shared__ int s_n;
  constexpr int KR = K > 0 ? K : 1;
  for (int64_t t = blockIdx.x; t < n_rows; t += gridDim.x) {
    uint32_t pos[KR];
    float unused[KR];
    int n;
    if constexpr (K > 0) {
      uniform_slots<K, false>(restore, nullptr, t, limit, pos, unused);
      n = 0;
#pragma unroll
      for (int j = 0; j < K; ++j) n += pos[j] != kSent ? 1 : 0;
    } else {
      n = gather_routed(restore, nullptr, t, top_k, limit, s_pos, nullptr, &s_n);
    }
    const int nj = K > 0 ? K : n;
    if (n > 0) {
      quantize_row<U>(
          x + t * units * 2, units, s_part,
          [&](int u, const u32x4& b) {
#pragma unroll
            for (int j = 0; j < nj; ++j) {
              const uint32_t p = K > 0 ? pos[j] : s_pos[j];
              if (p != kSent) __builtin_nontemporal_store(b, q + int64_t(p) * units + u);
            }
          },
          [&](float s) {
#pragma unroll
            for (int j = 0; j < nj; ++j) {
              const uint32_t p = K > 0 ? pos[j] : s_pos[j];
              if (p != kSent) scales[p] = s;
            }
          });
    }
    __syncthreads();  // s_part and s_pos are rewritten for the next token
  }
}

namespace {

// Lanes for a row: the fewest whole waves with a unit per lane, at most
// kMaxI8Threads.
int i8_threads(int units) {
  const int t = (units + kWave - 1) / kWave * kWave;
  return t < kMaxI8Threads ? t : kMaxI8Threads;
}

template <int K>
struct LaunchDispatchI8 {
  static hipError_t run(const u32x4* x, int64_t n_rows, int units, int top_k, const uint32_t* restore,
                        u32x4* q, float* scales, uint32_t limit, hipStream_t s) {
    const int threads = i8_threads(units), per = (units + threads - 1) / threads;
    const dim3 grid(row_grid(n_rows)), block(threads);
#define MOE_GO(U)                                                                                     \
  hipLaunchKernelGGL((k_dispatch_i8<K, U>), grid, block, 0, s, x, n_rows, units, top_k, restore, q, \
                     scales, limit)
    if (per == 1) MOE_GO(1);
    else if (per == 2) MOE_GO(2);
    else if (per <= 4) MOE_GO(4);
    else MOE_GO(0);
#undef MOE_GO
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_dispatch_i8(const uint16_t* x, int64_t n_rows, int hidden, int top_k,
                              const uint32_t* restore, int8_t* q, float* scales, int64_t out_rows,
                              hipStream_t s) {
  if (n_rows == 0) return hipSuccess;
  return by_top_k<LaunchDispatchI8>(top_k, reinterpret_cast<const u32x4*>(x), n_rows, hidden / 16, top_k,
                                    restore, reinterpret_cast<u32x4*>(q), scales,
                                    position_limit(out_rows), s);
}

hipError_t launch_quantize_i8(const uint16_t* x, int64_t n_rows, int hidden,
                              const uint32_t* row_count, int8_t* q, float* scales, hipStream_t s) {
  if (n_rows == 0) return hipSuccess;
  const int units = hidden / 16;
  const int threads = i8_threads(units), per = (units + threads - 1) / threads;
  const dim3 grid(row_grid(n_rows)), block(threads);
  const u32x4* xv = reinterpret_cast<const u32x4*>(x);
  u32x4* qv = reinterpret_cast<u32x4*>(q);
#define MOE_GO(U) \
  hipLaunchKernelGGL((k_quantize_i8<U>), grid, block, 0, s, xv, n_rows, units, row_count, qv, scales)
  if (per == 1) MOE_GO(1);
  else if (per == 2) MOE_GO(2);
  else if (per <= 4) MOE_GO(4);
  else MOE_GO(0);
#undef MOE_GO
  return hipGetLastError();
}

}  // namespace moe
