// Rows to e4m3 with one scale for each 128 values, in place order
// (moe_quantize_f8) or fanned out to the expert-contiguous buffer
// (moe_dispatch_f8).
//
//   a = max(max |x| over a block, 2^-116), scale = fl(a/448), inv = fl(448/a),
//   q = fl(x * inv) rounded to e4m3, ties to even.
//
// The floor 2^-116 keeps inv finite and scale a normal number for blocks of
// zeros and of subnormals.  |x| <= a gives |x*inv| <= 448*(1 + 2^-24), which
// rounds to at most 448.
//
// Bound by memory: 2 bytes read and top_k (or 1) written per value.  Blocks are
// independent, so a wave takes eight of them, 16 lanes each, with no exchange
// beyond the 16 lanes.  14000 rows of 14336 take 96 us (6.1 to 6.4 TB/s), 4096 rows of
// 7168 to 8 places each 46 us (6.5 TB/s, x out of the Infinity Cache).
#include "experts.h"
#include "rows.h"

namespace moe {

namespace {

constexpr int kChunk = 1024;    // values a wave takes: eight blocks
// Chunks of a row that a workgroup takes, one a wave: 14000 rows of 14336 in 95 us with 16, 99 with 8, 105 with 4, 111
// with 2.
constexpr int kMaxF8Waves = 16;
// moe_quantize_f8 loads and stores past the caches when what it reads and
// writes is more than the Infinity Cache holds.  moe_dispatch_f8 loads x
// plainly, as it mostly still lies in that cache, and streams its top_k times
// larger output.
constexpr int64_t kF8StreamMinBytes = int64_t(256) << 20;

constexpr int kDppRowRor1 = 0x121, kDppRowRor2 = 0x122, kDppRowRor4 = 0x124, kDppRowRor8 = 0x128;

// Largest value over each row of 16 lanes, returned to all of them.
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, dpp<kDppRowRor1, 0xF>(v));
  v = max(v, dpp<kDppRowRor2, 0xF>(v));
  v = max(v, dpp<kDppRowRor4, 0xF>(v));
  return max(v, dpp<kDppRowRor8, 0xF>(v));
}

// Four values in two words of bf16 to e4m3.
__device__ __forceinline__ uint32_t pack_f8(uint32_t w0, uint32_t w1, float inv) {
  const float a = __uint_as_float(w0 << 16) * inv, b = __uint_as_float(w0 & 0xFFFF0000u) * inv;
  const float c = __uint_as_float(w1 << 16) * inv, d = __uint_as_float(w1 & 0xFFFF0000u) * inv;
  const int low = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, low, true));
}

// The eight values of this lane, and the scale of the block that its row of 16 lanes holds.
__device__ __forceinline__ u32x2 block_f8(const u32x4& v, float& scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(v[i] & 0x7FFFu, (v[i] >> 16) & 0x7FFFu));
  const uint32_t bits = max(row_max(m) << 16, 0x05800000u);  // 2^-116; also orders infinities and NaNs above
  const float a = __uint_as_float(bits);
  scale = bits >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : a / 448.0f;
  const float inv = 448.0f / a;
  return u32x2{pack_f8(v.x, v.y, inv), pack_f8(v.z, v.w, inv)};
}

// One chunk of a row of `vecs` 16-byte vectors (an even number), from vector v0
// on.  Lane l loads vectors l and 64 + l, so that every load instruction reads
// whole cache lines, and stores the 16 bytes of payload of vectors l, l + 1
// (even lanes) or 63 + l, 64 + l (odd lanes).  `store(at, bytes)` writes 16
// bytes of the payload from byte 8*at, `scale_out(b, scale)` the scale of block b.
template <bool kNonTemporal, class Store, class ScaleOut>
__device__ __forceinline__ void quantize_chunk(const u32x4* __restrict__ src, int vecs, int v0, Store store,
                                               ScaleOut scale_out) {
  const int lane = threadIdx.x % kWave;
  const u32x4 zero{0u, 0u, 0u, 0u};
  const u32x4 lo = v0 + lane < vecs ? load_vec<kNonTemporal>(src + v0 + lane) : zero;
  const u32x4 hi = v0 + kWave + lane < vecs ? load_vec<kNonTemporal>(src + v0 + kWave + lane) : zero;
  float s_lo, s_hi;
  const u32x2 l = block_f8(lo, s_lo), h = block_f8(hi, s_hi);
  const bool odd = lane & 1;
  const u32x2 give{odd ? l.x : h.x, odd ? l.y : h.y};
  const u32x2 got{dpp<kDppQuadSwap1, 0xF>(give.x), dpp<kDppQuadSwap1, 0xF>(give.y)};
  const int at = odd ? v0 + kWave + lane - 1 : v0 + lane;
  if (at < vecs) store(at, odd ? u32x4{got.x, got.y, h.x, h.y} : u32x4{l.x, l.y, got.x, got.y});
  // Two lanes of each 16 write: blocks 0 to 3 of the chunk, blocks 4 to 7.
  const int b = v0 / 16 + (odd ? 4 : 0) + lane / 16;
  if (lane % 16 < 2 && b * 16 < vecs) scale_out(b, odd ? s_hi : s_lo);
}

}  // namespace

// kStream: loads and stores past the caches, for rows that do not fit them.
template <bool kStream>
__global__ __launch_bounds__(kMaxF8Waves* kWave) void k_quantize_f8(
    const u32x4* __restrict__ x, int64_t n_rows, int vecs, const uint32_t* __restrict__ row_count,
    uint8_t* __restrict__ q, float* __restrict__ scales) {
  const int64_t rows = row_count == nullptr ? n_rows : min(n_rows, int64_t(*row_count));
  const int v0 = int(blockIdx.y * (blockDim.x / kWave) + threadIdx.x / kWave) * (kChunk / 8);
  const int blocks = (vecs + 15) / 16;
  if (v0 >= vecs) return;
  for (int64_t t = blockIdx.x; t < rows; t += gridDim.x) {
    uint8_t* dst = q + t * vecs * 8;
    quantize_chunk<kStream>(
        x + t * vecs, vecs, v0,
        [&](int at, const u32x4& b) { store_vec<kStream>(reinterpret_cast<u32x4*>(dst + 8 * at), b); },
        [&](int b, float s) { scales[t * blocks + b] = s; });
  }
}

// K > 0: top_k == K, positions in scalar registers; K == 0: any top_k, positions read again for each store.
template <int K>
__global__ __launch_bounds__(kMaxF8Waves* kWave) void k_dispatch_f8(
    const u32x4* __restrict__ x, int64_t n_rows, int vecs, int top_k, const uint32_t* __restrict__ restore,
    uint8_t* __restrict__ q, float* __restrict__ scales, uint32_t limit) {
  constexpr int KR = K > 0 ? K : 1;
  const int v0 = int(blockIdx.y * (blockDim.x / kWave) + threadIdx.x / kWave) * (kChunk / 8);
  const int blocks = (vecs + 15) / 16;
  if (v0 >= vecs) return;
  for (int64_t t = blockIdx.x; t < n_rows; t += gridDim.x) {
    uint32_t pos[KR];
    float unused[KR];
    bool some = false;
    if constexpr (K > 0) {
      uniform_slots<K, false>(restore, nullptr, t, limit, pos, unused);
#pragma unroll
      for (int j = 0; j < K; ++j) some = some || pos[j] != kSent;
    } else {
      for (int j = 0; j < top_k; ++j) some = some || restore[t * top_k + j] < limit;
    }
    if (!some) continue;
    const int nj = K > 0 ? K : top_k;
    auto position = [&](int j) {
      const uint32_t p = K > 0 ? pos[j] : restore[t * top_k + j];
      return p < limit ? p : kSent;
    };
    quantize_chunk<false>(
        x + t * vecs, vecs, v0,
        [&](int at, const u32x4& b) {
#pragma unroll
          for (int j = 0; j < nj; ++j)
            if (const uint32_t p = position(j); p != kSent)
              __builtin_nontemporal_store(b, reinterpret_cast<u32x4*>(q + (int64_t(p) * vecs + at) * 8));
        },
        [&](int b, float s) {
#pragma unroll
          for (int j = 0; j < nj; ++j)
            if (const uint32_t p = position(j); p != kSent) scales[int64_t(p) * blocks + b] = s;
        });
  }
}

namespace {

// Workgroups for each row, and their waves: as few as hold its chunks, of nearly the same size.
dim3 f8_grid(int64_t n_rows, int vecs, dim3& block) {
  const int chunks = (vecs + kChunk / 8 - 1) / (kChunk / 8), parts = (chunks + kMaxF8Waves - 1) / kMaxF8Waves;
  block = dim3((chunks + parts - 1) / parts * kWave);
  return dim3(row_grid(n_rows), parts);
}

template <int K>
struct LaunchDispatchF8 {
  static hipError_t run(const u32x4* x, int64_t n_rows, int vecs, int top_k, const uint32_t* restore, uint8_t* q,
                        float* scales, uint32_t limit, hipStream_t s) {
    dim3 block;
    const dim3 grid = f8_grid(n_rows, vecs, block);
    hipLaunchKernelGGL((k_dispatch_f8<K>), grid, block, 0, s, x, n_rows, vecs, top_k, restore, q, scales, limit);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_dispatch_f8(const uint16_t* x, int64_t n_rows, int hidden, int top_k, const uint32_t* restore,
                              uint8_t* q, float* scales, int64_t out_rows, hipStream_t s) {
  if (n_rows == 0) return hipSuccess;
  return by_top_k<LaunchDispatchF8>(top_k, reinterpret_cast<const u32x4*>(x), n_rows, hidden / 8, top_k, restore, q,
                                    scales, position_limit(out_rows), s);
}

hipError_t launch_quantize_f8(const uint16_t* x, int64_t n_rows, int hidden, const uint32_t* row_count, uint8_t* q,
                              float* scales, hipStream_t s) {
  if (n_rows == 0) return hipSuccess;
  dim3 block;
  const dim3 grid = f8_grid(n_rows, hidden / 8, block);
  const u32x4* xv = reinterpret_cast<const u32x4*>(x);
  if (double(n_rows) * hidden * 3 >= double(kF8StreamMinBytes))
    hipLaunchKernelGGL((k_quantize_f8<true>), grid, block, 0, s, xv, n_rows, hidden / 8, row_count, q, scales);
  else
    hipLaunchKernelGGL((k_quantize_f8<false>), grid, block, 0, s, xv, n_rows, hidden / 8, row_count, q, scales);
  return hipGetLastError();
}

}  // namespace moe
