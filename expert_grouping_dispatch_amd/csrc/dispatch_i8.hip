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
// moe_quantize_i8 loads and stores past the caches when what it reads and
// writes is more than the Infinity Cache holds: 14000 rows of 14336 values
// (602 MB) took 93 us against 108 us with plain accesses.  moe_dispatch_i8
// loads x plainly, as it mostly still lies in that cache (4096 rows of 7168:
// 46 us against 59 us), and streams its top_k times larger output.
constexpr int64_t kI8StreamMinBytes = int64_t(256) << 20;

// Largest 15-bit magnitude of eight bf16 values.
__device__ __forceinline__ uint32_t vec_amax(const u32x4& v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(v[i] & 0x7FFFu, (v[i] >> 16) & 0x7FFFu));
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

// Sixteen bytes of payload of the eight values this lane has in `lo` and in
// `hi` and those of its neighbour: the even lane of a pair gets what follows
// from both `lo`, the odd lane what follows from both `hi`.
__device__ __forceinline__ u32x4 pair_i8(const u32x4& lo, const u32x4& hi, float inv) {
  const u32x2 l{pack_i8(lo.x, lo.y, inv), pack_i8(lo.z, lo.w, inv)};
  const u32x2 h{pack_i8(hi.x, hi.y, inv), pack_i8(hi.z, hi.w, inv)};
  const bool odd = threadIdx.x & 1;
  const u32x2 give{odd ? l.x : h.x, odd ? l.y : h.y};
  const u32x2 got{dpp<kDppQuadSwap1, 0xF>(give.x), dpp<kDppQuadSwap1, 0xF>(give.y)};
  return odd ? u32x4{got.x, got.y, h.x, h.y} : u32x4{l.x, l.y, got.x, got.y};
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

// One workgroup per row of `vecs` 16-byte vectors (an even number).  In turn i
// lane l of L loads vectors 2*L*i + l and 2*L*i + L + l, so that every load
// instruction reads whole cache lines, and stores the 16 bytes of payload of
// vectors 2*L*i + l, + 1 (even lanes) or 2*L*i + L + l - 1, + 1 (odd lanes).
// U > 0: at most U turns, held in registers; U == 0: any number, read twice.
// `store(at, bytes)` writes 16 bytes of the payload from byte 8*at,
// `scale_out(scale)` runs on lane 0.
template <int U, bool kNonTemporal, class Store, class ScaleOut>
__device__ __forceinline__ void quantize_row(const u32x4* __restrict__ src, int vecs, uint32_t* s_part,
                                             Store store, ScaleOut scale_out) {
  const int tid = threadIdx.x, lanes = blockDim.x;
  const u32x4 zero{0u, 0u, 0u, 0u};
  uint32_t amax = 0;
  float scale, inv;
  auto load = [&](int v) { return v < vecs ? load_vec<kNonTemporal>(src + v) : zero; };
  auto first_load = [&](int v) { return v < vecs ? load_vec<false>(src + v) : zero; };  // kept for the second
  auto write = [&](int base, const u32x4& lo, const u32x4& hi) {
    const u32x4 b = pair_i8(lo, hi, inv);
    const int at = tid % 2 == 0 ? base + tid : base + lanes + tid - 1;
    if (at < vecs) store(at, b);
  };
  if constexpr (U > 0) {
    u32x4 v[U][2];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      v[i][0] = load(2 * lanes * i + tid);
      v[i][1] = load(2 * lanes * i + lanes + tid);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) amax = max(amax, max(vec_amax(v[i][0]), vec_amax(v[i][1])));
    row_scale(block_max(amax, s_part), scale, inv);
#pragma unroll
    for (int i = 0; i < U; ++i) write(2 * lanes * i, v[i][0], v[i][1]);
  } else {
    for (int b = 0; b < vecs; b += 2 * lanes)
      amax = max(amax, max(vec_amax(first_load(b + tid)), vec_amax(first_load(b + lanes + tid))));
    row_scale(block_max(amax, s_part), scale, inv);
    for (int b = 0; b < vecs; b += 2 * lanes) write(b, load(b + tid), load(b + lanes + tid));
  }
  if (tid == 0) scale_out(scale);
}

}  // namespace

// kStream: loads and stores past the caches, for rows that do not fit them.
template <int U, bool kStream>
__global__ __launch_bounds__(kMaxI8Threads) void k_quantize_i8(
    const u32x4* __restrict__ x, int64_t n_rows, int vecs, const uint32_t* __restrict__ row_count,
    uint8_t* __restrict__ q, float* __restrict__ scales) {
  __shared__ uint32_t s_part[kMaxI8Threads / kWave];
  const int64_t rows = row_count == nullptr ? n_rows : min(n_rows, int64_t(*row_count));
  for (int64_t t = blockIdx.x; t < rows; t += gridDim.x) {
    uint8_t* dst = q + t * vecs * 8;
    quantize_row<U, kStream>(
        x + t * vecs, vecs, s_part,
        [&](int at, const u32x4& b) { store_vec<kStream>(reinterpret_cast<u32x4*>(dst + 8 * at), b); },
        [&](float s) { scales[t] = s; });
    __syncthreads();  // s_part is rewritten for the next row
  }
}

// K > 0: top_k == K, positions in scalar registers; K == 0: any top_k,
// positions compacted into LDS by wave 0.
template <int K, int U>
__global__ __launch_bounds__(kMaxI8Threads) void k_dispatch_i8(
    const u32x4* __restrict__ x, int64_t n_rows, int vecs, int top_k,
    const uint32_t* __restrict__ restore, uint8_t* __restrict__ q, float* __restrict__ scales,
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
      quantize_row<U, false>(
          x + t * vecs, vecs, s_part,
          [&](int at, const u32x4& b) {
#pragma unroll
            for (int j = 0; j < nj; ++j) {
              const uint32_t p = K > 0 ? pos[j] : s_pos[j];
              if (p != kSent)
                __builtin_nontemporal_store(b, reinterpret_cast<u32x4*>(q + (int64_t(p) * vecs + at) * 8));
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

// Turns of a row, and lanes: the fewest turns with at most kMaxI8Threads
// lanes, then the fewest whole waves that hold them.
int i8_turns(int vecs) { return (vecs + 2 * kMaxI8Threads - 1) / (2 * kMaxI8Threads); }
int i8_threads(int vecs, int turns) {
  if (turns > 4) return kMaxI8Threads;  // any number of them, in a loop
  const int held = turns == 3 ? 4 : turns;
  return ((vecs + 2 * held - 1) / (2 * held) + kWave - 1) / kWave * kWave;
}

template <int K>
struct LaunchDispatchI8 {
  static hipError_t run(const u32x4* x, int64_t n_rows, int vecs, int top_k, const uint32_t* restore,
                        uint8_t* q, float* scales, uint32_t limit, hipStream_t s) {
    const int per = i8_turns(vecs), threads = i8_threads(vecs, per);
    const dim3 grid(row_grid(n_rows)), block(threads);
#define MOE_GO(U)                                                                                     \
  hipLaunchKernelGGL((k_dispatch_i8<K, U>), grid, block, 0, s, x, n_rows, vecs, top_k, restore, q, \
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
  return by_top_k<LaunchDispatchI8>(top_k, reinterpret_cast<const u32x4*>(x), n_rows, hidden / 8, top_k,
                                    restore, reinterpret_cast<uint8_t*>(q), scales,
                                    position_limit(out_rows), s);
}

hipError_t launch_quantize_i8(const uint16_t* x, int64_t n_rows, int hidden,
                              const uint32_t* row_count, int8_t* q, float* scales, hipStream_t s) {
  if (n_rows == 0) return hipSuccess;
  const int vecs = hidden / 8;
  const int per = i8_turns(vecs), threads = i8_threads(vecs, per);
  const dim3 grid(row_grid(n_rows)), block(threads);
  const u32x4* xv = reinterpret_cast<const u32x4*>(x);
  uint8_t* qv = reinterpret_cast<uint8_t*>(q);
  const bool stream = double(n_rows) * hidden * 3 >= double(kI8StreamMinBytes);
#define MOE_GO(U)                                                                                              \
  do {                                                                                                       \
    if (stream)                                                                                              \
      hipLaunchKernelGGL((k_quantize_i8<U, true>), grid, block, 0, s, xv, n_rows, vecs, row_count, qv, scales); \
    else                                                                                                     \
      hipLaunchKernelGGL((k_quantize_i8<U, false>), grid, block, 0, s, xv, n_rows, vecs, row_count, qv, scales); \
  } while (0)
  if (per == 1) MOE_GO(1);
  else if (per == 2) MOE_GO(2);
  else if (per <= 4) MOE_GO(4);
  else MOE_GO(0);
#undef MOE_GO
  return hipGetLastError();
}

}  // namespace moe
