// The experts' products in 8-bit integers over the expert-contiguous buffer.
//
//   c[p, n] = sum_k a[p, k] * w[e(p), n, k]  (int32, exact in any order)
//   out = bf16(fl(fl(fl(c) * sa[p]) * sw[e, n])), or silu(gate) * up of two of them
//
// The rows of an expert are known on the device only.  Two kernels share the
// groups by their size, both reading the starts themselves:
//   k_matmul_few   groups of at most kFewRows rows, bound by reading the
//                  weights once: they stream into registers (stream.h).
//   k_matmul_tile  larger groups, in tiles of 256 rows by 256 weight rows,
//                  bound by the matrix units: both operands go through LDS.
#include "experts.h"
#include "rows.h"
#include "stream.h"

namespace moe {

namespace {

constexpr int kFewRows = 64;
constexpr int kFewWaves = 4, kFewThreads = kFewWaves * kWave;
constexpr int kTile = 256, kStepBytes = 128;  // tile edge, and values of k per step
constexpr int kTileThreads = 512;
constexpr int kMaxActive = 1024;

// Rows [lo, hi) of active expert j, inside the buffer whatever the starts hold.
__device__ __forceinline__ void group_rows(const uint32_t* starts, int j, uint32_t a_rows, uint32_t& lo,
                                           uint32_t& hi) {
  lo = min(starts[j], a_rows);
  hi = max(min(starts[j + 1], a_rows), lo);
}

__device__ __forceinline__ float scaled(int32_t c, float sa, float sw) { return float(c) * sa * sw; }

}  // namespace

// ---- few rows ------------------------------------------------------------------

// 32 weight rows (16 gate and 16 up rows, or 32 output channels) times n <= 16*NG rows from lo.
template <int NG, bool kSwiglu>
__device__ __forceinline__ void matmul_few_tile(const ExpertMatmul& p, uint32_t lo, int n, int e, int c0,
                                                i32x4* s_part) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int wide = kSwiglu ? 2 * p.n_out : p.n_out;
  const uint8_t* w = reinterpret_cast<const uint8_t*>(p.w) + int64_t(e) * wide * p.depth;
  const uint8_t* a = reinterpret_cast<const uint8_t*>(p.a) + int64_t(lo) * p.depth;
  const int second = kSwiglu ? p.n_out + c0 : min(c0 + 16, p.n_out - 16);  // first row of the second 16
  const uint8_t* wp[2] = {w + int64_t(c0 + lane % 16) * p.depth, w + int64_t(second + lane % 16) * p.depth};
  const uint8_t* ap[NG];
  i32x4 acc[2][NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    ap[g] = a + int64_t(min(g * 16 + lane % 16, n - 1)) * p.depth;
    acc[0][g] = acc[1][g] = i32x4{0, 0, 0, 0};
  }
  int begin, end;
  step_range(p.depth, wave, kFewWaves, begin, end);
  stream_products<CoreI8, 2, NG, (NG == 1 ? 8 : NG == 2 ? 4 : 2)>(wp, ap, begin, end, p.depth, acc);
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int g = 0; g < NG; ++g) s_part[((wave * 2 + r) * NG + g) * kWave + lane] = acc[r][g];
  __syncthreads();
  for (int g = wave; g < NG; g += kFewWaves) {
    const int row = g * 16 + lane % 16;
    i32x4 sum[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      sum[r] = s_part[(r * NG + g) * kWave + lane];
#pragma unroll
      for (int v = 1; v < kFewWaves; ++v) sum[r] += s_part[((v * 2 + r) * NG + g) * kWave + lane];
    }
    if (row >= n) continue;
    const float sa = p.a_scales[lo + row];
    const float* sw = p.w_scales + int64_t(e) * wide;
    uint16_t* o = p.out + int64_t(lo + row) * p.n_out;
    float v[2][4];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[r][i] = scaled(sum[r][i], sa, sw[(r == 0 ? c0 : second) + (lane / 16) * 4 + i]);
    if constexpr (kSwiglu) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[0][i] = silu_times(v[0][i], v[1][i]);
    }
#pragma unroll
    for (int r = 0; r < (kSwiglu ? 1 : 2); ++r) {
      const int c = c0 + r * 16;
      if (c < p.n_out)
        *reinterpret_cast<u32x2*>(o + c + (lane / 16) * 4) =
            u32x2{bf16_pair(v[r][0], v[r][1]), bf16_pair(v[r][2], v[r][3])};
    }
  }
}

template <bool kSwiglu>
__global__ __launch_bounds__(kFewThreads) void k_matmul_few(ExpertMatmul p) {
  __shared__ i32x4 s_part[kFewWaves * 2 * (kFewRows / 16) * kWave];
  uint32_t lo, hi;
  group_rows(p.starts, blockIdx.y, p.a_rows, lo, hi);
  const uint32_t n = hi - lo;
  if (n == 0 || n > uint32_t(kFewRows)) return;
  const int e = p.expert_ids[blockIdx.y];
  if (e < 0 || e >= p.n_experts) return;
  const int c0 = blockIdx.x * (kSwiglu ? 16 : 32);
  if (n <= 16) matmul_few_tile<1, kSwiglu>(p, lo, n, e, c0, s_part);
  else if (n <= 32) matmul_few_tile<2, kSwiglu>(p, lo, n, e, c0, s_part);
  else matmul_few_tile<4, kSwiglu>(p, lo, n, e, c0, s_part);
}

// ---- tiles ----------------------------------------------------------------------

namespace {

typedef __attribute__((address_space(3))) uint8_t lds_byte;

// 64 lanes x 16 bytes from `base + off` (per lane) to 1 KB of LDS at `dst`.
__device__ __forceinline__ void load_to_lds(const uint8_t* base, uint32_t off, uint8_t* dst) {
  __builtin_amdgcn_global_load_lds(
      reinterpret_cast<const __attribute__((address_space(1))) uint32_t*>(reinterpret_cast<uintptr_t>(base + off)),
      (__attribute__((address_space(3))) uint32_t*)(dst), 16, 0, 0);
}

}  // namespace

// One workgroup per CU takes tiles in turn.  Eight waves, 2 by 4: each forms
// 128 rows by 64 weight rows with the 32x32x32 instruction.  A step is 128
// values of k of 256 rows of both operands, 64 KB, in two buffers.  A row's
// 128 bytes lie in LDS as eight 16-byte pieces, piece c at c ^ (row % 8), so
// that the lanes of a read (consecutive rows, one piece) touch all banks.
// With SwiGLU each 64 weight rows are 32 gate rows and the 32 up rows of the
// same channels, so one lane holds both.
template <bool kSwiglu>
__global__ __launch_bounds__(kTileThreads, 2) void k_matmul_tile(ExpertMatmul p) {
  __shared__ __align__(16) uint8_t s_a[2][kTile * kStepBytes];
  __shared__ __align__(16) uint8_t s_w[2][kTile * kStepBytes];
  __shared__ uint32_t s_first[kMaxActive + 1];  // first tile of each active expert
  __shared__ uint32_t s_scan[kTileThreads / kWave];
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  constexpr int kChannels = kSwiglu ? kTile / 2 : kTile;
  const uint32_t col_tiles = (p.n_out + kChannels - 1) / kChannels;

  uint32_t tiles[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = 2 * tid + i;
    uint32_t lo = 0, hi = 0;
    if (j < p.n_experts) group_rows(p.starts, j, p.a_rows, lo, hi);
    tiles[i] = hi - lo > uint32_t(kFewRows) ? ((hi - lo + kTile - 1) / kTile) * col_tiles : 0u;
  }
  const uint32_t sum = wave_inclusive_sum(tiles[0] + tiles[1]);
  if (lane == kWave - 1) s_scan[wave] = sum;
  __syncthreads();
  uint32_t before = sum - tiles[0] - tiles[1], total = 0;
  for (int i = 0; i < kTileThreads / kWave; ++i) {
    if (i < wave) before += s_scan[i];
    total += s_scan[i];
  }
  s_first[2 * tid] = before;
  s_first[2 * tid + 1] = before + tiles[0];
  if (tid == kTileThreads - 1) s_first[kMaxActive] = total;
  __syncthreads();

  // Workgroups of one XCD (blockIdx % 8) take neighbouring tiles.
  const uint32_t grid = gridDim.x, per = grid / 8, rest = grid % 8, xcd = blockIdx.x % 8;
  const uint32_t place = xcd * per + min(xcd, rest) + blockIdx.x / 8;
  const int wr = wave / 4, wc = wave % 4;
  for (uint32_t tile = place; tile < total; tile += grid) {
    int j = 0;  // the last active expert with s_first[j] <= tile
    for (int step = kMaxActive / 2; step > 0; step /= 2)
      if (s_first[j + step] <= tile) j += step;
    uint32_t lo, hi;
    group_rows(p.starts, j, p.a_rows, lo, hi);
    if (hi == lo) continue;
    const int e = p.expert_ids[j];
    const uint32_t row_tiles = (hi - lo + kTile - 1) / kTile;
    const uint32_t in = tile - s_first[j];
    const uint32_t row0 = lo + (in % row_tiles) * kTile;
    const int c0 = int(in / row_tiles) * kChannels;
    if (e < 0 || e >= p.n_experts || row0 >= hi || c0 >= p.n_out) continue;
    const int n_rows = int(min(hi - row0, uint32_t(kTile)));
    const int wide = kSwiglu ? 2 * p.n_out : p.n_out;

    // This wave fills LDS rows [32*wave, +32) of both operands, eight rows an
    // instruction; rows past the tile's end repeat its last one.
    const int piece = (lane % 8) ^ (lane / 8);
    const uint8_t* a_base = reinterpret_cast<const uint8_t*>(p.a) + int64_t(row0) * p.depth;
    int w_first = c0 + 32 * wave, w_last = p.n_out - 1, w_shift = 0;
    if constexpr (kSwiglu) {
      w_first = c0 + 32 * (wave / 2);
      w_shift = wave % 2 == 0 ? 0 : p.n_out;
    }
    const int w_origin = min(w_first, w_last);
    const uint8_t* w_base =
        reinterpret_cast<const uint8_t*>(p.w) + (int64_t(e) * wide + w_shift + w_origin) * p.depth;
    uint32_t a_off[4], w_off[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 8 + lane / 8;
      a_off[i] = uint32_t(min(32 * wave + r, n_rows - 1)) * uint32_t(p.depth);
      w_off[i] = uint32_t(min(w_first + r, w_last) - w_origin) * uint32_t(p.depth);
    }
    const int steps = (p.depth + kStepBytes - 1) / kStepBytes;
    auto fetch = [&](int s, int buf) {
      const int k = s * kStepBytes;
      const uint32_t at = uint32_t(k + (k + piece * 16 < p.depth ? piece * 16 : 0));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        load_to_lds(a_base, a_off[i] + at, &s_a[buf][(32 * wave + 8 * i) * kStepBytes]);
        load_to_lds(w_base, w_off[i] + at, &s_w[buf][(32 * wave + 8 * i) * kStepBytes]);
      }
    };
    i32x16 acc[2][4];
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[f][g][i] = 0;
    auto compute = [&](int buf, int k, bool last) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const int c = kk * 2 + lane / 32;
        const int at = (c ^ (lane % 8)) * 16;
        i32x4 w[2], a[4];
#pragma unroll
        for (int f = 0; f < 2; ++f)
          w[f] = *reinterpret_cast<const i32x4*>(&s_w[buf][(64 * wc + 32 * f + lane % 32) * kStepBytes + at]);
#pragma unroll
        for (int g = 0; g < 4; ++g)
          a[g] = *reinterpret_cast<const i32x4*>(&s_a[buf][(128 * wr + 32 * g + lane % 32) * kStepBytes + at]);
        if (last && k + c * 16 >= p.depth) {  // pieces past the row's end add nothing
#pragma unroll
          for (int f = 0; f < 2; ++f) w[f] = i32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            acc[f][g] = __builtin_amdgcn_mfma_i32_32x32x32_i8(w[f], a[g], acc[f][g], 0, 0, 0);
      }
    };
    fetch(0, 0);
    for (int s = 0; s < steps; ++s) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      if (s + 1 < steps) fetch(s + 1, (s + 1) & 1);
      compute(s & 1, s * kStepBytes, s + 1 == steps);
    }
    __syncthreads();  // the buffers are refilled for the next tile

    const float* sw = p.w_scales + int64_t(e) * wide;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int r = 128 * wr + 32 * g + lane % 32;
      if (r >= n_rows) continue;
      const float sa = p.a_scales[row0 + r];
      uint16_t* o = p.out + int64_t(row0 + r) * p.n_out;
#pragma unroll
      for (int f = 0; f < (kSwiglu ? 1 : 2); ++f) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = c0 + (kSwiglu ? 32 * wc : 64 * wc + 32 * f) + 8 * q + 4 * (lane / 32);
          if (c >= p.n_out) continue;
          float v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] = scaled(acc[f][g][4 * q + i], sa, sw[c + i]);
            if constexpr (kSwiglu) v[i] = silu_times(v[i], scaled(acc[1][g][4 * q + i], sa, sw[p.n_out + c + i]));
          }
          *reinterpret_cast<u32x2*>(o + c) = u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
        }
      }
    }
  }
}

namespace {

template <bool kSwiglu>
hipError_t go(const ExpertMatmul& p, hipStream_t s) {
  const uint32_t groups = p.a_rows < uint32_t(p.n_experts) ? p.a_rows : uint32_t(p.n_experts);
  const int per = kSwiglu ? 16 : 32;
  hipLaunchKernelGGL((k_matmul_few<kSwiglu>), dim3((p.n_out + per - 1) / per, groups), dim3(kFewThreads), 0, s, p);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess || p.a_rows <= uint32_t(kFewRows)) return e;
  hipLaunchKernelGGL((k_matmul_tile<kSwiglu>), dim3(256), dim3(kTileThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_matmul_i8(const ExpertMatmul& p, bool swiglu, hipStream_t s) {
  if (p.a_rows == 0) return hipSuccess;
  return swiglu ? go<true>(p, s) : go<false>(p, s);
}

}  // namespace moe
