// The experts' products over the expert-contiguous buffer, for one type of
// operands, a core C:
//   kSize            bytes of a value
//   kFloat           sums in fp32, in an order that the launch fixes; int32 sums are exact in any
//   kChannels        a scale for each row and each output channel, on the sum
//   kBlocks          a scale for each 128 values of a row and each 128 x 128 block of weights
//   Acc, mac         the sums of 32 x 32 products and 128 bits (256 with kBlocks) of k a lane added to them
//   value            a sum's value
//   Few, FewAcc      the core of stream.h, and its sums
//   kFewPerSimd      waves a SIMD of k_matmul_few
//   kStripsMin       the smallest grid of strips
//   tiles            launches the kernel for large groups
//
// The rows of an expert are known on the device only.  Kernels share the
// groups by their size, each reading the starts itself:
//   k_matmul_strip  groups of at most kFewRows rows, bound by reading the
//                   weights once, 256 weight rows a workgroup, through LDS
//   k_matmul_few    the same groups where that makes too few workgroups: 32
//                   weight rows a workgroup, straight to registers (stream.h)
//   k_matmul_tile   larger groups, in tiles of 256 rows by 256 weight rows,
//                   bound by the matrix units and their clock
#pragma once

#include <type_traits>

#include "experts.h"
#include "lds_fill.h"
#include "rows.h"
#include "stream.h"

namespace moe {

namespace {

// Largest group of the first two.  256 experts with 33 and with 64 rows each, 2048
// -> 7168, as strips and as tiles: 672, 729 and 797, 853 us in int8, 1224, 1386
// and 1518, 1559 in bf16, 649, 691 and 701, 753 in e4m3.
constexpr int kFewRows = 64;
constexpr int kFewWaves = 4, kFewThreads = kFewWaves * kWave;
constexpr int kTile = 256, kStepBytes = 128;  // tile edge, and bytes of a row per step
constexpr int kTileThreads = 256, kStripThreads = 256;
constexpr int kStripFrags = 2;  // of 32 weight rows, for each wave
// Grids of k_matmul_strip have at least C::kStripsMin workgroups; smaller ones
// leave CUs idle and go to k_matmul_few.  Strips against k_matmul_few in us, int8,
// bf16 and e4m3:
//   64 workgroups (8 experts, 20 rows each, 7168 -> 2048)    67/27  138/52   69/35
//   128 (8, 20, 4096 -> 4096)                                39/32   70/60   39/40
//   160 (10, 20, 4096 -> 4096)                               40/42   72/73   40/55
//   192 (12, 20, 4096 -> 4096)                               41/52   75/87   41/63
//   192 (24, 4, 2048 -> 2048)                                22/18   37/38   21/20
//   256 (16, 20, 4096 -> 4096)                               45/66   83/113  45/83
//   896 (32, 16, 2048 -> 7168)                               81/97  149/174  79/121
// Between 160 and 256 int8 gains with many rows and loses with few.
// Buffers of up to kAloneRows rows over weights of up to kAloneWeights values an
// expert take one launch: all of their groups go to the first kernel, 64 rows at a
// time.  24 experts, 4 rows each, 1040 -> 528: 6.7 against 8.9 us in bf16, 5.1 and
// 7.3 in e4m3, 4.2 and 7.4 in int8; one expert with 100 rows, 4096 -> 1024: 41 and
// 59, 31 and 33, 23 and 34.  More rows would read the weights too often where one
// expert has them all (250 rows, 4096 -> 4096: 89 and 81 us in bf16, 74 and 50 in
// e4m3, 50 and 47 in int8), and so would larger weights (2 x 120 rows, 4096 ->
// 14336: 170 and 99, 120 and 41, 86 and 42).
constexpr uint32_t kAloneRows = 128;
constexpr int64_t kAloneWeights = int64_t(1) << 22;
constexpr int kMaxActive = 1024;
// Rows of tiles that are taken column by column together: 491366 rows on 253
// experts, 2048 -> 7168, with 8, 6, 4 and with all of an expert's 6.75, 6.74, 6.83
// and 7.07 ms in e4m3, 7.31, 7.32, 7.47 and 7.73 in int8, 12.4, 12.4, 12.6 and 13.0
// in bf16 (1750 rows an expert hardly depend on it).
constexpr uint32_t kRowGroup = 8;

// Rows [lo, hi) of active expert j, inside the buffer whatever the starts hold.
__device__ __forceinline__ void group_rows(const uint32_t* starts, int j, uint32_t a_rows, uint32_t& lo,
                                           uint32_t& hi) {
  lo = min(starts[j], a_rows);
  hi = max(min(starts[j + 1], a_rows), lo);
}

__device__ __forceinline__ float scaled(int32_t c, float sa, float sw) { return float(c) * sa * sw; }

// The sums of a block of k, times its scales, onto those of the others.
template <class Acc>
__device__ __forceinline__ void add_scaled(Acc& to, const Acc& part, float scale) {
#pragma unroll
  for (int i = 0; i < 16; ++i) to[i] = __builtin_fmaf(part[i], scale, to[i]);
}

}  // namespace

// ---- few rows ------------------------------------------------------------------

// 32 weight rows (16 gate and 16 up rows, or 32 output channels) times n <= 16*NG rows from lo.
template <class C, int NG, bool kSwiglu>
__device__ __forceinline__ void matmul_few_tile(const ExpertMatmul& p, uint32_t lo, int n, int e, int c0,
                                                typename C::FewAcc* s_part) {
  int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  // Numbers that the compiler knows nothing of, or it forms addresses of all three sizes ahead of the loop over the
  // group's rows and keeps them: 52 bytes a lane of scratch in int8.
  asm volatile("" : "+v"(lane), "+v"(wave));
  const int wide = kSwiglu ? 2 * p.n_out : p.n_out;
  const int64_t w_row = int64_t(p.depth) * C::kSize;  // bytes
  const uint8_t* w = static_cast<const uint8_t*>(p.w) + int64_t(e) * wide * w_row;
  const uint8_t* a = static_cast<const uint8_t*>(p.a) + int64_t(lo) * w_row;
  const int second = kSwiglu ? p.n_out + c0 : min(c0 + 16, p.n_out - 16);  // first row of the second 16
  const uint8_t* wp[2] = {w + (c0 + lane % 16) * w_row, w + (second + lane % 16) * w_row};
  const uint8_t* ap[NG];
  typename C::FewAcc acc[2][NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    ap[g] = a + min(g * 16 + lane % 16, n - 1) * w_row;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[0][g][i] = acc[1][g][i] = 0;
  }
  if constexpr (C::kBlocks) {
    const int blocks = (p.depth + kBlock - 1) / kBlock, half = (p.n_out + kBlock - 1) / kBlock;
    const float* sw = p.w_scales + int64_t(e) * (kSwiglu ? 2 : 1) * half * blocks;
    const float* swp[2] = {sw + int64_t(c0 / kBlock) * blocks,
                           sw + int64_t(kSwiglu ? half + c0 / kBlock : second / kBlock) * blocks};
    const float* sap[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) sap[g] = p.a_scales + (lo + min(g * 16 + lane % 16, n - 1)) * int64_t(blocks);
    stream_blocks<2, NG, 4 / NG>(wp, ap, swp, sap, blocks * wave / kFewWaves, blocks * (wave + 1) / kFewWaves, p.depth,
                                 acc);
  } else {
    int begin, end;
    step_range(p.depth, wave, kFewWaves, begin, end);
    stream_products<typename C::Few, 2, NG, C::kSize == 1 ? (NG == 4 ? 2 : 4) : 4 / NG>(wp, ap, begin, end, p.depth, acc);
  }
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int g = 0; g < NG; ++g) s_part[((wave * 2 + r) * NG + g) * kWave + lane] = acc[r][g];
  __syncthreads();
  for (int g = wave; g < NG; g += kFewWaves) {
    const int row = g * 16 + lane % 16;
    typename C::FewAcc sum[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      sum[r] = s_part[(r * NG + g) * kWave + lane];
#pragma unroll
      for (int v = 1; v < kFewWaves; ++v) {
        const typename C::FewAcc part = s_part[((v * 2 + r) * NG + g) * kWave + lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[r][i] += part[i];
      }
    }
    if (row >= n) continue;
    uint16_t* o = p.out + int64_t(lo + row) * p.n_out;
    float v[2][4];
    if constexpr (C::kChannels) {
      const float sa = p.a_scales[lo + row];
      const float* sw = p.w_scales + int64_t(e) * wide;
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[r][i] = scaled(sum[r][i], sa, sw[(r == 0 ? c0 : second) + (lane / 16) * 4 + i]);
    } else {
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[r][i] = sum[r][i];
    }
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

// C::kFewPerSimd waves a SIMD.  In int8 four hold all of a grid of 1024 workgroups at once (8 experts, 16 rows each,
// 2048 -> 2 x 2048: 16.5 against 18.2 us with three).  In bf16 and e4m3 the registers of four do not hold what is
// requested together, 2 rows of 4 steps, and with four and three 8 experts, 14 rows each, 4096 -> 4096, take 55.6 and
// 54.2 us in bf16, 35.7 and 32.4 in e4m3; 12 experts, 2 rows each, 7168 -> 2048, 62 and 60, 42 and 37.
template <class C, bool kSwiglu>
__global__ __launch_bounds__(kFewThreads, C::kFewPerSimd) void k_matmul_few(ExpertMatmul p, uint32_t most) {
  __shared__ typename C::FewAcc s_part[kFewWaves * 2 * (kFewRows / 16) * kWave];
  uint32_t lo, hi;
  group_rows(p.starts, blockIdx.y, p.a_rows, lo, hi);
  if (lo == hi || hi - lo > most) return;
  const int e = p.expert_ids[blockIdx.y];
  if (e < 0 || e >= p.n_experts) return;
  const int c0 = blockIdx.x * (kSwiglu ? 16 : 32);
  for (;; lo += kFewRows) {
    const int n = min(hi - lo, uint32_t(kFewRows));
    if (n <= 16) matmul_few_tile<C, 1, kSwiglu>(p, lo, n, e, c0, s_part);
    else if (n <= 32) matmul_few_tile<C, 2, kSwiglu>(p, lo, n, e, c0, s_part);
    else matmul_few_tile<C, 4, kSwiglu>(p, lo, n, e, c0, s_part);
    if (hi - lo <= uint32_t(kFewRows)) return;  // before lo, which may pass 2^32 with the buffer's last rows
    __syncthreads();                            // s_part is rewritten for the next rows
  }
}

// ---- strips ---------------------------------------------------------------------

// One workgroup: 128*F weight rows (with SwiGLU half of them gate rows, half
// the up rows of the same channels) times the n <= 32*G rows of one group.
// Bound by reading the weights: they go to LDS in whole cache lines,
// non-temporal, in two buffers of a step (128 bytes of a row).  Layout of a
// buffer, 16-byte pieces and their order as in k_matmul_tile; each wave takes
// 32*F weight rows, with SwiGLU first its gate and then its up rows.
template <class C, int G, bool kSwiglu>
__device__ __forceinline__ void strip(const ExpertMatmul& p, uint32_t lo, int n, int e, int c0, uint8_t* a0,
                                      uint8_t* a1, uint8_t* w0, uint8_t* w1) {
  constexpr int F = kStripFrags;
  const int lane = threadIdx.x % kWave, wave = uniform(int(threadIdx.x / kWave));
  const int wide = kSwiglu ? 2 * p.n_out : p.n_out;
  const uint32_t row = uint32_t(p.depth) * C::kSize;  // bytes
  const int steps = (row + kStepBytes - 1) / kStepBytes;
  const bool ragged = row % kStepBytes != 0;
  const int piece[2] = {(lane % 8) ^ (lane / 16), (lane % 8) ^ (4 + lane / 16)};
  const uint32_t lane_off[2] = {uint32_t(lane / 8) * row + piece[0] * 16,
                                uint32_t(lane / 8) * row + piece[1] * 16};
  // This wave's weight rows, LDS rows [32*F*wave, +32*F): channels c, c+1, ..
  constexpr int kWaveChannels = kSwiglu ? 16 * F : 32 * F;
  const int c = c0 + kWaveChannels * wave;
  // The activations' buffer ends with the group: rows behind it are zeros in LDS and not read.
  const uint64_t a_bytes = uint64_t(n) * row, w_rows = uint64_t(p.n_experts) * wide;
  const uint64_t w_row = uint64_t(e) * wide + min(c, p.n_out);
  const uint8_t* w = static_cast<const uint8_t*>(p.w);
  const __amdgpu_buffer_rsrc_t a_from = buffer_of(static_cast<const uint8_t*>(p.a) + uint64_t(lo) * row, a_bytes);
  const __amdgpu_buffer_rsrc_t w_from = buffer_of(w + w_row * row, (w_rows - w_row) * row);
  const uint64_t up_row = kSwiglu ? w_row + p.n_out : w_row;
  const __amdgpu_buffer_rsrc_t up_from = buffer_of(w + up_row * row, (w_rows - up_row) * row);
  // Workgroups begin at different steps: rows whose length is a power of two
  // would have all of them at the same few memory channels at any time (64
  // experts, 4 rows each, 4096 x 4096: 235 us against 171 us; no difference at
  // 2048 and 7168).  In int8 the sums are exact in any order; in fp32 a
  // workgroup's place fixes theirs.
  const int turn = ragged ? 0 : int((blockIdx.x * 5 + blockIdx.y * 3) % uint32_t(steps));
  const int blocks = C::kBlocks ? steps : 0;  // a step of e4m3 is a block of k
  const int half = (p.n_out + kBlock - 1) / kBlock, w_block = min(c, p.n_out - 1) / kBlock;
  const float* sw0 = p.w_scales + (int64_t(e) * (kSwiglu ? 2 : 1) * half + w_block) * blocks;
  const float* sw1 = sw0 + (kSwiglu ? int64_t(half) * blocks : 0);
  const __amdgpu_buffer_rsrc_t sa_from =
      buffer_of(reinterpret_cast<const uint8_t*>(p.a_scales + uint64_t(lo) * blocks), uint64_t(n) * blocks * 4);
  struct BlockScales {
    float a[G], w[2];
  };
  auto fetch = [&](int nth, uint8_t* to_a, uint8_t* to_w, BlockScales& to_s) __attribute__((always_inline)) {
    const int s = nth + turn < steps ? nth + turn : nth + turn - steps;
    if constexpr (C::kBlocks) {
#pragma unroll
      for (int g = 0; g < G; ++g)
        to_s.a[g] = __uint_as_float(
            __builtin_amdgcn_raw_buffer_load_b32(sa_from, uint32_t(32 * g + lane % 32) * blocks * 4, s * 4, 0));
      to_s.w[0] = sw0[s];
      to_s.w[1] = sw1[s];
    }
#pragma unroll
    for (int i = 0; i < 4 * F; ++i) {
      const int r = kSwiglu ? 8 * (i % (2 * F)) : 8 * i;
      if (c + r < p.n_out)
        load_to_lds<true>(kSwiglu && i >= 2 * F ? up_from : w_from, lane_off[i % 2],
                          uint32_t(s) * kStepBytes + uint32_t(r) * row, to_w + (32 * F * wave + 8 * i) * kStepBytes);
    }
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int r = 8 * (wave + 4 * i);
      if (r < n)
        load_to_lds(a_from, lane_off[wave % 2], uint32_t(s) * kStepBytes + uint32_t(r) * row, to_a + r * kStepBytes);
    }
  };
  static_assert(F == 2);  // with SwiGLU the first is gate rows and the second up rows
  typename C::Acc acc[F][G];
#pragma unroll
  for (int f = 0; f < F; ++f)
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[f][g][i] = 0;
  BlockScales by0{}, by1{};
  auto step = [&](int s, uint8_t* a, uint8_t* w, const BlockScales& by, uint8_t* next_a, uint8_t* next_w,
                  BlockScales& next_by) __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(kWaitLoads);
    asm volatile("" ::: "memory");
    if (ragged && s == steps - 1) {  // pieces past the row's end add nothing
#pragma unroll
      for (int i = 0; i < 4 * F; ++i)
        if (s * kStepBytes + piece[i % 2] * 16 >= int(row))
          *reinterpret_cast<u32x4*>(w + (32 * F * wave + 8 * i) * kStepBytes + lane * 16) = u32x4{0u, 0u, 0u, 0u};
      if constexpr (C::kFloat) {  // what was read there instead may be a NaN
#pragma unroll
        for (int i = 0; i < G; ++i)
          if (s * kStepBytes + piece[wave % 2] * 16 >= int(row))
            *reinterpret_cast<u32x4*>(a + 8 * (wave + 4 * i) * kStepBytes + lane * 16) = u32x4{0u, 0u, 0u, 0u};
      }
    }
    __builtin_amdgcn_s_waitcnt(kWaitLdsScalar);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (s + 1 < steps) fetch(s + 1, next_a, next_w, next_by);
    auto piece_of = [&](const uint8_t* rows, int r, int kk) __attribute__((always_inline)) {
      return *reinterpret_cast<const u32x4*>(rows + (r + lane % 32) * kStepBytes +
                                             ((kk * 2 + lane / 32) ^ (lane / 2 % 8)) * 16);
    };
    if constexpr (C::kBlocks) {
      typename C::Acc part[F][G];
#pragma unroll
      for (int kk = 0; kk < 4; kk += 2) {
        u32x4 fw[F][2], fa[G][2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int f = 0; f < F; ++f) fw[f][j] = piece_of(w, 32 * F * wave + 32 * f, kk + j);
#pragma unroll
          for (int g = 0; g < G; ++g) fa[g][j] = piece_of(a, 32 * g, kk + j);
        }
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
          for (int g = 0; g < G; ++g)
            part[f][g] = C::mac(fw[f], fa[g], kk == 0 ? typename C::Acc{} : part[f][g]);
      }
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int g = 0; g < G; ++g) add_scaled(acc[f][g], part[f][g], by.a[g] * by.w[f]);
    } else {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        u32x4 fw[F], fa[G];
#pragma unroll
        for (int f = 0; f < F; ++f) fw[f] = piece_of(w, 32 * F * wave + 32 * f, kk);
#pragma unroll
        for (int g = 0; g < G; ++g) fa[g] = piece_of(a, 32 * g, kk);
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
          for (int g = 0; g < G; ++g) acc[f][g] = C::mac(fw[f], fa[g], acc[f][g]);
      }
    }
  };
  fetch(0, a0, w0, by0);
  for (int s = 0; s < steps; s += 2) {
    step(s, a0, w0, by0, a1, w1, by1);
    if (s + 1 < steps) step(s + 1, a1, w1, by1, a0, w0, by0);
  }
  // A lane's weight rows: 8*q + 4*(lane/32) + i of each 32.  With SwiGLU the
  // second half of the wave's rows are the up rows of the first half's channels.
  const float* sw = p.w_scales + (C::kChannels ? int64_t(e) * wide : 0);
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int r = 32 * g + lane % 32;
    float sa = 1.0f;
    if constexpr (C::kChannels) sa = p.a_scales[lo + min(r, n - 1)];
    uint16_t* o = p.out + int64_t(lo + r) * p.n_out;
#pragma unroll
    for (int k = 0; k < kWaveChannels / 8; ++k) {  // eight channels, four of them this lane's
      constexpr int kUp = kSwiglu ? 2 * F : 0;     // eights from a gate row to its up row
      const int ch = c + 8 * k + 4 * (lane / 32);
      if (r >= n || ch >= p.n_out) continue;
      f32x4 s0{}, s1{};
      if constexpr (C::kChannels) {
        s0 = *reinterpret_cast<const f32x4*>(sw + ch);
        if constexpr (kSwiglu) s1 = *reinterpret_cast<const f32x4*>(sw + p.n_out + ch);
      }
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = C::value(acc[k / 4][g][4 * (k % 4) + i], sa, s0[i]);
      if constexpr (kSwiglu) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = silu_times(v[i], C::value(acc[(k + kUp) / 4][g][4 * ((k + kUp) % 4) + i], sa, s1[i]));
      }
      *reinterpret_cast<u32x2*>(o + ch) = u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    }
  }
}

template <class C, bool kSwiglu>
__global__ __launch_bounds__(kStripThreads, 2) void k_matmul_strip(ExpertMatmul p, uint32_t most) {
  __shared__ __align__(16) uint8_t s_a0[kFewRows * kStepBytes], s_a1[kFewRows * kStepBytes];
  __shared__ __align__(16) uint8_t s_w0[128 * kStripFrags * kStepBytes], s_w1[128 * kStripFrags * kStepBytes];
  uint32_t lo, hi;
  group_rows(p.starts, blockIdx.y, p.a_rows, lo, hi);
  if (lo == hi || hi - lo > most) return;
  const int e = p.expert_ids[blockIdx.y];
  if (e < 0 || e >= p.n_experts) return;
  const int c0 = blockIdx.x * (kSwiglu ? 64 * kStripFrags : 128 * kStripFrags);
  for (;; lo += kFewRows) {
    const int n = min(hi - lo, uint32_t(kFewRows));
    if (n <= 32) strip<C, 1, kSwiglu>(p, lo, n, e, c0, s_a0, s_a1, s_w0, s_w1);
    else strip<C, 2, kSwiglu>(p, lo, n, e, c0, s_a0, s_a1, s_w0, s_w1);
    if (hi - lo <= uint32_t(kFewRows)) return;  // before lo, which may pass 2^32 with the buffer's last rows
    __syncthreads();                            // the buffers are filled again for the next rows
  }
}

// ---- tiles ----------------------------------------------------------------------

// A tile: its rows of the buffer, its first output channel, its expert.
struct TilePlace {
  uint32_t row0;
  int n_rows, c0, e;
};

struct Walk {
  uint32_t tile;  // next tile to look at
  int j;          // place of its expert, found going forward
};

// Of any number of rows up to 2^32 - 1: a sum with kTile - 1 would pass 32 bits.
__device__ __forceinline__ uint32_t row_tiles(uint32_t rows) { return rows / kTile + (rows % kTile != 0); }

// The tiles of all groups of more than kFewRows rows, in the order of the groups, filled by the whole workgroup.
template <int kThreads>
struct TileList {
  uint32_t first[kMaxActive + 1];  // first tile of each active expert
  uint32_t row[kMaxActive + 1];    // its first row
  int32_t expert[kMaxActive];      // its id
  uint32_t scan[kThreads / kWave];

  // Returns the number of tiles.
  __device__ __forceinline__ uint32_t fill(const ExpertMatmul& p, uint32_t col_tiles) {
    const int tid = threadIdx.x, lane = tid % kWave, wave = uniform(tid / kWave);
    constexpr int kOwn = kMaxActive / kThreads;
    uint32_t tiles[kOwn], sum = 0;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int j = kOwn * tid + i;
      uint32_t lo, hi;
      group_rows(p.starts, min(j, p.n_experts - 1), p.a_rows, lo, hi);
      if (j >= p.n_experts) lo = hi;
      row[j] = lo;
      expert[j] = j < p.n_experts ? p.expert_ids[j] : -1;
      if (j == kMaxActive - 1) row[kMaxActive] = hi;
      tiles[i] = hi - lo > uint32_t(kFewRows) ? row_tiles(hi - lo) * col_tiles : 0u;
      sum += tiles[i];
    }
    const uint32_t upto = wave_inclusive_sum(sum);
    if (lane == kWave - 1) scan[wave] = upto;
    __syncthreads();
    uint32_t before = upto - sum, total = 0;
    for (int i = 0; i < kThreads / kWave; ++i) {
      if (i < wave) before += scan[i];
      total += scan[i];
    }
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      first[kOwn * tid + i] = before;
      before += tiles[i];
    }
    if (tid == 0) first[kMaxActive] = total;
    total = min(uniform(total), 0xFFFFFF00u);  // the walk's next tile, 256 on, stays below 2^32
    __syncthreads();
    return total;
  }

  // The walk's next tile with work; false when there is none left.
  __device__ __forceinline__ bool next(const ExpertMatmul& p, uint32_t total, uint32_t grid, int channels, Walk& at,
                                       TilePlace& t) const {
    for (; at.tile < total; at.tile += grid) {
      while (at.j + 1 < kMaxActive && uniform(first[at.j + 1]) <= at.tile) ++at.j;
      const uint32_t lo = uniform(row[at.j]), hi = max(min(uniform(row[at.j + 1]), p.a_rows), lo);
      const uint32_t down = row_tiles(hi - lo);
      if (down == 0) continue;
      // Rows by kRowGroup, within them columns, within a column its rows: the tiles that an XCD's workgroups take at
      // once then share both operands in its L2.
      const uint32_t in = at.tile - uniform(first[at.j]), col_tiles = (uint32_t(p.n_out) + channels - 1) / channels;
      const uint32_t group = in / (kRowGroup * col_tiles), rest = in % (kRowGroup * col_tiles);
      const uint32_t rows = min(down - group * kRowGroup, kRowGroup);
      t.row0 = lo + (group * kRowGroup + rest % rows) * kTile;
      t.c0 = int(rest / rows) * channels;
      t.e = uniform(expert[at.j]);
      if (t.e < 0 || t.e >= p.n_experts || t.row0 >= hi || t.c0 >= p.n_out) continue;
      t.n_rows = int(min(hi - t.row0, uint32_t(kTile)));
      at.tile += grid;
      return true;
    }
    return false;
  }
};

// One workgroup per CU takes tiles in turn.  Four waves, 2 by 2: each forms
// 128 rows by 128 weight rows with the 32x32 instruction that takes 16 bytes a
// lane, which halves what has to be read from LDS against eight waves of 128 by 64.
//
// A step is 128 bytes (128 values of k in int8, 64 in bf16) of 256 rows of both
// operands, 64 KB, in two buffers that are filled straight from global memory.  A
// row's 128 bytes lie in LDS as eight 16-byte pieces, piece c at c ^ (row/2 % 8),
// so that sixteen lanes of a read (consecutive rows, one piece) touch all 64 banks
// once.
//
// A step has four parts of 32 bytes of a row.  The fragments of a part are read
// while the matrix units work on the part before it; the last part's are in
// registers before its products start, so there the buffer is free: one
// barrier, then it is filled for the step after next.  The stream of steps runs
// on across tiles, so a tile's first steps arrive during the epilogue of the
// tile before.
//
// With SwiGLU each 128 weight rows are 64 gate rows and the 64 up rows of the
// same channels, so one lane holds both.
template <class C, bool kSwiglu>
__global__ __launch_bounds__(kTileThreads, 1) void k_matmul_tile(ExpertMatmul p) {
  // Named apart, so that the compiler sees that filling one does not touch the other.
  __shared__ __align__(16) uint8_t s_a0[kTile * kStepBytes], s_a1[kTile * kStepBytes];
  __shared__ __align__(16) uint8_t s_w0[kTile * kStepBytes], s_w1[kTile * kStepBytes];
  __shared__ TileList<kTileThreads> s_tiles;
  const int tid = threadIdx.x, lane = tid % kWave, wave = uniform(tid / kWave);
  constexpr int kChannels = kSwiglu ? kTile / 2 : kTile;
  const uint32_t col_tiles = (p.n_out + kChannels - 1) / kChannels;

  const uint32_t total = s_tiles.fill(p, col_tiles);

  // Workgroups of one XCD (blockIdx % 8) take neighbouring tiles.
  const uint32_t grid = gridDim.x, per = grid / 8, rest = grid % 8, xcd = blockIdx.x % 8;
  const uint32_t first = xcd * per + min(xcd, rest) + blockIdx.x / 8;

  // The walk's next tile with work; false when there is none left.
  auto advance = [&](Walk& at, TilePlace& t) __attribute__((always_inline)) {
    return s_tiles.next(p, total, grid, kChannels, at, t);
  };

  const int wide = kSwiglu ? 2 * p.n_out : p.n_out;
  const uint32_t row = uint32_t(p.depth) * C::kSize;  // bytes
  const int steps = (row + kStepBytes - 1) / kStepBytes;
  const bool ragged = row % kStepBytes != 0;
  const uint64_t w_bytes = uint64_t(p.n_experts) * wide * row;
  // This wave fills LDS rows [64*wave, +64) of both operands, eight rows an
  // instruction.  Rows past the tile's end lie past its buffer and are not
  // read; weight rows past the expert's end are the next one's, or nothing: what
  // they give is not stored.
  // of an instruction of even and of odd number: the piece this lane fills
  const int piece[2] = {(lane % 8) ^ (lane / 16), (lane % 8) ^ (4 + lane / 16)};
  const uint32_t lane_off[2] = {uint32_t(lane / 8) * row + piece[0] * 16,
                                uint32_t(lane / 8) * row + piece[1] * 16};
  __amdgpu_buffer_rsrc_t a_from, w_from;
  auto aim = [&](const TilePlace& t) __attribute__((always_inline)) {
    const int rows = max(t.n_rows - 64 * wave, 0);
    const uint64_t a0 = (uint64_t(t.row0) + (rows > 0 ? 64 * wave : 0)) * row;
    const int first_w = t.c0 + (kSwiglu ? 64 * (wave / 2) + (wave % 2) * p.n_out : 64 * wave);
    const uint64_t w0 = (uint64_t(t.e) * wide + first_w) * row;
    a_from = buffer_of(static_cast<const uint8_t*>(p.a) + a0, uint64_t(rows) * row);
    w_from = buffer_of(static_cast<const uint8_t*>(p.w) + min(w0, w_bytes), w0 < w_bytes ? w_bytes - w0 : 0);
  };
  // `ahead` is the tile being fetched, up to two steps in front of `now`, the
  // tile being formed; each walks the tiles on its own.  Past the last tile
  // its steps are fetched again, for nothing.
  TilePlace now, ahead;
  Walk at_now{first, 0}, at_ahead{first, 0};
  if (!advance(at_now, now)) return;
  advance(at_ahead, ahead);
  aim(ahead);
  int fs = 0;  // the next step of `ahead` to fetch
  auto fetched = [&]() __attribute__((always_inline)) {
    if (++fs == steps) {
      fs = 0;
      if (advance(at_ahead, ahead)) aim(ahead);
      __builtin_amdgcn_s_waitcnt(kWaitLdsScalar);
    }
  };

  // Eight of this wave's 64 rows of both operands, for a step.
  // The XCDs begin at different steps, so that they are not all at the same
  // memory channels; within one they keep step, for what they share in its L2.
  const int turn = ragged ? 0 : int(xcd * uint32_t(steps) / 8);
  auto fetch = [&](int nth, uint8_t* to_a, uint8_t* to_w, int i) __attribute__((always_inline)) {
    const int s = nth + turn < steps ? nth + turn : nth + turn - steps;
    const uint32_t at = uint32_t(s) * kStepBytes + uint32_t(8 * i) * row;
    load_to_lds(a_from, lane_off[i % 2], at, to_a + (64 * wave + 8 * i) * kStepBytes);
    load_to_lds(w_from, lane_off[i % 2], at, to_w + (64 * wave + 8 * i) * kStepBytes);
  };
  // Waits for everything this wave has asked for, its part of the buffer of
  // step s among it.  In a tile's first step that includes the stores of the
  // tile before it and the loads of this tile's scales; a wait that leaves them
  // out would count on how many operations the compiler makes of them, and made
  // no difference (16 steps a tile, 491520 rows: 7.56 to 7.61 ms either way).
  // Pieces past the row's end become zeros in the weights, so that they add
  // nothing.
  // Fragments of 32 channels for each wave; a lane has four of each eight, 8*q + (lane/32)*4 + i.
  constexpr int kOutFrags = kSwiglu ? 2 : 4;
  auto arrived = [&](int s, uint8_t* a, uint8_t* w) __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(kWaitLoads);
    asm volatile("" ::: "memory");
    if (ragged && s == steps - 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (s * kStepBytes + piece[i % 2] * 16 >= int(row)) {
          *reinterpret_cast<u32x4*>(w + (64 * wave + 8 * i) * kStepBytes + lane * 16) = u32x4{0u, 0u, 0u, 0u};
          if constexpr (C::kFloat)  // what was read there instead may be a NaN
            *reinterpret_cast<u32x4*>(a + (64 * wave + 8 * i) * kStepBytes + lane * 16) = u32x4{0u, 0u, 0u, 0u};
        }
      }
    }
    __builtin_amdgcn_s_waitcnt(kWaitLdsScalar);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  const int wr = wave / 2, wc = wave % 2;
  constexpr std::integral_constant<int, -1> none{};
  constexpr std::integral_constant<int, 0> zero{};
  constexpr std::integral_constant<int, 1> one{};

#pragma unroll
  for (int i = 0; i < 8; ++i) fetch(fs, s_a0, s_w0, i);
  fetched();
  arrived(0, s_a0, s_w0);
#pragma unroll
  for (int i = 0; i < 8; ++i) fetch(fs, s_a1, s_w1, i);
  fetched();
  bool odd = false;  // whether the tile's first step is in the second buffer

  // A tile of up to 64*G rows, 32*G for each wave.
  auto form = [&](auto frags) __attribute__((always_inline)) {
    constexpr int G = decltype(frags)::value;
    // The tile's scales, loaded now for the epilogue.
    float sa[G] = {};
    f32x4 s0[4][4] = {};
    if constexpr (C::kChannels) {
      const __amdgpu_buffer_rsrc_t rows = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<float*>(p.a_scales + now.row0), 0, now.n_rows * 4, 0x00027000);
      const __amdgpu_buffer_rsrc_t channels = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<float*>(p.w_scales + int64_t(now.e) * wide), 0, wide * 4, 0x00027000);
#pragma unroll
      for (int g = 0; g < G; ++g)
        sa[g] = __uint_as_float(
            __builtin_amdgcn_raw_buffer_load_b32(rows, (32 * G * wr + 32 * g + lane % 32) * 4, 0, 0));
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int c0 = now.c0 + 32 * kOutFrags * wc + 32 * (f % kOutFrags) + (f < kOutFrags ? 0 : p.n_out);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          s0[f][q] = __builtin_bit_cast(
              f32x4, __builtin_amdgcn_raw_buffer_load_b128(channels, (c0 + 8 * q + 4 * (lane / 32)) * 4, 0, 0));
      }
    }
    u32x4 fw[2][4], fa[2][G];
    typename C::Acc acc[4][G];
    auto read = [&](int set, const uint8_t* a, const uint8_t* w, int kk, int f) __attribute__((always_inline)) {
      const int at = ((kk * 2 + lane / 32) ^ (lane / 2 % 8)) * 16;
      fw[set][f] = *reinterpret_cast<const u32x4*>(w + (128 * wc + 32 * f + lane % 32) * kStepBytes + at);
      if (f < G) fa[set][f] = *reinterpret_cast<const u32x4*>(a + (32 * G * wr + 32 * f + lane % 32) * kStepBytes + at);
    };
    // The products of the fragments in `set`; between them part kk of (a, w) is
    // read into the other set and, with kHalf >= 0, half of a step is requested
    // for (to_a, to_w): spread out, because a request holds up the wave that
    // makes it while the other waves' are being taken.
    auto part = [&](auto set, const uint8_t* a, const uint8_t* w, int kk, auto half, uint8_t* to_a, uint8_t* to_w,
                    auto fresh) __attribute__((always_inline)) {
      constexpr int kSet = decltype(set)::value, kHalf = decltype(half)::value;
#pragma unroll
      for (int f = 0; f < 4; ++f) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          typename C::Acc c = acc[f][g];
          if constexpr (decltype(fresh)::value != 0)
#pragma unroll
            for (int i = 0; i < 16; ++i) c[i] = 0;
          acc[f][g] = C::mac(fw[kSet][f], fa[kSet][g], c);
          if (g == G / 2 - 1) {
            __builtin_amdgcn_sched_barrier(0);
            read(kSet ^ 1, a, w, kk, f);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (kHalf >= 0) {
          fetch(fs, to_a, to_w, 4 * kHalf + f);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    };
    // Step s of the tile, in the buffer (a, w); (na, nw) holds the step after it.
    auto step = [&](int s, uint8_t* a, uint8_t* w, uint8_t* na, uint8_t* nw) __attribute__((always_inline)) {
      if (s == 0) {
        part(zero, a, w, 1, none, na, nw, one);
      } else {
        part(zero, a, w, 1, one, na, nw, zero);
        fetched();
      }
      part(one, a, w, 2, none, na, nw, zero);
      part(zero, a, w, 3, none, na, nw, zero);
      arrived(s + 1 < steps ? s + 1 : 0, na, nw);
      part(one, na, nw, 0, zero, a, w, zero);
    };
    int s = 0;
    if (odd) {
#pragma unroll
      for (int f = 0; f < 4; ++f) read(0, s_a1, s_w1, 0, f);
      step(s++, s_a1, s_w1, s_a0, s_w0);
    } else {
#pragma unroll
      for (int f = 0; f < 4; ++f) read(0, s_a0, s_w0, 0, f);
    }
    for (; s + 1 < steps; s += 2) {
      step(s, s_a0, s_w0, s_a1, s_w1);
      step(s + 1, s_a1, s_w1, s_a0, s_w0);
    }
    odd = s < steps;
    if (odd) step(s, s_a0, s_w0, s_a1, s_w1);
    // The second half of the request that the last step began: before the stores.
#pragma unroll
    for (int i = 4; i < 8; ++i) {
      if (odd) fetch(fs, s_a0, s_w0, i);
      else fetch(fs, s_a1, s_w1, i);
    }
    fetched();

    // Stores go through a buffer of the tile's rows: what a lane has for a row
    // or channel past the end gets an offset past the buffer and is dropped.
    const uint32_t row_bytes = uint32_t(p.n_out) * 2, out_bytes = uint32_t(now.n_rows) * row_bytes;
    const __amdgpu_buffer_rsrc_t out =
        __builtin_amdgcn_make_buffer_rsrc(p.out + int64_t(now.row0) * p.n_out, 0, out_bytes, 0x00027000);
#pragma unroll
    for (int f = 0; f < kOutFrags; ++f) {
      const int c0 = now.c0 + 32 * kOutFrags * wc + 32 * f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        // The sums stay in accumulation registers until their turn.
        asm volatile("" : "+a"(acc[f][g]));
        if constexpr (kSwiglu) asm volatile("" : "+a"(acc[f + 2][g]));
        u32x2 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = C::value(acc[f][g][4 * q + i], sa[g], s0[f][q][i]);
            if constexpr (kSwiglu) x[i] = silu_times(x[i], C::value(acc[f + 2][g][4 * q + i], sa[g], s0[f + 2][q][i]));
          }
          v[q] = u32x2{bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3])};
        }
        // Lanes l and l+32 hold the two halves of each eight channels of one
        // row: the lower one takes all of the even q, the upper of the odd.
        const int r = 32 * G * wr + 32 * g + lane % 32;
        const uint32_t at = uint32_t(r) * row_bytes + uint32_t(c0 + 8 * (lane / 32)) * 2;
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
          const u32x2 x = permlane32_swap(v[q].x, v[q + 1].x), y = permlane32_swap(v[q].y, v[q + 1].y);
          const bool some = r < now.n_rows && c0 + 8 * q < p.n_out;
          __builtin_amdgcn_raw_buffer_store_b128(u32x4{x.x, y.x, x.y, y.y}, out, some ? at + 16 * q : 0xFFFFFFF0u, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);  // one fragment at a time, or the registers do not suffice
      }
    }
  };
  do {
    if (now.n_rows > kTile / 2) form(std::integral_constant<int, 4>{});
    else form(std::integral_constant<int, 2>{});
  } while (advance(at_now, now));
  __builtin_amdgcn_s_waitcnt(kWaitLoads);  // nothing may still be on its way to LDS
}

namespace {

template <class C, bool kSwiglu>
hipError_t go_matmul(const ExpertMatmul& p, hipStream_t s) {
  const uint32_t groups = p.a_rows < uint32_t(p.n_experts) ? p.a_rows : uint32_t(p.n_experts);
  const int per = kSwiglu ? 16 : 32, strip = (kSwiglu ? 64 : 128) * kStripFrags;
  const uint32_t strips = (p.n_out + strip - 1) / strip;
  const bool alone = p.a_rows <= uint32_t(kFewRows) ||
                     (p.a_rows <= kAloneRows && int64_t(p.n_out) * p.depth * (kSwiglu ? 2 : 1) <= kAloneWeights);
  const uint32_t most = alone ? kAloneRows : kFewRows;  // rows of the groups that the first kernel takes
  if (strips * groups >= C::kStripsMin)
    hipLaunchKernelGGL((k_matmul_strip<C, kSwiglu>), dim3(strips, groups), dim3(kStripThreads), 0, s, p, most);
  else
    hipLaunchKernelGGL((k_matmul_few<C, kSwiglu>), dim3((p.n_out + per - 1) / per, groups), dim3(kFewThreads), 0, s, p,
                       most);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess || alone) return e;
  C::template tiles<kSwiglu>(p, s);
  return hipGetLastError();
}

}  // namespace

}  // namespace moe
