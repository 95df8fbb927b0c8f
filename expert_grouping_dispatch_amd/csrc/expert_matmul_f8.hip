// The experts' products in e4m3 over the expert-contiguous buffer, with a scale
// for each 128 values of a row and for each 128 x 128 block of the weights.
//
//   v[p, n] = sum_b (sa[p, b] * sw[e(p), n/128, b]) * sum_{k in block b} a[p, k] * w[e(p), n, k]  (fp32)
//   out = bf16(v), or bf16(silu(gate) * up) of two of them
//
// The inner sums come from the matrix instruction, a block in two of K = 64, and
// are multiplied and added by the vector unit, 16 operations for each 128 cycles
// of the matrix unit.  So the sums have to lie in registers that the vector unit
// reads, of which a wave has 256 at most.
#include "expert_matmul.h"

namespace moe {

namespace {

constexpr int kF8Threads = 512;  // of the tiles: 2 x 4 waves, each 128 rows by 64 weight rows

__device__ __forceinline__ f32x16 mac_f8(const u32x4 (&w)[2], const u32x4 (&a)[2], const f32x16& c) {
  struct Both {
    u32x4 v[2];
  };
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(__builtin_bit_cast(i32x8, (Both{w[0], w[1]})),
                                                         __builtin_bit_cast(i32x8, (Both{a[0], a[1]})), c, 0, 0, 0, 0,
                                                         0, 0);
}

}  // namespace

// Tiles as in k_matmul_tile, with eight waves: a wave's 128 by 64 sums take 128
// registers, the sums of the block that is being formed 32 more.
template <bool kSwiglu>
__global__ __launch_bounds__(kF8Threads, 2) void k_matmul_tile_f8(ExpertMatmul p) {
  __shared__ __align__(16) uint8_t s_a0[kTile * kStepBytes], s_a1[kTile * kStepBytes];
  __shared__ __align__(16) uint8_t s_w0[kTile * kStepBytes], s_w1[kTile * kStepBytes];
  __shared__ float s_sa0[kTile], s_sa1[kTile], s_sw0[kWave], s_sw1[kWave];
  __shared__ TileList<kF8Threads> s_tiles;
  const int tid = threadIdx.x, lane = tid % kWave, wave = uniform(tid / kWave);
  constexpr int kChannels = kSwiglu ? kTile / 2 : kTile;
  const uint32_t col_tiles = (p.n_out + kChannels - 1) / kChannels;
  const uint32_t total = s_tiles.fill(p, col_tiles);

  // Workgroups of one XCD (blockIdx % 8) take neighbouring tiles.
  const uint32_t grid = gridDim.x, per = grid / 8, rest = grid % 8, xcd = blockIdx.x % 8;
  const uint32_t first = xcd * per + min(xcd, rest) + blockIdx.x / 8;
  auto advance = [&](Walk& at, TilePlace& t) __attribute__((always_inline)) {
    return s_tiles.next(p, total, grid, kChannels, at, t);
  };

  const int wide = kSwiglu ? 2 * p.n_out : p.n_out;
  const uint32_t row = uint32_t(p.depth);
  const int steps = (p.depth + kBlock - 1) / kBlock, half = (p.n_out + kBlock - 1) / kBlock;
  const bool ragged = p.depth % kBlock != 0;
  const uint64_t w_bytes = uint64_t(p.n_experts) * wide * row;
  const int piece[2] = {(lane % 8) ^ (lane / 16), (lane % 8) ^ (4 + lane / 16)};
  const uint32_t lane_off[2] = {uint32_t(lane / 8) * row + piece[0] * 16, uint32_t(lane / 8) * row + piece[1] * 16};
  // This wave fills LDS rows [32*wave, +32) of both operands; waves 0 to 3 the
  // scales of 64 rows each, wave 4 those of the two blocks of weight rows.
  __amdgpu_buffer_rsrc_t a_from, w_from, s_from;
  uint32_t s_off = 0;
  auto aim = [&](const TilePlace& t) __attribute__((always_inline)) {
    const int rows = max(t.n_rows - 32 * wave, 0);
    const uint64_t a0 = (uint64_t(t.row0) + (rows > 0 ? 32 * wave : 0)) * row;
    const int first_w = t.c0 + (kSwiglu ? 32 * (wave / 2) + (wave % 2) * p.n_out : 32 * wave);
    const uint64_t w0 = (uint64_t(t.e) * wide + first_w) * row;
    a_from = buffer_of(static_cast<const uint8_t*>(p.a) + a0, uint64_t(rows) * row);
    w_from = buffer_of(static_cast<const uint8_t*>(p.w) + min(w0, w_bytes), w0 < w_bytes ? w_bytes - w0 : 0);
    if (wave < 4) {
      s_from = buffer_of(reinterpret_cast<const uint8_t*>(p.a_scales + uint64_t(t.row0) * steps),
                         uint64_t(t.n_rows) * steps * 4);
      s_off = uint32_t(tid) * steps * 4;
    } else {
      const uint64_t blocks = uint64_t(kSwiglu ? 2 : 1) * half * steps;
      s_from = buffer_of(reinterpret_cast<const uint8_t*>(p.w_scales + t.e * blocks), blocks * 4);
      const int b = t.c0 / kBlock;
      s_off = uint32_t(lane == 0 ? b : kSwiglu ? half + b : min(b + 1, half - 1)) * steps * 4;
    }
  };
  TilePlace now, ahead;
  Walk at_now{first, 0}, at_ahead{first, 0};
  if (!advance(at_now, now)) return;
  advance(at_ahead, ahead);
  aim(ahead);
  int fs = 0;  // the next step of `ahead` to fetch
  const int turn = ragged ? 0 : int(xcd * uint32_t(steps) / 8);
  auto fetch = [&](uint8_t* to_a, uint8_t* to_w, float* to_sa, float* to_sw) __attribute__((always_inline)) {
    const int s = fs + turn < steps ? fs + turn : fs + turn - steps;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t at = uint32_t(s) * kStepBytes + uint32_t(8 * i) * row;
      load_to_lds(a_from, lane_off[i % 2], at, to_a + (32 * wave + 8 * i) * kStepBytes);
      load_to_lds(w_from, lane_off[i % 2], at, to_w + (32 * wave + 8 * i) * kStepBytes);
    }
    if (wave <= 4) load_word_to_lds(s_from, s_off, uint32_t(s) * 4, wave < 4 ? to_sa + 64 * wave : to_sw);
    if (++fs == steps) {
      fs = 0;
      if (advance(at_ahead, ahead)) aim(ahead);
      __builtin_amdgcn_s_waitcnt(kWaitLdsScalar);
    }
  };
  // Pieces past the row's end become zeros in both operands: what was read there instead may be a NaN.
  auto arrived = [&](int s, uint8_t* a, uint8_t* w) __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(kWaitLoads);
    asm volatile("" ::: "memory");
    if (ragged && s == steps - 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (s * kStepBytes + piece[i % 2] * 16 >= p.depth) {
          *reinterpret_cast<u32x4*>(w + (32 * wave + 8 * i) * kStepBytes + lane * 16) = u32x4{0u, 0u, 0u, 0u};
          *reinterpret_cast<u32x4*>(a + (32 * wave + 8 * i) * kStepBytes + lane * 16) = u32x4{0u, 0u, 0u, 0u};
        }
    }
    __builtin_amdgcn_s_waitcnt(kWaitLdsScalar);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  const int wr = wave / 4, wc = wave % 4;
  const uint32_t lane_at = (lane % 32) * kStepBytes + ((lane / 32) ^ (lane / 2 % 8)) * 16;
  fetch(s_a0, s_w0, s_sa0, s_sw0);
  bool odd = false;  // whether the tile's first step is in the second buffer

  // A tile of up to 64*G rows, 32*G for each wave.
  auto form = [&](auto frags) __attribute__((always_inline)) {
    constexpr int G = decltype(frags)::value;
    f32x16 acc[2][G];
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int g = 0; g < G; ++g) acc[f][g] = f32x16{};
    auto step = [&](int s, uint8_t* a, uint8_t* w, const float* sa, const float* sw, uint8_t* na, uint8_t* nw,
                    float* nsa, float* nsw) __attribute__((always_inline)) {
      arrived(s, a, w);
      fetch(na, nw, nsa, nsw);
      // Where this lane's pieces of fragment 0 lie; opaque, or the address of every fragment in every buffer is
      // kept in a register of its own.
      uint32_t at_a = lane_at + 32 * G * wr * kStepBytes, at_w = lane_at + 64 * wc * kStepBytes;
      asm volatile("" : "+v"(at_a), "+v"(at_w));
      auto piece_of = [&](const uint8_t* rows, uint32_t at, int f, int kk) __attribute__((always_inline)) {
        return *reinterpret_cast<const u32x4*>(rows + (at ^ (kk * 32)) + 32 * f * kStepBytes);
      };
      u32x4 fw[2][2][2];
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) fw[f][kk / 2][kk % 2] = piece_of(w, at_w, f, kk);
      float by[2];
#pragma unroll
      for (int f = 0; f < 2; ++f) by[f] = sw[kSwiglu ? f : wc / 2];
      u32x4 fa[2][2];
      auto read = [&](int g, int half) __attribute__((always_inline)) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) fa[half][kk] = piece_of(a, at_a, g, 2 * half + kk);
      };
      read(0, 0);
      read(0, 1);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float sr = sa[32 * G * wr + 32 * g + lane % 32];
        f32x16 part[2];
        __builtin_amdgcn_sched_barrier(0);
        part[0] = mac_f8(fw[0][0], fa[0], f32x16{});
        part[1] = mac_f8(fw[1][0], fa[0], f32x16{});
        __builtin_amdgcn_sched_barrier(0);
        if (g + 1 < G) read(g + 1, 0);
        __builtin_amdgcn_sched_barrier(0);
        part[0] = mac_f8(fw[0][1], fa[1], part[0]);
        part[1] = mac_f8(fw[1][1], fa[1], part[1]);
        __builtin_amdgcn_sched_barrier(0);
        if (g + 1 < G) read(g + 1, 1);
        __builtin_amdgcn_sched_barrier(0);
        add_scaled(acc[0][g], part[0], sr * by[0]);
        add_scaled(acc[1][g], part[1], sr * by[1]);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    int s = 0;
    if (odd) step(s++, s_a1, s_w1, s_sa1, s_sw1, s_a0, s_w0, s_sa0, s_sw0);
    for (; s + 1 < steps; s += 2) {
      step(s, s_a0, s_w0, s_sa0, s_sw0, s_a1, s_w1, s_sa1, s_sw1);
      step(s + 1, s_a1, s_w1, s_sa1, s_sw1, s_a0, s_w0, s_sa0, s_sw0);
    }
    odd = s < steps;
    if (odd) step(s, s_a0, s_w0, s_sa0, s_sw0, s_a1, s_w1, s_sa1, s_sw1);

    // Stores go through a buffer of the tile's rows: what a lane has for a row
    // or channel past the end gets an offset past the buffer and is dropped.
    constexpr int kOutFrags = kSwiglu ? 1 : 2;
    const uint32_t row_bytes = uint32_t(p.n_out) * 2, out_bytes = uint32_t(now.n_rows) * row_bytes;
    const __amdgpu_buffer_rsrc_t out =
        __builtin_amdgcn_make_buffer_rsrc(p.out + int64_t(now.row0) * p.n_out, 0, out_bytes, 0x00027000);
#pragma unroll
    for (int f = 0; f < kOutFrags; ++f) {
      const int c0 = now.c0 + 32 * kOutFrags * wc + 32 * f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        u32x2 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = acc[f][g][4 * q + i];
            if constexpr (kSwiglu) x[i] = silu_times(x[i], acc[1][g][4 * q + i]);
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

struct MatF8 {
  static constexpr int kSize = 1;
  static constexpr bool kFloat = true, kChannels = false, kBlocks = true;
  typedef f32x16 Acc;
  typedef f32x4 FewAcc;
  static __device__ __forceinline__ Acc mac(const u32x4 (&w)[2], const u32x4 (&a)[2], const Acc& c) {
    return mac_f8(w, a, c);
  }
  static __device__ __forceinline__ float value(float c, float, float) { return c; }
  template <bool kSwiglu>
  static void tiles(const ExpertMatmul& p, hipStream_t s) {
    hipLaunchKernelGGL((k_matmul_tile_f8<kSwiglu>), dim3(256), dim3(kF8Threads), 0, s, p);
  }
};

}  // namespace

hipError_t launch_expert_matmul_f8(const ExpertMatmul& p, bool swiglu, hipStream_t s) {
  if (p.a_rows == 0) return hipSuccess;
  return swiglu ? go_matmul<MatF8, true>(p, s) : go_matmul<MatF8, false>(p, s);
}

}  // namespace moe
