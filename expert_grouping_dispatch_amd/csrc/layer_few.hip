// The whole layer for a few tokens in two kernels.
//
// Both products read an active expert's weights once where few slots share it:
// 6*hidden*inter bytes per expert in bf16 (half in int8) against a few rows of
// activations, so the layer is bound by how fast HBM delivers the weights.
// With more slots the first product reads them once for every 64 of them, past
// the caches, and the second once for every 32, mostly from L2; and the second
// fetches all of h for each workgroup's few channels, so its time grows with
// the slots: 8 experts, 4096 x 2048, 32, 64 and 128 slots on each take 117, 208 and
// 368 us in int8, 123, 215 and 375 in e4m3, 142, 263 and 458 in bf16, the grouped
// calls 75, 142 and 111, 90, 153 and 105, 127, 263 and 187 us (replayed).  Grouping
// costs each workgroup one pass over the few ids instead of a kernel of its own.
//
//   k_few_up     one workgroup per (expert, 64 intermediate channels): lists the
//                expert's slots and forms gate, up and h = silu(gate)*up for up to
//                64 of them at a time.  Weights come in whole cache lines through
//                LDS: 247 active experts in int8, 7168 x 2048, 776 slots, 1105 us,
//                6.6 TB/s; two experts in bf16, 4096 x 14336, 73 us, 6.4 TB/s.  h
//                goes out as two bf16 values, the type of the second product's
//                matrix instruction: its rounding to bf16 and what that leaves.
//   k_few_up_split  the same for small grids: 16 channels a workgroup, its waves
//                share k.  4 experts, 1040 x 528, 13 tokens: 11 us, the latency of
//                two rounds of loads, the sums across waves and the launch.
//   k_few_down   one workgroup per 4 to 32 output channels: groups the slots, its
//                waves take (expert, part of k) items, every slot's result goes to
//                its own place in LDS in fp32, and then each token's choices are
//                summed in ascending order, so the result does not depend on which
//                wave came first.  Weights go straight to registers, since LDS
//                holds the results: in whole lines for 4x4 products where an
//                expert has up to four slots and long rows, in 16x16 products
//                else.  The int8 layer above 650 us, 5.6 TB/s; the bf16 one 43 us,
//                5.5 TB/s.  Both parts of h are multiplied whatever the sizes, so
//                that a token's result does not depend on how many others there
//                are and the output's own rounding is all the error there is
//                (0.0017 of the result's norm; 0.0023 with h in bf16 alone).  The
//                second part's loads show from about five slots an expert on: 97
//                tokens, 8 of 256 experts in int8, 7168 x 2048, the layer 1734 us,
//                1658 with h in bf16; 200 tokens, 2048 x 1024, 466 and 388; 256
//                tokens on all of 8 experts, 4096 x 2048, 644 and 393.
//
// e4m3 weights have a scale for each 128 values of k and 128 rows: a block's sums
// are multiplied with it and added in fp32.  The two experts above 40 us (5.9 TB/s)
// and 29 us (4.0: starts and ends are a larger part), the 247 experts 1085 us (6.7
// TB/s) and 666 us (5.4).
#include <algorithm>

#include "experts.h"
#include "lds_fill.h"
#include "stream.h"

namespace moe {

namespace {

constexpr int kFewMaxSlots = 2048;
constexpr int kUpWaves = 4, kUpThreads = kUpWaves * kWave;
// Slots at a time in k_few_down with RT row tiles: 128 KB of results.  Half of
// it read the weights of 64 experts, 1024 -> 4096, twice for 2048 slots: the
// layer 565 us against 521 us in bf16, 427 against 401 us in int8.
constexpr int down_slots(int rt) { return 2048 / rt; }

// Slots at or past the boundary row are unrouted.
__device__ __forceinline__ int real_slots(const PadMask& pad, int n_rows, int top_k) {
  if (pad.count == nullptr) return n_rows * top_k;
  const int64_t real = int64_t(*pad.count) - int64_t(pad.tp_rank) * n_rows;
  return int(real < 0 ? 0 : real > n_rows ? n_rows : real) * top_k;
}

template <typename IdT>
__device__ __forceinline__ int expert_of(const IdT* ids, int i, int n_experts) {
  const IdT e = ids[i];
  return e >= 0 && e < IdT(n_experts) ? int(e) : -1;
}

}  // namespace

// ---- gate, up and their product --------------------------------------------

constexpr int kUpChannels = 64;  // per workgroup: 64 gate and 64 up rows
constexpr int kUpWBytes = 2 * kUpChannels * 128, kUpXBytes = 8192;

// A step is 128 bytes of every weight row: 64 values of k in bf16, 128 in
// int8, against 128 or 256 bytes of every activation row.
struct UpBf16 {
  static constexpr int kStep = 64, kXRow = 128, kWSize = 2;
  static constexpr bool kBlocks = false;  // whether each 128 values of k and each 128 weight rows have a scale
  // Products of the 16 bytes this lane has of a weight row, piece c of 8, with n activation rows in x.
  static __device__ __forceinline__ f32x16 mac(const u32x4& w, const uint8_t* x, int row, int c, f32x16 acc) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(x + row * kXRow + (c ^ (row / 2 % 8)) * 16);
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, v), acc, 0,
                                                   0, 0);
  }
};
struct UpI8 {
  static constexpr int kStep = 128, kXRow = 256, kWSize = 1;
  static constexpr bool kBlocks = false;
  static __device__ __forceinline__ f32x16 mac(const u32x4& w, const uint8_t* x, int row, int c, f32x16 acc) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(x + row * kXRow + ((2 * c + j) ^ (row % 16)) * 16);
      const u32x2 lo = bf16_of_i8(w[2 * j]), hi = bf16_of_i8(w[2 * j + 1]);
      acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, (u32x4{lo.x, lo.y, hi.x, hi.y})),
                                                    __builtin_bit_cast(bf16x8, v), acc, 0, 0, 0);
    }
    return acc;
  }
};

struct UpF8 {  // a step is a block of k
  static constexpr int kStep = 128, kXRow = 256, kWSize = 1;
  static constexpr bool kBlocks = true;
  static __device__ __forceinline__ f32x16 mac(const u32x4& w, const uint8_t* x, int row, int c, f32x16 acc) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(x + row * kXRow + ((2 * c + j) ^ (row % 16)) * 16);
      const u32x2 lo = bf16_of_f8(w[2 * j]), hi = bf16_of_f8(w[2 * j + 1]);
      acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, (u32x4{lo.x, lo.y, hi.x, hi.y})),
                                                    __builtin_bit_cast(bf16x8, v), acc, 0, 0, 0);
    }
    return acc;
  }
};

__device__ __forceinline__ int blocks_of(int n) { return (n + kBlock - 1) / kBlock; }

// Grids of k_few_up of at least this many workgroups of 64 channels; smaller
// ones leave CUs idle and take 16 channels a workgroup (k_few_up_split).  The
// layer in us, 64 channels against 16, in bf16, int8 and e4m3:
//   32 workgroups (1 token, 1 of 8 experts, 8192 x 2048)    81/32   66/25  60/28
//   128 (4 tokens, 2 of 8, 4096 x 1024)                     53/34   40/24  37/25
//   256 (1 token, 8 of 64, 7168 x 2048)                    122/121  78/67  75/68
//   256 (2 tokens, 8 of 64, 4096 x 1024)                    69/68   49/42  46/44
//   512 (1 token, 8 of 32, 4096 x 4096)                    138/144  75/75  75/78
// At 256 itself the smaller form is still ahead with 8-bit weights.
constexpr int kUpStripsMin = 256;
// Output channels a workgroup of k_few_down: what spreads them over this many
// workgroups, in groups of four, at most 32; above 16 the workgroup has two
// row tiles.  Rows of a tile past the workgroup's are not read.
// Layers in int8, bf16 and e4m3: 256 experts, 776 slots, 7168 channels, 1765, 3218
// and 1726 us with 28 each, 1776, 3260 and 1733 with 32 on 224 workgroups, 1947, 3409
// and 1929 with 16; 2048 channels, 32 tokens, 8 of 64 experts, 188, 294 and 187 with 8
// each, 207, 333 and 205 with 16; 5120 channels, 1 token, 8 of 64, 47, 68 and 47 with
// 20 each, 59, 80 and 59 with 16.
constexpr int kDownGroups = 256;
constexpr int kDownWaves = 8;
// Rows of w_down of at least this many values are read in whole lines
// (few_down_lines) for experts with few slots.  The layer with and without, in
// int8, bf16 and e4m3:
//   97 tokens, 8 of 256 experts, 7168 x 2048  1750/1827  3217/3368  1710/1805
//   32 tokens, 8 of 64, 2048 x 1408            141/144    208/212    140/142
//   4 tokens, 8 of 64, 2048 x 2048              76/78     114/116     74/76
//   4 tokens, 8 of 64, 2048 x 1280              65/63      88/89      63/60
//   1 token, 8 of 64, 2048 x 1024               23/21      27/27      23/21
//   1 token, 2 of 8, 4096 x 14336               69/68     116/111     68/66.5
// Two long experts lose a little by it, many experts gain.
constexpr int kLinesMin = 1280;
constexpr int kUpMost = 3;  // buffers
// What bf16 leaves of two values whose bf16 forms are `hi`, in bf16; nothing
// where that is infinite or NaN.
__device__ __forceinline__ uint32_t rest_pair(float a, float b, uint32_t hi) {
  const float ra = a - __uint_as_float(hi << 16), rb = b - __uint_as_float(hi & 0xFFFF0000u);
  return bf16_pair(fabsf(ra) < INFINITY ? ra : 0.0f, fabsf(rb) < INFINITY ? rb : 0.0f);
}

// h of four channels of a slot, at `to`, and what bf16 leaves of it, h_rest further.
__device__ __forceinline__ void store_h(uint16_t* to, int64_t h_rest, const f32x4& gate, const f32x4& up) {
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = silu_times(gate[i], up[i]);
  const u32x2 hi{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
  *reinterpret_cast<u32x2*>(to) = hi;
  *reinterpret_cast<u32x2*>(to + h_rest) = u32x2{rest_pair(v[0], v[1], hi.x), rest_pair(v[2], v[3], hi.y)};
}

struct UpBuffers {
  uint8_t *w[kUpMost], *xa[kUpMost], *xb[kUpMost];  // weights; activation rows 0..31 and 32..63
};

// One expert's gate and up rows of channels [c0, c0 + 64) times n <= 32*G of
// its slots.  NB buffers of a step are filled straight from global memory, the
// weights non-temporal and in whole cache lines; each wave takes 16 gate and
// the 16 up rows of the same channels as one 32-row operand, so one lane has
// both.  16-byte pieces lie in an order that spreads a read over all banks:
// piece c of a 128-byte row r at c ^ (r/2 % 8), of a 256-byte row at c ^ (r % 16).
template <class C, int G, int NB, bool kScaled>
__device__ __forceinline__ void few_up(const uint8_t* x, int n_rows, int hidden, int top_k, const uint8_t* w,
                                       uint64_t w_bytes, const float* w_scales, int inter, int c0,
                                       const uint16_t* list, int n, uint16_t* h, int64_t h_rest, const UpBuffers& buf) {
  const int lane = threadIdx.x % kWave, wave = uniform(int(threadIdx.x / kWave));
  constexpr int kXFills = C::kXRow == 128 ? G : 2 * G;  // requests of activation rows per wave and step
  constexpr int kFills = 4 + kXFills;
  const uint32_t w_row = uint32_t(hidden) * C::kWSize;
  const int steps = (hidden + C::kStep - 1) / C::kStep;
  const bool ragged = hidden % C::kStep != 0;
  // Weights: LDS rows [32*wave, +32), eight per request: gate rows c, .., c+15, then up rows.
  const int c = min(c0 + 16 * wave, inter - 16);
  const uint64_t at_gate = uint64_t(c) * w_row, at_up = uint64_t(inter + c) * w_row;
  const __amdgpu_buffer_rsrc_t gate = buffer_of(w + at_gate, w_bytes - at_gate);
  const __amdgpu_buffer_rsrc_t up = buffer_of(w + at_up, w_bytes - at_up);
  const int w_piece[2] = {(lane % 8) ^ (lane / 16), (lane % 8) ^ (4 + lane / 16)};
  const uint32_t w_off[2] = {uint32_t(lane / 8) * w_row + w_piece[0] * 16,
                             uint32_t(lane / 8) * w_row + w_piece[1] * 16};
  // Activations: request i = wave + 4*j fills rows from i*8 (128-byte rows) or i*4.
  const __amdgpu_buffer_rsrc_t rows = buffer_of(x, uint64_t(n_rows) * hidden * 2);
  int x_piece[kXFills];
  uint32_t x_off[kXFills];
#pragma unroll
  for (int j = 0; j < kXFills; ++j) {
    const int i = wave + 4 * j;
    int r;
    if constexpr (C::kXRow == 128) {
      r = 8 * i + lane / 8;
      x_piece[j] = (lane % 8) ^ (r / 2 % 8);
    } else {
      r = 4 * i + lane / 16;
      x_piece[j] = (lane % 16) ^ (r % 16);
    }
    x_off[j] = uint32_t(list[min(r, n - 1)] / top_k) * uint32_t(hidden * 2) + x_piece[j] * 16;
  }
  // Where request j of the activations goes: 4 KB a half in bf16, 8 KB in int8.
  constexpr int kHalf = 32 * C::kXRow, kPerHalf = kHalf / 1024;
  auto x_place = [&](int j, uint8_t* xa, uint8_t* xb) {
    const int i = wave + 4 * j;
    return j * 4 < kPerHalf ? xa + i * 1024 : xb + (i - kPerHalf) * 1024;
  };
  // Workgroups begin at different steps: rows whose length is a power of two
  // would have all of them at the same few memory channels at any time.
  const int turn = ragged ? 0 : int((blockIdx.x * 5 + blockIdx.y * 3) % uint32_t(steps));
  struct BlockScales {
    float gate, up;
  };
  const float* s_gate = C::kBlocks ? w_scales + int64_t(c / kBlock) * steps : nullptr;
  const float* s_up = C::kBlocks ? s_gate + int64_t(blocks_of(inter)) * steps : nullptr;
  auto fetch = [&](int nth, uint8_t* to_w, uint8_t* xa, uint8_t* xb, BlockScales& by) {
    const int s = nth + turn < steps ? nth + turn : nth + turn - steps;
    if constexpr (C::kBlocks) by = BlockScales{s_gate[s], s_up[s]};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      load_to_lds<true>(i < 2 ? gate : up, w_off[i % 2], uint32_t(s) * 128 + uint32_t(8 * (i % 2)) * w_row,
                        to_w + (32 * wave + 8 * i) * 128);
#pragma unroll
    for (int j = 0; j < kXFills; ++j) load_to_lds(rows, x_off[j], uint32_t(s) * C::kXRow, x_place(j, xa, xb));
  };
  f32x16 acc[G];
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[g][i] = 0.0f;
  BlockScales by[NB] = {};
  auto step = [&](int s, uint8_t* w, uint8_t* xa, uint8_t* xb, const BlockScales& by, uint8_t* next_w, uint8_t* next_xa,
                  uint8_t* next_xb, BlockScales& next_by) {
    if (NB == 3 && s + 1 < steps) __builtin_amdgcn_s_waitcnt(wait_all_but(NB == 3 ? kFills : 0));
    else __builtin_amdgcn_s_waitcnt(kWaitLoads);
    asm volatile("" ::: "memory");
    if (ragged && s == steps - 1) {  // pieces past the rows' end: zeros in both, so that they add nothing
      const u32x4 zero{0u, 0u, 0u, 0u};
      const int left = (hidden - s * C::kStep) * C::kWSize, x_left = (hidden - s * C::kStep) * 2;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (w_piece[i % 2] * 16 >= left) *reinterpret_cast<u32x4*>(w + (32 * wave + 8 * i) * 128 + lane * 16) = zero;
#pragma unroll
      for (int j = 0; j < kXFills; ++j)
        if (x_piece[j] * 16 >= x_left) *reinterpret_cast<u32x4*>(x_place(j, xa, xb) + lane * 16) = zero;
    }
    __builtin_amdgcn_s_waitcnt(kWaitLdsScalar);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (s + NB - 1 < steps) fetch(s + NB - 1, next_w, next_xa, next_xb, next_by);
    f32x16 part[C::kBlocks ? G : 1];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const int c = 2 * kk + lane / 32, r = 32 * wave + lane % 32;
      const u32x4 v = *reinterpret_cast<const u32x4*>(w + r * 128 + (c ^ (r / 2 % 8)) * 16);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if constexpr (C::kBlocks) part[g] = C::mac(v, g == 0 ? xa : xb, lane % 32, c, kk == 0 ? f32x16{} : part[g]);
        else acc[g] = C::mac(v, g == 0 ? xa : xb, lane % 32, c, acc[g]);
      }
    }
    if constexpr (C::kBlocks) {  // gate rows in the first eight of a lane's sums, up rows in the others
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[g][i] = __builtin_fmaf(part[g][i], i < 8 ? by.gate : by.up, acc[g][i]);
    }
  };
#pragma unroll
  for (int b = 0; b < NB - 1; ++b)
    if (b < steps) fetch(b, buf.w[b], buf.xa[b], buf.xb[b], by[b]);
  for (int s = 0; s < steps; s += NB) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      constexpr int kBack = NB - 1;
      const int next = (b + kBack) % NB;
      if (s + b < steps)
        step(s + b, buf.w[b], buf.xa[b], buf.xb[b], by[b], buf.w[next], buf.xa[next], buf.xb[next], by[next]);
    }
  }
  // This lane's channels: 8*q + 4*(lane/32) + i of the wave's 16, gate in acc[8*.. of q 0, 1], up in q 2, 3.
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int at = 32 * g + lane % 32;
    if (at >= n) continue;
    uint16_t* row = h + int64_t(list[at]) * inter;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int ch = c + 8 * q + 4 * (lane / 32);
      f32x4 sg{1.0f, 1.0f, 1.0f, 1.0f}, su = sg;
      if constexpr (kScaled) {
        sg = *reinterpret_cast<const f32x4*>(w_scales + ch);
        su = *reinterpret_cast<const f32x4*>(w_scales + inter + ch);
      }
      f32x4 a, b;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = acc[g][4 * q + i];
        b[i] = acc[g][8 + 4 * q + i];
        if constexpr (kScaled) {
          a[i] *= sg[i];
          b[i] *= su[i];
        }
      }
      store_h(row + ch, h_rest, a, b);
    }
  }
  __syncthreads();  // the buffers are filled again for the next slots
}

// blockIdx.y: the expert, or, when there are fewer slots than experts, a slot,
// which stands for its expert if it is the first slot on it.  Lists the slots
// of the expert and returns their number, 0 where there is nothing to do.
template <typename IdT>
__device__ __forceinline__ int list_slots(const IdT* ids, int slots, int n_experts, bool by_slot, uint16_t* s_list,
                                          int* s_n, int& e) {
  const int tid = threadIdx.x;
  if (tid == 0) s_n[0] = s_n[1] = 0;
  e = blockIdx.y;
  if (by_slot) {
    if (e >= slots) return 0;
    e = expert_of(ids, e, n_experts);
    if (e < 0) return 0;
  }
  __syncthreads();
  for (int i = tid; i < slots; i += kUpThreads) {
    if (expert_of(ids, i, n_experts) == e) {
      if (by_slot && i < int(blockIdx.y)) s_n[1] = 1;
      s_list[atomicAdd(&s_n[0], 1)] = uint16_t(i);  // any order: a slot's result does not depend on its column
    }
  }
  __syncthreads();
  e = uniform(e);
  return uniform(s_n[1] != 0 ? 0 : s_n[0]);
}

// blockIdx.x: 64 channels.
template <class C, bool kScaled, typename IdT>
__global__ __launch_bounds__(kUpThreads, 2) void k_few_up(const uint8_t* __restrict__ x, int n_rows, int hidden,
                                                          int top_k, const IdT* __restrict__ ids, PadMask pad,
                                                          int n_experts, bool by_slot,
                                                          const uint8_t* __restrict__ w,
                                                          const float* __restrict__ w_scales, int inter,
                                                          uint16_t* __restrict__ h) {
  // Named apart, so that the compiler sees that filling one does not touch the others.
  __shared__ __align__(16) uint8_t s_w0[kUpWBytes], s_w1[kUpWBytes], s_w2[kUpWBytes];
  __shared__ __align__(16) uint8_t s_x0[kUpXBytes], s_x1[kUpXBytes], s_x2[kUpXBytes];
  __shared__ uint16_t s_list[kFewMaxSlots];
  __shared__ int s_n[2];
  int e;
  const int total = list_slots(ids, real_slots(pad, n_rows, top_k), n_experts, by_slot, s_list, s_n, e);
  const int64_t h_rest = int64_t(n_rows) * top_k * inter;
  const uint64_t each = uint64_t(2) * inter * hidden * C::kWSize;
  const uint8_t* we = w + e * each;
  const float* se = C::kBlocks  ? w_scales + int64_t(e) * 2 * blocks_of(inter) * blocks_of(hidden)
                    : kScaled ? w_scales + int64_t(e) * 2 * inter
                              : nullptr;
  const uint64_t w_bytes = (n_experts - e) * each;
  const int c0 = blockIdx.x * kUpChannels;
  for (int i = 0; i < total; i += 64) {
    const int n = total - i;
    UpBuffers buf{{s_w0, s_w1, s_w2}, {s_x0, s_x1, s_x2}, {s_x0, s_x1, s_x2}};
    if (n <= 32) {
      few_up<C, 1, 3, kScaled>(x, n_rows, hidden, top_k, we, w_bytes, se, inter, c0, s_list + i, n, h, h_rest, buf);
    } else if constexpr (C::kXRow == 128) {
#pragma unroll
      for (int b = 0; b < kUpMost; ++b) buf.xb[b] = buf.xa[b] + kUpXBytes / 2;
      few_up<C, 2, 3, kScaled>(x, n_rows, hidden, top_k, we, w_bytes, se, inter, c0, s_list + i, min(n, 64), h,
                               h_rest, buf);
    } else {
      // 64 rows of 256 bytes take the third weight buffer and two activation buffers: two steps deep
      const UpBuffers wide{{s_w0, s_w1}, {s_w2, s_x0}, {s_w2 + kUpXBytes, s_x1}};
      few_up<C, 2, 2, kScaled>(x, n_rows, hidden, top_k, we, w_bytes, se, inter, c0, s_list + i, min(n, 64), h,
                               h_rest, wide);
    }
  }
}

// The same for small grids: 16 channels a workgroup, k split over its waves,
// weights straight to registers (stream.h), the parts joined in LDS.
// list[0 .. n), n <= 16*NG.
template <class C, int NG, bool kScaled, bool kBlocks>
__device__ __forceinline__ void few_up_split(const uint8_t* x, int hidden, int top_k, const uint8_t* w,
                                             const float* w_scales, int inter, int tile, const uint16_t* list, int n,
                                             uint16_t* h, int64_t h_rest, f32x4* s_part) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int64_t w_row = int64_t(hidden) * (C::kWBytes / 16);
  const uint8_t* wp[2];
  const uint8_t* xp[NG];
  wp[0] = w + int64_t(tile * 16 + lane % 16) * w_row;
  wp[1] = wp[0] + int64_t(inter) * w_row;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int slot = list[min(g * 16 + lane % 16, n - 1)];
    xp[g] = x + int64_t(slot / top_k) * hidden * 2;
  }
  f32x4 acc[2][NG];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int g = 0; g < NG; ++g) acc[r][g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  int begin, end;
  step_range(hidden, wave, kUpWaves, begin, end);
  constexpr int U = 128 / C::kWBytes / NG;  // what the registers hold
  if constexpr (kBlocks) {
    const int blocks = blocks_of(hidden);
    const float* const sp[2] = {w_scales + int64_t(tile / (kBlock / 16)) * blocks,
                                w_scales + int64_t(blocks_of(inter) + tile / (kBlock / 16)) * blocks};
    stream_scaled<C, 2, NG, U>(wp, xp, sp, begin, end, hidden, acc);
  } else {
    stream_products<C, 2, NG, U>(wp, xp, begin, end, hidden, acc);
  }
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int g = 0; g < NG; ++g) s_part[((wave * 2 + r) * NG + g) * kWave + lane] = acc[r][g];
  __syncthreads();
  for (int g = wave; g < NG; g += kUpWaves) {
    f32x4 sum[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      sum[r] = s_part[(r * NG + g) * kWave + lane];
#pragma unroll
      for (int v = 1; v < kUpWaves; ++v) {
        const f32x4 p = s_part[((v * 2 + r) * NG + g) * kWave + lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[r][i] += p[i];
      }
    }
    const int at = g * 16 + lane % 16, c = tile * 16 + (lane / 16) * 4;
    if (at < n) {
      if constexpr (kScaled) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum[0][i] *= w_scales[c + i];
          sum[1][i] *= w_scales[inter + c + i];
        }
      }
      store_h(h + int64_t(list[at]) * inter + c, h_rest, sum[0], sum[1]);
    }
  }
  __syncthreads();  // s_part is rewritten for the next slots
}

// blockIdx.x: 16 channels.
template <class Up, class C, bool kScaled, typename IdT>
__global__ __launch_bounds__(kUpThreads, 2) void k_few_up_split(
    const uint8_t* __restrict__ x, int n_rows, int hidden, int top_k, const IdT* __restrict__ ids, PadMask pad,
    int n_experts, bool by_slot, const uint8_t* __restrict__ w, const float* __restrict__ w_scales, int inter,
    uint16_t* __restrict__ h) {
  __shared__ uint16_t s_list[kFewMaxSlots];
  __shared__ int s_n[2];
  __shared__ f32x4 s_part[kUpWaves * 2 * 4 * kWave];
  int e;
  const int total = list_slots(ids, real_slots(pad, n_rows, top_k), n_experts, by_slot, s_list, s_n, e);
  const int64_t h_rest = int64_t(n_rows) * top_k * inter;
  const uint8_t* we = w + int64_t(e) * 2 * inter * hidden * (C::kWBytes / 16);
  const float* se = Up::kBlocks ? w_scales + int64_t(e) * 2 * blocks_of(inter) * blocks_of(hidden)
                    : kScaled   ? w_scales + int64_t(e) * 2 * inter
                                : nullptr;
  for (int i = 0; i < total; i += 64) {
    const int n = min(total - i, 64);
    if (n <= 16)
      few_up_split<C, 1, kScaled, Up::kBlocks>(x, hidden, top_k, we, se, inter, blockIdx.x, s_list + i, n, h, h_rest, s_part);
    else if (n <= 32)
      few_up_split<C, 2, kScaled, Up::kBlocks>(x, hidden, top_k, we, se, inter, blockIdx.x, s_list + i, n, h, h_rest, s_part);
    else
      few_up_split<C, 4, kScaled, Up::kBlocks>(x, hidden, top_k, we, se, inter, blockIdx.x, s_list + i, n, h, h_rest, s_part);
  }
}

// ---- down and the weighted sum ------------------------------------------------

// The scales of a workgroup's rows of w_down, which lie in one block of 128 or in two.
struct BlockRows {
  const float* first;  // of the first row's block, one for each block of k
  int second_at, rows;  // the first row of the second block; blocks there are, 1 or 2
  // Whether row r (below the workgroup's own rows) is in the second one.
  __device__ __forceinline__ bool of(int r) const { return rows > 1 && r >= second_at; }
};

// The results of n <= 16*NG slots over steps [begin, end), U of them requested
// at a time.  Each slot has two columns: its h in bf16 and, `rest` bytes
// further, what bf16 left of it.
template <class D, int RT, int NG, int U>
__device__ __forceinline__ void few_down_tile(const uint8_t* h, uint32_t rest, int inter, const uint8_t* w,
                                              int w_rows, const BlockRows& by, const uint16_t* list, int n, int begin,
                                              int end, int base, f32x4* s_y) {
  typedef typename D::Core C;
  const int lane = threadIdx.x % kWave;
  const uint8_t* wp[RT];
  const uint8_t* hp[2 * NG];
  f32x4 acc[RT][2 * NG];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    wp[r] = w + int64_t(min(16 * r + lane % 16, w_rows - 1)) * inter * (C::kWBytes / 16);
#pragma unroll
    for (int g = 0; g < 2 * NG; ++g) acc[r][g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    hp[g] = h + int64_t(list[min(g * 16 + lane % 16, n - 1)]) * inter * 2;
    hp[NG + g] = hp[g] + rest;
  }
  if constexpr (D::kBlocks) {
    const float* sp[RT];  // of the four rows of this lane's sums
#pragma unroll
    for (int r = 0; r < RT; ++r) sp[r] = by.first + (by.of(16 * r + lane / 16 * 4) ? blocks_of(inter) : 0);
    stream_scaled<C, RT, 2 * NG, U>(wp, hp, sp, begin, end, inter, acc);
  } else {
    stream_products<C, RT, 2 * NG, U>(wp, hp, begin, end, inter, acc);
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int at = g * 16 + lane % 16;
    if (at < n)
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        f32x4 y = acc[r][g];
#pragma unroll
        for (int q = 0; q < 4; ++q) y[q] += acc[r][NG + g][q];
        s_y[((int(list[at]) - base) * RT + r) * 4 + lane / 16] = y;
      }
  }
}

// The results of the experts that `find` takes, with up to eight slots, or with
// kWide up to 16.  Of up to eight slots each has two of the 16 columns, its h
// in bf16 and, `rest` bytes further, what bf16 left of it, whose sums are
// added at the end; of more slots each has a column of two products, with its
// h and with the rest.  `find(item)` gives an item's rows and part of k, of
// 2^bits, or false; items first, first + NW, .. below `items` are taken.  Two
// batches of U steps are in registers or on their way, weights and activations
// together (loads end in order, so activations requested later would wait for
// the next weights); the requests walk on from expert to expert ahead of the
// products, so that the stream of weights does not stop at an expert's end.
// Past the last item, and in columns without one, requests point past their
// buffer and read nothing.
struct DownItem {
  const uint8_t* w;      // the expert's rows of weights, 16 for each of RT
  const float* scales;   // of their blocks, if there are such
  const uint16_t* list;  // its slots
  f32x4* y;              // where the results of this part of k go
  int n, part;
};
constexpr int kDppRowShl8 = 0x108;  // lane l of 16 reads lane l + 8, the upper eight read 0
template <class D, int RT, int NW, int U, bool kWide, class Find>
__device__ __forceinline__ void few_down_stream(const uint8_t* h, uint64_t h_bytes, uint32_t rest, int inter,
                                                int w_rows, const BlockRows& by, int base, int first, int items,
                                                int bits, Find find) {
  typedef typename D::Core C;
  const int lane = threadIdx.x % kWave, group = lane / 16;
  const int steps = (inter + kStreamStep - 1) / kStreamStep;
  // With block scales parts and batches begin with a block of two steps, whose sums are scaled together.
  constexpr int kPer = D::kBlocks ? 2 : 1, NS = D::kBlocks ? U / 2 : 1;
  static_assert(U % kPer == 0);
  const int whole = (steps + kPer - 1) / kPer;
  constexpr int WV = C::kWBytes / 16, XV = C::kXBytes / 16, NX = kWide ? 2 : 1;
  const uint32_t w_row = uint32_t(inter) * WV, nowhere = 0x80000000u;
  const __amdgpu_buffer_rsrc_t rows = buffer_of(h, h_bytes);
  struct Walk {
    DownItem i;
    int at, s, end;
  };
  auto turn = [&](Walk& k) {  // to the next item; at >= items when there is none
    do k.at += NW;
    while (k.at < items && !find(k.at, k.i));
    k.s = (whole * k.i.part >> bits) * kPer;
    k.end = min((whole * (k.i.part + 1) >> bits) * kPer, steps);
  };
  Walk ask{}, form;
  ask.at = first - NW;
  turn(ask);
  if (ask.at >= items) return;
  form = ask;
  uint32_t w_lane[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) w_lane[r] = uint32_t(16 * r + lane % 16) * w_row + group * C::kWBytes;
  const int column = lane % 16;
  auto row_of = [&](const DownItem& i) {
    const int at = kWide ? column : column % 8;
    if (at >= i.n) return nowhere;
    return uint32_t(i.list[at]) * uint32_t(inter * 2) + (at < column ? rest : 0u) + group * C::kXBytes;
  };
  uint32_t x_lane = row_of(ask.i);
  uint32_t s_lane[RT];
  if constexpr (D::kBlocks)
#pragma unroll
    for (int r = 0; r < RT; ++r) s_lane[r] = by.of(16 * r + 4 * group) ? uint32_t(blocks_of(inter)) * 4 : 0u;
  typedef float Scales[NS][RT];
  auto request = [&](typename C::W(&w)[U][RT], typename C::X(&x)[U][NX], Scales& sc) {
    const bool live = ask.at < items;
    // Scalars, or each load becomes a loop over the lanes' values.
    const __amdgpu_buffer_rsrc_t from = buffer_of(uniform(ask.i.w), uint64_t(w_rows) * w_row);
    const int s0 = uniform(ask.s);
    if constexpr (D::kBlocks) {
      const __amdgpu_buffer_rsrc_t from_s =
          buffer_of(uniform(reinterpret_cast<const uint8_t*>(ask.i.scales)), uint64_t(by.rows) * blocks_of(inter) * 4);
#pragma unroll
      for (int u = 0; u < NS; ++u) {
        uint32_t out = live && s0 + 2 * u < ask.end ? 0u : nowhere;
        asm("" : "+v"(out));
#pragma unroll
        for (int r = 0; r < RT; ++r)
          sc[u][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(from_s, (s_lane[r] | out) + 4 * u, s0 * 2, 0));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = s0 + u;
      uint32_t out = live && s < ask.end && s * kStreamStep + group * 16 < inter ? 0u : nowhere;
      asm("" : "+v"(out));  // or the loads go into branches, and the products wait for all of them
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int v = 0; v < WV; ++v)
          w[u][r].v[v] = __builtin_amdgcn_raw_buffer_load_b128(from, (w_lane[r] | out) + 4 * C::kWBytes * u + 16 * v,
                                                               s0 * 4 * C::kWBytes, 0);
#pragma unroll
      for (int b = 0; b < NX; ++b)
#pragma unroll
        for (int v = 0; v < XV; ++v)
          x[u][b].v[v] = __builtin_amdgcn_raw_buffer_load_b128(
              rows, ((x_lane + b * rest) | out) + 4 * C::kXBytes * u + 16 * v, s0 * 4 * C::kXBytes, 0);
    }
    ask.s += U;
    if (live && ask.s >= ask.end) {
      turn(ask);
      if (ask.at < items) x_lane = row_of(ask.i);
    }
  };
  f32x4 acc[RT];
  auto clear = [&] {
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  };
  clear();
  auto products = [&](const typename C::W(&w)[U][RT], const typename C::X(&x)[U][NX], const Scales& sc) {
    if constexpr (D::kBlocks) {
#pragma unroll
      for (int u = 0; u < U; u += 2) {
        f32x4 part[RT];
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
          for (int b = 0; b < NX; ++b)
#pragma unroll
            for (int r = 0; r < RT; ++r) part[r] = C::mac(w[u + v][r], x[u + v][b], v + b == 0 ? f32x4{} : part[r]);
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[r][q] = __builtin_fmaf(part[r][q], sc[u / 2][r], acc[r][q]);
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int b = 0; b < NX; ++b)
#pragma unroll
          for (int r = 0; r < RT; ++r) acc[r] = C::mac(w[u][r], x[u][b], acc[r]);
    }
    form.s += U;
    if (form.at < items && form.s >= form.end) {
      if constexpr (!kWide) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[r][q] += __uint_as_float(dpp<kDppRowShl8, 0xF>(__float_as_uint(acc[r][q])));
      }
      if (column < form.i.n)
#pragma unroll
        for (int r = 0; r < RT; ++r) form.i.y[((int(form.i.list[column]) - base) * RT + r) * 4 + group] = acc[r];
      clear();
      turn(form);
    }
  };
  typename C::W w0[U][RT], w1[U][RT];
  typename C::X x0[U][NX], x1[U][NX];
  Scales c0, c1;
  request(w0, x0, c0);
  request(w1, x1, c1);
  while (form.at < items) {
    products(w0, x0, c0);
    request(w0, x0, c0);
    products(w1, x1, c1);  // of zeros after the last item; a way out here would let the first products wait for both
    request(w1, x1, c1);
  }
}

// Weights and activations of 4x4 products, 16 of them an instruction: lane l
// has 16 bytes of weight row l%4 and the same k of the slot in column l%4, and
// the 16 blocks l/4 are sixteen pieces of k whose sums are joined at an item's
// end.  So a load takes two whole cache lines of each of four rows, 8 lines;
// in the 16x16 instruction's layout it takes pieces of 16 lines, and the
// address unit needs about two cycles a line.
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ f32x4 mac_4x4(uint32_t w0, uint32_t w1, uint32_t x0, uint32_t x1, f32x4 acc) {
  return __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(s16x4, (u32x2{w0, w1})),
                                                __builtin_bit_cast(s16x4, (u32x2{x0, x1})), acc, 0, 0, 0);
}
struct DownBf16 {  // kStep values of k are 256 bytes of a weight row
  typedef CoreBf16 Core;
  static constexpr bool kBlocks = false;
  static constexpr int kStep = 128, kWSize = 2, kXLoads = 1;
  struct W { u32x4 v; };
  static __device__ __forceinline__ W weights(const u32x4& w) { return W{w}; }
  static __device__ __forceinline__ f32x4 mac(const W& w, const u32x4 (&x)[1], f32x4 acc) {
#pragma unroll
    for (int j = 0; j < 2; ++j) acc = mac_4x4(w.v[2 * j], w.v[2 * j + 1], x[0][2 * j], x[0][2 * j + 1], acc);
    return acc;
  }
};
struct DownI8 {
  typedef CoreI8Bf16 Core;
  static constexpr bool kBlocks = false;
  static constexpr int kStep = 256, kWSize = 1, kXLoads = 2;
  struct W { u32x2 v[4]; };
  static __device__ __forceinline__ W weights(const u32x4& w) {
    return W{{bf16_of_i8(w[0]), bf16_of_i8(w[1]), bf16_of_i8(w[2]), bf16_of_i8(w[3])}};
  }
  static __device__ __forceinline__ f32x4 mac(const W& w, const u32x4 (&x)[2], f32x4 acc) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc = mac_4x4(w.v[j].x, w.v[j].y, x[j / 2][j % 2 * 2], x[j / 2][j % 2 * 2 + 1], acc);
    return acc;
  }
};

struct DownF8 {
  typedef CoreF8Bf16 Core;
  static constexpr bool kBlocks = true;
  static constexpr int kStep = 256, kWSize = 1, kXLoads = 2;
  struct W { u32x2 v[4]; };
  static __device__ __forceinline__ W weights(const u32x4& w) {
    return W{{bf16_of_f8(w[0]), bf16_of_f8(w[1]), bf16_of_f8(w[2]), bf16_of_f8(w[3])}};
  }
  static __device__ __forceinline__ f32x4 mac(const W& w, const u32x4 (&x)[2], f32x4 acc) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc = mac_4x4(w.v[j].x, w.v[j].y, x[j / 2][j % 2 * 2], x[j / 2][j % 2 * 2 + 1], acc);
    return acc;
  }
};

// The four values that a (or b, c, d) has in lanes l%16 + 16*i, added: lane l
// gets those of a, b, c or d by l/16.
__device__ __forceinline__ float sum_rows(float a, float b, float c, float d) {
  const u32x2 ac = permlane32_swap(__float_as_uint(a), __float_as_uint(c));
  const u32x2 bd = permlane32_swap(__float_as_uint(b), __float_as_uint(d));
  const float p = __uint_as_float(ac.x) + __uint_as_float(ac.y), q = __uint_as_float(bd.x) + __uint_as_float(bd.y);
  const u32x2 r = permlane16_swap(__float_as_uint(p), __float_as_uint(q));
  return __uint_as_float(r.x) + __uint_as_float(r.y);
}

// The same for experts with up to four slots, in two groups of four columns: of
// h, and of what bf16 left of it.
constexpr int kOnce = 2;  // non-temporal: data that no other read wants
constexpr int kDppRowRor4 = 0x124, kDppRowRor8 = 0x128;  // lane l of 16 reads lane l - 4 or l - 8, cyclically
template <class D, int RT, int NW, int U, class Find>
__device__ __forceinline__ void few_down_lines(const uint8_t* h, uint64_t h_bytes, uint32_t rest, int inter,
                                              int w_rows, const BlockRows& by, int base, int first, int items,
                                               int bits, Find find) {
  constexpr int RG = 4 * RT, XV = D::kXLoads, kStep = D::kStep;
  const int lane = threadIdx.x % kWave, column = lane % 4, block = lane / 4;
  const uint32_t w_row = uint32_t(inter) * D::kWSize, nowhere = 0x80000000u;
  const __amdgpu_buffer_rsrc_t rows = buffer_of(h, h_bytes);
  const int steps = (inter + kStep - 1) / kStep;
  struct Walk {
    DownItem i;
    int at, s, end;
  };
  auto turn = [&](Walk& k) {  // to the next item; at >= items when there is none
    do k.at += NW;
    while (k.at < items && !find(k.at, k.i));
    k.s = steps * k.i.part >> bits;
    k.end = steps * (k.i.part + 1) >> bits;
  };
  Walk ask{}, form;
  ask.at = first - NW;
  turn(ask);
  if (ask.at >= items) return;
  form = ask;
  uint32_t w_lane[RG], x_lane[2];
#pragma unroll
  for (int q = 0; q < RG; ++q) w_lane[q] = uint32_t(4 * q + column) * w_row + block * 16;
  auto columns = [&] {  // of the item asked for
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      x_lane[g] = nowhere;
      if (column < ask.i.n)
        x_lane[g] = uint32_t(ask.i.list[column]) * uint32_t(inter * 2) + g * rest + block * (16 * XV);
    }
  };
  columns();
  // A lane's sums are of its own piece of k, in one block of it: a scale for either block of rows.
  typedef float Scales[U][2];
  auto request = [&](u32x4(&w)[U][RG], u32x4(&x)[U][2][XV], Scales& sc) {
    const bool live = ask.at < items;
    const __amdgpu_buffer_rsrc_t from = buffer_of(uniform(ask.i.w), uint64_t(w_rows) * w_row);
    const int s0 = uniform(ask.s);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = s0 + u;
      uint32_t out = live && s < ask.end && s * kStep + block * (16 / D::kWSize) < inter ? 0u : nowhere;
      asm("" : "+v"(out));
      if constexpr (D::kBlocks) {
        const uint32_t k_blocks = blocks_of(inter);
        const __amdgpu_buffer_rsrc_t from_s =
            buffer_of(uniform(reinterpret_cast<const uint8_t*>(ask.i.scales)), uint64_t(by.rows) * k_blocks * 4);
#pragma unroll
        for (int b = 0; b < 2; ++b)
          sc[u][b] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
              from_s, (uint32_t(block / 8 * 4) | out) + b * k_blocks * 4 + 8 * u, s0 * 8, 0));
      }
#pragma unroll
      for (int q = 0; q < RG; ++q)
        w[u][q] = __builtin_amdgcn_raw_buffer_load_b128(from, (w_lane[q] | out) + 256 * u, s0 * 256, kOnce);
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int v = 0; v < XV; ++v)
          x[u][g][v] = __builtin_amdgcn_raw_buffer_load_b128(rows, (x_lane[g] | out) + 2 * kStep * u + 16 * v,
                                                             s0 * 2 * kStep, 0);
    }
    ask.s += U;
    if (live && ask.s >= ask.end) {
      turn(ask);
      if (ask.at < items) columns();
    }
  };
  f32x4 acc[RG][2];
  auto clear = [&] {
#pragma unroll
    for (int q = 0; q < RG; ++q) acc[q][0] = acc[q][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  };
  clear();
  auto products = [&](const u32x4(&w)[U][RG], const u32x4(&x)[U][2][XV], const Scales& sc) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int q = 0; q < RG; ++q) {
        const typename D::W wq = D::weights(w[u][q]);
        if constexpr (D::kBlocks) {
          const float scale = by.of(4 * q) ? sc[u][1] : sc[u][0];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const f32x4 part = D::mac(wq, x[u][g], f32x4{});
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[q][g][i] = __builtin_fmaf(part[i], scale, acc[q][g][i]);
          }
        } else {
          acc[q][0] = D::mac(wq, x[u][0], acc[q][0]);
          acc[q][1] = D::mac(wq, x[u][1], acc[q][1]);
        }
      }
    form.s += U;
    if (form.at < items && form.s >= form.end) {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        f32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float t[2];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            t[g] = sum_rows(acc[4 * r][g][i], acc[4 * r + 1][g][i], acc[4 * r + 2][g][i], acc[4 * r + 3][g][i]);
            t[g] += __uint_as_float(dpp<kDppRowRor4, 0xF>(__float_as_uint(t[g])));
            t[g] += __uint_as_float(dpp<kDppRowRor8, 0xF>(__float_as_uint(t[g])));
          }
          v[i] = t[0] + t[1];
        }
        if (block % 4 == 0 && column < form.i.n)
          form.i.y[((int(form.i.list[column]) - base) * RT + r) * 4 + lane / 16] = v;
      }
      clear();
      turn(form);
    }
  };
  u32x4 w0[U][RG], w1[U][RG], x0[U][2][XV], x1[U][2][XV];
  Scales c0, c1;
  request(w0, x0, c0);
  request(w1, x1, c1);
  while (form.at < items) {
    products(w0, x0, c0);
    request(w0, x0, c0);
    products(w1, x1, c1);
    request(w1, x1, c1);
  }
}

// s_y (dynamic LDS): parts x chunk slots x 16*RT channels of fp32.  Slots are
// taken `chunk` at a time, a whole number of tokens; with more than one chunk
// an expert's weights are read for each that has a slot on it.
template <class D, int RT, bool kScaled, typename IdT>
__global__ __launch_bounds__(kDownWaves* kWave, 2) void k_few_down(
    const uint8_t* __restrict__ h, int n_rows, int hidden, int top_k, const IdT* __restrict__ ids,
    const float* __restrict__ router_weights, PadMask pad, int n_experts, const uint8_t* __restrict__ w,
    const float* __restrict__ w_scales, int inter, int channels, int chunk, int max_parts,
    uint16_t* __restrict__ out) {
  extern __shared__ f32x4 s_y[];
  __shared__ uint32_t s_count[1024];  // slots per expert, then their first place in s_list
  __shared__ uint16_t s_list[down_slots(RT)];
  __shared__ int16_t s_of[down_slots(RT)];  // a slot's expert, -1: none
  __shared__ float s_weight[down_slots(RT)];
  __shared__ uint16_t s_expert[1024], s_start[1025];  // active experts
  __shared__ uint32_t s_scan[kDownWaves];
  __shared__ int s_forms;  // which of the forms below have an expert
  typedef typename D::Core C;
  constexpr int NW = kDownWaves, kThreads = NW * kWave, kQuads = 4 * RT;
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int all = n_rows * top_k, routed_end = real_slots(pad, n_rows, top_k);
  const int c0 = blockIdx.x * channels, w_rows = min(channels, hidden - c0);
  const int second_at = kBlock - c0 % kBlock;
  const BlockRows by{nullptr, second_at, w_rows > second_at ? 2 : 1};
  constexpr int kBatch = 64 / (C::kWBytes * RT);  // steps: 4 KB of weights a wave
  for (int base = 0; base < all; base += chunk) {
    const int end = min(base + chunk, all), slots = min(end, routed_end);
    constexpr int kOwn = down_slots(RT) / kThreads;
    for (int e = tid; e < n_experts; e += kThreads) s_count[e] = 0;
    if (tid == 0) s_forms = 0;
    __syncthreads();
    int own_e[kOwn];
    uint32_t own_rank[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int slot = base + tid + i * kThreads;
      own_e[i] = slot < slots ? expert_of(ids, slot, n_experts) : -1;
      if (slot < end) {
        s_of[slot - base] = int16_t(own_e[i]);
        s_weight[slot - base] = router_weights[slot];
      }
      if (own_e[i] >= 0) own_rank[i] = atomicAdd(&s_count[own_e[i]], 1u);
    }
    __syncthreads();
    // Each lane scans two experts: slots in the low half, active experts in the high.
    const uint32_t n0 = 2 * tid < n_experts ? s_count[2 * tid] : 0u;
    const uint32_t n1 = 2 * tid + 1 < n_experts ? s_count[2 * tid + 1] : 0u;
    const int lines = inter < kLinesMin ? 0 : 4;  // slots of an expert up to which whole lines are read
    auto form_of = [&](int n) { return n == 0 ? 0 : n <= lines ? 1 : n <= 8 ? 2 : n <= 16 ? 4 : 8; };
    if (const int f = form_of(n0) | form_of(n1); f != 0) atomicOr(&s_forms, f);
    const uint32_t v0 = n0 | (n0 != 0 ? 0x10000u : 0u), v1 = n1 | (n1 != 0 ? 0x10000u : 0u);
    const uint32_t sum = wave_inclusive_sum(v0 + v1);
    if (lane == kWave - 1) s_scan[wave] = sum;
    __syncthreads();
    uint32_t before = sum - v0 - v1, total = 0;
    for (int i = 0; i < NW; ++i) {
      if (i < wave) before += s_scan[i];
      total += s_scan[i];
    }
    const int active = uniform(int(total >> 16)), routed = int(total & 0xFFFFu);
    if (n0 != 0) {
      s_expert[before >> 16] = uint16_t(2 * tid);
      s_start[before >> 16] = uint16_t(before);
    }
    if (n1 != 0) {
      s_expert[(before + v0) >> 16] = uint16_t(2 * tid + 1);
      s_start[(before + v0) >> 16] = uint16_t(before + v0);
    }
    if (tid == 0) s_start[active] = uint16_t(routed);
    if (2 * tid < n_experts) s_count[2 * tid] = before & 0xFFFFu;
    if (2 * tid + 1 < n_experts) s_count[2 * tid + 1] = (before + v0) & 0xFFFFu;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      if (own_e[i] >= 0) s_list[s_count[own_e[i]] + own_rank[i]] = uint16_t(base + tid + i * kThreads);
    __syncthreads();

    // With fewer experts than waves, k is split so that every wave has work.  Every part has a step; with block scales,
    // whose parts are whole blocks, some may have none and give zeros.
    int bits = 0;  // of the number of parts
    while ((2 << bits) <= max_parts && (2 << bits) * kStreamStep <= inter && (active << bits) < 2 * NW) ++bits;
    const int parts = 1 << bits;
    auto item_of = [&](int item, DownItem& i) {
      const int a = item >> bits, p = item & (parts - 1);
      const int first = uniform(s_start[a]);
      i.n = uniform(s_start[a + 1]) - first;
      i.list = s_list + first;
      i.w = w + (int64_t(uniform(s_expert[a])) * hidden + c0) * inter * (C::kWBytes / 16);
      if constexpr (D::kBlocks)
        i.scales = w_scales + (int64_t(uniform(s_expert[a])) * blocks_of(hidden) + c0 / kBlock) * blocks_of(inter);
      i.y = s_y + p * chunk * kQuads;
      i.part = p;
    };
    const uint32_t rest = uint32_t(all) * inter * 2;
    const uint64_t h_bytes = uint64_t(all) * inter * 4;
    const int forms = uniform(s_forms);
    if (forms & 1)
      few_down_lines<D, RT, NW, 2 / RT>(h, h_bytes, rest, inter, w_rows, by, base, uniform(wave), active * parts, bits,
                                        [&](int item, DownItem& i) {
                                          item_of(item, i);
                                          return i.n <= lines;
                                        });
    if (forms & 2)
      few_down_stream<D, RT, NW, kBatch, false>(h, h_bytes, rest, inter, w_rows, by, base, uniform(wave), active * parts,
                                                bits, [&](int item, DownItem& i) {
                                                  item_of(item, i);
                                                  return i.n > lines && i.n <= 8;
                                                });
    if (forms & 4)
      few_down_stream<D, RT, NW, kBatch, true>(h, h_bytes, rest, inter, w_rows, by, base, uniform(wave), active * parts,
                                               bits, [&](int item, DownItem& i) {
                                                 item_of(item, i);
                                                 return i.n > 8 && i.n <= 16;
                                               });
    for (int item = uniform(wave); (forms & 8) && item < active * parts; item += NW) {  // more than 16 slots
      DownItem i;
      item_of(item, i);
      if (i.n <= 16) continue;
      int begin, end;
      step_range(inter, i.part, parts, begin, end);
      for (int j = 0; j < i.n; j += 32)
        few_down_tile<D, RT, 2, 2>(h, rest, inter, i.w, w_rows, BlockRows{i.scales, by.second_at, by.rows}, i.list + j,
                                   min(i.n - j, 32), begin, end, base, i.y);
    }
    __syncthreads();

    for (int i = tid; i < (end - base) / top_k * kQuads; i += kThreads) {
      const int t = base / top_k + i / kQuads, quad = i % kQuads, c = c0 + quad * 4;
      if (quad * 4 >= w_rows) continue;
      float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      const int from = i / kQuads * top_k;
      constexpr int kAhead = kScaled ? 4 : 1;  // choices whose scales are requested together
      for (int first = 0; first < top_k; first += kAhead) {
        f32x4 scale[kAhead];
        if constexpr (kScaled)
#pragma unroll
          for (int j = 0; j < kAhead; ++j)
            scale[j] = *reinterpret_cast<const f32x4*>(
                w_scales + int64_t(max(int(s_of[from + min(first + j, top_k - 1)]), 0)) * hidden + c);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int slot = from + first + j;
          if (first + j >= top_k || s_of[slot] < 0) continue;
          f32x4 y = s_y[slot * kQuads + quad];
          for (int p = 1; p < parts; ++p) {
            const f32x4 v = s_y[(p * chunk + slot) * kQuads + quad];
#pragma unroll
            for (int q = 0; q < 4; ++q) y[q] += v[q];
          }
          const float rw = s_weight[slot];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if constexpr (kScaled) y[q] *= scale[j][q];
            o[q] += rw * y[q];
          }
        }
      }
      *reinterpret_cast<u32x2*>(out + int64_t(t) * hidden + c) = u32x2{bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3])};
    }
    __syncthreads();  // the lists and s_y are written again for the next slots
  }
}

namespace {

template <class Up, class D, bool kScaled, typename IdT>
hipError_t go(const FewLayer<IdT>& p, hipStream_t s) {
  const int slots = p.n_rows * p.top_k;
  const bool by_slot = slots < p.n_experts;
  const uint32_t strips = (p.inter + kUpChannels - 1) / kUpChannels, groups = by_slot ? slots : p.n_experts;
#define MOE_GO(KERNEL, ...)                                                                                        \
  hipLaunchKernelGGL((KERNEL<__VA_ARGS__, kScaled, IdT>), grid, dim3(kUpThreads), 0, s, reinterpret_cast<const uint8_t*>(p.x), \
                     p.n_rows, p.hidden, p.top_k, p.ids, p.pad, p.n_experts, by_slot,                              \
                     static_cast<const uint8_t*>(p.w_gate_up), p.gate_up_scales, p.inter, p.h)
  if (strips * groups >= uint32_t(kUpStripsMin)) {
    const dim3 grid(strips, groups);
    MOE_GO(k_few_up, Up);
  } else {
    const dim3 grid(p.inter / 16, groups);
    MOE_GO(k_few_up_split, Up, typename D::Core);
  }
#undef MOE_GO
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  const int channels = std::min((p.hidden / 4 + kDownGroups - 1) / kDownGroups * 4, 32);
  const int most = down_slots(channels > 16 ? 2 : 1);
  // Room for the results of the slots of a chunk, and for several parts of k while that stays within 512 slots' room.
  const int chunk = slots <= most ? slots : most / p.top_k * p.top_k;
  int max_parts = 1;
  while (max_parts < 8 && max_parts * 2 * chunk <= 512) max_parts *= 2;
  const size_t lds = size_t(max_parts) * chunk * 16 * sizeof(float);
#define MOE_GO(RT)                                                                                                  \
  hipLaunchKernelGGL((k_few_down<D, RT, kScaled, IdT>), dim3((p.hidden + channels - 1) / channels),                 \
                     dim3(kDownWaves * kWave), lds * RT, s, reinterpret_cast<const uint8_t*>(p.h), p.n_rows,        \
                     p.hidden, p.top_k, p.ids, p.router_weights, p.pad, p.n_experts, static_cast<const uint8_t*>(p.w_down),   \
                     p.down_scales, p.inter, channels, chunk, max_parts, p.out)
  if (channels > 16) MOE_GO(2);
  else MOE_GO(1);
#undef MOE_GO
  return hipGetLastError();
}

}  // namespace

template <typename IdT>
hipError_t launch_layer_few(const FewLayer<IdT>& p, hipStream_t s) {
  if (p.n_rows == 0) return hipSuccess;
  if (p.f8) return go<UpF8, DownF8, false, IdT>(p, s);
  return p.gate_up_scales != nullptr ? go<UpI8, DownI8, true, IdT>(p, s) : go<UpBf16, DownBf16, false, IdT>(p, s);
}

template hipError_t launch_layer_few<int32_t>(const FewLayer<int32_t>&, hipStream_t);
template hipError_t launch_layer_few<int64_t>(const FewLayer<int64_t>&, hipStream_t);

}  // namespace moe
