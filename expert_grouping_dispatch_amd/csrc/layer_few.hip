// The whole layer for a few tokens in two kernels.
//
// Both products read every active expert's weights once: 6*hidden*inter bytes
// per expert in bf16 (half in int8) against at most a few dozen rows of
// activations, so the layer is bound by how fast HBM delivers the weights.
// They go straight to registers (stream.h); grouping costs each workgroup one
// pass over the few ids instead of a kernel of its own.
//
//   k_few_up     one workgroup per (expert, 16 intermediate channels): lists the
//                expert's slots, forms gate and up for up to 64 slots at a time
//                with k split over the waves, joins the parts in LDS and writes
//                h = silu(gate)*up as bf16, the type the second product's
//                matrix instruction takes.
//   k_few_down   one workgroup per 16 output channels: groups all slots, its
//                waves take (expert, part of k) items, every slot's result goes
//                to its own place in LDS in fp32, and then each token's choices
//                are summed in ascending order, so the result does not depend on
//                which wave came first.
#include "experts.h"
#include "stream.h"

namespace moe {

namespace {

constexpr int kFewMaxSlots = 2048;
constexpr int kUpWaves = 4, kUpThreads = kUpWaves * kWave;
constexpr int kDownWaves = 8, kDownThreads = kDownWaves * kWave;
constexpr int kMaxGroups = 4;  // 16 slots each, per pass over the weights

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

// NG groups of 16 slots, list[0 .. n), n <= 16*NG.
template <class C, int NG, bool kScaled>
__device__ __forceinline__ void few_up_tile(const uint8_t* x, int hidden, int top_k, const uint8_t* w,
                                            const float* w_scales, int inter, int tile,
                                            const uint16_t* list, int n, uint16_t* h, f32x4* s_part) {
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
  stream_products<C, 2, NG, (NG == 1 ? 4 : NG == 2 ? 2 : 1)>(wp, xp, begin, end, hidden, acc);
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
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = silu_times(sum[0][i], sum[1][i]);
      *reinterpret_cast<u32x2*>(h + int64_t(list[at]) * inter + c) =
          u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    }
  }
  __syncthreads();  // s_part is rewritten for the next slots
}

// blockIdx.x: tile of 16 channels.  blockIdx.y: the expert, or, when there
// are fewer slots than experts, a slot, which stands for its expert if it is
// the first slot on it.
template <class C, bool kScaled, typename IdT>
__global__ __launch_bounds__(kUpThreads, 4) void k_few_up(const uint8_t* __restrict__ x, int n_rows, int hidden,
                                                       int top_k, const IdT* __restrict__ ids, PadMask pad,
                                                       int n_experts, bool by_slot,
                                                       const uint8_t* __restrict__ w,
                                                       const float* __restrict__ w_scales, int inter,
                                                       uint16_t* __restrict__ h) {
  __shared__ uint16_t s_list[kFewMaxSlots];
  __shared__ int s_n, s_earlier;
  __shared__ f32x4 s_part[kUpWaves * 2 * kMaxGroups * kWave];
  const int tid = threadIdx.x;
  const int slots = real_slots(pad, n_rows, top_k);
  if (tid == 0) s_n = s_earlier = 0;
  int e = blockIdx.y;
  if (by_slot) {
    if (e >= slots) return;
    e = expert_of(ids, e, n_experts);
    if (e < 0) return;
  }
  __syncthreads();
  for (int i = tid; i < slots; i += kUpThreads) {
    if (expert_of(ids, i, n_experts) == e) {
      if (by_slot && i < int(blockIdx.y)) s_earlier = 1;
      s_list[atomicAdd(&s_n, 1)] = uint16_t(i);  // any order: a slot's result does not depend on its column
    }
  }
  __syncthreads();
  if (s_earlier != 0) return;
  const int n = s_n;
  const uint8_t* we = w + int64_t(e) * 2 * inter * hidden * (C::kWBytes / 16);
  const float* se = kScaled ? w_scales + int64_t(e) * 2 * inter : nullptr;
  for (int c0 = 0; c0 < n; c0 += 16 * kMaxGroups) {
    const int m = min(n - c0, 16 * kMaxGroups);
    if (m <= 16)
      few_up_tile<C, 1, kScaled>(x, hidden, top_k, we, se, inter, blockIdx.x, s_list + c0, m, h, s_part);
    else if (m <= 32)
      few_up_tile<C, 2, kScaled>(x, hidden, top_k, we, se, inter, blockIdx.x, s_list + c0, m, h, s_part);
    else
      few_up_tile<C, 4, kScaled>(x, hidden, top_k, we, se, inter, blockIdx.x, s_list + c0, m, h, s_part);
  }
}

// ---- down and the weighted sum ------------------------------------------------

template <class C, int NG>
__device__ __forceinline__ void few_down_tile(const uint8_t* h, int inter, const uint8_t* w, int tile,
                                              const uint16_t* list, int n, int begin, int end, f32x4* s_y) {
  const int lane = threadIdx.x % kWave;
  const uint8_t* wp[1] = {w + int64_t(tile * 16 + lane % 16) * inter * (C::kWBytes / 16)};
  const uint8_t* hp[NG];
  f32x4 acc[1][NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    hp[g] = h + int64_t(list[min(g * 16 + lane % 16, n - 1)]) * inter * 2;
    acc[0][g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  stream_products<C, 1, NG, (NG == 1 ? 8 : NG == 2 ? 4 : 2)>(wp, hp, begin, end, inter, acc);
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int at = g * 16 + lane % 16;
    if (at < n) s_y[int(list[at]) * 4 + lane / 16] = acc[0][g];
  }
}

// s_y (dynamic LDS): parts x slots x 16 channels of fp32.
template <class C, bool kScaled, typename IdT>
__global__ __launch_bounds__(kDownThreads, 4) void k_few_down(
    const uint8_t* __restrict__ h, int n_rows, int hidden, int top_k, const IdT* __restrict__ ids,
    const float* __restrict__ router_weights, PadMask pad, int n_experts, const uint8_t* __restrict__ w,
    const float* __restrict__ w_scales, int inter, int max_parts, uint16_t* __restrict__ out) {
  extern __shared__ f32x4 s_y[];
  __shared__ uint32_t s_count[1024];  // slots per expert, then their first place in s_list
  __shared__ uint16_t s_list[kFewMaxSlots];
  __shared__ uint16_t s_expert[1024], s_start[1025];  // active experts
  __shared__ uint32_t s_scan[kDownWaves];
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int all = n_rows * top_k, slots = real_slots(pad, n_rows, top_k);
  constexpr int kOwn = kFewMaxSlots / kDownThreads;
  for (int e = tid; e < n_experts; e += kDownThreads) s_count[e] = 0;
  __syncthreads();
  int own_e[kOwn];
  uint32_t own_rank[kOwn];
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int slot = tid + i * kDownThreads;
    own_e[i] = slot < slots ? expert_of(ids, slot, n_experts) : -1;
    if (own_e[i] >= 0) own_rank[i] = atomicAdd(&s_count[own_e[i]], 1u);
  }
  __syncthreads();
  // Each lane scans two experts: slots in the low half, active experts in the high.
  uint32_t c0 = 2 * tid < n_experts ? s_count[2 * tid] : 0u;
  uint32_t c1 = 2 * tid + 1 < n_experts ? s_count[2 * tid + 1] : 0u;
  const uint32_t v0 = c0 | (c0 != 0 ? 0x10000u : 0u), v1 = c1 | (c1 != 0 ? 0x10000u : 0u);
  const uint32_t sum = wave_inclusive_sum(v0 + v1);
  if (lane == kWave - 1) s_scan[wave] = sum;
  __syncthreads();
  uint32_t base = sum - v0 - v1, total = 0;
  for (int i = 0; i < kDownWaves; ++i) {
    if (i < wave) base += s_scan[i];
    total += s_scan[i];
  }
  const int active = int(total >> 16), routed = int(total & 0xFFFFu);
  if (c0 != 0) {
    s_expert[base >> 16] = uint16_t(2 * tid);
    s_start[base >> 16] = uint16_t(base);
  }
  if (c1 != 0) {
    s_expert[(base + v0) >> 16] = uint16_t(2 * tid + 1);
    s_start[(base + v0) >> 16] = uint16_t(base + v0);
  }
  if (tid == 0) s_start[active] = uint16_t(routed);
  if (2 * tid < n_experts) s_count[2 * tid] = base & 0xFFFFu;
  if (2 * tid + 1 < n_experts) s_count[2 * tid + 1] = (base + v0) & 0xFFFFu;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kOwn; ++i)
    if (own_e[i] >= 0) s_list[s_count[own_e[i]] + own_rank[i]] = uint16_t(tid + i * kDownThreads);
  __syncthreads();

  // With fewer experts than waves, k is split so that every wave has work.
  int parts = 1;
  while (parts * 2 <= max_parts && parts * active < 2 * kDownWaves) parts *= 2;
  for (int item = wave; item < active * parts; item += kDownWaves) {
    const int a = item / parts, p = item - a * parts;
    const int first = s_start[a], n = int(s_start[a + 1]) - first;
    const uint8_t* we = w + int64_t(s_expert[a]) * hidden * inter * (C::kWBytes / 16);
    f32x4* y = s_y + int64_t(p) * all * 4;
    int begin, end;
    step_range(inter, p, parts, begin, end);
    for (int i = 0; i < n; i += 16 * kMaxGroups) {
      const int m = min(n - i, 16 * kMaxGroups);
      if (m <= 16) few_down_tile<C, 1>(h, inter, we, blockIdx.x, s_list + first + i, m, begin, end, y);
      else if (m <= 32) few_down_tile<C, 2>(h, inter, we, blockIdx.x, s_list + first + i, m, begin, end, y);
      else few_down_tile<C, 4>(h, inter, we, blockIdx.x, s_list + first + i, m, begin, end, y);
    }
  }
  __syncthreads();

  for (int i = tid; i < n_rows * 4; i += kDownThreads) {
    const int t = i / 4, quad = i % 4, c = blockIdx.x * 16 + quad * 4;
    float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j = 0; j < top_k; ++j) {
      const int slot = t * top_k + j;
      const int e = slot < slots ? expert_of(ids, slot, n_experts) : -1;
      if (e < 0) continue;
      f32x4 y = s_y[slot * 4 + quad];
      for (int p = 1; p < parts; ++p) {
        const f32x4 v = s_y[(p * all + slot) * 4 + quad];
#pragma unroll
        for (int q = 0; q < 4; ++q) y[q] += v[q];
      }
      const float rw = router_weights[slot];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (kScaled) y[q] *= w_scales[int64_t(e) * hidden + c + q];
        o[q] += rw * y[q];
      }
    }
    *reinterpret_cast<u32x2*>(out + int64_t(t) * hidden + c) = u32x2{bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3])};
  }
}

namespace {

template <class C, bool kScaled, typename IdT>
hipError_t go(const FewLayer<IdT>& p, hipStream_t s) {
  const int slots = p.n_rows * p.top_k;
  const bool by_slot = slots < p.n_experts;
  hipLaunchKernelGGL((k_few_up<C, kScaled, IdT>), dim3(p.inter / 16, by_slot ? slots : p.n_experts),
                     dim3(kUpThreads), 0, s, reinterpret_cast<const uint8_t*>(p.x), p.n_rows, p.hidden, p.top_k,
                     p.ids, p.pad, p.n_experts, by_slot, static_cast<const uint8_t*>(p.w_gate_up),
                     p.gate_up_scales, p.inter, p.h);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  // Room for the results of every slot, and for several parts of k while that stays within 512 slots' room.
  int max_parts = 1;
  while (max_parts < kDownWaves && max_parts * 2 * slots <= 512) max_parts *= 2;
  const size_t lds = size_t(max_parts) * slots * 16 * sizeof(float);
  hipLaunchKernelGGL((k_few_down<C, kScaled, IdT>), dim3(p.hidden / 16), dim3(kDownThreads), lds, s,
                     reinterpret_cast<const uint8_t*>(p.h), p.n_rows, p.hidden, p.top_k, p.ids, p.router_weights,
                     p.pad, p.n_experts, static_cast<const uint8_t*>(p.w_down), p.down_scales, p.inter, max_parts,
                     p.out);
  return hipGetLastError();
}

}  // namespace

template <typename IdT>
hipError_t launch_layer_few(const FewLayer<IdT>& p, hipStream_t s) {
  if (p.n_rows == 0) return hipSuccess;
  return p.gate_up_scales != nullptr ? go<CoreI8Bf16, true, IdT>(p, s) : go<CoreBf16, false, IdT>(p, s);
}

template hipError_t launch_layer_few<int32_t>(const FewLayer<int32_t>&, hipStream_t);
template hipError_t launch_layer_few<int64_t>(const FewLayer<int64_t>&, hipStream_t);

}  // namespace moe
