// Filling LDS straight from global memory, and the waits that go with it.
#pragma once

#include "experts.h"

namespace moe {

// A buffer of `bytes` bytes at `base`: reads past it give zeros, in registers
// and in LDS, away from memory.  What is compared with the size is the whole
// offset, the per-lane and the scalar part together, also where the scalar part
// alone is past it (seen on a buffer over the start of a larger allocation).
// No kernel reads further than 2^30 bytes from its base.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const uint8_t* base, uint64_t bytes) {
  const uint32_t size = bytes < (uint64_t(1) << 31) ? uint32_t(bytes) : 0x7FFFFFF0u;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, size, 0x00027000);
}

// 64 lanes x 16 bytes from `off` (per lane) + `at` to 1 KB of LDS at `dst`.
template <bool kNonTemporal = false>
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t from, uint32_t off, uint32_t at, uint8_t* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)(dst), 16, off, at, 0,
                                           kNonTemporal ? 2 : 0);
}

constexpr int kWaitLoads = 0x0F70;     // s_waitcnt vmcnt(0)
// s_waitcnt vmcnt(n), n <= 63
constexpr int wait_all_but(int n) { return 0x0F70 | (n & 15) | ((n >> 4) << 14); }
constexpr int kWaitLdsScalar = 0xC07F;  // s_waitcnt lgkmcnt(0)

}  // namespace moe
