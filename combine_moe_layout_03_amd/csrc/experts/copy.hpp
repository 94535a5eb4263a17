// Copies from memory to LDS that pass no registers, bounded by a buffer
// descriptor: what lies past the descriptor's end arrives as zeros.
#pragma once

#include "experts.hpp"

namespace moe {

typedef int ex_i32x4 __attribute__((ext_vector_type(4)));

// Wave-uniform values, moved to scalar registers.
__device__ __forceinline__ int scalar_i(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ uint64_t scalar_u64(uint64_t v) {
  return (uint64_t)(uint32_t)scalar_i((int)(uint32_t)v) |
         (uint64_t)(uint32_t)scalar_i((int)(uint32_t)(v >> 32)) << 32;
}

// Offset of a lane whose bytes are to arrive as zeros: past every descriptor.
constexpr uint32_t kOutside = 0xffffffffu;

// The `left` bytes (at most 2^32 - 32 of them; none if left <= 0) from `base`.
__device__ __forceinline__ ex_i32x4 buffer_at(uint64_t base, int64_t left) {
  const uint32_t n = left <= 0 ? 0u : left > 0xffffffe0ll ? 0xffffffe0u : (uint32_t)left;
  return ex_i32x4{(int)(uint32_t)base, (int)((uint32_t)(base >> 32) & 0xffffu), (int)n, 0x00020000};
}

// Copies 16 bytes per lane from byte `off` of the buffer to LDS at byte `to` +
// 16 * lane. Written in asm because the compiler, not knowing which LDS bytes a
// copy in flight writes, would wait for all copies before any LDS read; callers
// count them. No register is written, so nothing can be reused too early.
__device__ __forceinline__ void copy16_bounded(ex_i32x4 buf, uint32_t off, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(scalar_i((int)to)), "v"(off), "s"(buf) : "memory", "m0");
}
// The same to LDS byte `to` + kMore, in one instruction less.
template <int kMore>
__device__ __forceinline__ void copy16_bounded(ex_i32x4 buf, uint32_t off, uint32_t to) {
  asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(scalar_i((int)to)), "v"(off), "s"(buf), "i"(kMore) : "memory", "m0", "scc");
}
// The same for bytes that nobody reads again: marked to leave L2 first.
__device__ __forceinline__ void copy16_bounded_once(ex_i32x4 buf, uint32_t off, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds"
               :: "s"(scalar_i((int)to)), "v"(off), "s"(buf) : "memory", "m0");
}

__device__ __forceinline__ uint32_t lds_offset(const void *p) {  // address of a shared object
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}

}  // namespace moe
