// Device helpers of the products that fill LDS by direct loads: loads that go
// past the registers, their waits, and fragments of the matrix core's operands.
#pragma once

#include "common.h"

namespace bsq {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

// Buffer resource of `records` bytes (in range 0 .. 2^32 - 1) from `base`;
// reads past it give zeros.
__device__ __forceinline__ i32x4 rsrc(const uint8_t* base, int64_t records) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  const uint32_t n = uint32_t(records < 0 ? 0 : (records > int64_t(0xFFFFFFFF) ? int64_t(0xFFFFFFFF) : records));
  return i32x4{__builtin_amdgcn_readfirstlane(int(uint32_t(b))),
               __builtin_amdgcn_readfirstlane(int(uint32_t(b >> 32) & 0xFFFFu)),
               __builtin_amdgcn_readfirstlane(int(n)), 0x00020000};
}

// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t scalar(int64_t v) {
  return int64_t(uint64_t(uint32_t(scalar(int(v)))) | (uint64_t(uint32_t(scalar(int(v >> 32)))) << 32));
}
__device__ __forceinline__ const uint8_t* scalar(const uint8_t* v) {
  return reinterpret_cast<const uint8_t*>(scalar(reinterpret_cast<int64_t>(v)));
}

// 16 bytes per lane straight into LDS: lane i fills [lds + 16 i, + 16).  In
// inline asm, so that the compiler does not order it against the reads of
// the other stage; the caller waits with vmcnt before the barrier that
// publishes the stage.  No register is written.  The compiler does not know
// what these are, so the waits that the hardware leaves to software are in
// them: one state from m0 to its use, five from a descriptor that a vector
// instruction may have written.
__device__ __forceinline__ void dma16(const uint8_t* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(lds), "v"(p) : "memory");
}
__device__ __forceinline__ void dma16(i32x4 r, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(scalar(int(lds))), "v"(voff), "s"(r)
               : "memory");
}
// 4 bytes per lane: lane i fills [lds + 4 i, + 4).
__device__ __forceinline__ void dma4(i32x4 r, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :
               : "s"(scalar(int(lds))), "v"(voff), "s"(r)
               : "memory");
}
// From a 32-bit offset to a base in scalar registers, to `at` (a constant
// where it is inlined) past lds.
__device__ __forceinline__ void dma16(const uint8_t* base, uint32_t off, uint32_t lds, int at) {
  asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(lds), "v"(off), "s"(base), "i"(at)
               : "memory", "scc");
}

// The same, to be dropped from the L2 first.
__device__ __forceinline__ void dma16_stream(const uint8_t* base, uint32_t off, uint32_t lds, int at) {
  asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt"
               :
               : "s"(lds), "v"(off), "s"(base), "i"(at)
               : "memory", "scc");
}

// s_waitcnt's operand: at most n vector memory operations under way.
constexpr int vmcnt(int n) { return (n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14); }
// A barrier that no access of the compiler's moves across.
__device__ __forceinline__ void barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ uint32_t lds_of(const uint8_t* p) {
  return __builtin_amdgcn_readfirstlane(
      uint32_t(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) uint8_t*)(p))));
}

__device__ __forceinline__ v8i frag(const uint8_t* tile, int off0, int off1) {
  const uint4 lo = *reinterpret_cast<const uint4*>(tile + off0);
  const uint4 hi = *reinterpret_cast<const uint4*>(tile + off1);
  return v8i{int(lo.x), int(lo.y), int(lo.z), int(lo.w), int(hi.x), int(hi.y), int(hi.z), int(hi.w)};
}

}  // namespace bsq
