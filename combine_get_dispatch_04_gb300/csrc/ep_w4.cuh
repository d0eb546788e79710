// ep_w4.cuh -- what the kernels that multiply 4-bit weights in registers share
// (ep_experts_w4.cu, ep_layer_w4.cu): the matrix instruction, the order of the
// channels within a step, and the layout of a step's codes in shared memory.
#pragma once

#include "ep_common.cuh"

namespace ep {

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// The B fragments of 8 channels: the pairs (0,4) (1,5) (2,6) (3,7).
__device__ __forceinline__ void pairs_bf16(const uint4& x, uint32_t (&b)[4]) {
  b[0] = __byte_perm(x.x, x.z, 0x5410);
  b[1] = __byte_perm(x.x, x.z, 0x7632);
  b[2] = __byte_perm(x.y, x.w, 0x5410);
  b[3] = __byte_perm(x.y, x.w, 0x7632);
}
// First channel, within a step, of word j (8 channels) of thread t of a quad:
// the t-th quarter of every 64 channels, or of every 32 where those have
// scales of their own.
template <int kGroup>
__device__ __forceinline__ int word_channel(int t, int j) {
  return kGroup == 32 ? j * 32 + t * 8 : (j >> 1) * 64 + t * 16 + (j & 1) * 8;
}

// The 16-byte chunks of a staged weight row are permuted by its place among
// eight rows, so that the loads of fragments meet no bank twice.
__device__ __forceinline__ int chunk_swizzle(int g) { return (g & 2) | (g >> 2 & 1); }

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
}  // namespace ep
