// Device helpers of the attention kernels (gfx950).
#pragma once

#include "device_common.h"

namespace misa {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2 lds_i32x2;
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Softmax reference of a row that has seen no key: finite, so that a masked
// score (-inf) minus it is -inf and weighs 0, and below every score.
constexpr float kNoMax = -3.0e38f;
// A row's reference is raised when a score passes it by this much (in powers
// of two): weights stay below 2^8 and the accumulated sums are rescaled in few
// tiles only. The reference cancels in the quotient, so results do not change
// beyond fp32 rounding.
constexpr float kSlack = 8.0f;

// Starts a copy of 16 bytes a lane from global memory to LDS at lds + 16 * lane
// (lds: wave-uniform byte address). It counts in vmcnt and is waited for with
// wait_copies() before the barrier that hands the tile over; written as one
// instruction here because the compiler would otherwise wait for every copy in
// flight before any LDS read. No vector register is written, so nothing can be
// overwritten while it is in flight; M0 is set where it is used, and nothing
// else in these kernels reads it.
__device__ __forceinline__ void copy16_to_lds(const void* src, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, off"
      :
      : "s"(lds), "v"(src)
      : "memory");
}
__device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Workgroup barrier that waits for this wave's LDS accesses only (copies to
// LDS stay in flight).
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <typename Tp>
__device__ __forceinline__ uint32_t lds_addr(Tp* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) Tp*)p;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_fast(float x) { return __builtin_amdgcn_logf(x); }

// Maximum / sum over the four lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float max_over_groups(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, kWave));
  return fmaxf(v, __shfl_xor(v, 32, kWave));
}
__device__ __forceinline__ float sum_over_groups(float v) {
  v += __shfl_xor(v, 16, kWave);
  return v + __shfl_xor(v, 32, kWave);
}

// Eight E4M3FN codes -> eight bf16 values (exact).
__device__ __forceinline__ bf16x8 codes_to_bf16(u32x2 v) {
  u32x4 r;
  r.x = fp8x2_to_bf16x2<false>(v.x);
  r.y = fp8x2_to_bf16x2<true>(v.x);
  r.z = fp8x2_to_bf16x2<false>(v.y);
  r.w = fp8x2_to_bf16x2<true>(v.y);
  return __builtin_bit_cast(bf16x8, r);
}

// Keys 0 .. pos of a prefix of `left` keys (0 for pos < 0).
__device__ __forceinline__ int visible_keys(int pos, int left) { return pos < 0 ? 0 : (pos < left ? pos + 1 : left); }

// A tile whose keys are not the same for all rows of a wave: a value that is
// not finite must reach the rows that see its key and no other, but weight 0
// times infinity or NaN is NaN in a matrix product. Operands without such
// values (the normal case) are used as they are.
__device__ __forceinline__ bool any_odd(bf16x8 a) {
  const u32x4 v = __builtin_bit_cast(u32x4, a);
  bool odd = false;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    odd |= (v[i] & 0x7f80u) == 0x7f80u || (v[i] & 0x7f800000u) == 0x7f800000u;
  return odd;
}
// The values of an operand that are (ODD) or are not infinite or NaN; of the
// first kind only element `keep`, or none if it is negative.
template <bool ODD>
__device__ __forceinline__ bf16x8 part_of(bf16x8 a, int keep) {
  const u32x4 v = __builtin_bit_cast(u32x4, a);
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool o0 = (v[i] & 0x7f80u) == 0x7f80u, o1 = (v[i] & 0x7f800000u) == 0x7f800000u;
    const bool k0 = ODD ? (o0 && keep == 2 * i) : !o0, k1 = ODD ? (o1 && keep == 2 * i + 1) : !o1;
    r[i] = (k0 ? v[i] & 0xffffu : 0u) | (k1 ? v[i] & 0xffff0000u : 0u);
  }
  return __builtin_bit_cast(bf16x8, r);
}

}  // namespace misa
