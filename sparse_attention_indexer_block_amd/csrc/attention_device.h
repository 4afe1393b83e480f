// Device helpers of the attention kernels (gfx950).
#pragma once

#include "device_common.h"

namespace misa {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2 lds_i32x2;
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Softmax reference of a row that has seen no key: the lowest finite number, so
// that a masked score (-inf) minus it is -inf and weighs 0, and no finite score is
// below it. (A reference of this size plus kSlack rounds to itself, so that any
// score but the lowest one raises it, and that one weighs 1 against it.)
constexpr float kNoMax = -0x1.fffffep127f;
// A row's reference is raised when a score passes it by this much (in powers
// of two): weights stay below 2^32, far inside fp32 and bf16 (and sums over n keys
// inside fp32 while n times the largest value is below 2^96), and the
// accumulated sums are rescaled in hardly any tile but the first (with 2^8 one
// of 32 rows passed it every few tiles). The reference cancels in the quotient,
// so results do not change beyond fp32 rounding. Each row's is raised by its own
// scores alone: a weight is rounded to bf16 against it, and a row's bits must not
// depend on the rows beside it.
constexpr float kSlack = 32.0f;

// Starts a copy of 16 bytes a lane from global memory to LDS at lds + 16 * lane
// (lds: wave-uniform byte address). It counts in vmcnt and is waited for with
// wait_copies() before the barrier that hands the tile over; written as one
// instruction here because the compiler would otherwise wait for every copy in
// flight before any LDS read. No vector register is written, so nothing can be
// overwritten while it is in flight. M0 is set where it is used and nothing else
// in these files touches it; the compiler reserves it and does not honour a
// clobber, so a test reads the generated code for that instead.
__device__ __forceinline__ void copy16_to_lds(const void* src, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, off"
      :
      : "s"(lds), "v"(src)
      : "memory");
}
// The same from base + off, base uniform over the wave. It may come from a lane
// read, after which a memory instruction would have to wait five states for it;
// a scalar move of it waits by itself.
__device__ __forceinline__ void copy16_to_lds_at(const void* base, uint32_t off, uint32_t lds) {
  const void* b;
  asm volatile(
      "s_mov_b64 %0, %3\n\t"
      "s_mov_b32 m0, %1\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %2, %0"
      : "=&s"(b)
      : "s"(lds), "v"(off), "s"(base)
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

// A row's total as it leaves a kernel: -0 says that the row has no keys (the weights of
// keys add up to +0 or more; +0 if they all score -inf).
__device__ __forceinline__ float row_total(bool has_keys, float total) { return has_keys ? total : -0.f; }
__device__ __forceinline__ bool no_keys(float total) { return __float_as_uint(total) == 0x80000000u; }
// What a row's sums are divided by its total with: a row without keys is zeros, and one
// whose keys all score -inf is 0 / 0 = NaN, here 0 times infinity.
__device__ __forceinline__ float row_inverse(float total) { return no_keys(total) ? 0.f : 1.f / total; }
// log sum exp of a row with reference m (in powers of two): -inf without keys, or if they all score -inf.
__device__ __forceinline__ float row_log_sum(float m, float total) {
  return no_keys(total) ? -INFINITY : (m + log2_fast(total)) * 0.6931471805599453f;
}

// The larger value, NaN if one is (fmaxf would first have every operand quieted by
// an instruction of its own). A row with a NaN score ends as NaN whatever its reference.
__device__ __forceinline__ float max_or_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// Values of lane l ^ 32 (and l ^ 16) exchanged in registers: with both operands
// the same, the two results hold the lower and the upper halves (odd and even
// rows of 16 lanes) for every lane.
__device__ __forceinline__ float max_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// Maximum / sum over the four lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float max_over_groups(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return max_halves(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float sum_over_groups(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return sum_halves(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// LDS reads at a byte address (and the transposing ones: 16 lanes read rows of
// 16 values, a lane gets one value of each row).
template <typename Tp>
__device__ __forceinline__ Tp lds_read(uint32_t at) {
  return *(const __attribute__((address_space(3))) Tp*)(uintptr_t)at;
}
__device__ __forceinline__ s16x4 lds_read_tr16(uint32_t at) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)at);
}
__device__ __forceinline__ u32x2 lds_read_tr8(uint32_t at) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2*)(uintptr_t)at));
}
__device__ __forceinline__ bf16x8 join_rows(s16x4 a, s16x4 b) {
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// The softmax scale as the kernels use it: positive (queries change sign with
// it) and not zero, so that a masked score (-inf) times it stays -inf. The
// smallest number, 2^-149, weighs all finite scores (below 2^128) alike to
// within 2^-21, as a scale of zero does.
__device__ __forceinline__ float scale_magnitude(float sm_log2) { return fmaxf(fabsf(sm_log2), 0x1p-149f); }
__device__ __forceinline__ bf16x8 flip_sign(bf16x8 a, uint32_t mask) {
  u32x4 v = __builtin_bit_cast(u32x4, a);
  v ^= mask;
  return __builtin_bit_cast(bf16x8, v);
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

// A 32x32x16 product with its accumulator in vector registers, for a kernel whose
// accumulation registers are all taken (the compiler's own choice is one kind
// for a whole kernel). The compiler does not know that the asm is an MFMA, so
// the waits it would insert stand here: two wait states after a vector
// instruction that wrote an operand, none for the same accumulator, and
// mfma_done() (16; 12 are required for this shape) before any other use of it.
__device__ __forceinline__ void mfma_vgpr_first(f32x16& d, bf16x8 a, bf16x8 b) {
  asm("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, 0" : "=&v"(d) : "v"(a), "v"(b));
}
__device__ __forceinline__ void mfma_vgpr(f32x16& d, bf16x8 a, bf16x8 b) {
  asm("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+v"(d) : "v"(a), "v"(b));
}
__device__ __forceinline__ void mfma_done(f32x16& d) { asm volatile("s_nop 15" : "+v"(d)); }

// The same value, taken anew: what is derived from it is formed where it is
// used, instead of once before the loop and kept in registers.
template <typename Tp>
__device__ __forceinline__ Tp anew(Tp x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Keeps an accumulator in the accumulation registers on both sides of this
// point: at the entry of a rare branch that changes it, the copies that the
// change needs stay in the branch.
__device__ __forceinline__ void in_agprs(f32x16& d) { asm volatile("" : "+a"(d)); }

// In a tile whose keys are not the same for all rows of a wave a value that is
// not finite must reach the rows that see its key and no other, but weight 0
// times infinity or NaN is NaN in a matrix product.
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
