// Small device helpers shared by the head product, the scoring kernels and
// the gradient clip.
#ifndef MARKOV_NUMBERS_H_
#define MARKOV_NUMBERS_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float bf_one(uint16_t w) { return __uint_as_float((uint32_t)w << 16); }

// Two binary32 -> one word of two bf16 (nearest, ties to even), `a` low.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){a, b}, bf16x2_t));
}

__host__ __device__ __forceinline__ bool aligned_to(const void* p, uintptr_t n) {
  return ((uintptr_t)p & (n - 1)) == 0;
}

// A workgroup barrier after which the LDS writes of every wave before it are
// seen, and those of its asynchronous loads but for each wave's latest N memory
// operations (which leave their count in order). A __syncthreads would wait for
// all of them.
template <int N>
__device__ __forceinline__ void barrier_but() {
  static_assert(N >= 0 && N < 16, "");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | N);   // vmcnt(N) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace

#endif  // MARKOV_NUMBERS_H_
