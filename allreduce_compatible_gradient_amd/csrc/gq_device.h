// gq_device.h -- what the matrix kernels share on the device: vector types, loads of eight
// neighbouring elements of either type, rounding to bf16, the draws of stochastic rounding.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// rows of an odd length start at any element: vectors that need no more than its alignment
typedef u32x4 u32x4_e2 __attribute__((aligned(2)));
typedef u32x2 u32x2_e2 __attribute__((aligned(2)));
typedef f32x4 f32x4_e4 __attribute__((aligned(4)));

#define LDS_PTR __attribute__((address_space(3)))

// Between writes of a wave's lanes to its own part of LDS and other lanes' reads of them, and back.
// The hardware executes a wave's LDS accesses in order; the fences keep the compiler from moving
// them across (the barrier alone is nothing to memory), and cost no instruction.
__device__ __forceinline__ void wave_exchange() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// MurmurHash3's 32-bit finaliser of (counter XOR key), its first step already applied to the key.
__device__ __forceinline__ uint32_t draw(uint32_t counter, uint32_t key_mix) {
  uint32_t h = (counter ^ (counter >> 16)) ^ key_mix;
  h *= 0x85EBCA6Bu;
  h ^= h >> 13;
  h *= 0xC2B2AE35u;
  return h ^ (h >> 16);
}

template <int DT>
__device__ __forceinline__ float load_one(const void *p, int64_t i) {
  if constexpr (DT == 0)
    return static_cast<const float *>(p)[i];
  else
    return __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[i] << 16);
}

// Eight consecutive elements at any element's alignment.
template <int DT>
__device__ __forceinline__ void load_eight(const void *p, int64_t i, float (&x)[8]) {
  if constexpr (DT == 0) {
    const f32x4_e4 *q = reinterpret_cast<const f32x4_e4 *>(static_cast<const float *>(p) + i);
    const f32x4 a = q[0], b = q[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = a[j];
      x[4 + j] = b[j];
    }
  } else {
    const u32x4 a = *reinterpret_cast<const u32x4_e2 *>(static_cast<const uint16_t *>(p) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(a[j] << 16);
      x[2 * j + 1] = __uint_as_float(a[j] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ uint16_t to_bf16(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x40u);
  return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Two fp32 rounded to bf16 (nearest even) in one word, the first in its low half.
__device__ __forceinline__ uint32_t to_bf16_pair(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// Eight elements of a row from `first` on, zeros past its end.
template <int DT>
__device__ __forceinline__ void load_word(const void *x, int64_t row_at, int64_t first, int64_t cols,
                                          float (&v)[8]) {
  if (first + 8 <= cols) {
    load_eight<DT>(x, row_at + first, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = first + i < cols ? load_one<DT>(x, row_at + first + i) : 0.0f;
  }
}

__device__ __forceinline__ uint32_t top_of(const float (&x)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  return top;
}

}  // namespace
}  // namespace gq
