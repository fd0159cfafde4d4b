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
typedef u32x4 u32x4_e4 __attribute__((aligned(4)));

#define LDS_PTR __attribute__((address_space(3)))
#define GLOBAL_PTR __attribute__((address_space(1)))

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

// E neighbouring elements (4 or 8) as they lie in memory.  Loads that should be on their way together
// are made by raw_word, which has no branch: a row's end moves the place, within the row as long as it
// has E elements at all, else to a place of its own (after a load that may or may not have been made,
// the wait for an earlier one is a wait for all).  open_word reads a row's last few elements one by
// one.
template <int DT, int E>
struct Raw {
  u32x4 a, b;
};

[[maybe_unused]] __device__ const uint32_t kElsewhere[8] = {};

template <int DT, int E>
__device__ __forceinline__ Raw<DT, E> raw_word(const void *p, int64_t row_at, int64_t first, int64_t cols) {
  Raw<DT, E> r = {};
  uint64_t at = reinterpret_cast<uint64_t>(p) + (uint64_t)(row_at + min(first, cols - E)) * (DT == 0 ? 4 : 2);
  at = cols >= E ? at : reinterpret_cast<uint64_t>(kElsewhere);
  if constexpr (DT == 0) {
    const GLOBAL_PTR u32x4_e4 *q = reinterpret_cast<const GLOBAL_PTR u32x4_e4 *>(at);
    r.a = q[0];
    if constexpr (E == 8) r.b = q[1];
  } else if constexpr (E == 8) {
    r.a = *reinterpret_cast<const GLOBAL_PTR u32x4_e2 *>(at);
  } else {
    const u32x2 v = *reinterpret_cast<const GLOBAL_PTR u32x2_e2 *>(at);
    r.a.x = v.x;
    r.a.y = v.y;
  }
  return r;
}

// The elements of raw_word(p, row_at, first, cols), zeros past the row's end.
template <int DT, int E>
__device__ __forceinline__ void open_word(const Raw<DT, E> &r, const void *p, int64_t row_at, int64_t first,
                                          int64_t cols, float (&x)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) {
    if constexpr (DT == 0)
      x[i] = __uint_as_float(i < 4 ? r.a[i & 3] : r.b[i & 3]);
    else
      x[i] = __uint_as_float(i & 1 ? r.a[i >> 1] & 0xFFFF0000u : r.a[i >> 1] << 16);
  }
  if (first + E > cols) {
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = first + i < cols ? load_one<DT>(p, row_at + first + i) : 0.0f;
  }
}

}  // namespace
}  // namespace gq
