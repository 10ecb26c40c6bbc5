// Shared device helpers of the verify-round operators (gfx950, wave64).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "verify_ops.h"

namespace verify {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// The same word of every lane, as a scalar.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ int64_t wave_sum64(int64_t v) {
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) v += __shfl_xor(v, s);
  return v;
}

// Inclusive prefix sum over the wave.
__device__ __forceinline__ int64_t wave_scan64(int64_t v, int lane) {
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const int64_t up = __shfl_up(v, s);
    if (lane >= s) v += up;
  }
  return v;
}

__device__ __forceinline__ int max0(int v) { return v > 0 ? v : 0; }

}  // namespace verify
