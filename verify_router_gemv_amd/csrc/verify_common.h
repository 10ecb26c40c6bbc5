// Shared device helpers of the verify-round operators (gfx950, wave64).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "moe_common.h"
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

// The word of lane ^ 16 (X = 16) or lane ^ 32 beside the lane's own, in either order.
template <int X>
__device__ __forceinline__ float2 across(float v) {
  const uint32_t w = __builtin_bit_cast(uint32_t, v);
  uint32_t a, b;  // scalars: a bit cast of a vector's element would read its first element
  if constexpr (X == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    a = r[0], b = r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    a = r[0], b = r[1];
  }
  return make_float2(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}
// Reductions over the wave on the vector ALUs; every lane gets the result. Maxima skip NaN.
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, moe::dpp_f32<moe::kDppXor1>(v));
  v = fmaxf(v, moe::dpp_f32<moe::kDppXor2>(v));
  v = fmaxf(v, moe::dpp_f32<moe::kDppHalfMirror>(v));
  v = fmaxf(v, moe::dpp_f32<moe::kDppMirror>(v));
  float2 a = across<16>(v);
  a = across<32>(fmaxf(a.x, a.y));
  return fmaxf(a.x, a.y);
}
__device__ __forceinline__ float wave_sum(float v) {
  v += moe::dpp_f32<moe::kDppXor1>(v);
  v += moe::dpp_f32<moe::kDppXor2>(v);
  v += moe::dpp_f32<moe::kDppHalfMirror>(v);
  v += moe::dpp_f32<moe::kDppMirror>(v);
  float2 a = across<16>(v);
  a = across<32>(a.x + a.y);
  return a.x + a.y;
}
__device__ __forceinline__ int wave_max(int v) {
  v = max(v, static_cast<int>(moe::dpp_u32<moe::kDppXor1>(v)));
  v = max(v, static_cast<int>(moe::dpp_u32<moe::kDppXor2>(v)));
  v = max(v, static_cast<int>(moe::dpp_u32<moe::kDppHalfMirror>(v)));
  v = max(v, static_cast<int>(moe::dpp_u32<moe::kDppMirror>(v)));
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(static_cast<int>(a[0]), static_cast<int>(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(static_cast<int>(b[0]), static_cast<int>(b[1]));
}

__device__ __forceinline__ int max0(int v) { return v > 0 ? v : 0; }

}  // namespace verify
