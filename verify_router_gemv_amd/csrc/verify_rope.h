// RMS norm of each query and key head, the rotary position, and the cache write, in one pass.
//
// A head's D values lie in D / 8 lanes, eight each (one 16-byte load of 16-bit values), so the norm is
// a reduction over 8, 16 or 32 neighbouring lanes and the pair of value i in the half layout, i + R/2, is
// the same element of a lane R / 16 further: no shared memory but the row's angles.  A block of 256
// threads takes one row; its first R / 2 threads compute the angles while the heads' loads are under
// way.  Angle and reduction to a turn are float64 (position * inv_freq * 1/(2 pi), 53 bits: a position of
// 2^20 keeps its fraction of a turn to 2^-33), the sine and cosine of the remaining turn float32.  One
// rounding at the end, to the cache's type.
// Bound: memory from about a thousand rows, launch and two dependent load latencies below.  Measured: 8191
// rows of 16 + 2 heads of 256, fp16, 42 us (4.0 TB/s read and written); 64 rows of 32 + 8 heads of 128, fp32 in,
// 4.2; one row of 16 + 2 heads 3.2.
#pragma once

#include "verify_common.h"

namespace verify {

constexpr int kRopeThreads = 256;

__device__ __forceinline__ f32x8 load8(const float* p) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
  return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
__device__ __forceinline__ void store8(__bf16* p, f32x8 v) {
  *reinterpret_cast<bf16x8*>(p) = __builtin_convertvector(v, bf16x8);
}
__device__ __forceinline__ void store8(_Float16* p, f32x8 v) {
  *reinterpret_cast<f16x8*>(p) = __builtin_convertvector(v, f16x8);
}

template <typename T>
struct Raw8 {  // eight values as they lie in memory
  typedef T V __attribute__((ext_vector_type(8)));
  V v;
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (sizeof(T) == 4) {
      const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
      v = V{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    } else {
      v = *reinterpret_cast<const V*>(p);
    }
  }
  __device__ __forceinline__ f32x8 get() const { return __builtin_convertvector(v, f32x8); }
};

template <typename TI, typename TC, int D>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(verify_rope_args a) {
  constexpr int L = D / 8;                 // lanes per head
  constexpr int HB = kRopeThreads / L;     // heads per step of the block
  constexpr int U = 3;                     // steps whose heads are asked for at once
  __shared__ float2 turn[D / 2];
  const int t = blockIdx.x, l = threadIdx.x % L;
  const int items = a.heads + 2 * a.kv_heads;
  const int slot = a.slots[t];
  const int position = a.positions[t];
  const int half = a.n_freq;

  auto source = [&](int item) -> const TI* {
    if (item < a.heads) return static_cast<const TI*>(a.q) + t * a.q_row + item * a.q_head;
    item -= a.heads;
    if (item < a.kv_heads) return static_cast<const TI*>(a.k) + t * a.k_row + item * a.k_head;
    return static_cast<const TI*>(a.v) + t * a.v_row + (item - a.kv_heads) * a.v_head;
  };
  const int mine = threadIdx.x / L;
  Raw8<TI> x[U];
  auto ask = [&](int step) {  // a thread past the last head takes the last one again, and stores nothing
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int item = (step + u * static_cast<int>(gridDim.y)) * HB + mine;
      x[u].load(source(item < items ? item : items - 1) + 8 * l);
    }
  };
  int step = blockIdx.y;
  ask(step);
  f32x8 wq{}, wk{};
  if (a.q_weight) wq = load8(a.q_weight + 8 * l);
  if (a.k_weight) wk = load8(a.k_weight + 8 * l);
  if (static_cast<int>(threadIdx.x) < half) {
    const double angle = static_cast<double>(position) * static_cast<double>(a.inv_freq[threadIdx.x]);
    const double turns = angle * 0.15915494309189533577;  // 1 / (2 pi)
    float s, c;
    sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &s, &c);
    turn[threadIdx.x] = make_float2(c, s);
  }
  const int page = slot / a.page_size, place = slot - page * a.page_size;
  if (slot < 0 || page >= a.n_pages) return;  // the whole block
  __syncthreads();
  TC* const ko = static_cast<TC*>(a.k_cache) + page * a.kc_page + place * a.kc_token;
  TC* const vo = static_cast<TC*>(a.v_cache) + page * a.vc_page + place * a.vc_token;

  for (;;) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = (step + u * static_cast<int>(gridDim.y)) * HB;
      if (at >= items) break;  // uniform over the block
      const int item = at + mine;
      const bool is_q = item < a.heads, is_v = item >= a.heads + a.kv_heads;
      f32x8 y = x[u].get();
      if (item < items && is_v) store8(vo + (item - a.heads - a.kv_heads) * a.vc_head + 8 * l, y);
      float ss = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += y[j] * y[j];
      ss = moe::group_sum<L>(ss);
      if (is_q ? a.q_weight : a.k_weight) y *= (is_q ? wq : wk) * (1.0f / sqrtf(ss * (1.0f / D) + a.eps));
      f32x8 z = y;
      if (a.interleaved) {
        if (8 * l < 2 * half) {
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const float2 cs = turn[4 * l + j / 2];
            z[j] = y[j] * cs.x - y[j + 1] * cs.y;
            z[j + 1] = y[j + 1] * cs.x + y[j] * cs.y;
          }
        }
      } else {
        const int hop = half / 8;  // lanes to the other half of the pair
        const bool low = l < hop, in = l < 2 * hop;
        const int lane = threadIdx.x & 63;
        const int from = in ? (low ? lane + hop : lane - hop) : lane;
        f32x8 o;
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = __shfl(y[j], from);
        if (in) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 cs = turn[8 * (low ? l : l - hop) + j];
            z[j] = y[j] * cs.x + (low ? -o[j] : o[j]) * cs.y;
          }
        }
      }
      if (item < items && !is_v) {
        if (is_q) store8(static_cast<TC*>(a.q_out) + t * a.o_row + item * a.o_head + 8 * l, z);
        else store8(ko + (item - a.heads) * a.kc_head + 8 * l, z);
      }
    }
    step += U * gridDim.y;
    if (step * HB >= items) break;
    ask(step);
  }
}

// Rows alone fill the chip from 512 on; below, a row's heads are spread over blocks too, each of which
// computes the row's angles again (32 + 8 heads of 128, bf16, spread against one block a row: 64 rows 3.5, 4.4
// us; 256 4.8, 5.4; 512 7.1, 6.7; 4096 40, 26).
template <typename TI, typename TC, int D>
hipError_t launch_rope_t(const verify_rope_args& a, hipStream_t stream) {
  constexpr int HB = kRopeThreads / (D / 8);
  const int steps = (a.heads + 2 * a.kv_heads + HB - 1) / HB;
  rope_kernel<TI, TC, D><<<dim3(a.n_rows, a.n_rows < 512 ? steps : 1), kRopeThreads, 0, stream>>>(a);
  return hipGetLastError();
}

template <typename TI, typename TC>
hipError_t launch_rope_d(const verify_rope_args& a, hipStream_t stream) {
  switch (a.dim) {
    case 64: return launch_rope_t<TI, TC, 64>(a, stream);
    case 128: return launch_rope_t<TI, TC, 128>(a, stream);
    default: return launch_rope_t<TI, TC, 256>(a, stream);
  }
}

inline hipError_t launch_rope(const verify_rope_args& a, hipStream_t stream) {
  if (a.cache_type == VERIFY_BF16)
    return a.in_type == VERIFY_F32 ? launch_rope_d<float, __bf16>(a, stream) : launch_rope_d<__bf16, __bf16>(a, stream);
  return a.in_type == VERIFY_F32 ? launch_rope_d<float, _Float16>(a, stream)
                                 : launch_rope_d<_Float16, _Float16>(a, stream);
}

}  // namespace verify
