// The cut of a call with many requests, worked out once, ahead of the attention kernel.
//
// Up to kScanRequests the attention's blocks do this themselves: one or two reads per lane. Beyond, the
// reads of all lengths in every block cost more than this kernel and a search in what it writes (one row
// each, bf16, all kernels, every block for itself against this: 256 requests of up to 1024 tokens, 8 kv heads
// 139, 129 us; 1024 of them 602, 463; 4096 of up to 256 tokens, 4 kv heads 1826, 495; at 128 requests of up to
// 2048 tokens this would add 6 us to 113).
// One thread a request; every block sums the work of all requests itself, in the same order.
#pragma once

#include "verify_attention.h"

namespace verify {

constexpr int kCutThreads = 1024;
constexpr int kCutWaves = kCutThreads / 64;

__global__ void __launch_bounds__(kCutThreads) attn_cut_kernel(verify_attention_args a, AttnLaunch p) {
  __shared__ float works[kCutWaves];
  __shared__ int befores[kCutWaves], owns[kCutWaves];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int group = a.heads / a.kv_heads, first = blockIdx.x * kCutThreads;
  float work = 0;
  for (int b = threadIdx.x; b < a.n_requests; b += kCutThreads) work += attn_work(p, attn_request(a, b), group);
  work = wave_sum(work);
  if (lane == 0) works[wave] = work;
  __syncthreads();
  work = 0;
#pragma unroll
  for (int w = 0; w < kCutWaves; ++w) work += works[w];
  const unsigned chunk = attn_chunk(a, p, work);

  int before = 0, parts = 0, mbs;
  for (int b = threadIdx.x; b < first; b += kCutThreads)
    before += attn_blocks(a, p, attn_request(a, b), group, chunk, &parts, &mbs);
  const int b = first + static_cast<int>(threadIdx.x);
  const int blocks = b < a.n_requests ? attn_blocks(a, p, attn_request(a, b), group, chunk, &parts, &mbs) : 0;
  before = wave_scan(before, lane);
  const int scan = wave_scan(blocks, lane);
  if (lane == 63) befores[wave] = before, owns[wave] = scan;
  __syncthreads();
  int base = scan - blocks;
#pragma unroll
  for (int w = 0; w < kCutWaves; ++w) base += befores[w] + (w < wave ? owns[w] : 0);
  if (b < a.n_requests) {
    p.plan[2 * b] = base;
    p.plan[2 * b + 1] = parts;
  }
}

inline hipError_t launch_attn_cut(const verify_attention_args& a, const AttnLaunch& p, hipStream_t stream) {
  attn_cut_kernel<<<dim3((a.n_requests + kCutThreads - 1) / kCutThreads), kCutThreads, 0, stream>>>(a, p);
  return hipGetLastError();
}

}  // namespace verify
