// Block table, slot map, positions and tree masks of a round, in one launch.
//
// Everything follows from two prefix sums over the requests (rows, and pages to take).  B is small
// (hundreds of requests, 8 B each), so every block sums the requests before its own four itself, 256
// threads at a time: that read hits the L2 and costs less than a second launch or a wait between
// blocks.  A wave then owns one request (several past thousands): its pages and rows are written lane by lane
// (coalesced), and grid.y waves share a request whose rows are many.  A request's tree (up to 64 rows) lies in one wave:
// lane i holds row i's parent, and six rounds of pointer doubling over lane shuffles give every row its
// ancestors' bits and depth, instead of a walk of up to 63 dependent loads.
// Bound: latency (a few dependent loads) up to some 10^5 rows, then the writes.  Measured: 8 requests with
// trees of up to 8 rows 4.2 us; 1000 prompts of up to 1025 rows, all pages new, 9.1 us (6.6 MB read and written).
#pragma once

#include "verify_common.h"

namespace verify {

constexpr int kSlotThreads = 256;
constexpr int kSlotWaves = kSlotThreads / 64;

__device__ __forceinline__ int slot_pages(int64_t tokens, int P, int W) {
  const int64_t n = (tokens + P - 1) / P;
  return n < W ? static_cast<int>(n) : W;
}

// The slots, positions and masks of request b, whose rows and new pages begin at `rows` and `pages`.
__device__ __forceinline__ void slots_request(const verify_slots_args& a, int b, int64_t rows, int64_t pages, int64_t step,
                                              int lane) {
  const int64_t N = a.total_rows;
  const int P = a.page_size, W = a.width;
  const int c = max0(a.cached[b]), r = max0(a.rows[b]);
  const int old = slot_pages(c, P, W);
  const int need = slot_pages(static_cast<int64_t>(c) + r, P, W) - old;
  int32_t* const row = a.table + b * a.table_stride;
  const int64_t head = (a.free_head ? *a.free_head : 0) + pages;  // list place of the request's first new page
  auto fresh = [&](int64_t j) {
    const int64_t at = head + j;
    return at >= 0 && at < a.n_free ? a.free_pages[at] : -1;
  };
  const int64_t first = static_cast<int64_t>(blockIdx.y) * 64 + lane;
  if (first == 0) a.row_start[b] = static_cast<int32_t>(rows < N ? rows : N);
  for (int64_t j = first; j < need; j += step) row[old + j] = fresh(j);

  auto slot = [&](int64_t index) {
    const int64_t col = index / P;
    if (col >= W) return -1;
    const int page = col < old ? row[col] : fresh(col - old);
    const int64_t s = static_cast<int64_t>(page) * P + index % P;
    return page < 0 || s > INT32_MAX ? -1 : static_cast<int>(s);
  };
  if (!a.parents) {
    for (int64_t i = first; i < r && rows + i < N; i += step) {
      const int64_t index = c + i;
      a.slots[rows + i] = slot(index);
      a.positions[rows + i] = static_cast<int32_t>(index < INT32_MAX ? index : INT32_MAX);
    }
    return;
  }
  if (blockIdx.y == 0) {  // the tree's rows: row i in lane i
    const bool mine = lane < r && rows + lane < N;
    int up = mine ? a.parents[rows + lane] : -1;
    if (up < 0 || up >= lane) up = -1;
    uint64_t mask = uint64_t(1) << lane;
    int depth = up >= 0;
#pragma unroll
    for (int s = 0; s < 6; ++s) {
      const int from = up >= 0 ? up : lane;
      const uint64_t m = __shfl(mask, from);
      const int d = __shfl(depth, from), u = __shfl(up, from);
      if (up >= 0) {
        mask |= m;
        depth += d;
        up = u;
      }
    }
    if (mine) {
      a.slots[rows + lane] = slot(static_cast<int64_t>(c) + lane);
      a.positions[rows + lane] = min(c, INT32_MAX - depth) + depth;
      a.masks[rows + lane] = static_cast<int64_t>(mask);
    }
  }
  for (int64_t i = 64 + first; i < r && rows + i < N; i += step) {
    a.slots[rows + i] = -1;
    a.positions[rows + i] = c;
    a.masks[rows + i] = 0;
  }
}

__global__ void __launch_bounds__(kSlotThreads) slots_kernel(verify_slots_args a, int each) {
  __shared__ int64_t part[kSlotWaves][2];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int B = a.n_requests, P = a.page_size, W = a.width;
  const int own = kSlotWaves * each, groups = (B + own - 1) / own;
  const int g = blockIdx.x;  // the last one writes the totals and the padding
  const bool last = g == groups;
  const int before = last ? B : g * own;

  int64_t rows = 0, pages = 0;
  auto count = [&](int b) {
    const int64_t c = max0(a.cached[b]), r = max0(a.rows[b]);
    rows += r;
    pages += slot_pages(c + r, P, W) - slot_pages(c, P, W);
  };
  for (int b = threadIdx.x; b < before; b += kSlotThreads) count(b);
  rows = wave_sum64(rows);
  pages = wave_sum64(pages);
  if (lane == 0) part[wave][0] = rows, part[wave][1] = pages;
  __syncthreads();
  rows = pages = 0;
#pragma unroll
  for (int w = 0; w < kSlotWaves; ++w) rows += part[w][0], pages += part[w][1];

  const int64_t N = a.total_rows;
  const int64_t step = static_cast<int64_t>(gridDim.y) * 64;
  if (last) {
    const int64_t id = (static_cast<int64_t>(blockIdx.y) * kSlotWaves + wave) * 64 + lane;
    for (int64_t t = rows + id; t < N; t += step * kSlotWaves) {
      a.slots[t] = -1;
      a.positions[t] = 0;
      if (a.masks) a.masks[t] = 0;
    }
    if (id == 0) {
      a.row_start[B] = static_cast<int32_t>(rows < N ? rows : N);
      a.counts[0] = static_cast<int32_t>(rows < INT32_MAX ? rows : INT32_MAX);
      a.counts[1] = static_cast<int32_t>(pages < INT32_MAX ? pages : INT32_MAX);
    }
    return;
  }

  const int mine = g * own + wave * each;
  if (mine >= B) return;
  for (int b = g * own; b < mine; ++b) count(b);  // the block's own earlier requests
  slots_request(a, mine, rows, pages, step, lane);
  for (int b = mine + 1; b < min(mine + each, B); ++b) {
    count(b - 1);
    slots_request(a, b, rows, pages, step, lane);
  }
}

// grid.y: enough waves that an average request's rows take a wave a few rounds, not more. From 4096 requests on
// a wave takes several, as the number of blocks and the sums in each grow with the requests (calls of
// 4095, 4096 and 65536 requests of one row: 11.5, 11.4, 145 us; 65536 with one a wave 774).
inline hipError_t launch_slots(const verify_slots_args& a, hipStream_t stream) {
  const int each = a.n_requests / 4096 + 1;
  const int groups = (a.n_requests + kSlotWaves * each - 1) / (kSlotWaves * each);
  const int64_t per = static_cast<int64_t>(a.total_rows) / (groups ? a.n_requests : 1) / 256 + 1;
  const unsigned y = per < 256 ? static_cast<unsigned>(per) : 256u;
  slots_kernel<<<dim3(groups + 1, y), kSlotThreads, 0, stream>>>(a, each);
  return hipGetLastError();
}

}  // namespace verify
