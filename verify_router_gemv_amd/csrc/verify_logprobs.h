// Log probabilities of given tokens, entropy and top alternatives of each row of logits, in one read.
//
// Per lane, online over its elements, in powers of two (t = x log2 e - M, M the lane's running maximum):
//   l = sum 2^t,  e = sum 2^t t;   raising M by s:  e <- 2^-s (e - s l),  l <- 2^-s l.
// At the end z = ln 2 (M + log2 l) and the entropy is ln 2 (log2 l - e / l).
// The top alternatives ride along: a wave keeps its best K in the registers of its first K lanes, sorted,
// and looks at a chunk's elements again only when some lane's maximum (known already) beats the K-th;
// the wave then takes the chunk's best elements out one by one, largest first, so a chunk costs at most K
// insertions, and a random row about K ln(n / K) in all.
//
// All rows' chunks of 1024 logits form one sequence that is cut evenly over the waves the chip holds (a
// chunk is not cut: a wave's second chunk costs 2.5 us with 8 alternatives, its list in the second kernel
// less), so every wave reads the same amount whatever the rows and the vocabulary are; a wave that crosses
// from one row into the next writes a part per row, and a second kernel joins each row's parts.
// Bound: memory from a few dozen rows of 10^5 logits (a 16-bit row is near the vector rate too, about
// twelve issue slots an element); below, launch, load and insertion latency.
// Measured, first kernel + join: 2048 rows of 131072 bf16, 1 alternative, 98 + 4.9 us (5.5 TB/s; with 8
// alternatives 112 + 4.9); 24 rows of 151001 bf16, 8 alternatives, 9.8 + 7.4; one row of 248000 fp32, 8
// alternatives, 6.4 + 6.8 (4.3 + 2.5 without).
#pragma once

#include "verify_common.h"

namespace verify {

constexpr int kLpThreads = 256;
constexpr int kLpWaves = kLpThreads / 64;
constexpr int kLpChunk = 1024;      // logits per wave step: 16 a lane
constexpr int kLpEach = kLpChunk / 64;
// Waves a SIMD holds at the kernel's registers, by the element's size.
constexpr int lp_waves(int size) { return size == 4 ? 5 : 6; }
constexpr int kTop = VERIFY_MAX_ALTERNATIVES;
static_assert(kTop <= 16, "the list lies in one 16-lane row");
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLpNegInf = -__builtin_inff();

// Running statistics of a lane.
struct LpStat {
  float m, l, e;  // reference (in powers of two), sums
};

// The lanes' statistics as one; every lane gets it.
__device__ __forceinline__ LpStat lp_wave(LpStat s) {
  const float m = wave_max(s.m);
  const float ref = m == kLpNegInf ? 0.0f : m;
  const float d = s.m == kLpNegInf ? 0.0f : s.m - ref;  // a lane that saw nothing: sums 0 (or NaN)
  const float f = __builtin_amdgcn_exp2f(d);
  return {m, wave_sum(s.l * f), wave_sum(f == 0 ? 0.0f : f * (s.e + d * s.l))};
}

// Two lanes' statistics as one.
__device__ __forceinline__ LpStat lp_join(LpStat a, LpStat b) {
  const float m = fmaxf(a.m, b.m);
  const float ref = m == kLpNegInf ? 0.0f : m;
  const float da = a.m == kLpNegInf ? 0.0f : a.m - ref, db = b.m == kLpNegInf ? 0.0f : b.m - ref;
  const float fa = __builtin_amdgcn_exp2f(da), fb = __builtin_amdgcn_exp2f(db);
  return {m, a.l * fa + b.l * fb, (fa == 0 ? 0.0f : fa * (a.e + da * a.l)) + (fb == 0 ? 0.0f : fb * (b.e + db * b.l))};
}

// Logits as signed integers of the same order, equal exactly where the logits are equal (-0 and 0); NaN is
// below them all.
constexpr int kLpNone = INT32_MIN;
__device__ __forceinline__ int lp_key(float x) {
  const int b = __builtin_bit_cast(int, x + 0.0f);
  return x == x ? b ^ ((b >> 31) & 0x7fffffff) : kLpNone;
}
__device__ __forceinline__ float lp_unkey(int k) { return __builtin_bit_cast(float, k ^ ((k >> 31) & 0x7fffffff)); }

// The wave's best elements as keys, sorted: lane i < n holds the i-th; `cut` and `cut_id` are the K-th once
// n = K.
struct LpTop {
  int k = 0;
  int id = -1;
  int n = 0;
  int cut = kLpNone;
  int cut_id = -1;
};

// All but the lists are the same in every lane (scalars).
__device__ __forceinline__ void lp_insert(LpTop& top, int key, int id, int K, int lane) {
  // after everything larger, and after equal ones of lower id
  const bool before = (lane < top.n) & ((top.k > key) | ((top.k == key) & (top.id < id)));
  const int at = __popcll(__ballot(before));
  // every lane's left neighbour within its 16 lanes
  const int ku = static_cast<int>(moe::dpp_u32<0x111>(static_cast<uint32_t>(top.k)));
  const int iu = static_cast<int>(moe::dpp_u32<0x111>(static_cast<uint32_t>(top.id)));
  top.k = lane == at ? key : lane > at ? ku : top.k;
  top.id = lane == at ? id : lane > at ? iu : top.id;
  top.n = uniform(top.n < K ? top.n + 1 : K);
  if (top.n == K) {
    top.cut = __builtin_amdgcn_readlane(top.k, K - 1);
    top.cut_id = __builtin_amdgcn_readlane(top.id, K - 1);
  }
}
__device__ __forceinline__ bool lp_good(const LpTop& top, int key, int id, int K) {
  return top.n < K || key > top.cut || (key == top.cut && id < top.cut_id);
}

// The best K of one candidate per lane (key kLpNone: none), as a new list. Equal keys in ascending order of id.
__device__ __forceinline__ void lp_first(LpTop& top, int key, int id, int K, int lane) {
  for (int i = 0; i < K; ++i) {
    const int w = uniform(wave_max(key));
    if (w == kLpNone) break;
    const uint64_t who = __ballot(key == w);
    int from = __ffsll(static_cast<unsigned long long>(who)) - 1;
    int lo = __builtin_amdgcn_readlane(id, from);
    if (who & (who - 1)) {  // equal ones
      lo = ~uniform(wave_max(key == w ? ~id : INT32_MIN));
      from = __ffsll(static_cast<unsigned long long>(__ballot(key == w && id == lo))) - 1;
    }
    top.k = lane == i ? w : top.k;
    top.id = lane == i ? lo : top.id;
    key = lane == from ? kLpNone : key;
    top.n = i + 1;
  }
  if (top.n == K) {
    top.cut = __builtin_amdgcn_readlane(top.k, K - 1);
    top.cut_id = __builtin_amdgcn_readlane(top.id, K - 1);
  }
}

// Inserts the candidates of the lanes in `who` that are still good enough, one by one.
__device__ __forceinline__ void lp_each(LpTop& top, uint64_t who, int key, int id, int K, int lane) {
  while (who) {
    const int from = __ffsll(static_cast<unsigned long long>(who)) - 1;
    who &= who - 1;
    const int ck = __builtin_amdgcn_readlane(key, from), ci = __builtin_amdgcn_readlane(id, from);
    if (lp_good(top, ck, ci, K)) lp_insert(top, ck, ci, K, lane);
  }
}

// Element j of a lane in a chunk.
template <int VEC>
__device__ __forceinline__ int lp_place(int j, int lane) {
  return (j / VEC * 64 + lane) * VEC + j % VEC;
}

// Takes those of a chunk's elements that are among the best K: x the lanes' elements (NaN: none), best their
// largest, base the id of the chunk's first. Every lane offers its best element, then its second best, until
// none is good enough. With a list that is not full, or with many lanes that have something to offer, the
// first offers go as a list of their own: its K are a list already, or raise the cut, so that little is left
// to insert one by one, whatever the order of the row. (One loop, not one branch per element: the code is
// fetched anew in each launch, and sixteen skipped copies of the insertion cost more than the work.)
template <int VEC>
__device__ __forceinline__ void lp_take(LpTop& top, float (&x)[kLpEach], float best, int K, int lane, int base) {
  for (;;) {
    const int key = lp_key(best);
    int at = 0;  // the lane's first element that is its best
#pragma unroll
    for (int j = kLpEach - 1; j >= 0; --j) at = x[j] == best ? j : at;
    const int id = base + lp_place<VEC>(at, lane);
    uint64_t who = __ballot(key != kLpNone && lp_good(top, key, id, K));
    if (!who) break;
    int ok = key, oi = id;  // what is offered
    if (top.n < K || __popcll(who) > 4 + K) {
      LpTop mine;
      lp_first(mine, key, id, K, lane);
      ok = mine.k;
      oi = mine.id;
      who = (uint64_t(1) << mine.n) - 1;
      if (top.n == 0) {
        top = mine;
        who = 0;
      }
    }
    lp_each(top, who, ok, oi, K, lane);
    best = __builtin_nanf("");
#pragma unroll
    for (int j = 0; j < kLpEach; ++j) {
      x[j] = j == at ? __builtin_nanf("") : x[j];
      best = fmaxf(best, x[j]);
    }
  }
}

struct LpPlan {
  int32_t chunks;    // per row
  int64_t per_wave;  // chunks of a wave, of n_rows * chunks
  int64_t waves;
  float* stat;       // [waves + rows][3]: the part of wave w in row t lies at w + t
  int32_t* tk;       // [waves + rows][top] keys
  int32_t* ti;       // the same of ids
};

// Chunk 0 of a row starts at the row's last 16-byte boundary at or before its first element, so all loads
// but the row's edges are whole and aligned.
template <typename T>
__device__ __forceinline__ int lp_offset(const T* row) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads, lp_waves(sizeof(T))) logprobs_kernel(verify_logprobs_args a, LpPlan p) {
  constexpr int VEC = 16 / sizeof(T), U = kLpEach / VEC;  // logits of a load, loads of a chunk
  typedef T TV __attribute__((ext_vector_type(VEC)));
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kLpWaves + wave;
  const int64_t all = static_cast<int64_t>(a.n_rows) * p.chunks;
  const int64_t g0 = w * p.per_wave;
  const int64_t g1 = g0 + p.per_wave < all ? g0 + p.per_wave : all;
  if (g0 >= g1) return;
  const int V = a.vocab, K = a.top;

  TV buf[U];
  auto load = [&](int t, int c) {
    const T* const row = static_cast<const T*>(a.logits) + t * a.row_stride;
    const int first = c * kLpChunk - lp_offset(row);
    if (first >= 0 && first + kLpChunk <= V) {
      const T* const src = row + first;
#pragma unroll
      for (int u = 0; u < U; ++u) buf[u] = *reinterpret_cast<const TV*>(src + (u * 64 + lane) * VEC);
    } else {  // an edge of the row: element by element, from inside it
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const int i = first + (u * 64 + lane) * VEC + j;
          const T v = row[i < 0 ? 0 : i < V ? i : V - 1];
          buf[u][j] = i >= 0 && i < V ? v : static_cast<T>(kLpNegInf);
        }
    }
  };

  LpStat st{kLpNegInf, 0, 0};
  LpTop top;
  int t = static_cast<int>(g0 / p.chunks), c = static_cast<int>(g0 - static_cast<int64_t>(t) * p.chunks);
  load(t, c);
  for (int left = static_cast<int>(g1 - g0); left > 0; --left) {
    float x[kLpEach];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < VEC; ++j) x[u * VEC + j] = static_cast<float>(static_cast<T>(buf[u][j]));
    const int t0 = t, c0 = c;
    const bool row_ends = c + 1 == p.chunks;
    if (row_ends) c = 0, ++t;
    else ++c;
    if (left > 1) load(t, c);  // the next chunk is under way while this one is worked on
    float best = x[0];
#pragma unroll
    for (int j = 1; j < kLpEach; ++j) best = fmaxf(best, x[j]);
    const float m = fmaxf(st.m, best * kLog2e);
    if (m > st.m) {
      if (st.l != 0) {
        const float s = st.m - m, f = __builtin_amdgcn_exp2f(s);
        st.e = f == 0 ? 0.0f : f * (st.e + s * st.l);
        st.l *= f;
      }
      st.m = m;
    }
    const float ref = m == kLpNegInf ? 0.0f : m;
    float e = st.e;
#pragma unroll
    for (int j = 0; j < kLpEach; ++j) {
      const float s = fmaf(x[j], kLog2e, -ref);
      const float q = __builtin_amdgcn_exp2f(s);
      st.l += q;
      e = fmaf(q, s, e);
    }
    if (e != e) {  // a logit of -inf (0 times -inf) or a NaN: once more, as -inf adds nothing
      e = st.e;
#pragma unroll
      for (int j = 0; j < kLpEach; ++j) {
        const float s = fmaf(x[j], kLog2e, -ref);
        e = fmaf(__builtin_amdgcn_exp2f(s), fmaxf(s, -256.0f), e);
      }
    }
    st.e = e;
    if (K && __ballot(top.n < K || best > lp_unkey(top.cut))) {
      const T* const row = static_cast<const T*>(a.logits) + t0 * a.row_stride;
      const int base = c0 * kLpChunk - lp_offset(row);
      if (c0 == 0 || row_ends) {  // what lies outside the row is no element
        best = __builtin_nanf("");
#pragma unroll
        for (int j = 0; j < kLpEach; ++j) {
          const int id = base + lp_place<VEC>(j, lane);
          x[j] = id >= 0 && id < V ? x[j] : __builtin_nanf("");
          best = fmaxf(best, x[j]);
        }
      }
      lp_take<VEC>(top, x, best, K, lane, base);
    }
    if (row_ends || left == 1) {
      const LpStat s = lp_wave(st);
      const int64_t at = w + t0;
      if (lane == 0) {
        p.stat[3 * at] = s.m;
        p.stat[3 * at + 1] = s.l;
        p.stat[3 * at + 2] = s.e;
      }
      if (lane < K) {
        p.tk[at * K + lane] = lane < top.n ? top.k : kLpNone;
        p.ti[at * K + lane] = top.id;
      }
      st = LpStat{kLpNegInf, 0, 0};
      top = LpTop{};
    }
  }
}

// One block a row, of a wave per 64 parts up to kJoinWaves; the first wave joins what the waves found.
constexpr int kJoinWaves = 4;
static_assert(kJoinWaves * kTop <= 64, "their lists' entries lie in one wave");

template <typename T>
__global__ void __launch_bounds__(64 * kJoinWaves) logprobs_join_kernel(verify_logprobs_args a, LpPlan p) {
  __shared__ LpStat stats[kJoinWaves];
  __shared__ int keys[kJoinWaves * kTop], ids[kJoinWaves * kTop];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int t = blockIdx.x, K = a.top;
  const T* const row = static_cast<const T*>(a.logits) + t * a.row_stride;
  // The given tokens' logits, asked for first.
  const int64_t tok0 = static_cast<int64_t>(t) * a.n_tokens;
  auto token = [&](int n) {
    return a.tokens_64 ? static_cast<const int64_t*>(a.tokens)[tok0 + n]
                       : static_cast<int64_t>(static_cast<const int32_t*>(a.tokens)[tok0 + n]);
  };
  int64_t id0 = -1;
  float x0 = 0;
  if (wave == 0 && lane < a.n_tokens) {
    id0 = token(lane);
    if (id0 >= 0 && id0 < a.vocab) x0 = static_cast<float>(row[id0]);
  }

  // The row's parts: of the waves from the one that has its first chunk to the one that has its last.
  const int64_t w0 = static_cast<int64_t>(t) * p.chunks / p.per_wave;
  const int64_t w1 = (static_cast<int64_t>(t + 1) * p.chunks - 1) / p.per_wave;
  const int parts = static_cast<int>(w1 - w0 + 1);
  const int64_t at0 = w0 + t;
  LpStat st{kLpNegInf, 0, 0};
  const bool flat = waves == 1 && parts * K <= 64;  // the lists' entries, one a lane
  int fk = kLpNone, fid = -1;
  if (flat && lane < parts * K) {
    fk = p.tk[at0 * K + lane];
    fid = p.ti[at0 * K + lane];
  }
  for (int i = 64 * wave + lane; i < parts; i += 64 * waves)
    st = lp_join(st, LpStat{p.stat[3 * (at0 + i)], p.stat[3 * (at0 + i) + 1], p.stat[3 * (at0 + i) + 2]});
  LpTop top;
  if (flat) {
    if (K) lp_first(top, fk, fid, K, lane);
  } else {
    // The lists are sorted: the best of each first, then the second best, until none is good enough. All of
    // 64 lists are asked for at once.
    for (int i0 = 64 * wave; i0 < parts && K; i0 += 64 * waves) {
      const int i = i0 + lane;
      int k[kTop], id[kTop];
#pragma unroll
      for (int r = 0; r < kTop; ++r) {
        k[r] = kLpNone, id[r] = -1;
        if (r < K && i < parts) {
          k[r] = p.tk[(at0 + i) * K + r];
          id[r] = p.ti[(at0 + i) * K + r];
        }
      }
      const bool first = i0 == 64 * wave;
      if (first) lp_first(top, k[0], id[0], K, lane);
      for (int r = first; r < K; ++r) {
        if (r) {  // the next of each list, to the front
#pragma unroll
          for (int q = 0; q + 1 < kTop; ++q) k[q] = k[q + 1], id[q] = id[q + 1];
        }
        const uint64_t who = __ballot(k[0] != kLpNone && lp_good(top, k[0], id[0], K));
        if (!who) break;
        lp_each(top, who, k[0], id[0], K, lane);
      }
    }
  }
  st = lp_wave(st);
  if (waves > 1) {
    if (lane == 0) stats[wave] = st;
    if (lane < kTop) {
      keys[wave * kTop + lane] = lane < top.n ? top.k : kLpNone;
      ids[wave * kTop + lane] = top.id;
    }
    __syncthreads();
    if (wave) return;
    st = lp_wave(lane < waves ? stats[lane] : LpStat{kLpNegInf, 0, 0});
    top = LpTop{};
    const int at = lane < waves * kTop ? lane : 0;
    if (K) lp_first(top, lane < waves * kTop ? keys[at] : kLpNone, ids[at], K, lane);
  }

  const float lg = __builtin_amdgcn_logf(st.l);  // log2
  const bool none = st.m == kLpNegInf && st.l == 0;  // every logit is -inf
  const float z = kLn2 * (st.m + lg);
  for (int n = lane; n < a.n_tokens; n += 64) {
    if (n != lane) {
      id0 = token(n);
      if (id0 >= 0 && id0 < a.vocab) x0 = static_cast<float>(row[id0]);
    }
    a.logprobs[tok0 + n] = none || id0 < 0 || id0 >= a.vocab ? kLpNegInf : x0 - z;
  }
  if (a.entropy && lane == 0) a.entropy[t] = none ? 0.0f : kLn2 * (lg - st.e / st.l);
  if (lane < K) {
    const int64_t at = static_cast<int64_t>(t) * K + lane;
    const bool there = lane < top.n;
    a.top_ids[at] = there ? top.id : -1;
    a.top_logprobs[at] = !there ? __builtin_nanf("") : none ? kLpNegInf : lp_unkey(top.k) - z;
  }
}

// The cut of the rows into waves, and the workspace for the parts.
inline LpPlan lp_plan(const verify_logprobs_args& a, void* workspace, int64_t* bytes) {
  LpPlan p{};
  const int vec = a.type == VERIFY_F32 ? 4 : 8;
  p.chunks = static_cast<int32_t>((static_cast<int64_t>(a.vocab) + vec - 1 + kLpChunk - 1) / kLpChunk);
  const int64_t all = static_cast<int64_t>(a.n_rows) * p.chunks;
  const int64_t resident = 256 * 4 * lp_waves(a.type == VERIFY_F32 ? 4 : 2);
  p.per_wave = (all + resident - 1) / resident;
  p.waves = (all + p.per_wave - 1) / p.per_wave;
  const int64_t parts = p.waves + a.n_rows;
  *bytes = parts * (12 + 8 * a.top);
  p.stat = static_cast<float*>(workspace);
  p.tk = reinterpret_cast<int32_t*>(p.stat + 3 * parts);
  p.ti = p.tk + parts * a.top;
  return p;
}

template <typename T>
hipError_t launch_logprobs_t(const verify_logprobs_args& a, const LpPlan& p, hipStream_t stream) {
  logprobs_kernel<T><<<dim3(static_cast<unsigned>((p.waves + kLpWaves - 1) / kLpWaves)), kLpThreads, 0, stream>>>(a, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t parts = (p.chunks - 1) / p.per_wave + 2;  // of a row, at most
  const int waves = static_cast<int>(parts >= 64 * kJoinWaves ? kJoinWaves : (parts + 63) / 64);
  logprobs_join_kernel<T><<<dim3(a.n_rows), 64 * waves, 0, stream>>>(a, p);
  return hipGetLastError();
}

inline hipError_t launch_logprobs(const verify_logprobs_args& a, const LpPlan& p, hipStream_t stream) {
  if (a.type == VERIFY_F32) return launch_logprobs_t<float>(a, p, stream);
  if (a.type == VERIFY_BF16) return launch_logprobs_t<__bf16>(a, p, stream);
  return launch_logprobs_t<_Float16>(a, p, stream);
}

}  // namespace verify
