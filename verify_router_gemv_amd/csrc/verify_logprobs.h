// Log probabilities of given tokens, entropy and top alternatives of each row of logits, in one read.
//
// Per lane, online over its elements, in powers of two (t = x log2 e - M, M the lane's running maximum):
//   l = sum 2^t,  e = sum 2^t t;   raising M by s:  e <- 2^-s (e - s l),  l <- 2^-s l.
// At the end z = ln 2 (M + log2 l) and the entropy is ln 2 (log2 l - e / l).
// The top alternatives ride along: a wave keeps its best K in the registers of its first K lanes, sorted,
// and looks at a chunk's elements again only when some lane's maximum (known already) beats the K-th;
// the wave then takes the chunk's best elements out one by one, largest first, so a chunk costs at most K
// insertions, and a random row about K ln(n / K) in all.
// Rows are cut over blocks while there are fewer rows than the chip has room for; a second kernel joins
// the parts. With enough rows, one block takes a whole row and joins its waves itself.
// Bound: memory from a few rows of 10^5 logits; a 16-bit row is near the vector rate too (about ten
// operations an element).
#pragma once

#include "verify_common.h"

namespace verify {

constexpr int kLpThreads = 256;
constexpr int kLpWaves = kLpThreads / 64;
constexpr int kTop = VERIFY_MAX_ALTERNATIVES;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLpNegInf = -__builtin_inff();

// Running statistics of a lane.
struct LpStat {
  float m, l, e;  // reference (in powers of two), sums
};

__device__ __forceinline__ LpStat lp_join(LpStat a, LpStat b) {
  const float m = fmaxf(a.m, b.m);
  const float ref = m == kLpNegInf ? 0.0f : m;
  // an empty side (m = -inf, sums 0) has factor 0 and shift 0
  const float da = a.m == kLpNegInf ? 0.0f : a.m - ref, db = b.m == kLpNegInf ? 0.0f : b.m - ref;
  const float fa = __builtin_amdgcn_exp2f(da), fb = __builtin_amdgcn_exp2f(db);
  LpStat r;
  r.m = m;
  // a factor of 0 times a shift of many thousand must not meet an infinite shift: shifts are finite here
  r.l = a.l * fa + b.l * fb;
  r.e = (fa == 0 ? 0.0f : fa * (a.e + da * a.l)) + (fb == 0 ? 0.0f : fb * (b.e + db * b.l));
  return r;
}

// The wave's best elements, sorted: lane i < K holds the i-th. `n` of them are there; `cut` is the K-th
// value once n = K.
struct LpTop {
  float v;
  int id;
  int n;
  float cut;
};

__device__ __forceinline__ void lp_insert(LpTop& top, float v, int id, int K, int lane) {
  // after everything larger, and after equal ones of lower id
  const bool before = lane < top.n && (top.v > v || (top.v == v && top.id < id));
  const int at = __popcll(__ballot(before));
  const float vu = __shfl_up(top.v, 1);
  const int iu = __shfl_up(top.id, 1);
  if (lane > at) top.v = vu, top.id = iu;
  if (lane == at) top.v = v, top.id = id;
  if (top.n < K) ++top.n;
  if (top.n == K) top.cut = __shfl(top.v, K - 1);
}

// Takes the elements of x (E per lane, element j of the lane has id ids(j), ascending in j) that are among
// the best. Every lane calls it; NaN elements are never taken.
template <int E, typename F>
__device__ __forceinline__ void lp_take(LpTop& top, const float (&x)[E], int K, int lane, F ids) {
  uint64_t left = 0;  // elements of this lane not yet taken
  static_assert(E <= 64, "one bit an element");
#pragma unroll
  for (int j = 0; j < E; ++j) left |= (x[j] == x[j] && ids(j) >= 0) ? uint64_t(1) << j : 0;
  for (;;) {
    float best = kLpNegInf;
    int at = -1;
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (((left >> j) & 1) && (at < 0 || x[j] > best)) best = x[j], at = j;
    float w = best;
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) w = fmaxf(w, __shfl_xor(w, s));
    int id = INT32_MAX;
    if (at >= 0 && best == w) {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (j == at) id = ids(j);
    }
    int lo = id;
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) lo = min(lo, __shfl_xor(lo, s));
    if (lo == INT32_MAX) return;  // nothing left
    if (top.n == K) {  // full: it must beat the last (a tie goes to the lower id)
      const float lv = __shfl(top.v, K - 1);
      const int li = __shfl(top.id, K - 1);
      if (!(w > lv || (w == lv && lo < li))) return;
    }
    lp_insert(top, w, lo, K, lane);
    if (id == lo) left &= ~(uint64_t(1) << at);
  }
}

struct LpPlan {
  int32_t splits;   // blocks per row
  float* stat;      // [rows][splits * 4][3]
  float* tv;        // [rows][splits * 4][top]
  int32_t* ti;      // the same
};

template <typename T>
__device__ __forceinline__ float lp_value(T v) { return static_cast<float>(v); }

template <typename T>
__device__ __forceinline__ void lp_outputs(const verify_logprobs_args& a, int t, const LpStat& st, const LpTop& top,
                                           int lane) {
  // every lane holds the row's statistics, the first `top` lanes the alternatives
  const float lg = __builtin_amdgcn_logf(st.l);  // log2
  const bool none = st.m == kLpNegInf && st.l == 0;  // every logit is -inf
  const float z = kLn2 * (st.m + lg);
  const T* row = static_cast<const T*>(a.logits) + t * a.row_stride;
  for (int n = lane; n < a.n_tokens; n += 64) {
    const int64_t at = static_cast<int64_t>(t) * a.n_tokens + n;
    const int64_t id = a.tokens_64 ? static_cast<const int64_t*>(a.tokens)[at] : static_cast<const int32_t*>(a.tokens)[at];
    float lp = kLpNegInf;
    if (id >= 0 && id < a.vocab) {
      const float x = lp_value(row[id]);
      lp = none ? kLpNegInf : x - z;
    }
    a.logprobs[at] = lp;
  }
  if (a.entropy && lane == 0) a.entropy[t] = none ? 0.0f : kLn2 * (lg - st.e / st.l);
  if (lane < a.top) {
    const int64_t at = static_cast<int64_t>(t) * a.top + lane;
    const bool there = lane < top.n;
    a.top_ids[at] = there ? top.id : -1;
    a.top_logprobs[at] = !there ? __builtin_nanf("") : none ? kLpNegInf : top.v - z;
  }
}

// Joins `parts` partial results (statistics and sorted lists of K), one wave.
template <typename FS, typename FV, typename FI>
__device__ __forceinline__ void lp_join_parts(int parts, int K, int lane, FS stat, FV value, FI ident, LpStat* st,
                                              LpTop* top) {
  LpStat s{kLpNegInf, 0, 0};
  for (int i = lane; i < parts; i += 64) s = lp_join(s, stat(i));
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const LpStat o{__shfl_xor(s.m, d), __shfl_xor(s.l, d), __shfl_xor(s.e, d)};
    // the lower lane's side first on both sides, so that all lanes agree bit for bit
    s = (lane & d) ? lp_join(o, s) : lp_join(s, o);
  }
  *st = s;
  *top = LpTop{0, -1, 0, 0};
  for (int i0 = 0; i0 < parts * K; i0 += 64) {
    const int i = i0 + lane;
    float x[1] = {0};
    int id = -1;
    if (i < parts * K) x[0] = value(i), id = ident(i);
    lp_take<1>(*top, x, K, lane, [&](int) { return id; });
  }
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads) logprobs_kernel(verify_logprobs_args a, LpPlan p) {
  constexpr int VEC = 16 / sizeof(T);  // elements of a load
  constexpr int U = sizeof(T) == 4 ? 4 : 2;
  constexpr int E = VEC * U, CHUNK = 64 * E;
  typedef T TV __attribute__((ext_vector_type(VEC)));
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int t = blockIdx.x / p.splits, split = blockIdx.x - t * p.splits;
  const T* const row = static_cast<const T*>(a.logits) + t * a.row_stride;
  const int V = a.vocab, K = a.top;

  // The row from its first 16-byte boundary on is cut into chunks, the chunks evenly over the row's waves;
  // the elements before it go to the first wave, those behind the last whole chunk to the last.
  const int miss = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / static_cast<int>(sizeof(T));
  const int lead = miss < V ? miss : V;
  const int chunks = (V - lead) / CHUNK;
  const int waves = p.splits * kLpWaves, w = split * kLpWaves + wave;
  const int c0 = static_cast<int>(static_cast<int64_t>(chunks) * w / waves);
  const int c1 = static_cast<int>(static_cast<int64_t>(chunks) * (w + 1) / waves);

  LpStat st{kLpNegInf, 0, 0};
  LpTop top{0, -1, 0, 0};
  auto add = [&](const float (&x)[E], auto ids) {
    float best = kLpNegInf;
#pragma unroll
    for (int j = 0; j < E; ++j) best = fmaxf(best, x[j]);
    const float m = fmaxf(st.m, best * kLog2e);
    if (m > st.m) {
      if (st.l != 0) {
        const float d = st.m - m, f = __builtin_amdgcn_exp2f(d);
        st.e = f == 0 ? 0.0f : f * (st.e + d * st.l);
        st.l *= f;
      }
      st.m = m;
    }
    const float ref = m == kLpNegInf ? 0.0f : m;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float d = fmaf(x[j], kLog2e, -ref);
      const float q = __builtin_amdgcn_exp2f(d);
      st.l += q;
      st.e = fmaf(q, fmaxf(d, -256.0f), st.e);  // 2^d is 0 there: a logit of -inf adds 0, not NaN
    }
    if (K && __ballot(top.n < K || best > top.cut)) lp_take<E>(top, x, K, lane, ids);
  };
  auto edge = [&](int from, int to) {  // fewer than 64 * E elements, one by one
    float x[E];
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int i = from + j * 64 + lane;
      x[j] = i < to ? lp_value(row[i]) : kLpNegInf;
    }
    add(x, [&](int j) { const int i = from + j * 64 + lane; return i < to ? i : -1; });
  };
  if (w == 0 && lead) edge(0, lead);
  const T* const base = row + lead;
  if (c0 < c1) {
    TV buf[U], nxt[U];
    auto load = [&](TV (&d)[U], int ch) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        d[u] = *reinterpret_cast<const TV*>(base + static_cast<int64_t>(ch) * CHUNK + (u * 64 + lane) * VEC);
    };
    load(buf, c0);
    for (int ch = c0; ch < c1; ++ch) {
      if (ch + 1 < c1) load(nxt, ch + 1);
      float x[E];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[u * VEC + j] = lp_value(static_cast<T>(buf[u][j]));
      const int first = lead + ch * CHUNK + lane * VEC;
      add(x, [&](int j) { return first + (j / VEC) * 64 * VEC + j % VEC; });
#pragma unroll
      for (int u = 0; u < U; ++u) buf[u] = nxt[u];
    }
  }
  if (w == waves - 1 && lead + chunks * CHUNK < V) edge(lead + chunks * CHUNK, V);

#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const LpStat o{__shfl_xor(st.m, d), __shfl_xor(st.l, d), __shfl_xor(st.e, d)};
    st = (lane & d) ? lp_join(o, st) : lp_join(st, o);
  }
  if (p.splits == 1) {
    __shared__ float ss[kLpWaves][3], sv[kLpWaves * kTop];
    __shared__ int si[kLpWaves * kTop];
    if (lane == 0) ss[wave][0] = st.m, ss[wave][1] = st.l, ss[wave][2] = st.e;
    if (lane < K) {
      sv[wave * K + lane] = top.v;
      si[wave * K + lane] = lane < top.n ? top.id : -1;
    }
    __syncthreads();
    if (wave) return;
    LpStat all;
    LpTop best;
    lp_join_parts(kLpWaves, K, lane, [&](int i) { return LpStat{ss[i][0], ss[i][1], ss[i][2]}; },
                  [&](int i) { return sv[i]; }, [&](int i) { return si[i]; }, &all, &best);
    lp_outputs<T>(a, t, all, best, lane);
    return;
  }
  const int64_t at = static_cast<int64_t>(t) * waves + w;
  if (lane == 0) {
    p.stat[3 * at] = st.m;
    p.stat[3 * at + 1] = st.l;
    p.stat[3 * at + 2] = st.e;
  }
  if (lane < K) {
    p.tv[at * K + lane] = top.v;
    p.ti[at * K + lane] = lane < top.n ? top.id : -1;
  }
}

template <typename T>
__global__ void __launch_bounds__(64) logprobs_join_kernel(verify_logprobs_args a, LpPlan p) {
  const int lane = threadIdx.x, t = blockIdx.x, K = a.top;
  const int parts = p.splits * kLpWaves;
  const int64_t at = static_cast<int64_t>(t) * parts;
  LpStat all;
  LpTop best;
  lp_join_parts(parts, K, lane,
                [&](int i) { return LpStat{p.stat[3 * (at + i)], p.stat[3 * (at + i) + 1], p.stat[3 * (at + i) + 2]}; },
                [&](int i) { return p.tv[at * K + i]; }, [&](int i) { return p.ti[at * K + i]; }, &all, &best);
  lp_outputs<T>(a, t, all, best, lane);
}

// Blocks per row, and the workspace for the parts.
inline LpPlan lp_plan(const verify_logprobs_args& a, void* workspace, int64_t* bytes) {
  LpPlan p{};
  const int chunk = 64 * 16;  // logprobs_kernel's, either type
  const int64_t most = (static_cast<int64_t>(a.vocab) / chunk + kLpWaves - 1) / kLpWaves;  // a chunk a wave
  const int64_t want = (1024 + a.n_rows - 1) / a.n_rows;  // about four blocks a CU
  int64_t s = want < most ? want : most;
  p.splits = static_cast<int32_t>(s < 1 ? 1 : s);
  const int64_t parts = static_cast<int64_t>(a.n_rows) * p.splits * kLpWaves;
  *bytes = p.splits > 1 ? parts * (12 + 8 * a.top) : 0;
  p.stat = static_cast<float*>(workspace);
  p.tv = p.stat + 3 * parts;
  p.ti = reinterpret_cast<int32_t*>(p.tv + parts * a.top);
  return p;
}

template <typename T>
hipError_t launch_logprobs_t(const verify_logprobs_args& a, const LpPlan& p, hipStream_t stream) {
  logprobs_kernel<T><<<dim3(static_cast<unsigned>(p.splits) * a.n_rows), kLpThreads, 0, stream>>>(a, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  logprobs_join_kernel<T><<<dim3(a.n_rows), 64, 0, stream>>>(a, p);
  return hipGetLastError();
}

inline hipError_t launch_logprobs(const verify_logprobs_args& a, const LpPlan& p, hipStream_t stream) {
  if (a.type == VERIFY_F32) return launch_logprobs_t<float>(a, p, stream);
  if (a.type == VERIFY_BF16) return launch_logprobs_t<__bf16>(a, p, stream);
  return launch_logprobs_t<_Float16>(a, p, stream);
}

}  // namespace verify
