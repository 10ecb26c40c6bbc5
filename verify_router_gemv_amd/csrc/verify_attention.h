// Attention of each request's tree of drafted rows over its paged cache.
//
// For one request and one kv head the M = rows * (heads / kv_heads) query rows share every key and
// value, so a block holds all of them (up to 256) and streams the cache once.  Online softmax: with the
// running maximum m, sum l and output O of the tokens so far, a tile of 32 tokens with scores s adds
//   m' = max(m, max s), p = exp(s - m'), l' = l e^(m - m') + sum p, O' = O e^(m - m') + p V.
//
// Both products are 16x16x32 matrix instructions, computed transposed so that no operand crosses lanes:
//   S^T (token x row)  = K Q^T : lane (c = lane % 16, g = lane / 16) loads 16 bytes of token c's key as it
//                        lies in the cache; the result leaves it with row c's scores of tokens 4g..4g+3;
//   O^T (value x row) += V^T P^T : the scores of the tile's two 16-token halves, rounded, ARE the lane's
//                        part of P^T (the order of the 32 tokens along the reduction is free as long as
//                        V^T follows it: tokens 4g..4g+3 of the first half, then of the second).  V^T needs
//                        eight tokens of one value column in a lane: the lane loads columns 8c..8c+7 of
//                        its eight tokens (whole 256-byte cache rows per load) and transposes the 8 x 8
//                        block in its own registers; column 8c + i goes to the i-th product, which only
//                        permutes the output's columns (undone by the store).
// So keys and values go from memory to registers to the matrix cores, without LDS and without a
// barrier in the loop; every wave has its own tokens (or, with many rows, its own rows) and loads a
// tile ahead.
//
// The context is split over blocks: the blocks that fit on the chip at once are handed out by
// rows * tokens of each request (computed by every block from the lengths, see AttnPlan), and a second
// kernel joins the parts of requests with more than one.
// Bound: memory (each K/V byte is read once) up to about 64 query rows a kv head; above, the matrix
// cores and the exponentials.
#pragma once

#include "verify_common.h"

namespace verify {

constexpr int kAttnThreads = 256;
constexpr int kTile = 32;          // tokens per step of a wave
constexpr int kMinChunk = 256;     // fewest tokens a block is split down to
constexpr float kNegInf = -__builtin_inff();

// How the work of one call is cut up. The host fixes `target` (blocks that may be resident) and the
// grid from the sizes it knows; the rest follows from the lengths on the GPU, the same in every block.
struct AttnLaunch {
  int32_t m_block;   // query rows (rows * group) per block
  int32_t target;    // blocks to spread the work over, all heads together
  int32_t grid;      // blocks launched
  int32_t swizzle;   // 1: several row blocks per request, kept on one XCD (8 neighbours)
  float* part;       // [grid][m_block][D] partial outputs, then [grid][m_block][2] (maximum, sum)
};

struct AttnItem {
  int b, rows, start;       // request, its rows, its first row
  int cached, len;          // tokens before the round, tokens in all
  int chunk, chunks;        // this block's part of the context, of how many
  int mb, head;             // this block's row block and kv head
  int first;                // index of the request's first block
};

template <typename A>
__device__ __forceinline__ void attn_request(const A& a, int b, int* start, int* rows, int* cached, int* len) {
  int s = a.row_start[b], e = a.row_start[b + 1];
  s = s < 0 ? 0 : s > a.n_rows ? a.n_rows : s;
  e = e < s ? s : e > a.n_rows ? a.n_rows : e;
  int r = e - s;
  r = r > a.max_rows ? a.max_rows : r;
  const int64_t most = static_cast<int64_t>(a.width) * a.page_size;  // tokens the table can hold
  int64_t c = max0(a.cached[b]);
  c = c < most ? c : most;
  int64_t n = c + r;
  n = n < most ? n : most;
  *start = s;
  *rows = r;
  *cached = static_cast<int>(c);
  *len = static_cast<int>(n);
}

// Tokens per block so that the whole call makes about `target` blocks.
__device__ __forceinline__ int attn_chunk(const verify_attention_args& a, const AttnLaunch& p, int lane) {
  const int group = a.heads / a.kv_heads;
  int64_t work = 0;
  for (int b = lane; b < a.n_requests; b += 64) {
    int s, r, c, n;
    attn_request(a, b, &s, &r, &c, &n);
    work += static_cast<int64_t>((r * group + p.m_block - 1) / p.m_block) * n;
  }
  work = wave_sum64(work) * a.kv_heads;
  int64_t c = (work + p.target - 1) / p.target;
  c = (c + kTile - 1) / kTile * kTile;
  c = c < kMinChunk ? kMinChunk : c;
  return c < INT32_MAX / 2 ? static_cast<int>(c) : INT32_MAX / 2;
}

// Blocks of one request: row blocks x kv heads x chunks, the last two rounded up together to a multiple
// of 8 when there are several row blocks.
__device__ __forceinline__ int attn_blocks(const verify_attention_args& a, const AttnLaunch& p, int rows, int len,
                                           int chunk, int* chunks) {
  const int mbs = (rows * (a.heads / a.kv_heads) + p.m_block - 1) / p.m_block;
  const int n = len > chunk ? (len + chunk - 1) / chunk : 1;
  *chunks = n;
  int u = n * a.kv_heads;
  if (p.swizzle) u = (u + 7) & ~7;
  return mbs * u;
}

// The request that block `at` works on (want_b < 0), or the plan of request want_b. False: none.
__device__ __forceinline__ bool attn_find(const verify_attention_args& a, const AttnLaunch& p, int lane, int at,
                                          int want_b, AttnItem* it) {
  const int chunk = attn_chunk(a, p, lane);
  int64_t base = 0;
  for (int b0 = 0; b0 < a.n_requests; b0 += 64) {
    const int b = b0 + lane;
    int s = 0, r = 0, c = 0, n = 0, chunks = 1, blocks = 0;
    if (b < a.n_requests) {
      attn_request(a, b, &s, &r, &c, &n);
      blocks = r ? attn_blocks(a, p, r, n, chunk, &chunks) : 0;
    }
    const int64_t end = base + wave_scan64(blocks, lane);
    const uint64_t hit = want_b >= 0 ? (want_b - b0 < 64 ? uint64_t(1) << (want_b - b0) : 0) : __ballot(end > at);
    if (hit) {
      const int from = __ffsll(static_cast<unsigned long long>(hit)) - 1;
      it->b = b0 + from;
      it->start = uniform(__shfl(s, from));
      it->rows = uniform(__shfl(r, from));
      it->cached = uniform(__shfl(c, from));
      it->len = uniform(__shfl(n, from));
      it->chunks = uniform(__shfl(chunks, from));
      const int last = uniform(__shfl(static_cast<int>(end), from));  // blocks fit 31 bits (checked by the host)
      it->first = last - uniform(__shfl(blocks, from));
      return true;
    }
    base += __shfl(end - base, 63);
  }
  return false;
}

// A request's blocks in launch order: with the swizzle, groups of 8 (chunk, head) units, row blocks in
// between, so that the row blocks of one unit are 8 apart and reach the same XCD (and its L2).
__device__ __forceinline__ int attn_unit_block(const AttnLaunch& p, int unit, int mb, int mbs) {
  return p.swizzle ? (unit >> 3) * 8 * mbs + mb * 8 + (unit & 7) : unit;
}

template <typename T>
struct Mfma;
template <>
struct Mfma<__bf16> {
  typedef bf16x8 V;
  static __device__ __forceinline__ f32x4 mul(V a, V b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static constexpr uint32_t kExp = 0x7f80;  // the exponent bits: all set in infinities and NaN
  static constexpr float kLift = 0.0f;
};
template <>
struct Mfma<_Float16> {
  typedef f16x8 V;
  static __device__ __forceinline__ f32x4 mul(V a, V b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  static constexpr uint32_t kExp = 0x7c00;
  // Probabilities are held 2^7 times as large (a factor of the sums too, so it cancels): up to 2^15, below
  // the type's largest value, and 2^-21 of the running maximum still has the type's full precision.
  static constexpr float kLift = 7.0f;
};

// Maximum / sum over the lanes that hold the other tokens of the same query row.
__device__ __forceinline__ float rows_max(float v) {
  const float2 a = across<16>(v);
  const float2 b = across<32>(fmaxf(a.x, a.y));
  return fmaxf(b.x, b.y);
}
__device__ __forceinline__ float rows_sum(float v) {
  const float2 a = across<16>(v);
  const float2 b = across<32>(a.x + a.y);
  return b.x + b.y;
}

// One wave's view of the tile of 32 tokens at `tok`: its keys (16-byte pieces) and values.
template <int D>
struct KV {
  static constexpr int KK = D / 32;            // matrix steps along the head
  static constexpr int VW = D == 64 ? 2 : 4;   // dwords of a value load (D = 64: 4 columns per lane)
  static constexpr int VH = D == 256 ? 2 : 1;  // 128-column halves
  u32x4 k[2][KK];
  uint32_t v[8][VH][VW];
  bool ok[2];                                  // the half tile's page exists
};

template <typename T, int D, int NM, int WK>
__global__ void __launch_bounds__(kAttnThreads) attn_kernel(verify_attention_args a, AttnLaunch p) {
  typedef Mfma<T> MM;
  typedef typename MM::V V8;
  typedef KV<D> Tile;
  constexpr int KK = Tile::KK, VW = Tile::VW, VH = Tile::VH, DV = 2 * VW;  // DV columns of a lane per half
  constexpr int NT = VH * DV;                                              // output tiles (16 columns each)
  constexpr int WM = 4 / WK, MB = 16 * NM * WM;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int wk = wave % WK, wm = wave / WK;
  const int group = a.heads / a.kv_heads;

  AttnItem it;
  if (!attn_find(a, p, lane, blockIdx.x, -1, &it)) return;
  const int mbs = (it.rows * group + MB - 1) / MB;
  int unit;
  {
    const int at = blockIdx.x - it.first;
    if (p.swizzle) {
      const int q = at / (8 * mbs), r = at - q * 8 * mbs;
      it.mb = r >> 3;
      unit = q * 8 + (r & 7);
    } else {
      it.mb = 0;
      unit = at;
    }
    if (unit >= it.chunks * a.kv_heads) return;  // rounding of the swizzle
    it.head = unit % a.kv_heads;
    it.chunk = unit / a.kv_heads;
  }
  // Chunks of equal length, whole tiles.
  const int step = ((it.len + it.chunks - 1) / it.chunks + kTile - 1) / kTile * kTile;
  const int t0 = it.chunk * step;
  const int t1 = t0 + step < it.len ? t0 + step : it.len;

  // Query rows: row m = 16 (NM wm + n) + c of the block, in the order of the matrix operand.
  V8 q[NM][KK];
  uint64_t mask[NM];
  const int m0 = it.mb * MB + wm * 16 * NM;
  const int total = it.rows * group;
  const uint64_t inside = it.rows >= 64 ? ~uint64_t(0) : (uint64_t(1) << it.rows) - 1;
#pragma unroll
  for (int n = 0; n < NM; ++n) {
    const int m = m0 + 16 * n + c;
    const int mm = m < total ? m : 0;
    const int i = mm / group, h = it.head * group + (mm - i * group);
    const T* src = static_cast<const T*>(a.q) + static_cast<int64_t>(it.start + i) * a.q_row + h * a.q_head + 8 * g;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) q[n][kk] = *reinterpret_cast<const V8*>(src + 32 * kk);
    mask[n] = a.masks ? static_cast<uint64_t>(a.masks[it.start + i]) : (uint64_t(2) << i) - 1;
    mask[n] &= inside;
  }

  f32x4 o[NM][NT] = {};
  float mx[NM], sum[NM];  // running maximum of the raw scores, sum of the lane's own probabilities
#pragma unroll
  for (int n = 0; n < NM; ++n) mx[n] = kNegInf, sum[n] = 0;
  const float sc = a.scale * 1.4426950408889634f;  // exponentials are powers of two

  const int shift = __builtin_ctz(a.page_size), in_page = a.page_size - 1;
  const int32_t* const pages = a.table + it.b * a.table_stride;
  const T* const kbase = static_cast<const T*>(a.k_cache) + it.head * a.kc_head;
  const T* const vbase = static_cast<const T*>(a.v_cache) + it.head * a.vc_head;
  // 16 tokens never cross a page. A page past the table or the cache is not read: its tokens count as
  // unseen (page 0 is read instead, and dropped).
  auto page_of = [&](int tok) {
    const int col = tok >> shift;
    const int page = col < a.width ? pages[col] : -1;
    return page < a.n_pages ? page : -1;
  };
  auto load = [&](Tile& x, int tok, const int (&page)[2]) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      x.ok[s] = page[s] >= 0;
      const int64_t pg = page[s] >= 0 ? page[s] : 0;
      const int place = (tok + 16 * s) & in_page;
      const T* kp = kbase + pg * a.kc_page + place * a.kc_token + (c * static_cast<int>(a.kc_token) + 8 * g);
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) x.k[s][kk] = *reinterpret_cast<const u32x4*>(kp + 32 * kk);
      const T* vp = vbase + pg * a.vc_page + place * a.vc_token;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int hv = 0; hv < VH; ++hv) {
          const T* src = vp + ((4 * g + j) * static_cast<int>(a.vc_token) + DV * c + 128 * hv);
          if constexpr (VW == 4) {
            const u32x4 w = *reinterpret_cast<const u32x4*>(src);
#pragma unroll
            for (int e = 0; e < 4; ++e) x.v[4 * s + j][hv][e] = w[e];
          } else {
            const u32x2 w = *reinterpret_cast<const u32x2*>(src);
#pragma unroll
            for (int e = 0; e < 2; ++e) x.v[4 * s + j][hv][e] = w[e];
          }
        }
    }
  };

  auto compute = [&](Tile& x, int tok) {
    const bool edge = tok + kTile > it.cached || !x.ok[0] || !x.ok[1];  // some token may be unseen
    f32x4 s[NM][2] = {};
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int kk = 0; kk < KK; ++kk)
#pragma unroll
        for (int n = 0; n < NM; ++n)
          s[n][h] = MM::mul(__builtin_bit_cast(V8, x.k[h][kk]), q[n][kk], s[n][h]);
    bool slow = false;
    if (edge) {
      // Scores of unseen tokens are replaced, whatever they are; values of tokens that nobody may see
      // (past the end, on no page) are zeroed, and a drafted token's infinity or NaN is kept out of the
      // matrix product, which would spread it to the rows that do not see the token.
      uint32_t bad = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = tok + 16 * h + 4 * g + r, d = t - it.cached;
          const bool real = x.ok[h] && t < t1;
#pragma unroll
          for (int n = 0; n < NM; ++n) {
            const bool seen = real && (d < 0 || (d < 64 && ((mask[n] >> (d & 63)) & 1)));
            s[n][h][r] = seen ? s[n][h][r] : kNegInf;
          }
#pragma unroll
          for (int hv = 0; hv < VH; ++hv)
#pragma unroll
            for (int e = 0; e < VW; ++e) {
              uint32_t w = real ? x.v[4 * h + r][hv][e] : 0;
              if (d >= 0) {
                const bool lo = (w & MM::kExp) == MM::kExp;
                const bool hi = ((w >> 16) & MM::kExp) == MM::kExp;
                bad |= lo | hi;
                w = (lo ? 0 : w & 0xffffu) | (hi ? 0 : w & 0xffff0000u);
              }
              x.v[4 * h + r][hv][e] = w;
            }
        }
      slow = __ballot(bad) != 0;
    }
    // Probabilities relative to a running maximum that a row raises only when its own grows by more than
    // 8 powers of two: until then p <= 2^8, which both 16-bit types hold with their full precision. (Each
    // row by itself: its result does not depend on the other rows' values.)
    float raised[NM];
    bool grow = false;
#pragma unroll
    for (int n = 0; n < NM; ++n) {
      float v = fmaxf(fmaxf(fmaxf(s[n][0][0], s[n][0][1]), fmaxf(s[n][0][2], s[n][0][3])),
                      fmaxf(fmaxf(s[n][1][0], s[n][1][1]), fmaxf(s[n][1][2], s[n][1][3])));
      v = rows_max(v);
      const bool up = (v - mx[n]) * sc > 8.0f;  // also from -inf; not for NaN (-inf after -inf)
      raised[n] = up ? v : mx[n];
      grow |= up;
    }
    if (__ballot(grow)) {
#pragma unroll
      for (int n = 0; n < NM; ++n) {
        const float m = raised[n];
        const float f = mx[n] == m ? 1.0f : __builtin_amdgcn_exp2f((mx[n] - m) * sc);
        mx[n] = m;
        sum[n] *= f;
#pragma unroll
        for (int i = 0; i < NT; ++i) o[n][i] *= f;
      }
    }
    V8 pt[NM];
#pragma unroll
    for (int n = 0; n < NM; ++n) {
      const float ref = (mx[n] == kNegInf ? 0.0f : mx[n] * sc) - MM::kLift;
      f32x8 e;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        e[j] = __builtin_amdgcn_exp2f(fmaf(s[n][j >> 2][j & 3], sc, -ref));
        sum[n] += e[j];
      }
      pt[n] = __builtin_convertvector(e, V8);
    }
    // V^T: element i of the lane's columns, of its eight tokens.
#pragma unroll
    for (int hv = 0; hv < VH; ++hv)
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        u32x4 lo, hi;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w0 = x.v[2 * j][hv][e], w1 = x.v[2 * j + 1][hv][e];
          lo[j] = __builtin_amdgcn_perm(w1, w0, 0x05040100);
          hi[j] = __builtin_amdgcn_perm(w1, w0, 0x07060302);
        }
#pragma unroll
        for (int n = 0; n < NM; ++n) {
          o[n][hv * DV + 2 * e] = MM::mul(__builtin_bit_cast(V8, lo), pt[n], o[n][hv * DV + 2 * e]);
          o[n][hv * DV + 2 * e + 1] = MM::mul(__builtin_bit_cast(V8, hi), pt[n], o[n][hv * DV + 2 * e + 1]);
        }
      }
    if (slow) {
      // The infinities and NaN left out above, token by token, added to the rows that see the token.
      for (int t = 0; t < kTile; ++t) {
        const int d = tok + t - it.cached;
        const bool ok = t < 16 ? x.ok[0] : x.ok[1];
        if (d < 0 || !ok || tok + t >= t1) continue;
        const int64_t pg = page_of(tok + t);
        const T* vp = vbase + pg * a.vc_page + ((tok + t) & in_page) * a.vc_token;
#pragma unroll
        for (int n = 0; n < NM; ++n) {
          const bool seen = d < 64 && ((mask[n] >> (d & 63)) & 1);
          float pr = 0;  // this row's probability of the token, from the lane that holds it
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float v = __shfl(static_cast<float>(pt[n][j]), ((t & 15) >> 2) * 16 + c);
            if (((t >> 4) * 4 + (t & 3)) == j) pr = v;
          }
#pragma unroll
          for (int hv = 0; hv < VH; ++hv)
#pragma unroll
            for (int i = 0; i < DV; ++i)
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const float v = static_cast<float>(vp[128 * hv + DV * (4 * g + r) + i]);
                if (seen && !(fabsf(v) < __builtin_inff())) o[n][hv * DV + i][r] += pr * v;
              }
        }
      }
    }
  };

  // Tiles wk, wk + WK, ... of the chunk, loaded one ahead, their page numbers two ahead.
  {
    Tile x[2];
    int tok = t0 + wk * kTile;
    constexpr int kStep = WK * kTile;
    auto next_pages = [&](int t, int (&pg)[2]) {
      pg[0] = page_of(t);
      pg[1] = page_of(t + 16);
    };
    if (tok < t1) {
      int pg[2], pn[2];
      next_pages(tok, pg);
      next_pages(tok + kStep, pn);
      load(x[0], tok, pg);
      for (;;) {
        if (tok + kStep < t1) {
          load(x[1], tok + kStep, pn);
          next_pages(tok + 2 * kStep, pn);
        }
        compute(x[0], tok);
        tok += kStep;
        if (tok >= t1) break;
        if (tok + kStep < t1) {
          load(x[0], tok + kStep, pn);
          next_pages(tok + 2 * kStep, pn);
        }
        compute(x[1], tok);
        tok += kStep;
        if (tok >= t1) break;
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NM; ++n) sum[n] = rows_sum(sum[n]);

  // Join the waves that shared rows, through LDS, and store: the output of a request in one part, or
  // this part's output, maximum and sum.
  const bool whole = it.chunks == 1;
  const int64_t slot = blockIdx.x;
  float* const part_o = p.part + slot * MB * D;
  float* const part_ml = p.part + static_cast<int64_t>(p.grid) * MB * D + slot * MB * 2;
  typedef float FV __attribute__((ext_vector_type(DV)));
  typedef FV FVM __attribute__((aligned(16)));  // in memory
  auto store = [&](int m, int col, FV value) {  // `value`: DV columns from col of the block's row m
    const int row = it.mb * MB + m;
    if (row >= total) return;
    if (whole) {
      const int i = row / group, h = it.head * group + (row - i * group);
      T* dst = static_cast<T*>(a.out) + static_cast<int64_t>(it.start + i) * a.o_row + h * a.o_head + col;
      typedef T TV __attribute__((ext_vector_type(DV)));
      *reinterpret_cast<TV*>(dst) = __builtin_convertvector(value, TV);
    } else {
      *reinterpret_cast<FVM*>(part_o + m * D + col) = value;
    }
  };
  if constexpr (WK == 1) {
#pragma unroll
    for (int n = 0; n < NM; ++n) {
      const int m = wm * 16 * NM + 16 * n + c;
      const float inv = whole ? (sum[n] == 0 ? 0.0f : 1.0f / sum[n]) : 1.0f;
#pragma unroll
      for (int hv = 0; hv < VH; ++hv)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          FV v;
#pragma unroll
          for (int i = 0; i < DV; ++i) v[i] = o[n][hv * DV + i][r] * inv;
          store(m, 128 * hv + DV * (4 * g + r), v);
        }
      if (!whole && g == 0) {
        part_ml[2 * m] = mx[n];
        part_ml[2 * m + 1] = sum[n];
      }
    }
  } else {
    constexpr int MW = 16 * NM, LD = D + 4;  // rows of a wave; padded row
    __shared__ __align__(16) float so[4][MW][LD];
    __shared__ float sml[4][MW][2];
#pragma unroll
    for (int n = 0; n < NM; ++n) {
#pragma unroll
      for (int hv = 0; hv < VH; ++hv)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          FV v;
#pragma unroll
          for (int i = 0; i < DV; ++i) v[i] = o[n][hv * DV + i][r];
          *reinterpret_cast<FVM*>(&so[wave][16 * n + c][128 * hv + DV * (4 * g + r)]) = v;
        }
      if (g == 0) {
        sml[wave][16 * n + c][0] = mx[n];
        sml[wave][16 * n + c][1] = sum[n];
      }
    }
    __syncthreads();
    constexpr int CH = D / DV;  // pieces of a row
    for (int e = threadIdx.x; e < MB * CH; e += kAttnThreads) {
      const int m = e / CH, col = (e % CH) * DV;
      const int w0 = m / MW * WK, mw = m % MW;
      float top = kNegInf;
#pragma unroll
      for (int w = 0; w < WK; ++w) top = fmaxf(top, sml[w0 + w][mw][0]);
      FV v = {};
      float l = 0;
#pragma unroll
      for (int w = 0; w < WK; ++w) {
        const float mw_max = sml[w0 + w][mw][0];
        const float f = mw_max == kNegInf ? 0.0f : __builtin_amdgcn_exp2f((mw_max - top) * sc);
        // A wave that saw nothing holds zeros only.
        v += *reinterpret_cast<const FVM*>(&so[w0 + w][mw][col]) * f;
        l += sml[w0 + w][mw][1] * f;
      }
      if (whole) v *= l == 0 ? 0.0f : 1.0f / l;
      store(m, col, v);
      if (!whole && col == 0 && it.mb * MB + m < total) {
        part_ml[2 * m] = top;
        part_ml[2 * m + 1] = l;
      }
    }
  }
}

// Joins the parts of a (row, head): one wave each, D / 64 values a lane. Rows of requests in one part are
// stored already.
template <typename T, int D>
__global__ void __launch_bounds__(kAttnThreads) attn_join_kernel(verify_attention_args a, AttnLaunch p) {
  constexpr int E = D / 64;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int id = blockIdx.x * 4 + wave;
  const int t = id / a.heads, h = id - t * a.heads;
  if (t >= a.n_rows) return;
  // The row's request: the last one that starts at or before it and has rows there.
  int b = -1;
  for (int b0 = 0; b0 < a.n_requests && b < 0; b0 += 64) {
    const int x = b0 + lane;
    int s = 0, r = 0, c = 0, n = 0;
    if (x < a.n_requests) attn_request(a, x, &s, &r, &c, &n);
    const uint64_t hit = __ballot(t >= s && t < s + r);
    if (hit) b = b0 + __ffsll(static_cast<unsigned long long>(hit)) - 1;
  }
  if (b < 0) return;
  AttnItem it;
  if (!attn_find(a, p, lane, 0, b, &it) || it.chunks == 1) return;
  const int group = a.heads / a.kv_heads;
  const int kvh = h / group;
  const int m_all = (t - it.start) * group + (h - kvh * group);
  const int mb = m_all / p.m_block, m = m_all - mb * p.m_block;
  const int mbs = (it.rows * group + p.m_block - 1) / p.m_block;
  const float sc = a.scale * 1.4426950408889634f;
  const float* const ml = p.part + static_cast<int64_t>(p.grid) * p.m_block * D;
  auto part = [&](int ch) {
    return static_cast<int64_t>(it.first + attn_unit_block(p, ch * a.kv_heads + kvh, mb, mbs)) * p.m_block + m;
  };
  float top = kNegInf;
  for (int ch = lane; ch < it.chunks; ch += 64) top = fmaxf(top, ml[2 * part(ch)]);
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) top = fmaxf(top, __shfl_xor(top, s));
  float v[E] = {}, l = 0;
#pragma unroll 4
  for (int ch = 0; ch < it.chunks; ++ch) {
    const int64_t at = part(ch);
    const float mc = ml[2 * at], lc = ml[2 * at + 1];
    const float f = mc == kNegInf ? 0.0f : __builtin_amdgcn_exp2f((mc - top) * sc);
    const float* src = p.part + at * D + E * lane;
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] += src[e] * f;
    l += lc * f;
  }
  const float inv = l == 0 ? 0.0f : 1.0f / l;
  T* dst = static_cast<T*>(a.out) + static_cast<int64_t>(t) * a.o_row + h * a.o_head + E * lane;
#pragma unroll
  for (int e = 0; e < E; ++e) dst[e] = static_cast<T>(v[e] * inv);
}

// Launch shapes: rows a block holds, by the most query rows a (request, kv head) can have.
struct AttnShape {
  int nm, wk, m_block, per_cu;  // 16-row tiles a wave, waves along the tokens, rows a block, blocks a CU holds
};

inline AttnShape attn_shape(const verify_attention_args& a) {
  const int m = a.max_rows * (a.heads / a.kv_heads);
  if (m <= 16) return {1, 4, 16, a.dim == 256 ? 1 : 2};
  if (m <= 32) return {2, 4, 32, 1};
  if (a.dim == 256) return m <= 64 ? AttnShape{2, 2, 64, 1} : AttnShape{2, 1, 128, 1};
  if (m <= 64) return {4, 4, 64, 1};
  if (m <= 128) return {4, 2, 128, 1};
  return {4, 1, 256, 1};
}

// The grid and the workspace of a call; false if the blocks do not fit 31 bits.
inline bool attn_plan(const verify_attention_args& a, AttnLaunch* p, int64_t* bytes) {
  const AttnShape s = attn_shape(a);
  const int m = a.max_rows * (a.heads / a.kv_heads);
  const int64_t per_request = (m + s.m_block - 1) / s.m_block;
  p->m_block = s.m_block;
  p->target = 256 * s.per_cu;
  p->swizzle = per_request > 1;
  // sum over requests of row blocks x (heads x chunks, rounded): at most target for the chunks in all, one
  // more chunk per row block and head, and the rounding.
  const int64_t rowblocks = static_cast<int64_t>(a.n_requests) * per_request;
  const int64_t grid = p->target + rowblocks * (a.kv_heads + (p->swizzle ? 7 : 0));
  if (grid > INT32_MAX) return false;
  p->grid = static_cast<int32_t>(grid);
  p->part = nullptr;
  // A table that holds no more tokens than one chunk never splits.
  const bool split = static_cast<int64_t>(a.width) * a.page_size > kMinChunk;
  *bytes = split ? grid * s.m_block * (a.dim + 2) * 4 : 0;
  return true;
}

template <typename T, int D>
hipError_t launch_attention_d(const verify_attention_args& a, const AttnLaunch& p, bool join, hipStream_t stream) {
  const AttnShape s = attn_shape(a);
  const dim3 grid(p.grid), block(kAttnThreads);
  if (s.nm == 1) {
    attn_kernel<T, D, 1, 4><<<grid, block, 0, stream>>>(a, p);
  } else if (s.nm == 2 && s.wk == 4) {
    attn_kernel<T, D, 2, 4><<<grid, block, 0, stream>>>(a, p);
  } else if constexpr (D == 256) {
    if (s.wk == 2) attn_kernel<T, D, 2, 2><<<grid, block, 0, stream>>>(a, p);
    else attn_kernel<T, D, 2, 1><<<grid, block, 0, stream>>>(a, p);
  } else {
    if (s.wk == 4) attn_kernel<T, D, 4, 4><<<grid, block, 0, stream>>>(a, p);
    else if (s.wk == 2) attn_kernel<T, D, 4, 2><<<grid, block, 0, stream>>>(a, p);
    else attn_kernel<T, D, 4, 1><<<grid, block, 0, stream>>>(a, p);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !join) return e;
  const int64_t waves = static_cast<int64_t>(a.n_rows) * a.heads;
  attn_join_kernel<T, D><<<dim3(static_cast<unsigned>((waves + 3) / 4)), block, 0, stream>>>(a, p);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_attention(const verify_attention_args& a, const AttnLaunch& p, bool join, hipStream_t stream) {
  switch (a.dim) {
    case 64: return launch_attention_d<T, 64>(a, p, join, stream);
    case 128: return launch_attention_d<T, 128>(a, p, join, stream);
    default: return launch_attention_d<T, 256>(a, p, join, stream);
  }
}

extern template hipError_t launch_attention<__bf16>(const verify_attention_args&, const AttnLaunch&, bool, hipStream_t);
extern template hipError_t launch_attention<_Float16>(const verify_attention_args&, const AttnLaunch&, bool, hipStream_t);

}  // namespace verify
