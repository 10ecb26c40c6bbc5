// Attention of each request's tree of drafted rows over its paged cache.
//
// For one request and one kv head the M = rows * (heads / kv_heads) query rows share every key and
// value, so a block holds up to 256 of them and streams the cache once.  Online softmax: with the
// running maximum m, sum l and output O of the tokens so far, a tile of 32 tokens with scores s adds
//   m' = max(m, max s), p = exp(s - m'), l' = l e^(m - m') + sum p, O' = O e^(m - m') + p V.
//
// A wave holds 32 query rows and works on tiles of 32 tokens with 32x32x16 matrix instructions, both
// products transposed so that no operand crosses lanes (c = lane % 32, h = lane / 32):
//   S^T (token x row)  = K Q^T : lane (c, h) loads token c's key as it lies in the cache, 16 bytes a step;
//                        the result leaves it with row c's scores of tokens 8q + 4h + r (q, r < 4);
//   O^T (value x row) += V^T P^T : the lane's 16 probabilities, rounded, ARE its part of P^T (the order of
//                        the tokens along the reduction is free as long as V^T follows it).  V^T needs
//                        eight tokens of one value column in a lane: the lane loads D / 32 neighbouring
//                        columns of its own 16 tokens (whole cache rows per load) and transposes them in
//                        its own registers; its i-th column goes to the i-th product, which only permutes
//                        the output's columns (undone by the store).
// A tile goes from memory straight into LDS (loads that write LDS, 16 bytes a lane), some tiles ahead of its
// use, and from there into the operands.  The waves of a block split the rows (WM) and the tokens (WK):
// the WM waves of a token stream share its tiles and fetch a part of each; a stream has as many stages as
// LDS holds (1 with WM = 1: the wave takes the tile into registers and refills the stage while it works).
// Keys lie in LDS with their 16-byte pieces exchanged within the token (piece ^ token), so that the reads of
// 32 tokens' same piece hit different banks; values as they are.
//
// The context is split over blocks: the blocks that the chip holds at once are handed out by
// rows * tokens of each request (worked out from the lengths, by every block or, with many requests, by a
// kernel of its own), and a last kernel joins the parts of requests with more than one.
// Bound: memory (each K/V byte is read once) up to about 64 query rows a kv head; above, the
// exponentials and the matrix cores, which wait for each other with two waves a SIMD; launch and three
// dependent latencies (lengths, page table, tile) with few tokens.  Measured, D = 128, with the join: 5 rows of
// 32 / 8 heads over 131071 tokens 94 + 5 us (5.7 TB/s); 8 requests of up to 8 rows, 32 / 4 heads, up to 8192
// tokens 27.5 + 4.8 (106 MB); 4 of up to 64 rows, up to 16384 tokens 80 + 9 (510 TFLOP/s); one row over 1000
// tokens 12.8.
#pragma once

#include "verify_common.h"

namespace verify {

constexpr int kTile = 32;          // tokens per step of a wave
// A context of more than kSplitTiles tiles per wave of a block is split, into parts of at least kMinTiles: a
// tile more costs a wave about 2 us of latency, a split the second kernel, 5 us.
constexpr int kSplitTiles = 4, kMinTiles = 2;
constexpr int kScanRequests = 128;  // with more, a kernel of its own works the cut out (verify_attention_cut.h)
constexpr int kCus = 256;
constexpr float kNegInf = -__builtin_inff();

typedef float f32x16 __attribute__((ext_vector_type(16)));

// How the work of one call is cut up. The host fixes `target` and the grid from the sizes it knows; the
// rest follows from the lengths on the GPU, the same in every block.
struct AttnLaunch {
  int32_t m_shift;   // log2 of the query rows (rows * group) per block
  int32_t target;    // blocks to spread the work over, all heads together
  int32_t grid;      // blocks launched
  int32_t least;     // fewest tiles of a part ...
  int32_t whole;     // ... and most of a context that is not split for the sake of the chip's width
  int32_t split;     // 1: contexts may come in parts, joined by the second kernel
  int32_t swizzle;   // 1: several row blocks per request, kept on one XCD (8 neighbours)
  float* part;       // [grid][rows][D] partial outputs, then [grid][rows][2] (maximum, sum)
  int32_t* plan;     // [B][2] first block and number of parts of each request
};

struct AttnRequest {
  int start, rows, cached, len;  // first row, rows, tokens before the round, tokens in all
};

__device__ __forceinline__ AttnRequest attn_request(const verify_attention_args& a, int b) {
  int s = a.row_start[b], e = a.row_start[b + 1];
  int c = a.cached[b];
  s = min(max(s, 0), a.n_rows);
  e = min(max(e, s), a.n_rows);
  const int r = min(e - s, a.max_rows);
  const int most = a.width * a.page_size;  // tokens the table can hold, at most 2^30
  c = min(max(c, 0), most);
  return {s, r, c, min(c + r, most)};
}

// Inclusive prefix sum over the wave.
__device__ __forceinline__ int wave_scan(int v, int lane) {
  auto up = [&](int w, auto ctrl) {
    return static_cast<int>(moe::dpp_u32<decltype(ctrl)::value>(static_cast<uint32_t>(w)));
  };
  // within rows of 16 lanes (lanes shifted in from outside the row are 0), then the rows' totals
  v += up(v, std::integral_constant<int, 0x111>{});
  v += up(v, std::integral_constant<int, 0x112>{});
  v += up(v, std::integral_constant<int, 0x114>{});
  v += up(v, std::integral_constant<int, 0x118>{});
  const int t0 = __builtin_amdgcn_readlane(v, 15), t1 = __builtin_amdgcn_readlane(v, 31),
            t2 = __builtin_amdgcn_readlane(v, 47);
  return v + (lane >= 16 ? t0 : 0) + (lane >= 32 ? t1 : 0) + (lane >= 48 ? t2 : 0);
}

// The last of n ascending numbers, `stride` apart, that is at most x (the first if none is): 64 of them a
// step. Other than ascending numbers give some place of the n.
__device__ __forceinline__ int wave_search(const int32_t* v, int stride, int n, int x, int lane) {
  int lo = 0;
  while (n > 1) {
    const int step = (n + 63) / 64, at = lane * step;
    const uint64_t hit = __ballot(at < n && v[static_cast<int64_t>(lo + (at < n ? at : 0)) * stride] <= x);
    const int k = hit ? 63 - __clzll(static_cast<long long>(hit)) : 0;
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// Tiles of a request, counted once per row block.
__device__ __forceinline__ float attn_work(const AttnLaunch& p, const AttnRequest& q, int group) {
  const int mbs = (q.rows * group + (1 << p.m_shift) - 1) >> p.m_shift;
  return static_cast<float>(mbs) * static_cast<float>((q.len + kTile - 1) / kTile);
}
// Tiles per block so that the whole call makes about `target` blocks. (As float: rounding moves the cut,
// alike in all blocks, and the grid has blocks to spare.)
__device__ __forceinline__ unsigned attn_chunk(const verify_attention_args& a, const AttnLaunch& p, float work) {
  const float c = ceilf(work * static_cast<float>(a.kv_heads) / static_cast<float>(p.target));
  return max(static_cast<unsigned>(c), static_cast<unsigned>(p.least));
}
// The blocks of a request.
__device__ __forceinline__ int attn_blocks(const verify_attention_args& a, const AttnLaunch& p, const AttnRequest& q,
                                           int group, unsigned chunk, int* parts, int* mbs) {
  const unsigned tiles = static_cast<unsigned>(q.len + kTile - 1) / kTile;
  const bool split = tiles > max(chunk, static_cast<unsigned>(p.whole));
  *parts = split ? static_cast<int>((tiles + chunk - 1) / chunk) : 1;
  *mbs = (q.rows * group + (1 << p.m_shift) - 1) >> p.m_shift;
  const int units = *parts * a.kv_heads;
  return *mbs * (p.swizzle ? (units + 7) & ~7 : units);
}

// The request, row block, kv head and part of the context that block `at` works on; false: none. Called
// by all lanes of a wave.
struct AttnItem {
  AttnRequest q;
  int b, mb, head, part, parts;
};

__device__ __forceinline__ bool attn_item(const verify_attention_args& a, const AttnLaunch& p, int lane, int group,
                                          int at, AttnItem* it) {
  const int B = a.n_requests;
  int blocks = 0, first = 0, n_mb = 0;
  if (B > kScanRequests) {
    it->b = wave_search(p.plan, 2, B, at, lane);
    it->q = attn_request(a, it->b);
    first = p.plan[2 * it->b];
    it->parts = p.plan[2 * it->b + 1];
    n_mb = (it->q.rows * group + (1 << p.m_shift) - 1) >> p.m_shift;
    if (n_mb == 0) return false;
  } else {
    float work = 0;
    AttnRequest q{0, 0, 0, 0};
    for (int b = lane; b < B; b += 64) {
      q = attn_request(a, b);
      work += attn_work(p, q, group);
    }
    const unsigned chunk = attn_chunk(a, p, wave_sum(work));
    int base = 0, b0 = 0;
    for (;; b0 += 64) {
      if (b0 >= B) return false;
      const int b = b0 + lane;
      if (B > 64) q = b < B ? attn_request(a, b) : AttnRequest{0, 0, 0, 0};
      int parts, mbs;
      blocks = attn_blocks(a, p, q, group, chunk, &parts, &mbs);
      const int end = base + wave_scan(blocks, lane);
      const uint64_t hit = __ballot(end > at);
      if (hit) {
        const int from = __ffsll(static_cast<unsigned long long>(hit)) - 1;
        it->b = b0 + from;
        it->q.start = __builtin_amdgcn_readlane(q.start, from);
        it->q.rows = __builtin_amdgcn_readlane(q.rows, from);
        it->q.cached = __builtin_amdgcn_readlane(q.cached, from);
        it->q.len = __builtin_amdgcn_readlane(q.len, from);
        it->parts = __builtin_amdgcn_readlane(parts, from);
        n_mb = __builtin_amdgcn_readlane(mbs, from);
        first = __builtin_amdgcn_readlane(end - blocks, from);
        break;
      }
      base = __builtin_amdgcn_readlane(end, 63);
    }
  }
  // A request's blocks in launch order: (part, head) units; with the swizzle in groups of 8, row blocks
  // in between, so that the row blocks of one unit are 8 apart and reach the same XCD (and its L2).
  int unit = at - first;
  it->mb = 0;
  if (p.swizzle) {
    const int group8 = unit / (8 * n_mb), r = unit - group8 * 8 * n_mb;
    it->mb = r >> 3;
    unit = group8 * 8 + (r & 7);
  }
  if (B <= kScanRequests && p.plan && unit == 0 && it->mb == 0 && threadIdx.x == 0) {
    p.plan[2 * it->b] = first;
    p.plan[2 * it->b + 1] = it->parts;
  }
  it->part = unit / a.kv_heads;
  it->head = unit - it->part * a.kv_heads;
  return it->part < it->parts;  // the swizzle's rounding
}

__device__ __forceinline__ int64_t attn_slot(const AttnLaunch& p, int first, int unit, int mb, int mbs) {
  return first + (p.swizzle ? (unit >> 3) * 8 * mbs + mb * 8 + (unit & 7) : unit);
}

template <typename T>
struct Mfma;
template <>
struct Mfma<__bf16> {
  typedef bf16x8 V;
  static __device__ __forceinline__ f32x16 mul(V a, V b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  // A half word's exponent bits are all set (infinity, NaN) when this step carries into its top bit.
  static constexpr uint32_t kExp = 0x7f807f80, kExpStep = 0x00800080;
  static constexpr float kLift = 0.0f;
};
template <>
struct Mfma<_Float16> {
  typedef f16x8 V;
  static __device__ __forceinline__ f32x16 mul(V a, V b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
  static constexpr uint32_t kExp = 0x7c007c00, kExpStep = 0x04000400;
  // Probabilities are held 2^7 times as large (a factor of the sums too, so it cancels): up to 2^15, below
  // the type's largest value, and 2^-21 of the running maximum still has the type's full precision.
  static constexpr float kLift = 7.0f;
};

// With the lane that holds the other half of a row's tokens.
__device__ __forceinline__ float row_max(float v) {
  const float2 a = across<32>(v);
  return fmaxf(a.x, a.y);
}
__device__ __forceinline__ float row_sum(float v) {
  const float2 a = across<32>(v);
  return a.x + a.y;
}

// Which of the four tokens at `at` .. `at` + 3 a row sees, as bits: all before `cached`, drafted ones by the
// row's mask, none from `end` on. (Arithmetic, no branches, as in all of the edge's work below: with lanes
// taking different ways there, the wide heads' kernel, which keeps part of its registers in accumulation
// registers, came out with wrong values in the lanes that had been away.)
__device__ __forceinline__ uint32_t attn_seen(int at, int cached, int end, uint64_t mask) {
  const int d = at - cached;
  const int before = min(max(-d, 0), 4);
  const uint32_t past = static_cast<uint32_t>(mask >> min(max(d, 0), 63)) & static_cast<uint32_t>((d - 64) >> 31);
  const uint32_t bits = (past << before) | ((1u << before) - 1u);
  return bits & ((1u << min(max(end - at, 0), 4)) - 1u);
}
// All bits of a word where x < y.
__device__ __forceinline__ uint32_t less_mask(int x, int y) { return static_cast<uint32_t>((x - y) >> 31); }

template <typename T, int D, int WM, int WK>
__global__ void __launch_bounds__(64 * WM * WK, D == 256 ? 1 : 2)
attn_kernel(verify_attention_args a, AttnLaunch p) {
  typedef Mfma<T> MM;
  typedef typename MM::V V8;
  constexpr int KK = D / 16;          // matrix steps along the head
  constexpr int DV = D / 32;          // value columns of a lane
  constexpr int VW = DV / 2;          // their dwords
  constexpr int MB = 32 * WM, NT = 64 * WM * WK;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int c = lane & 31, h = lane >> 5;
  const int wk = wave % WK, wm = wave / WK;
  const int group = a.heads / a.kv_heads;

  AttnItem it;
  if (!attn_item(a, p, lane, group, blockIdx.x, &it)) return;
  // Parts of equal length, whole tiles.
  const int tiles = (it.q.len + kTile - 1) / kTile;
  const int each = (tiles + it.parts - 1) / it.parts;
  const int t0 = it.part * each * kTile;
  const int t1 = min(t0 + each * kTile, it.q.len);

  f32x16 o[DV] = {};
  float mx = kNegInf, sum = 0;  // running maximum of the raw scores, sum of the lane's own probabilities
  const float sc = a.scale * 1.4426950408889634f;  // exponentials are powers of two

  const int shift = __builtin_ctz(a.page_size), in_page = a.page_size - 1;
  const int32_t* const pages = a.table + it.b * a.table_stride;
  const char* const kbase = static_cast<const char*>(a.k_cache) + it.head * a.kc_head * 2;
  const char* const vbase = static_cast<const char*>(a.v_cache) + it.head * a.vc_head * 2;
  const uint32_t k_token = static_cast<uint32_t>(a.kc_token) * 2, v_token = static_cast<uint32_t>(a.vc_token) * 2;

  // 16 tokens never cross a page. A page past the table or the cache is not read: its tokens count as
  // unseen (page 0 is read instead, and dropped).
  auto page_of = [&](int tok) {
    const int col = tok >> shift;
    const bool in = tok < t1 && col < a.width;
    const int page = pages[in ? col : 0];
    return in && page < a.n_pages ? page : -1;
  };

  // A stage: 32 tokens' keys, then their values, 2 D bytes a token. One load of a wave writes 1 KB of it,
  // lane l the 16 bytes at 16 l: whole tokens, CR lanes each.
  constexpr int CR = D / 8, RB = 2 * D, KI = D / 16;  // pieces and bytes of a token; loads of the keys
  constexpr int NI = 2 * KI / WM;                     // loads of a wave per tile
  constexpr uint32_t kStage = 2 * kTile * RB;
  constexpr int NS = WM == 1 ? 1 : WM == 2 ? 2 : 4;   // stages of a stream
  constexpr int LD = D + 4;                           // padded row of the waves' outputs, joined at the end
  constexpr uint32_t kOut = WK > 1 ? WM * WK * 32 * (LD + 2) * 4 : 0;
  __shared__ __align__(1024) char lds[WK * NS * kStage > kOut ? WK * NS * kStage : kOut];
  char* const stream = lds + wk * NS * kStage;
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) char*)stream));
  auto twist = [](int token) { return (D == 64 ? token >> 1 : token) & (CR < 16 ? CR - 1 : 15); };
  const int lr = lane / CR, lc = lane % CR;           // a load's token and piece of this lane
  // The wave's j-th load: the j WM + wm-th of a tile, whose first token is row `row` of keys or values.
  struct Part {
    bool is_k;
    int n, row;
  };
  auto part_of = [&](int j) {
    const int n = j * WM + wm;
    return Part{n < KI, n, (n < KI ? n : n - KI) * (512 / D)};
  };
  auto offset_of = [&](int j) {  // of this lane's piece from the half tile's first token
    const Part l = part_of(j);
    const uint32_t token = (l.row & 15) + lr;
    return l.is_k ? token * k_token + 16 * (lc ^ twist(token)) : token * v_token + 16 * lc;
  };
  constexpr bool kKeep = WM > 1;  // the offsets stay in registers; of a wave that has all 2 KI loads only ...
  uint32_t offset[kKeep ? NI : 1];
  if constexpr (kKeep) {
#pragma unroll
    for (int j = 0; j < NI; ++j) offset[j] = offset_of(j);
  }
  // ... the first ones, and what a load lies further on is added.
  const uint32_t k_near = lr * k_token, v_near = lr * v_token + 16 * lc;
  auto tok_of = [&](int tile) { return t0 + (tile * WK + wk) * kTile; };
  // Lane i: where the keys and values of half i % 2 of the tile i / 2 after the last multiple of 32 begin. The
  // lanes work this out for 32 tiles at a time, so that the loop waits for nothing but its tiles and has
  // no address arithmetic; halves without a page are marked.
  uint32_t k_lo = 0, k_hi = 0, v_lo = 0, v_hi = 0;
  uint64_t no_page = 0;
  auto look_up = [&](int tile) {
    const int half = tok_of(tile + (lane >> 1)) + 16 * (lane & 1);
    const int page = page_of(half);
    const int64_t pg = max(page, 0);
    const uint64_t place = half & in_page;
    const uint64_t ka = reinterpret_cast<uint64_t>(kbase) + pg * (a.kc_page * 2) + place * k_token;
    const uint64_t va = reinterpret_cast<uint64_t>(vbase) + pg * (a.vc_page * 2) + place * v_token;
    k_lo = static_cast<uint32_t>(ka), k_hi = static_cast<uint32_t>(ka >> 32);
    v_lo = static_cast<uint32_t>(va), v_hi = static_cast<uint32_t>(va >> 32);
    no_page = __ballot(page < 0);
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
  };
  auto read_base = [](uint32_t lo, uint32_t hi, int i) {
    return static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(hi, i))) << 32 |
           static_cast<uint32_t>(__builtin_amdgcn_readlane(lo, i));
  };
  uint32_t lost = 0;          // two bits a tile in flight, the one in use lowest: its halves without a page
  auto ask = [&](int tile) {  // the wave's loads of a tile
    if ((tile & 31) == 0) look_up(tile);
    const int i = 2 * (tile & 31);
    const uint32_t to = lds0 + (NS > 1 ? tile % NS * kStage : 0);
    uint64_t k0, k1, v0, v1;
    if constexpr (WM < 4) {
      k0 = read_base(k_lo, k_hi, i), k1 = read_base(k_lo, k_hi, i + 1);
      v0 = read_base(v_lo, v_hi, i), v1 = read_base(v_lo, v_hi, i + 1);
    }
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const Part l = part_of(j);
      uint64_t src;
      if constexpr (WM < 4) src = l.is_k ? (l.row < 16 ? k0 : k1) : l.row < 16 ? v0 : v1;
      else if constexpr (KI % WM == 0) src = j < NI / 2 ? read_base(k_lo, k_hi, i + (l.row >> 4)) : read_base(v_lo, v_hi, i + (l.row >> 4));
      else src = l.is_k ? read_base(k_lo, k_hi, i + (l.row >> 4)) : read_base(v_lo, v_hi, i + (l.row >> 4));
      uint32_t off;
      if constexpr (kKeep) off = offset[j];
      else off = l.is_k ? k_near + (l.row & 15) * k_token + 16 * (lc ^ twist(lr) ^ twist(l.row)) : v_near + (l.row & 15) * v_token;
      // (The wait states: a vector instruction has just written the address's scalars, and the compiler
      // does not see that this text reads them.)
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2"
                   :: "s"(to + l.n * 1024), "v"(off), "s"(src) : "memory");
    }
    lost |= (static_cast<uint32_t>(no_page >> i) & 3u) << (2 * (NS > 1 ? NS - 1 : 0));
  };

  // Tiles of the stream with the most of them: all waves of the block go round as often.
  const int all = (max(t1 - t0, 0) + kTile - 1) / kTile;
  const int rounds = (all + WK - 1) / WK, mine = (all - wk + WK - 1) / WK;
  if constexpr (NS == 1) {
    if (mine > 0) ask(0);
  } else {
#pragma unroll
    for (int i = 0; i < NS - 1; ++i) {
      if (i < mine) ask(i);
      lost >>= 2;
    }
  }
  // Query rows: row m = 32 wm + c of the block, in the order of the matrix operand.
  V8 q[KK];
  uint64_t mask;
  const int total = it.q.rows * group;
  {
    const int m = (it.mb << p.m_shift) + wm * 32 + c;
    const int mm = m < total ? m : 0;
    const int i = mm / group, hq = it.head * group + (mm - i * group);
    const T* src = static_cast<const T*>(a.q) + static_cast<int64_t>(it.q.start + i) * a.q_row + hq * a.q_head + 8 * h;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) q[kk] = *reinterpret_cast<const V8*>(src + 16 * kk);
    mask = a.masks ? static_cast<uint64_t>(a.masks[it.q.start + i]) : (uint64_t(2) << i) - 1;
    if (it.q.rows < 64) mask &= (uint64_t(1) << it.q.rows) - 1;
  }
  // Waited for here, as the compiler would in every round of the loop, and for all that is asked there too.
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)

  const int k_row = c * RB, k_twist = h ^ twist(c);
  const int v_row = kTile * RB + 4 * h * RB + 2 * DV * c;

  auto load_keys = [&](const char* at, u32x4 (&k)[KK]) {
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) k[kk] = *reinterpret_cast<const u32x4*>(at + k_row + 16 * (2 * kk ^ k_twist));
  };
  auto scores = [&](const u32x4 (&k)[KK]) {
    f32x16 s = {};
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) s = MM::mul(__builtin_bit_cast(V8, k[kk]), q[kk], s);
    return s;
  };
  // With four stages the rows are many and the matrix cores count: a tile is scored in the round before
  // its own, between the exponentials of the tile before it, which the matrix cores would else wait for.
  constexpr bool kAhead = NS == 4;
  constexpr int kWait = kAhead ? NS - 3 : NS - 2;  // tiles that may still be under way when a round begins
  f32x16 s;
  if constexpr (kAhead) {
    if (mine > 2) asm volatile("s_waitcnt vmcnt(%0)" :: "n"(2 * NI) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    asm volatile("s_barrier" ::: "memory");
    u32x4 k[KK];
    load_keys(stream, k);
    s = scores(k);
  }
  for (int tile = 0; tile < rounds; ++tile) {
    const int tok = tok_of(tile);
    if constexpr (NS == 1) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    } else {
      // The tile (scored ahead: the one after it) has arrived when at most the loads of the tiles after it are
      // still under way; every wave has also finished with the stage that is asked for next.
      if (tile + NS - 2 < mine) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" :: "n"(kWait * NI) : "memory");
      else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      asm volatile("s_barrier" ::: "memory");
      if (tile + NS - 1 < mine) ask(tile + NS - 1);
    }
    if (tile >= mine) {
      if constexpr (NS == 1) break;
      continue;
    }
    const char* const at0 = stream + (NS > 1 ? tile % NS * kStage : 0);
    u32x4 k[KK];
    if constexpr (!kAhead) load_keys(at0, k);
    uint32_t v[16][VW];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const char* const src = at0 + v_row + (8 * (j >> 2) + (j & 3)) * RB;
      if constexpr (VW == 4) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(src);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[j][e] = w[e];
      } else if constexpr (VW == 2) {
        const u32x2 w = *reinterpret_cast<const u32x2*>(src);
        v[j][0] = w[0], v[j][1] = w[1];
      } else {
        v[j][0] = *reinterpret_cast<const uint32_t*>(src);
      }
    }
    const bool lost0 = lost & 1, lost1 = lost & 2;
    lost >>= 2;
    if constexpr (NS == 1) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (tile + 1 < mine) ask(tile + 1);
    }
    if constexpr (!kAhead) s = scores(k);

    const bool edge = tok + kTile > it.q.cached || lost0 || lost1;  // some token may be unseen
    int first = tok + 4 * h;  // the lane's first token; opaque, or its sixteen tokens' numbers would be
    asm("" : "+v"(first));    // kept in registers through the loop
    bool bad = false;
    if (edge) {
      // Scores of unseen tokens are replaced, whatever they are; values of tokens that nobody may see
      // (past the end, on no page) are zeroed, and a drafted token's infinity or NaN is found, which the
      // matrix product would spread to the rows that do not see the token.
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = first + 8 * j;
        const uint32_t bits = attn_seen(at, it.q.cached, (j < 2 ? lost0 : lost1) ? at : t1, mask);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t keep = -((bits >> r) & 1);
          const float x = s[4 * j + r];
          s[4 * j + r] = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, x) & keep) | (0xff800000u & ~keep));
        }
      }
      if (tok + kTile > t1 || lost0 || lost1) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const uint32_t real = less_mask(first + 8 * (j >> 2) + (j & 3), (j < 8 ? lost0 : lost1) ? 0 : t1);
#pragma unroll
          for (int e = 0; e < VW; ++e) v[j][e] &= real;
        }
      }
      uint32_t found = 0;
#pragma unroll
      for (int j = 0; j < 16; ++j)
#pragma unroll
        for (int e = 0; e < VW; ++e) found |= (v[j][e] & MM::kExp) + MM::kExpStep;
      bad = __ballot((found & 0x80008000u) != 0) != 0;
      if (bad) {  // keep the drafted tokens' out of the product
#pragma unroll
        for (int j = 0; j < 16; ++j)
#pragma unroll
          for (int e = 0; e < VW; ++e) {
            const uint32_t w = v[j][e];
            const uint32_t x = (w & MM::kExp) + MM::kExpStep;
            const uint32_t wrong = ((x >> 15) & 0x00010001u) * 0xffffu;  // the halves that are no number
            v[j][e] = w & ~(wrong & ~less_mask(first + 8 * (j >> 2) + (j & 3), it.q.cached));
          }
      }
    }
    // Probabilities relative to a running maximum that a row raises only when its own grows by more than
    // 8 powers of two: until then p <= 2^8, which both 16-bit types hold with their full precision. (Each
    // row by itself: its result does not depend on the other rows' values.)
    float top = fmaxf(fmaxf(s[0], s[1]), s[2]);
#pragma unroll
    for (int r = 3; r < 15; r += 2) top = fmaxf(fmaxf(top, s[r]), s[r + 1]);
    top = row_max(fmaxf(top, s[15]));
    const bool up = (top - mx) * sc > 8.0f;  // also from -inf; not for NaN (-inf after -inf)
    if (__ballot(up)) {
      const float f = up ? __builtin_amdgcn_exp2f((mx - top) * sc) : 1.0f;
      mx = up ? top : mx;
      sum *= f;
#pragma unroll
      for (int i = 0; i < DV; ++i) o[i] *= f;
    }
    const float ref = (mx == kNegInf ? 0.0f : mx * sc) - MM::kLift;
    V8 pt[2];
    {
      f32x16 e;
      float part[2] = {0, 0};
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        e[r] = __builtin_amdgcn_exp2f(fmaf(s[r], sc, -ref));
        part[r & 1] += e[r];
      }
      sum += part[0] + part[1];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        f32x8 half;
#pragma unroll
        for (int j = 0; j < 8; ++j) half[j] = e[8 * w + j];
        pt[w] = __builtin_convertvector(half, V8);
      }
    }
    if constexpr (kAhead) {  // (past the wave's last tile: of whatever the stage holds, for nothing)
      u32x4 k[KK];
      load_keys(stream + (tile + 1) % NS * kStage, k);
      s = scores(k);
    }
    // V^T: a column of the lane's, its eight tokens of a matrix step.
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        u32x4 lo, hi;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w0 = v[8 * w + 2 * j][e], w1 = v[8 * w + 2 * j + 1][e];
          lo[j] = __builtin_amdgcn_perm(w1, w0, 0x05040100);
          hi[j] = __builtin_amdgcn_perm(w1, w0, 0x07060302);
        }
        o[2 * e] = MM::mul(__builtin_bit_cast(V8, lo), pt[w], o[2 * e]);
        o[2 * e + 1] = MM::mul(__builtin_bit_cast(V8, hi), pt[w], o[2 * e + 1]);
      }
    if (bad) {
      // The infinities and NaN left out above, token by token, added to the rows that see the token.
#pragma unroll 1
      for (int t = 0; t < kTile; ++t) {
        const int d = tok + t - it.q.cached;
        if (d < 0 || d >= 64 || (t < 16 ? lost0 : lost1) || tok + t >= t1) continue;
        const T* vp = reinterpret_cast<const T*>(vbase + page_of(tok + t) * (a.vc_page * 2) +
                                                 static_cast<uint64_t>((tok + t) & in_page) * v_token);
        float pr = 0;  // this row's probability of the token, from the lane that holds it
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float x = __shfl(static_cast<float>(pt[j >> 3][j & 7]), ((t >> 2) & 1) * 32 + c);
          if ((t >> 3) * 4 + (t & 3) == j) pr = x;
        }
        const bool seen = (mask >> d) & 1;
#pragma unroll
        for (int i = 0; i < DV; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const float x = static_cast<float>(vp[DV * (8 * (r >> 2) + 4 * h + (r & 3)) + i]);
            const uint32_t add = -static_cast<uint32_t>(seen & !(fabsf(x) < __builtin_inff()));
            o[i][r] += __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, pr * x) & add);
          }
      }
    }
  }
  sum = row_sum(sum);

  // Join the waves that shared rows, through LDS, and store: the output of a request in one part, or
  // this part's output, maximum and sum.
  const bool whole = it.parts == 1;
  const int64_t slot = blockIdx.x;
  float* const part_o = p.part + slot * MB * D;
  float* const part_ml = p.part + static_cast<int64_t>(p.grid) * MB * D + slot * MB * 2;
  constexpr int SV = DV < 4 ? DV : 4;  // columns stored at a time
  typedef float FV __attribute__((ext_vector_type(SV)));
  typedef T TV __attribute__((ext_vector_type(SV)));
  // where row m of the block goes: the output, or the part
  auto out_of = [&](int m) {
    const int row = (it.mb << p.m_shift) + m, i = row / group;
    return static_cast<T*>(a.out) + static_cast<int64_t>(it.q.start + i) * a.o_row +
           (it.head * group + (row - i * group)) * a.o_head;
  };
  if constexpr (WK == 1) {
    const int m = wm * 32 + c;
    if ((it.mb << p.m_shift) + m >= total) return;
    const float inv = whole ? (sum == 0 ? 0.0f : 1.0f / sum) : 1.0f;
    T* const dst = whole ? out_of(m) : nullptr;
#pragma unroll
    for (int r = 0; r < 16; ++r)
#pragma unroll
      for (int i0 = 0; i0 < DV; i0 += SV) {
        const int col = DV * (8 * (r >> 2) + 4 * h + (r & 3)) + i0;
        FV x;
#pragma unroll
        for (int i = 0; i < SV; ++i) x[i] = o[i0 + i][r] * inv;
        if (whole) *reinterpret_cast<TV*>(dst + col) = __builtin_convertvector(x, TV);
        else *reinterpret_cast<FV*>(part_o + m * D + col) = x;
      }
    if (!whole && h == 0) {
      part_ml[2 * m] = mx;
      part_ml[2 * m + 1] = sum;
    }
  } else {
    // over the stages, once every wave is through with them
    float (*const so)[32][LD] = reinterpret_cast<float (*)[32][LD]>(lds);
    float (*const sml)[32][2] = reinterpret_cast<float (*)[32][2]>(lds + WM * WK * 32 * LD * 4);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 16; ++r)
#pragma unroll
      for (int i0 = 0; i0 < DV; i0 += SV) {
        FV x;
#pragma unroll
        for (int i = 0; i < SV; ++i) x[i] = o[i0 + i][r];
        *reinterpret_cast<FV*>(&so[wave][c][DV * (8 * (r >> 2) + 4 * h + (r & 3)) + i0]) = x;
      }
    if (h == 0) {
      sml[wave][c][0] = mx;
      sml[wave][c][1] = sum;
    }
    __syncthreads();
    constexpr int CH = D / SV;  // pieces of a row
    const int rows = min(MB, total - (it.mb << p.m_shift));
    for (int e = threadIdx.x; e < rows * CH; e += NT) {
      const int m = e / CH, col = (e % CH) * SV;
      const int w0 = m / 32 * WK, mw = m % 32;
      float top = kNegInf;
#pragma unroll
      for (int w = 0; w < WK; ++w) top = fmaxf(top, sml[w0 + w][mw][0]);
      FV x = {};
      float l = 0;
#pragma unroll
      for (int w = 0; w < WK; ++w) {
        const float mw_max = sml[w0 + w][mw][0];
        const float f = mw_max == kNegInf ? 0.0f : __builtin_amdgcn_exp2f((mw_max - top) * sc);
        // A wave that saw nothing holds zeros (or NaN) only, and no maximum.
        x += *reinterpret_cast<const FV*>(&so[w0 + w][mw][col]) * (mw_max == kNegInf ? 1.0f : f);
        l += sml[w0 + w][mw][1] * (mw_max == kNegInf ? 1.0f : f);
      }
      if (whole) x *= l == 0 ? 0.0f : 1.0f / l;
      if (whole) *reinterpret_cast<TV*>(out_of(m) + col) = __builtin_convertvector(x, TV);
      else *reinterpret_cast<FV*>(part_o + m * D + col) = x;
      if (!whole && col == 0) {
        part_ml[2 * m] = top;
        part_ml[2 * m + 1] = l;
      }
    }
  }
}

// Joins the parts of a (row, head), one wave each: lane i first takes part i's maximum and sum, then the
// wave's halves take every other part's output, D / 32 values a lane: sixteen parts at once, or the last eight
// (one row of 16 heads, 128 parts: 6.2 us, always eight 7.7; 32 at once 5.8, but 10.1 instead of 8.8 with 8192
// rows of few parts, which miss the registers). Rows of requests in one part are stored already.
template <typename T, int D>
__global__ void __launch_bounds__(256) attn_join_kernel(verify_attention_args a, AttnLaunch p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int id = blockIdx.x * 4 + wave;
  const int t = id / a.heads, hq = id - t * a.heads;
  if (t >= a.n_rows) return;
  int b = -1, start = 0, rows = 0;
  if (a.n_requests > kScanRequests) {
    const int x = wave_search(a.row_start, 1, a.n_requests, t, lane);
    const AttnRequest q = attn_request(a, x);
    if (t >= q.start && t < q.start + q.rows) b = x, start = q.start, rows = q.rows;
  }
  for (int b0 = 0; b0 < (a.n_requests > kScanRequests ? 0 : a.n_requests) && b < 0; b0 += 64) {
    const int x = b0 + lane;
    AttnRequest q{0, 0, 0, 0};
    if (x < a.n_requests) q = attn_request(a, x);
    const uint64_t hit = __ballot(t >= q.start && t < q.start + q.rows);
    if (hit) {
      const int from = __ffsll(static_cast<unsigned long long>(hit)) - 1;
      b = b0 + from;
      start = __builtin_amdgcn_readlane(q.start, from);
      rows = __builtin_amdgcn_readlane(q.rows, from);
    }
  }
  if (b < 0) return;
  const int first = p.plan[2 * b], parts = p.plan[2 * b + 1];
  if (parts == 1) return;
  const int group = a.heads / a.kv_heads, kvh = hq / group;
  const int m_all = (t - start) * group + (hq - kvh * group);
  const int mb = m_all >> p.m_shift, m = m_all - (mb << p.m_shift);
  const int mbs = (rows * group + (1 << p.m_shift) - 1) >> p.m_shift;
  const float sc = a.scale * 1.4426950408889634f;
  const float* const ml = p.part + (static_cast<int64_t>(p.grid) << p.m_shift) * D;
  auto part = [&](int i) { return (attn_slot(p, first, i * a.kv_heads + kvh, mb, mbs) << p.m_shift) + m; };
  const int h = lane >> 5, c = lane & 31;
  typedef float FV __attribute__((ext_vector_type(E)));
  FV o = {};
  float l = 0, mx = kNegInf;
  for (int i0 = 0; i0 < parts; i0 += 64) {
    float pm = kNegInf, pl = 0;
    if (i0 + lane < parts) {
      const int64_t at = part(i0 + lane);
      pm = ml[2 * at];
      pl = ml[2 * at + 1];
    }
    const float top = fmaxf(mx, wave_max(pm));
    const float ref = top == kNegInf ? 0.0f : top;
    const float back = mx == kNegInf ? 1.0f : __builtin_amdgcn_exp2f((mx - ref) * sc);  // what is there so far
    // a part that saw nothing holds zeros (or NaN)
    const float f = pm == kNegInf ? 1.0f : __builtin_amdgcn_exp2f((pm - ref) * sc);
    mx = top;
    l = l * back + wave_sum(pl * f);
    o *= back;
    const int n = min(64, parts - i0);
    auto add = [&](int i, auto wide) {  // so many parts a half wave, asked for at once
      constexpr int U = decltype(wide)::value;
      FV x[U];
      float w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = min(i + 2 * u + h, n - 1);
        x[u] = *reinterpret_cast<const FV*>(p.part + part(i0 + at) * D + E * c);
        w[u] = __shfl(f, at);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + 2 * u + h < n) o += x[u] * w[u];
    };
    int i = 0;
    for (; n - i > 8; i += 16) add(i, std::integral_constant<int, 8>{});
    if (i < n) add(i, std::integral_constant<int, 4>{});
  }
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = row_sum(o[e]);
  const float inv = l == 0 ? 0.0f : 1.0f / l;
  if (h) return;
  T* dst = static_cast<T*>(a.out) + static_cast<int64_t>(t) * a.o_row + hq * a.o_head + E * c;
  typedef T TV __attribute__((ext_vector_type(E)));
  TV x;
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = static_cast<T>(o[e] * inv);
  *reinterpret_cast<TV*>(dst) = x;
}

// Waves along the rows of a block, by the most query rows a (request, kv head) can have. A block has 8
// waves, as many as a CU holds at the kernel's registers; 4 with 256 values a head. (From 256 rows on eight
// against four, each with two streams of tokens: 4 requests of 512 rows over up to 16384 tokens 90, 94 us; one
// of 384 rows over 131071 194, 254; 32 of 256 rows over up to 2048 155, 139.)
inline int attn_wm(const verify_attention_args& a) {
  const int m = a.max_rows * (a.heads / a.kv_heads), most = a.dim == 256 ? 4 : 8;
  int wm = 1;
  while (wm < most && 32 * wm < m) wm *= 2;
  return wm;
}

// The grid and the workspace of a call; false if a launch would reach 2^32 threads.
inline bool attn_plan(const verify_attention_args& a, AttnLaunch* p, int64_t* bytes) {
  const int m = a.max_rows * (a.heads / a.kv_heads), rows = 32 * attn_wm(a);
  const int64_t per_request = (m + rows - 1) / rows;
  p->m_shift = __builtin_ctz(rows);
  const int wk = (a.dim == 256 ? 4 : 8) / (rows / 32);
  p->least = kMinTiles * wk;
  p->whole = kSplitTiles * wk;
  p->swizzle = per_request > 1;
  // Each (row block, head) rounds up to a whole number of parts, so the call makes up to `once` blocks more
  // than the target. While that leaves room, all blocks fit the chip at once; with more, the target is
  // twice what the chip holds: smaller parts even the blocks out but write and join more partial outputs
  // (once, twice, four times, both kernels, us: 32 requests of 8 rows, up to 8192 tokens, 8 kv heads 166,
  // 162, 165; 40 of 32 rows, 4096 tokens 157, 152, 168; 48 of one row, 8192 tokens 233, 222, 218).
  const int64_t row_blocks = static_cast<int64_t>(a.n_requests) * per_request, once = row_blocks * a.kv_heads;
  p->target = static_cast<int32_t>(once <= kCus / 2 ? kCus - once : 2 * kCus);
  const int64_t grid = p->target + once + (p->swizzle ? 7 * row_blocks : 0) + 8;
  constexpr int64_t kThreads = UINT32_MAX;
  if (grid > kThreads / 512) return false;
  p->grid = static_cast<int32_t>(grid);
  p->part = nullptr;
  p->plan = nullptr;
  // A table that holds no more than that never splits.
  const bool split = static_cast<int64_t>(a.width) * a.page_size > p->whole * kTile;
  if (split && (static_cast<int64_t>(a.n_rows) * a.heads + 3) / 4 > kThreads / 256) return false;
  p->split = split;
  *bytes = split ? grid * rows * (a.dim + 2) * 4 : 0;
  if (split || a.n_requests > kScanRequests) *bytes += a.n_requests * 8;
  return true;
}

inline void attn_workspace(const verify_attention_args& a, AttnLaunch* p, void* workspace) {
  p->part = static_cast<float*>(workspace);
  p->plan = reinterpret_cast<int32_t*>(p->part + (p->split ? (static_cast<int64_t>(p->grid) << p->m_shift) * (a.dim + 2) : 0));
}

template <typename T, int D>
hipError_t launch_attention_d(const verify_attention_args& a, const AttnLaunch& p, hipStream_t stream) {
  constexpr int W = D == 256 ? 4 : 8;
  const dim3 grid(p.grid), block(64 * W);
  switch (attn_wm(a)) {
    case 1: attn_kernel<T, D, 1, W><<<grid, block, 0, stream>>>(a, p); break;
    case 2: attn_kernel<T, D, 2, W / 2><<<grid, block, 0, stream>>>(a, p); break;
    case 4: attn_kernel<T, D, 4, W / 4><<<grid, block, 0, stream>>>(a, p); break;
    default:
      if constexpr (D != 256) attn_kernel<T, D, 8, 1><<<grid, block, 0, stream>>>(a, p);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !p.split) return e;
  const int64_t waves = static_cast<int64_t>(a.n_rows) * a.heads;
  attn_join_kernel<T, D><<<dim3(static_cast<unsigned>((waves + 3) / 4)), dim3(256), 0, stream>>>(a, p);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_attention(const verify_attention_args& a, const AttnLaunch& p, hipStream_t stream) {
  switch (a.dim) {
    case 64: return launch_attention_d<T, 64>(a, p, stream);
    case 128: return launch_attention_d<T, 128>(a, p, stream);
    default: return launch_attention_d<T, 256>(a, p, stream);
  }
}

extern template hipError_t launch_attention<__bf16>(const verify_attention_args&, const AttnLaunch&, hipStream_t);
extern template hipError_t launch_attention<_Float16>(const verify_attention_args&, const AttnLaunch&, hipStream_t);

}  // namespace verify
