// Host-only validation of the verify-round operators' arguments. Kept free of HIP so that it runs (and
// is tested) on a machine without a GPU.
#include "verify_internal.h"

#include <math.h>

namespace verify {

static bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
static bool good(const void* p, unsigned n) { return p && aligned(p, n); }
static int size_of(int type) { return type == VERIFY_F32 ? 4 : 2; }
static bool type16(int t) { return t == VERIFY_BF16 || t == VERIFY_F16; }
static bool dim_ok(int d) { return d == 64 || d == 128 || d == 256; }

// A stride (in elements) that keeps 16-byte alignment and lies in the range the kernels multiply in.
static bool stride_ok(int64_t s, int size, int64_t most) { return s >= 0 && s <= most && (s * size) % 16 == 0; }
// A written tensor's elements must not share memory: no dimension of several elements has stride 0.
static bool apart(int64_t s, int64_t n) { return s > 0 || n <= 1; }
constexpr int64_t kWide = int64_t(1) << 40;   // rows, heads and pages: 64-bit products
constexpr int64_t kNear = int64_t(1) << 24;   // tokens of a page: 32-bit products with up to 15

// An output over the queries: the same elements, or none.
static bool over_ok(const void* q, int q_type, int64_t q_row, int64_t q_head, const void* out, int o_type, int64_t o_row,
                    int64_t o_head, int64_t rows, int64_t heads, int64_t dim) {
  const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), o0 = reinterpret_cast<uintptr_t>(out);
  if (q0 == o0) return q_type == o_type && q_row == o_row && q_head == o_head;
  const uintptr_t q1 = q0 + ((rows - 1) * q_row + (heads - 1) * q_head + dim) * size_of(q_type);
  const uintptr_t o1 = o0 + ((rows - 1) * o_row + (heads - 1) * o_head + dim) * size_of(o_type);
  return q0 >= o1 || o0 >= q1;
}

moe_status validate_slots(const verify_slots_args* a) {
  if (!a || a->struct_bytes != static_cast<int64_t>(sizeof(*a)) || a->reserved) return MOE_ERR_INVALID_ARG;
  if (a->n_requests < 0 || a->width < 1 || a->n_free < 0 || a->page_size < 1 || a->total_rows < 0 ||
      a->table_stride < a->width)
    return MOE_ERR_INVALID_ARG;
  if (a->n_requests > VERIFY_MAX_REQUESTS || a->page_size > 65536 || a->total_rows > VERIFY_MAX_TOTAL_ROWS ||
      a->table_stride > kWide)
    return MOE_ERR_UNSUPPORTED;
  if ((a->parents != nullptr) != (a->masks != nullptr)) {
    // an empty tensor has no address
    if (a->total_rows > 0) return MOE_ERR_INVALID_ARG;
  }
  if (!good(a->row_start, 4) || !good(a->counts, 4)) return MOE_ERR_INVALID_ARG;
  if (a->n_requests > 0 && (!good(a->cached, 4) || !good(a->rows, 4) || !good(a->table, 4))) return MOE_ERR_INVALID_ARG;
  if (a->total_rows > 0 && (!good(a->slots, 4) || !good(a->positions, 4))) return MOE_ERR_INVALID_ARG;
  if (a->n_free > 0 && !good(a->free_pages, 4)) return MOE_ERR_INVALID_ARG;
  if (!aligned(a->free_head, 4) || !aligned(a->parents, 4) || !aligned(a->masks, 8)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status validate_rope(const verify_rope_args* a) {
  if (!a || a->struct_bytes != static_cast<int64_t>(sizeof(*a))) return MOE_ERR_INVALID_ARG;
  if (a->n_rows < 0 || a->heads < 1 || a->kv_heads < 1 || a->page_size < 1 || a->n_pages < 1 || a->n_freq < 0 ||
      !(a->eps >= 0) || isinf(a->eps) || (a->interleaved != 0 && a->interleaved != 1))
    return MOE_ERR_INVALID_ARG;
  if (!type16(a->cache_type) || (a->in_type != a->cache_type && a->in_type != VERIFY_F32)) return MOE_ERR_UNSUPPORTED;
  if (!dim_ok(a->dim) || a->n_freq % 8 || 2 * a->n_freq > a->dim) return MOE_ERR_UNSUPPORTED;
  if (a->heads > 1024 || a->kv_heads > 1024 || a->n_rows > VERIFY_MAX_TOTAL_ROWS || a->n_pages > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  const int in = size_of(a->in_type), out = 2;
  if (!stride_ok(a->q_row, in, kWide) || !stride_ok(a->q_head, in, kWide) || !stride_ok(a->k_row, in, kWide) ||
      !stride_ok(a->k_head, in, kWide) || !stride_ok(a->v_row, in, kWide) || !stride_ok(a->v_head, in, kWide) ||
      !stride_ok(a->o_row, out, kWide) || !stride_ok(a->o_head, out, kWide) || !stride_ok(a->kc_page, out, kWide) ||
      !stride_ok(a->kc_head, out, kWide) || !stride_ok(a->kc_token, out, kNear) ||
      !stride_ok(a->vc_page, out, kWide) || !stride_ok(a->vc_head, out, kWide) || !stride_ok(a->vc_token, out, kNear))
    return MOE_ERR_INVALID_ARG;
  if (!apart(a->o_row, a->n_rows) || !apart(a->o_head, a->heads) || !apart(a->kc_page, a->n_pages) ||
      !apart(a->kc_head, a->kv_heads) || !apart(a->kc_token, a->page_size) || !apart(a->vc_page, a->n_pages) ||
      !apart(a->vc_head, a->kv_heads) || !apart(a->vc_token, a->page_size))
    return MOE_ERR_INVALID_ARG;
  if (a->n_rows == 0) return MOE_OK;
  if (!good(a->q, 16) || !good(a->k, 16) || !good(a->v, 16) || !good(a->q_out, 16) || !good(a->k_cache, 16) ||
      !good(a->v_cache, 16) || !good(a->positions, 4) || !good(a->slots, 4) || !aligned(a->q_weight, 16) ||
      !aligned(a->k_weight, 16) || (a->n_freq > 0 && !good(a->inv_freq, 4)))
    return MOE_ERR_INVALID_ARG;
  if (!over_ok(a->q, a->in_type, a->q_row, a->q_head, a->q_out, a->cache_type, a->o_row, a->o_head, a->n_rows, a->heads,
               a->dim))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status validate_attention(const verify_attention_args* a) {
  if (!a || a->struct_bytes != static_cast<int64_t>(sizeof(*a))) return MOE_ERR_INVALID_ARG;
  if (a->n_rows < 0 || a->n_requests < 0 || a->heads < 1 || a->kv_heads < 1 || a->heads % a->kv_heads ||
      a->width < 1 || a->n_pages < 1 || a->max_rows < 1 || a->table_stride < a->width || a->page_size < 1 ||
      !(a->scale > 0) || isinf(a->scale))
    return MOE_ERR_INVALID_ARG;
  if (!type16(a->type) || !dim_ok(a->dim)) return MOE_ERR_UNSUPPORTED;
  if (a->page_size < 16 || a->page_size > 65536 || (a->page_size & (a->page_size - 1))) return MOE_ERR_UNSUPPORTED;
  // token numbers and a few tiles behind the last stay within 31 bits
  if (static_cast<int64_t>(a->width) * a->page_size > (int64_t(1) << 30)) return MOE_ERR_UNSUPPORTED;
  if (a->max_rows > VERIFY_MAX_TREE_ROWS || a->heads / a->kv_heads > 64 || a->heads > 1024 ||
      a->n_requests > VERIFY_MAX_REQUESTS || a->n_rows > VERIFY_MAX_TOTAL_ROWS || a->n_pages > INT32_MAX ||
      a->table_stride > kWide)
    return MOE_ERR_UNSUPPORTED;
  if (!stride_ok(a->q_row, 2, kWide) || !stride_ok(a->q_head, 2, kWide) || !stride_ok(a->o_row, 2, kWide) ||
      !stride_ok(a->o_head, 2, kWide) || !stride_ok(a->kc_page, 2, kWide) || !stride_ok(a->kc_head, 2, kWide) ||
      !stride_ok(a->kc_token, 2, kNear) || !stride_ok(a->vc_page, 2, kWide) || !stride_ok(a->vc_head, 2, kWide) ||
      !stride_ok(a->vc_token, 2, kNear))
    return MOE_ERR_INVALID_ARG;
  if (!apart(a->o_row, a->n_rows) || !apart(a->o_head, a->heads)) return MOE_ERR_INVALID_ARG;
  if (a->n_rows == 0 || a->n_requests == 0) return MOE_OK;
  if (!good(a->q, 16) || !good(a->out, 16) || !good(a->k_cache, 16) || !good(a->v_cache, 16) || !good(a->table, 4) ||
      !good(a->cached, 4) || !good(a->row_start, 4) || !aligned(a->masks, 8))
    return MOE_ERR_INVALID_ARG;
  if (!over_ok(a->q, a->type, a->q_row, a->q_head, a->out, a->type, a->o_row, a->o_head, a->n_rows, a->heads, a->dim))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status validate_logprobs(const verify_logprobs_args* a) {
  if (!a || a->struct_bytes != static_cast<int64_t>(sizeof(*a))) return MOE_ERR_INVALID_ARG;
  if (a->n_rows < 0 || a->vocab < 1 || a->n_tokens < 0 || a->top < 0 || a->row_stride < 0 ||
      (a->n_rows > 1 && a->row_stride < a->vocab) || (a->tokens_64 != 0 && a->tokens_64 != 1) || a->top > a->vocab)
    return MOE_ERR_INVALID_ARG;
  if (a->type != VERIFY_F32 && !type16(a->type)) return MOE_ERR_UNSUPPORTED;
  if (a->top > VERIFY_MAX_ALTERNATIVES || a->n_rows > VERIFY_MAX_TOTAL_ROWS || a->vocab > (1 << 30) ||
      a->row_stride > kWide)
    return MOE_ERR_UNSUPPORTED;
  if (a->n_rows == 0) return MOE_OK;
  if (!good(a->logits, size_of(a->type)) || !aligned(a->entropy, 4)) return MOE_ERR_INVALID_ARG;
  if (a->n_tokens > 0 && (!good(a->tokens, a->tokens_64 ? 8 : 4) || !good(a->logprobs, 4))) return MOE_ERR_INVALID_ARG;
  if (a->top > 0 && (!good(a->top_ids, 4) || !good(a->top_logprobs, 4))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace verify
