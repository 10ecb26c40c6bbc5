// The C entries of the verify-round operators: checks, launch shapes, launches.
#include "verify_attention_cut.h"
#include "verify_internal.h"
#include "verify_logprobs.h"
#include "verify_rope.h"
#include "verify_slots.h"

using namespace verify;

static thread_local int32_t g_last_hip = 0;

static moe_status hip_status(hipError_t e) {
  if (e == hipSuccess) return MOE_OK;
  g_last_hip = static_cast<int32_t>(e);
  return MOE_ERR_HIP;
}

// A workspace of at least `need` bytes, 16-byte aligned (none is needed for 0).
static bool workspace_ok(const void* p, int64_t have, int64_t need) {
  return need == 0 || (p && have >= need && (reinterpret_cast<uintptr_t>(p) & 15u) == 0);
}

extern "C" moe_status verify_round_slots(const verify_slots_args* a, void* stream) {
  const moe_status st = validate_slots(a);
  if (st != MOE_OK) return st;
  return hip_status(launch_slots(*a, static_cast<hipStream_t>(stream)));
}

extern "C" moe_status verify_qk_norm_rope(const verify_rope_args* a, void* stream) {
  const moe_status st = validate_rope(a);
  if (st != MOE_OK || a->n_rows == 0) return st;
  return hip_status(launch_rope(*a, static_cast<hipStream_t>(stream)));
}

extern "C" int64_t verify_tree_attention_workspace(const verify_attention_args* a) {
  const moe_status st = validate_attention(a);
  if (st != MOE_OK) return st;
  if (a->n_rows == 0 || a->n_requests == 0) return 0;
  AttnLaunch p;
  int64_t bytes = 0;
  return attn_plan(*a, &p, &bytes) ? bytes : MOE_ERR_UNSUPPORTED;
}

extern "C" moe_status verify_tree_attention(const verify_attention_args* a, void* workspace, int64_t workspace_bytes,
                                            void* stream) {
  const moe_status st = validate_attention(a);
  if (st != MOE_OK || a->n_rows == 0 || a->n_requests == 0) return st;
  AttnLaunch p;
  int64_t bytes = 0;
  if (!attn_plan(*a, &p, &bytes)) return MOE_ERR_UNSUPPORTED;
  if (!workspace_ok(workspace, workspace_bytes, bytes)) return MOE_ERR_INVALID_ARG;
  if (bytes) attn_workspace(*a, &p, workspace);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (a->n_requests > kScanRequests) {
    const hipError_t e = launch_attn_cut(*a, p, s);
    if (e != hipSuccess) return hip_status(e);
  }
  return hip_status(a->type == VERIFY_BF16 ? launch_attention<__bf16>(*a, p, s) : launch_attention<_Float16>(*a, p, s));
}

extern "C" int64_t verify_token_logprobs_workspace(const verify_logprobs_args* a) {
  const moe_status st = validate_logprobs(a);
  if (st != MOE_OK) return st;
  int64_t bytes = 0;
  if (a->n_rows) lp_plan(*a, nullptr, &bytes);
  return bytes;
}

extern "C" moe_status verify_token_logprobs(const verify_logprobs_args* a, void* workspace, int64_t workspace_bytes,
                                            void* stream) {
  const moe_status st = validate_logprobs(a);
  if (st != MOE_OK || a->n_rows == 0) return st;
  int64_t bytes = 0;
  const LpPlan p = lp_plan(*a, workspace, &bytes);
  if (!workspace_ok(workspace, workspace_bytes, bytes)) return MOE_ERR_INVALID_ARG;
  return hip_status(launch_logprobs(*a, p, static_cast<hipStream_t>(stream)));
}

extern "C" int32_t verify_last_hip_error(void) { return g_last_hip; }
