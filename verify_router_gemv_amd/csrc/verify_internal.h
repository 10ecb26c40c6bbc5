// Host-only checks of the verify-round operators' arguments (no HIP: tested without a GPU).
#pragma once

#include "verify_ops.h"

namespace verify {

moe_status validate_slots(const verify_slots_args* a);
moe_status validate_rope(const verify_rope_args* a);
moe_status validate_attention(const verify_attention_args* a);
moe_status validate_logprobs(const verify_logprobs_args* a);

}  // namespace verify
