// Tree attention over float16 caches.
#include "verify_attention.h"
namespace verify {
template hipError_t launch_attention<_Float16>(const verify_attention_args&, const AttnLaunch&, hipStream_t);
}  // namespace verify
