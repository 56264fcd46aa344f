// Prompt attention over the 8-bit pool: launches of prompt_kernel.h.
#include "context/prompt_kernel.h"
#include "serving/serving_internal.h"

namespace pkv {

pkv_status launch_prompt8(const pkv_problem& p, const PromptArgs& a, hipStream_t s) {
  const bool bf = p.dtype == PKV_BF16;
  if (p.head_dim == 128)
    return bf ? launch_prompt_shares<128, true, Cache::k8, false>(a, s)
              : launch_prompt_shares<128, false, Cache::k8, false>(a, s);
  return bf ? launch_prompt_shares<64, true, Cache::k8, false>(a, s)
            : launch_prompt_shares<64, false, Cache::k8, false>(a, s);
}

}  // namespace pkv
