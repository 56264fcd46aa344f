// Prompt attention over 16-bit pages and the 4-bit pool: launches of
// prompt_kernel.h.
#include "context/prompt_kernel.h"

namespace pkv {
namespace {

template <int D, bool BF16>
pkv_status launch_fmt(bool kv4, const PromptArgs& a, hipStream_t s) {
  return kv4 ? launch_prompt_kernel<D, BF16, Cache::k4, false>(a, s)
             : launch_prompt_kernel<D, BF16, Cache::k16, false>(a, s);
}

}  // namespace

pkv_status launch_prompt(const pkv_problem& p, bool kv4, const PromptArgs& a, hipStream_t s) {
  const bool bf = p.dtype == PKV_BF16;
  if (p.head_dim == 128)
    return bf ? launch_fmt<128, true>(kv4, a, s) : launch_fmt<128, false>(kv4, a, s);
  return bf ? launch_fmt<64, true>(kv4, a, s) : launch_fmt<64, false>(kv4, a, s);
}

}  // namespace pkv
