// Cross attention of many queries a row: launches of prompt_kernel.h.
#include "context/prompt_kernel.h"
#include "serving/serving_internal.h"

namespace pkv {
namespace {

template <int D, bool BF16>
pkv_status launch_kind(Cache kind, const PromptArgs& a, hipStream_t s) {
  switch (kind) {
    case Cache::k16: return launch_prompt_shares<D, BF16, Cache::k16, true>(a, s);
    case Cache::k4: return launch_prompt_shares<D, BF16, Cache::k4, true>(a, s);
    default: return launch_prompt_shares<D, BF16, Cache::k8, true>(a, s);
  }
}

}  // namespace

pkv_status launch_cross_many(const pkv_problem& p, Cache kind, const PromptArgs& a,
                             hipStream_t s) {
  const bool bf = p.dtype == PKV_BF16;
  if (p.head_dim == 128)
    return bf ? launch_kind<128, true>(kind, a, s) : launch_kind<128, false>(kind, a, s);
  return bf ? launch_kind<64, true>(kind, a, s) : launch_kind<64, false>(kind, a, s);
}

}  // namespace pkv
