// Cross attention of few queries a row, sixteen packed together: launches of
// attend_kernel.h.
#include "context/attend_kernel.h"
#include "serving/serving_internal.h"

namespace pkv {
namespace {

template <int D, bool BF16>
void launch_kind(Cache kind, int64_t tiles, const AttendArgs& a, hipStream_t s) {
  const dim3 grid(a.num_kv_heads, a.splits, static_cast<uint32_t>(tiles));
  if (kind == Cache::k16)
    hipLaunchKernelGGL((attend_kernel<D, BF16, Cache::k16, true, 16, 4, 1, 1>), grid, dim3(256),
                       0, s, a);
  else if (kind == Cache::k4)
    hipLaunchKernelGGL((attend_kernel<D, BF16, Cache::k4, true, 16, 4, 2, 2>), grid, dim3(256), 0,
                       s, a);
  else
    hipLaunchKernelGGL((attend_kernel<D, BF16, Cache::k8, true, 16, 4, 1, 2>), grid, dim3(256), 0,
                       s, a);
}

}  // namespace

pkv_status launch_cross_few(const pkv_problem& p, Cache kind, int64_t tiles,
                            const AttendArgs& args, hipStream_t s) {
  AttendArgs a = args;
  if (a.splits > 1 && (a.cus = current_compute_units()) <= 0) return PKV_EHIP;
  const bool bf = p.dtype == PKV_BF16;
  if (p.head_dim == 128) {
    if (bf) launch_kind<128, true>(kind, tiles, a, s);
    else launch_kind<128, false>(kind, tiles, a, s);
  } else {
    if (bf) launch_kind<64, true>(kind, tiles, a, s);
    else launch_kind<64, false>(kind, tiles, a, s);
  }
  return hipGetLastError() == hipSuccess ? PKV_OK : PKV_EHIP;
}

}  // namespace pkv
