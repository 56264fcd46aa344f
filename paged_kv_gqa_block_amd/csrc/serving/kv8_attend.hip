// Decode attention over the 8-bit pool: launches of attend_kernel.h.
#include "context/attend_kernel.h"
#include "serving/serving_internal.h"

namespace pkv {
namespace {

template <int D, bool BF16, int GP>
void launch_one(const AttendArgs& a, hipStream_t s) {
  const dim3 grid(a.num_kv_heads, a.splits, a.batch);
  hipLaunchKernelGGL((attend_kernel<D, BF16, Cache::k8, false, GP, 4, 1, 2>), grid, dim3(256), 0,
                     s, a);
}

template <int D, bool BF16>
void launch_gp(const AttendArgs& a, hipStream_t s) {
  if (a.group <= 4) launch_one<D, BF16, 4>(a, s);
  else if (a.group <= 8) launch_one<D, BF16, 8>(a, s);
  else launch_one<D, BF16, 16>(a, s);
}

}  // namespace

pkv_status launch_attend8(const pkv_problem& p, const AttendArgs& args, hipStream_t s) {
  AttendArgs a = args;
  if (a.splits > 1) {
    if ((a.cus = current_compute_units()) <= 0) return PKV_EHIP;
    ranges_of_device(int64_t(a.batch) * a.num_kv_heads, a.cus, &a.fill, &a.even);
  }
  const bool bf = p.dtype == PKV_BF16;
  if (p.head_dim == 128) {
    if (bf) launch_gp<128, true>(a, s);
    else launch_gp<128, false>(a, s);
  } else {
    if (bf) launch_gp<64, true>(a, s);
    else launch_gp<64, false>(a, s);
  }
  return hipGetLastError() == hipSuccess ? PKV_OK : PKV_EHIP;
}

}  // namespace pkv
