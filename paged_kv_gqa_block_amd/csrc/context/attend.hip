// Decode attention over 16-bit pages and the 4-bit pool: launches of
// attend_kernel.h.
#include <atomic>

#include "context/attend_kernel.h"

namespace pkv {
namespace {

template <int D, bool BF16, bool KV4, int GP>
void launch_one(const AttendArgs& a, hipStream_t s) {
  const dim3 grid(a.num_kv_heads, a.splits, a.batch);
  hipLaunchKernelGGL((attend_kernel<D, BF16, KV4 ? Cache::k4 : Cache::k16, false, GP, 4,
                                    KV4 ? 2 : 1, KV4 ? 2 : 1>),
                     grid, dim3(256), 0, s, a);
}

template <int D, bool BF16, bool KV4>
void launch_gp(const AttendArgs& a, hipStream_t s) {
  if (a.group <= 4) launch_one<D, BF16, KV4, 4>(a, s);
  else if (a.group <= 8) launch_one<D, BF16, KV4, 8>(a, s);
  else launch_one<D, BF16, KV4, 16>(a, s);
}

template <int D, bool BF16>
void launch_fmt(bool kv4, const AttendArgs& a, hipStream_t s) {
  if (kv4) launch_gp<D, BF16, true>(a, s);
  else launch_gp<D, BF16, false>(a, s);
}

}  // namespace

int current_compute_units() {
  static std::atomic<int> known[64];
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess) return 0;
  if (dev < 64 && (cus = known[dev].load(std::memory_order_relaxed)) > 0) return cus;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
    return 0;
  if (dev < 64) known[dev].store(cus, std::memory_order_relaxed);
  return cus;
}

pkv_status launch_attend(const pkv_problem& p, bool kv4, const AttendArgs& args, hipStream_t s) {
  const bool bf = p.dtype == PKV_BF16;
  AttendArgs a = args;
  if (a.splits > 1) {
    if ((a.cus = current_compute_units()) <= 0) return PKV_EHIP;
    ranges_of_device(int64_t(a.batch) * a.num_kv_heads, a.cus, &a.fill, &a.even);
  }
  if (p.head_dim == 128) {
    if (bf) launch_fmt<128, true>(kv4, a, s);
    else launch_fmt<128, false>(kv4, a, s);
  } else {
    if (bf) launch_fmt<64, true>(kv4, a, s);
    else launch_fmt<64, false>(kv4, a, s);
  }
  return hipGetLastError() == hipSuccess ? PKV_OK : PKV_EHIP;
}

}  // namespace pkv
