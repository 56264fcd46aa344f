// Launcher stubs of the serving operators for the sanitizer build of the host
// code: an entry point that gets as far as a launch returns PKV_EHIP.
#include "serving/serving_internal.h"

namespace pkv {

pkv_status launch_attend8(const pkv_problem&, const AttendArgs&, hipStream_t) { return PKV_EHIP; }
pkv_status launch_prompt8(const pkv_problem&, const PromptArgs&, hipStream_t) { return PKV_EHIP; }
pkv_status launch_cross_few(const pkv_problem&, Cache, int64_t, const AttendArgs&, hipStream_t) {
  return PKV_EHIP;
}
pkv_status launch_cross_many(const pkv_problem&, Cache, const PromptArgs&, hipStream_t) {
  return PKV_EHIP;
}
pkv_status launch_store8(const pkv_problem&, const Store8Args&, hipStream_t) { return PKV_EHIP; }
pkv_status launch_load8(const pkv_problem&, const Load8Args&, hipStream_t) { return PKV_EHIP; }
pkv_status launch_take(const TakeArgs&, hipStream_t) { return PKV_EHIP; }
pkv_status launch_release(const ReleaseArgs&, hipStream_t) { return PKV_EHIP; }

}  // namespace pkv
