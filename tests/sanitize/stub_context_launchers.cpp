// Launcher stubs of the context operators for the sanitizer build of the host
// code: an entry point that gets as far as a launch returns PKV_EHIP.
#include "context/context_internal.h"

namespace pkv {

pkv_status launch_attend(const pkv_problem&, bool, const AttendArgs&, hipStream_t) {
  return PKV_EHIP;
}
pkv_status launch_prompt(const pkv_problem&, bool, const PromptArgs&, hipStream_t) {
  return PKV_EHIP;
}
pkv_status launch_store(const pkv_problem&, bool, const StoreArgs&, hipStream_t) {
  return PKV_EHIP;
}
pkv_status launch_load(const pkv_problem&, const LoadArgs&, hipStream_t) { return PKV_EHIP; }

}  // namespace pkv
