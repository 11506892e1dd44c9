// abi_common.h -- what the C ABI's translation units share: pointer and type
// checks and the debug finiteness mode.  Internal to libssmvjp.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdlib>
#include <cstring>

#include "../../include/ssmvjp.h"
#include "kernels.h"

namespace {

using namespace ssmvjp;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

size_t big_elem(int32_t dtype) { return dtype == SSMVJP_BF16 ? 2 : 4; }

bool valid_dtype(int32_t dtype) { return dtype == SSMVJP_F32 || dtype == SSMVJP_BF16; }

ssmvjp_status hip_status(hipError_t e) { return e == hipSuccess ? SSMVJP_OK : SSMVJP_EHIP; }

// ---- debug finiteness mode (SSMVJP_CHECK_FINITE set and not "0") ----
// The flag lives in FLAG_BYTES at the end of the workspace, after the plan's
// own bytes rounded up to 256; the workspace queries include it while the
// mode is on.
constexpr size_t FLAG_BYTES = 256;

bool check_finite_on() {
  const char* e = std::getenv("SSMVJP_CHECK_FINITE");
  return e && e[0] && std::strcmp(e, "0") != 0;
}
size_t round256(size_t n) { return (n + 255) / 256 * 256; }
size_t with_flag(size_t plan_bytes) { return check_finite_on() ? round256(plan_bytes) + FLAG_BYTES : plan_bytes; }

struct OutSpan {
  const void* p;
  int64_t n;
  bool bf16;
};

// After the launches: clear the flag, scan every output (`more`: those that the
// call writes in part), read the flag back (this synchronises the stream) and
// turn a raised flag into ENONFINITE.
template <size_t K, typename More>
ssmvjp_status finite_check(void* workspace, size_t plan_bytes, const OutSpan (&outs)[K], hipStream_t stream, More more) {
  unsigned* flag = (unsigned*)((char*)workspace + round256(plan_bytes));
  launch_flag_clear(flag, stream);
  for (const OutSpan& o : outs) launch_nonfinite_check(o.p, o.n, o.bf16, flag, stream);
  more(flag);
  unsigned host = 0;
  if (hipMemcpyAsync(&host, flag, sizeof(host), hipMemcpyDeviceToHost, stream) != hipSuccess) return SSMVJP_EHIP;
  if (hipStreamSynchronize(stream) != hipSuccess) return SSMVJP_EHIP;
  return host ? SSMVJP_ENONFINITE : SSMVJP_OK;
}
template <size_t K>
ssmvjp_status finite_check(void* workspace, size_t plan_bytes, const OutSpan (&outs)[K], hipStream_t stream) {
  return finite_check(workspace, plan_bytes, outs, stream, [](unsigned*) {});
}

}  // namespace
