// Host-side checks of abi_block.cpp for the sanitizer build: descriptors, the
// workspace plans up to the largest accepted sizes, pointers that are never
// dereferenced on the host and no call that reaches a launch.  Exit status =
// number of failed checks.
#include <cstdint>
#include <cstdio>
#include <limits>

#include "ssmvjp.h"

static int failures = 0;
#define CHECK(expr, want)                                                                       \
  do {                                                                                          \
    const int got_ = (int)(expr);                                                               \
    if (got_ != (int)(want)) {                                                                  \
      std::fprintf(stderr, "line %d: %s returned %d, expected %d\n", __LINE__, #expr, got_, (int)(want)); \
      ++failures;                                                                               \
    }                                                                                           \
  } while (0)

static const int64_t TOP = std::numeric_limits<int64_t>::max(), SIZES[] = {
    0, 1, 2, 7, 8, 63, 64, 65, 128, 129, 4096, 65535, 65536, (1 << 20) - 8, 1 << 20, (1 << 24) - 1, 1 << 24,
    0x7fffffff, (int64_t)1 << 32, (int64_t)1 << 40, (int64_t)1 << 62, TOP};

// every plan that is accepted has a size; a workspace one byte short is refused, before anything is read
template <typename Desc, typename Query>
static int sized(const Desc& d, Query query) {
  size_t n = 12345;
  const int st = (int)query(&d, &n);
  if (st == SSMVJP_OK) CHECK(n < (size_t)1 << 62, 1);
  return st;
}

int main() {
  int accepted = 0;
  for (int64_t b : SIZES)
    for (int64_t T : SIZES)
      for (int64_t D : SIZES)
        for (int packed = 0; packed < 2; ++packed) {
          const ssmvjp_linear_scan_desc d{b, T, D, 8.0f, SSMVJP_SCAN_GATED, SSMVJP_BF16, packed};
          const int st = sized(d, linear_scan_fwd_workspace);
          CHECK(sized(d, linear_scan_bwd_workspace), st);
          accepted += st == SSMVJP_OK;
          if (st != SSMVJP_OK) {
            CHECK(linear_scan_fwd(&d, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0), st);
            CHECK(linear_scan_bwd(&d, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0), st);
          }
        }
  for (int64_t b : SIZES)
    for (int64_t n : SIZES)
      for (int64_t D : SIZES) {
        const ssmvjp_linear_step_desc d{b, n, D, 8.0f, SSMVJP_SCAN_LOG, SSMVJP_F32, 0};
        accepted += sized(d, linear_scan_step_workspace) == SSMVJP_OK;
      }
  for (int64_t M : SIZES)
    for (int64_t D : SIZES)
      for (int64_t F : SIZES)
        for (int dtype = 0; dtype < 2; ++dtype) {
          const ssmvjp_ffn_desc d{M, D, F, SSMVJP_ACT_GELU, dtype};
          const int st = sized(d, gated_ffn_fwd_workspace);
          CHECK(sized(d, gated_ffn_bwd_workspace), st);
          accepted += st == SSMVJP_OK;
          if (st != SSMVJP_OK) {
            CHECK(gated_ffn_fwd(&d, 0, 0, 0, 0, 0, 0, 0, 0, 0), st);
            CHECK(gated_ffn_bwd(&d, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0), st);
          }
        }
  for (int64_t n : SIZES) {
    const ssmvjp_dropout_desc d{n, 0.5, SSMVJP_BF16, 0};
    const int st = sized(d, dropout_fwd_workspace);
    CHECK(sized(d, dropout_bwd_workspace), st);
    accepted += st == SSMVJP_OK;
    if (n > 0 && st == SSMVJP_OK) {
      CHECK(dropout_fwd(&d, 0, 0, 0, 0, 0, 0, 0), SSMVJP_EINVAL);
      CHECK(dropout_bwd(&d, 0, 0, 0, 0, 0, 0), SSMVJP_EINVAL);
    }
  }
  CHECK(accepted > 1000, 1);
  std::printf("%d accepted, %d failure(s)\n", accepted, failures);
  return failures;
}
