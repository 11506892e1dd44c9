// Host-side checks of abi_layers.cpp for the sanitizer build: descriptors, the
// workspace plans up to the largest accepted sizes, pointers that are never
// dereferenced on the host and no call that reaches a launch.  Exit status =
// number of failed checks.
#include <cstdint>
#include <cstdio>

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

static char* fake(int i) { return (char*)(uintptr_t)(0x100000u * (unsigned)(i + 1)); }  // 256-aligned, never read

static void chunk_checks() {
  const ssmvjp_delta_chunk_desc d{2, 100, 2, 4, 128, 64, 0.1f, SSMVJP_BF16, 0, 0};
  auto fwd = [&](const ssmvjp_delta_chunk_desc* dd, char** p, void* ws, size_t n) {
    return delta_chunk_fwd(dd, p[0], p[1], p[2], (float*)p[3], (float*)p[4], (float*)p[5], (int32_t*)p[6], p[7],
                           (float*)p[8], ws, n, nullptr);
  };
  auto bwd = [&](const ssmvjp_delta_chunk_desc* dd, char** p, void* ws, size_t n) {
    return delta_chunk_bwd(dd, p[0], p[1], p[2], (float*)p[3], (float*)p[4], (float*)p[5], p[6], (float*)p[7],
                           (int32_t*)p[8], p[9], p[10], p[11], (float*)p[12], (float*)p[13], (float*)p[14], ws, n, nullptr);
  };
  size_t nf = 0, nb = 0;
  CHECK(delta_chunk_fwd_workspace(&d, &nf), SSMVJP_OK);
  CHECK(delta_chunk_bwd_workspace(&d, &nb), SSMVJP_OK);
  CHECK(nf > 0 && nb > nf, 1);
  CHECK(delta_chunk_fwd_workspace(nullptr, &nf), SSMVJP_EINVAL);
  CHECK(delta_chunk_bwd_workspace(&d, nullptr), SSMVJP_EINVAL);
  char* f[9];
  char* b[15];
  for (int i = 0; i < 9; ++i) f[i] = i == 6 ? nullptr : fake(i);
  for (int i = 0; i < 15; ++i) b[i] = i == 8 ? nullptr : fake(i);
  CHECK(fwd(nullptr, f, fake(20), nf), SSMVJP_EINVAL);
  CHECK(bwd(nullptr, b, fake(20), nb), SSMVJP_EINVAL);
  CHECK(fwd(&d, f, fake(20), nf - 1), SSMVJP_EWORKSPACE);
  CHECK(bwd(&d, b, fake(20), nb - 1), SSMVJP_EWORKSPACE);
  CHECK(fwd(&d, f, nullptr, nf), SSMVJP_EWORKSPACE);
  CHECK(bwd(&d, b, fake(20) + 8, nb), SSMVJP_EWORKSPACE);
  f[0] += 8;
  CHECK(fwd(&d, f, fake(20), nf), SSMVJP_EINVAL);
  f[0] = nullptr;
  CHECK(fwd(&d, f, fake(20), nf), SSMVJP_EINVAL);
  b[13] += 2;
  CHECK(bwd(&d, b, fake(20), nb), SSMVJP_EINVAL);
  b[13] = nullptr;
  CHECK(bwd(&d, b, fake(20), nb), SSMVJP_EINVAL);
  // at and past every bound: the plans stay inside 64 bits
  const int64_t top = 0x7fffffff;
  const int64_t sizes[][6] = {
      {top, 1, 1, 1, 128, 16},        {1, top, 1, 1, 128, 16},      {top, top, 1, 1, 128, 16},
      {1, 1, (1 << 17) - 1, (1 << 17) - 1, 128, 16}, {1, top, 1, 32, 16, 65536},   {1, 1, 1, 255, 128, 65536},
      {INT64_MAX, INT64_MAX, 1, 1, 16, 16}, {1, INT64_MAX, INT64_MAX, INT64_MAX, 16, 16}, {0, INT64_MAX, 1, 1, 16, 16},
      {1, 1, 1, 1, INT64_MAX - 15, 16}, {1, 1, 1, 1, 16, INT64_MAX - 15},
  };
  for (const auto& s : sizes)
    for (int packed = 0; packed < 2; ++packed)
      for (int t = 0; t < 2; ++t) {
        const ssmvjp_delta_chunk_desc e{s[0], s[1], s[2], s[3], s[4], s[5], 1.0f, t, packed, 0};
        size_t n = 0;
        const int st = delta_chunk_fwd_workspace(&e, &n);
        CHECK(st == SSMVJP_OK || st == SSMVJP_EUNSUPPORTED, 1);
        CHECK(n < ((size_t)1 << 62), 1);
        n = 0;
        const int sb = delta_chunk_bwd_workspace(&e, &n);
        CHECK(sb, t == SSMVJP_BF16 ? st : SSMVJP_EUNSUPPORTED);
        CHECK(n < ((size_t)1 << 62), 1);
      }
}

static void step_checks() {
  const ssmvjp_delta_step_desc d{3, 5, 2, 4, 128, 64, 0.1f, SSMVJP_BF16, SSMVJP_GATE_PER_HEAD, 0};
  auto call = [&](const ssmvjp_delta_step_desc* dd, char** p) {
    return delta_step(dd, p[0], p[1], p[2], (float*)p[3], (float*)p[4], (float*)p[5], (int32_t*)p[6], p[7], nullptr, 0,
                      nullptr);
  };
  size_t n = 1;
  CHECK(delta_step_workspace(&d, &n), SSMVJP_OK);
  CHECK(n, 0);
  CHECK(delta_step_workspace(nullptr, &n), SSMVJP_EINVAL);
  char* p[8];
  for (int i = 0; i < 8; ++i) p[i] = fake(i);
  CHECK(call(nullptr, p), SSMVJP_EINVAL);
  for (int i = 0; i < 8; ++i) {
    if (i == 6) continue;
    char* const old = p[i];
    p[i] = nullptr;
    CHECK(call(&d, p), SSMVJP_EINVAL);
    p[i] = old + 2;
    CHECK(call(&d, p), SSMVJP_EINVAL);
    p[i] = old;
  }
  ssmvjp_delta_step_desc few = d;
  few.nslots = 2;
  p[6] = nullptr;
  CHECK(call(&few, p), SSMVJP_EINVAL);
  for (int64_t big : {(int64_t)0x7fffffff, INT64_MAX}) {
    ssmvjp_delta_step_desc e = d;
    e.batch = big;
    CHECK(delta_step_workspace(&e, &n), SSMVJP_EUNSUPPORTED);
    e = d;
    e.nslots = big;
    CHECK(delta_step_workspace(&e, &n), big > 0x7fffffff ? SSMVJP_EUNSUPPORTED : SSMVJP_OK);
    e = d;
    e.nqk_heads = e.nv_heads = big;
    CHECK(delta_step_workspace(&e, &n), SSMVJP_EUNSUPPORTED);
  }
}

static void norm_checks() {
  const ssmvjp_norm_desc d{10, 1, 100, 1e-5f, SSMVJP_BF16};
  size_t nf = 1, nb = 0;
  CHECK(layer_norm_fwd_workspace(&d, &nf), SSMVJP_OK);
  CHECK(nf, 0);
  CHECK(layer_norm_bwd_workspace(&d, &nb), SSMVJP_OK);
  CHECK(nb > 0, 1);
  CHECK(layer_norm_fwd_workspace(nullptr, &nf), SSMVJP_EINVAL);
  CHECK(layer_norm_bwd_workspace(&d, nullptr), SSMVJP_EINVAL);
  auto bwd = [&](char* dy, char* x, char* x8, char* s8, void* ws, size_t n) {
    return layer_norm_bwd(&d, dy, x, (int8_t*)x8, (float*)s8, (float*)fake(4), (float*)fake(5), (float*)fake(6), fake(7),
                          (float*)fake(8), (float*)fake(9), ws, n, nullptr);
  };
  CHECK(bwd(fake(0), fake(1), nullptr, nullptr, fake(20), nb - 1), SSMVJP_EWORKSPACE);
  CHECK(bwd(fake(0), fake(1), nullptr, nullptr, nullptr, nb), SSMVJP_EWORKSPACE);
  CHECK(bwd(fake(0), fake(1), fake(2), fake(3), fake(20), nb), SSMVJP_EINVAL);
  CHECK(bwd(fake(0), nullptr, nullptr, nullptr, fake(20), nb), SSMVJP_EINVAL);
  CHECK(bwd(fake(0), nullptr, fake(2), nullptr, fake(20), nb), SSMVJP_EINVAL);
  CHECK(bwd(fake(0) + 1, fake(1), nullptr, nullptr, fake(20), nb), SSMVJP_EINVAL);
  CHECK(layer_norm_fwd(&d, fake(0), nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr),
        SSMVJP_EINVAL);
  CHECK(layer_norm_fwd(&d, fake(0), nullptr, nullptr, fake(1), nullptr, nullptr, (int8_t*)fake(2), nullptr, nullptr, 0,
                       nullptr),
        SSMVJP_EINVAL);
  const int64_t top = 0x7fffffff;
  const int64_t sizes[][3] = {{top, 1, 1},  {1, top, 1},  {1, top, 16}, {1, 1, (int64_t)1 << 35}, {top, 1, (int64_t)1 << 35},
                              {INT64_MAX, 1, 1}, {1, INT64_MAX, 1}, {1, 1, INT64_MAX}, {0, 1, INT64_MAX}, {1 << 15, 1 << 15, 1 << 15}};
  for (const auto& s : sizes)
    for (int t = 0; t < 2; ++t) {
      const ssmvjp_norm_desc e{s[0], s[1], s[2], 0.0f, t};
      size_t n = 0;
      const int st = layer_norm_bwd_workspace(&e, &n);
      CHECK(st == SSMVJP_OK || st == SSMVJP_EUNSUPPORTED, 1);
      CHECK(n < ((size_t)1 << 62), 1);
    }
}

int main() {
  chunk_checks();
  step_checks();
  norm_checks();
  std::printf("%d failure(s)\n", failures);
  return failures != 0;
}
