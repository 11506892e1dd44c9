// dropout.hip -- dropout whose mask is drawn from a counter-based generator
// each time it is needed, in the forward (added to a residual) and the backward.
//
// The generator is Philox 4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011): ten rounds of two 32 x 32 -> 64-bit
// products on a 128-bit counter.  One counter gives eight 16-bit draws, which is
// one 16-byte vector of bf16: the probability is a multiple of 2^-16 then, and
// the scale is the exact one for it.
#include "common.cuh"
#include "kernels.h"

namespace ssmvjp {
namespace {

struct DropArgs {
  i64 n;
  unsigned t;   // kept: draw >= t
  float scale;
  const void *x, *res;
  const i64* rng;
  void* y;
};

struct Words {
  unsigned w[4];
};

__device__ __forceinline__ Words philox(unsigned long long block, unsigned long long offset, unsigned long long seed) {
  unsigned c0 = (unsigned)block, c1 = (unsigned)(block >> 32), c2 = (unsigned)offset, c3 = (unsigned)(offset >> 32);
  unsigned k0 = (unsigned)seed, k1 = (unsigned)(seed >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const unsigned long long p0 = 0xD2511F53ull * c0, p1 = 0xCD9E8D57ull * c2;
    c0 = (unsigned)(p1 >> 32) ^ c1 ^ k0;
    c1 = (unsigned)p1;
    c2 = (unsigned)(p0 >> 32) ^ c3 ^ k1;
    c3 = (unsigned)p0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return {{c0, c1, c2, c3}};
}

// element j of the block's eight
__device__ __forceinline__ bool keep(const Words& w, int j, unsigned t) {
  return ((j & 1) ? w.w[j >> 1] >> 16 : w.w[j >> 1] & 0xffffu) >= t;
}

template <typename T, bool RES>
__global__ void __launch_bounds__(256) dropout_kernel(DropArgs a) {
  const unsigned long long seed = (unsigned long long)a.rng[0], offset = (unsigned long long)a.rng[1];
  const i64 blocks = (a.n + 7) / 8;
  for (i64 b = (i64)blockIdx.x * 256 + threadIdx.x; b < blocks; b += (i64)gridDim.x * 256) {
    const Words w = philox((unsigned long long)b, offset, seed);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const i64 e = 8 * b + j;
      if (e >= a.n) break;
      const float v = keep(w, j, a.t) ? ld((const T*)a.x, e) * a.scale : 0.0f;
      st((T*)a.y, e, RES ? ld((const T*)a.res, e) + v : v);
    }
  }
}

}  // namespace

hipError_t launch_dropout(int64_t n, double p, int32_t dtype, const void* in, const void* residual, const int64_t* rng,
                          void* out, hipStream_t stream) {
  const unsigned t = (unsigned)__builtin_rint(65536.0 * p);
  const DropArgs a{n, t, t < 65536u ? (float)(65536.0 / (65536.0 - t)) : 0.0f, in, residual, rng, out};
  const i64 blocks = ((n + 7) / 8 + 255) / 256;
  const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536));
  if (dtype == SSMVJP_BF16) {
    if (residual) hipLaunchKernelGGL((dropout_kernel<bf16, true>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((dropout_kernel<bf16, false>), grid, dim3(256), 0, stream, a);
  } else {
    if (residual) hipLaunchKernelGGL((dropout_kernel<float, true>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((dropout_kernel<float, false>), grid, dim3(256), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace ssmvjp
