// dropout.hip -- dropout whose mask is drawn from a counter-based generator
// each time it is needed, in the forward (added to a residual) and the backward.
//
// The generator is Philox 4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011): ten rounds of two 32 x 32 -> 64-bit
// products on a 128-bit counter.  One counter gives eight 16-bit draws, which is
// one 16-byte vector of bf16: the probability is a multiple of 2^-16 then, and
// the scale is the exact one for it.  So the generator hides behind the memory
// (32-bit draws would need twice its products): 8192 x 4096 bf16 with a residual,
// 201 MB, takes 36 us (5.6 TB/s), 29 where the memory-side cache holds a part.
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

// eight elements of a 16-byte aligned tensor
struct Eight {
  float v[8];
};
__device__ __forceinline__ Eight load8(const bf16* p) {
  const uint4 u = *(const uint4*)p;
  const unsigned d[4] = {u.x, u.y, u.z, u.w};
  Eight e;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e.v[2 * i] = __uint_as_float(d[i] << 16);
    e.v[2 * i + 1] = __uint_as_float(d[i] & 0xffff0000u);
  }
  return e;
}
__device__ __forceinline__ Eight load8(const float* p) {
  const float4 a = *(const float4*)p, b = *(const float4*)(p + 4);
  return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ void store8(bf16* p, const Eight& e) {
  *(uint4*)p = make_uint4(pk_bf16(e.v[0], e.v[1]), pk_bf16(e.v[2], e.v[3]), pk_bf16(e.v[4], e.v[5]), pk_bf16(e.v[6], e.v[7]));
}
__device__ __forceinline__ void store8(float* p, const Eight& e) {
  *(float4*)p = make_float4(e.v[0], e.v[1], e.v[2], e.v[3]);
  *(float4*)(p + 4) = make_float4(e.v[4], e.v[5], e.v[6], e.v[7]);
}

// A thread takes one counter's eight elements at a time.  WIDE: 16-byte aligned tensors.
template <typename T, bool RES, bool WIDE>
__global__ void __launch_bounds__(256) dropout_kernel(DropArgs a) {
  const unsigned long long seed = (unsigned long long)a.rng[0], offset = (unsigned long long)a.rng[1];
  const T *x = (const T*)a.x, *res = (const T*)a.res;
  T* y = (T*)a.y;
  const i64 blocks = (a.n + 7) / 8;
  for (i64 b = (i64)blockIdx.x * 256 + threadIdx.x; b < blocks; b += (i64)gridDim.x * 256) {
    const i64 e = 8 * b;
    if (WIDE && e + 8 <= a.n) {
      Eight v = load8(x + e), r;
      if (RES) r = load8(res + e);
      const Words w = philox((unsigned long long)b, offset, seed);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v.v[j] = keep(w, j, a.t) ? v.v[j] * a.scale : 0.0f;
        if (RES) v.v[j] += r.v[j];
      }
      store8(y + e, v);
    } else {
      const Words w = philox((unsigned long long)b, offset, seed);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (e + j < a.n) {
          const float v = keep(w, j, a.t) ? ld(x, e + j) * a.scale : 0.0f;
          st(y, e + j, RES ? ld(res, e + j) + v : v);
        }
    }
  }
}

template <typename T, bool RES>
void launch_wide(const DropArgs& a, hipStream_t s) {
  const i64 blocks = ((a.n + 7) / 8 + 255) / 256;
  const dim3 grid((unsigned)(blocks < (1 << 22) ? blocks : 1 << 22));
  const bool wide = (uintptr_t)a.x % 16 == 0 && (uintptr_t)a.res % 16 == 0 && (uintptr_t)a.y % 16 == 0;
  if (wide) hipLaunchKernelGGL((dropout_kernel<T, RES, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((dropout_kernel<T, RES, false>), grid, dim3(256), 0, s, a);
}

}  // namespace

hipError_t launch_dropout(int64_t n, double p, int32_t dtype, const void* in, const void* residual, const int64_t* rng,
                          void* out, hipStream_t stream) {
  const unsigned t = (unsigned)__builtin_rint(65536.0 * p);
  const DropArgs a{n, t, t < 65536u ? (float)(65536.0 / (65536.0 - t)) : 0.0f, in, residual, rng, out};
  if (dtype == SSMVJP_BF16) residual ? launch_wide<bf16, true>(a, stream) : launch_wide<bf16, false>(a, stream);
  else residual ? launch_wide<float, true>(a, stream) : launch_wide<float, false>(a, stream);
  return hipGetLastError();
}

}  // namespace ssmvjp
