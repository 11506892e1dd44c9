// layer_norm.hip -- layer norm of the last axis, its gradients, and the 8-bit
// form of its input that the backward can read in place of the input.
//
// x is [rows][G][D]; row (t, g) uses the weights w[g], b[g] (G = 1: one weight
// vector for all rows; G = heads: every head of a readout has its own).
//   mean = sum x / D;  rstd = 1 / sqrt(sum (x - mean)^2 / D + eps)
//   h = (x - mean) rstd;  y = h w + b
//   t = dy w;  dx = rstd (t - sum(t) / D - h sum(t h) / D)
//   dw[g] = sum over rows of dy h;  db[g] = sum over rows of dy
// 8-bit form: per block of 64 values of a row, scale = max|x| (1/127) and
// code = rint(x (127 (1/max|x|))), each operation rounded to float32 (bf16
// inputs often fall on the half between two codes, so the order is part of the
// format); a block below 1e-36 is stored as zeros.
//
// All sums are float32.  The variance is the second pass over values that are
// already in registers, not E[x^2] - mean^2, which would cancel.
//
// MI355X organisation.  These kernels are bound by HBM: every value of x, dy,
// y, dx crosses it once.  A row is held in registers by TPR threads (16, 64 or
// 256, the fewest that hold it: short rows need no cross-wave exchange, and
// several share a wave), NV vectors of 16 bytes each.  A workgroup keeps one
// g, so that its weights stay in registers over all of its rows, and walks the
// rows of that group with a stride.  dw, db are summed over a workgroup's rows
// in registers, over its row slots in LDS and over the workgroups by a second
// launch, in a fixed order (no atomics: equal inputs give equal bits).
// Rows that are too long for the registers, or whose length or pointers do not
// allow 16-byte accesses at that length, are walked in passes over memory
// (the second and third pass mostly hit L2).
//
// Measured (bf16): forward of 8192 x 32 rows of 128 in 26.1 us, 5.2 TB/s, the rate
// of a device copy; backward of 8192 x 4096 in 40.9 us (4.9 TB/s) and 4.6 us for the
// second launch; with the 8-bit form 42.1 and 40.2 us.  The two launches of the
// backward took 69 us a call before a row was loaded ahead and 32 partial sums were
// summed at a time, 50 since.  Widths that are no multiple of a vector go value by
// value: 8192 x 1001 takes 14.5 us forward and 20.5 backward in registers (8192 x
// 1000: 13.2 and 18.4), 8192 x 4097 in passes 64 and 107 us a call (8192 x 4096: 25
// and 45), 4096 x 5001 45 and 70.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace ssmvjp {
namespace {

struct NormArgs {
  i64 rows, G, D, NB;  // NB: 8-bit blocks of a row
  i64 parts;           // workgroups per group
  float eps;
  const void* x;
  const float* w;
  const float* b;
  const void* dy;
  void* out;  // y or dx
  float* mean;
  float* rstd;
  int8_t* x8;
  float* x8s;
  float* part;  // [parts][2][G][D] partial dw, db (NULL: not wanted)
};

constexpr float TINY8 = 1e-36f;  // below it 127 / max|x| would leave float32's range

// ---- VEC consecutive elements as floats ----
template <int VEC>
__device__ __forceinline__ void load_vec(const float* p, float (&o)[VEC]) {
  if constexpr (VEC == 4) {
    const float4 u = *(const float4*)p;
    o[0] = u.x; o[1] = u.y; o[2] = u.z; o[3] = u.w;
  } else if constexpr (VEC == 8) {
    const float4 u = ((const float4*)p)[0], v = ((const float4*)p)[1];
    o[0] = u.x; o[1] = u.y; o[2] = u.z; o[3] = u.w;
    o[4] = v.x; o[5] = v.y; o[6] = v.z; o[7] = v.w;
  } else {
    o[0] = *p;
  }
}
template <int VEC>
__device__ __forceinline__ void load_vec(const bf16* p, float (&o)[VEC]) {
  if constexpr (VEC == 8) {
    const u32x4 u = *(const u32x4*)p;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o[2 * e] = __uint_as_float(u[e] << 16);
      o[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
    }
  } else {
    o[0] = (float)*p;
  }
}
template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[VEC]) {
  if constexpr (VEC == 4)
    *(float4*)p = make_float4(v[0], v[1], v[2], v[3]);
  else
    *p = v[0];
}
template <int VEC>
__device__ __forceinline__ void store_vec(bf16* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const u32x4 u = {pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]), pk_bf16(v[4], v[5]), pk_bf16(v[6], v[7])};
    *(u32x4*)p = u;
  } else {
    *p = (bf16)v[0];
  }
}
// VEC codes times their block's scale
template <int VEC>
__device__ __forceinline__ void load_codes(const int8_t* p, float s, float (&o)[VEC]) {
  if constexpr (VEC == 1) {
    o[0] = (float)*p * s;
  } else {
    int8_t c[VEC];
    __builtin_memcpy(c, __builtin_assume_aligned(p, VEC), VEC);
#pragma unroll
    for (int e = 0; e < VEC; ++e) o[e] = (float)c[e] * s;
  }
}

// ---- reductions over the TPR threads of a row; every thread gets the result ----
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* lds) {
  if constexpr (TPR == 16) return sum16(v);
  v = wave_sum(v);
  if constexpr (TPR == 256) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (lds[0] + lds[1]) + (lds[2] + lds[3]);
  }
  return v;
}
// max over the 64 / VEC lanes that hold one block's values (8, 16 or 64)
template <int VEC>
__device__ __forceinline__ float block_max(float v) {
  if constexpr (VEC == 8) {
    v = fmaxf(v, dpp_f<0xB1>(v));   // quad_perm [1,0,3,2]
    v = fmaxf(v, dpp_f<0x4E>(v));   // quad_perm [2,3,0,1]
    v = fmaxf(v, dpp_f<0x141>(v));  // row_half_mirror: the other quad of the eight
  } else {
    v = fmaxf(v, dpp_f<0x128>(v));
    v = fmaxf(v, dpp_f<0x124>(v));
    v = fmaxf(v, dpp_f<0x122>(v));
    v = fmaxf(v, dpp_f<0x121>(v));
    if constexpr (VEC == 1) {
      v = fmaxf(v, __shfl_xor(v, 16, 64));
      v = fmaxf(v, __shfl_xor(v, 32, 64));
    }
  }
  return v;
}

// the codes and the scale of this thread's vector `vec` of row r (every lane of
// a block calls it; `live`: the vector lies inside the row)
template <int VEC>
__device__ __forceinline__ void store_codes(const NormArgs& a, i64 r, i64 vec, const float (&x)[VEC], bool live) {
  float top = 0.0f;
  if (live) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) top = fmaxf(top, fabsf(x[e]));
  }
  top = block_max<VEC>(top);
  const bool some = top >= TINY8;
  const float inv = some ? 127.0f * (1.0f / top) : 0.0f;
  if (!live) return;
  int8_t c[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) c[e] = (int8_t)(int)rintf(x[e] * inv);
  __builtin_memcpy(__builtin_assume_aligned(a.x8 + r * a.D + vec * VEC, VEC), c, VEC);
  constexpr int LPB = 64 / VEC;
  if (vec % LPB == 0) a.x8s[r * a.NB + vec / LPB] = some ? top * (1.0f / 127.0f) : 0.0f;
}

// ---------------------------------------------------------------------------
// forward, rows in registers
// ---------------------------------------------------------------------------
template <typename T, int VEC, int TPR, int NV, bool CK>
__global__ void __launch_bounds__(256) norm_fwd_kernel(NormArgs a) {
  constexpr int RPB = 256 / TPR;
  __shared__ float red[2][2][4];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const i64 g = blockIdx.x % a.G, part = blockIdx.x / a.G;
  const float invD = 1.0f / (float)a.D;
  float w[NV][VEC], b[NV][VEC];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const i64 e = (i64)(t + TPR * n) * VEC;
#pragma unroll
    for (int k = 0; k < VEC; ++k) w[n][k] = 1.0f, b[n][k] = 0.0f;
    if (e < a.D) {
      if (a.w) load_vec<VEC>(a.w + g * a.D + e, w[n]);
      if (a.b) load_vec<VEC>(a.b + g * a.D + e, b[n]);
    }
  }
  int flip = 0;
  for (i64 row = part * RPB + sub; row < a.rows; row += a.parts * RPB, flip ^= 1) {
    const i64 r = row * a.G + g;
    const T* x = (const T*)a.x + r * a.D;
    float v[NV][VEC];
    float s = 0.0f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const i64 e = (i64)(t + TPR * n) * VEC;
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[n][k] = 0.0f;
      if (e < a.D) load_vec<VEC>(x + e, v[n]);
    }
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int k = 0; k < VEC; ++k) s += v[n][k];
    const float mean = row_sum<TPR>(s, red[flip][0]) * invD;
    float q = 0.0f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const bool live = (i64)(t + TPR * n) * VEC < a.D;
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const float d = v[n][k] - mean;
        q += live ? d * d : 0.0f;
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<TPR>(q, red[flip][1]) * invD + a.eps);
    T* y = (T*)a.out + r * a.D;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const i64 vec = t + TPR * n;
      const bool live = vec * VEC < a.D;
      if constexpr (CK) store_codes<VEC>(a, r, vec, v[n], live);
      if (live) {
        float o[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) o[k] = (v[n][k] - mean) * rstd * w[n][k] + b[n][k];
        store_vec<VEC>(y + vec * VEC, o);
      }
    }
    if (t == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
  }
}

// forward, a row per workgroup at a time in three passes over memory
template <typename T, int VEC, bool CK>
__global__ void __launch_bounds__(256) norm_fwd_long_kernel(NormArgs a) {
  __shared__ float red[2][4];
  for (i64 r = blockIdx.x; r < a.rows * a.G; r += gridDim.x) {
    const i64 g = r % a.G;
    const T* x = (const T*)a.x + r * a.D;
    T* y = (T*)a.out + r * a.D;
    const float invD = 1.0f / (float)a.D;
    const i64 nv = (a.D + VEC - 1) / VEC;
    float s = 0.0f, v[VEC];
    for (i64 i = threadIdx.x; i < nv; i += 256) {
      load_vec<VEC>(x + i * VEC, v);
#pragma unroll
      for (int k = 0; k < VEC; ++k) s += v[k];
    }
    const float mean = row_sum<256>(s, red[0]) * invD;
    float q = 0.0f;
    for (i64 i = threadIdx.x; i < nv; i += 256) {
      load_vec<VEC>(x + i * VEC, v);
#pragma unroll
      for (int k = 0; k < VEC; ++k) q += (v[k] - mean) * (v[k] - mean);
    }
    const float rstd = 1.0f / sqrtf(row_sum<256>(q, red[1]) * invD + a.eps);
    const i64 nround = (nv + 255) / 256 * 256;  // whole waves: every lane of a block takes part in its maximum
    for (i64 i = threadIdx.x; i < nround; i += 256) {
      const bool live = i < nv;
      if (live) load_vec<VEC>(x + i * VEC, v);
      if constexpr (CK) store_codes<VEC>(a, r, i, v, live);
      if (live) {
        float w[VEC], b[VEC], o[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) w[k] = 1.0f, b[k] = 0.0f;
        if (a.w) load_vec<VEC>(a.w + g * a.D + i * VEC, w);
        if (a.b) load_vec<VEC>(a.b + g * a.D + i * VEC, b);
#pragma unroll
        for (int k = 0; k < VEC; ++k) o[k] = (v[k] - mean) * rstd * w[k] + b[k];
        store_vec<VEC>(y + i * VEC, o);
      }
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
  }
}

// ---------------------------------------------------------------------------
// backward, rows in registers
// ---------------------------------------------------------------------------
// x values of vector `vec` of row r: the input itself or its 8-bit form
template <typename T, int VEC, bool CK>
__device__ __forceinline__ void load_x(const NormArgs& a, i64 r, i64 vec, float (&o)[VEC]) {
  if constexpr (CK)
    load_codes<VEC>(a.x8 + r * a.D + vec * VEC, a.x8s[r * a.NB + vec / (64 / VEC)], o);
  else
    load_vec<VEC>((const T*)a.x + r * a.D + vec * VEC, o);
}

// one vector of x (or of its codes, and their scale) and of dy as they are in
// memory: the next row's are loaded while a row is computed
template <typename T, int VEC, bool CK>
struct NormRaw {
  T dy[VEC], x[CK ? 1 : VEC];
  int8_t c[CK ? VEC : 1];
  float s;
  __device__ __forceinline__ void load(const NormArgs& a, i64 r, i64 vec) {
    constexpr int B = VEC * (int)sizeof(T), AL = VEC > 1 ? 16 : (int)sizeof(T);
    const i64 e = r * a.D + vec * VEC;
    __builtin_memcpy(dy, __builtin_assume_aligned((const T*)a.dy + e, AL), B);
    if constexpr (CK) {
      __builtin_memcpy(c, __builtin_assume_aligned(a.x8 + e, VEC), VEC);
      s = a.x8s[r * a.NB + vec / (64 / VEC)];
    } else {
      __builtin_memcpy(x, __builtin_assume_aligned((const T*)a.x + e, AL), B);
    }
  }
  __device__ __forceinline__ float x_at(int k) const {
    if constexpr (CK) return (float)c[k] * s;
    else return (float)x[k];
  }
};

template <typename T, int VEC, int TPR, int NV, bool CK>
__global__ void __launch_bounds__(256) norm_bwd_kernel(NormArgs a) {
  constexpr int RPB = 256 / TPR, W = TPR * NV * VEC;  // W: columns a row slot can hold
  __shared__ float red[2][2][4];
  __shared__ float acc[RPB > 1 ? RPB * W : 1];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const i64 g = blockIdx.x % a.G, part = blockIdx.x / a.G;
  const float invD = 1.0f / (float)a.D;
  float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const i64 e = (i64)(t + TPR * n) * VEC;
#pragma unroll
    for (int k = 0; k < VEC; ++k) w[n][k] = 1.0f, dw[n][k] = 0.0f, db[n][k] = 0.0f;
    if (a.w && e < a.D) load_vec<VEC>(a.w + g * a.D + e, w[n]);
  }
  NormRaw<T, VEC, CK> raw[NV];
  float mean_n = 0.0f, rstd_n = 0.0f;
  auto fetch = [&](i64 row) {
    const i64 r = row * a.G + g;
    mean_n = a.mean[r];
    rstd_n = a.rstd[r];
#pragma unroll
    for (int n = 0; n < NV; ++n)
      if ((i64)(t + TPR * n) * VEC < a.D) raw[n].load(a, r, t + TPR * n);
  };
  i64 row = part * RPB + sub;
  if (row < a.rows) fetch(row);
  int flip = 0;
  for (; row < a.rows; row += a.parts * RPB, flip ^= 1) {
    const i64 r = row * a.G + g;
    float h[NV][VEC], dy[NV][VEC];
    const float mean = mean_n, rstd = rstd_n;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const bool live = (i64)(t + TPR * n) * VEC < a.D;
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        h[n][k] = live ? raw[n].x_at(k) : mean;
        dy[n][k] = live ? (float)raw[n].dy[k] : 0.0f;
      }
    }
    if (row + a.parts * RPB < a.rows) fetch(row + a.parts * RPB);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        h[n][k] = (h[n][k] - mean) * rstd;
        const float tw = dy[n][k] * w[n][k];
        s1 += tw;
        s2 += tw * h[n][k];
        dw[n][k] += dy[n][k] * h[n][k];
        db[n][k] += dy[n][k];
      }
    float c1, c2;
    if constexpr (TPR == 256) {
      s1 = wave_sum(s1);
      s2 = wave_sum(s2);
      float(*l)[4] = red[flip];
      if ((threadIdx.x & 63) == 0) l[0][threadIdx.x >> 6] = s1, l[1][threadIdx.x >> 6] = s2;
      __syncthreads();
      c1 = ((l[0][0] + l[0][1]) + (l[0][2] + l[0][3])) * invD;
      c2 = ((l[1][0] + l[1][1]) + (l[1][2] + l[1][3])) * invD;
    } else {
      c1 = row_sum<TPR>(s1, nullptr) * invD;
      c2 = row_sum<TPR>(s2, nullptr) * invD;
    }
    T* dx = (T*)a.out + r * a.D;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const i64 e = (i64)(t + TPR * n) * VEC;
      if (e < a.D) {
        float o[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) o[k] = rstd * (dy[n][k] * w[n][k] - c1 - h[n][k] * c2);
        store_vec<VEC>(dx + e, o);
      }
    }
  }
  if (!a.part) return;
  // this workgroup's dw, then db: over its row slots in slot order, then out
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* p = a.part + ((part * 2 + which) * a.G + g) * a.D;
    float(&s)[NV][VEC] = which ? db : dw;
    if constexpr (RPB > 1) {
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int k = 0; k < VEC; ++k) acc[sub * W + (t + TPR * n) * VEC + k] = s[n][k];
      __syncthreads();
      for (i64 e = threadIdx.x; e < a.D; e += 256) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < RPB; ++i) v += acc[i * W + e];
        p[e] = v;
      }
    } else {
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const i64 e = (i64)(t + TPR * n) * VEC + k;
          if (e < a.D) p[e] = s[n][k];
        }
    }
  }
}

// backward, a row per workgroup at a time in two passes over memory (dx only)
template <typename T, int VEC, bool CK>
__global__ void __launch_bounds__(256) norm_bwd_long_kernel(NormArgs a) {
  __shared__ float red[2][4];
  for (i64 r = blockIdx.x; r < a.rows * a.G; r += gridDim.x) {
    const i64 g = r % a.G;
    const float invD = 1.0f / (float)a.D, mean = a.mean[r], rstd = a.rstd[r];
    const i64 nv = (a.D + VEC - 1) / VEC;
    const T* dyp = (const T*)a.dy + r * a.D;
    const float* wp = a.w ? a.w + g * a.D : nullptr;
    float h[VEC], dy[VEC], w[VEC], s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int k = 0; k < VEC; ++k) w[k] = 1.0f;
    for (i64 i = threadIdx.x; i < nv; i += 256) {
      load_x<T, VEC, CK>(a, r, i, h);
      load_vec<VEC>(dyp + i * VEC, dy);
      if (wp) load_vec<VEC>(wp + i * VEC, w);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        s1 += dy[k] * w[k];
        s2 += dy[k] * w[k] * ((h[k] - mean) * rstd);
      }
    }
    const float c1 = row_sum<256>(s1, red[0]) * invD, c2 = row_sum<256>(s2, red[1]) * invD;
    T* dx = (T*)a.out + r * a.D;
    for (i64 i = threadIdx.x; i < nv; i += 256) {
      load_x<T, VEC, CK>(a, r, i, h);
      load_vec<VEC>(dyp + i * VEC, dy);
      if (wp) load_vec<VEC>(wp + i * VEC, w);
      float o[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) o[k] = rstd * (dy[k] * w[k] - c1 - (h[k] - mean) * rstd * c2);
      store_vec<VEC>(dx + i * VEC, o);
    }
  }
}

// dw, db of 256 columns of one group over one share of the rows (partial sums)
template <typename T, bool CK>
__global__ void __launch_bounds__(256) norm_cols_kernel(NormArgs a, i64 cblocks) {
  const i64 g = blockIdx.x / cblocks % a.G, part = blockIdx.x / cblocks / a.G;
  const i64 d = blockIdx.x % cblocks * 256 + threadIdx.x;
  if (d >= a.D) return;
  float dw = 0.0f, db = 0.0f;
  for (i64 row = part; row < a.rows; row += a.parts) {
    const i64 r = row * a.G + g;
    float x[1], dy[1];
    load_x<T, 1, CK>(a, r, d, x);
    load_vec<1>((const T*)a.dy + r * a.D + d, dy);
    dw += dy[0] * ((x[0] - a.mean[r]) * a.rstd[r]);
    db += dy[0];
  }
  a.part[(part * 2 * a.G + g) * a.D + d] = dw;
  a.part[((part * 2 + 1) * a.G + g) * a.D + d] = db;
}

// dw, db = sums of the workgroups' partial sums: 32 columns x 32 shares per
// workgroup, each share's parts in ascending order, then the shares in a tree
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float* part, i64 parts, i64 GD, float* dw, float* db) {
  __shared__ float acc[32][33];
  const int c = threadIdx.x & 31, sh = threadIdx.x >> 5;
  const i64 col = (i64)blockIdx.x * 32 + c;
  float s = 0.0f;
  if (col < 2 * GD) {
#pragma unroll 8
    for (i64 p = sh; p < parts; p += 32) s += part[p * 2 * GD + col];
  }
  acc[sh][c] = s;
  __syncthreads();
  // thread (column sh, share c): the sum over the shares lies in one half wave
  s = acc[c][sh];
  s = sum16(s);
  s += __shfl_xor(s, 16, 64);
  const i64 oc = (i64)blockIdx.x * 32 + sh;
  if (c == 0 && oc < 2 * GD) {
    float* out = oc < GD ? dw : db;
    if (out) out[oc < GD ? oc : oc - GD] = s;
  }
}

__global__ void __launch_bounds__(256) norm_zero_kernel(float* a, float* b, i64 n) {
  const i64 i = (i64)blockIdx.x * 256 + threadIdx.x;
  if (i < n) {
    if (a) a[i] = 0.0f;
    if (b) b[i] = 0.0f;
  }
}

bool on16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// 16-byte accesses: the row length is a whole number of vectors and every
// tensor starts on a vector
bool vec_ok(const ssmvjp_norm_desc& d, std::initializer_list<const void*> ps) {
  if (d.dim % (d.dtype == SSMVJP_BF16 ? 8 : 4)) return false;
  for (const void* p : ps)
    if (p && !on16(p)) return false;
  return true;
}

// workgroups per group: enough to fill the card (about `total` of 4 waves), not
// more than there are shares of `per` rows for each of a workgroup's rpb slots
i64 norm_parts(i64 rows, i64 G, int rpb, int per, i64 total) {
  const i64 most = (rows + rpb * per - 1) / (rpb * per), want = (total + G - 1) / G;
  return most < want ? most : want;
}

// threads per row, by what TPR threads of NV vectors hold (0: walked in passes)
int norm_tpr(i64 D, int vec, bool backward) {
  const i64 n = (D + vec - 1) / vec;
  if (vec > 1 && n <= 32) return 16;
  if (n <= 256) return 64;
  if (n <= (backward ? 1024 : 2048)) return 256;
  return 0;
}

// a launch has fewer than 2^32 threads
unsigned long_grid(const NormArgs& a) { return (unsigned)std::min<i64>(a.rows * a.G, 1 << 20); }

constexpr i64 FWD_GROUPS = 2048, BWD_GROUPS = 512;
constexpr int BWD_ROWS = 2;  // a workgroup's partial dw, db cost as much as a row of dx each
constexpr i64 COLS_GROUPS = (1 << 24) - 1;  // norm_cols_kernel: a launch has fewer than 2^32 threads

i64 col_blocks(i64 D) { return (D + 255) / 256; }

// partial dw, db of a group: one for each of its workgroups, or (tpr = 0) of its shares of the rows in norm_cols_kernel
i64 bwd_parts(i64 rows, i64 G, i64 D, int tpr) {
  const i64 p = norm_parts(rows, G, tpr ? 256 / tpr : 1, BWD_ROWS, BWD_GROUPS);
  return tpr ? p : std::min(p, COLS_GROUPS / (col_blocks(D) * G));
}

template <typename T, int VEC, bool CK>
void fwd_vec(const NormArgs& in, hipStream_t s) {
  NormArgs a = in;
  const int tpr = norm_tpr(a.D, VEC, false);
  const i64 n = (a.D + VEC - 1) / VEC;
  a.parts = norm_parts(a.rows, a.G, tpr ? 256 / tpr : 1, 1, FWD_GROUPS);
  const dim3 grid((unsigned)(a.parts * a.G)), wg(256);
  if constexpr (VEC > 1) {
    if (tpr == 16) {
      if (n <= 16) hipLaunchKernelGGL((norm_fwd_kernel<T, VEC, 16, 1, CK>), grid, wg, 0, s, a);
      else hipLaunchKernelGGL((norm_fwd_kernel<T, VEC, 16, 2, CK>), grid, wg, 0, s, a);
      return;
    }
  }
  if (tpr == 64) {
    if (n <= 128) hipLaunchKernelGGL((norm_fwd_kernel<T, VEC, 64, 2, CK>), grid, wg, 0, s, a);
    else hipLaunchKernelGGL((norm_fwd_kernel<T, VEC, 64, 4, CK>), grid, wg, 0, s, a);
  } else if (tpr == 256) {
    if (n <= 512) hipLaunchKernelGGL((norm_fwd_kernel<T, VEC, 256, 2, CK>), grid, wg, 0, s, a);
    else if (n <= 1024) hipLaunchKernelGGL((norm_fwd_kernel<T, VEC, 256, 4, CK>), grid, wg, 0, s, a);
    else hipLaunchKernelGGL((norm_fwd_kernel<T, VEC, 256, 8, CK>), grid, wg, 0, s, a);
  } else {
    hipLaunchKernelGGL((norm_fwd_long_kernel<T, VEC, CK>), dim3(long_grid(a)), wg, 0, s, a);
  }
}

template <typename T, int VEC, bool CK>
void bwd_vec(const NormArgs& in, hipStream_t s) {
  NormArgs a = in;
  const int tpr = norm_tpr(a.D, VEC, true);
  const i64 n = (a.D + VEC - 1) / VEC;
  a.parts = bwd_parts(a.rows, a.G, a.D, tpr);
  const dim3 grid((unsigned)(a.parts * a.G)), wg(256);
  if (VEC > 1 && tpr == 16) {
    if constexpr (VEC > 1) {
      if (n <= 16) hipLaunchKernelGGL((norm_bwd_kernel<T, VEC, 16, 1, CK>), grid, wg, 0, s, a);
      else hipLaunchKernelGGL((norm_bwd_kernel<T, VEC, 16, 2, CK>), grid, wg, 0, s, a);
    }
  } else if (tpr == 64) {
    if (n <= 128) hipLaunchKernelGGL((norm_bwd_kernel<T, VEC, 64, 2, CK>), grid, wg, 0, s, a);
    else hipLaunchKernelGGL((norm_bwd_kernel<T, VEC, 64, 4, CK>), grid, wg, 0, s, a);
  } else if (tpr == 256) {
    if (n <= 512) hipLaunchKernelGGL((norm_bwd_kernel<T, VEC, 256, 2, CK>), grid, wg, 0, s, a);
    else hipLaunchKernelGGL((norm_bwd_kernel<T, VEC, 256, 4, CK>), grid, wg, 0, s, a);
  } else {
    hipLaunchKernelGGL((norm_bwd_long_kernel<T, VEC, CK>), dim3(long_grid(a)), wg, 0, s, a);
    if (a.part) {
      const i64 cb = col_blocks(a.D);
      hipLaunchKernelGGL((norm_cols_kernel<T, CK>), dim3((unsigned)(cb * a.G * a.parts)), wg, 0, s, a, cb);
    }
  }
}

NormArgs norm_args(const ssmvjp_norm_desc& d) {
  NormArgs a{};
  a.rows = d.rows; a.G = d.groups; a.D = d.dim; a.NB = (d.dim + 63) / 64; a.eps = d.eps;
  return a;
}

}  // namespace

size_t norm_bwd_workspace_bytes(const ssmvjp_norm_desc& d) {
  // the largest number of partial sums over the variants: one row a workgroup, and no cap by norm_cols_kernel's grid
  // unless every variant walks the row in passes
  const int tpr = norm_tpr(d.dim, d.dtype == SSMVJP_BF16 ? 8 : 4, true) ? 256 : 0;
  return (size_t)(bwd_parts(d.rows, d.groups, d.dim, tpr) * 2 * d.groups * d.dim * 4);
}

hipError_t launch_norm_fwd(const ssmvjp_norm_desc& d, const NormFwdPointers& p, hipStream_t s) {
  NormArgs a = norm_args(d);
  a.x = p.x; a.w = p.weight; a.b = p.bias; a.out = p.y; a.mean = p.mean; a.rstd = p.rstd;
  a.x8 = p.x8; a.x8s = p.x8_scale;
  const bool v = vec_ok(d, {p.x, p.weight, p.bias, p.y, p.x8}), ck = p.x8 != nullptr;
  if (d.dtype == SSMVJP_BF16) {
    if (v) ck ? fwd_vec<bf16, 8, true>(a, s) : fwd_vec<bf16, 8, false>(a, s);
    else ck ? fwd_vec<bf16, 1, true>(a, s) : fwd_vec<bf16, 1, false>(a, s);
  } else {
    if (v) ck ? fwd_vec<float, 4, true>(a, s) : fwd_vec<float, 4, false>(a, s);
    else ck ? fwd_vec<float, 1, true>(a, s) : fwd_vec<float, 1, false>(a, s);
  }
  return hipGetLastError();
}

hipError_t launch_norm_bwd(const ssmvjp_norm_desc& d, const NormBwdPointers& p, hipStream_t s) {
  NormArgs a = norm_args(d);
  const i64 GD = d.groups * d.dim;
  const bool wants = p.dweight || p.dbias;
  if (d.rows == 0) {
    if (wants)
      hipLaunchKernelGGL(norm_zero_kernel, dim3((unsigned)((GD + 255) / 256)), dim3(256), 0, s, p.dweight, p.dbias, GD);
    return hipGetLastError();
  }
  a.x = p.x; a.w = p.weight; a.dy = p.dy; a.out = p.dx;
  a.mean = const_cast<float*>(p.mean); a.rstd = const_cast<float*>(p.rstd);
  a.x8 = const_cast<int8_t*>(p.x8); a.x8s = const_cast<float*>(p.x8_scale);
  a.part = wants ? (float*)p.workspace : nullptr;
  const bool v = vec_ok(d, {p.x, p.weight, p.dy, p.dx, p.x8}), ck = p.x8 != nullptr;
  if (d.dtype == SSMVJP_BF16) {
    if (v) ck ? bwd_vec<bf16, 8, true>(a, s) : bwd_vec<bf16, 8, false>(a, s);
    else ck ? bwd_vec<bf16, 1, true>(a, s) : bwd_vec<bf16, 1, false>(a, s);
  } else {
    if (v) ck ? bwd_vec<float, 4, true>(a, s) : bwd_vec<float, 4, false>(a, s);
    else ck ? bwd_vec<float, 1, true>(a, s) : bwd_vec<float, 1, false>(a, s);
  }
  if (wants) {
    const int tpr = norm_tpr(d.dim, v ? (d.dtype == SSMVJP_BF16 ? 8 : 4) : 1, true);
    const i64 parts = bwd_parts(d.rows, d.groups, d.dim, tpr);
    hipLaunchKernelGGL(norm_reduce_kernel, dim3((unsigned)((2 * GD + 31) / 32)), dim3(1024), 0, s, (const float*)p.workspace, parts,
                       GD, p.dweight, p.dbias);
  }
  return hipGetLastError();
}

}  // namespace ssmvjp
