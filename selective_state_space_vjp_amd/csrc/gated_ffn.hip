// gated_ffn.hip -- the projections of a gated feed-forward block and their
// gradients: h = act(x Wg^T) * (x Wu^T).
//
// Every product is C(m,n) = sum_k A(m,k) B(n,k) on tiles of the matrix cores:
//   forward        A = x, B = Wg and Wu (two products that share A; the
//                  activation and the product are applied to the sums)
//   dx             A = dgate, dup (one behind the other along k), B = Wg^T, Wu^T
//   dWg, dWu       A = dgate^T, dup^T, B = x^T
// k runs along the rows of an operand in memory (KC) or down its columns.
#include "common.cuh"
#include "kernels.h"

namespace ssmvjp {
namespace {

struct Operand {
  const void* p;
  i64 ld;
};

struct FfnArgs {
  i64 M, N, K;          // K: of one segment
  Operand A[2], B[2];   // PAIR: A[0] with both B; else segments of k
  int segs;
  i64 ldc;
  void* C[3];           // h, gate, up | dgate, dup | C
  const void *dh;       // BACK: [M, N]
};

enum { EPI_PLAIN, EPI_GLU, EPI_GLU_BACK };

// act and its derivative at z
template <int ACT>
__device__ __forceinline__ void act_pair(float z, float& f, float& df) {
  if constexpr (ACT == SSMVJP_ACT_SILU) {
    const float s = __builtin_amdgcn_rcpf(1.0f + exp_hw(-z));
    f = z * s;
    df = fmaf(f, 1.0f - s, s);
  } else {
    // (1 + tanh(v)) / 2 = sigmoid(2 v)
    const float k = 1.5957691216057308f, z2 = z * z;
    const float s = __builtin_amdgcn_rcpf(1.0f + exp_hw(-k * z * fmaf(0.044715f, z2, 1.0f)));
    f = z * s;
    df = fmaf(f * (1.0f - s), k * fmaf(0.134145f, z2, 1.0f), s);
  }
}
template <int ACT>
__device__ __forceinline__ float act_of(float z) {
  float f, df;
  act_pair<ACT>(z, f, df);
  return f;
}

constexpr int TM = 64, TN = 64, TK = 32;

// TMN x TK values of an operand into LDS, [mn][k] (KC) or [k][mn]; zeros outside
template <typename T, bool KC>
__device__ __forceinline__ void stage(T* lds, const Operand& o, i64 mn0, i64 MN, i64 k0, i64 K, int tid) {
  constexpr int W = 16 / sizeof(T), cols = KC ? TK : TM, rows = KC ? TM : TK, pitch = cols + W;
  for (int i = tid; i < rows * cols / W; i += 256) {
    const int r = i / (cols / W), c = i % (cols / W) * W;
    const i64 gr = (KC ? mn0 : k0) + r, gc = (KC ? k0 : mn0) + c;
    uint4 v = {0u, 0u, 0u, 0u};
    if (gr < (KC ? MN : K) && gc < (KC ? K : MN)) v = *(const uint4*)((const T*)o.p + gr * o.ld + gc);
    *(uint4*)(lds + r * pitch + c) = v;
  }
}

template <typename T, bool KC>
__device__ __forceinline__ Frag<T> frag_of(const T* lds, int mn, int k, int lane) {
  constexpr int W = 16 / sizeof(T);
  if constexpr (KC) return ld_colk(lds, TK + W, mn, k, lane);
  else return ld_rowk(lds, TM + W, k, mn, lane);
}

template <typename T, bool AKC, bool BKC, int EPI, int ACT>
__global__ void __launch_bounds__(256) ffn_gemm_kernel(FfnArgs a) {
  constexpr bool PAIR = EPI != EPI_PLAIN;
  constexpr int LDSN = 64 * 40 > 32 * 72 ? 64 * 40 : 32 * 72;
  __shared__ __align__(16) T sA[LDSN], sB[PAIR ? 2 : 1][LDSN];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const i64 m0 = (i64)blockIdx.y * TM, n0 = (i64)blockIdx.x * TN;
  const int wm = (wave & 1) * 32, wn = (wave >> 1) * 32;
  f32x4 acc[PAIR ? 2 : 1][2][2];
#pragma unroll
  for (int p = 0; p < (PAIR ? 2 : 1); ++p)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[p][i >> 1][i & 1] = zero4();
  for (int s = 0; s < (PAIR ? 1 : a.segs); ++s)
    for (i64 k0 = 0; k0 < a.K; k0 += TK) {
      stage<T, AKC>(sA, a.A[s], m0, a.M, k0, a.K, tid);
      stage<T, BKC>(sB[0], a.B[s], n0, a.N, k0, a.K, tid);
      if constexpr (PAIR) stage<T, BKC>(sB[1], a.B[1], n0, a.N, k0, a.K, tid);
      __syncthreads();
#pragma unroll
      for (int k = 0; k < TK; k += 16) {
        Frag<T> fa[2], fb[PAIR ? 2 : 1][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) fa[i] = frag_of<T, AKC>(sA, wm + 16 * i, k, lane);
#pragma unroll
        for (int p = 0; p < (PAIR ? 2 : 1); ++p)
#pragma unroll
          for (int j = 0; j < 2; ++j) fb[p][j] = frag_of<T, BKC>(sB[p], wn + 16 * j, k, lane);
#pragma unroll
        for (int p = 0; p < (PAIR ? 2 : 1); ++p)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) mma(acc[p][i][j], fa[i], fb[p][j]);
      }
      __syncthreads();
    }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const i64 m = m0 + wm + 16 * i + 4 * (lane >> 4) + r, n = n0 + wn + 16 * j + (lane & 15);
        if (m >= a.M || n >= a.N) continue;
        const i64 e = m * a.ldc + n;
        if constexpr (EPI == EPI_PLAIN) {
          st((T*)a.C[0], e, acc[0][i][j][r]);
        } else if constexpr (EPI == EPI_GLU) {
          const float g = acc[0][i][j][r], u = acc[1][i][j][r];
          st((T*)a.C[0], e, act_of<ACT>(g) * u);
          if (a.C[1]) {
            st((T*)a.C[1], e, g);
            st((T*)a.C[2], e, u);
          }
        } else {
          float f, df;
          act_pair<ACT>(acc[0][i][j][r], f, df);
          const float dh = ld((const T*)a.dh, e);
          st((T*)a.C[0], e, dh * acc[1][i][j][r] * df);
          st((T*)a.C[1], e, dh * f);
        }
      }
}

// dgate, dup from the kept gate and up
template <typename T, int ACT>
__global__ void __launch_bounds__(256) ffn_grad_kernel(const T* dh, const T* gate, const T* up, T* dgate, T* dup, i64 n) {
  for (i64 e = (i64)blockIdx.x * 256 + threadIdx.x; e < n; e += (i64)gridDim.x * 256) {
    float f, df;
    act_pair<ACT>(ld(gate, e), f, df);
    const float d = ld(dh, e);
    st(dgate, e, d * ld(up, e) * df);
    st(dup, e, d * f);
  }
}

template <typename T, bool AKC, bool BKC, int EPI, int ACT>
void launch_gemm(const FfnArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.N + TN - 1) / TN), (unsigned)((a.M + TM - 1) / TM));
  hipLaunchKernelGGL((ffn_gemm_kernel<T, AKC, BKC, EPI, ACT>), grid, dim3(256), 0, s, a);
}

template <typename T, int ACT>
void ffn_fwd(const ssmvjp_ffn_desc& d, const FfnFwdPointers& p, hipStream_t s) {
  FfnArgs a{d.rows, d.hidden, d.dim, {{p.x, d.dim}}, {{p.w_gate, d.dim}, {p.w_up, d.dim}}, 1, d.hidden, {p.h, p.gate, p.up}, nullptr};
  launch_gemm<T, true, true, EPI_GLU, ACT>(a, s);
}

template <typename T, int ACT>
void ffn_bwd(const ssmvjp_ffn_desc& d, const FfnBwdPointers& p, hipStream_t s) {
  const i64 n = d.rows * d.hidden;
  T *dgate = (T*)p.workspace, *dup = dgate + n;
  if (n > 0) {
    if (p.gate) {
      const i64 blocks = (n + 255) / 256 < 65536 ? (n + 255) / 256 : 65536;
      hipLaunchKernelGGL((ffn_grad_kernel<T, ACT>), dim3((unsigned)blocks), dim3(256), 0, s, (const T*)p.dh, (const T*)p.gate,
                         (const T*)p.up, dgate, dup, n);
    } else {
      FfnArgs a{d.rows, d.hidden, d.dim, {{p.x, d.dim}}, {{p.w_gate, d.dim}, {p.w_up, d.dim}}, 1, d.hidden, {dgate, dup}, p.dh};
      launch_gemm<T, true, true, EPI_GLU_BACK, ACT>(a, s);
    }
    if (p.dx) {
      FfnArgs a{d.rows, d.dim, d.hidden, {{dgate, d.hidden}, {dup, d.hidden}}, {{p.w_gate, d.dim}, {p.w_up, d.dim}}, 2, d.dim, {p.dx}, nullptr};
      launch_gemm<T, true, false, EPI_PLAIN, 0>(a, s);
    }
  }
  for (int w = 0; w < 2; ++w) {
    void* out = w ? p.dw_up : p.dw_gate;
    if (!out) continue;
    FfnArgs a{d.hidden, d.dim, d.rows, {{w ? dup : dgate, d.hidden}}, {{p.x, d.dim}}, 1, d.dim, {out}, nullptr};
    launch_gemm<T, false, false, EPI_PLAIN, 0>(a, s);
  }
}

}  // namespace

size_t ffn_fwd_workspace_bytes(const ssmvjp_ffn_desc&) { return 0; }
size_t ffn_bwd_workspace_bytes(const ssmvjp_ffn_desc& d) {
  return (size_t)(2 * d.rows * d.hidden * (d.dtype == SSMVJP_BF16 ? 2 : 4));
}

hipError_t launch_ffn_fwd(const ssmvjp_ffn_desc& d, const FfnFwdPointers& p, hipStream_t stream) {
  const bool gelu = d.act == SSMVJP_ACT_GELU;
  if (d.dtype == SSMVJP_BF16) {
    if (gelu) ffn_fwd<bf16, SSMVJP_ACT_GELU>(d, p, stream);
    else ffn_fwd<bf16, SSMVJP_ACT_SILU>(d, p, stream);
  } else {
    if (gelu) ffn_fwd<float, SSMVJP_ACT_GELU>(d, p, stream);
    else ffn_fwd<float, SSMVJP_ACT_SILU>(d, p, stream);
  }
  return hipGetLastError();
}

hipError_t launch_ffn_bwd(const ssmvjp_ffn_desc& d, const FfnBwdPointers& p, hipStream_t stream) {
  const bool gelu = d.act == SSMVJP_ACT_GELU;
  if (d.dtype == SSMVJP_BF16) {
    if (gelu) ffn_bwd<bf16, SSMVJP_ACT_GELU>(d, p, stream);
    else ffn_bwd<bf16, SSMVJP_ACT_SILU>(d, p, stream);
  } else {
    if (gelu) ffn_bwd<float, SSMVJP_ACT_GELU>(d, p, stream);
    else ffn_bwd<float, SSMVJP_ACT_SILU>(d, p, stream);
  }
  return hipGetLastError();
}

}  // namespace ssmvjp
