// delta_step.hip -- the gated delta rule token by token: one token per request
// on a pool of states (serving), and whole sequences where the chunked kernels
// do not apply or not pay (float32, up to 16 tokens).
//
//   S_dec = a_t S_{t-1} (a_t = exp(g_t): one per value head, or one per key
//   channel);  r = v_t - k_t^T S_dec;  u = beta_t r;  S_t = S_dec + k_t (x) u
//   o_t = scale q_t^T S_t = scale (q_t^T S_dec + (q_t . k_t) u)
// The second form of o_t needs S_dec only, so k^T S_dec, q^T S_dec and q . k are
// summed over the rows in one exchange.  States and sums are float32.
//
// One token reads and writes K V floats per head and does 6 K V operations on
// them: it is bound by the states' traffic.  Columns of S are independent, so a
// wave owns 16 columns (64-byte row segments; the four waves of a workgroup
// own 256 adjacent bytes of each row) and all K rows: lane (row group lane / 4,
// column quad lane % 4) holds K/16 consecutive rows of four columns in
// registers, the row sums are two DPP rotations and two permlane swaps, and
// there is no LDS and no barrier.
// 256 requests of HV=32 K=V=128: 221 us, 1.08 GB at 4.9 TB/s (a device copy moves
// 5.2); one request: 4.4 us, a launch and one round trip to memory.
//
// Whole sequences: the same with the state kept in registers from the first
// token to the last; the inputs of the next four tokens are in flight while
// one is computed (a token takes less time than a load's latency).
#include "common.cuh"
#include "delta_seq.cuh"
#include "kernels.h"

namespace ssmvjp {
namespace {

struct StepArgs {
  DeltaSeqs seq;
  i64 nslots, H, HV, V, ncol, rep;
  float scale;
  const void *q, *k, *v;
  const float *beta, *g;
  const float* S0;
  float* S;  // step: the pool; walk: the final states (NULL: not wanted)
  const int* slots;
  void* o;
};

// M consecutive elements (a lane's rows) as floats
template <int M, typename T>
__device__ __forceinline__ void load_rows(const T* p, float (&o)[M]) {
  constexpr int B = M * (int)sizeof(T), AL = B % 16 == 0 ? 16 : B % 8 == 0 ? 8 : B % 4 == 0 ? 4 : 2;
  T t[M];
  __builtin_memcpy(t, __builtin_assume_aligned(p, AL), B);
#pragma unroll
  for (int i = 0; i < M; ++i) o[i] = (float)t[i];
}
__device__ __forceinline__ void load4(const float* p, float (&o)[4]) {
  const float4 u = *(const float4*)p;
  o[0] = u.x; o[1] = u.y; o[2] = u.z; o[3] = u.w;
}
__device__ __forceinline__ void load4(const bf16* p, float (&o)[4]) {
  const uint2 u = *(const uint2*)p;
  o[0] = __uint_as_float(u.x << 16); o[1] = __uint_as_float(u.x & 0xffff0000u);
  o[2] = __uint_as_float(u.y << 16); o[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void store_o(float* p, const float (&o)[4]) { *(float4*)p = make_float4(o[0], o[1], o[2], o[3]); }
__device__ __forceinline__ void store_o(bf16* p, const float (&o)[4]) {
  *(uint2*)p = make_uint2(pk_bf16(o[0], o[1]), pk_bf16(o[2], o[3]));
}

// sum over the 16 lanes of the same lane % 4
__device__ __forceinline__ float sum_rows(float v) {
  v += dpp_f<0x128>(v);  // row_ror:8
  v += dpp_f<0x124>(v);  // row_ror:4
  return sum4q(v);
}

template <int M, bool KEYG>
struct Token {
  float k[M], q[M], v[4], beta, g[KEYG ? M : 1];
};

template <typename T, int M, bool KEYG>
__device__ __forceinline__ Token<M, KEYG> load_token(const StepArgs& a, i64 tok, i64 hv, int rg, i64 col) {
  constexpr i64 K = 16 * M;
  Token<M, KEYG> x;
  const i64 qk = (tok * a.H + hv / a.rep) * K + rg * M, th = tok * a.HV + hv;
  load_rows<M>((const T*)a.k + qk, x.k);
  load_rows<M>((const T*)a.q + qk, x.q);
  load4((const T*)a.v + th * a.V + col, x.v);
  x.beta = a.beta[th];
  if constexpr (KEYG)
    load_rows<M>(a.g + th * K + rg * M, x.g);
  else
    x.g[0] = a.g[th];
  return x;
}

// one token on this lane's part of the state; o: its four columns of the readout
template <int M, bool KEYG>
__device__ __forceinline__ void token_update(const Token<M, KEYG>& x, float scale, float (&S)[M][4], float (&o)[4]) {
  float kd[4] = {0.f, 0.f, 0.f, 0.f}, qd[4] = {0.f, 0.f, 0.f, 0.f}, qk = 0.0f;
  const float ah = KEYG ? 0.0f : expf(x.g[0]);
#pragma unroll
  for (int i = 0; i < M; ++i) {
    const float ai = KEYG ? expf(x.g[KEYG ? i : 0]) : ah;
    qk = fmaf(x.q[i], x.k[i], qk);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      S[i][c] *= ai;
      kd[c] = fmaf(x.k[i], S[i][c], kd[c]);
      qd[c] = fmaf(x.q[i], S[i][c], qd[c]);
    }
  }
  qk = sum_rows(qk);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float u = x.beta * (x.v[c] - sum_rows(kd[c]));
    o[c] = scale * fmaf(qk, u, sum_rows(qd[c]));
#pragma unroll
    for (int i = 0; i < M; ++i) S[i][c] = fmaf(x.k[i], u, S[i][c]);
  }
}

template <int M>
__device__ __forceinline__ void load_state(const float* p, i64 V, int rg, i64 col, float (&S)[M][4]) {
#pragma unroll
  for (int i = 0; i < M; ++i) load4(p + (i64)(rg * M + i) * V + col, S[i]);
}
template <int M>
__device__ __forceinline__ void store_state(float* p, i64 V, int rg, i64 col, const float (&S)[M][4]) {
#pragma unroll
  for (int i = 0; i < M; ++i) store_o(p + (i64)(rg * M + i) * V + col, S[i]);
}

template <typename T, int M, bool KEYG>
__global__ void __launch_bounds__(256) delta_step_kernel(StepArgs a) {
  const int lane = threadIdx.x & 63, rg = lane >> 2;
  const i64 hv = blockIdx.x / a.ncol % a.HV, n = blockIdx.x / a.ncol / a.HV;
  const i64 c0 = (blockIdx.x % a.ncol) * 64 + (threadIdx.x >> 6) * 16, col = c0 + 4 * (lane & 3);
  if (c0 >= a.V) return;
  i64 slot = n;
  bool run = true;
  if (a.slots) {
    slot = a.slots[n];
    run = slot >= 0 && slot < a.nslots;
    // a slot named again belongs to the first request that names it: two
    // updates of one state would race
    int dup = 0;
    for (i64 j = lane; j < n; j += 64) dup |= a.slots[j] == (int)slot;
    run = run && !__any(dup);
  }
  T* o = (T*)a.o + (n * a.HV + hv) * a.V + col;
  float out[4] = {0.f, 0.f, 0.f, 0.f};
  if (run) {
    float S[M][4];
    float* st = a.S + (slot * a.HV + hv) * (16 * M) * a.V;
    load_state<M>(st, a.V, rg, col, S);
    const Token<M, KEYG> x = load_token<T, M, KEYG>(a, n, hv, rg, col);
    token_update<M, KEYG>(x, a.scale, S, out);
    store_state<M>(st, a.V, rg, col, S);
  }
  if (rg == 0) store_o(o, out);
}

constexpr int AHEAD = 4;

template <typename T, int M>
__global__ void __launch_bounds__(256) delta_walk_kernel(StepArgs a) {
  const int lane = threadIdx.x & 63, rg = lane >> 2;
  const i64 hv = blockIdx.x / a.ncol % a.HV, n = blockIdx.x / a.ncol / a.HV;
  const i64 c0 = (blockIdx.x % a.ncol) * 64 + (threadIdx.x >> 6) * 16, col = c0 + 4 * (lane & 3);
  if (c0 >= a.V) return;
  const DeltaSpan sp = a.seq.span(n);
  float S[M][4];
  const i64 sb = (n * a.HV + hv) * (16 * M) * a.V;
  if (a.S0) {
    load_state<M>(a.S0 + sb, a.V, rg, col, S);
  } else {
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) S[i][c] = 0.0f;
  }
  if (sp.len > 0) {
    Token<M, false> x[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
      x[j] = load_token<T, M, false>(a, sp.start + (j < sp.len ? j : sp.len - 1), hv, rg, col);
    for (i64 t = 0; t < sp.len; t += AHEAD) {
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        if (t + j < sp.len) {
          float o[4];
          token_update<M, false>(x[j], a.scale, S, o);
          if (rg == 0) store_o((T*)a.o + ((sp.start + t + j) * a.HV + hv) * a.V + col, o);
          const i64 nx = t + j + AHEAD;
          x[j] = load_token<T, M, false>(a, sp.start + (nx < sp.len ? nx : sp.len - 1), hv, rg, col);
        }
      }
    }
  }
  if (a.S) store_state<M>(a.S + sb, a.V, rg, col, S);
}

template <typename T, int M>
void launch_step_m(const StepArgs& a, bool keyg, i64 blocks, hipStream_t s) {
  if (keyg) hipLaunchKernelGGL((delta_step_kernel<T, M, true>), dim3((unsigned)blocks), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((delta_step_kernel<T, M, false>), dim3((unsigned)blocks), dim3(256), 0, s, a);
}
template <typename T, int M>
void launch_walk_m(const StepArgs& a, i64 blocks, hipStream_t s) {
  hipLaunchKernelGGL((delta_walk_kernel<T, M>), dim3((unsigned)blocks), dim3(256), 0, s, a);
}

template <typename T, bool STEP>
void launch_rows(const StepArgs& a, int m, bool keyg, i64 blocks, hipStream_t s) {
#define SSMVJP_M(N)                                       \
  case N:                                                 \
    if constexpr (STEP) launch_step_m<T, N>(a, keyg, blocks, s); \
    else launch_walk_m<T, N>(a, blocks, s);               \
    break;
  switch (m) {
    SSMVJP_M(1) SSMVJP_M(2) SSMVJP_M(3) SSMVJP_M(4) SSMVJP_M(5) SSMVJP_M(6) SSMVJP_M(7) SSMVJP_M(8)
  }
#undef SSMVJP_M
}

}  // namespace

hipError_t launch_delta_step(const ssmvjp_delta_step_desc& d, const DeltaStepPointers& p, hipStream_t stream) {
  StepArgs a{};
  a.nslots = d.nslots; a.H = d.nqk_heads; a.HV = d.nv_heads; a.V = d.dv; a.ncol = (d.dv + 63) / 64;
  a.rep = d.nv_heads / d.nqk_heads; a.scale = d.scale;
  a.q = p.q; a.k = p.k; a.v = p.v; a.beta = p.beta; a.g = p.g; a.S = p.state; a.slots = p.slots; a.o = p.o;
  const i64 blocks = d.batch * d.nv_heads * a.ncol;
  const bool keyg = d.gate == SSMVJP_GATE_PER_KEY;
  if (d.dtype == SSMVJP_BF16) launch_rows<bf16, true>(a, (int)(d.dk / 16), keyg, blocks, stream);
  else launch_rows<float, true>(a, (int)(d.dk / 16), keyg, blocks, stream);
  return hipGetLastError();
}

hipError_t launch_delta_walk(const ssmvjp_delta_chunk_desc& d, const DeltaChunkPointers& p, hipStream_t stream) {
  StepArgs a{};
  a.seq = delta_seqs(d, p.seq_offsets);
  a.H = d.nqk_heads; a.HV = d.nv_heads; a.V = d.dv; a.ncol = (d.dv + 63) / 64;
  a.rep = d.nv_heads / d.nqk_heads; a.scale = d.scale;
  a.q = p.q; a.k = p.k; a.v = p.v; a.beta = p.beta; a.g = p.g; a.S0 = p.S0; a.S = p.S_final; a.o = p.o;
  const i64 blocks = d.batch * d.nv_heads * a.ncol;
  if (d.dtype == SSMVJP_BF16) launch_rows<bf16, false>(a, (int)(d.dk / 16), false, blocks, stream);
  else launch_rows<float, false>(a, (int)(d.dk / 16), false, blocks, stream);
  return hipGetLastError();
}

}  // namespace ssmvjp
