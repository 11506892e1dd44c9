// linear_scan.hip -- the linear recurrence with one state value per channel:
// whole sequences, their gradients, and one token on a pool of states.
//
//   log form:    a_t = exp(g_t),  u_t = x_t
//   gated form:  L_t = c softplus(decay) sigmoid(r_t), a_t = exp(-L_t),
//                u_t = m_t w_t x_t with m_t = sqrt(1 - a_t^2), w_t = sigmoid(i_t)
//   h_t = a_t h_{t-1} + u_t
// Adjoint, with l_t the gradient of h_t (l_t = dh_t + a_{t+1} l_{t+1}):
//   log form:    dx = l, dg = l a h_{t-1}
//   gated form:  dx = l m w, di = l m w x (1 - w),
//                E = L dJ/dL = l (w x a^2 (L/m) - L a h_{t-1}),
//                dr = E (1 - sigmoid(r)), ddecay = sigmoid(decay)/softplus(decay) sum E
// E is formed with L/m, which stays finite (sqrt(L/2)) where L and m go to zero.
#include "common.cuh"
#include "delta_seq.cuh"
#include "kernels.h"

namespace ssmvjp {
namespace {

struct ScanArgs {
  DeltaSeqs seq;
  i64 D;
  float c;
  const void *x, *gate, *igate;
  const float *decay, *h0;
  void* h;
  float *h_final, *ckpt;
  // backward
  const float* kept;
  const void* dh;
  const float* dh_final;
  void *dx, *dgate, *digate;
  float *part, *dh0;
};

__device__ __forceinline__ float sigmoid_hw(float z) { return __builtin_amdgcn_rcpf(1.0f + exp_hw(-z)); }

// per channel: c softplus(decay), and sigmoid(decay) / softplus(decay) (1 where both go to exp(decay))
__device__ __forceinline__ float decay_rate(float c, float z) { return c * softplus_f(z); }
__device__ __forceinline__ float decay_slope(float z) { return z < -16.0f ? 1.0f : sigmoid_f(z) / softplus_f(z); }

struct Token {
  float a, u;              // h = a h + u
  float L, m, sr, w, rm;   // gated form; rm = 1/m, 0 where m = 0
};

// 1 - exp(-y) loses what a has rounded away where y is small: there its series
__device__ __forceinline__ Token gated_token(float x, float r, float i, float rate) {
  Token t;
  t.sr = sigmoid_hw(r);
  t.w = sigmoid_hw(i);
  t.L = rate * t.sr;
  t.a = exp_hw(-t.L);
  const float y = 2.0f * t.L;
  const float series = y * fmaf(y, fmaf(y, fmaf(y, fmaf(y, fmaf(y, -1.0f / 720, 1.0f / 120), -1.0f / 24), 1.0f / 6), -0.5f), 1.0f);
  const float m2 = y < 0.25f ? series : fmaf(-t.a, t.a, 1.0f);
  t.rm = m2 >= 1.17549435e-38f ? __builtin_amdgcn_rsqf(m2) : 0.0f;  // the instruction takes denormals as zeros
  t.m = m2 * t.rm;
  t.u = t.m * t.w * x;
  return t;
}

template <typename T, bool GATED>
__device__ __forceinline__ Token load_token(const ScanArgs& a, i64 e, float rate, float& x) {
  x = ld((const T*)a.x, e);
  if constexpr (GATED) return gated_token(x, ld((const T*)a.gate, e), ld((const T*)a.igate, e), rate);
  Token t{};
  t.a = exp_hw(((const float*)a.gate)[e]);
  t.u = x;
  return t;
}

template <typename T, bool GATED>
__global__ void __launch_bounds__(64) scan_fwd_kernel(ScanArgs a) {
  const i64 ch = (i64)blockIdx.x * 64 + threadIdx.x, s = blockIdx.y;
  if (ch >= a.D) return;
  const DeltaSpan sp = a.seq.span(s);
  const float rate = GATED ? decay_rate(a.c, a.decay[ch]) : 0.0f;
  float h = a.h0 ? a.h0[s * a.D + ch] : 0.0f;
  for (i64 t = 0; t < sp.len; ++t) {
    if (a.ckpt && t % DCH == 0) a.ckpt[(sp.slot0 + t / DCH) * a.D + ch] = h;
    const i64 e = (sp.start + t) * a.D + ch;
    float x;
    const Token k = load_token<T, GATED>(a, e, rate, x);
    h = fmaf(k.a, h, k.u);
    if (a.h) st((T*)a.h, e, h);
  }
  if (a.h_final) a.h_final[s * a.D + ch] = h;
}

template <typename T, bool GATED>
__global__ void __launch_bounds__(64) scan_bwd_kernel(ScanArgs a) {
  const i64 ch = (i64)blockIdx.x * 64 + threadIdx.x, s = blockIdx.y;
  if (ch >= a.D) return;
  const DeltaSpan sp = a.seq.span(s);
  const float rate = GATED ? decay_rate(a.c, a.decay[ch]) : 0.0f;
  float carry = a.dh_final ? a.dh_final[s * a.D + ch] : 0.0f, sum = 0.0f;
  for (i64 j = (sp.len + DCH - 1) / DCH - 1; j >= 0; --j) {
    const int n = (int)(sp.len - j * DCH < DCH ? sp.len - j * DCH : DCH);
    float prev[DCH], x;
    float h = a.kept[(sp.slot0 + j) * a.D + ch];
    for (int t = 0; t < n; ++t) {
      prev[t] = h;
      const Token k = load_token<T, GATED>(a, (sp.start + j * DCH + t) * a.D + ch, rate, x);
      h = fmaf(k.a, h, k.u);
    }
    for (int t = n - 1; t >= 0; --t) {
      const i64 e = (sp.start + j * DCH + t) * a.D + ch;
      const Token k = load_token<T, GATED>(a, e, rate, x);
      const float l = ld((const T*)a.dh, e) + carry;
      carry = k.a * l;
      if constexpr (GATED) {
        const float lm = l * k.m * k.w, E = l * (k.w * x * k.a * k.a * (k.L * k.rm) - k.L * k.a * prev[t]);
        st((T*)a.dx, e, lm);
        st((T*)a.digate, e, lm * x * (1.0f - k.w));
        st((T*)a.dgate, e, E * (1.0f - k.sr));
        sum += E;
      } else {
        st((T*)a.dx, e, l);
        ((float*)a.dgate)[e] = carry * prev[t];
      }
    }
  }
  if (GATED) a.part[s * a.D + ch] = sum;
  if (a.dh0) a.dh0[s * a.D + ch] = carry;
}

__global__ void __launch_bounds__(64) decay_sum_kernel(const float* part, i64 n, i64 D, const float* decay, float* out) {
  const i64 ch = (i64)blockIdx.x * 64 + threadIdx.x;
  if (ch >= D) return;
  float sum = 0.0f;
  for (i64 i = 0; i < n; ++i) sum += part[i * D + ch];
  out[ch] = n > 0 ? sum * decay_slope(decay[ch]) : 0.0f;
}

// rows of ckpt that no token has
__global__ void __launch_bounds__(64) ckpt_clear_kernel(float* ckpt, i64 n) {
  for (i64 i = (i64)blockIdx.x * 64 + threadIdx.x; i < n; i += (i64)gridDim.x * 64) ckpt[i] = 0.0f;
}

struct StepArgs {
  i64 nslots, D, nblk;
  float c;
  const void *x, *gate, *igate;
  const float* decay;
  float* state;
  const int* slots;
  void* h;
};

template <typename T, bool GATED>
__global__ void __launch_bounds__(256) scan_step_kernel(StepArgs a) {
  const i64 req = blockIdx.x / a.nblk, ch = (blockIdx.x % a.nblk) * 256 + threadIdx.x;
  i64 slot = req;
  if (a.slots) {
    // every wave looks through the earlier requests for the same slot
    slot = a.slots[req];
    bool taken = slot < 0 || slot >= a.nslots;
    for (i64 j = threadIdx.x & 63; j < req; j += 64) taken |= a.slots[j] == (int)slot;
    if (__any(taken)) slot = -1;
  }
  if (ch >= a.D) return;
  const i64 e = req * a.D + ch;
  if (slot < 0) {
    st((T*)a.h, e, 0.0f);
    return;
  }
  const float x = ld((const T*)a.x, e);
  Token k{};
  if constexpr (GATED) {
    k = gated_token(x, ld((const T*)a.gate, e), ld((const T*)a.igate, e), decay_rate(a.c, a.decay[ch]));
  } else {
    k.a = exp_hw(((const float*)a.gate)[e]);
    k.u = x;
  }
  float* p = a.state + slot * a.D + ch;
  const float h = fmaf(k.a, *p, k.u);
  *p = h;
  st((T*)a.h, e, h);
}

DeltaSeqs scan_seqs(const ssmvjp_linear_scan_desc& d, const int* off) {
  return {d.packed ? off : nullptr, d.batch, d.seqlen, (d.seqlen + DCH - 1) / DCH};
}

}  // namespace

int64_t linear_scan_ckpt_rows(const ssmvjp_linear_scan_desc& d) {
  return d.packed ? d.seqlen / DCH + d.batch : d.batch * ((d.seqlen + DCH - 1) / DCH);
}

size_t linear_scan_fwd_workspace_bytes(const ssmvjp_linear_scan_desc&) { return 0; }

size_t linear_scan_bwd_workspace_bytes(const ssmvjp_linear_scan_desc& d) {
  return (size_t)(4 * (linear_scan_ckpt_rows(d) + d.batch) * d.dim);
}

hipError_t launch_linear_scan_fwd(const ssmvjp_linear_scan_desc& d, const LinearScanPointers& p, hipStream_t stream) {
  ScanArgs a{};
  a.seq = scan_seqs(d, p.seq_offsets);
  a.D = d.dim; a.c = d.c; a.x = p.x; a.gate = p.gate; a.igate = p.input_gate; a.decay = p.decay; a.h0 = p.h0;
  a.h = p.h; a.h_final = p.h_final; a.ckpt = p.ckpt;
  if (p.ckpt && linear_scan_ckpt_rows(d) > 0) hipLaunchKernelGGL(ckpt_clear_kernel, dim3(1024), dim3(64), 0, stream, p.ckpt, linear_scan_ckpt_rows(d) * d.dim);
  const dim3 grid((unsigned)((d.dim + 63) / 64), (unsigned)d.batch);
  const bool gated = d.form == SSMVJP_SCAN_GATED;
  if (d.dtype == SSMVJP_BF16) {
    if (gated) hipLaunchKernelGGL((scan_fwd_kernel<bf16, true>), grid, dim3(64), 0, stream, a);
    else hipLaunchKernelGGL((scan_fwd_kernel<bf16, false>), grid, dim3(64), 0, stream, a);
  } else {
    if (gated) hipLaunchKernelGGL((scan_fwd_kernel<float, true>), grid, dim3(64), 0, stream, a);
    else hipLaunchKernelGGL((scan_fwd_kernel<float, false>), grid, dim3(64), 0, stream, a);
  }
  return hipGetLastError();
}

hipError_t launch_linear_scan_bwd(const ssmvjp_linear_scan_desc& d, const LinearScanBwdPointers& p, hipStream_t stream) {
  float* states = (float*)p.workspace;
  float* part = states + linear_scan_ckpt_rows(d) * d.dim;
  const bool gated = d.form == SSMVJP_SCAN_GATED;
  if (d.batch > 0) {
    if (!p.ckpt) {
      const LinearScanPointers f{p.x, p.gate, p.input_gate, p.decay, p.h0, p.seq_offsets, nullptr, nullptr, states, nullptr};
      const hipError_t e = launch_linear_scan_fwd(d, f, stream);
      if (e != hipSuccess) return e;
    }
    ScanArgs a{};
    a.seq = scan_seqs(d, p.seq_offsets);
    a.D = d.dim; a.c = d.c; a.x = p.x; a.gate = p.gate; a.igate = p.input_gate; a.decay = p.decay; a.h0 = p.h0;
    a.kept = p.ckpt ? p.ckpt : states; a.dh = p.dh; a.dh_final = p.dh_final;
    a.dx = p.dx; a.dgate = p.dgate; a.digate = p.dinput_gate; a.part = part; a.dh0 = p.dh0;
    const dim3 grid((unsigned)((d.dim + 63) / 64), (unsigned)d.batch);
    if (d.dtype == SSMVJP_BF16) {
      if (gated) hipLaunchKernelGGL((scan_bwd_kernel<bf16, true>), grid, dim3(64), 0, stream, a);
      else hipLaunchKernelGGL((scan_bwd_kernel<bf16, false>), grid, dim3(64), 0, stream, a);
    } else {
      if (gated) hipLaunchKernelGGL((scan_bwd_kernel<float, true>), grid, dim3(64), 0, stream, a);
      else hipLaunchKernelGGL((scan_bwd_kernel<float, false>), grid, dim3(64), 0, stream, a);
    }
  }
  if (gated)
    hipLaunchKernelGGL(decay_sum_kernel, dim3((unsigned)((d.dim + 63) / 64)), dim3(64), 0, stream, part, d.batch, d.dim, p.decay, p.ddecay);
  return hipGetLastError();
}

hipError_t launch_linear_step(const ssmvjp_linear_step_desc& d, const LinearStepPointers& p, hipStream_t stream) {
  const StepArgs a{d.nslots, d.dim, (d.dim + 255) / 256, d.c, p.x, p.gate, p.input_gate, p.decay, p.state, p.slots, p.h};
  const dim3 grid((unsigned)(d.batch * a.nblk));
  const bool gated = d.form == SSMVJP_SCAN_GATED;
  if (d.dtype == SSMVJP_BF16) {
    if (gated) hipLaunchKernelGGL((scan_step_kernel<bf16, true>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((scan_step_kernel<bf16, false>), grid, dim3(256), 0, stream, a);
  } else {
    if (gated) hipLaunchKernelGGL((scan_step_kernel<float, true>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((scan_step_kernel<float, false>), grid, dim3(256), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace ssmvjp
