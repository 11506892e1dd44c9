// finite.hip -- the debug finiteness check behind SSMVJP_CHECK_FINITE: a scan
// of an output tensor that raises a flag if any element is NaN or infinite.
// Every writer stores the same value, so the flag does not depend on the order
// in which the threads run.
#include "common.cuh"
#include "delta_seq.cuh"
#include "kernels.h"

namespace ssmvjp {
namespace {

__global__ void __launch_bounds__(256) flag_clear_kernel(unsigned* flag) {
  if (threadIdx.x == 0) *flag = 0u;
}

template <typename T>
__global__ void __launch_bounds__(256) nonfinite_scan_kernel(const T* p, i64 n, unsigned* flag) {
  bool bad = false;
  for (i64 i = (i64)blockIdx.x * 256 + threadIdx.x; i < n; i += (i64)gridDim.x * 256) bad |= nonfinite((float)p[i]);
  if (bad) *flag = 1u;
}

// ---- outputs of which a call writes a part that only device memory knows ----
// elements [lo, hi) of part i: the rows of a packed call's sequence (rising: a border below one before it counts as that
// one, as in the linear recurrence; called by whole waves) ...
struct OwnedRows {
  DeltaSeqs seq;
  i64 n;  // elements of a row
  bool rising;
  __device__ __forceinline__ void part(i64 i, i64& lo, i64& hi) const {
    const DeltaSpan sp = seq.span(i);
    const i64 start = rising ? seq.risen(i, threadIdx.x & 63) : sp.start, end = sp.start + sp.len;
    lo = start * n;
    hi = end > start ? end * n : lo;
  }
};
// ... or the state that request i names (nothing where it names none)
struct NamedStates {
  const int* slots;
  i64 nslots, n;  // n: elements of a state
  __device__ __forceinline__ void part(i64 i, i64& lo, i64& hi) const {
    const i64 s = slots[i];
    const bool in = s >= 0 && s < nslots;
    lo = in ? s * n : 0;
    hi = in ? lo + n : 0;
  }
};

template <typename T, typename Parts>
__global__ void __launch_bounds__(256) nonfinite_parts_kernel(const T* p, Parts parts, i64 count, unsigned* flag) {
  bool bad = false;
  for (i64 i = blockIdx.y; i < count; i += gridDim.y) {
    i64 lo, hi;
    parts.part(i, lo, hi);
    for (i64 e = lo + (i64)blockIdx.x * 256 + threadIdx.x; e < hi; e += (i64)gridDim.x * 256) bad |= nonfinite((float)p[e]);
  }
  if (bad) *flag = 1u;
}

dim3 parts_grid(i64 count) { return dim3(64, (unsigned)(count < 1024 ? count : 1024)); }

}  // namespace

void launch_flag_clear(unsigned* flag, hipStream_t stream) {
  hipLaunchKernelGGL(flag_clear_kernel, dim3(1), dim3(64), 0, stream, flag);
}

void launch_nonfinite_check(const void* p, int64_t n, bool is_bf16, unsigned* flag, hipStream_t stream) {
  if (!p || n <= 0) return;
  const i64 blocks = (n + 255) / 256 < 1024 ? (n + 255) / 256 : 1024;
  if (is_bf16)
    hipLaunchKernelGGL(nonfinite_scan_kernel<bf16>, dim3((unsigned)blocks), dim3(256), 0, stream, (const bf16*)p, n,
                       flag);
  else
    hipLaunchKernelGGL(nonfinite_scan_kernel<float>, dim3((unsigned)blocks), dim3(256), 0, stream, (const float*)p, n,
                       flag);
}

void launch_nonfinite_check_rows(const void* p, int64_t n, bool is_bf16, const int32_t* seq_offsets, int64_t nseq,
                                 int64_t tokens, bool rising, unsigned* flag, hipStream_t stream) {
  if (!p || n <= 0 || nseq <= 0) return;
  const OwnedRows parts{{seq_offsets, nseq, tokens, 0}, n, rising};
  if (is_bf16)
    hipLaunchKernelGGL((nonfinite_parts_kernel<bf16, OwnedRows>), parts_grid(nseq), dim3(256), 0, stream, (const bf16*)p,
                       parts, nseq, flag);
  else
    hipLaunchKernelGGL((nonfinite_parts_kernel<float, OwnedRows>), parts_grid(nseq), dim3(256), 0, stream, (const float*)p,
                       parts, nseq, flag);
}

void launch_nonfinite_check_states(const float* p, int64_t n, const int32_t* slots, int64_t batch, int64_t nslots,
                                   unsigned* flag, hipStream_t stream) {
  if (!p || n <= 0 || batch <= 0) return;
  hipLaunchKernelGGL((nonfinite_parts_kernel<float, NamedStates>), parts_grid(batch), dim3(256), 0, stream, p,
                     NamedStates{slots, nslots, n}, batch, flag);
}

}  // namespace ssmvjp
