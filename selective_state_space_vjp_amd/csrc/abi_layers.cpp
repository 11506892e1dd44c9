// abi_layers.cpp -- the C ABI of the gated delta rule with one gate per head
// (chunked and one token) and of layer norm: argument validation, workspace
// sizing and dispatch.  Validation runs on the host and returns before anything
// is enqueued; nothing here allocates device memory or throws.
#include "abi_common.h"

namespace {

constexpr int64_t DIM_MAX = 0x7fffffff;

bool fits(double n) { return n <= (double)DIM_MAX; }
// a launch has fewer than 2^32 threads
bool launches(double groups, int threads) { return groups * threads < 4294967296.0; }

ssmvjp_status delta_dims_check(int64_t H, int64_t HV, int64_t K, int64_t V, int32_t dtype) {
  if (H <= 0 || HV <= 0 || K <= 0 || V <= 0 || HV % H || !valid_dtype(dtype)) return SSMVJP_EINVAL;
  if (K % 16 || K > 128 || V % 16) return SSMVJP_EUNSUPPORTED;
  // 32-bit byte offsets inside one chunk's rows and inside one state
  if (V > 65536 || H > (1 << 24) || HV > (1 << 24) || H * K >= (1 << 24) || HV * V >= (1 << 24)) return SSMVJP_EUNSUPPORTED;
  return SSMVJP_OK;
}

ssmvjp_status delta_chunk_check(const ssmvjp_delta_chunk_desc* d) {
  if (!d || d->batch < 0 || d->seqlen < 0 || d->reserved != 0 || (d->packed != 0 && d->packed != 1)) return SSMVJP_EINVAL;
  const ssmvjp_status s = delta_dims_check(d->nqk_heads, d->nv_heads, d->dk, d->dv, d->dtype);
  if (s != SSMVJP_OK) return s;
  // grids and workspace cells: 31-bit counts
  const double slots = d->packed ? (double)d->seqlen / 64 + (double)d->batch : (double)d->batch * ((double)d->seqlen / 64 + 1);
  if (!fits((double)d->batch) || !fits((double)d->seqlen) || !fits(slots * (double)d->nv_heads) ||
      !launches(slots * (double)d->nqk_heads, 512) ||
      !launches(2 * ((double)d->batch * (double)d->nv_heads + 8) * ((double)d->dv / 32 + 1), 320))
    return SSMVJP_EUNSUPPORTED;
  return SSMVJP_OK;
}

int64_t chunk_tokens(const ssmvjp_delta_chunk_desc& d) { return d.packed ? d.seqlen : d.batch * d.seqlen; }

// finite_check of a call's token tensors (`rows`, by the elements of one token) beside `outs`: with packed
// sequences only the tokens that one owns, since the call leaves the others alone
template <size_t K, size_t R>
ssmvjp_status finite_check_tokens(const ssmvjp_delta_chunk_desc& d, const int32_t* seq_offsets, void* workspace,
                                  size_t plan_bytes, const OutSpan (&outs)[K], const OutSpan (&rows)[R], hipStream_t stream) {
  return finite_check(workspace, plan_bytes, outs, stream, [&](unsigned* flag) {
    for (const OutSpan& r : rows)
      if (d.packed) launch_nonfinite_check_rows(r.p, r.n, r.bf16, seq_offsets, d.batch, d.seqlen, flag, stream);
      else launch_nonfinite_check(r.p, r.n * chunk_tokens(d), r.bf16, flag, stream);
  });
}

ssmvjp_status delta_step_check(const ssmvjp_delta_step_desc* d) {
  if (!d || d->batch < 0 || d->nslots < 0 || d->reserved != 0) return SSMVJP_EINVAL;
  if (d->gate != SSMVJP_GATE_PER_HEAD && d->gate != SSMVJP_GATE_PER_KEY) return SSMVJP_EINVAL;
  const ssmvjp_status s = delta_dims_check(d->nqk_heads, d->nv_heads, d->dk, d->dv, d->dtype);
  if (s != SSMVJP_OK) return s;
  if (!launches((double)d->batch * (double)d->nv_heads * ((double)d->dv / 64 + 1), 256) || !fits((double)d->nslots))
    return SSMVJP_EUNSUPPORTED;
  return SSMVJP_OK;
}

ssmvjp_status norm_check(const ssmvjp_norm_desc* d) {
  if (!d || d->rows < 0 || d->groups <= 0 || d->dim <= 0 || !valid_dtype(d->dtype)) return SSMVJP_EINVAL;
  if (!(d->eps >= 0.0f)) return SSMVJP_EINVAL;  // also NaN
  const double rows = (double)d->rows * (double)d->groups;
  if (rows * (double)d->dim * 4 > 9e18) return SSMVJP_EUNSUPPORTED;  // 64-bit byte offsets
  // the sums over the workgroups (32 of 2 groups dim columns each) and the kernels with one or more workgroups per
  // group, 2048 more than groups at most
  if (!fits(rows) || !launches((double)d->groups * (double)d->dim / 16 + 1, 1024) || !launches((double)d->groups + 2048, 256))
    return SSMVJP_EUNSUPPORTED;
  return SSMVJP_OK;
}

// every non-NULL pointer aligned to `a` bytes
template <size_t N>
bool all_aligned(const void* const (&ps)[N], size_t a) {
  for (const void* p : ps)
    if (p && !aligned(p, a)) return false;
  return true;
}

ssmvjp_status workspace_check(size_t need, const void* workspace, size_t workspace_bytes) {
  return need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)) ? SSMVJP_EWORKSPACE : SSMVJP_OK;
}

}  // namespace

extern "C" {

// ------------------------------ delta_chunk_fwd ------------------------------

ssmvjp_status delta_chunk_fwd_workspace(const ssmvjp_delta_chunk_desc* desc, size_t* bytes) {
  if (!bytes) return SSMVJP_EINVAL;
  const ssmvjp_status s = delta_chunk_check(desc);
  if (s != SSMVJP_OK) return s;
  *bytes = with_flag(delta_fwd_workspace_bytes(*desc));
  return SSMVJP_OK;
}

ssmvjp_status delta_chunk_fwd(const ssmvjp_delta_chunk_desc* desc, const void* q, const void* k, const void* v,
                              const float* beta, const float* g, const float* S0, const int32_t* seq_offsets, void* o,
                              float* S_final, void* workspace, size_t workspace_bytes, void* stream) {
  ssmvjp_status s = delta_chunk_check(desc);
  if (s != SSMVJP_OK) return s;
  const ssmvjp_delta_chunk_desc& d = *desc;
  const int64_t tokens = chunk_tokens(d);
  if (tokens > 0 && (!q || !k || !v || !beta || !g || !o)) return SSMVJP_EINVAL;
  if ((d.packed != 0) != (seq_offsets != nullptr)) return SSMVJP_EINVAL;
  const void* p16[] = {q, k, v, o, S0, S_final};
  const void* p4[] = {beta, g, seq_offsets};
  if (!all_aligned(p16, 16) || !all_aligned(p4, 4)) return SSMVJP_EINVAL;
  const size_t plan = delta_fwd_workspace_bytes(d);
  s = workspace_check(with_flag(plan), workspace, workspace_bytes);
  if (s != SSMVJP_OK) return s;
  if (d.batch == 0) return SSMVJP_OK;
  const DeltaChunkPointers ptr{q, k, v, beta, g, S0, seq_offsets, o, S_final, workspace};
  s = hip_status(launch_delta_fwd(d, ptr, (hipStream_t)stream));
  if (s != SSMVJP_OK || !check_finite_on()) return s;
  const OutSpan outs[] = {{S_final, d.batch * d.nv_heads * d.dk * d.dv, false}};
  const OutSpan rows[] = {{o, d.nv_heads * d.dv, d.dtype == SSMVJP_BF16}};
  return finite_check_tokens(d, seq_offsets, workspace, plan, outs, rows, (hipStream_t)stream);
}

// ------------------------------ delta_chunk_bwd ------------------------------

ssmvjp_status delta_chunk_bwd_workspace(const ssmvjp_delta_chunk_desc* desc, size_t* bytes) {
  if (!bytes) return SSMVJP_EINVAL;
  const ssmvjp_status s = delta_chunk_check(desc);
  if (s != SSMVJP_OK) return s;
  if (desc->dtype != SSMVJP_BF16) return SSMVJP_EUNSUPPORTED;
  *bytes = with_flag(delta_bwd_workspace_bytes(*desc));
  return SSMVJP_OK;
}

ssmvjp_status delta_chunk_bwd(const ssmvjp_delta_chunk_desc* desc, const void* q, const void* k, const void* v,
                              const float* beta, const float* g, const float* S0, const void* d_o,
                              const float* dS_final, const int32_t* seq_offsets, void* dq, void* dk, void* dv,
                              float* dbeta, float* dg, float* dS0, void* workspace, size_t workspace_bytes,
                              void* stream) {
  ssmvjp_status s = delta_chunk_check(desc);
  if (s != SSMVJP_OK) return s;
  const ssmvjp_delta_chunk_desc& d = *desc;
  if (d.dtype != SSMVJP_BF16) return SSMVJP_EUNSUPPORTED;
  const int64_t tokens = chunk_tokens(d);
  if (tokens > 0 && (!q || !k || !v || !beta || !g || !d_o || !dq || !dk || !dv || !dbeta || !dg)) return SSMVJP_EINVAL;
  if ((d.packed != 0) != (seq_offsets != nullptr)) return SSMVJP_EINVAL;
  const void* p16[] = {q, k, v, d_o, dq, dk, dv, S0, dS_final, dS0};
  const void* p4[] = {beta, g, seq_offsets, dbeta, dg};
  if (!all_aligned(p16, 16) || !all_aligned(p4, 4)) return SSMVJP_EINVAL;
  const size_t plan = delta_bwd_workspace_bytes(d);
  s = workspace_check(with_flag(plan), workspace, workspace_bytes);
  if (s != SSMVJP_OK) return s;
  if (d.batch == 0) return SSMVJP_OK;
  const DeltaChunkBwdPointers ptr{q, k, v, d_o, beta, g, S0, dS_final, seq_offsets, dq, dk, dv, dbeta, dg, dS0, workspace};
  s = hip_status(launch_delta_chunk_bwd(d, ptr, (hipStream_t)stream));
  if (s != SSMVJP_OK || !check_finite_on()) return s;
  const OutSpan outs[] = {{dS0, d.batch * d.nv_heads * d.dk * d.dv, false}};
  const OutSpan rows[] = {{dq, d.nqk_heads * d.dk, true}, {dk, d.nqk_heads * d.dk, true}, {dv, d.nv_heads * d.dv, true},
                          {dbeta, d.nv_heads, false}, {dg, d.nv_heads, false}};
  return finite_check_tokens(d, seq_offsets, workspace, plan, outs, rows, (hipStream_t)stream);
}

// -------------------------------- delta_step ---------------------------------

ssmvjp_status delta_step_workspace(const ssmvjp_delta_step_desc* desc, size_t* bytes) {
  if (!bytes) return SSMVJP_EINVAL;
  const ssmvjp_status s = delta_step_check(desc);
  if (s != SSMVJP_OK) return s;
  *bytes = with_flag(0);
  return SSMVJP_OK;
}

ssmvjp_status delta_step(const ssmvjp_delta_step_desc* desc, const void* q, const void* k, const void* v,
                         const float* beta, const float* g, float* state, const int32_t* slots, void* o,
                         void* workspace, size_t workspace_bytes, void* stream) {
  ssmvjp_status s = delta_step_check(desc);
  if (s != SSMVJP_OK) return s;
  const ssmvjp_delta_step_desc& d = *desc;
  if (d.batch > 0 && (!q || !k || !v || !beta || !g || !o || (d.nslots > 0 && !state))) return SSMVJP_EINVAL;
  if (!slots && d.nslots < d.batch) return SSMVJP_EINVAL;
  const void* p16[] = {q, k, v, o, state};
  const void* p4[] = {beta, g, slots};
  if (!all_aligned(p16, 16) || !all_aligned(p4, 4)) return SSMVJP_EINVAL;
  // per-key gates are read in vectors, like the keys they belong to
  if (d.gate == SSMVJP_GATE_PER_KEY && !aligned(g, 16)) return SSMVJP_EINVAL;
  s = workspace_check(with_flag(0), workspace, workspace_bytes);
  if (s != SSMVJP_OK || d.batch == 0) return s;
  const DeltaStepPointers ptr{q, k, v, beta, g, state, slots, o};
  s = hip_status(launch_delta_step(d, ptr, (hipStream_t)stream));
  if (s != SSMVJP_OK || !check_finite_on()) return s;
  const int64_t n = d.nv_heads * d.dk * d.dv;
  const OutSpan outs[] = {{o, d.batch * d.nv_heads * d.dv, d.dtype == SSMVJP_BF16}, {slots ? nullptr : state, d.batch * n, false}};
  return finite_check(workspace, 0, outs, (hipStream_t)stream, [&](unsigned* flag) {
    if (slots) launch_nonfinite_check_states(state, n, slots, d.batch, d.nslots, flag, (hipStream_t)stream);
  });
}

// -------------------------------- layer_norm ---------------------------------

ssmvjp_status layer_norm_fwd_workspace(const ssmvjp_norm_desc* desc, size_t* bytes) {
  if (!bytes) return SSMVJP_EINVAL;
  const ssmvjp_status s = norm_check(desc);
  if (s != SSMVJP_OK) return s;
  *bytes = with_flag(0);
  return SSMVJP_OK;
}

ssmvjp_status layer_norm_fwd(const ssmvjp_norm_desc* desc, const void* x, const float* weight, const float* bias, void* y,
                             float* mean, float* rstd, int8_t* x8, float* x8_scale, void* workspace,
                             size_t workspace_bytes, void* stream) {
  ssmvjp_status s = norm_check(desc);
  if (s != SSMVJP_OK) return s;
  const ssmvjp_norm_desc& d = *desc;
  if (d.rows > 0 && (!x || !y)) return SSMVJP_EINVAL;
  if ((x8 != nullptr) != (x8_scale != nullptr)) return SSMVJP_EINVAL;
  const void* pe[] = {x, y};
  const void* p4[] = {weight, bias, mean, rstd, x8_scale};
  if (!all_aligned(pe, big_elem(d.dtype)) || !all_aligned(p4, 4)) return SSMVJP_EINVAL;
  s = workspace_check(with_flag(0), workspace, workspace_bytes);
  if (s != SSMVJP_OK || d.rows == 0) return s;
  const NormFwdPointers ptr{x, weight, bias, y, mean, rstd, x8, x8_scale};
  s = hip_status(launch_norm_fwd(d, ptr, (hipStream_t)stream));
  if (s != SSMVJP_OK || !check_finite_on()) return s;
  const int64_t r = d.rows * d.groups;
  const OutSpan outs[] = {{y, r * d.dim, d.dtype == SSMVJP_BF16}, {mean, r, false}, {rstd, r, false},
                          {x8_scale, r * ((d.dim + 63) / 64), false}};
  return finite_check(workspace, 0, outs, (hipStream_t)stream);
}

ssmvjp_status layer_norm_bwd_workspace(const ssmvjp_norm_desc* desc, size_t* bytes) {
  if (!bytes) return SSMVJP_EINVAL;
  const ssmvjp_status s = norm_check(desc);
  if (s != SSMVJP_OK) return s;
  *bytes = with_flag(norm_bwd_workspace_bytes(*desc));
  return SSMVJP_OK;
}

ssmvjp_status layer_norm_bwd(const ssmvjp_norm_desc* desc, const void* dy, const void* x, const int8_t* x8,
                             const float* x8_scale, const float* mean, const float* rstd, const float* weight, void* dx,
                             float* dweight, float* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  ssmvjp_status s = norm_check(desc);
  if (s != SSMVJP_OK) return s;
  const ssmvjp_norm_desc& d = *desc;
  if (d.rows > 0 && (!dy || !mean || !rstd || !dx)) return SSMVJP_EINVAL;
  if ((x8 != nullptr) != (x8_scale != nullptr)) return SSMVJP_EINVAL;
  if (d.rows > 0 ? (x != nullptr) == (x8 != nullptr) : (x && x8)) return SSMVJP_EINVAL;  // one form of the input
  const void* pe[] = {dy, x, dx};
  const void* p4[] = {x8_scale, mean, rstd, weight, dweight, dbias};
  if (!all_aligned(pe, big_elem(d.dtype)) || !all_aligned(p4, 4)) return SSMVJP_EINVAL;
  const size_t plan = norm_bwd_workspace_bytes(d);
  s = workspace_check(with_flag(plan), workspace, workspace_bytes);
  if (s != SSMVJP_OK) return s;
  const NormBwdPointers ptr{dy, x, x8, x8_scale, mean, rstd, weight, dx, dweight, dbias, workspace};
  s = hip_status(launch_norm_bwd(d, ptr, (hipStream_t)stream));
  if (s != SSMVJP_OK || !check_finite_on()) return s;
  const OutSpan outs[] = {{dx, d.rows * d.groups * d.dim, d.dtype == SSMVJP_BF16},
                          {dweight, d.groups * d.dim, false}, {dbias, d.groups * d.dim, false}};
  return finite_check(workspace, plan, outs, (hipStream_t)stream);
}

}  // extern "C"
