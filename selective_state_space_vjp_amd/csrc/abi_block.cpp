// abi_block.cpp -- the C ABI of the parts of a residual layer around a scan: the
// linear recurrence (sequences, gradients, one token), the gated feed-forward
// projections and dropout: argument validation, workspace sizing and dispatch.
// Validation runs on the host and returns before anything is enqueued; nothing
// here allocates device memory or throws.
#include "abi_common.h"

namespace {

// a launch has fewer than 2^32 threads
bool launches(double groups, int threads) { return groups * threads < 4294967296.0; }
constexpr double DIM_MAX = 0x7fffffff;

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

ssmvjp_status scan_form_check(int32_t form, int32_t dtype, float c, int64_t dim) {
  if (dim <= 0 || !valid_dtype(dtype) || (form != SSMVJP_SCAN_LOG && form != SSMVJP_SCAN_GATED)) return SSMVJP_EINVAL;
  if (form == SSMVJP_SCAN_GATED && !(c > 0.0f && c <= 3.402823466e38f)) return SSMVJP_EINVAL;  // also NaN
  return dim >= (1 << 24) ? SSMVJP_EUNSUPPORTED : SSMVJP_OK;  // 32-bit byte offsets inside a wave's 16 tokens
}

ssmvjp_status linear_scan_check(const ssmvjp_linear_scan_desc* d) {
  if (!d || d->batch < 0 || d->seqlen < 0 || (d->packed != 0 && d->packed != 1)) return SSMVJP_EINVAL;
  const ssmvjp_status s = scan_form_check(d->form, d->dtype, d->c, d->dim);
  if (s != SSMVJP_OK) return s;
  const double slots = d->packed ? (double)d->seqlen / 64 + (double)d->batch : (double)d->batch * ((double)d->seqlen / 64 + 1);
  if ((double)d->batch > DIM_MAX || (double)d->seqlen > DIM_MAX || !launches((slots + 1) * ((double)d->dim / 64 + 1), 512))
    return SSMVJP_EUNSUPPORTED;
  return SSMVJP_OK;
}

int64_t scan_tokens(const ssmvjp_linear_scan_desc& d) { return d.packed ? d.seqlen : d.batch * d.seqlen; }

// what both directions ask of their inputs; `tokens` > 0: the token tensors are read
ssmvjp_status scan_inputs_check(const ssmvjp_linear_scan_desc& d, const void* x, const void* gate, const void* input_gate,
                                const float* decay, const float* h0, const int32_t* seq_offsets) {
  const bool gated = d.form == SSMVJP_SCAN_GATED;
  if (scan_tokens(d) > 0 && (!x || !gate || (gated && (!input_gate || !decay)))) return SSMVJP_EINVAL;
  if (!gated && (input_gate || decay)) return SSMVJP_EINVAL;
  if ((d.packed != 0) != (seq_offsets != nullptr)) return SSMVJP_EINVAL;
  const void* pe[] = {x, input_gate, gated ? gate : nullptr};
  const void* p4[] = {gated ? nullptr : gate, decay, h0, seq_offsets};
  return all_aligned(pe, big_elem(d.dtype)) && all_aligned(p4, 4) ? SSMVJP_OK : SSMVJP_EINVAL;
}

// finite_check of a call's token tensors (`rows`) beside `outs`: with packed sequences only the tokens that one owns
template <size_t K, size_t R>
ssmvjp_status finite_check_tokens(const ssmvjp_linear_scan_desc& d, const int32_t* seq_offsets, void* workspace,
                                  size_t plan_bytes, const OutSpan (&outs)[K], const OutSpan (&rows)[R], hipStream_t stream) {
  return finite_check(workspace, plan_bytes, outs, stream, [&](unsigned* flag) {
    for (const OutSpan& r : rows)
      if (d.packed) launch_nonfinite_check_rows(r.p, r.n, r.bf16, seq_offsets, d.batch, d.seqlen, true, flag, stream);
      else launch_nonfinite_check(r.p, r.n * scan_tokens(d), r.bf16, flag, stream);
  });
}

ssmvjp_status linear_step_check(const ssmvjp_linear_step_desc* d) {
  if (!d || d->batch < 0 || d->nslots < 0 || d->reserved != 0) return SSMVJP_EINVAL;
  const ssmvjp_status s = scan_form_check(d->form, d->dtype, d->c, d->dim);
  if (s != SSMVJP_OK) return s;
  if (!launches((double)d->batch * ((double)d->dim / 256 + 1), 256) || (double)d->nslots > DIM_MAX) return SSMVJP_EUNSUPPORTED;
  return SSMVJP_OK;
}

ssmvjp_status ffn_check(const ssmvjp_ffn_desc* d) {
  if (!d || d->rows < 0 || d->dim <= 0 || d->hidden <= 0 || !valid_dtype(d->dtype)) return SSMVJP_EINVAL;
  if (d->act != SSMVJP_ACT_SILU && d->act != SSMVJP_ACT_GELU) return SSMVJP_EINVAL;
  if (d->dim % 8 || d->hidden % 8 || d->dim >= (1 << 20) || d->hidden >= (1 << 20)) return SSMVJP_EUNSUPPORTED;
  const double wide = (double)(d->dim > d->hidden ? d->dim : d->hidden);
  if ((double)d->rows > DIM_MAX || !launches(((double)d->rows / 32 + 1) * (wide / 32 + 1), 256) ||
      !launches(((double)d->hidden / 128 + 1) * ((double)d->dim / 128 + 1), 512))
    return SSMVJP_EUNSUPPORTED;
  return SSMVJP_OK;
}

ssmvjp_status dropout_check(const ssmvjp_dropout_desc* d) {
  if (!d || d->n < 0 || d->reserved != 0 || !valid_dtype(d->dtype)) return SSMVJP_EINVAL;
  if (!(d->p >= 0.0 && d->p <= 1.0)) return SSMVJP_EINVAL;  // also NaN
  return d->n >= ((int64_t)1 << 60) ? SSMVJP_EUNSUPPORTED : SSMVJP_OK;
}

template <typename Desc>
ssmvjp_status query(ssmvjp_status (*check)(const Desc*), size_t (*plan)(const Desc&), const Desc* desc, size_t* bytes) {
  if (!bytes) return SSMVJP_EINVAL;
  const ssmvjp_status s = check(desc);
  if (s != SSMVJP_OK) return s;
  *bytes = with_flag(plan ? plan(*desc) : 0);
  return SSMVJP_OK;
}

}  // namespace

extern "C" {

// ------------------------------ linear_scan_fwd ------------------------------

ssmvjp_status linear_scan_fwd_workspace(const ssmvjp_linear_scan_desc* desc, size_t* bytes) {
  return query(linear_scan_check, linear_scan_fwd_workspace_bytes, desc, bytes);
}

ssmvjp_status linear_scan_fwd(const ssmvjp_linear_scan_desc* desc, const void* x, const void* gate, const void* input_gate,
                              const float* decay, const float* h0, const int32_t* seq_offsets, void* h, float* h_final,
                              float* ckpt, void* workspace, size_t workspace_bytes, void* stream) {
  ssmvjp_status s = linear_scan_check(desc);
  if (s != SSMVJP_OK) return s;
  const ssmvjp_linear_scan_desc& d = *desc;
  s = scan_inputs_check(d, x, gate, input_gate, decay, h0, seq_offsets);
  if (s != SSMVJP_OK) return s;
  if ((scan_tokens(d) > 0 && !h) || (h_final && h_final == h0)) return SSMVJP_EINVAL;
  const void* p4[] = {h_final, ckpt};
  if (!aligned(h, big_elem(d.dtype)) || !all_aligned(p4, 4)) return SSMVJP_EINVAL;
  const size_t plan = linear_scan_fwd_workspace_bytes(d);
  s = workspace_check(with_flag(plan), workspace, workspace_bytes);
  // without a sequence there may still be rows of ckpt, zeros then
  if (s != SSMVJP_OK || (d.batch == 0 && !(ckpt && linear_scan_ckpt_rows(d) > 0))) return s;
  const LinearScanPointers ptr{x, gate, input_gate, decay, h0, seq_offsets, h, h_final, ckpt, workspace};
  s = hip_status(launch_linear_scan_fwd(d, ptr, (hipStream_t)stream));
  if (s != SSMVJP_OK || !check_finite_on()) return s;
  const OutSpan outs[] = {{h_final, d.batch * d.dim, false}, {ckpt, linear_scan_ckpt_rows(d) * d.dim, false}};
  const OutSpan rows[] = {{h, d.dim, d.dtype == SSMVJP_BF16}};
  return finite_check_tokens(d, seq_offsets, workspace, plan, outs, rows, (hipStream_t)stream);
}

// ------------------------------ linear_scan_bwd ------------------------------

ssmvjp_status linear_scan_bwd_workspace(const ssmvjp_linear_scan_desc* desc, size_t* bytes) {
  return query(linear_scan_check, linear_scan_bwd_workspace_bytes, desc, bytes);
}

ssmvjp_status linear_scan_bwd(const ssmvjp_linear_scan_desc* desc, const void* x, const void* gate, const void* input_gate,
                              const float* decay, const float* h0, const float* ckpt, const void* dh,
                              const float* dh_final, const int32_t* seq_offsets, void* dx, void* dgate,
                              void* dinput_gate, float* ddecay, float* dh0, void* workspace, size_t workspace_bytes,
                              void* stream) {
  ssmvjp_status s = linear_scan_check(desc);
  if (s != SSMVJP_OK) return s;
  const ssmvjp_linear_scan_desc& d = *desc;
  s = scan_inputs_check(d, x, gate, input_gate, decay, h0, seq_offsets);
  if (s != SSMVJP_OK) return s;
  const bool gated = d.form == SSMVJP_SCAN_GATED;
  if (scan_tokens(d) > 0 && (!dh || !dx || !dgate || (gated && !dinput_gate))) return SSMVJP_EINVAL;
  if (gated ? !ddecay : (dinput_gate || ddecay)) return SSMVJP_EINVAL;
  if (dh0 && dh0 == dh_final) return SSMVJP_EINVAL;
  const void* pe[] = {dh, dx, dinput_gate, gated ? dgate : nullptr};
  const void* p4[] = {ckpt, dh_final, ddecay, dh0, gated ? nullptr : dgate};
  if (!all_aligned(pe, big_elem(d.dtype)) || !all_aligned(p4, 4)) return SSMVJP_EINVAL;
  const size_t plan = linear_scan_bwd_workspace_bytes(d);
  s = workspace_check(with_flag(plan), workspace, workspace_bytes);
  if (s != SSMVJP_OK) return s;
  const LinearScanBwdPointers ptr{x, gate, input_gate, decay, h0, ckpt, dh, dh_final, seq_offsets, dx, dgate, dinput_gate,
                                  ddecay, dh0, workspace};
  s = hip_status(launch_linear_scan_bwd(d, ptr, (hipStream_t)stream));
  if (s != SSMVJP_OK || !check_finite_on()) return s;
  const bool half = d.dtype == SSMVJP_BF16;
  const OutSpan outs[] = {{ddecay, d.dim, false}, {dh0, d.batch * d.dim, false}};
  const OutSpan rows[] = {{dx, d.dim, half}, {dgate, d.dim, gated && half}, {dinput_gate, d.dim, half}};
  return finite_check_tokens(d, seq_offsets, workspace, plan, outs, rows, (hipStream_t)stream);
}

// ------------------------------ linear_scan_step -----------------------------

ssmvjp_status linear_scan_step_workspace(const ssmvjp_linear_step_desc* desc, size_t* bytes) {
  return query<ssmvjp_linear_step_desc>(linear_step_check, nullptr, desc, bytes);
}

ssmvjp_status linear_scan_step(const ssmvjp_linear_step_desc* desc, const void* x, const void* gate,
                               const void* input_gate, const float* decay, float* state, const int32_t* slots, void* h,
                               void* workspace, size_t workspace_bytes, void* stream) {
  ssmvjp_status s = linear_step_check(desc);
  if (s != SSMVJP_OK) return s;
  const ssmvjp_linear_step_desc& d = *desc;
  const bool gated = d.form == SSMVJP_SCAN_GATED;
  if (d.batch > 0 && (!x || !gate || !h || (gated && (!input_gate || !decay)) || (d.nslots > 0 && !state))) return SSMVJP_EINVAL;
  if ((!gated && (input_gate || decay)) || (!slots && d.nslots < d.batch)) return SSMVJP_EINVAL;
  const void* pe[] = {x, input_gate, h, gated ? gate : nullptr};
  const void* p4[] = {gated ? nullptr : gate, decay, state, slots};
  if (!all_aligned(pe, big_elem(d.dtype)) || !all_aligned(p4, 4)) return SSMVJP_EINVAL;
  s = workspace_check(with_flag(0), workspace, workspace_bytes);
  if (s != SSMVJP_OK || d.batch == 0) return s;
  const LinearStepPointers ptr{x, gate, input_gate, decay, state, slots, h};
  s = hip_status(launch_linear_step(d, ptr, (hipStream_t)stream));
  if (s != SSMVJP_OK || !check_finite_on()) return s;
  const OutSpan outs[] = {{h, d.batch * d.dim, d.dtype == SSMVJP_BF16}, {slots ? nullptr : state, d.batch * d.dim, false}};
  return finite_check(workspace, 0, outs, (hipStream_t)stream, [&](unsigned* flag) {
    if (slots) launch_nonfinite_check_states(state, d.dim, slots, d.batch, d.nslots, flag, (hipStream_t)stream);
  });
}

// ------------------------------- gated_ffn -----------------------------------

ssmvjp_status gated_ffn_fwd_workspace(const ssmvjp_ffn_desc* desc, size_t* bytes) {
  return query(ffn_check, ffn_fwd_workspace_bytes, desc, bytes);
}

ssmvjp_status gated_ffn_fwd(const ssmvjp_ffn_desc* desc, const void* x, const void* w_gate, const void* w_up, void* h,
                            void* gate, void* up, void* workspace, size_t workspace_bytes, void* stream) {
  ssmvjp_status s = ffn_check(desc);
  if (s != SSMVJP_OK) return s;
  const ssmvjp_ffn_desc& d = *desc;
  if (d.rows > 0 && (!x || !w_gate || !w_up || !h)) return SSMVJP_EINVAL;
  if ((gate != nullptr) != (up != nullptr)) return SSMVJP_EINVAL;
  const void* p16[] = {x, w_gate, w_up, h, gate, up};
  if (!all_aligned(p16, 16)) return SSMVJP_EINVAL;
  const size_t plan = ffn_fwd_workspace_bytes(d);
  s = workspace_check(with_flag(plan), workspace, workspace_bytes);
  if (s != SSMVJP_OK || d.rows == 0) return s;
  const FfnFwdPointers ptr{x, w_gate, w_up, h, gate, up, workspace};
  s = hip_status(launch_ffn_fwd(d, ptr, (hipStream_t)stream));
  if (s != SSMVJP_OK || !check_finite_on()) return s;
  const int64_t n = d.rows * d.hidden;
  const bool half = d.dtype == SSMVJP_BF16;
  const OutSpan outs[] = {{h, n, half}, {gate, n, half}, {up, n, half}};
  return finite_check(workspace, plan, outs, (hipStream_t)stream);
}

ssmvjp_status gated_ffn_bwd_workspace(const ssmvjp_ffn_desc* desc, size_t* bytes) {
  return query(ffn_check, ffn_bwd_workspace_bytes, desc, bytes);
}

ssmvjp_status gated_ffn_bwd(const ssmvjp_ffn_desc* desc, const void* dh, const void* x, const void* w_gate,
                            const void* w_up, const void* gate, const void* up, void* dx, void* dw_gate, void* dw_up,
                            void* workspace, size_t workspace_bytes, void* stream) {
  ssmvjp_status s = ffn_check(desc);
  if (s != SSMVJP_OK) return s;
  const ssmvjp_ffn_desc& d = *desc;
  if (d.rows > 0 && (!dh || !x || !w_gate || !w_up)) return SSMVJP_EINVAL;
  if ((gate != nullptr) != (up != nullptr)) return SSMVJP_EINVAL;
  const void* p16[] = {dh, x, w_gate, w_up, gate, up, dx, dw_gate, dw_up};
  if (!all_aligned(p16, 16)) return SSMVJP_EINVAL;
  const size_t plan = ffn_bwd_workspace_bytes(d);
  s = workspace_check(with_flag(plan), workspace, workspace_bytes);
  if (s != SSMVJP_OK) return s;
  const FfnBwdPointers ptr{dh, x, w_gate, w_up, gate, up, dx, dw_gate, dw_up, workspace};
  s = hip_status(launch_ffn_bwd(d, ptr, (hipStream_t)stream));
  if (s != SSMVJP_OK || !check_finite_on()) return s;
  const bool half = d.dtype == SSMVJP_BF16;
  const OutSpan outs[] = {{dx, d.rows * d.dim, half}, {dw_gate, d.hidden * d.dim, half}, {dw_up, d.hidden * d.dim, half}};
  return finite_check(workspace, plan, outs, (hipStream_t)stream);
}

// -------------------------------- dropout ------------------------------------

ssmvjp_status dropout_fwd_workspace(const ssmvjp_dropout_desc* desc, size_t* bytes) {
  return query<ssmvjp_dropout_desc>(dropout_check, nullptr, desc, bytes);
}

ssmvjp_status dropout_fwd(const ssmvjp_dropout_desc* desc, const void* x, const void* residual, const int64_t* rng, void* y,
                          void* workspace, size_t workspace_bytes, void* stream) {
  ssmvjp_status s = dropout_check(desc);
  if (s != SSMVJP_OK) return s;
  const ssmvjp_dropout_desc& d = *desc;
  if (d.n > 0 && (!x || !rng || !y)) return SSMVJP_EINVAL;
  const void* pe[] = {x, residual, y};
  if (!all_aligned(pe, big_elem(d.dtype)) || !aligned(rng, 8)) return SSMVJP_EINVAL;
  s = workspace_check(with_flag(0), workspace, workspace_bytes);
  if (s != SSMVJP_OK || d.n == 0) return s;
  s = hip_status(launch_dropout(d.n, d.p, d.dtype, x, residual, rng, y, (hipStream_t)stream));
  if (s != SSMVJP_OK || !check_finite_on()) return s;
  const OutSpan outs[] = {{y, d.n, d.dtype == SSMVJP_BF16}};
  return finite_check(workspace, 0, outs, (hipStream_t)stream);
}

ssmvjp_status dropout_bwd_workspace(const ssmvjp_dropout_desc* desc, size_t* bytes) {
  return query<ssmvjp_dropout_desc>(dropout_check, nullptr, desc, bytes);
}

ssmvjp_status dropout_bwd(const ssmvjp_dropout_desc* desc, const void* dy, const int64_t* rng, void* dx, void* workspace,
                          size_t workspace_bytes, void* stream) {
  return dropout_fwd(desc, dy, nullptr, rng, dx, workspace, workspace_bytes, stream);
}

}  // extern "C"
