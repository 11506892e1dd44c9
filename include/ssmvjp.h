/*
 * ssmvjp.h -- C ABI of libssmvjp: the backward pass (VJP) of the selective
 * state-space scan on AMD Instinct MI355X (gfx950).
 *
 * The operation.  The forward scan keeps a state s_t[h,p,n] per (batch, head):
 *     delta_t,h = softplus(dt_t,h)                  (dt is the raw, pre-softplus value)
 *     a_t       = exp(delta_t,h * A)                (A = A_h: Mamba-2, one decay per head;
 *                                                    A = A_h,n: Mamba-1, one decay per state)
 *     s_t       = a_t * s_{t-1} + delta_t,h * x_t[h,p] * B_t[g,n]
 *     y_t[h,p]  = sum_n C_t[g,n] * s_t[h,p,n]       (reads the state after the update)
 * with s_{-1} = s0 and head h reading group g = h / (H/G).  Given the upstream
 * gradients dy (of y) and ds_final (of the final state s_{T-1}), the library
 * returns the five gradients dx, d_dt, dB, dC, d_s0 of
 *     J = <dy, y> + <ds_final, s_{T-1}>.
 * This is the reverse-time recurrence of llama.cpp PR "S1-31: SSM_SCAN_BACK --
 * Mamba has a backward" (the op paragraph: five gradients from one op, both the
 * per-head and the per-state decay branch), seeded at t = T with the non-zero
 * final-state gradient (its point 1) and needing s_{t-1} for the decay path of
 * d_dt (its point 2).
 *
 * The chunked entry point computes the same gradients with the chunked SSD
 * algorithm of burn-mamba "combined_backward.rs" (combined_backward: K1..K4
 * recompute, reverse chunk loop over the BLUE / ORANGE / K4 backwards, batched
 * K3 / K2 / K1 backwards), including the fused L*M length of the MIMO form.
 * The delta-rule entry point is the KDA backward of the K3 notes section
 * "反向传播推导" (forward F1..F6, BPTT steps 1..6, GVA view+sum).
 *
 * Conventions shared by every entry point
 *  - All tensors are dense, row-major, innermost axis last, and live in device
 *    memory of the current HIP device.  The caller allocates every input,
 *    output and workspace buffer; the library allocates nothing and keeps no
 *    state between calls, so concurrent calls on different streams are safe.
 *  - `stream` is a hipStream_t (NULL = the null stream).  Work is enqueued
 *    asynchronously; the caller synchronises.
 *  - Outputs are overwritten, never accumulated into.  Inputs, outputs and the
 *    workspace must not overlap, unless the entry point says that they may.
 *  - Validation errors (SSMVJP_EINVAL, SSMVJP_EUNSUPPORTED, SSMVJP_EWORKSPACE)
 *    are returned before anything is enqueued.  SSMVJP_EHIP means a launch
 *    failed; outputs are then undefined.
 *  - Results are deterministic: the same inputs give bitwise-identical outputs
 *    on every call (all reductions run in a fixed order, no float atomics).
 *  - "big" tensors (x or v, B, C, dy and their gradients) are float32 or
 *    bfloat16 as selected by `dtype`; everything else is float32.
 *  - Debug finiteness mode: with the environment variable SSMVJP_CHECK_FINITE
 *    set (to anything but "0") when a call is made, every entry point scans
 *    the outputs it wrote for NaN and infinite values after its launches,
 *    synchronises the stream and returns SSMVJP_ENONFINITE if it found one
 *    (the outputs are still written).  While the mode is on, the *_workspace
 *    queries report 256 more bytes, which hold the scan's flag (burn-mamba's
 *    combined_backward checks its intermediates for NaNs in the same spirit;
 *    here the intermediates stay inside the kernels, so the outputs are
 *    checked).  Off by default: the normal calls neither scan nor synchronise.
 */
#ifndef SSMVJP_H
#define SSMVJP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SSMVJP_OK = 0,
  SSMVJP_EINVAL = 1,        /* bad descriptor, NULL required pointer, misaligned pointer */
  SSMVJP_EUNSUPPORTED = 2,  /* valid arguments outside what the kernels implement */
  SSMVJP_EWORKSPACE = 3,    /* workspace NULL or smaller than the *_workspace query */
  SSMVJP_EHIP = 4,          /* a HIP launch or runtime call failed */
  SSMVJP_ENONFINITE = 5     /* debug mode only: an output holds a NaN or an infinity */
} ssmvjp_status;

enum { SSMVJP_F32 = 0, SSMVJP_BF16 = 1 };                         /* dtype of the big tensors */
enum { SSMVJP_DECAY_PER_HEAD = 0, SSMVJP_DECAY_PER_STATE = 1 };   /* Mamba-2 / Mamba-1 */
enum { SSMVJP_FORM_MAMBA2 = 0, SSMVJP_FORM_RAW = 1 };             /* (x, dt, A) or (v, da) */

/* ------------------------------------------------------------------------ */
/* ssm_scan_bwd: sequential reverse recurrence                               */
/* ------------------------------------------------------------------------ */

typedef struct {
  int64_t batch, seqlen, nheads, headdim, dstate, ngroups; /* b, T, H, P, N, G */
  int32_t decay;      /* SSMVJP_DECAY_PER_HEAD (A is [H]) or SSMVJP_DECAY_PER_STATE (A is [H,N]) */
  int32_t dtype;      /* SSMVJP_F32 or SSMVJP_BF16 for x, B, C, dy, dx, dB, dC */
  int32_t ckpt_every; /* K: states are checkpointed every K steps and recomputed per
                         segment (llama.cpp PR, point 2: checkpoint-every-K against
                         store-all).  0 = library default.  Outputs are bitwise
                         identical for every K. */
  int32_t reserved;   /* must be 0 */
} ssmvjp_scan_desc;

/* Bytes of device workspace ssm_scan_bwd needs for `desc` (0 is valid). */
ssmvjp_status ssm_scan_bwd_workspace(const ssmvjp_scan_desc* desc, size_t* bytes);

/* Backward of the sequential selective scan.
 *   x [b,T,H,P] (dtype)   dt [b,T,H] f32 (raw)   A [H] or [H,N] f32
 *   B, C [b,T,G,N] (dtype)   s0 [b,H,P,N] f32 (NULL = zeros)
 *   dy [b,T,H,P] (dtype)   ds_final [b,H,P,N] f32 (NULL = zeros)
 * Outputs:
 *   dx [b,T,H,P] (dtype)   d_dt [b,T,H] f32   dB, dC [b,T,G,N] (dtype)
 *   d_s0 [b,H,P,N] f32
 * Constraints: b, T >= 0 (an empty batch or sequence enqueues nothing except
 * d_s0 = ds_final for T = 0); H % G == 0 (SSMVJP_EINVAL otherwise).  One
 * workgroup per (batch, head) holds the head's state in LDS, so with
 * Q = ceil(P / min(P, 16)) groups of p values
 *     N <= 1024,  P*N <= 32768,  Q*N <= 1024  and
 *     4 * (P*(N+1) + 2*Q*N + ceil(Q*N / 64)) <= 65536 bytes of LDS
 * (SSMVJP_EUNSUPPORTED otherwise; e.g. P = N = 128 needs 74,304 bytes and is
 * refused, P = 64, N = 128 fits).
 * Pointers must be 4-byte aligned (f32) or 2-byte aligned (bf16). */
ssmvjp_status ssm_scan_bwd(const ssmvjp_scan_desc* desc,
                           const void* x, const float* dt, const float* A,
                           const void* B, const void* C, const float* s0,
                           const void* dy, const float* ds_final,
                           void* dx, float* d_dt, void* dB, void* dC, float* d_s0,
                           void* workspace, size_t workspace_bytes, void* stream);

/* ssm_scan_bwd plus dA, the gradient of the decay coefficients A: dA [H]
 * (per-head decay) or [H,N] (per-state decay), float32, written (not
 * accumulated).  With a_t = exp(delta_t A) the state update gives
 * d s_t / d A = delta_t a_t s_{t-1}, so dA = sum over the batch and time of
 * delta_t a_t <dS_t, s_{t-1}> (per state: per column n).  burn-mamba's
 * combined_backward returns the decay gradient d_da; dA is its sum
 * sum_{b,t} d_da * delta, the gradient training needs for A.  The other
 * arguments and outputs are exactly those of ssm_scan_bwd; dA must not be NULL
 * when batch > 0.  The sums over the batch run in a fixed order (deterministic). */
ssmvjp_status ssm_scan_bwd_dA(const ssmvjp_scan_desc* desc,
                              const void* x, const float* dt, const float* A,
                              const void* B, const void* C, const float* s0,
                              const void* dy, const float* ds_final,
                              void* dx, float* d_dt, void* dB, void* dC, float* d_s0, float* dA,
                              void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* ssd_chunk_bwd: chunked SSD backward (Mamba-2 and Mamba-3 MIMO)            */
/* ------------------------------------------------------------------------ */

typedef struct {
  int64_t batch, seqlen, nheads, headdim, dstate, ngroups; /* b, T, H, P, N, G */
  int64_t mimo_rank;  /* M: rank of the per-step input (1 for Mamba-2) */
  int64_t chunk_len;  /* L: steps per chunk; the fused chunk length is L*M */
  int32_t form;       /* SSMVJP_FORM_MAMBA2: inputs x, dt, A (requires M == 1);
                         SSMVJP_FORM_RAW: pre-scaled inputs v, da (burn-mamba's
                         combined_backward arguments) */
  int32_t dtype;      /* SSMVJP_F32 or SSMVJP_BF16 for x/v, B, C, dy and their gradients */
} ssmvjp_ssd_desc;

ssmvjp_status ssd_chunk_bwd_workspace(const ssmvjp_ssd_desc* desc, size_t* bytes);

/* Chunked backward.  Layouts (all row-major):
 *   FORM_MAMBA2: x_or_v = x [b,T,H,P], dt_or_da = dt [b,T,H] (raw), A [H]
 *   FORM_RAW:    x_or_v = v [b,T,M,H,P], dt_or_da = da [b,T,H] (= delta*A), A = NULL
 *   B, C [b,T,M,G,N]   s0, ds_final, d_s0 [b,H,P,N] f32 (s0/ds_final NULL = zeros)
 *   dy, dx_or_dv like x_or_v;  d_dt_or_dda like dt_or_da;  dB, dC like B.
 * A last chunk shorter than L (T % L != 0) is handled as a shorter chunk.
 * Constraints (SSMVJP_EUNSUPPORTED otherwise): H % G == 0; P % 16 == 0,
 * N % 16 == 0, P <= 128, N <= 128; (P/16) * (N/16) <= 32 unless N is a
 * multiple of 32; and the fused chunk length L*M is either
 *   - a multiple of 16 up to 64 (one kernel holds the whole chunk): its
 *     working set must fit 160 KiB of LDS (P*N <= 8192 with bf16 at
 *     L*M = 64; P*N <= 4096 more or less with float32), or
 *   - a multiple of 64 above 64 with L <= 64 and M dividing 64 (row-blocked
 *     kernels, e.g. the rank-4 MIMO form with L = 64): 64 rows of B, C, x and
 *     dy plus one state must fit 160 KiB of LDS (any P, N <= 128 with bf16;
 *     P*N <= 8192 more or less with float32).
 * Alignment (SSMVJP_EINVAL otherwise): x_or_v, B, C, dy, dx_or_dv, dB and dC
 * 16-byte aligned (the kernels move them in 16-byte vectors); the float32
 * tensors 4-byte aligned; the workspace 256-byte aligned. */
ssmvjp_status ssd_chunk_bwd(const ssmvjp_ssd_desc* desc,
                            const void* x_or_v, const float* dt_or_da, const float* A,
                            const void* B, const void* C, const float* s0,
                            const void* dy, const float* ds_final,
                            void* dx_or_dv, float* d_dt_or_dda, void* dB, void* dC, float* d_s0,
                            void* workspace, size_t workspace_bytes, void* stream);

/* ssd_chunk_bwd plus dA [H] (FORM_MAMBA2 only, SSMVJP_EINVAL otherwise):
 * dA_h = sum over the batch and time of d_da * delta for head h, with d_da the
 * decay gradient the chunked backward forms on the way to d_dt (burn-mamba
 * combined_backward's d_da).  Each chunk's per-head sum is formed in the
 * chunk kernel, and the sums over (batch, chunk) run in a fixed order.  The
 * other arguments and outputs are exactly those of ssd_chunk_bwd (same
 * workspace size, same shape limits and 16-byte alignment of the big
 * tensors); dA must not be NULL when batch > 0. */
ssmvjp_status ssd_chunk_bwd_dA(const ssmvjp_ssd_desc* desc,
                               const void* x, const float* dt, const float* A,
                               const void* B, const void* C, const float* s0,
                               const void* dy, const float* ds_final,
                               void* dx, float* d_dt, void* dB, void* dC, float* d_s0, float* dA,
                               void* workspace, size_t workspace_bytes, void* stream);

/* The two stages of ssd_chunk_bwd as separate calls, for callers that want to
 * schedule or time them apart.  ssd_chunk_bwd_states followed by
 * ssd_chunk_bwd_grads on the same stream, with the same descriptor, inputs and
 * workspace, is exactly ssd_chunk_bwd.
 *  - ssd_chunk_bwd_states: the forward and reverse state passing over chunks
 *    (burn-mamba combined_backward's K1..K4 recompute and the K4 backward with
 *    the BLUE state gradient).  Writes d_s0 and leaves the chunk-input states
 *    and the chunk-output state gradients in the workspace.
 *  - ssd_chunk_bwd_grads: the per-chunk BLUE / ORANGE / K3 / K2 / K1 backwards
 *    and the Mamba-2 chain, reading the states the previous call left in the
 *    workspace.  The workspace must not be modified in between.
 * Arguments mean what they mean for ssd_chunk_bwd, with the same shape limits
 * and the same alignment (the big tensors 16-byte aligned, the workspace 256). */
ssmvjp_status ssd_chunk_bwd_states(const ssmvjp_ssd_desc* desc,
                                   const void* x_or_v, const float* dt_or_da, const float* A,
                                   const void* B, const void* C, const float* s0,
                                   const void* dy, const float* ds_final, float* d_s0,
                                   void* workspace, size_t workspace_bytes, void* stream);
ssmvjp_status ssd_chunk_bwd_grads(const ssmvjp_ssd_desc* desc,
                                  const void* x_or_v, const float* dt_or_da, const float* A,
                                  const void* B, const void* C, const void* dy,
                                  void* dx_or_dv, float* d_dt_or_dda, void* dB, void* dC,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* ssd_chunk_bwd without a workspace argument, for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc.  The workspace is a device array of
 * SSMVJP_NOALLOC_SCRATCH_BYTES (96 MiB) that the library owns: each device
 * holds its own copy from the first call on that device until the process
 * ends.  The call allocates nothing (no hipMalloc, no hipFree); the caller
 * still passes every input and output.  Arguments, layouts, limits, alignment
 * and results are exactly those of ssd_chunk_bwd; a shape whose
 * ssd_chunk_bwd_workspace size exceeds SSMVJP_NOALLOC_SCRATCH_BYTES returns
 * SSMVJP_EWORKSPACE before anything is enqueued (the Mamba-2 head shape
 * H = 32, P = 64, N = 128 in bf16 fits up to b*T = 4096 tokens, e.g. one
 * sequence of 4096).  Every call on one device shares that device's array:
 * calls whose work overlaps on one device (other streams, other host threads)
 * race and must be serialised by the caller. */
#define SSMVJP_NOALLOC_SCRATCH_BYTES (96u << 20)
ssmvjp_status ssd_chunk_bwd_noalloc(const ssmvjp_ssd_desc* desc,
                                    const void* x_or_v, const float* dt_or_da, const float* A,
                                    const void* B, const void* C, const float* s0,
                                    const void* dy, const float* ds_final,
                                    void* dx_or_dv, float* d_dt_or_dda, void* dB, void* dC, float* d_s0,
                                    void* stream);

/* ------------------------------------------------------------------------ */
/* ssd_chunk_fwd: chunked SSD forward (the step before the backward)         */
/* ------------------------------------------------------------------------ */

/* The forward scan in the chunked SSD form of burn-mamba's chunked forward
 * (K1 chunk cumsum, K2 C.B^T, K3 intra-chunk state, K4 state passing, K5
 * output = BLUE inter-chunk term + ORANGE causal intra-chunk term): returns
 * y and the final state s_{T-1} (s0 when T = 0).
 *   Inputs as for ssd_chunk_bwd (FORM_MAMBA2: x, dt, A; FORM_RAW: v, da).
 *   y like x_or_v ([b,T,H,P] or [b,T,M,H,P], dtype); s_final [b,H,P,N] f32
 *   (NULL: not written); s0 NULL = zeros.
 * The running state of each (batch, head) stays on chip; with bf16 the
 * workspace holds the scores C.B^T of every chunk (from ssd_chunk_fwd_workspace;
 * none with float32).  The kernel walks chunks of chunk_len steps when
 * chunk_len * M <= 64, else of 64 / M steps; the results do not depend on the
 * chunk length apart from rounding.
 * Constraints (SSMVJP_EUNSUPPORTED otherwise): P % 16 == 0, N % 16 == 0,
 * N <= 128, M <= 64.  x_or_v, B, C and y 16-byte aligned. */
ssmvjp_status ssd_chunk_fwd_workspace(const ssmvjp_ssd_desc* desc, size_t* bytes);
ssmvjp_status ssd_chunk_fwd(const ssmvjp_ssd_desc* desc,
                            const void* x_or_v, const float* dt_or_da, const float* A,
                            const void* B, const void* C, const float* s0,
                            void* y, float* s_final,
                            void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* delta_rule_bwd: KDA gated delta rule backward                             */
/* ------------------------------------------------------------------------ */

typedef struct {
  int64_t batch, seqlen, nqk_heads, nv_heads, dk, dv; /* b, T, H, HV, K, V */
  float scale;        /* q enters the output as scale * q */
  int32_t reserved;   /* must be 0 */
} ssmvjp_delta_desc;

ssmvjp_status delta_rule_bwd_workspace(const ssmvjp_delta_desc* desc, size_t* bytes);

/* KDA backward (all float32), K3 notes section "反向传播推导": the forward
 *   S_dec = exp(g_t) (.) S_{t-1};  r = v_t - k_t^T S_dec;  S_t = S_dec + (beta_t k_t) (x) r;
 *   o_t = (scale q_t)^T S_t
 * (F1..F6) with S_{-1} = S0, and its reverse-time backward (BPTT steps 1..5)
 * seeded with dS_final, followed by the GVA sum of dq and dk over the value
 * heads of each qk head (step 6).  The gradients are those of
 *     J = <d_o, o> + <dS_final, S_{T-1}>.
 *   q, k [b,T,H,K]   v [b,T,HV,V]   beta [b,T,HV]   g [b,T,HV,K] (log gate)
 *   S0 [b,HV,K,V] (NULL = zeros)   d_o [b,T,HV,V]   dS_final [b,HV,K,V] (NULL = zeros)
 * Outputs: dq, dk [b,T,H,K]   dv [b,T,HV,V]   dg [b,T,HV,K]   dbeta [b,T,HV]
 *   dS0 [b,HV,K,V] (NULL = not written).
 * Value head hv reads qk head hv / (HV/H).
 * Constraints: HV % H == 0 (SSMVJP_EINVAL otherwise); K == 128 and V a
 * multiple of 32 (SSMVJP_EUNSUPPORTED otherwise).  Every pointer must be
 * 16-byte aligned.  T = 0 writes dS0 = dS_final only. */
ssmvjp_status delta_rule_bwd(const ssmvjp_delta_desc* desc,
                             const float* q, const float* k, const float* v, const float* beta,
                             const float* g, const float* S0, const float* d_o, const float* dS_final,
                             float* dq, float* dk, float* dv, float* dg, float* dbeta, float* dS0,
                             void* workspace, size_t workspace_bytes, void* stream);

/* The three stages of delta_rule_bwd as separate calls, for callers that
 * schedule or time them apart.  `stages` is a non-empty bit mask of
 *  - SSMVJP_DELTA_CKPT:   forward walk that leaves the state at the start of
 *                         every checkpoint segment in the workspace;
 *  - SSMVJP_DELTA_BWD:    reverse walk (recompute from the checkpoints, BPTT
 *                         steps 1..5): writes dv and dS0 and leaves per-slice
 *                         partial sums of the per-key outputs in the workspace;
 *  - SSMVJP_DELTA_REDUCE: slice sums and the GVA sum: writes dq, dk, dg, dbeta.
 * The stages run in that order; calls for the three stages in order on one
 * stream, with the same descriptor, arguments and workspace, are exactly
 * delta_rule_bwd (the workspace must not be modified in between).  Arguments
 * mean what they mean for delta_rule_bwd and are validated the same way. */
enum { SSMVJP_DELTA_CKPT = 1, SSMVJP_DELTA_BWD = 2, SSMVJP_DELTA_REDUCE = 4, SSMVJP_DELTA_ALL = 7 };
ssmvjp_status delta_rule_bwd_stages(const ssmvjp_delta_desc* desc, int32_t stages,
                                    const float* q, const float* k, const float* v, const float* beta,
                                    const float* g, const float* S0, const float* d_o, const float* dS_final,
                                    float* dq, float* dk, float* dv, float* dg, float* dbeta, float* dS0,
                                    void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* delta_chunk_fwd: gated delta rule, one log gate per value head             */
/* ------------------------------------------------------------------------ */

/* The delta rule above with one gate per value head instead of one per key
 * channel, over whole sequences:
 *   S_dec = exp(g_t) S_{t-1};  r = v_t - k_t^T S_dec;  S_t = S_dec + (beta_t k_t) (x) r;
 *   o_t = (scale q_t)^T S_t.
 * Sequences: with packed = 0, `batch` sequences of `seqlen` tokens (token
 * tensors [batch, seqlen, ...]).  With packed = 1, `batch` sequences behind one
 * another in `seqlen` tokens (token tensors [seqlen, ...]): sequence i owns the
 * tokens seq_offsets[i] .. seq_offsets[i+1] - 1, seq_offsets in device memory,
 * ascending.  Borders outside [0, seqlen] are clamped, so that no value there
 * can lead outside the tensors; an empty sequence's final state is its initial
 * state; tokens that no sequence owns are neither read nor written. */
typedef struct {
  int64_t batch, seqlen, nqk_heads, nv_heads, dk, dv; /* sequences, T, H, HV, K, V */
  float scale;
  int32_t dtype;    /* SSMVJP_F32 or SSMVJP_BF16 for q, k, v, o (and their gradients) */
  int32_t packed;   /* 0 or 1, see above */
  int32_t reserved; /* must be 0 */
} ssmvjp_delta_chunk_desc;

/* Forward.
 *   q, k [.., H, K]   v [.., HV, V] (dtype)   beta, g [.., HV] f32 (g the log gate)
 *   S0 [batch, HV, K, V] f32 (NULL = zeros)   seq_offsets [batch + 1] int32 (packed; else NULL)
 * Outputs: o like v;  S_final [batch, HV, K, V] f32 (NULL = not written).
 * Value head hv reads qk head hv / (HV/H).  bf16 runs the chunked form on the
 * matrix cores (states to about 1e-5 of their norm), float32 and calls of up to
 * 16 tokens (seqlen: of all sequences of a packed call together) run token by
 * token in float32 throughout.  bf16 values given as float32 therefore leave the
 * states at float32's accuracy, at 0.7 us a token of the longest sequence.
 * g may be -infinity (a reset); the chunked form takes every g below -88 as -88.
 * There the decay between two tokens is the exponential of a difference of sums
 * of g over their chunk of 64 tokens, relatively off by up to 2^-24 of the larger
 * sum's size (1e-5 after two resets, 6e-5 after twelve in one chunk).
 * A NaN or an infinity in a token of one value head reaches that token and those
 * behind it in that head, as in the definition: garbage in the padding behind the
 * end of a sequence leaves the tokens before it alone (its final state not).  In
 * the backward it reaches the head's whole sequence, and dq and dk of its qk head;
 * in both, nothing else.
 * S_final may be S0.
 * Constraints: HV % H == 0 (SSMVJP_EINVAL otherwise); K % 16 == 0, K <= 128,
 * V % 16 == 0, V <= 65536, H*K and HV*V below 2^24, and launches of fewer than
 * 2^32 threads: chunks * H below 2^23 with seqlen/64 + 1 chunks a sequence (packed:
 * seqlen/64 + batch of all) and (batch*HV + 8) * (V/32 + 1) at most 6,710,886
 * (SSMVJP_EUNSUPPORTED otherwise).  q, k, v, o, S0, S_final 16-byte aligned. */
ssmvjp_status delta_chunk_fwd_workspace(const ssmvjp_delta_chunk_desc* desc, size_t* bytes);
ssmvjp_status delta_chunk_fwd(const ssmvjp_delta_chunk_desc* desc,
                              const void* q, const void* k, const void* v, const float* beta, const float* g,
                              const float* S0, const int32_t* seq_offsets, void* o, float* S_final,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Backward: the gradients of J = <d_o, o> + <dS_final, S_final>.
 *   q, k, v, beta, g, S0, seq_offsets as for delta_chunk_fwd;  d_o like o;
 *   dS_final [batch, HV, K, V] f32 (NULL = zeros)
 * Outputs: dq, dk like q (summed over the value heads of each qk head), dv like v,
 *   dbeta, dg [.., HV] f32, dS0 [batch, HV, K, V] f32 (NULL = not written).
 * dq, dk and dv are rounded to bf16, dbeta, dg and dS0 come out to about 1e-5
 * of their norm.  The gradient of a g below -88 is that at -88.
 * dS0 may be dS_final or S0 (over S0 the two state walks run one behind the
 * other where they would share a launch).
 * Constraints as for delta_chunk_fwd, and dtype SSMVJP_BF16 (SSMVJP_EUNSUPPORTED
 * otherwise).  d_o, dq, dk, dv, dS_final and dS0 are 16-byte aligned too.
 * There is no float32 form.  delta_rule_bwd computes the same gradients in
 * float32, with g repeated over the key channels and dg summed over them, but
 * takes only K = 128, V a multiple of 32 and equal sequences: narrower heads have
 * to be padded with zeros (q, k, S0 and dS_final to 128 keys; v, d_o, S0 and
 * dS_final to a multiple of 32 columns), packed sequences called one by one. */
ssmvjp_status delta_chunk_bwd_workspace(const ssmvjp_delta_chunk_desc* desc, size_t* bytes);
ssmvjp_status delta_chunk_bwd(const ssmvjp_delta_chunk_desc* desc,
                              const void* q, const void* k, const void* v, const float* beta, const float* g,
                              const float* S0, const void* d_o, const float* dS_final, const int32_t* seq_offsets,
                              void* dq, void* dk, void* dv, float* dbeta, float* dg, float* dS0,
                              void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* delta_step: one token per request on a pool of states                      */
/* ------------------------------------------------------------------------ */

enum { SSMVJP_GATE_PER_HEAD = 0, SSMVJP_GATE_PER_KEY = 1 }; /* g [batch, HV] or [batch, HV, K] */

typedef struct {
  int64_t batch, nslots, nqk_heads, nv_heads, dk, dv; /* requests, states in the pool, H, HV, K, V */
  float scale;
  int32_t dtype;    /* SSMVJP_F32 or SSMVJP_BF16 for q, k, v, o */
  int32_t gate;     /* SSMVJP_GATE_PER_HEAD (as delta_chunk_fwd) or SSMVJP_GATE_PER_KEY (as delta_rule_bwd) */
  int32_t reserved; /* must be 0 */
} ssmvjp_delta_step_desc;

/* One token of the delta rule for every request, the states updated in place.
 *   q, k [batch, H, K]   v [batch, HV, V] (dtype)   beta [batch, HV] f32   g f32 (see gate)
 *   state [nslots, HV, K, V] f32, read and written   slots [batch] int32 in device memory
 *   (NULL: request i uses state i)
 * Output: o [batch, HV, V].
 * A request whose slot is outside [0, nslots) (padding of a captured batch) or
 * was named by an earlier request of the call gets zeros in o and touches no
 * state.  Constraints on the heads and alignment as for delta_chunk_fwd (state
 * 16-byte aligned; g too with per-key gates); batch * HV * (V/64 + 1) below 2^24
 * (SSMVJP_EUNSUPPORTED otherwise). */
ssmvjp_status delta_step_workspace(const ssmvjp_delta_step_desc* desc, size_t* bytes);
ssmvjp_status delta_step(const ssmvjp_delta_step_desc* desc,
                         const void* q, const void* k, const void* v, const float* beta, const float* g,
                         float* state, const int32_t* slots, void* o,
                         void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* layer_norm_fwd, layer_norm_bwd                                             */
/* ------------------------------------------------------------------------ */

/* Layer norm of the last axis of x [rows, groups, dim]; the row (t, j) uses
 * weight[j] and bias[j] (groups = 1: one weight vector; groups = heads: the
 * norm of every head of a scan's readout, each head with its own):
 *   mean = sum x / dim;  rstd = 1 / sqrt(sum (x - mean)^2 / dim + eps)
 *   h = (x - mean) rstd;  y = h weight + bias. */
typedef struct {
  int64_t rows, groups, dim;
  float eps;
  int32_t dtype; /* SSMVJP_F32 or SSMVJP_BF16 for x, y, dy, dx */
} ssmvjp_norm_desc;

/* Forward: y like x; mean, rstd [rows, groups] f32 (NULL = not written);
 * weight, bias [groups, dim] f32 (NULL = ones, zeros).
 * x8 [rows, groups, dim] int8 and x8_scale [rows, groups, ceil(dim / 64)] f32
 * (both or neither): the 8-bit form of x that layer_norm_bwd can read in its
 * place.  For every block of 64 values of a row (the last may be shorter)
 *   x8_scale = max|x| * (1/127),  x8 = rint(x * (127 * (1/max|x|)))
 * (each operation rounded to float32, ties to even),
 * zeros where max|x| < 1e-36: the value kept is off by max|x| / 254, half a code, and
 * the float32 roundings at most.
 * Any dim and any element alignment (groups * dim below 2^26 - 16, groups below
 * 2^24 - 2048, rows * groups below 2^31: SSMVJP_EUNSUPPORTED otherwise); 16-byte
 * aligned tensors and a dim that is a multiple of 8 (bf16) or 4 (f32) are the
 * fast ones. */
ssmvjp_status layer_norm_fwd_workspace(const ssmvjp_norm_desc* desc, size_t* bytes);
ssmvjp_status layer_norm_fwd(const ssmvjp_norm_desc* desc,
                             const void* x, const float* weight, const float* bias, void* y, float* mean, float* rstd,
                             int8_t* x8, float* x8_scale, void* workspace, size_t workspace_bytes, void* stream);

/* Backward from the upstream gradient dy, the forward's mean and rstd and
 * either x or (x NULL) x8 and x8_scale, whose values x8 * x8_scale then stand
 * for x:
 *   t = dy weight;  dx = rstd (t - sum(t)/dim - h sum(t h)/dim)
 *   dweight = sum over rows of dy h,  dbias = sum over rows of dy  ([groups, dim] f32,
 *   each NULL = not computed; zeros when rows = 0).  eps is not used. */
ssmvjp_status layer_norm_bwd_workspace(const ssmvjp_norm_desc* desc, size_t* bytes);
ssmvjp_status layer_norm_bwd(const ssmvjp_norm_desc* desc,
                             const void* dy, const void* x, const int8_t* x8, const float* x8_scale,
                             const float* mean, const float* rstd, const float* weight,
                             void* dx, float* dweight, float* dbias,
                             void* workspace, size_t workspace_bytes, void* stream);

/* Human-readable name of a status code (static storage). */
const char* ssmvjp_status_str(ssmvjp_status status);

/* Library version, e.g. "0.1.0" (static storage). */
const char* ssmvjp_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SSMVJP_H */
