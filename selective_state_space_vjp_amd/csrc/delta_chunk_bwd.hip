// delta_chunk_bwd.hip -- gradients of the chunked gated delta rule on MFMA.
//
// With lambda_i the adjoint of u_i and mu = beta lambda (delta_chunk.cuh has
// the forward's algebra; dS the gradient of the state behind the chunk, N_ij =
// mu_i . r_j, M the pair terms):
//     dU = scale P^T dO + e^{G_63 - G} (K dS)
//     mu = T^T (beta dU)  = dv
//     dS0 = e^{G_63} dS + Q^T (scale e^G dO) - K^T (e^G mu)
//     dD_ij = scale beta_j (dO_i . r_j) Gam_ij  (i >= j),  E_ij = -beta_j N_ij Gam_ij  (i > j)
//     dq = scale e^G dO S0^T + dD K
//     dk = -e^G mu S0^T + (e^{G_63 - G} beta r) dS^T + dD^T Q + E K + E^T K
//     dbeta_j = r_j . dU_j - sum_{i > j} a_ij N_ij
//     M_ij = dD_ij q_i . k_j + E_ij k_i . k_j
//     dG_i = q_i . (scale e^G dO S0^T)_i - k_i . (e^G mu S0^T)_i + sum_{j < i} M_ij - sum_{j > i} M_ji
//     su_i = k_i . ((e^{G_63 - G} beta r) dS^T)_i
//     dg_t = sum_{i >= t} dG_i + sum_{i < t} su_i + e^{G_63} <S0, dS>
//     r_j . dU_j = scale sum_{i >= j} P_ij (dO_i . r_j) + su_j / beta_j
// (dG_i without -su_i, which the gate of the chunk's end cancels for i >= t; the
// last sum is formed without beta.)  In the sum over i >= t the pairs with
// both tokens behind t cancel between the row and the column sums, exactly,
// since both add the same float32 M_ij; that is why r, mu and the states enter
// with both bf16 parts, and dg comes out at about 4e-6.
//
// delta_prep_kernel (T, T^T, scale P^T of every chunk), then the two walks:
// delta_chunk_walk<., 1> (the state before every chunk, r) and delta_chunk_rev
// (mu and the state's gradient behind every chunk, 16 columns per wave as the
// forward), then delta_chunk_grads_kernel (all chunks at once: dv, dq, dk summed
// over the value heads of a qk head, dg, dbeta).  The
// walks are bound by the chain from one state to the next, so that everything
// that a chunk can do on its own is left to the last kernel.
#include <algorithm>

#include "delta_walk.cuh"

namespace ssmvjp {
namespace {

// ---------------------------------------------------------------------------
// reverse walk
// ---------------------------------------------------------------------------
// As the forward walk: waves 0 and 1 carry the gradients of 16 columns of the
// state each, waves 2 and 3 work one chunk ahead on the part that does not
// depend on them, B = Q^T (scale e^G dO), and hand it over through LDS, wave 4
// loads and prepares the gates.  195 us for b=2 T=4096 HV=32 K=V=128 (64 chunks
// in a row, 393 MB stored), 150 of them without the stores of mu and dS; a second
// loading wave made it 211, the gates waited for among the loads 225.
template <int KP>
struct RevLds {  // byte offsets
  static constexpr int K = 0, T = K + 64 * KP * 2, P = T + 12 * 1024, ABUF = P + 12 * 1024;    // [2] waves 0, 1
  static constexpr int Q = 2 * ABUF, O = Q + 2 * 64 * KP * 2, B = O + 3 * 4096, BT = KP * 64;  // q [2], d_o [3], B [2][2 tiles]
  static constexpr int G = B + 4 * BT, TOTAL = G + 3 * 768;  // gates: [3][e^G, e^{G_63 - G}, beta]
};
constexpr int REV_NTH = 320;

template <int KP, bool X32>
__device__ __forceinline__ void delta_chunk_rev(const DeltaChunkArgs& a, unsigned block) {
  constexpr int KS = KP / 32, KT = KP / 16;
  typedef RevLds<KP> L;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, q = lane >> 4;
  const int t16 = w & 1;
  const WalkUnit wu = walk_unit(block, (a.V + 31) / 32);
  const i64 unit = wu.unit, slice = wu.slice;
  if (unit >= a.seq.nseq * a.HV) return;
  const i64 n = unit / a.HV, hv = unit % a.HV, h = hv / a.rep;
  const DeltaSpan sp = a.seq.span(n);
  const int nch = (int)((sp.len + DCH - 1) / DCH);
  const i64 v0 = slice * 32 + t16 * 16, vt = slice * 2 + t16;
  const bool act = v0 < a.V;
  const i64 cell0 = sp.slot0 * a.HV + hv;
  auto gates = [&](int ch) { return (float*)(smem_raw + L::G + ch % 3 * 768); };
  auto d_o = [&](int ch) { return (const bf16*)(smem_raw + L::O + ch % 3 * 4096); };
  auto at4 = [&](const float* p, int m) { return *(const f32x4*)(p + 16 * m + 4 * q); };
  auto Bof = [&](int ch) { return (f32x4*)(smem_raw + L::B + ((ch & 1) * 2 + t16) * L::BT) + lane; };

  if (w < 2) {
    // ------------------------------------------------------ the state's gradient
    __builtin_amdgcn_s_setprio(3);
    f32x4 dS[KT];
    Frag8 dh[KS], dl[KS];  // its two parts
    const brsrc rs = state_rsrc(a.dSf, a, unit, act);
#pragma unroll
    for (int t = 0; t < KT; ++t) dS[t] = load_state4(rs, a, t, q, v0 + c);
#pragma unroll
    for (int s = 0; s < KS; ++s) split8(dS[2 * s], dS[2 * s + 1], dh[s], dl[s]);
    __syncthreads();
    __syncthreads();  // the period in which B of the last chunk is made
    for (int ch = nch - 1; ch >= 0; --ch) {
      if (act) {
        if constexpr (X32) store_state32(a.dS32 + (cell0 + ch * a.HV) * a.K * a.V, dS, a.K, a.V, q, v0 + c);
        const unsigned char* const buf = smem_raw + (ch & 1) * L::ABUF;
        const bf16* Kt = (const bf16*)(buf + L::K);
        const u32x4 *Tt = (const u32x4*)(buf + L::T) + lane, *Pt = (const u32x4*)(buf + L::P) + lane;
        const bf16* Ot = d_o(ch);
        const f32x4* B = Bof(ch);
        const i64 tile = (cell0 + ch * a.HV) * a.nvt + vt;
        u32x4* Dw = (u32x4*)(a.dSw + tile * 2 * KS * 512) + state_slot(lane);
        s16x4* Mw = (s16x4*)(a.muw + tile * 4 * 512) + row_slot(lane);
        const float *eG = gates(ch), *eE = eG + 64, *be = eG + 128;
        // 1: z = K dS, row tiles 2 and 3, both parts of dS
        f32x4 z[4], du[4], e[4], b[4];
        Frag8 kf[2][KS], kg[2][KS], of[2], ph[6], pl[6];
#pragma unroll
        for (int s = 0; s < KS; ++s) kf[0][s] = row_frag(Kt, KP, 2, s, lane), kf[1][s] = row_frag(Kt, KP, 3, s, lane);
        SSMVJP_FENCE();
#pragma unroll
        for (int m = 0; m < 4; ++m) z[m] = zero4(), du[m] = zero4();
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          z[2] = mma32(kf[0][s], dl[s], z[2]);
          z[3] = mma32(kf[1][s], dl[s], z[3]);
          z[2] = mma32(kf[0][s], dh[s], z[2]);
          z[3] = mma32(kf[1][s], dh[s], z[3]);
        }
#pragma unroll
        for (int i = 0; i < 6; ++i) ph[i] = as_frag(Pt[i * 128]), pl[i] = as_frag(Pt[i * 128 + 64]);
#pragma unroll
        for (int s = 0; s < 2; ++s) of[s] = {col4(Ot, 32, 2 * s, t16, lane), col4(Ot, 32, 2 * s + 1, t16, lane)};
#pragma unroll
        for (int s = 0; s < KS; ++s) stream_store(Dw + s * 64, as_u4(dh[s])), stream_store(Dw + (KS + s) * 64, as_u4(dl[s]));
        pipe<4 * KS, 2, 1>();
        SSMVJP_FENCE();
        // 2: scale P^T dO
#pragma unroll
        for (int s = 1; s >= 0; --s) {
#pragma unroll
          for (int m = 0; m < 2 * s + 2; ++m) du[m] = mma32(pl[frag_up(m, s)], of[s], du[m]);
#pragma unroll
          for (int m = 0; m < 2 * s + 2; ++m) du[m] = mma32(ph[frag_up(m, s)], of[s], du[m]);
        }
#pragma unroll
        for (int s = 0; s < KS; ++s) kg[0][s] = row_frag(Kt, KP, 0, s, lane), kg[1][s] = row_frag(Kt, KP, 1, s, lane);
#pragma unroll
        for (int m = 0; m < 4; ++m) e[m] = at4(eE, m), b[m] = at4(be, m);
        pipe<12, 2, 2>();
        SSMVJP_FENCE();
        // 3: z, row tiles 0 and 1; beta dU of tiles 2 and 3, dU = scale P^T dO + e^{G_63 - G} z
        Frag8 bh[2], bl[2], th[6], tl[6];
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          z[0] = mma32(kg[0][s], dl[s], z[0]);
          z[1] = mma32(kg[1][s], dl[s], z[1]);
          z[0] = mma32(kg[0][s], dh[s], z[0]);
          z[1] = mma32(kg[1][s], dh[s], z[1]);
        }
        f32x4 mu[4];
        auto bdu = [&](int s) {
#pragma unroll
          for (int m = 2 * s; m < 2 * s + 2; ++m) mu[m] = b[m] * (du[m] + e[m] * z[m]);
          split8(mu[2 * s], mu[2 * s + 1], bh[s], bl[s]);
        };
        bdu(1);
#pragma unroll
        for (int i = 0; i < 6; ++i) th[i] = as_frag(Tt[i * 128]), tl[i] = as_frag(Tt[i * 128 + 64]);
        pipe<4 * KS, 3, 1>();
        SSMVJP_FENCE();
        // 4: mu = T^T (beta dU), contraction over tiles 2 and 3; the decay of dS, plus B
        f32x4 y[2];  // tiles 0 and 1 get this part later
        y[0] = mma32(th[frag_up(0, 1)], bl[1], zero4());
        y[1] = mma32(th[frag_up(1, 1)], bl[1], zero4());
        mu[2] = mma32(th[frag_up(2, 1)], bl[1], mu[2]);
        mu[3] = mma32(th[frag_up(3, 1)], bl[1], mu[3]);
        y[0] = mma32(tl[frag_up(0, 1)], bh[1], y[0]);
        y[1] = mma32(tl[frag_up(1, 1)], bh[1], y[1]);
        mu[2] = mma32(tl[frag_up(2, 1)], bh[1], mu[2]);
        mu[3] = mma32(tl[frag_up(3, 1)], bh[1], mu[3]);
        y[0] = mma32(th[frag_up(0, 1)], bh[1], y[0]);
        y[1] = mma32(th[frag_up(1, 1)], bh[1], y[1]);
        mu[2] = mma32(th[frag_up(2, 1)], bh[1], mu[2]);
        mu[3] = mma32(th[frag_up(3, 1)], bh[1], mu[3]);
        bdu(0);
        const float eEnd = eG[63];
#pragma unroll
        for (int t = 0; t < KT; ++t) dS[t] = eEnd * dS[t] + B[t * 64];
        pipe<12, 5, 1>();
        SSMVJP_FENCE();
        // 5: contraction over tiles 0 and 1; -e^G mu of tiles 2 and 3
        y[0] = mma32(th[frag_up(0, 0)], bl[0], y[0]);
        y[1] = mma32(th[frag_up(1, 0)], bl[0], y[1]);
        y[0] = mma32(tl[frag_up(0, 0)], bh[0], y[0]);
        y[1] = mma32(tl[frag_up(1, 0)], bh[0], y[1]);
        y[0] = mma32(th[frag_up(0, 0)], bh[0], y[0]);
        y[1] = mma32(th[frag_up(1, 0)], bh[0], y[1]);
        Frag8 nh[2], nl[2], ct[2][KT];
        auto turn = [&](int s) {
          split8(-at4(eG, 2 * s) * mu[2 * s], -at4(eG, 2 * s + 1) * mu[2 * s + 1], nh[s], nl[s]);
        };
        auto keep = [&](int s) {
          Frag8 hi, lo;
          split8(mu[2 * s], mu[2 * s + 1], hi, lo);
          stream_store(Mw + 2 * s * 64, hi.a);
          stream_store(Mw + (2 * s + 1) * 64, hi.b);
          stream_store(Mw + 256 + 2 * s * 64, lo.a);
          stream_store(Mw + 256 + (2 * s + 1) * 64, lo.b);
        };
        turn(1);
#pragma unroll
        for (int t = 0; t < KT; ++t) ct[1][t] = key_frag(Kt, KP, t, 1, lane);
        pipe<6, 8, 3>();
        SSMVJP_FENCE();
        // 6: dS0 = e^{G_63} dS + B - K^T (e^G mu), tokens of tiles 2 and 3
#pragma unroll
        for (int t = 0; t < KT; ++t) dS[t] = mma32(ct[1][t], nl[1], dS[t]);
#pragma unroll
        for (int t = 0; t < KT; ++t) dS[t] = mma32(ct[1][t], nh[1], dS[t]);
        mu[0] += y[0];
        mu[1] += y[1];
        turn(0);
        keep(1);
#pragma unroll
        for (int t = 0; t < KT; ++t) ct[0][t] = key_frag(Kt, KP, t, 0, lane);
        pipe<2 * KT, 5, 1>();
        SSMVJP_FENCE();
        // 7: tokens of tiles 0 and 1; the parts of the state tiles that are done
        constexpr int PT = KT < 4 ? KT : 4;  // state tiles at a time
#pragma unroll
        for (int g = 0; g < KT; g += PT) {
#pragma unroll
          for (int t = g; t < g + PT; ++t) dS[t] = mma32(ct[0][t], nl[0], dS[t]);
#pragma unroll
          for (int t = g; t < g + PT; ++t) dS[t] = mma32(ct[0][t], nh[0], dS[t]);
          if (g == 0) {
            keep(0);
          } else {
#pragma unroll
            for (int s = (g - PT) / 2; s < g / 2; ++s) split8(dS[2 * s], dS[2 * s + 1], dh[s], dl[s]);
          }
          pipe<2 * PT, 6, 0>();
          SSMVJP_FENCE();
        }
#pragma unroll
        for (int s = (KT - PT) / 2; s < KS; ++s) split8(dS[2 * s], dS[2 * s + 1], dh[s], dl[s]);
      }
      __syncthreads();
    }
    if (a.dS0 && act) {
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int k = state_row(t, q) + r;
          if (k < a.K) a.dS0[(unit * a.K + k) * a.V + v0 + c] = dS[t][r];
        }
    }
  } else if (w < 4) {
    // ------------------------------------------------- B = Q^T (scale e^G dO) ahead
    __syncthreads();
    for (int p = nch; p >= 0; --p) {  // chunk p - 1 here, chunk p at the gradients
      if (act && p > 0) {
        const int ch = p - 1;
        const bf16 *Qt = (const bf16*)(smem_raw + L::Q + (ch & 1) * 64 * KP * 2), *Ot = d_o(ch);
        const float* eG = gates(ch);
        f32x4* B = Bof(ch);
        Frag8 oh[2], ol[2], ct[2][KT];
#pragma unroll
        for (int t = 0; t < KT; ++t) ct[0][t] = key_frag(Qt, KP, t, 0, lane);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          f32x4 o[2];
#pragma unroll
          for (int m = 0; m < 2; ++m) o[m] = a.scale * at4(eG, 2 * s + m) * unpack4(col4(Ot, 32, 2 * s + m, t16, lane));
          split8(o[0], o[1], oh[s], ol[s]);
        }
        SSMVJP_FENCE();
        f32x4 x[KT];
#pragma unroll
        for (int t = 0; t < KT; ++t) x[t] = mma32(ct[0][t], ol[0], zero4());
#pragma unroll
        for (int t = 0; t < KT; ++t) x[t] = mma32(ct[0][t], oh[0], x[t]);
#pragma unroll
        for (int t = 0; t < KT; ++t) ct[1][t] = key_frag(Qt, KP, t, 1, lane);
        SSMVJP_FENCE();
#pragma unroll
        for (int t = 0; t < KT; ++t) x[t] = mma32(ct[1][t], ol[1], x[t]);
#pragma unroll
        for (int t = 0; t < KT; ++t) x[t] = mma32(ct[1][t], oh[1], x[t]);
#pragma unroll
        for (int t = 0; t < KT; ++t) B[t * 64] = x[t];
      }
      __syncthreads();
    }
  } else {
    // --------------------------------------------------------------- the loader
    const unsigned lds0 = lds_base(smem_raw);
    RowDma<KP, 1> rows_dma;
    ColDma<2, 1> cols_dma;
    rows_dma.init(0, lane, a.H * a.K, a.K);
    cols_dma.init(0, lane, a.HV * a.V, slice * 32, a.V);
    auto rows_of = [&](int ch) { return (int)(sp.len - (i64)ch * DCH < DCH ? sp.len - (i64)ch * DCH : DCH); };
    auto issue_a = [&](int ch) {  // k, T^T and P^T of chunk ch
      const unsigned b = lds0 + (unsigned)((ch & 1) * L::ABUF);
      const i64 cu = cell0 + ch * a.HV;
      rows_dma.issue(b + L::K, 0, row_words(a.k, sp.start + (i64)ch * DCH, rows_of(ch), a.H, h, a.K, 0));
      flat_dma<12, 1>(b + L::T, 0, lane, rsrc_words_u(a.Tt + cu * 6 * 2 * 512, 12 * 1024));
      flat_dma<12, 1>(b + L::P, 0, lane, rsrc_words_u(a.Pt + cu * 6 * 2 * 512, 12 * 1024));
    };
    auto issue_b = [&](int ch) {  // q and d_o
      const i64 tok0 = sp.start + (i64)ch * DCH;
      rows_dma.issue(lds0 + (unsigned)(L::Q + (ch & 1) * 64 * KP * 2), 0, row_words(a.q, tok0, rows_of(ch), a.H, h, a.K, 0));
      cols_dma.issue(lds0 + (unsigned)(L::O + ch % 3 * 4096), 0,
                     row_words(a.d_o, tok0, rows_of(ch), a.HV, hv, a.V, slice * 32));
    };
    float sG = 0.0f, sB = 0.0f;
    auto fetch_gates = [&](int ch) {
      sG = a.G[(cell0 + ch * a.HV) * 64 + lane];
      const i64 t = (i64)ch * DCH + lane;
      sB = t < sp.len ? a.beta[(sp.start + t) * a.HV + hv] : 0.0f;
    };
    auto commit_gates = [&](int ch) {
      float* g = gates(ch) + lane;
      const float end = __shfl(sG, 63, 64);
      g[0] = exp_hw(sG);
      g[64] = exp_hw(end - sG);
      g[128] = sB;
    };
    // gates are fetched a period before they are prepared: a wait for them among the loads would be one for all
    if (nch > 0) {
      fetch_gates(nch - 1);
      issue_b(nch - 1);
      commit_gates(nch - 1);
      if (nch > 1) fetch_gates(nch - 2);
    }
    dma_wait();
    __syncthreads();
    for (int p = nch; p >= 0; --p) {
      if (p > 1) commit_gates(p - 2);
      SSMVJP_FENCE();
      if (p > 2) fetch_gates(p - 3);
      if (p > 0) issue_a(p - 1);
      if (p > 1) issue_b(p - 2);
      dma_wait();
      __syncthreads();
    }
  }
}

// The two walks need nothing of each other unless dS0 is written over S0: with
// BOTH, blocks below `half` are reverse walks (they take longer and go first),
// the others forward walks.  X32: both keep what they keep in float32 too.
template <int KP, bool BOTH, bool X32>
__global__ void __launch_bounds__(REV_NTH) __attribute__((amdgpu_waves_per_eu(2, 2)))
delta_chunk_rev_kernel(DeltaChunkArgs a, unsigned half) {
  if (!BOTH || blockIdx.x < half) delta_chunk_rev<KP, X32>(a, blockIdx.x);
  else if (threadIdx.x < walk_nth(1)) delta_chunk_walk<KP, X32 ? 2 : 1>(a, blockIdx.x - half);  // two waves end here
}
template <int KP, bool X32>
__global__ void __launch_bounds__(walk_nth(1)) __attribute__((amdgpu_waves_per_eu(2, 2)))
delta_chunk_states_kernel(DeltaChunkArgs a) {
  delta_chunk_walk<KP, X32 ? 2 : 1>(a, blockIdx.x);
}

// su_i = e^{G_63 - G_i} r_i . (K dS)_i and <S0, dS> of one cell from float32 r, S0
// and dS (K dS in three parts of dS), for few cells.  dg is a sum of a few such
// terms of either sign, and with r and dS in two bf16 parts (2e-6 of each value)
// it comes out at 5e-6 of its norm where many cells make up the norm, but at 1e-5
// and more for a short sequence of a few heads (1.4e-5 for 30 tokens of 2).
// Eight waves, each every eighth tile of 16 columns.
template <int KP>
__global__ void __launch_bounds__(512) delta_su_kernel(DeltaChunkArgs a) {
  constexpr int KS = KP / 32;
  __shared__ float red[8][64], dots[8];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, q = lane >> 4;
  const i64 cell = blockIdx.x, slot = cell / a.HV, hv = cell % a.HV, h = hv / a.rep;
  const ChunkAt at = chunk_at(a.seq, slot, lane);
  if (at.rows == 0) return;
  const brsrc rd = state_rsrc(a.dS32, a, cell, true), rs = state_rsrc(a.S32, a, cell, true);
  const brsrc rk = row_rsrc(a.k, at.tok0, at.rows, a.H, h, a.K);
  u32x4 kf[4][KS];
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int col = 32 * s + 8 * q;
      kf[m][s] = bload16(rk, col < a.K ? (unsigned)(((16 * m + c) * a.H * a.K + col) * 2) : BUF_OOB);
    }
  f32x4 su[4];
#pragma unroll
  for (int m = 0; m < 4; ++m) su[m] = zero4();
  float dot = 0.0f;
  for (i64 vt = w; vt < a.nvt; vt += 8) {
    const i64 v = 16 * vt + c;
    f32x4 z[4], x[2 * KS];
#pragma unroll
    for (int m = 0; m < 4; ++m) z[m] = zero4();
#pragma unroll
    for (int t = 0; t < 2 * KS; ++t) x[t] = load_state4(rd, a, t, q, v);  // rows 32s + 8q + 4 (t & 1) ..
#pragma unroll
    for (int t = 0; t < 2 * KS; ++t) {
      const f32x4 s0 = load_state4(rs, a, t, q, v);
#pragma unroll
      for (int r = 0; r < 4; ++r) dot = fmaf(s0[r], x[t][r], dot);
    }
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      Frag8 hi, mid, lo;
      split8x3(x[2 * s], x[2 * s + 1], hi, mid, lo);
#pragma unroll
      for (int m = 0; m < 4; ++m) z[m] = mma32(kf[m][s], as_u4(lo), z[m]);
#pragma unroll
      for (int m = 0; m < 4; ++m) z[m] = mma32(kf[m][s], as_u4(mid), z[m]);
#pragma unroll
      for (int m = 0; m < 4; ++m) z[m] = mma32(kf[m][s], as_u4(hi), z[m]);
    }
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) su[m][r] = fmaf(z[m][r], a.r32[(cell * 64 + 16 * m + 4 * q + r) * a.V + v], su[m][r]);
  }
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float x = sum16(su[m][r]);
      if (c == 0) red[w][16 * m + 4 * q + r] = x;
    }
  dot = wave_sum(dot);
  if (lane == 0) dots[w] = dot;
  __syncthreads();
  if (w == 0) {
    const float G = a.G[cell * 64 + lane], end = __shfl(G, 63, 64);
    float s = 0.0f, t = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += red[i][lane], t += dots[i];
    a.su[cell * 64 + lane] = exp_hw(end - G) * s;
    if (lane == 0) a.dot[cell] = t;
  }
}

// ---------------------------------------------------------------------------
// gradients of one chunk of one qk head
// ---------------------------------------------------------------------------
// Eight waves: wave (wr = w % 4, half = w / 4) owns row tile wr of every 64-row
// result and one half of its columns (of the keys, or of the pairs' tokens j).
// The columns of V go by 32 (one contraction step): r, mu, S0 and dS of the
// slice, both parts, and d_o come to LDS by LDS-direct loads, one slice ahead
// and over the border between two value heads (two buffers), and are read
// transposed, the contraction running over v.  dD and E then take the place of
// the last slice.
//
// A workgroup takes a CU, and what it waits for (the barriers between the steps of
// a head, loads) nobody fills, so that it goes from unit to unit with the next
// one's first slice, k, q and gates on their way: b=2 T=4096 H=16 HV=32 K=V=128
// takes 285 us for 4096 chunks of a head, 208 KB each (3.0 TB/s; a workgroup per
// unit: 295; 60 us less if the blocks came from the L2), the matrix cores 20 % busy
// (442 MFMAs of 16 cycles a wave and unit) and the LDS 34 %, 43 % of that bank
// conflicts (the pitches below): most of the time the waves wait.  Two workgroups
// per CU would need half the registers (1024 threads spilled and were slower).
constexpr int GRADS_NTH = 512;

// Row pitches of the padded tiles: 40 bytes past a multiple of 128.  The 16 rows
// of a fragment read meet 16 different pairs of banks, the 4 rows of a transposed
// read overlap in 24 bytes of 128, and, unlike in a swizzled tile, every
// fragment is the lane's own address plus a constant: swizzled, the addresses
// alone took more registers than there are.
constexpr int P64 = 64 + 20;
__device__ __forceinline__ Frag8 prow(const bf16* t, int pitch, int m, int s, int lane) {
  return {ld_colk(t, pitch, 16 * m, 32 * s, lane).v, ld_colk(t, pitch, 16 * m, 32 * s + 16, lane).v};
}
__device__ __forceinline__ Frag8 pcol(const bf16* t, int pitch, int m, int s, int lane) {
  return {ld_rowk(t, pitch, 32 * s, 16 * m, lane).v, ld_rowk(t, pitch, 32 * s + 16, 16 * m, lane).v};
}
__device__ __forceinline__ void pstore(bf16* t, int pitch, int row, int col, const u32x4& u) {
  typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
  u32x2* d = (u32x2*)(t + row * pitch + col);
  d[0] = u32x2{u[0], u[1]};
  d[1] = u32x2{u[2], u[3]};
}

template <int KP>
struct GradsLds {  // byte offsets
  static constexpr int KS = KP / 32, PK = KP + 20;
  static constexpr int R = 0, MU = 8 * 1024, S = 16 * 1024, DS = S + 4 * KS * 1024, DO = DS + 4 * KS * 1024, SLICE = DO + 4096;
  static constexpr int PAIRS = 4 * 64 * P64 * 2;  // dD^T, E^T, two parts each
  static constexpr int BUF = SLICE > PAIRS ? SLICE : PAIRS;
  static constexpr int K = 2 * BUF, Q = K + 64 * PK * 2, F = Q + 64 * PK * 2, TOTAL = F + 4 * (2 * 2 * 64 + 3 * 2 * 64 + 2 * 4 * 64 + 8);
};

template <int KP>
__global__ void __launch_bounds__(GRADS_NTH, 2) delta_chunk_grads_kernel(DeltaChunkArgs a) {
  constexpr int KS = KP / 32, KT = KP / 16, PK = KP + 20, HT = KT / 2;  // HT: key tiles of a wave
  typedef GradsLds<KP> L;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  bf16 *const Kb = (bf16*)(smem_raw + L::K), *const Qb = (bf16*)(smem_raw + L::Q);
  float* const gates = (float*)(smem_raw + L::F);  // [2 heads][G, beta]
  // row terms of dG, su without beta, row sums of M (by half); column sums of M and of dbeta's pairs (by row tile);
  // <S0, dS> by wave
  float(*const rowT)[64] = (float(*)[64])(gates + 256), (*const rowU)[64] = rowT + 2, (*const rowM)[64] = rowT + 4;
  float(*const colM)[64] = (float(*)[64])(gates + 640), (*const colA)[64] = colM + 4;
  float* const dots = gates + 640 + 512;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, q = lane >> 4;
  const int wr = w & 3, half = w >> 2;
  const unsigned H32 = (unsigned)a.H;
  // the workgroup's units (slot, qk head): from one to the next that has tokens
  const unsigned units = (unsigned)(a.nslots * a.H);
  unsigned un = blockIdx.x;
  i64 tok0 = 0;
  int rows = 0;
  for (; un < units; un += gridDim.x) {
    const ChunkAt x = chunk_at(a.seq, un / H32, lane);
    tok0 = x.tok0;
    rows = x.rows;
    if (rows) break;
  }
  if (un >= units) return;
  i64 h = un % H32, slot = un / H32;
  const int nsl = (int)(a.nvt + 1) / 2, nvt = (int)a.nvt;
  const unsigned lds0 = lds_base(smem_raw);
  const int orow = 16 * wr + (lane >> 2), ocol = (lane & 3) * 8;  // this lane's piece of d_o
  const unsigned ooff = (unsigned)((orow * a.HV * a.V + ocol) * 2);
  // slice sl of value head hv into buffer bf, in three parts (r, mu and d_o; S0; dS), tiles past V as zeros
  auto issue = [&](int part, i64 tok0, int rows, i64 slot, i64 hv, int sl, int bf) {
    const i64 tile = (slot * a.HV + hv) * nvt + 2 * sl;
    const unsigned b = lds0 + (unsigned)(bf * L::BUF), left = nvt - 2 * sl > 1 ? 2u : 1u;
    if (part == 0) {
      flat_dma<8, 8>(b + L::R, w, lane, rsrc_words_u(a.rw + tile * 2048, left * 4096u));
      flat_dma<8, 8>(b + L::MU, w, lane, rsrc_words_u(a.muw + tile * 2048, left * 4096u));
      if (half == 0)
        dma_dwordx4(b + L::DO + 1024u * (unsigned)wr, sl * 32 + ocol < a.V ? ooff : BUF_OOB,
                    row_words(a.d_o, tok0, rows, a.HV, hv, a.V, sl * 32));
    } else if (part == 1) {
      flat_dma<4 * KS, 8>(b + L::S, w, lane, rsrc_words_u(a.Sw + tile * KS * 1024, left * KS * 2048u));
    } else {
      flat_dma<4 * KS, 8>(b + L::DS, w, lane, rsrc_words_u(a.dSw + tile * KS * 1024, left * KS * 2048u));
    }
  };
#pragma unroll
  for (int i = 0; i < 3; ++i) issue(i, tok0, rows, slot, h * a.rep, 0, 0);
  int bf = 0;  // the buffer of the slice at hand
  // k and q of a unit, a value head's gates: loaded ahead
  constexpr int N = 64 * KP / 8 / GRADS_NTH;
  u32x4 tk[N], tq[N];
  float G1 = 0.0f, b1 = 0.0f;
  // the thread's number, anew: addresses made from it are not kept in registers from unit to unit
  auto thread = [&] {
    int t = tid;
    asm volatile("" : "+v"(t));
    return t;
  };
  auto load_kq = [&](i64 tok0, int rows, i64 h) {
    const int tid = thread();
    const brsrc rk = row_rsrc(a.k, tok0, rows, a.H, h, a.K), rq = row_rsrc(a.q, tok0, rows, a.H, h, a.K);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int p = tid + GRADS_NTH * i, row = p / (KP / 8), col = p % (KP / 8) * 8;
      const unsigned o = col < a.K ? (unsigned)(((i64)row * a.H * a.K + col) * 2) : BUF_OOB;
      tk[i] = bload16(rk, o);
      tq[i] = bload16(rq, o);
    }
  };
  auto load_gates = [&](i64 tok0, int rows, i64 slot, i64 hv) {
    G1 = a.G[(slot * a.HV + hv) * 64 + lane];
    b1 = lane < rows ? a.beta[(tok0 + lane) * a.HV + hv] : 0.0f;
  };
  load_kq(tok0, rows, h);
  if (w == 0) load_gates(tok0, rows, slot, h * a.rep);
  for (;;) {
    un += gridDim.x;
    i64 ntok0 = 0;  // the next unit
    int nrows = 0;
    for (; un < units; un += gridDim.x) {
      const ChunkAt x = chunk_at(a.seq, un / H32, lane);
      ntok0 = x.tok0;
      nrows = x.rows;
      if (nrows) break;
    }
    const i64 nslot = un / H32, nh = un % H32;
    const bool next = un < units;
    const int tn = thread();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int p = tn + GRADS_NTH * i;
      pstore(Kb, PK, p / (KP / 8), p % (KP / 8) * 8, tk[i]);
      pstore(Qb, PK, p / (KP / 8), p % (KP / 8) * 8, tq[i]);
    }
    if (w == 0) {
      gates[lane] = G1;
      gates[64 + lane] = b1;
    }
    __syncthreads();
    f32x4 qk[2], kk[2];  // q_i . k_j and k_i . k_j of column tiles 2 half and 2 half + 1, for every value head
    {
      Frag8 fq[KS], fk[KS];
#pragma unroll
      for (int s = 0; s < KS; ++s) fq[s] = prow(Qb, PK, wr, s, lane), fk[s] = prow(Kb, PK, wr, s, lane);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        qk[e] = kk[e] = zero4();
        if (2 * half + e <= wr) {
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            const Frag8 f = prow(Kb, PK, 2 * half + e, s, lane);
            qk[e] = mma32(fq[s], f, qk[e]);
            kk[e] = mma32(fk[s], f, kk[e]);
          }
        }
      }
    }
    f32x4 dq[HT], dk[HT];  // rows i = 16 wr + 4 q + r, column 16 (HT half + t) + c
#pragma unroll
    for (int t = 0; t < HT; ++t) dq[t] = zero4(), dk[t] = zero4();

    for (i64 rr = 0; rr < a.rep; ++rr) {
      const i64 hv = h * a.rep + rr;
      const float *const Gs = gates + (rr & 1) * 128, *const Bs = Gs + 64;
      if (w == 0 && rr + 1 < a.rep) load_gates(tok0, rows, slot, hv + 1);
      f32x4 po[2], pm[2], x1[HT], y2[HT], y3[HT];  // dO . r, mu . r; dO S0^T, mu S0^T, r dS^T
#pragma unroll
      for (int e = 0; e < 2; ++e) po[e] = zero4(), pm[e] = zero4();
#pragma unroll
      for (int t = 0; t < HT; ++t) x1[t] = zero4(), y2[t] = zero4(), y3[t] = zero4();
      f32x4 dot = zero4();
      dma_wait();
      __syncthreads();  // the first slice has landed
      if (w == 0) {
        float* const g = gates + ((rr + 1) & 1) * 128 + lane;  // the previous head's: its readers are past a barrier
        g[0] = G1;
        g[64] = b1;
      }
      for (int sl = 0; sl < nsl; ++sl) {
        const bool last = sl + 1 == nsl;
        // the next slice's loads, spread over this one's products: all at once they block for 2,000 cycles
        const bool over = last && rr + 1 == a.rep, ahead = !over || next;
        const i64 nhv = over ? nh * a.rep : last ? hv + 1 : hv, nsl2 = over ? nslot : slot;
        const i64 tok2 = over ? ntok0 : tok0;
        const int rows2 = over ? nrows : rows;
        const int nxt = last ? 0 : sl + 1;
        if (ahead) issue(0, tok2, rows2, nsl2, nhv, nxt, bf ^ 1);
        const unsigned char* const buf = smem_raw + bf * L::BUF;
        const bf16 *R = (const bf16*)(buf + L::R), *MU = (const bf16*)(buf + L::MU), *S = (const bf16*)(buf + L::S),
                   *DS = (const bf16*)(buf + L::DS);
        const s16x4* const orp = (const s16x4*)(buf + L::DO) + (16 * wr + c) * 8 + q;  // rows of 32 columns
        const Frag8 of = {orp[0], orp[4]};
        // [tile][hi, lo]: 1024 values each of r and mu, 512 KS of the states
        const Frag8 mh = kept_rows(MU, MU + 2048, wr, lane), ml = kept_rows(MU + 1024, MU + 2048 + 1024, wr, lane);
        const Frag8 rh = kept_rows(R, R + 2048, wr, lane), rl = kept_rows(R + 1024, R + 2048 + 1024, wr, lane);
#pragma unroll
        for (int t = 0; t < HT; ++t) {
          const int k = HT * half + t;
          const Frag8 sh = kept_keys(S, S + 1024 * KS, k, lane), sl2 = kept_keys(S + 512 * KS, S + 1536 * KS, k, lane);
          const Frag8 dh = kept_keys(DS, DS + 1024 * KS, k, lane), dl = kept_keys(DS + 512 * KS, DS + 1536 * KS, k, lane);
          x1[t] = mma32(of, sl2, x1[t]);
          y2[t] = mma32(ml, sh, y2[t]);
          y3[t] = mma32(rl, dh, y3[t]);
          y2[t] = mma32(mh, sl2, y2[t]);
          y3[t] = mma32(rh, dl, y3[t]);
          x1[t] = mma32(of, sh, x1[t]);
          y2[t] = mma32(mh, sh, y2[t]);
          y3[t] = mma32(rh, dh, y3[t]);
        }
        if (ahead) issue(1, tok2, rows2, nsl2, nhv, nxt, bf ^ 1);
        // also where all of a tile lies above the diagonal and is dropped later: straight code is read ahead
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const Frag8 bh = kept_rows(R, R + 2048, 2 * half + e, lane), bl = kept_rows(R + 1024, R + 2048 + 1024, 2 * half + e, lane);
          po[e] = mma32(of, bl, po[e]);
          pm[e] = mma32(mh, bl, pm[e]);
          po[e] = mma32(of, bh, po[e]);
          pm[e] = mma32(ml, bh, pm[e]);
          pm[e] = mma32(mh, bh, pm[e]);
        }
        if (ahead) issue(2, tok2, rows2, nsl2, nhv, nxt, bf ^ 1);
        if (w < 2 * KS) {  // this wave's 64 pieces of each array
          const int o = (w / KS) * 1024 * KS + (w % KS) * 512 + lane * 8;
          const Frag8 s0 = as_frag(*(const u32x4*)(S + o)), s1 = as_frag(*(const u32x4*)(S + o + 512 * KS));
          const Frag8 d0 = as_frag(*(const u32x4*)(DS + o)), d1 = as_frag(*(const u32x4*)(DS + o + 512 * KS));
          dot += (unpack4(s0.a) + unpack4(s1.a)) * (unpack4(d0.a) + unpack4(d1.a));
          dot += (unpack4(s0.b) + unpack4(s1.b)) * (unpack4(d0.b) + unpack4(d1.b));
        }
        // dv = mu, rounded: its hi part
        if (half == 1) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int col = sl * 32 + 16 * e + 4 * q;
            if (16 * wr + c < rows && col < a.V)
              *(s16x4*)(a.dv + ((tok0 + 16 * wr + c) * a.HV + hv) * a.V + col) = e ? mh.b : mh.a;
          }
        }
        if (!last) {
          dma_wait();
          __syncthreads();
          bf ^= 1;
        }
      }
      // rows i = 16 wr + 4 q + r
      const f32x4 Gi = *(const f32x4*)(Gs + 16 * wr + 4 * q), Bi = *(const f32x4*)(Bs + 16 * wr + 4 * q);
      const float Ge = Gs[63];
      f32x4 eg, ee, rt = zero4(), ru = zero4();
#pragma unroll
      for (int r = 0; r < 4; ++r) eg[r] = exp_hw(Gi[r]), ee[r] = exp_hw(Ge - Gi[r]);
#pragma unroll
      for (int t = 0; t < HT; ++t) {
        const f32x4 q4 = unpack4(ld_rowk(Qb, PK, 16 * wr, 16 * (HT * half + t), lane).v);
        const f32x4 k4 = unpack4(ld_rowk(Kb, PK, 16 * wr, 16 * (HT * half + t), lane).v);
        x1[t] *= a.scale * eg;
        y2[t] *= eg;
        y3[t] *= ee;
        dq[t] += x1[t];
        dk[t] += Bi * y3[t] - y2[t];
        rt += q4 * x1[t] - k4 * y2[t];
        ru += k4 * y3[t];
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) rt[r] = sum16(rt[r]), ru[r] = sum16(ru[r]);
      if (c == 0) {
        *(f32x4*)(rowT[half] + 16 * wr + 4 * q) = rt;
        *(f32x4*)(rowU[half] + 16 * wr + 4 * q) = ru;
      }
      const float dsum = wave_sum((dot[0] + dot[1]) + (dot[2] + dot[3]));
      if (lane == 0) dots[w] = dsum;
      __syncthreads();  // the last slice's readers are done
      // pair terms; column j = 16 b + c
      f32x4 rm = zero4();
      bf16* const pairs = (bf16*)(smem_raw + bf * L::BUF);  // dD hi, lo, E hi, lo: [64][64], transposed: row j
      bf ^= 1;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        f32x4 xd = zero4(), xe = zero4();
        float cm = 0.0f, ca = 0.0f;
        const int b = 2 * half + e, j = 16 * b + c;
        if (b <= wr) {
          const float Gj = Gs[j], bj = Bs[j];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int i = 16 * wr + 4 * q + r;
            const float gam = exp_hw(i >= j ? Gi[r] - Gj : 0.0f);
            const float d = i >= j ? a.scale * gam * po[e][r] : 0.0f, m = i > j ? gam * pm[e][r] : 0.0f;
            xd[r] = bj * d;
            xe[r] = -bj * m;
            ca += d * qk[e][r] - m * kk[e][r];  // P_ij (dO_i . r_j) - a_ij N_ij
            const float t = (i > j ? xd[r] * qk[e][r] : 0.0f) + xe[r] * kk[e][r];
            rm[r] += t;
            cm += t;
          }
        }
        cm = sum4q(cm);
        ca = sum4q(ca);
        if (q == 0) {
          colM[wr][j] = cm;
          colA[wr][j] = ca;
        }
        bf16* const o = pairs + j * P64 + 16 * wr + 4 * q;
        s16x4 hi, lo;
        split4(xd, hi, lo);
        *(s16x4*)o = hi;
        *(s16x4*)(o + 64 * P64) = lo;
        split4(xe, hi, lo);
        *(s16x4*)(o + 2 * 64 * P64) = hi;
        *(s16x4*)(o + 3 * 64 * P64) = lo;
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) rm[r] = sum16(rm[r]);
      if (c == 0) *(f32x4*)(rowM[half] + 16 * wr + 4 * q) = rm;
      __syncthreads();
      // dq += dD K, dk += E K (rows i); dk += dD^T Q + E^T K (rows j)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const bool lower = s <= wr >> 1, upper = s >= wr >> 1;
        Frag8 dr[2], er[2], dc[2], ec[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bf16 *D = pairs + e * 64 * P64, *E = pairs + (2 + e) * 64 * P64;
          dr[e] = pcol(D, P64, wr, s, lane);
          er[e] = pcol(E, P64, wr, s, lane);
          dc[e] = prow(D, P64, wr, s, lane);
          ec[e] = prow(E, P64, wr, s, lane);
        }
#pragma unroll
        for (int t = 0; t < HT; ++t) {
          const Frag8 kf = pcol(Kb, PK, HT * half + t, s, lane);
          if (lower) {
            dq[t] = mma32(dr[1], kf, dq[t]);
            dk[t] = mma32(er[1], kf, dk[t]);
            dq[t] = mma32(dr[0], kf, dq[t]);
            dk[t] = mma32(er[0], kf, dk[t]);
          }
          if (upper) {
            const Frag8 qf = pcol(Qb, PK, HT * half + t, s, lane);
            dk[t] = mma32(ec[1], kf, dk[t]);
            dk[t] = mma32(dc[1], qf, dk[t]);
            dk[t] = mma32(ec[0], kf, dk[t]);
            dk[t] = mma32(dc[0], qf, dk[t]);
          }
        }
      }
      // dbeta, dg
      if (w == 0) {
        float col = 0.0f, db = 0.0f, dot0 = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) col += colM[i][lane], db += colA[i][lane];
#pragma unroll
        for (int i = 0; i < 8; ++i) dot0 += dots[i];
        float u = rowU[0][lane] + rowU[1][lane];
        if (a.su) {
          u = a.su[(slot * a.HV + hv) * 64 + lane];
          dot0 = a.dot[slot * a.HV + hv];
        }
        const float dG = rowT[0][lane] + rowT[1][lane] + rowM[0][lane] + rowM[1][lane] - col;
        // true one-sided sums: under strong gates a result is far smaller than the sum over the whole chunk
        const float after = __shfl(wave_incl_scan(__shfl(dG, 63 - lane, 64), lane), 63 - lane, 64);
        const float su = __shfl_up(Bs[lane] * u, 1, 64), before = wave_incl_scan(lane ? su : 0.0f, lane);
        const float sum = after + before + exp_hw(Gs[63]) * dot0;
        if (lane < rows) {
          const i64 o = (tok0 + lane) * a.HV + hv;
          a.dg[o] = sum;
          a.dbeta[o] = db + u;
        }
      }
    }
    if (next) {
      load_kq(ntok0, nrows, nh);
      if (w == 0) load_gates(ntok0, nrows, nslot, nh * a.rep);
    }
    // out, through LDS: 16-byte stores of whole rows in place of two bytes of sixteen columns
    __syncthreads();  // the last pair terms' readers are done
    constexpr int PO = KP + 8;
    const int to = thread(), lo = to & 63, row0 = 16 * wr + 4 * (lo >> 4), col0 = 16 * HT * half + (lo & 15);
    bf16 *const dqb = (bf16*)(smem_raw + (bf ^ 1) * L::BUF), *const dkb = dqb + 64 * PO;
#pragma unroll
    for (int t = 0; t < HT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int o = (row0 + r) * PO + col0 + 16 * t;
        dqb[o] = (bf16)dq[t][r];
        dkb[o] = (bf16)dk[t][r];
      }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 64 * KP / 8 / GRADS_NTH; ++i) {
      const int p = to + GRADS_NTH * i, row = p / (KP / 8), col = p % (KP / 8) * 8;
      if (row < rows && col < a.K) {
        const i64 o = ((tok0 + row) * a.H + h) * a.K + col;
        *(u32x4*)(a.dq + o) = *(const u32x4*)(dqb + row * PO + col);
        *(u32x4*)(a.dk + o) = *(const u32x4*)(dkb + row * PO + col);
      }
    }
    if (!next) return;
    tok0 = ntok0;
    rows = nrows;
    h = nh;
    slot = nslot;
  }
}

template <int KP, bool X32>
void launch_walks(const DeltaChunkArgs& a, unsigned half, bool together, hipStream_t s) {
  static_assert(RevLds<KP>::TOTAL >= WalkLds<KP, 1>::TOTAL && walk_nth(1) == walk_nth(2) &&
                    WalkLds<KP, 1>::TOTAL == WalkLds<KP, 2>::TOTAL, "one launch for both walks");
  const size_t lds = RevLds<KP>::TOTAL;
  if (together) {
    hipLaunchKernelGGL((delta_chunk_rev_kernel<KP, true, X32>), dim3(2 * half), dim3(REV_NTH), lds, s, a, half);
  } else {
    hipLaunchKernelGGL((delta_chunk_states_kernel<KP, X32>), dim3(half), dim3(walk_nth(1)), (WalkLds<KP, 1>::TOTAL), s, a);
    hipLaunchKernelGGL((delta_chunk_rev_kernel<KP, false, X32>), dim3(half), dim3(REV_NTH), lds, s, a, half);
  }
}

// dS0 lies over S0: the reverse walk writes what the forward walk reads, and blocks of one launch have no order
bool writes_over_s0(const DeltaChunkArgs& a) {
  const uintptr_t bytes = (uintptr_t)(a.seq.nseq * a.HV * a.K * a.V * 4), r = (uintptr_t)a.S0, w = (uintptr_t)a.dS0;
  return a.S0 && a.dS0 && r < w + bytes && w < r + bytes;
}

template <int KP>
void launch_walks_grads(const DeltaChunkArgs& a, hipStream_t s) {
  const unsigned half = (unsigned)walk_blocks(a.seq.nseq * a.HV, (a.V + 31) / 32);
  const bool apart = writes_over_s0(a);
  // A workgroup takes a CU, so that the walks run in rounds of 256 workgroups.  Where a walk's last round is not
  // full, one launch of both lets the other fill it: 123 us against 177 us for the whole backward at 64 workgroups
  // per walk (b=1 T=2048 HV=16, K = V = 128), 279 against 292 at 192, 267 against 285 at 384.  Full rounds gain
  // nothing, and the walks' inputs push each other out of the caches: 686 against 675 us at 256 (b=2 T=4096 HV=32),
  // 352 against 348 at 512 and 785 against 719 at 1024 (T=1024).
  if (a.su) {  // few cells
    launch_walks<KP, true>(a, half, !apart, s);
    if (a.nslots > 0)
      hipLaunchKernelGGL((delta_su_kernel<KP>), dim3((unsigned)(a.nslots * a.HV)), dim3(512), 0, s, a);
  } else {
    launch_walks<KP, false>(a, half, !apart && half % 256 != 0 && half < 512, s);
  }
  if (a.nslots > 0)
    hipLaunchKernelGGL((delta_chunk_grads_kernel<KP>), dim3((unsigned)std::min<i64>(a.nslots * a.H, 256)), dim3(GRADS_NTH),
                       (GradsLds<KP>::TOTAL), s, a);
}

struct BwdPlan {
  i64 off_T, off_Tt, off_Pt, off_G, off_S, off_dS, off_r, off_mu;
  i64 off_S32, off_dS32, off_r32, off_su, off_dot;  // few cells only
  bool few;
  size_t bytes;
};
BwdPlan bwd_plan(const ssmvjp_delta_chunk_desc& d) {
  const i64 cells = delta_slots(d) * d.nv_heads, tiles = cells * (d.dv / 16), KP = d.dk <= 64 ? 64 : 128;
  BwdPlan p{};
  i64 off = 0;
  auto carve = [&](i64 bytes) {
    const i64 o = off;
    off += (bytes + 255) / 256 * 256;
    return o;
  };
  p.off_T = carve(cells * 12 * 1024);
  p.off_Tt = carve(cells * 12 * 1024);
  p.off_Pt = carve(cells * 12 * 1024);
  p.off_G = carve(cells * 64 * 4);
  p.off_S = carve(tiles * KP * 16 * 2 * 2);
  p.off_dS = carve(tiles * KP * 16 * 2 * 2);
  p.off_r = carve(tiles * 4 * 1024);
  p.off_mu = carve(tiles * 4 * 1024);
  // few: dg's norm is made up of few sums (delta_su_kernel): 16 cells of K = V = 128, where 48 come out within 8e-6
  // without and the call takes longer (105 against 67 us at 128 cells, b=1 T=512 HV=16).  Narrow keys come out worse
  // (K = 16, V = 48: 9.8e-6 at 140 cells, 8.3e-6 with) and cost less (152 against 129 us at 256 cells).  At most 6 MB
  // of workspace.
  p.few = cells * d.dk * d.dv <= 1 << 18;
  if (p.few) {
    p.off_S32 = carve(cells * d.dk * d.dv * 4);
    p.off_dS32 = carve(cells * d.dk * d.dv * 4);
    p.off_r32 = carve(cells * 64 * d.dv * 4);
    p.off_su = carve(cells * 64 * 4);
    p.off_dot = carve(cells * 4);
  }
  p.bytes = (size_t)off;
  return p;
}

}  // namespace

size_t delta_bwd_workspace_bytes(const ssmvjp_delta_chunk_desc& d) { return bwd_plan(d).bytes; }

hipError_t launch_delta_chunk_bwd(const ssmvjp_delta_chunk_desc& d, const DeltaChunkBwdPointers& p, hipStream_t stream) {
  DeltaChunkArgs a = delta_chunk_args(d, p.seq_offsets);
  const BwdPlan pl = bwd_plan(d);
  char* ws = (char*)p.workspace;
  a.q = (const bf16*)p.q; a.k = (const bf16*)p.k; a.v = (const bf16*)p.v; a.d_o = (const bf16*)p.d_o;
  a.beta = p.beta; a.g = p.g; a.S0 = p.S0; a.dSf = p.dS_final;
  a.dq = (bf16*)p.dq; a.dk = (bf16*)p.dk; a.dv = (bf16*)p.dv; a.dbeta = p.dbeta; a.dg = p.dg; a.dS0 = p.dS0;
  auto b16 = [&](i64 off) { return (bf16*)(ws + off); };
  a.Tf = b16(pl.off_T); a.Tt = b16(pl.off_Tt); a.Pt = b16(pl.off_Pt); a.G = (float*)(ws + pl.off_G);
  a.Sw = b16(pl.off_S); a.dSw = b16(pl.off_dS); a.rw = b16(pl.off_r); a.muw = b16(pl.off_mu);
  if (pl.few) {
    auto f32 = [&](i64 off) { return (float*)(ws + off); };
    a.S32 = f32(pl.off_S32); a.dS32 = f32(pl.off_dS32); a.r32 = f32(pl.off_r32); a.su = f32(pl.off_su);
    a.dot = f32(pl.off_dot);
  }
  if (a.nslots > 0) {
    const hipError_t e = launch_delta_prep(a, true, stream);
    if (e != hipSuccess) return e;
  }
  if (a.K <= 64) launch_walks_grads<64>(a, stream);
  else launch_walks_grads<128>(a, stream);
  return hipGetLastError();
}

}  // namespace ssmvjp
