// delta_walk.cuh -- the walk over a sequence's chunks that carries the state.
//
// Columns of the state are independent, so a wave owns 16 columns of one
// head for a whole sequence, with the state in its accumulators, and nothing is
// exchanged between waves: r, u and the next state come out of the MFMAs in the
// layout that the following MFMA wants.  The waves of a workgroup share the
// chunk's K, Q, V rows and fragments in LDS.  LDS-direct loads bring the next
// chunk's while this one is computed (two buffers): one barrier per chunk, no
// load in the chain that leads from one state to the next.
//
// MODE 0: the forward (o, S_final); 1: for the backward, the state before every
// chunk and r; 2: those in float32 too.
//
// Waves 0 and 1 carry the states of 16 columns each and do nothing that the next
// state does not wait for.  Forward only: waves 2 and 3 follow one chunk behind
// with the readout of the same columns, from the state's fragments and r, which
// they get through LDS.  The last wave sends for the next chunks' data and
// prepares the gates.  One wave that does all of it takes 7,600 cycles a chunk
// at K = 128, 2,000 of them for the readout and 1,100 for issuing the loads.
//
// Bound by the chain from one state to the next: 136 us for b=2 T=4096 HV=32
// K=V=128, 256 workgroups for 256 CUs, 2.1 us or 4,330 cycles a chunk.  The 98
// MFMAs of a state wave issue in 1,570 of them.  By the clock the six stretches
// take K S0 and the residual 943 + 710 cycles (32 MFMAs), T 539 + 394 (18), K^T u
// 891 + 788 (48), the barrier 69: each begins with what the one before it ends
// with (the last MFMAs' results, their split into parts) and with its LDS reads,
// and there is one such wave on a SIMD to fill the time.  The matrix cores are 27 %
// busy over all SIMDs.  MODE 1 takes 155 us there, 85 of them without its stores
// (393 MB, 2.5 TB/s); stored through the L2 it took 193, and loads two chunks ahead
// made it 176 to 181.
#pragma once

#include "delta_chunk.cuh"

namespace ssmvjp {
namespace {

template <int KP, int MODE>
struct WalkLds {  // byte offsets
  static constexpr int K = 0, V = K + 64 * KP * 2, T = V + 4096, ABUF = T + 12 * 1024;  // for waves 0, 1
  static constexpr int Q = 0, BBUF = MODE ? 0 : 64 * KP * 2;  // for the followers
  static constexpr int B = 2 * ABUF, S = B + 2 * BBUF, SBUF = MODE ? 0 : 2 * KP * 64, R = S + 2 * SBUF;  // [2 buffers][2 tiles]
  static constexpr int G = R + (MODE ? 0 : 2 * 2 * 4096), TOTAL = G + 3 * 512;  // gates: [3][e^G, e^{G_63 - G} beta]
};
constexpr int walk_nth(int mode) { return mode ? 192 : 320; }

// ---- values that are not finite ----
// A product over a chunk's tokens multiplies a later token's NaN or infinity by
// the zeros of T and P above the diagonal and so carries it to earlier tokens.
// The state is not harmed by that: a column that meets such a value is lost from
// there on.  Where r comes out with one, the follower forms r and the readout once
// more, with zeros in place of the column's rows from the first such value on, and
// puts NaN there afterwards.  To look for them costs it 16 multiply-adds a chunk, no
// time of the walk; the same look and path in the state wave cost 4 us of 136.

// the first of the column's 64 rows that is not finite (64: none); zeros from there on.  x: rows 16m + 4q ..
__device__ __forceinline__ int drop_from_first_nonfinite(f32x4 (&x)[4], int q) {
  int first = 64;
#pragma unroll
  for (int m = 3; m >= 0; --m)
#pragma unroll
    for (int r = 3; r >= 0; --r)
      if (nonfinite(x[m][r])) first = 16 * m + 4 * q + r;
  first = min(first, __shfl_xor(first, 16, 64));
  first = min(first, __shfl_xor(first, 32, 64));
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (16 * m + 4 * q + r >= first) x[m][r] = 0.0f;
  return first;
}

// r of a chunk from memory and the state's parts before it (So), in the order of the walk's own products: rows before
// the column's first value that is not finite come out as if it were not there.  Columns without one keep theirs.
template <int KP>
__device__ __forceinline__ void causal_residual(const DeltaChunkArgs& a, i64 tok0, int rows, i64 h, i64 hv, i64 cell,
                                                i64 col, const u32x4* So, const float* eG, f32x4 (&r)[4], int lane) {
  constexpr int KS = KP / 32;
  const int c = lane & 15, q = lane >> 4;
  const brsrc rk = row_rsrc(a.k, tok0, rows, a.H, h, a.K);
  const u32x4* Tf = (const u32x4*)(a.Tf + cell * 6 * 2 * 512) + lane;
  f32x4 x[4], y[4];
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    x[m] = y[m] = zero4();
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int kc = 32 * s + 8 * q;
      const Frag8 k = as_frag(bload16(rk, kc < a.K ? (unsigned)(((i64)(16 * m + c) * a.H * a.K + kc) * 2) : BUF_OOB));
      x[m] = mma32(k, as_frag(So[(KS + s) * 64]), x[m]);
      x[m] = mma32(k, as_frag(So[s * 64]), x[m]);
    }
    const f32x4 e = *(const f32x4*)(eG + 16 * m + 4 * q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 16 * m + 4 * q + i;
      x[m][i] = (row < rows ? (float)a.v[((tok0 + row) * a.HV + hv) * a.V + col] : 0.0f) - e[i] * x[m][i];
    }
  }
  const int first = drop_from_first_nonfinite(x, q);
  y[0] = x[0];
  y[1] = x[1];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    Frag8 xh, xl;
    split8(x[2 * s], x[2 * s + 1], xh, xl);
#pragma unroll
    for (int m = 2 * s; m < 4; ++m) {
      const Frag8 th = as_frag(Tf[frag_lo(m, s) * 128]), tl = as_frag(Tf[frag_lo(m, s) * 128 + 64]);
      y[m] = mma32(th, xl, y[m]);
      y[m] = mma32(tl, xh, y[m]);
      y[m] = mma32(th, xh, y[m]);
    }
  }
  y[2] += x[2];
  y[3] += x[3];
  if (first == 64) return;
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) r[m][i] = 16 * m + 4 * q + i >= first ? __builtin_nanf("") : y[m][i];
}

// block `block` of walk_blocks
template <int KP, int MODE>
__device__ __forceinline__ void delta_chunk_walk(const DeltaChunkArgs& a, unsigned block) {
  constexpr int KS = KP / 32, KT = KP / 16;  // 32-steps and 16-tiles of K
  constexpr bool FWD = MODE == 0, X32 = MODE == 2;
  typedef WalkLds<KP, MODE> L;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, q = lane >> 4;
  const int t16 = w & 1;  // this wave's column tile of the two
  const WalkUnit wu = walk_unit(block, (a.V + 31) / 32);
  const i64 unit = wu.unit, slice = wu.slice;
  if (unit >= a.seq.nseq * a.HV) return;
  const i64 n = unit / a.HV, hv = unit % a.HV, h = hv / a.rep;
  const DeltaSpan sp = a.seq.span(n);
  const int nch = (int)((sp.len + DCH - 1) / DCH);
  const i64 v0 = slice * 32 + t16 * 16, vt = slice * 2 + t16;
  const bool act = v0 < a.V;  // V is a multiple of 16: all of a wave's columns or none
  const i64 cell0 = sp.slot0 * a.HV + hv;  // chunk ch: cell0 + ch * HV
  auto gates = [&](int ch) { return (float*)(smem_raw + L::G + ch % 3 * 512); };
  auto at4 = [&](const float* p, int m) { return *(const f32x4*)(p + 16 * m + 4 * q); };

  if (w < 2) {
    // ---------------------------------------------------------------- the state
    __builtin_amdgcn_s_setprio(3);  // what every other wave waits for goes first
    f32x4 S[KT];
    Frag8 sh[KS], sl[KS];  // its two parts
    const brsrc rs = state_rsrc(a.S0, a, unit, act);
#pragma unroll
    for (int t = 0; t < KT; ++t) S[t] = load_state4(rs, a, t, q, v0 + c);
#pragma unroll
    for (int s = 0; s < KS; ++s) split8(S[2 * s], S[2 * s + 1], sh[s], sl[s]);
    __syncthreads();
    for (int ch = 0; ch < nch; ++ch) {
      const int bf = ch & 1;
      if (act) {
        const unsigned char* const buf = smem_raw + bf * L::ABUF;
        const bf16 *Kt = (const bf16*)(buf + L::K), *Vt = (const bf16*)(buf + L::V);
        const u32x4* Tf = (const u32x4*)(buf + L::T) + lane;
        // the state's parts and r: to the follower, or to memory
        const i64 tile = (cell0 + ch * a.HV) * a.nvt + vt;
        u32x4* So = (u32x4*)(smem_raw + L::S + bf * L::SBUF + t16 * (L::SBUF / 2)) + lane;
        u32x4* Sw = (u32x4*)(a.Sw + tile * 2 * KS * 512) + state_slot(lane);
        f32x4* Ro = (f32x4*)(smem_raw + L::R + (bf * 2 + t16) * 4096) + lane;
        s16x4* Rw = (s16x4*)(a.rw + tile * 4 * 512) + row_slot(lane);
        const float *eG = gates(ch), *wB = eG + 64;
        if constexpr (X32) store_state32(a.S32 + (cell0 + ch * a.HV) * a.K * a.V, S, a.K, a.V, q, v0 + c);
        // Six stretches of MFMAs, each with the vector and LDS work of its neighbours between them: a 16x16x32
        // MFMA holds the matrix pipe for 16 cycles, in which three vector instructions issue.
        // 1: K S0, row tiles 0 and 1, both parts of S0; the state's decay
        f32x4 x[4], e[4], wb[4];
        s16x4 v[4];
        Frag8 kf[2][KS];
#pragma unroll
        for (int s = 0; s < KS; ++s) kf[0][s] = row_frag(Kt, KP, 0, s, lane), kf[1][s] = row_frag(Kt, KP, 1, s, lane);
        const float eEnd = eG[63];
        SSMVJP_FENCE();
#pragma unroll
        for (int m = 0; m < 4; ++m) x[m] = zero4();
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          x[0] = mma32(kf[0][s], sl[s], x[0]);
          x[1] = mma32(kf[1][s], sl[s], x[1]);
          x[0] = mma32(kf[0][s], sh[s], x[0]);
          x[1] = mma32(kf[1][s], sh[s], x[1]);
        }
        Frag8 kg[2][KS];
#pragma unroll
        for (int s = 0; s < KS; ++s) kg[0][s] = row_frag(Kt, KP, 2, s, lane), kg[1][s] = row_frag(Kt, KP, 3, s, lane);
#pragma unroll
        for (int m = 0; m < 4; ++m) v[m] = col4(Vt, 32, m, t16, lane), e[m] = at4(eG, m);
#pragma unroll
        for (int t = 0; t < KT; ++t) S[t] *= eEnd;
        pipe<4 * KS, 2, 1>();
        SSMVJP_FENCE();
        // 2: K S0, row tiles 2 and 3; V - e^G K S0 of tiles 0 and 1; the state's parts to the follower
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          x[2] = mma32(kg[0][s], sl[s], x[2]);
          x[3] = mma32(kg[1][s], sl[s], x[3]);
          x[2] = mma32(kg[0][s], sh[s], x[2]);
          x[3] = mma32(kg[1][s], sh[s], x[3]);
        }
        Frag8 xh[2], xl[2], th[6], tl[6];
        auto residual = [&](int s) {
#pragma unroll
          for (int m = 2 * s; m < 2 * s + 2; ++m) {
            x[m] = unpack4(v[m]) - e[m] * x[m];
          }
          split8(x[2 * s], x[2 * s + 1], xh[s], xl[s]);
        };
        residual(0);
#pragma unroll
        for (int i = 0; i < 6; ++i) th[i] = as_frag(Tf[i * 128]), tl[i] = as_frag(Tf[i * 128 + 64]);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          if constexpr (FWD) {
            So[s * 64] = as_u4(sh[s]);
            So[(KS + s) * 64] = as_u4(sl[s]);
          } else {
            stream_store(Sw + s * 64, as_u4(sh[s]));
            stream_store(Sw + (KS + s) * 64, as_u4(sl[s]));
          }
        }
        pipe<4 * KS, 3, 1>();
        SSMVJP_FENCE();
        // 3: r = T (V - e^G K S0), contraction over tiles 0 and 1; the other residual
#pragma unroll
        for (int m = 0; m < 4; ++m) x[m] = m < 2 ? mma32(th[frag_lo(m, 0)], xl[0], x[m]) : x[m];
        f32x4 y[2];  // tiles 2 and 3 get this part later: their own residual is still to be formed
        y[0] = mma32(th[frag_lo(2, 0)], xl[0], zero4());
        y[1] = mma32(th[frag_lo(3, 0)], xl[0], zero4());
#pragma unroll
        for (int m = 0; m < 2; ++m) x[m] = mma32(tl[frag_lo(m, 0)], xh[0], x[m]);
        y[0] = mma32(tl[frag_lo(2, 0)], xh[0], y[0]);
        y[1] = mma32(tl[frag_lo(3, 0)], xh[0], y[1]);
#pragma unroll
        for (int m = 0; m < 2; ++m) x[m] = mma32(th[frag_lo(m, 0)], xh[0], x[m]);
        y[0] = mma32(th[frag_lo(2, 0)], xh[0], y[0]);
        y[1] = mma32(th[frag_lo(3, 0)], xh[0], y[1]);
        residual(1);
        Frag8 ct[2][KT];
#pragma unroll
        for (int t = 0; t < KT; ++t) ct[0][t] = key_frag(Kt, KP, t, 0, lane);
#pragma unroll
        for (int m = 0; m < 4; ++m) wb[m] = at4(wB, m);
        pipe<12, 4, 2>();
        SSMVJP_FENCE();
        // 4: contraction over tiles 2 and 3; u = e^{G_63 - G} beta r of tiles 0 and 1, in three parts
        y[0] = mma32(th[frag_lo(2, 1)], xl[1], y[0]);
        y[1] = mma32(th[frag_lo(3, 1)], xl[1], y[1]);
        y[0] = mma32(tl[frag_lo(2, 1)], xh[1], y[0]);
        y[1] = mma32(tl[frag_lo(3, 1)], xh[1], y[1]);
        y[0] = mma32(th[frag_lo(2, 1)], xh[1], y[0]);
        y[1] = mma32(th[frag_lo(3, 1)], xh[1], y[1]);
        Frag8 uh[2], um[2], ul[2];
        split8x3(x[0] * wb[0], x[1] * wb[1], uh[0], um[0], ul[0]);
        auto keep = [&](int s) {
          if constexpr (FWD) {
            Ro[2 * s * 64] = x[2 * s];
            Ro[(2 * s + 1) * 64] = x[2 * s + 1];
          } else {
            if constexpr (X32) {
              float* p = a.r32 + ((cell0 + ch * a.HV) * 64 + 32 * s + 4 * q) * a.V + v0 + c;
#pragma unroll
              for (int i = 0; i < 8; ++i) p[(16 * (i >> 2) + (i & 3)) * a.V] = x[2 * s + (i >> 2)][i & 3];
            }
            Frag8 rh, rl;
            split8(x[2 * s], x[2 * s + 1], rh, rl);
            stream_store(Rw + 2 * s * 64, rh.a);
            stream_store(Rw + (2 * s + 1) * 64, rh.b);
            stream_store(Rw + 256 + 2 * s * 64, rl.a);
            stream_store(Rw + 256 + (2 * s + 1) * 64, rl.b);
          }
        };
        keep(0);
        pipe<6, 8, 0>();
        SSMVJP_FENCE();
        // 5: S = e^{G_63} S0 + K^T u, tokens of tiles 0 and 1; u of tiles 2 and 3
#pragma unroll
        for (int t = 0; t < KT; ++t) S[t] = mma32(ct[0][t], ul[0], S[t]);
#pragma unroll
        for (int t = 0; t < KT; ++t) S[t] = mma32(ct[0][t], um[0], S[t]);
#pragma unroll
        for (int t = 0; t < KT; ++t) S[t] = mma32(ct[0][t], uh[0], S[t]);
        x[2] += y[0];
        x[3] += y[1];
        split8x3(x[2] * wb[2], x[3] * wb[3], uh[1], um[1], ul[1]);
        keep(1);
#pragma unroll
        for (int t = 0; t < KT; ++t) ct[1][t] = key_frag(Kt, KP, t, 1, lane);
        pipe<3 * KT, 3, 1>();
        SSMVJP_FENCE();
        // 6: tokens of tiles 2 and 3, two state tiles at a time; the parts of those that are done
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          S[2 * s] = mma32(ct[1][2 * s], ul[1], S[2 * s]);
          S[2 * s + 1] = mma32(ct[1][2 * s + 1], ul[1], S[2 * s + 1]);
          S[2 * s] = mma32(ct[1][2 * s], um[1], S[2 * s]);
          S[2 * s + 1] = mma32(ct[1][2 * s + 1], um[1], S[2 * s + 1]);
          S[2 * s] = mma32(ct[1][2 * s], uh[1], S[2 * s]);
          S[2 * s + 1] = mma32(ct[1][2 * s + 1], uh[1], S[2 * s + 1]);
          if (s > 0) {
            split8(S[2 * s - 2], S[2 * s - 1], sh[s - 1], sl[s - 1]);
            pipe<6, 4, 0>();
          }
          SSMVJP_FENCE();
        }
        split8(S[KT - 2], S[KT - 1], sh[KS - 1], sl[KS - 1]);
      }
      __syncthreads();
    }
    if constexpr (FWD) __syncthreads();  // the period in which the followers finish the last chunk
    if (FWD && a.Sf && act) {
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int k = state_row(t, q) + r;
          if (k < a.K) a.Sf[(unit * a.K + k) * a.V + v0 + c] = S[t][r];
        }
    }
  } else if (FWD && w < 4) {
    // ------------------------------------------------------------ the followers
    // P comes straight from memory, a period ahead: both parts would not fit into LDS beside the rest
    u32x4 pf[12];
    auto fetch_p = [&](int ch) {
      const u32x4* f = (const u32x4*)(a.Pf + (cell0 + ch * a.HV) * 6 * 2 * 512) + lane;
#pragma unroll
      for (int i = 0; i < 12; ++i) pf[i] = f[i * 64];
    };
    if (nch > 0) fetch_p(0);
    __syncthreads();
    for (int p = 0; p <= nch; ++p) {  // chunk p - 1 here, chunk p at the states
      if (act && p > 0) {
        const int ch = p - 1, bf = ch & 1;
        const unsigned char* const buf = smem_raw + L::B + bf * L::BBUF;
        const bf16* Qt = (const bf16*)(buf + L::Q);
        const u32x4* So = (const u32x4*)(smem_raw + L::S + bf * L::SBUF + t16 * (L::SBUF / 2)) + lane;
        const f32x4* Ro = (const f32x4*)(smem_raw + L::R + (bf * 2 + t16) * 4096) + lane;
        const float* eG = gates(ch);
        // (Q S0)^T, both parts of S0
        u32x4 h4[KS], l4[KS];
        Frag8 qf[KS][4];
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          h4[s] = So[s * 64];
          l4[s] = So[(KS + s) * 64];
#pragma unroll
          for (int m = 0; m < 4; ++m) qf[s][m] = row_frag(Qt, KP, m, s, lane);
        }
        SSMVJP_FENCE();
        f32x4 y[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) y[m] = zero4();
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const Frag8 hi = as_frag(h4[s]), lo = as_frag(l4[s]);
#pragma unroll
          for (int m = 0; m < 4; ++m) y[m] = mma32(lo, qf[s][m], y[m]);
#pragma unroll
          for (int m = 0; m < 4; ++m) y[m] = mma32(hi, qf[s][m], y[m]);
        }
        Frag8 rh[2], rl[2];
        f32x4 r[4], rz = zero4();
#pragma unroll
        for (int m = 0; m < 4; ++m) r[m] = Ro[m * 64], rz += 0.0f * r[m];
        const bool bad = __any(!(rz[0] + rz[1] + rz[2] + rz[3] == 0.0f));  // see above
        int first = 64;
        if (__builtin_expect(bad, 0)) {
          const i64 left = sp.len - (i64)ch * DCH;
          causal_residual<KP>(a, sp.start + (i64)ch * DCH, (int)(left < DCH ? left : DCH), h, hv, cell0 + ch * a.HV, v0 + c,
                              So, eG, r, lane);
          first = drop_from_first_nonfinite(r, q);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) split8(r[2 * s], r[2 * s + 1], rh[s], rl[s]);
        // O^T = scale e^G (Q S0)^T + r^T (scale P beta)^T
        float e[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) e[m] = a.scale * eG[16 * m + c];
        SSMVJP_FENCE();
#pragma unroll
        for (int m = 0; m < 4; ++m) y[m] *= e[m];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
          for (int m = 2 * s; m < 4; ++m) y[m] = mma32(rl[s], as_frag(pf[2 * frag_lo(m, s)]), y[m]);
#pragma unroll
          for (int m = 2 * s; m < 4; ++m) y[m] = mma32(rh[s], as_frag(pf[2 * frag_lo(m, s) + 1]), y[m]);
#pragma unroll
          for (int m = 2 * s; m < 4; ++m) y[m] = mma32(rh[s], as_frag(pf[2 * frag_lo(m, s)]), y[m]);
        }
        if (__builtin_expect(bad, 0)) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int from = __shfl(first, 4 * q + j, 64);
#pragma unroll
            for (int m = 0; m < 4; ++m)
              if (16 * m + c >= from) y[m][j] = __builtin_nanf("");
          }
        }
        if (p < nch) fetch_p(p);
        const i64 row0 = (i64)ch * DCH + c;
        bf16* o = a.o + ((sp.start + row0) * a.HV + hv) * a.V + v0 + 4 * q;
#pragma unroll
        for (int m = 0; m < 4; ++m)
          if (row0 + 16 * m < sp.len) *(s16x4*)(o + 16 * m * a.HV * a.V) = pack4(y[m]);
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
    auto issue_a = [&](int ch) {  // k, v and T of chunk ch
      const unsigned b = lds0 + (unsigned)((ch & 1) * L::ABUF);
      const i64 tok0 = sp.start + (i64)ch * DCH;
      rows_dma.issue(b + L::K, 0, row_words(a.k, tok0, rows_of(ch), a.H, h, a.K, 0));
      cols_dma.issue(b + L::V, 0, row_words(a.v, tok0, rows_of(ch), a.HV, hv, a.V, slice * 32));
      flat_dma<12, 1>(b + L::T, 0, lane, rsrc_words_u(a.Tf + (cell0 + ch * a.HV) * 6 * 2 * 512, 12 * 1024));
    };
    auto issue_b = [&](int ch) {  // q
      const unsigned b = lds0 + (unsigned)(L::B + (ch & 1) * L::BBUF);
      const i64 tok0 = sp.start + (i64)ch * DCH;
      rows_dma.issue(b + L::Q, 0, row_words(a.q, tok0, rows_of(ch), a.H, h, a.K, 0));
    };
    float sG = 0.0f, sB = 0.0f;
    auto fetch_gates = [&](int ch) {
      sG = a.G[(cell0 + ch * a.HV) * 64 + lane];
      const i64 t = (i64)ch * DCH + lane;
      sB = t < sp.len ? a.beta[(sp.start + t) * a.HV + hv] : 0.0f;
    };
    auto commit_gates = [&](int ch) {
      float* g = gates(ch);
      const float end = __shfl(sG, 63, 64);
      g[lane] = exp_hw(sG);
      g[64 + lane] = exp_hw(end - sG) * sB;
    };
    if (nch > 0) {
      fetch_gates(0);
      issue_a(0);
      commit_gates(0);
    }
    dma_wait();
    __syncthreads();
    for (int p = 0; p < nch + (FWD ? 1 : 0); ++p) {
      const bool more = p + 1 < nch;
      if (more) {
        fetch_gates(p + 1);
        issue_a(p + 1);
      }
      if (FWD && p < nch) issue_b(p);
      if (more) commit_gates(p + 1);
      dma_wait();
      __syncthreads();
    }
  }
}

}  // namespace
}  // namespace ssmvjp
