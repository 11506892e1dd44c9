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
//     dG_i = scale e^G_i dO_i . (Q S0)_i - e^G_i mu_i . (K S0)_i - su_i + sum_j M_ij - sum_j M_ji
//     su_i = e^{G_63 - G_i} beta_i r_i . (K dS)_i
//     dg_t = sum_{i >= t} dG_i + sum_i su_i + e^{G_63} <S0, dS>
// In the sum over i >= t the pairs with both tokens behind t cancel between the
// row and the column sums, exactly, since both add the same float32 M_ij; that
// is why r, mu and the states enter M and the row terms with both bf16 parts,
// and dg comes out at about 6e-6.  dq and dk are bf16: one part is enough.
//
// Four launches: delta_prep_kernel (T, T^T, scale P^T of every chunk),
// delta_chunk_walk_kernel<., 1> (the state before every chunk, r),
// delta_chunk_rev_kernel (the reverse walk, 16 columns per wave as the forward:
// mu, dS, row sums over its columns) and delta_chunk_grads_kernel (all chunks at
// once: dv, dq, dk summed over the value heads of a qk head, dg, dbeta).
#include "delta_chunk.cuh"

namespace ssmvjp {
namespace {

// ---------------------------------------------------------------------------
// reverse walk
// ---------------------------------------------------------------------------
// The chunk's q, k, d_o rows and the fragments of T^T and P^T come as in the
// forward walk, by LDS-direct loads into the other of two buffers while a chunk
// is computed.  What belongs to one wave's columns (S0, e^G K S0, r) has one
// buffer per wave: it is read early in a chunk, and the wave then sends for the
// next chunk's.
template <int KP, int NW>
struct RevLds {
  static constexpr int KS = KP / 32;
  static constexpr int K = 0, Q = K + 64 * KP * 2, O = Q + 64 * KP * 2, T = O + 2048 * NW, P = T + 12 * 1024,
                       BUF = P + 12 * 1024;
  static constexpr int S = 2 * BUF, X = 2 * KS * 1024, R = X + 4096, OWN = R + 4096;  // per wave: X, R inside it
  static constexpr int G = S + NW * OWN, TOTAL = G + 6 * 256;
};

template <int KP, int NW>
__global__ void __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(2, 2))) delta_chunk_rev_kernel(DeltaChunkArgs a) {
  constexpr int KS = KP / 32, KT = KP / 16, VPITCH = 16 * NW;
  typedef RevLds<KP, NW> L;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  float* const gates = (float*)(smem_raw + L::G);  // [2][e^G, e^{G_63 - G}, beta][64]
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, q = lane >> 4;
  i64 unit, slice;
  if (!walk_unit(a.seq.nseq * a.HV, (a.V + VPITCH - 1) / VPITCH, unit, slice)) return;
  const i64 n = unit / a.HV, hv = unit % a.HV, h = hv / a.rep;
  const DeltaSpan sp = a.seq.span(n);
  const i64 nch = (sp.len + DCH - 1) / DCH;
  const i64 v0 = slice * VPITCH + w * 16, vt = slice * NW + w;
  const bool act = v0 < a.V;

  const unsigned lds0 = lds_base(smem_raw);
  RowDma<KP, NW> rows_dma;
  ColDma<NW, NW> cols_dma;
  rows_dma.init(w, lane, a.H * a.K, a.K);
  cols_dma.init(w, lane, a.HV * a.V, slice * VPITCH, a.V);
  auto issue = [&](i64 ch, int bf) {
    const i64 tok0 = sp.start + ch * DCH;
    const int rows = (int)(sp.len - ch * DCH < DCH ? sp.len - ch * DCH : DCH);
    const unsigned b = lds0 + (unsigned)(bf * L::BUF);
    const i64 cu = (sp.slot0 + ch) * a.HV + hv;
    rows_dma.issue(b + L::K, w, row_words(a.k, tok0, rows, a.H, h, a.K, 0));
    rows_dma.issue(b + L::Q, w, row_words(a.q, tok0, rows, a.H, h, a.K, 0));
    cols_dma.issue(b + L::O, w, row_words(a.d_o, tok0, rows, a.HV, hv, a.V, slice * VPITCH));
    flat_dma<12, NW>(b + L::T, w, lane, rsrc_words_u(a.Tt + cu * 6 * 2 * 512, 12 * 1024));
    flat_dma<12, NW>(b + L::P, w, lane, rsrc_words_u(a.Pt + cu * 6 * 2 * 512, 12 * 1024));
  };
  const unsigned own = (unsigned)(L::S + w * L::OWN);
  auto issue_own = [&](i64 ch) {
    const i64 tile = ((sp.slot0 + ch) * a.HV + hv) * a.nvt + vt;
    flat_dma<2 * KS, 1>(lds0 + own, 0, lane, rsrc_words_u(a.Sw + tile * 2 * KS * 512, 2 * KS * 1024));
    flat_dma<4, 1>(lds0 + own + L::X, 0, lane, rsrc_words_u(a.Xw + tile * 1024, 4096));
    flat_dma<4, 1>(lds0 + own + L::R, 0, lane, rsrc_words_u(a.rw + tile * 4 * 512, 4096));
  };
  float sG = 0.0f, sB = 0.0f;
  auto fetch_gates = [&](i64 ch) {
    const i64 tok0 = sp.start + ch * DCH;
    sG = a.G[((sp.slot0 + ch) * a.HV + hv) * 64 + lane];
    sB = ch * DCH + lane < sp.len ? a.beta[(tok0 + lane) * a.HV + hv] : 0.0f;
  };
  auto commit_gates = [&](int bf) {
    const float end = __shfl(sG, 63, 64);
    float* g = gates + bf * 192 + lane;
    g[0] = exp_hw(sG);
    g[64] = exp_hw(end - sG);
    g[128] = sB;
  };

  f32x4 dS[KT];
  const brsrc rs = state_rsrc(a.dSf, a, unit, act);
#pragma unroll
  for (int t = 0; t < KT; ++t) dS[t] = load_state4(rs, a, t, q, v0 + c);
  if (nch > 0) {
    const int bf = (nch - 1) & 1;
    if (w == 0) fetch_gates(nch - 1);
    issue(nch - 1, bf);
    if (act) issue_own(nch - 1);
    if (w == 0) commit_gates(bf);
  }
  dma_wait();
  __syncthreads();
  for (i64 ch = nch - 1; ch >= 0; --ch) {
    const int bf = ch & 1;
    const i64 tile = ((sp.slot0 + ch) * a.HV + hv) * a.nvt + vt;
    if (ch > 0) {
      if (w == 0) fetch_gates(ch - 1);
      issue(ch - 1, bf ^ 1);
    }
    if (act) {
      const unsigned char* const buf = smem_raw + bf * L::BUF;
      const bf16 *Kt = (const bf16*)(buf + L::K), *Qt = (const bf16*)(buf + L::Q), *Ot = (const bf16*)(buf + L::O);
      const u32x4 *Tt = (const u32x4*)(buf + L::T) + lane, *Pt = (const u32x4*)(buf + L::P) + lane;
      const u32x4 *So = (const u32x4*)(smem_raw + own) + lane, *Ro = (const u32x4*)(smem_raw + own + L::R) + lane;
      const f32x4* Xo = (const f32x4*)(smem_raw + own + L::X) + lane;
      const float *eG = gates + bf * 192, *eE = eG + 64, *be = eG + 128;
      auto at4 = [&](const float* p, int m) { return *(const f32x4*)(p + 16 * m + 4 * q); };
      // K dS (both parts of dS) and <S0, dS>
      f32x4 z[4], x[4], r[4];
      f32x4 dot = zero4();
#pragma unroll
      for (int m = 0; m < 4; ++m) z[m] = zero4();
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const Frag8 sh = as_frag(So[s * 64]), sl = as_frag(So[(KS + s) * 64]);
        Frag8 dh, dl;
        split8(dS[2 * s], dS[2 * s + 1], dh, dl);
        *((u32x4*)(a.dSw + tile * KS * 512) + s * 64 + lane) = as_u4(dh);
        dot += (unpack4(sh.a) + unpack4(sl.a)) * dS[2 * s];
        dot += (unpack4(sh.b) + unpack4(sl.b)) * dS[2 * s + 1];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const Frag8 kf = row_frag(Kt, KP, m, s, lane);
          z[m] = mma32(kf, dl, z[m]);
          z[m] = mma32(kf, dh, z[m]);
        }
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const Frag8 rh = as_frag(Ro[s * 64]), rl = as_frag(Ro[(2 + s) * 64]);
        r[2 * s] = unpack4(rh.a) + unpack4(rl.a);
        r[2 * s + 1] = unpack4(rh.b) + unpack4(rl.b);
        x[2 * s] = Xo[2 * s * 64];
        x[2 * s + 1] = Xo[(2 * s + 1) * 64];
      }
      if (ch > 0) {
        lds_wait();  // what this wave had of its own is in registers
        issue_own(ch - 1);
      }
      // dU = scale P^T dO + e^{G_63 - G} K dS
      Frag8 of[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) of[s] = {col4(Ot, VPITCH, 2 * s, w, lane), col4(Ot, VPITCH, 2 * s + 1, w, lane)};
      f32x4 du[4], mu[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        z[m] *= at4(eE, m);
        du[m] = z[m];
#pragma unroll
        for (int s = m / 2; s < 2; ++s) {
          du[m] = mma32(as_frag(Pt[frag_up(m, s) * 128 + 64]), of[s], du[m]);
          du[m] = mma32(as_frag(Pt[frag_up(m, s) * 128]), of[s], du[m]);
        }
      }
      // mu = T^T (beta dU)
      {
        Frag8 bh[2], bl[2];
#pragma unroll
        for (int m = 0; m < 4; ++m) mu[m] = at4(be, m) * du[m];
#pragma unroll
        for (int s = 0; s < 2; ++s) split8(mu[2 * s], mu[2 * s + 1], bh[s], bl[s]);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
#pragma unroll
          for (int s = m / 2; s < 2; ++s) {
            const Frag8 th = as_frag(Tt[frag_up(m, s) * 128]), tl = as_frag(Tt[frag_up(m, s) * 128 + 64]);
            mu[m] = mma32(th, bl[s], mu[m]);
            mu[m] = mma32(tl, bh[s], mu[m]);
            mu[m] = mma32(th, bh[s], mu[m]);
          }
        }
      }
      u32x4* mo = (u32x4*)(a.muw + tile * 4 * 512) + lane;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Frag8 hi, lo;
        split8(mu[2 * s], mu[2 * s + 1], hi, lo);
        mo[s * 64] = as_u4(hi);
        mo[128 + s * 64] = as_u4(lo);
      }
      // row terms, summed over this wave's 16 columns; the operands of the state's update
      const float eEnd = eG[63];
      float tail = eEnd * ((dot[0] + dot[1]) + (dot[2] + dot[3]));
      float* rp = a.rowp + tile * 3 * 64 + 64;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const f32x4 eg = at4(eG, m);
        const f32x4 o = unpack4(m & 1 ? of[m / 2].b : of[m / 2].a);
        const f32x4 su = at4(be, m) * r[m] * z[m];
        f32x4 t = -mu[m] * x[m] - su, d = r[m] * du[m];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          tail += su[j];
          t[j] = sum16(t[j]);
          d[j] = sum16(d[j]);
        }
        if (c == 0) {
          *(f32x4*)(rp + 16 * m + 4 * q) = t;
          *(f32x4*)(rp + 64 + 16 * m + 4 * q) = d;
        }
        mu[m] *= -eg;
        x[m] = a.scale * eg * o;
      }
      tail = wave_sum(tail);
      if (lane == 0) a.endp[tile] = tail;
      // dS0 = e^{G_63} dS + Q^T (scale e^G dO) - K^T (e^G mu)
      Frag8 mh[2], ml[2], oh[2], ol[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        split8(mu[2 * s], mu[2 * s + 1], mh[s], ml[s]);
        split8(x[2 * s], x[2 * s + 1], oh[s], ol[s]);
      }
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        dS[t] *= eEnd;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const Frag8 kf = key_frag(Kt, KP, t, s, lane), qf = key_frag(Qt, KP, t, s, lane);
          dS[t] = mma32(kf, ml[s], dS[t]);
          dS[t] = mma32(qf, ol[s], dS[t]);
          dS[t] = mma32(kf, mh[s], dS[t]);
          dS[t] = mma32(qf, oh[s], dS[t]);
        }
      }
    }
    if (ch > 0 && w == 0) commit_gates(bf ^ 1);
    dma_wait();
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
}

// ---------------------------------------------------------------------------
// gradients of one chunk of one qk head
// ---------------------------------------------------------------------------
// Eight waves: wave (wr = w % 4, half = w / 4) owns row tile wr of every 64-row
// result and one half of the key columns; of the pair terms, half 0 forms dD
// and half 1 E.  The columns of V go by 32 (one contraction step): r, mu (two
// parts), S0, dS (one part) of the slice are brought to LDS as [v][row] tiles,
// whose transposed reads are the operands with the contraction over v.
constexpr int GRADS_NTH = 512;

// Row pitches of the tiles: 40 bytes past a multiple of 128.  The 16 rows of a
// fragment read meet 16 different pairs of banks, the 4 rows of a transposed
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
__global__ void __launch_bounds__(GRADS_NTH, 2) delta_chunk_grads_kernel(DeltaChunkArgs a) {
  constexpr int KS = KP / 32, KT = KP / 16, PK = KP + 20, HT = KT / 2;  // HT: key tiles of a wave
  constexpr int NP = 4 * KS * 64 / GRADS_NTH;             // 16-byte pieces per thread of a slice of S0 and dS
  __shared__ __attribute__((aligned(16))) bf16 Kb[64 * PK], Qb[64 * PK];
  // the slice's tiles; behind the slices the same memory holds dD^T and E^T, two parts each
  __shared__ __attribute__((aligned(16))) bf16 buf[16 * P64 * 16];
  __shared__ __attribute__((aligned(16))) float Gs[64], Bs[64], rowM[2][64], colM[2][4][64], colA[4][64];
  __shared__ float rowG[8][64], rowB[8][64], tails[8];  // the reverse walk's row sums, by wave
  typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
  bf16 *rH = buf, *mH = buf + 2 * 32 * P64;  // each followed by its lo part
  bf16* sT = buf + 4 * 32 * P64;             // [S0, dS][32][KP]
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, q = lane >> 4;
  const int wr = w & 3, half = w >> 2;
  const unsigned H32 = (unsigned)a.H;
  const i64 h = blockIdx.x % H32, slot = blockIdx.x / H32;
  const ChunkAt at = chunk_at(a.seq, slot, lane);
  if (at.rows == 0) return;
  {
    constexpr int N = 64 * KP / 8 / GRADS_NTH;
    const brsrc rk = row_rsrc(a.k, at.tok0, at.rows, a.H, h, a.K), rq = row_rsrc(a.q, at.tok0, at.rows, a.H, h, a.K);
    u32x4 tk[N], tq[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int p = tid + GRADS_NTH * i, row = p / (KP / 8), col = p % (KP / 8) * 8;
      const unsigned o = col < a.K ? (unsigned)(((i64)row * a.H * a.K + col) * 2) : BUF_OOB;
      tk[i] = bload16(rk, o);
      tq[i] = bload16(rq, o);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int p = tid + GRADS_NTH * i;
      pstore(Kb, PK, p / (KP / 8), p % (KP / 8) * 8, tk[i]);
      pstore(Qb, PK, p / (KP / 8), p % (KP / 8) * 8, tq[i]);
    }
  }
  f32x4 dq[HT], dk[HT];  // rows i = 16 wr + 4 q + r, column 16 (HT half + t) + c
#pragma unroll
  for (int t = 0; t < HT; ++t) dq[t] = zero4(), dk[t] = zero4();

  const int nsl = (int)(a.nvt + 1) / 2;
  for (i64 rr = 0; rr < a.rep; ++rr) {
    const i64 hv = h * a.rep + rr, cu = slot * a.HV + hv;
    u32x4 pr[2], ps[NP];
    u32x2 po[2];
    const brsrc ro = row_rsrc(a.d_o, at.tok0, at.rows, a.HV, hv, a.V);
    // tiles past V lie past the resources: zeros, without a branch
    const brsrc rm4 = make_rsrc((w < 4 ? a.rw : a.muw) + cu * a.nvt * 2048, (unsigned)(a.nvt * 4096));
    const brsrc rS = make_rsrc(a.Sw + cu * a.nvt * KS * 1024, (unsigned)(a.nvt * KS * 2048));
    const brsrc rD = make_rsrc(a.dSw + cu * a.nvt * KS * 512, (unsigned)(a.nvt * KS * 1024));
    auto fetch = [&](int sl) {
      {  // waves 0 .. 3: r, the others mu; hi and lo of one fragment
        const unsigned o = (unsigned)(((sl * 2 + (w >> 1 & 1)) * 256 + (w & 1) * 64 + lane) * 16);
        pr[0] = bload16(rm4, o);
        pr[1] = bload16(rm4, o + 2048u);
      }
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int p = w + GRADS_NTH / 64 * i, t = sl * 2 + p / KS % 2, st = p % KS;
        if (p < 2 * KS) ps[i] = bload16(rS, (unsigned)(((t * 2 * KS + st) * 64 + lane) * 16));
        else ps[i] = bload16(rD, (unsigned)(((t * KS + st) * 64 + lane) * 16));
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = sl * 32 + 16 * e + 4 * q;
        po[e] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(
            ro, col < a.V ? (int)(((16 * wr + c) * a.HV * a.V + col) * 2) : (int)BUF_OOB, 0, 0));
      }
    };
    auto put = [&](bf16* t, int row, int s, const u32x4& u) {  // a fragment's two 4-element runs
      *(u32x2*)(t + row * P64 + 32 * s + 4 * q) = u32x2{u[0], u[1]};
      *(u32x2*)(t + row * P64 + 32 * s + 16 + 4 * q) = u32x2{u[2], u[3]};
    };
    fetch(0);
    // this wave's share of the walks' row sums (tiles w, w + 8, ..) and, for wave 0, the gates
    float dG = 0.0f, db = 0.0f, tail = 0.0f, G0 = 0.0f, b0 = 0.0f;
    for (int t = w; t < (int)a.nvt; t += 8) {
      const float* rp = a.rowp + (cu * a.nvt + t) * 192 + lane;
      dG += rp[0] + rp[64];
      db += rp[128];
      tail += a.endp[cu * a.nvt + t];
    }
    if (w == 0) {
      G0 = a.G[cu * 64 + lane];
      b0 = lane < at.rows ? a.beta[(at.tok0 + lane) * a.HV + hv] : 0.0f;
    }
    __syncthreads();  // the previous head's readers are done; k and q are in LDS
    rowG[w][lane] = dG;
    rowB[w][lane] = db;
    if (lane == 0) tails[w] = tail;
    if (w == 0) {
      Gs[lane] = G0;
      Bs[lane] = b0;
    }
    f32x4 pp[4], x1[HT], y2[HT], y3[HT];  // pp: dO . r (half 0) or mu . r; dO S0^T, mu S0^T, r dS^T
#pragma unroll
    for (int b = 0; b < 4; ++b) pp[b] = zero4();
#pragma unroll
    for (int t = 0; t < HT; ++t) x1[t] = zero4(), y2[t] = zero4(), y3[t] = zero4();
    for (int sl = 0; sl < nsl; ++sl) {
      if (sl) __syncthreads();
      {
        bf16* d = w < 4 ? rH : mH;
        const int row = 16 * (w >> 1 & 1) + c;
        put(d, row, w & 1, pr[0]);
        put(d + 32 * P64, row, w & 1, pr[1]);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int p = w + GRADS_NTH / 64 * i, arr = p / (2 * KS), t2 = p / KS % 2, st = p % KS;
          pstore(sT + arr * 32 * PK, PK, 16 * t2 + c, 32 * st + 8 * q, ps[i]);
        }
      }
      const Frag8 of = {__builtin_bit_cast(s16x4, po[0]), __builtin_bit_cast(s16x4, po[1])};
      __syncthreads();
      if (sl + 1 < nsl) fetch(sl + 1);
      const Frag8 mh = pcol(mH, P64, wr, 0, lane), ml = pcol(mH + 32 * P64, P64, wr, 0, lane);
      const Frag8 rh = pcol(rH, P64, wr, 0, lane), rl = pcol(rH + 32 * P64, P64, wr, 0, lane);
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (b <= wr) {
          const Frag8 bh = pcol(rH, P64, b, 0, lane), bl = pcol(rH + 32 * P64, P64, b, 0, lane);
          if (half == 0) {
            pp[b] = mma32(of, bl, pp[b]);
            pp[b] = mma32(of, bh, pp[b]);
          } else {
            pp[b] = mma32(mh, bl, pp[b]);
            pp[b] = mma32(ml, bh, pp[b]);
            pp[b] = mma32(mh, bh, pp[b]);
          }
        }
#pragma unroll
      for (int t = 0; t < HT; ++t) {
        const Frag8 sf = pcol(sT, PK, HT * half + t, 0, lane), df = pcol(sT + 32 * PK, PK, HT * half + t, 0, lane);
        x1[t] = mma32(of, sf, x1[t]);
        y2[t] = mma32(ml, sf, y2[t]);
        y3[t] = mma32(rl, df, y3[t]);
        y2[t] = mma32(mh, sf, y2[t]);
        y3[t] = mma32(rh, df, y3[t]);
      }
      // dv = mu, rounded: its hi part
      if (half == 1) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = sl * 32 + 16 * e + 4 * q;
          if (16 * wr + c < at.rows && col < a.V)
            *(s16x4*)(a.dv + ((at.tok0 + 16 * wr + c) * a.HV + hv) * a.V + col) = e ? mh.b : mh.a;
        }
      }
    }
    // rows i = 16 wr + 4 q + r
    const f32x4 Gi = *(const f32x4*)(Gs + 16 * wr + 4 * q), Bi = *(const f32x4*)(Bs + 16 * wr + 4 * q);
    const float Ge = Gs[63];
    f32x4 eg, we;
#pragma unroll
    for (int r = 0; r < 4; ++r) eg[r] = exp_hw(Gi[r]), we[r] = exp_hw(Ge - Gi[r]) * Bi[r];
#pragma unroll
    for (int t = 0; t < HT; ++t) {
      dq[t] += a.scale * eg * x1[t];
      dk[t] += we * y3[t] - eg * y2[t];
    }
    __syncthreads();  // the slices' tiles are free
    // pair terms: dD (half 0) or E (half 1); column j = 16 b + c
    f32x4 rm = zero4();
    bf16* const Pt = buf + half * 2 * 64 * P64;  // [hi, lo][64][64], transposed: row j
    Frag8 rf[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) rf[s] = prow(half ? Kb : Qb, PK, wr, s, lane);
    f32x4 kq[4];  // q_i . k_j (half 0) or k_i . k_j
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      kq[b] = zero4();
      if (b <= wr) {
#pragma unroll
        for (int s = 0; s < KS; ++s) kq[b] = mma32(rf[s], prow(Kb, PK, b, s, lane), kq[b]);
      }
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      f32x4 x = zero4();
      float cm = 0.0f, ca = 0.0f;
      const int j = 16 * b + c;
      if (b <= wr) {
        const float Gj = Gs[j], bj = Bs[j] * (half ? -1.0f : a.scale);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = 16 * wr + 4 * q + r;
          const float gam = exp_hw(i >= j ? Gi[r] - Gj : 0.0f);
          if (i > j || (half == 0 && i == j)) x[r] = bj * pp[b][r] * gam;
          if (i > j) {
            const float m = x[r] * kq[b][r];
            rm[r] += m;
            cm += m;
            ca += gam * kq[b][r] * pp[b][r];
          }
        }
      }
      cm = sum4q(cm);
      if (half) ca = sum4q(ca);
      if (q == 0) {
        colM[half][wr][j] = cm;
        if (half) colA[wr][j] = ca;
      }
      s16x4 hi, lo;
      split4(x, hi, lo);
      const int o = j * P64 + 16 * wr + 4 * q;
      *(s16x4*)(Pt + o) = hi;
      *(s16x4*)(Pt + 64 * P64 + o) = lo;
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
        const bf16 *D = buf + e * 64 * P64, *E = buf + (2 + e) * 64 * P64;
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
      float dG = 0.0f, db = 0.0f, tail = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) dG += rowG[i][lane], db += rowB[i][lane], tail += tails[i];
      float col = 0.0f, ca = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) col += colM[0][i][lane] + colM[1][i][lane], ca += colA[i][lane];
      dG += rowM[0][lane] + rowM[1][lane] - col;
      const float sum = wave_incl_suffix(dG, lane) + tail;
      if (lane < at.rows) {
        const i64 o = (at.tok0 + lane) * a.HV + hv;
        a.dg[o] = sum;
        a.dbeta[o] = db - ca;
      }
    }
  }
  // out: row i, 16 columns at a time
#pragma unroll
  for (int t = 0; t < HT; ++t) {
    const int k0 = 16 * (HT * half + t);
    if (k0 < a.K) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * wr + 4 * q + r;
        if (i < at.rows) {
          const i64 o = ((at.tok0 + i) * a.H + h) * a.K + k0 + c;
          a.dq[o] = (bf16)dq[t][r];
          a.dk[o] = (bf16)dk[t][r];
        }
      }
    }
  }
}

template <int KP>
void launch_rev_grads(const DeltaChunkArgs& a, hipStream_t s) {
  const i64 blocks = walk_blocks(a.seq.nseq * a.HV, (a.V + 31) / 32);
  hipLaunchKernelGGL((delta_chunk_rev_kernel<KP, 2>), dim3((unsigned)blocks), dim3(128), (RevLds<KP, 2>::TOTAL), s, a);
  if (a.nslots > 0)
    hipLaunchKernelGGL((delta_chunk_grads_kernel<KP>), dim3((unsigned)(a.nslots * a.H)), dim3(GRADS_NTH), 0, s, a);
}

struct BwdPlan {
  i64 off_T, off_Tt, off_Pt, off_G, off_S, off_dS, off_r, off_X, off_mu, off_row, off_end;
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
  p.off_dS = carve(tiles * KP * 16 * 2);
  p.off_r = carve(tiles * 4 * 1024);
  p.off_X = carve(tiles * 4 * 1024);
  p.off_mu = carve(tiles * 4 * 1024);
  p.off_row = carve(tiles * 3 * 64 * 4);
  p.off_end = carve(tiles * 4);
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
  a.Xw = (float*)(ws + pl.off_X);
  a.rowp = (float*)(ws + pl.off_row); a.endp = (float*)(ws + pl.off_end);
  if (a.nslots > 0) {
    hipError_t e = launch_delta_prep(a, true, stream);
    if (e == hipSuccess) e = launch_delta_states(a, stream);
    if (e != hipSuccess) return e;
  }
  if (a.K <= 64) launch_rev_grads<64>(a, stream);
  else launch_rev_grads<128>(a, stream);
  return hipGetLastError();
}

}  // namespace ssmvjp
