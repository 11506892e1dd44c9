// delta_chunk.hip -- the chunked gated delta rule on MFMA: what each chunk needs
// that does not depend on the state (delta_prep_kernel, all chunks at once) and
// the walk over the chunks that carries the state (delta_chunk_walk_kernel).
// delta_chunk.cuh has the algebra, the number formats and the fragment order.
//
// Prep.  One workgroup per (chunk, qk head), four waves, wave w owning row tile
// w of the 64 x 64 products K K^T and Q K^T (16-byte fragments straight from
// memory: both operands run along the rows).  (I + a diag(beta))^-1 is formed in
// float32: the four 16 x 16 diagonal blocks by forward substitution, one wave
// each, then the blocks below them from the inverses of the halves
// ([A 0; C D]^-1 = [A^-1 0; -D^-1 C A^-1 D^-1], twice) on float32 MFMA.
// Substitution, not powers of a: those cancel when keys repeat.
//
// Walk.  Columns of the state are independent, so a wave owns 16 columns of one
// head for a whole sequence, with the state in its accumulators, and nothing is
// exchanged between waves: r, u and the next state come out of the MFMAs in the
// layout that the following MFMA wants.  Two waves share a workgroup and the
// K, Q, V rows in LDS, double-buffered: one barrier per chunk.
#include "delta_chunk.cuh"

namespace ssmvjp {
namespace {

constexpr int TP = 68;  // row pitch (floats) of the 64 x 64 matrices in LDS: 16-byte rows, 4 banks apart

// ---------------------------------------------------------------------------
// prep
// ---------------------------------------------------------------------------
// D = X Y for 16 x 16 blocks of float32 matrices in LDS; X block (xr, xc), Y block (yr, yc)
__device__ __forceinline__ void mm_block(f32x4& d, const float* X, int xr, int xc, const Frag<float>& y, int lane) {
  mma(d, ld_colk(X, TP, 16 * xr, 16 * xc, lane), y);
}
__device__ __forceinline__ Frag<float> as_b(const f32x4& v) {  // D as the B operand of the next product
  Frag<float> f;
#pragma unroll
  for (int j = 0; j < 4; ++j) f.v[j] = v[j];
  return f;
}

// Ts = (I + As)^-1 for As strictly lower triangular; every thread of the four waves calls it
__device__ __forceinline__ void invert64(const float* As, float* Ts, int w, int lane) {
  const int c = lane & 15, q = lane >> 4;
  {
    float x[16];
    const float* A = As + 16 * w * TP + 16 * w;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == c ? 1.0f : 0.0f;
#pragma unroll
      for (int j = 0; j < i; ++j) s = fmaf(-A[i * TP + j], x[j], s);
      x[i] = s;
    }
    if (q == 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) Ts[(16 * w + i) * TP + 16 * w + c] = x[i];
    }
  }
  __syncthreads();
  if (w < 2) {  // blocks (1,0) and (3,2)
    const int i = 2 * w + 1, j = 2 * w;
    f32x4 x = zero4(), y = zero4();
    mm_block(x, As, i, j, ld_rowk(Ts, TP, 16 * j, 16 * j, lane), lane);
    mm_block(y, Ts, i, i, as_b(x), lane);
#pragma unroll
    for (int r = 0; r < 4; ++r) Ts[(16 * i + 4 * q + r) * TP + 16 * j + c] = -y[r];
  }
  __syncthreads();
  {  // blocks (2..3, 0..1): wave w takes block (2 + w / 2, w % 2)
    const int j = w & 1, i = 2 + (w >> 1);
    f32x4 x2 = zero4(), x3 = zero4(), y = zero4();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k < j) continue;
      const Frag<float> t = ld_rowk(Ts, TP, 16 * k, 16 * j, lane);
      mm_block(x2, As, 2, k, t, lane);
      if (i == 3) mm_block(x3, As, 3, k, t, lane);
    }
    mm_block(y, Ts, i, 2, as_b(x2), lane);
    if (i == 3) mm_block(y, Ts, 3, 3, as_b(x3), lane);
#pragma unroll
    for (int r = 0; r < 4; ++r) Ts[(16 * i + 4 * q + r) * TP + 16 * j + c] = -y[r];
  }
  __syncthreads();
}

template <int KP, bool BWD>
__global__ void __launch_bounds__(256) delta_prep_kernel(DeltaChunkArgs a) {
  constexpr int KS = KP / 32;
  __shared__ float As[64 * TP], Ts[64 * TP];
  __shared__ float Gs[64], Bs[64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, c = lane & 15, q = lane >> 4;
  const i64 h = blockIdx.x % a.H, slot = blockIdx.x / a.H;
  const ChunkAt at = chunk_at(a.seq, slot, lane);
  if (at.rows == 0) return;
  const brsrc rk = row_rsrc(a.k, at.tok0, at.rows, a.H, h, a.K), rq = row_rsrc(a.q, at.tok0, at.rows, a.H, h, a.K);
  auto off = [&](int tile, int s) {
    const int col = 32 * s + 8 * q;
    return col < a.K ? (unsigned)(((i64)(16 * tile + c) * a.H * a.K + col) * 2) : BUF_OOB;
  };
  u32x4 kw[KS], qw[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) kw[s] = bload16(rk, off(w, s)), qw[s] = bload16(rq, off(w, s));
  // lane: row i = 16 w + c, columns j = 16 b + 4 q + r (kt: row j = 16 w + c, columns i)
  f32x4 kk[4], qk[4], kt[BWD ? 4 : 1];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    kk[b] = zero4();
    qk[b] = zero4();
    if (b <= w) {
      u32x4 x[KS];
#pragma unroll
      for (int s = 0; s < KS; ++s) x[s] = bload16(rk, off(b, s));
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        kk[b] = mma32(x[s], kw[s], kk[b]);
        qk[b] = mma32(x[s], qw[s], qk[b]);
      }
    }
    if constexpr (BWD) {
      kt[b] = zero4();
      if (b >= w) {
        u32x4 x[KS];
#pragma unroll
        for (int s = 0; s < KS; ++s) x[s] = bload16(rq, off(b, s));
#pragma unroll
        for (int s = 0; s < KS; ++s) kt[b] = mma32(x[s], kw[s], kt[b]);
      }
    }
  }
  for (i64 rr = 0; rr < a.rep; ++rr) {
    const i64 hv = h * a.rep + rr, unit = slot * a.HV + hv;
    __syncthreads();  // the previous head's readers are done with LDS
    if (w == 0) {
      const i64 at1 = (at.tok0 + lane) * a.HV + hv;
      const bool in = lane < at.rows;
      const float G = wave_incl_scan(in ? gate_clamp(a.g[at1]) : 0.0f, lane);
      Gs[lane] = G;
      Bs[lane] = in ? a.beta[at1] : 0.0f;
      a.G[unit * 64 + lane] = G;
    }
    __syncthreads();
    const int row = 16 * w + c;
    const float Gr = Gs[row];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const f32x4 Gc = *(const f32x4*)(Gs + 16 * b + 4 * q), Bc = *(const f32x4*)(Bs + 16 * b + 4 * q);
      if (b <= w) {
        f32x4 x;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 16 * b + 4 * q + r;
          x[r] = row > j ? kk[b][r] * exp_hw(Gr - Gc[r]) * Bc[r] : 0.0f;
        }
        *(f32x4*)(As + row * TP + 16 * b + 4 * q) = x;
      }
    }
    // fragments of scale P beta (lower) and, for the backward, of scale P^T
    auto p_tile = [&](int b) {
      f32x4 x = zero4();
      if (b <= w) {
        const f32x4 Gc = *(const f32x4*)(Gs + 16 * b + 4 * q), Bc = *(const f32x4*)(Bs + 16 * b + 4 * q);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (row >= 16 * b + 4 * q + r) x[r] = a.scale * qk[b][r] * exp_hw(Gr - Gc[r]) * Bc[r];
      }
      return x;
    };
    if constexpr (!BWD) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (s <= w >> 1) {
          const Frag8 f = {pack4(p_tile(2 * s)), pack4(p_tile(2 * s + 1))};
          *(u32x4*)(a.Pf + ((unit * 6 + frag_lo(w, s)) * 64 + lane) * 8) = as_u4(f);
        }
    } else {
      auto pt_tile = [&](int b) {
        f32x4 x = zero4();
        if (b >= w) {
          const f32x4 Gc = *(const f32x4*)(Gs + 16 * b + 4 * q);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (16 * b + 4 * q + r >= row) x[r] = a.scale * kt[b][r] * exp_hw(Gc[r] - Gr);
        }
        return x;
      };
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (s >= w >> 1) {
          Frag8 hi, lo;
          split8(pt_tile(2 * s), pt_tile(2 * s + 1), hi, lo);
          u32x4* f = (u32x4*)(a.Pt + ((unit * 6 + frag_up(w, s)) * 2 * 64 + lane) * 8);
          f[0] = as_u4(hi);
          f[64] = as_u4(lo);
        }
    }
    __syncthreads();
    invert64(As, Ts, w, lane);
    // T: lane row i = 16 w + c, columns 16 b + 4 q + r; blocks above the diagonal are zero
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (s <= w >> 1) {
        const f32x4 x = *(const f32x4*)(Ts + row * TP + 32 * s + 4 * q);
        const f32x4 y = 2 * s + 1 <= w ? *(const f32x4*)(Ts + row * TP + 32 * s + 16 + 4 * q) : zero4();
        Frag8 hi, lo;
        split8(x, y, hi, lo);
        u32x4* f = (u32x4*)(a.Tf + ((unit * 6 + frag_lo(w, s)) * 2 * 64 + lane) * 8);
        f[0] = as_u4(hi);
        f[64] = as_u4(lo);
      }
    if constexpr (BWD) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (s >= w >> 1) {
          f32x4 x = zero4(), y;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if (2 * s >= w) x[r] = Ts[(32 * s + 4 * q + r) * TP + row];
            y[r] = Ts[(32 * s + 16 + 4 * q + r) * TP + row];
          }
          Frag8 hi, lo;
          split8(x, y, hi, lo);
          u32x4* f = (u32x4*)(a.Tt + ((unit * 6 + frag_up(w, s)) * 2 * 64 + lane) * 8);
          f[0] = as_u4(hi);
          f[64] = as_u4(lo);
        }
    }
  }
}

// ---------------------------------------------------------------------------
// walk
// ---------------------------------------------------------------------------
constexpr int WNT = 128;  // threads of a walk's workgroup

// MODE 0: the forward (o, S_final); 1: the states before every chunk, for the backward
template <int KP, int MODE>
__global__ void __launch_bounds__(WNT, 1) delta_chunk_walk_kernel(DeltaChunkArgs a) {
  constexpr int KS = KP / 32, KT = KP / 16;       // 32-steps and 16-tiles of K
  constexpr bool FWD = MODE == 0;
  __shared__ __attribute__((aligned(16))) bf16 Kb[2][64 * KP];
  __shared__ __attribute__((aligned(16))) bf16 Qb[FWD ? 2 : 1][FWD ? 64 * KP : 8];
  __shared__ __attribute__((aligned(16))) bf16 Vb[2][64 * VP];
  __shared__ __attribute__((aligned(16))) float eGs[2][64], wBs[2][64];  // e^G; e^{G_63 - G} beta
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, c = lane & 15, q = lane >> 4;
  i64 unit, slice;
  if (!walk_unit(a.seq.nseq * a.HV, (a.V + 31) / 32, unit, slice)) return;
  const i64 n = unit / a.HV, hv = unit % a.HV, h = hv / a.rep;
  const DeltaSpan sp = a.seq.span(n);
  const i64 nch = (sp.len + DCH - 1) / DCH;
  const i64 v0 = slice * 32 + w * 16;  // this wave's first column
  const bool act = v0 < a.V;           // V is a multiple of 16: all of a wave's columns or none

  RowTile<KP, WNT> sk, sq;
  ColTile<WNT> sv;
  float sG = 0.0f, sB = 0.0f;
  auto fetch = [&](i64 ch) {
    const i64 tok0 = sp.start + ch * DCH;
    const int rows = (int)(sp.len - ch * DCH < DCH ? sp.len - ch * DCH : DCH);
    sk.fetch(row_rsrc(a.k, tok0, rows, a.H, h, a.K), tid, a.H * a.K, a.K);
    if constexpr (FWD) sq.fetch(row_rsrc(a.q, tok0, rows, a.H, h, a.K), tid, a.H * a.K, a.K);
    sv.fetch(row_rsrc(a.v, tok0, rows, a.HV, hv, a.V), tid, a.HV * a.V, slice * 32, a.V);
    if (w == 0) {
      sG = a.G[((sp.slot0 + ch) * a.HV + hv) * 64 + lane];
      sB = lane < rows ? a.beta[(tok0 + lane) * a.HV + hv] : 0.0f;
    }
  };
  auto commit = [&](int bf) {
    sk.commit(Kb[bf], tid);
    if constexpr (FWD) sq.commit(Qb[bf], tid);
    sv.commit(Vb[bf], tid);
    if (w == 0) {
      const float end = __shfl(sG, 63, 64);
      eGs[bf][lane] = exp_hw(sG);
      wBs[bf][lane] = exp_hw(end - sG) * sB;
    }
  };

  f32x4 S[KT];
#pragma unroll
  for (int t = 0; t < KT; ++t) {
    S[t] = zero4();
    if (a.S0 && act) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int k = 16 * t + 4 * q + r;
        if (k < a.K) S[t][r] = a.S0[(unit * a.K + k) * a.V + v0 + c];
      }
    }
  }
  if (nch > 0) {
    fetch(0);
    commit(0);
  }
  __syncthreads();
  for (i64 ch = 0; ch < nch; ++ch) {
    const int bf = ch & 1;
    const i64 cu = (sp.slot0 + ch) * a.HV + hv;
    u32x4 tf[6][2], pf[FWD ? 6 : 1];
    if (act) {
#pragma unroll
      for (int i = 0; i < 6; ++i) {
        const u32x4* f = (const u32x4*)(a.Tf + (cu * 6 + i) * 2 * 64 * 8) + lane;
        tf[i][0] = f[0];
        tf[i][1] = f[64];
        if constexpr (FWD) pf[i] = ((const u32x4*)(a.Pf + (cu * 6 + i) * 64 * 8))[lane];
      }
    }
    if (ch + 1 < nch) fetch(ch + 1);
    if (act) {
      const bf16* Kt = Kb[bf];
      const bf16* Qt = Qb[FWD ? bf : 0];
      // K S0 (two parts of S0) and (Q S0)^T (one part)
      f32x4 x[4], ot[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) x[m] = zero4(), ot[m] = zero4();
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        Frag8 hi, lo;
        split8(S[2 * s], S[2 * s + 1], hi, lo);
        if constexpr (!FWD) {
          const i64 o = (((cu * a.nvt + slice * 2 + w) * KS + s) * 64 + lane) * 8;
          *(u32x4*)(a.Sh + o) = as_u4(hi);
          *(u32x4*)(a.Sl + o) = as_u4(lo);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const Frag8 kf = row_frag(Kt, KP, m, s, lane);
          x[m] = mma32(kf, hi, x[m]);
          x[m] = mma32(kf, lo, x[m]);
          if constexpr (FWD) {
            const Frag8 qf = row_frag(Qt, KP, m, s, lane);
            ot[m] = mma32(hi, qf, ot[m]);
          }
        }
      }
      // V - e^G K S0
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const f32x4 v = unpack4(ld_rowk(Vb[bf], VP, 16 * m, 16 * w, lane).v);
        const f32x4 e = *(const f32x4*)(eGs[bf] + 16 * m + 4 * q);
        x[m] = v - e * x[m];
      }
      Frag8 xh[2], xl[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) split8(x[2 * s], x[2 * s + 1], xh[s], xl[s]);
      // r = T (V - e^G K S0)
      f32x4 r[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        r[m] = zero4();
#pragma unroll
        for (int s = 0; s <= m / 2; ++s) {
          const Frag8 th = as_frag(tf[frag_lo(m, s)][0]), tl = as_frag(tf[frag_lo(m, s)][1]);
          r[m] = mma32(th, xl[s], r[m]);
          r[m] = mma32(tl, xh[s], r[m]);
          r[m] = mma32(th, xh[s], r[m]);
        }
      }
      // O^T = scale e^G (Q S0)^T + r^T (scale P beta)^T
      if constexpr (FWD) {
        const i64 tok0 = sp.start + ch * DCH;
        const i64 left = sp.len - ch * DCH;
        const Frag8 rf[2] = {{pack4(r[0]), pack4(r[1])}, {pack4(r[2]), pack4(r[3])}};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float e = a.scale * eGs[bf][16 * m + c];
          ot[m] *= e;
#pragma unroll
          for (int s = 0; s <= m / 2; ++s) ot[m] = mma32(rf[s], as_frag(pf[frag_lo(m, s)]), ot[m]);
          if (16 * m + c < left)
            *(s16x4*)(a.o + ((tok0 + 16 * m + c) * a.HV + hv) * a.V + v0 + 4 * q) = pack4(ot[m]);
        }
      }
      // S = e^{G_63} S0 + K^T (e^{G_63 - G} beta r)
      const float eEnd = eGs[bf][63];
#pragma unroll
      for (int m = 0; m < 4; ++m) r[m] *= *(const f32x4*)(wBs[bf] + 16 * m + 4 * q);
      Frag8 uh[2], ul[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) split8(r[2 * s], r[2 * s + 1], uh[s], ul[s]);
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        S[t] *= eEnd;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const Frag8 kf = col_frag(Kt, KP, t, s, lane);
          S[t] = mma32(kf, ul[s], S[t]);
          S[t] = mma32(kf, uh[s], S[t]);
        }
      }
    }
    if (ch + 1 < nch) commit(bf ^ 1);
    __syncthreads();
  }
  if (FWD && a.Sf && act) {
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int k = 16 * t + 4 * q + r;
        if (k < a.K) a.Sf[(unit * a.K + k) * a.V + v0 + c] = S[t][r];
      }
  }
}

// workspace of the forward: T and P fragments and G of every (slot, value head)
struct FwdPlan {
  i64 off_T, off_P, off_G;
  size_t bytes;
};
FwdPlan fwd_plan(i64 cells) {
  FwdPlan p{};
  i64 off = 0;
  auto carve = [&](i64 bytes) {
    const i64 o = off;
    off += (bytes + 255) / 256 * 256;
    return o;
  };
  p.off_T = carve(cells * 6 * 2 * 64 * 8 * 2);
  p.off_P = carve(cells * 6 * 64 * 8 * 2);
  p.off_G = carve(cells * 64 * 4);
  p.bytes = (size_t)off;
  return p;
}

}  // namespace

hipError_t launch_delta_prep(const DeltaChunkArgs& a, bool backward, hipStream_t stream) {
  const dim3 grid((unsigned)(a.nslots * a.H)), wg(256);
  if (a.K <= 64) {
    if (backward) hipLaunchKernelGGL((delta_prep_kernel<64, true>), grid, wg, 0, stream, a);
    else hipLaunchKernelGGL((delta_prep_kernel<64, false>), grid, wg, 0, stream, a);
  } else {
    if (backward) hipLaunchKernelGGL((delta_prep_kernel<128, true>), grid, wg, 0, stream, a);
    else hipLaunchKernelGGL((delta_prep_kernel<128, false>), grid, wg, 0, stream, a);
  }
  return hipGetLastError();
}

hipError_t launch_delta_states(const DeltaChunkArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)walk_blocks(a.seq.nseq * a.HV, (a.V + 31) / 32)), wg(WNT);
  if (a.K <= 64) hipLaunchKernelGGL((delta_chunk_walk_kernel<64, 1>), grid, wg, 0, stream, a);
  else hipLaunchKernelGGL((delta_chunk_walk_kernel<128, 1>), grid, wg, 0, stream, a);
  return hipGetLastError();
}

// Chunked MFMA kernels or the token walk.  float32 inputs take the walk.
bool delta_fwd_walks(const ssmvjp_delta_chunk_desc& d) { return d.dtype == SSMVJP_F32; }

size_t delta_fwd_workspace_bytes(const ssmvjp_delta_chunk_desc& d) {
  return delta_fwd_walks(d) ? 0 : fwd_plan(delta_slots(d) * d.nv_heads).bytes;
}

DeltaChunkArgs delta_chunk_args(const ssmvjp_delta_chunk_desc& d, const int* off) {
  DeltaChunkArgs a{};
  a.seq = delta_seqs(d, off);
  a.nslots = delta_slots(d);
  a.H = d.nqk_heads; a.HV = d.nv_heads; a.K = d.dk; a.V = d.dv;
  a.rep = d.nv_heads / d.nqk_heads; a.nvt = d.dv / 16; a.scale = d.scale;
  return a;
}

hipError_t launch_delta_fwd(const ssmvjp_delta_chunk_desc& d, const DeltaChunkPointers& p, hipStream_t stream) {
  if (delta_fwd_walks(d)) return launch_delta_walk(d, p, stream);
  DeltaChunkArgs a = delta_chunk_args(d, p.seq_offsets);
  const FwdPlan pl = fwd_plan(a.nslots * a.HV);
  char* ws = (char*)p.workspace;
  a.q = (const bf16*)p.q; a.k = (const bf16*)p.k; a.v = (const bf16*)p.v;
  a.beta = p.beta; a.g = p.g; a.S0 = p.S0; a.Sf = p.S_final; a.o = (bf16*)p.o;
  a.Tf = (bf16*)(ws + pl.off_T); a.Pf = (bf16*)(ws + pl.off_P); a.G = (float*)(ws + pl.off_G);
  if (a.nslots > 0) {
    const hipError_t e = launch_delta_prep(a, false, stream);
    if (e != hipSuccess) return e;
  }
  const dim3 grid((unsigned)walk_blocks(a.seq.nseq * a.HV, (a.V + 31) / 32)), wg(WNT);
  if (a.K <= 64) hipLaunchKernelGGL((delta_chunk_walk_kernel<64, 0>), grid, wg, 0, stream, a);
  else hipLaunchKernelGGL((delta_chunk_walk_kernel<128, 0>), grid, wg, 0, stream, a);
  return hipGetLastError();
}

}  // namespace ssmvjp
