// delta_chunk.hip -- the chunked gated delta rule on MFMA: what each chunk needs
// that does not depend on the state (delta_prep_kernel, all chunks at once) and
// the walk over the chunks that carries the state (delta_walk.cuh).
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
// Bound by writing the fragments (24 KB of a chunk and value head, backward 36
// KB): b=2 T=4096 H=16 HV=32 K=V=128 takes 41 us, 100 MB written at 2.4 TB/s
// (backward 62 us, 150 MB), with two loads in a row exposed per workgroup; with
// the loads of k and q not all up front it was 55 us.
#include "delta_walk.cuh"

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
      for (int j = 0; j < i; j += 4) {
        const f32x4 r = *(const f32x4*)(A + i * TP + j);  // the same for every lane
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (j + k < i) s = fmaf(-r[k], x[j + k], s);
      }
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
__global__ void __launch_bounds__(256, 3) delta_prep_kernel(DeltaChunkArgs a) {
  constexpr int KS = KP / 32;
  __shared__ float As[64 * TP], Ts[64 * TP];
  __shared__ float Gs[64], Bs[64];
  __shared__ int lost;  // forward: the first row of a beta with a value that is not finite (64: none)
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, q = lane >> 4;
  const unsigned H32 = (unsigned)a.H;
  const i64 h = blockIdx.x % H32, slot = blockIdx.x / H32;
  const ChunkAt at = chunk_at(a.seq, slot, lane);
  if (at.rows == 0) return;
  const brsrc rk = row_rsrc(a.k, at.tok0, at.rows, a.H, h, a.K), rq = row_rsrc(a.q, at.tok0, at.rows, a.H, h, a.K);
  auto off = [&](int tile, int s) {
    const int col = 32 * s + 8 * q;
    return col < a.K ? (unsigned)(((i64)(16 * tile + c) * a.H * a.K + col) * 2) : BUF_OOB;
  };
  // everything this wave needs of k and q is on its way before the first product
  u32x4 kx[4][KS], qw[KS], qx[BWD ? 4 : 1][KS];
#pragma unroll
  for (int b = 0; b < 4; ++b)
    if (b <= w) {
#pragma unroll
      for (int s = 0; s < KS; ++s) kx[b][s] = bload16(rk, off(b, s));
    }
#pragma unroll
  for (int s = 0; s < KS; ++s) qw[s] = bload16(rq, off(w, s));
  if constexpr (BWD) {
#pragma unroll
    for (int b = 0; b < 4; ++b)
      if (b > w) {
#pragma unroll
        for (int s = 0; s < KS; ++s) qx[b][s] = bload16(rq, off(b, s));
      }
  }
  const bool in = lane < at.rows;
  float gn = in ? a.g[(at.tok0 + lane) * a.HV + h * a.rep] : 0.0f, bn = in ? a.beta[(at.tok0 + lane) * a.HV + h * a.rep] : 0.0f;
  u32x4 kw[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) kw[s] = w == 0 ? kx[0][s] : w == 1 ? kx[1][s] : w == 2 ? kx[2][s] : kx[3][s];
  // lane: row i = 16 w + c, columns j = 16 b + 4 q + r (kt: row j = 16 w + c, columns i)
  f32x4 kk[4], qk[4], kt[BWD ? 4 : 1];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    kk[b] = zero4();
    qk[b] = zero4();
    if (b <= w) {
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        kk[b] = mma32(kx[b][s], kw[s], kk[b]);
        qk[b] = mma32(kx[b][s], qw[s], qk[b]);
      }
    }
    if constexpr (BWD) {
      kt[b] = zero4();
      if (b >= w) {
#pragma unroll
        for (int s = 0; s < KS; ++s) kt[b] = mma32(b == w ? qw[s] : qx[b][s], kw[s], kt[b]);
      }
    }
  }
  for (i64 rr = 0; rr < a.rep; ++rr) {
    const i64 hv = h * a.rep + rr, unit = slot * a.HV + hv;
    __syncthreads();  // the previous head's readers are done with LDS
    if (w == 0) {
      const float G = wave_incl_scan(gate_clamp(gn), lane);
      Gs[lane] = G;
      Bs[lane] = bn;
      a.G[unit * 64 + lane] = G;
      if (!BWD && lane == 0) lost = 64;
    }
    __syncthreads();
    if (rr + 1 < a.rep && in) {  // the next head's gates
      gn = a.g[(at.tok0 + lane) * a.HV + hv + 1];
      bn = a.beta[(at.tok0 + lane) * a.HV + hv + 1];
    }
    const int row = 16 * w + c;
    const float Gr = Gs[row];
    // a beta into LDS and, for the forward, the tiles of scale P beta
    f32x4 p[4], az = zero4();
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      p[b] = zero4();
      if (b <= w) {
        const f32x4 Gc = *(const f32x4*)(Gs + 16 * b + 4 * q), Bc = *(const f32x4*)(Bs + 16 * b + 4 * q);
        f32x4 x;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 16 * b + 4 * q + r;
          const float gb = exp_hw(row >= j ? Gr - Gc[r] : 0.0f) * Bc[r];
          x[r] = row > j ? kk[b][r] * gb : 0.0f;
          if (!BWD && row >= j) p[b][r] = a.scale * qk[b][r] * gb;
        }
        *(f32x4*)(As + row * TP + 16 * b + 4 * q) = x;
        az += 0.0f * x;
      }
    }
    if constexpr (!BWD) {
      // T is formed without the rows that hold such values and gets NaN from the first of them on: its products run
      // over the zeros above the diagonal and would carry them to rows before
      if (__builtin_expect(!(az[0] + az[1] + az[2] + az[3] == 0.0f), 0)) {
        atomicMin(&lost, row);
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (b <= w) *(f32x4*)(As + row * TP + 16 * b + 4 * q) = zero4();
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (s <= w >> 1) {
          Frag8 hi, lo;
          split8(p[2 * s], p[2 * s + 1], hi, lo);
          u32x4* f = (u32x4*)(a.Pf + ((unit * 6 + frag_lo(w, s)) * 2 * 64 + lane) * 8);
          f[0] = as_u4(hi);
          f[64] = as_u4(lo);
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
    // T - I: lane row i = 16 w + c, columns 16 b + 4 q + r; blocks above the diagonal are zero
    const bool gone = !BWD && row >= lost;
    auto off_diag = [&](f32x4 x, int col) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (col + r == row) x[r] = 0.0f;
        if (gone) x[r] = __builtin_nanf("");
      }
      return x;
    };
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (s <= w >> 1) {
        const f32x4 x = *(const f32x4*)(Ts + row * TP + 32 * s + 4 * q);
        const f32x4 y = 2 * s + 1 <= w ? *(const f32x4*)(Ts + row * TP + 32 * s + 16 + 4 * q) : zero4();
        Frag8 hi, lo;
        split8(off_diag(x, 32 * s + 4 * q), off_diag(y, 32 * s + 16 + 4 * q), hi, lo);
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
          split8(off_diag(x, 32 * s + 4 * q), off_diag(y, 32 * s + 16 + 4 * q), hi, lo);
          u32x4* f = (u32x4*)(a.Tt + ((unit * 6 + frag_up(w, s)) * 2 * 64 + lane) * 8);
          f[0] = as_u4(hi);
          f[64] = as_u4(lo);
        }
    }
  }
}

template <int KP>
__global__ void __launch_bounds__(walk_nth(0)) __attribute__((amdgpu_waves_per_eu(2, 2)))
delta_chunk_walk_kernel(DeltaChunkArgs a) {
  delta_chunk_walk<KP, 0>(a, blockIdx.x);
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
  p.off_P = carve(cells * 6 * 2 * 64 * 8 * 2);
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

// Chunked MFMA kernels or the token walk: float32 inputs take the walk at any length, since the chunked kernels read
// bf16 operands and keep what they compute in two bf16 parts, short of float32 results.  It is slow where sequences
// are long, 0.7 us a token: b=2 HV=32 K=V=128 takes 45 us for T=64, 174 for 256, 2,770 for 4096 (bf16, chunked: 22,
// 28, 175).  Up to 16 tokens take it in bf16 too, since a chunk costs the same whether it is full or not while the
// walk grows with its tokens.  Chunked against walk at K = V = 128, HV = 32: 17 against 9 us for 8 tokens, 17 against
// 14 for 16, 18 against 25 for 32 (1 sequence); 40 against 24 for 16, 40 against 33 for 24, 40 against 42 for 32 (8);
// 115 against 69 for 16, 117 against 122 for 32 (32).  At 24 tokens one sequence takes 18 against 20.  A packed call
// goes by all its tokens together, since the lengths are in device memory: many short sequences take the chunked
// kernels there (32 of 16 tokens: 119 us packed, 65 as a batch), and one long one among them never takes the walk.
bool delta_fwd_walks(const ssmvjp_delta_chunk_desc& d) { return d.dtype == SSMVJP_F32 || d.seqlen <= 16; }

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
  const dim3 grid((unsigned)walk_blocks(a.seq.nseq * a.HV, (a.V + 31) / 32)), wg(walk_nth(0));
  if (a.K <= 64) hipLaunchKernelGGL((delta_chunk_walk_kernel<64>), grid, wg, (WalkLds<64, 0>::TOTAL), stream, a);
  else hipLaunchKernelGGL((delta_chunk_walk_kernel<128>), grid, wg, (WalkLds<128, 0>::TOTAL), stream, a);
  return hipGetLastError();
}

}  // namespace ssmvjp
