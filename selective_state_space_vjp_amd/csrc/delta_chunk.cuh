// delta_chunk.cuh -- what the chunked gated delta rule's kernels share: the
// chunk algebra, its operand fragments and the workspace.
//
// One chunk of 64 tokens of one value head, S0 the state before it, G_i the
// running sum of the log gates inside the chunk, Gam_ij = exp(G_i - G_j):
//     r = (I + a diag(beta))^-1 (V - e^G K S0),   a_ij = Gam_ij k_i . k_j  (i > j)
//     u = beta r
//     O = scale (e^G Q S0 + P u),                 P_ij = Gam_ij q_i . k_j  (i >= j)
//     S = e^{G_63} S0 + K^T (e^{G_63 - G} u)
// (r is the whole residual v_t - k_t^T S_dec of every token: the triangular
// inverse, called T below, undoes the dependence of each on the ones before.)
//
// Number formats.  K, Q, V, dO are bf16 inputs and enter the products exactly.
// States, T, r and every other computed operand is split into two bf16 parts
// (x = hi + lo up to 2^-16 |x|, about 3e-6 in the mean), and the products keep
// hi hi, hi lo and lo hi, with float32 accumulation: states and the float32
// gradients come out at about 5e-6 instead of the 3e-3 of one bf16 part, and
// an error in the state is carried over thousands of tokens.  What only leads
// to a bf16 output (the readout, dq, dk) takes the hi part alone.
//
// Layouts.  D of a 16x16 MFMA tile has lane (c = lane % 16, q = lane / 16) hold
// column c, rows 4q .. 4q+3.  Two such tiles stacked (rows 32s .. 32s+31) are,
// without any exchange, the B operand (or the A operand of the transpose) of a
// 16x16x32 MFMA whose contraction runs over those rows in the order
//     slot e of lane group q  <->  row 32s + 16 (e / 4) + 4q + e % 4,
// as long as the other operand uses the same order.  "Fragment" below means
// that order.
#pragma once

#include "delta_seq.cuh"
#include "ssd_common.cuh"

namespace ssmvjp {

struct DeltaChunkArgs {
  DeltaSeqs seq;
  i64 nslots, H, HV, K, V, rep, nvt;  // nvt: 16-column tiles of V
  float scale;
  const bf16 *q, *k, *v, *d_o;
  const float *beta, *g, *S0, *dSf;
  bf16 *o, *dq, *dk, *dv;
  float *Sf, *dbeta, *dg, *dS0;
  // workspace, all per (slot, value head)
  bf16* Tf;   // [6][2][64][8] lower fragments of T, hi and lo
  bf16* Pf;   // [6][64][8] lower fragments of scale P beta
  float* G;   // [64]
  bf16* Tt;   // [6][2][64][8] fragments of T^T                      (backward from here on)
  bf16* Pt;   // [6][2][64][8] fragments of scale P^T
  bf16 *Sh, *Sl, *dSh;          // [nvt][KP/32][64][8] fragments of the state before the chunk (two parts) and of
                                // the state's gradient behind it
  bf16 *rh, *rl, *muh, *mul;    // [nvt][2][64][8] fragments of r and mu (two parts each)
  float* rowp;                  // [nvt][2][64] sums over a tile's columns, see delta_chunk_rev_kernel
  float* endp;                  // [nvt]
};

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
struct Frag8 {
  s16x4 a, b;
};
__device__ __forceinline__ f32x4 mma32(const Frag8& x, const Frag8& y, f32x4 d) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), d, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma32(const u32x4& x, const u32x4& y, f32x4 d) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), d, 0, 0, 0);
}
__device__ __forceinline__ Frag8 as_frag(const u32x4& u) { return __builtin_bit_cast(Frag8, u); }
__device__ __forceinline__ u32x4 as_u4(const Frag8& f) { return __builtin_bit_cast(u32x4, f); }

__device__ __forceinline__ s16x4 pack4(const f32x4& v) {
  typedef unsigned u32x2_t __attribute__((ext_vector_type(2)));
  const u32x2_t u = {pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])};
  return __builtin_bit_cast(s16x4, u);
}
__device__ __forceinline__ f32x4 unpack4(const s16x4& s) {
  f32x4 v;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = bits_bf16(s[j]);
  return v;
}
// v = hi + lo, two bf16 parts
__device__ __forceinline__ void split4(const f32x4& v, s16x4& hi, s16x4& lo) {
  hi = pack4(v);
  lo = pack4(v - unpack4(hi));
}
// the fragments of two stacked tiles
__device__ __forceinline__ void split8(const f32x4& x, const f32x4& y, Frag8& hi, Frag8& lo) {
  split4(x, hi.a, lo.a);
  split4(y, hi.b, lo.b);
}

// position of the fragment of row tile mt, contraction step s: lower triangular
// (steps 0 .. mt / 2) and its transpose (steps mt / 2 .. 1)
__device__ __forceinline__ constexpr int frag_lo(int mt, int s) { return mt < 2 ? mt : 2 * mt - 2 + s; }
__device__ __forceinline__ constexpr int frag_up(int mt, int s) { return mt < 2 ? 2 * mt + s : mt + 2; }

// a log gate as the kernels use it: e^-88 is where float32 ends, and a bounded
// sum keeps -inf (a hard reset) from turning differences of sums into NaN
__device__ __forceinline__ float gate_clamp(float g) { return g < -88.0f ? -88.0f : g; }

// resource over the rows [tok0, tok0 + rows) of head h of a [tokens][heads][cols] tensor
// (rows past the end read as zeros)
__device__ __forceinline__ brsrc row_rsrc(const bf16* p, i64 tok0, int rows, i64 heads, i64 h, i64 cols) {
  return make_rsrc(p + (tok0 * heads + h) * cols, (unsigned)((((i64)rows - 1) * heads * cols + cols) * 2));
}

// The rows of a chunk on their way to LDS: registers <- memory (fetch), LDS <-
// registers (commit), so that the loads of the next chunk are in flight while
// this one is computed.  NT threads take part.
template <int KP, int NT>
struct RowTile {  // [64][KP] of q or k, swizzled rows, columns past K zero
  static constexpr int N = 64 * KP / 8 / NT;
  u32x4 r[N];
  __device__ __forceinline__ void fetch(brsrc rs, int tid, i64 stride, i64 K) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int p = tid + NT * i, row = p / (KP / 8), col = p % (KP / 8) * 8;
      r[i] = bload16(rs, col < K ? (unsigned)((row * stride + col) * 2) : BUF_OOB);
    }
  }
  __device__ __forceinline__ void commit(bf16* lds, int tid) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int p = tid + NT * i;
      st16_xs(lds, KP, p / (KP / 8), p % (KP / 8) * 8, r[i]);
    }
  }
};
constexpr int VP = 36;  // row pitch of a staged [64][32] tile: 8-byte rows, shifted by 2 banks each
template <int NT>
struct ColTile {  // [64][32] of v or d_o, the columns from v0
  static constexpr int N = 256 / NT;
  u32x4 r[N];
  __device__ __forceinline__ void fetch(brsrc rs, int tid, i64 stride, i64 v0, i64 V) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int p = tid + NT * i, row = p / 4;
      const i64 col = v0 + p % 4 * 8;
      r[i] = bload16(rs, col < V ? (unsigned)((row * stride + col) * 2) : BUF_OOB);
    }
  }
  __device__ __forceinline__ void commit(bf16* lds, int tid) const {
    typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int p = tid + NT * i;
      u32x2* d = (u32x2*)(lds + p / 4 * VP + p % 4 * 8);
      d[0] = u32x2{r[i][0], r[i][1]};
      d[1] = u32x2{r[i][2], r[i][3]};
    }
  }
};
// fragment of rows 16m .. 16m+15 of a swizzled row tile, contraction over its columns
__device__ __forceinline__ Frag8 row_frag(const bf16* t, int KP, int m, int s, int lane) {
  return {ld_colk_xs(t, KP, 16 * m, 32 * s, lane).v, ld_colk_xs(t, KP, 16 * m, 32 * s + 16, lane).v};
}
// fragment of columns 16t .. 16t+15, contraction over its rows
__device__ __forceinline__ Frag8 col_frag(const bf16* x, int pitch, int t, int s, int lane) {
  return {ld_rowk_xs(x, pitch, 32 * s, 16 * t, lane).v, ld_rowk_xs(x, pitch, 32 * s + 16, 16 * t, lane).v};
}

struct ChunkAt {
  DeltaSpan sp;
  i64 seq, tok0;
  int rows;  // 0: nothing here
};
__device__ __forceinline__ ChunkAt chunk_at(const DeltaSeqs& q, i64 slot, int lane) {
  ChunkAt c;
  c.seq = q.of_slot(slot, lane);
  c.sp = q.span(c.seq);
  const i64 ch = slot - c.sp.slot0, left = c.sp.len - ch * DCH;
  c.tok0 = c.sp.start + ch * DCH;
  c.rows = ch < 0 || left <= 0 ? 0 : left < DCH ? (int)left : DCH;
  return c;
}

// (sequence, value head, slice) of a walk's workgroup: ids go round the 8 XCDs,
// and the slices of one head, which read the same q, k and fragments, share one
// XCD's L2.  unit = sequence * HV + head; false: no work.
__device__ __forceinline__ bool walk_unit(i64 units, i64 nslice, i64& unit, i64& slice) {
  const i64 x = blockIdx.x & 7, y = blockIdx.x >> 3;
  unit = y / nslice * 8 + x;
  slice = y % nslice;
  return unit < units;
}
inline i64 walk_blocks(i64 units, i64 nslice) { return (units + 7) / 8 * 8 * nslice; }

DeltaChunkArgs delta_chunk_args(const ssmvjp_delta_chunk_desc& d, const int* off);
hipError_t launch_delta_prep(const DeltaChunkArgs& a, bool backward, hipStream_t stream);
hipError_t launch_delta_states(const DeltaChunkArgs& a, hipStream_t stream);

}  // namespace ssmvjp
