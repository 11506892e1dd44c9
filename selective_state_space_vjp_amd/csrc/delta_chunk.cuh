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
// an error in the state is carried over thousands of tokens.  T is applied as
// I + (T - I), the identity without any rounding, and u enters the state in
// three parts.  What leads to a bf16 output (o, dq, dk) keeps both parts too: it
// comes out at the output's own rounding, 1.7e-3 of the norm; with the hi parts
// alone o had 2.0e-3 to 2.6e-3, dk 3.1e-3.
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
#include "lds_dma.cuh"
#include "ssd_common.cuh"

namespace ssmvjp {

struct DeltaChunkArgs {
  DeltaSeqs seq;
  i64 nslots, H, HV, K, V, rep, nvt;  // nvt: 16-column tiles of V
  const bf16 *q, *k, *v, *d_o;
  const float *beta, *g, *S0, *dSf;
  bf16 *o, *dq, *dk, *dv;
  float *Sf, *dbeta, *dg, *dS0;
  // workspace, all per (slot, value head)
  bf16* Tf;   // [6][2][64][8] lower fragments of T - I, hi and lo
  bf16* Pf;   // [6][2][64][8] lower fragments of scale P beta
  float* G;   // [64]
  bf16* Tt;   // [6][2][64][8] fragments of T^T - I                  (backward from here on)
  bf16* Pt;   // [6][2][64][8] fragments of scale P^T
  // per 16-column tile (cell * nvt + tile), hi and lo parts, in the order in which the gradients kernel reads
  // them from LDS (state_slot, row_slot):
  bf16* Sw;   // [2][KP/32][64][8] the state before the chunk
  bf16* dSw;  // [2][KP/32][64][8] the state's gradient behind the chunk
  bf16* rw;   // [2][4][64][4] r
  bf16* muw;  // [2][4][64][4] mu
  // few cells only (NULL otherwise): the states before and the gradients behind every chunk [K][V] and r [64][V] in
  // float32, and what comes of them: r . (K dS) e^{G_63 - G} per token [64], <S0, dS>
  float *S32, *dS32, *r32, *su, *dot;
  float scale;
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

// x = hi + mid + lo up to 2^-24 |x|
__device__ __forceinline__ void split8x3(const f32x4& x, const f32x4& y, Frag8& hi, Frag8& mid, Frag8& lo) {
  hi.a = pack4(x);
  hi.b = pack4(y);
  split8(x - unpack4(hi.a), y - unpack4(hi.b), mid, lo);
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

// ---- row tiles in LDS ----
// [64][KP] rows of q or k, no padding, columns past K zero.  The 16-byte unit u
// of a row is stored at u ^ row_swz(KP, row).  LDS takes 16 lanes of 16 bytes or 32
// of 8 at a time over 256 bytes (a row of KP = 128, two of KP = 64): the 16 rows
// of one unit that a fragment read takes meet 16 different places; the 8 rows of
// four half units that a transposed read takes fill every place twice, the least
// that half units allow.
__device__ __forceinline__ int row_swz(int KP, int row) {
  return KP == 128 ? ((row & 3) << 2) | ((row >> 2) & 3) : ((row & 2) << 1) | ((row >> 2) & 3);
}

// Contraction over K.  A fragment of rows is 16 contiguous bytes: slot e of lane
// group q <-> column 32s + 8q + e.  The state's tiles match it by their rows:
// row 4q + r of tile 2s + b is key 32s + 8q + 4b + r.
__device__ __forceinline__ int state_row(int tile, int q) { return 32 * (tile >> 1) + 8 * q + 4 * (tile & 1); }

// a store that the L2 need not keep: the walks write more than it holds, and what it holds (k, q, fragments) is
// read by the other slices of the head
template <typename T>
__device__ __forceinline__ void stream_store(T* p, const T& v) {
  __builtin_nontemporal_store(v, p);
}

// What the walks keep is read by columns, 4 rows of 4 units of 8 bytes at a time
// (a transposed read of 16 lanes): these orders put each such group into 128
// bytes of its own, so that the blocks go to LDS as they are.
// The 8-key pieces of a state's fragment, lane (c, q): 16-byte slots.
__device__ __forceinline__ int state_slot(int lane) {
  const int c = lane & 15, q = lane >> 4;
  return (c >> 2) * 16 + q * 4 + (c & 3);
}
// The four rows 4q .. of one row tile, lane (c, q): 8-byte slots.
__device__ __forceinline__ int row_slot(int lane) {
  const int c = lane & 15, q = lane >> 4;
  return (c >> 2) * 16 + (c & 3) * 4 + q;
}
// column tile b of r or mu, contraction over 32 columns of V: t0, t1 are the blocks [4][64][4] of two tiles
__device__ __forceinline__ Frag8 kept_rows(const bf16* t0, const bf16* t1, int b, int lane) {
  return {lds_tr_b16(t0 + b * 256 + lane * 4).v, lds_tr_b16(t1 + b * 256 + lane * 4).v};
}
// keys 16t .. of a state, contraction over 32 columns of V: t0, t1 are the blocks [KP/32][64][8] of two tiles
__device__ __forceinline__ Frag8 kept_keys(const bf16* t0, const bf16* t1, int t, int lane) {
  const int m = lane & 15, o = (t >> 1) * 512 + ((lane >> 4) * 16 + ((t & 1) * 2 + ((m >> 1) & 1)) * 4 + (m >> 2)) * 8 + (m & 1) * 4;
  return {lds_tr_b16(t0 + o).v, lds_tr_b16(t1 + o).v};
}

// a state [K][V] in memory (NULL, or a wave without columns: zeros): four rows of column v of tile t
__device__ __forceinline__ brsrc state_rsrc(const float* S, const DeltaChunkArgs& a, i64 unit, bool act) {
  const float* p = S + unit * a.K * a.V;
  return make_rsrc(S ? p : S, S && act ? (unsigned)(a.K * a.V * 4) : 0u);
}
__device__ __forceinline__ f32x4 load_state4(brsrc rs, const DeltaChunkArgs& a, int t, int q, i64 v) {
  const int k = state_row(t, q);
  f32x4 x;
#pragma unroll
  for (int r = 0; r < 4; ++r) x[r] = bload_f32(rs, k < a.K ? (unsigned)(((k + r) * a.V + v) * 4) : BUF_OOB);
  return x;
}

// rows 16m .. 16m+15, contraction over the columns 32s .. 32s+31
__device__ __forceinline__ Frag8 row_frag(const bf16* t, int KP, int m, int s, int lane) {
  const int row = 16 * m + (lane & 15);
  return as_frag(*(const u32x4*)(t + row * KP + (((4 * s + (lane >> 4)) ^ row_swz(KP, row)) << 3)));
}
// the keys of state tile t as rows, contraction over the tokens 32s .. 32s+31 (slot order of the token fragments)
__device__ __forceinline__ Frag8 key_frag(const bf16* x, int KP, int t, int s, int lane) {
  const int m = lane & 15, row = 32 * s + 4 * (lane >> 4) + (m >> 2), u = 4 * (t >> 1) + (m & 3);
  return {lds_tr_b16(x + row * KP + ((u ^ row_swz(KP, row)) << 3) + 4 * (t & 1)).v,
          lds_tr_b16(x + (row + 16) * KP + ((u ^ row_swz(KP, row + 16)) << 3) + 4 * (t & 1)).v};
}
// LDS-direct loads of one chunk's tiles, shared out over NW waves, 1 KB (64
// pieces of 16 bytes) an instruction.  A wave's instructions are consecutive; the
// swizzle repeats every 16 rows, VAR instructions.
template <int KP, int NW>
struct RowDma {
  static constexpr int N = KP / 8 / NW, VAR = KP == 128 ? 4 : 2;  // instructions a wave; rows 4 or 8 an instruction
  unsigned off[VAR], step;
  __device__ __forceinline__ void init(int w, int lane, i64 stride, i64 K) {
#pragma unroll
    for (int j = 0; j < VAR; ++j) {
      const int p = 64 * (N * w + j) + lane, row = p / (KP / 8), col = ((p % (KP / 8)) ^ row_swz(KP, row)) * 8;
      off[j] = col < K ? (unsigned)((row * stride + col) * 2) : BUF_OOB;
    }
    step = (unsigned)(16 * stride * 2);
  }
  __device__ __forceinline__ void issue(unsigned lds, int w, u32x4 rs) const {
#pragma unroll
    for (int j = 0; j < N; ++j)
      dma_dwordx4(lds + 1024u * (unsigned)(N * w + j), off[j % VAR] + (unsigned)(j / VAR) * step, rs);
  }
};
// [64][16 NT] of v or d_o, the columns from v0 (zero past V)
template <int NT, int NW>
struct ColDma {
  static constexpr int N = 2 * NT / NW, ROWS = 32 / NT;  // instructions a wave; rows an instruction
  unsigned off, step;
  __device__ __forceinline__ void init(int w, int lane, i64 stride, i64 v0, i64 V) {
    const int row = N * w * ROWS + lane / (2 * NT), col = lane % (2 * NT) * 8;
    off = v0 + col < V ? (unsigned)((row * stride + col) * 2) : BUF_OOB;
    step = (unsigned)(ROWS * stride * 2);
  }
  __device__ __forceinline__ void issue(unsigned lds, int w, u32x4 rs) const {
#pragma unroll
    for (int j = 0; j < N; ++j) dma_dwordx4(lds + 1024u * (unsigned)(N * w + j), off + (unsigned)j * step, rs);
  }
};
// N KB as they are
template <int N, int NW>
__device__ __forceinline__ void flat_dma(unsigned lds, int w, int lane, u32x4 rs) {
#pragma unroll
  for (int i = 0; i < N; i += NW)
    if (N % NW == 0 || i + w < N) dma_dwordx4(lds + 1024u * (unsigned)(i + w), (unsigned)((i + w) * 1024 + lane * 16), rs);
}
// four values down column 16w + c of a [64][16 NW] tile: rows 16m + 4q ..
__device__ __forceinline__ s16x4 col4(const bf16* t, int pitch, int m, int w, int lane) {
  return ld_rowk(t, pitch, 16 * m, 16 * w, lane).v;
}

// words of a resource over the rows [tok0, tok0 + rows) of head h of a [tokens][heads][cols] tensor, from column
// col0 (rows past the end read as zeros)
__device__ __forceinline__ u32x4 row_words(const bf16* p, i64 tok0, int rows, i64 heads, i64 h, i64 cols, i64 col0) {
  return rsrc_words_u(p + (tok0 * heads + h) * cols + col0, (unsigned)((((i64)rows - 1) * heads * cols + cols - col0) * 2));
}

// no instruction moves past here: operands that are read ahead stay ahead
#define SSMVJP_FENCE() __builtin_amdgcn_sched_barrier(0)
// asks the scheduler for N times: an MFMA, VALU vector instructions, READ LDS reads
template <int N, int VALU, int READ>
__device__ __forceinline__ void pipe() {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
    if (VALU) __builtin_amdgcn_sched_group_barrier(0x2, VALU, 0);
    if (READ) __builtin_amdgcn_sched_group_barrier(0x100, READ, 0);
  }
}

// a wave's 16 columns of a state into the float32 matrix m [K][V] (col: the lane's)
template <int KT>
__device__ __forceinline__ void store_state32(float* m, const f32x4 (&S)[KT], i64 K, i64 V, int q, i64 col) {
  const brsrc rs = make_rsrc(m, (unsigned)(K * V * 4));
  unsigned o = (unsigned)((8 * q * V + col) * 4);
  asm volatile("" : "+v"(o));  // anew for every chunk: 32 addresses kept over the loop would not fit
#pragma unroll
  for (int t = 0; t < KT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float x = S[t][r];
      const unsigned at = state_row(t, q) + r < K ? o + (unsigned)((state_row(t, 0) + r) * V * 4) : BUF_OOB;
      __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, x), rs, (int)at, 0, 0);
    }
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
// XCD's L2.  unit = sequence * HV + head, past the last one: no work.
struct WalkUnit {
  i64 unit, slice;
};
__device__ __forceinline__ WalkUnit walk_unit(unsigned block, i64 nslice) {
  const unsigned x = block & 7, y = block >> 3, ns = (unsigned)nslice;
  return {(i64)(y / ns * 8 + x), (i64)(y % ns)};
}
inline i64 walk_blocks(i64 units, i64 nslice) { return (units + 7) / 8 * 8 * nslice; }

DeltaChunkArgs delta_chunk_args(const ssmvjp_delta_chunk_desc& d, const int* off);
hipError_t launch_delta_prep(const DeltaChunkArgs& a, bool backward, hipStream_t stream);

}  // namespace ssmvjp
