// gated_ffn.hip -- the projections of a gated feed-forward block and their
// gradients: h = act(x Wg^T) * (x Wu^T).
//
// Every product is C(m,n) = sum_k A(m,k) B(n,k) on tiles of the matrix cores:
//   forward        A = x, B = Wg and Wu (two products that share A; the
//                  activation and the product are applied to the sums)
//   dx             A = dgate, dup (one behind the other along k), B = Wg^T, Wu^T
//   dWg, dWu       A = dgate^T, dup^T, B = x^T
// k runs along the rows of an operand in memory (KC) or down its columns.
//
// dgate and dup are rounded to the type between the products, as gate and up are
// when they are kept: the gradients of bf16 come out at 2.3e-3 of the norm, the
// two roundings of 1.7e-3 together.  In two parts each (the value's rounding and
// what that leaves) they take twice the products, and the gradients come out at
// 1.7e-3: that is done where a result has few values or few roundings in it,
// whose errors do not average out (up to 2.6e-3 otherwise), and the time is the
// launches' (TWO_PARTS).
//
// The matrix cores and what feeds them are the bound: bf16 at 8192 x 4096 ->
// 12288 runs at 1.31 PFLOP/s without and 1.24 with gate and up (their 400 MB are
// stored in bursts at the tiles' ends), dx and the weights' gradients at 1.30,
// where a library product of 8192^3 reaches 1.40.  Matrix cores busy 61 % of the
// cycles, at 2.0 GHz under this load.  Measured and not kept: 32 x 32 x 16
// products (1410 us forward against 1320), four buffers of 64 bytes of k (1497
// against 1385), the next step's fragments read before the barrier (3 % faster
// forward, 1 % slower backward), a higher wave priority for the products (2 %
// slower), four waves of 128 x 128 (4 % faster forward, 3 % slower weights'
// gradients, and only with the accumulators pinned by hand), streaming stores.
// Few rows are bound by the weights: 5 rows of 4096 -> 12288 take 41 us (201 MB,
// 4.9 TB/s), 33 where the memory-side cache still holds them.
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "lds_dma.cuh"

namespace ssmvjp {
namespace {

struct Operand {
  const void* p;
  i64 ld;
};

struct FfnArgs {
  i64 M, N, K;          // K: of one segment
  Operand A[4], B[2];   // PAIR: A[0] with both B; else segments of k, segment s of A with B[s % 2]
  int segs;
  i64 ldc;
  void* C[4];           // h, gate, up | dgate, dup and, in two parts, what their roundings leave | C
  const void *dh;       // BACK: [M, N]
  int items;            // products of one shape in one launch: A[i segs ..], C[i] (EPI_PLAIN)
  int split;            // parts of k, each a workgroup's; more than one: sums to part
  float* part;          // [items][split][PAIR ? 2 : 1][M][N]
};

enum { EPI_PLAIN, EPI_GLU, EPI_GLU_BACK };

// act and its derivative at z
template <int ACT>
__device__ __forceinline__ void act_pair(float z, float& f, float& df) {
  if constexpr (ACT == SSMVJP_ACT_SILU) {
    const float s = __builtin_amdgcn_rcpf(1.0f + exp_hw(-z));
    f = z * s;
    df = fmaf(f, 1.0f - s, s);
  } else {
    // (1 + tanh(v)) / 2 = sigmoid(2 v); a z^2 that overflows would meet the 0 of f (1 - s)
    const float k = 1.5957691216057308f, z2 = fminf(z * z, 1e30f);
    const float s = __builtin_amdgcn_rcpf(1.0f + exp_hw(-k * z * fmaf(0.044715f, z2, 1.0f)));
    f = z * s;
    df = fmaf(f * (1.0f - s), k * fmaf(0.134145f, z2, 1.0f), s);
  }
}
template <int ACT>
__device__ __forceinline__ float act_of(float z) {
  float f, df;
  act_pair<ACT>(z, f, df);
  return f;
}

// ---------------------------------------------------------------------------
// Tiles.  A workgroup forms BM x BN values of C; every step of its loop brings
// 128 bytes of k (64 values of bf16, 32 of float32) of both operands into one
// of two buffers in LDS by LDS-direct loads while the other is multiplied.
//
// In LDS a tile lies as in memory, in 16-byte chunks: rows of 8 chunks (KC: a
// row is one m or n), or rows of BM or BN values (a row is one k).  Chunk p of
// row r holds the row's chunk p ^ swizzle(r), which spreads the rows that one
// read touches over the banks; the loads write LDS in order, so it is the
// addresses in memory that are permuted.
//
// The products run with the roles of A and B exchanged, which leaves a lane
// with four consecutive n of one m.
// ---------------------------------------------------------------------------
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
constexpr int ROWB = 128;  // bytes of k per step
constexpr int LDS_BYTES = 160 * 1024;
constexpr int SCHED_MFMA = 0x008, SCHED_LDS_READ = 0x100;  // kinds of instructions of sched_group_barrier

template <typename T>
struct Fragment;  // 16 values of m or n, half a step of k
template <>
struct Fragment<bf16> {
  bf16x8 v;
};
template <>
struct Fragment<float> {
  f32x4 v;
};

__device__ __forceinline__ void multiply(f32x4& d, const Fragment<bf16>& a, const Fragment<bf16>& b) {
  d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, d, 0, 0, 0);
}
__device__ __forceinline__ void multiply(f32x4& d, const Fragment<float>& a, const Fragment<float>& b) {
#pragma unroll
  for (int j = 0; j < 4; ++j) d = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[j], b.v[j], d, 0, 0, 0);
}

template <typename T, bool KC, int MN>
struct TileOf {
  static constexpr int CPR = KC ? ROWB / 16 : MN * (int)sizeof(T) / 16;  // chunks of a row
  static constexpr int ROWS = KC ? MN : ROWB / (int)sizeof(T);
  static constexpr int BYTES = MN * ROWB;
  static constexpr int READS = KC ? 1 : sizeof(T) == 2 ? 2 : 4;  // instructions of a fragment
  static __device__ __forceinline__ int swizzle(int r) {
    if constexpr (KC) return r & 7;
    else if constexpr (sizeof(T) == 2) return (((r & 3) | ((r >> 3) & 3) << 2) << 1) & (CPR - 1);
    else return ((r >> 2) & 3) << 2;
  }
  // the byte in memory, from the tile's first, that chunk i of LDS holds
  static __device__ __forceinline__ unsigned source(int i, unsigned ldb) {
    const int r = i / CPR, p = i % CPR;
    return r * ldb + ((p ^ swizzle(r)) << 4);
  }
  // the k (in values from the step's first) of that chunk's first value
  static __device__ __forceinline__ int source_k(int i) {
    const int r = i / CPR, p = i % CPR;
    return KC ? (p ^ swizzle(r)) * (16 / (int)sizeof(T)) : r;
  }
  // values mn .. mn + 15, half `kk` of the step
  static __device__ __forceinline__ Fragment<T> fragment(const char* lds, int mn, int kk, int lane) {
    const int q = lane >> 4, c = lane & 15;
    Fragment<T> f;
    if constexpr (KC) {
      const int r = mn + c;
      f.v = *(const decltype(f.v)*)(lds + r * ROWB + (((q + 4 * kk) ^ swizzle(r)) << 4));
    } else if constexpr (sizeof(T) == 2) {
      // two transposing reads of 4 k x 16 values
      typedef short s16x8 __attribute__((ext_vector_type(8)));
      s16x4 h[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = kk * 32 + 8 * q + 4 * i + (c >> 2);
        const int chunk = ((mn >> 3) + ((c & 3) >> 1)) ^ swizzle(r);
        h[i] = lds_tr_b16((const bf16*)(lds + r * (CPR * 16) + chunk * 16 + (c & 1) * 8)).v;
      }
      f.v = __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = kk * 16 + 4 * q + j;
        const int chunk = ((mn >> 2) + (c >> 2)) ^ swizzle(r);
        f.v[j] = *(const float*)(lds + r * (CPR * 16) + chunk * 16 + (c & 3) * 4);
      }
    }
    return f;
  }
};

// Where the tile mn0 .. of an operand begins at step k0, and how many bytes behind that may be read: rows of KC past
// the last m or n, and rows of k past the last, come back as zeros.  Columns past the last m or n reach C there only.
template <typename T, bool KC>
__device__ __forceinline__ u32x4 tile_rsrc(const Operand& o, i64 mn0, i64 MN, i64 k0, i64 K, int tile) {
  constexpr int KB = ROWB / (int)sizeof(T);
  const i64 r0 = KC ? mn0 : k0, c0 = KC ? k0 : mn0, all = KC ? MN : K;
  const i64 rows = all - r0 < (KC ? tile : KB) ? all - r0 : (KC ? tile : KB);
  return rsrc_words_u((const T*)o.p + r0 * o.ld + c0, (unsigned)((rows * o.ld - c0) * (i64)sizeof(T)));
}

// Tile number -> (m, n).  Workgroups go round the eight XCDs, each with an L2 of its own: an XCD gets a contiguous run
// of tiles, in bands of 4 tiles of m, so that those it works on at one time share rows of A and of B.
__device__ __forceinline__ void place(unsigned id, unsigned nm, unsigned nn, unsigned& m, unsigned& n) {
  const unsigned total = nm * nn, each = total / 8, rest = total % 8, xcd = id % 8;
  const unsigned t = xcd * each + (xcd < rest ? xcd : rest) + id / 8;
  const unsigned band = t / (4 * nn), m0 = band * 4, h = nm - m0 < 4 ? nm - m0 : 4, in = t - band * 4 * nn;
  m = m0 + in % h;
  n = in / h;
}

// act(gate) up and what the backward makes of it, four n of one m
template <typename T>
__device__ __forceinline__ void store4(void* p, i64 e, const float (&v)[4]) {
  if constexpr (sizeof(T) == 2) *(uint2*)((bf16*)p + e) = make_uint2(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]));
  else *(float4*)((float*)p + e) = make_float4(v[0], v[1], v[2], v[3]);
}
template <typename T>
__device__ __forceinline__ void fetch4(const void* p, i64 e, float (&v)[4]) {
  if constexpr (sizeof(T) == 2) {
    const uint2 u = *(const uint2*)((const bf16*)p + e);
    v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xffff0000u);
    v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xffff0000u);
  } else {
    const float4 u = *(const float4*)((const float*)p + e);
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
  }
}

// all but the last N loads have come, and every read of LDS has its data: behind a barrier the buffer read last is free
template <int N>
__device__ __forceinline__ void step_wait() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"i"(N) : "memory");
}

__device__ __forceinline__ void step_barrier() {
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// what the rounding of v leaves; nothing of a value that is rounded to an infinity or is none
template <typename T>
__device__ __forceinline__ float left_over(float v) {
  const float r = (float)(T)v;
  return fabsf(r) < INFINITY ? v - r : 0.0f;
}

// What the sums v[0] (and v[1], PAIR) of four n of one m become: the values of the outputs.  e: where dh has them.
template <typename T, int EPI, int ACT>
__device__ __forceinline__ void finish4(const FfnArgs& a, i64 e, float (&v)[4][4]) {
  if constexpr (EPI == EPI_GLU) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      v[2][r] = v[1][r];
      v[1][r] = v[0][r];
      v[0][r] = act_of<ACT>(v[1][r]) * v[2][r];
    }
  } else if constexpr (EPI == EPI_GLU_BACK) {
    fetch4<T>(a.dh, e, v[2]);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float f, df;
      act_pair<ACT>(v[0][r], f, df);
      v[0][r] = v[2][r] * v[1][r] * df;
      v[1][r] = v[2][r] * f;
    }
    if (a.C[2])
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        v[2][r] = left_over<T>(v[0][r]);
        v[3][r] = left_over<T>(v[1][r]);
      }
  }
}
template <int EPI>
__device__ __forceinline__ int outputs(const FfnArgs& a) {
  return EPI == EPI_PLAIN ? 1 : EPI == EPI_GLU_BACK ? (a.C[2] ? 4 : 2) : a.C[1] ? 3 : 1;
}

// The outputs on their way through LDS: ROWS of a wave's FM rows of 16 at a time, the most that fit, in 1, 2, 4 .. parts.
template <typename T, int EPI, int BM, int NOUT, int FM>
struct StoreOf {
  static constexpr int PITCH = NOUT * (int)sizeof(T) + 16, ALL = (EPI == EPI_PLAIN ? 1 : EPI == EPI_GLU ? 3 : 4) * BM * PITCH;
  static constexpr int PARTS = FM > 2 && ALL / 2 > LDS_BYTES ? 4 : FM > 1 ? 2 : 1;
  static constexpr int ROWS = FM / PARTS, BYTES = ALL / PARTS;
  static_assert(FM % PARTS == 0 && BYTES <= LDS_BYTES, "");
};

// WM x WN waves, NB buffers.  PAIR: the tile's BN columns are BN/2 of each of two products, side by side in every wave.
// block: the workgroup's number among those of this product.
template <typename T, bool AKC, bool BKC, int EPI, int ACT, int BM, int BN, int WM, int WN, int NB>
__device__ __forceinline__ void gemm_tile(const FfnArgs& a, const unsigned block, char* lds) {
  constexpr bool PAIR = EPI != EPI_PLAIN;
  constexpr int W = WM * WN, KB = ROWB / (int)sizeof(T), NOUT = PAIR ? BN / 2 : BN;
  constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  typedef TileOf<T, AKC, BM> TA;
  typedef TileOf<T, BKC, NOUT> TB;
  static_assert(BM >= 32 && FM > 0 && FN > 0, "");
  constexpr int IA = TA::BYTES / 1024 / W, IB = TB::BYTES / 1024 / W;  // loads of a wave, each product's B by itself
  constexpr int BUF = TA::BYTES + (PAIR ? 2 : 1) * TB::BYTES;
  static_assert(IA * 1024 * W == TA::BYTES && IB * 1024 * W == TB::BYTES, "");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN * (BM / WM), wn = wave % WN * (NOUT / WN);
  const unsigned nm = (unsigned)((a.M + BM - 1) / BM), nn = (unsigned)((a.N + NOUT - 1) / NOUT);
  unsigned tm, tn;
  place(block % (nm * nn), nm, nn, tm, tn);
  const i64 m0 = (i64)tm * BM, n0 = (i64)tn * NOUT;
  const int steps1 = (int)((a.K + KB - 1) / KB), all = (PAIR ? 1 : a.segs) * steps1;
  const int which = block / (nm * nn), item = PAIR ? 0 : which / a.split, share = which - item * a.split;
  const int first = (int)((i64)all * share / a.split), steps = (int)((i64)all * (share + 1) / a.split) - first;
  const unsigned base = lds_base(lds);

  unsigned offA[IA], offB[IB];
#pragma unroll
  for (int i = 0; i < IA; ++i) offA[i] = TA::source((wave * IA + i) * 64 + lane, (unsigned)(a.A[0].ld * sizeof(T)));
#pragma unroll
  for (int i = 0; i < IB; ++i) offB[i] = TB::source((wave * IB + i) * 64 + lane, (unsigned)(a.B[0].ld * sizeof(T)));

  auto load = [&](int at, int buf) {
    const int step = first + at, s = PAIR ? 0 : (step >= steps1) + (step >= 2 * steps1) + (step >= 3 * steps1);
    const i64 k0 = (i64)(step - s * steps1) * KB;
    const bool part = k0 + KB > a.K;  // KC: chunks past the last k would be the next row's
    const unsigned to = base + buf * BUF;
    const u32x4 ra = tile_rsrc<T, AKC>(a.A[s + item * a.segs], m0, a.M, k0, a.K, BM);
#pragma unroll
    for (int i = 0; i < IA; ++i) {
      unsigned off = offA[i];
      if (AKC && part && k0 + TA::source_k((wave * IA + i) * 64 + lane) >= a.K) off = BUF_OOB;
      dma_dwordx4(to + (wave * IA + i) * 1024, off, ra);
    }
#pragma unroll
    for (int p = 0; p < (PAIR ? 2 : 1); ++p) {
      const u32x4 rb = tile_rsrc<T, BKC>(a.B[PAIR ? p : s & 1], n0, a.N, k0, a.K, NOUT);
#pragma unroll
      for (int i = 0; i < IB; ++i) {
        unsigned off = offB[i];
        if (BKC && part && k0 + TB::source_k((wave * IB + i) * 64 + lane) >= a.K) off = BUF_OOB;
        dma_dwordx4(to + TA::BYTES + p * TB::BYTES + (wave * IB + i) * 1024, off, rb);
      }
    }
  };

  // float32: the halves of the steps are summed apart, which takes sqrt(2) off the error of a sum of thousands (1.0e-6 -> 0.7e-6
  // of 2456 terms); the tiles from 128 x 128 on have no registers for it
  constexpr int HALVES = sizeof(T) == 4 && FM * FN <= 8 ? 2 : 1;
  f32x4 acc[HALVES][FM][FN];
#pragma unroll
  for (int h = 0; h < HALVES; ++h)
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[h][i][j] = zero4();

  // the next NB - 1 steps are on their way while one is multiplied
  constexpr int LOADS = IA + (PAIR ? 2 : 1) * IB;
#pragma unroll
  for (int i = 0; i < NB - 1; ++i)
    if (i < steps) load(i, i);
  int at = 0;
  for (int step = 0; step < steps; ++step) {
    if (step + NB - 1 <= steps) step_wait<(NB - 2) * LOADS>();
    else step_wait<0>();
    step_barrier();
    const char* buf = lds + at * BUF;
    if (step + NB - 1 < steps) load(step + NB - 1, at == 0 ? NB - 1 : at - 1);
    at = at + 1 == NB ? 0 : at + 1;
    Fragment<T> fa[2][FM], fb[2][FN];
    auto read = [&](int kk) {
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        constexpr int half = PAIR ? FN / 2 : FN;
        const int p = j / half;
        fb[kk][j] = TB::fragment(buf + TA::BYTES + p * TB::BYTES, wn + 16 * (j - p * half), kk, lane);
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) fa[kk][i] = TA::fragment(buf, wm + 16 * i, kk, lane);
    };
    read(0);
    read(1);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) multiply(kk < HALVES ? acc[kk][i][j] : acc[0][i][j], fb[kk][j], fa[kk][i]);
    // The order of the step: the fragments of B and of the first LEAD rows of A are read, then one more read goes with
    // every few products, so that a wave does not stop for LDS at each (left to the compiler, which reads a fragment right
    // before its use, the forward at 8192 x 4096 -> 12288 takes 1308 us instead of 1250).
    constexpr int LEAD = FM < 4 ? FM : 4, MM = 2 * FM * FN * (sizeof(T) == 2 ? 1 : 4);
    constexpr int FIRST = FN * TB::READS + LEAD * TA::READS, REST = 2 * (FN * TB::READS + FM * TA::READS) - FIRST;
    constexpr int PER = (MM - FN * LEAD) / REST > 0 ? (MM - FN * LEAD) / REST : 1;
    __builtin_amdgcn_sched_group_barrier(SCHED_LDS_READ, FIRST, 0);
#pragma unroll
    for (int i = 0; i < REST; ++i) {
      __builtin_amdgcn_sched_group_barrier(SCHED_MFMA, PER, 0);
      __builtin_amdgcn_sched_group_barrier(SCHED_LDS_READ, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(SCHED_MFMA, MM - PER * REST, 0);
  }
  if constexpr (HALVES > 1)
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[0][i][j] += acc[HALVES - 1][i][j];

  if (a.split > 1) {
    const i64 each = a.M * a.N;
    float* part = a.part + (PAIR ? 2 : 1) * each * which;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const i64 m = m0 + wm + 16 * i + (lane & 15);
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int second = PAIR && j >= FN / 2;
        const i64 n = n0 + wn + 16 * (second ? j - FN / 2 : j) + 4 * (lane >> 4);
        if (m < a.M && n < a.N) *(f32x4*)(part + second * each + m * a.N + n) = acc[0][i][j];
      }
    }
    return;
  }
  // Through LDS, so that whole rows of the tile are stored by 16 bytes a lane: a part of every wave's rows at a time, all
  // outputs side by side (8192 x 4096 -> 12288 with gate and up: 1350 us; 1440 with stores of 32 bytes of a row from the
  // registers).
  typedef StoreOf<T, EPI, BM, NOUT, FM> SO;
  constexpr int ROWS = SO::ROWS, ER = WM * 16 * ROWS, PITCH = SO::PITCH, CHUNKS = NOUT * (int)sizeof(T) / 16;
  const int nout = outputs<EPI>(a);
#pragma unroll
  for (int h = 0; h < FM / ROWS; ++h) {
    step_wait<0>();
    step_barrier();
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
#pragma unroll
      for (int j = 0; j < (PAIR ? FN / 2 : FN); ++j) {
        const int col = wn + 16 * j + 4 * (lane >> 4);
        const i64 m = m0 + wm + 16 * (h * ROWS + i) + (lane & 15), n = n0 + col;
        const bool in = m < a.M && n < a.N;
        float v[4][4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          v[0][r] = acc[0][h * ROWS + i][j][r];
          if constexpr (PAIR) v[1][r] = acc[0][h * ROWS + i][j + FN / 2][r];
        }
        finish4<T, EPI, ACT>(a, in ? m * a.ldc + n : 0, v);
        char* to = lds + ((wave / WN) * 16 * ROWS + 16 * i + (lane & 15)) * PITCH + col * (int)sizeof(T);
        store4<T>(to, 0, v[0]);
        if constexpr (PAIR)
          if (nout > 1) {
            store4<T>(to + ER * PITCH, 0, v[1]);
            if (EPI == EPI_GLU || nout > 2) store4<T>(to + 2 * ER * PITCH, 0, v[2]);
            if (EPI == EPI_GLU_BACK && nout > 2) store4<T>(to + 3 * ER * PITCH, 0, v[3]);
          }
      }
    step_wait<0>();
    step_barrier();
    for (int i = threadIdx.x; i < nout * ER * CHUNKS; i += 64 * W) {
      const int o = i / (ER * CHUNKS), r = i / CHUNKS % ER, c = i % CHUNKS;
      const i64 m = m0 + r / (16 * ROWS) * (BM / WM) + h * 16 * ROWS + r % (16 * ROWS), n = n0 + c * (16 / (int)sizeof(T));
      if (m < a.M && n < a.N)
        *(uint4*)((T*)a.C[EPI == EPI_PLAIN ? item : o] + m * a.ldc + n) = *(const uint4*)(lds + (o * ER + r) * PITCH + c * 16);
    }
  }
}

template <typename T, bool AKC, bool BKC, int EPI, int ACT, int BM, int BN, int WM, int WN, int NB>
__global__ void __launch_bounds__(64 * WM * WN) ffn_gemm_kernel(FfnArgs a) {
  extern __shared__ __align__(1024) char lds[];
  gemm_tile<T, AKC, BKC, EPI, ACT, BM, BN, WM, WN, NB>(a, blockIdx.x, lds);
}

// dx by the first workgroups, the weights' gradients by the others, which need nothing of each other: a launch less (the
// backward of 20 x 512 -> 1024 takes 13.4 us, 16.2 with two; of 777 x 1000 -> 2712 60, 68).
template <typename T, int BMX, int BNX, int WX, int NBX, int BNW, int NBW>
__global__ void __launch_bounds__(256) ffn_grads_kernel(FfnArgs dx, FfnArgs dw, unsigned blocks) {
  extern __shared__ __align__(1024) char lds[];
  if (blockIdx.x < blocks) gemm_tile<T, true, false, EPI_PLAIN, 0, BMX, BNX, WX, 4 / WX, NBX>(dx, blockIdx.x, lds);
  else gemm_tile<T, false, false, EPI_PLAIN, 0, 128, BNW, 2, 2, NBW>(dw, blockIdx.x - blocks, lds);
}

// the parts' sums in order, and what becomes of them: the share `block` of `blocks`
template <typename T, int EPI, int ACT>
__device__ __forceinline__ void join_parts(const FfnArgs& a, const i64 block, const i64 blocks) {
  constexpr bool PAIR = EPI != EPI_PLAIN;
  const i64 each = a.M * a.N;
  for (i64 i = (block * 256 + threadIdx.x) * 4; i < each * a.items; i += blocks * 1024) {
    const int item = (int)(i / each);
    const i64 e = i - item * each;
    float v[4][4];
#pragma unroll
    for (int p = 0; p < (PAIR ? 2 : 1); ++p) {
      const float* part = a.part + ((PAIR ? 2 : 1) * (i64)item * a.split + p) * each + e;
      fetch4<float>(part, 0, v[p]);
      for (int s = 1; s < a.split; ++s) {
        float w[4];
        fetch4<float>(part, (PAIR ? 2 : 1) * s * each, w);
#pragma unroll
        for (int r = 0; r < 4; ++r) v[p][r] += w[r];
      }
    }
    const i64 at = e / a.N * a.ldc + e % a.N;
    finish4<T, EPI, ACT>(a, at, v);
    store4<T>(a.C[EPI == EPI_PLAIN ? item : 0], at, v[0]);
    if constexpr (PAIR) {
      const int nout = outputs<EPI>(a);
      if (nout > 1) store4<T>(a.C[1], at, v[1]);
      if (nout > 2) store4<T>(a.C[2], at, v[2]);
      if (nout > 3) store4<T>(a.C[3], at, v[3]);
    }
  }
}

template <typename T, int EPI, int ACT>
__global__ void __launch_bounds__(256) ffn_join_kernel(FfnArgs a) {
  join_parts<T, EPI, ACT>(a, blockIdx.x, gridDim.x);
}
template <typename T>
__global__ void __launch_bounds__(256) ffn_join_grads_kernel(FfnArgs dx, FfnArgs dw, unsigned blocks) {
  if (blockIdx.x < blocks) join_parts<T, EPI_PLAIN, 0>(dx, blockIdx.x, blocks);
  else join_parts<T, EPI_PLAIN, 0>(dw, blockIdx.x - blocks, gridDim.x - blocks);
}

// dgate, dup (TWO: and what their roundings leave, n further on each) from the kept gate and up, 16 bytes a lane; n a
// multiple of 8
template <typename T, int ACT, bool TWO>
__global__ void __launch_bounds__(256) ffn_grad_kernel(const T* dh, const T* gate, const T* up, T* dgate, T* dup, i64 n) {
  constexpr int W = 16 / sizeof(T);
  typedef T vec __attribute__((ext_vector_type(W)));
  for (i64 e = ((i64)blockIdx.x * 256 + threadIdx.x) * W; e < n; e += (i64)gridDim.x * 256 * W) {
    const vec d = *(const vec*)(dh + e), g = *(const vec*)(gate + e), u = *(const vec*)(up + e);
    vec og, ou, og2, ou2;
#pragma unroll
    for (int r = 0; r < W; ++r) {
      float f, df;
      act_pair<ACT>((float)g[r], f, df);
      const float vg = (float)d[r] * (float)u[r] * df, vu = (float)d[r] * f;
      og[r] = (T)vg;
      ou[r] = (T)vu;
      if constexpr (TWO) {
        og2[r] = (T)left_over<T>(vg);
        ou2[r] = (T)left_over<T>(vu);
      }
    }
    *(vec*)(dgate + e) = og;
    *(vec*)(dup + e) = ou;
    if constexpr (TWO) {
      *(vec*)(dgate + 2 * n + e) = og2;
      *(vec*)(dup + 2 * n + e) = ou2;
    }
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
enum { TILE_LARGE, TILE_MID, TILE_NARROW, TILE_FEW };  // 256 x 256, 128 x 128, 128 x 64, 32 x 64

struct GemmPlan {
  int tile, split;
};

// A product's shape as the rules below see it.  kc: k along the rows of A.
struct Shape {
  i64 M, N, steps;
  int items;
  bool pair, kc, two;  // two: bf16
};
Shape shape_of(i64 M, i64 N, i64 K, int segs, int items, bool pair, bool kc, size_t elem) {
  return {M, N, segs * ((K * (i64)elem + ROWB - 1) / ROWB), items, pair, kc, elem == 2};
}
i64 tiles_of(const Shape& p, i64 bm, i64 bn) {
  return p.items * ((p.M + bm - 1) / bm) * ((p.N * (p.pair ? 2 : 1) + bn - 1) / bn);
}

// Parts of at least 4 steps, together at most 512 workgroups.
constexpr int PARTS = 16, WORKGROUPS = 512;
bool may_cut(const Shape& p, i64 tiles, int split) { return split == 1 || (p.steps >= 4 * split && tiles * split <= WORKGROUPS); }

// The smaller tiles: the time of a step of bf16 and float32 in steps of 128 x 128, alone and beside another product.
struct Kind {
  int tile;
  i64 bm, bn;
  float step[2], beside[2];
};
constexpr Kind KINDS[] = {{TILE_MID, 128, 128, {1.0f, 1.0f}, {1.0f, 1.0f}},
                          {TILE_NARROW, 128, 64, {0.7f, 0.6f}, {0.7f, 0.6f}},
                          {TILE_FEW, 32, 64, {0.35f, 0.15f}, {0.45f, 0.25f}}};
// Up to 32 rows are one tile of the small kind, which is for operands with k along the rows.
bool single(const Shape& p) { return p.kc && p.M <= 32; }
bool fits(const Shape& p, const Kind& k) { return k.tile == TILE_FEW ? p.kc : !single(p); }

// what the second launch takes that adds the parts, in steps: a launch, and the parts' bytes
float sum_time(const Shape& p, int split, float launch) {
  return split > 1 ? launch + (float)(split * p.items * p.M * p.N * (p.pair ? 8 : 4)) / (p.two ? 2e6f : 4e6f) : 0.0f;
}

// Whether the large tile fills the 256 CUs by itself (4096 x 2048 -> 8192 dw: 278 us, 327 with 128 x 128) or with k cut into
// long parts (dx of the same: 317, uncut 446, 128 x 128 347; of 1024 x 4096 -> 12288: 215, 552, 270).
bool large_plan(const Shape& p, GemmPlan& g) {
  const i64 large = tiles_of(p, 256, 256);
  if (large == 0 || single(p)) return false;
  const i64 cut = large >= 256 ? 1 : 256 / large;
  g = {TILE_LARGE, (int)cut};
  return large >= 256 || (cut * large >= 232 && p.steps >= 96 * cut);
}

// Which tile, and into how many parts k is cut, for a product by itself: by the time of the busiest CU.  bf16 waits for its
// loads, so that two workgroups of a CU take 1.2 of the time of one; with the small tile and in float32 they take 2.  The
// constants come from a sweep of the tiles in 1 to 16 parts over 125 products of 1 to 8000 rows: the choice is 1.4 % above
// the fastest on average.  Forward at 100 x 1024 -> 2048: 6.9 us with 32 x 64, 9.8 with 128 x 64, 12.7 with 128 x 128; at
// 777 x 1000 -> 2712: 22.8 with 128 x 64, 19 with 128 x 128; dx of 512 x 1024 -> 4096 in 8 parts: 28, 31.
GemmPlan gemm_plan(const Shape& p) {
  GemmPlan best;
  if (large_plan(p, best)) return best;
  best = {single(p) ? TILE_FEW : TILE_MID, 1};
  float least = INFINITY;
  for (const Kind& k : KINDS) {
    if (!fits(p, k)) continue;
    const i64 tiles = tiles_of(p, k.bm, k.bn);
    for (int split = 1; split <= PARTS && may_cut(p, tiles, split); ++split) {
      const i64 per_cu = (split * tiles + 255) / 256;
      float time = (float)((p.steps + split - 1) / split) * k.step[p.two ? 0 : 1];
      if (per_cu > 1) time *= (p.two && k.tile != TILE_FEW ? 0.6f : 1.0f) * (float)per_cu;
      time += sum_time(p, split, p.two ? 4.0f : 1.5f);
      if (time < least) {
        least = time;
        best = {k.tile, split};
      }
    }
  }
  return best;
}

// The same for dx and the weights' gradients in one launch, neither on the large tile (else false): 512 workgroups run at
// one time, those of dx begin first, and dx in few long parts leaves room beside it.  A workgroup takes its steps and 2 more
// (float32: half of one), two on a CU 1.4 (1.6) of that.  From a sweep of both products' tiles and parts over 18 sizes: 3 % above
// the fastest on average, the plans that are best alone 13 % (float32 16 %).  Both of 777 x 1000 -> 2712 from the kept gate and
// up: 42 us with dx in 3 parts of 128 x 128, 50 in 4 of 128 x 64.
bool grads_plan(const Shape& x, const Shape& w, GemmPlan& px, GemmPlan& pw) {
  if (large_plan(x, px) || large_plan(w, pw)) return false;
  const int dt = x.two ? 0 : 1;
  const float more = x.two ? 2.0f : 0.5f, crowd = x.two ? 1.4f : 1.6f, launch = x.two ? 4.0f : 1.5f;
  float least = INFINITY;
  px = {single(x) ? TILE_FEW : TILE_MID, 1};
  pw = {TILE_MID, 1};
  for (const Kind& kw : KINDS) {
    if (!fits(w, kw)) continue;
    const i64 tw = tiles_of(w, kw.bm, kw.bn);
    for (int sw = 1; sw <= PARTS && may_cut(w, tw, sw); sw *= 2) {
      const float nw = (float)(tw * sw), lw = (float)((w.steps + sw - 1) / sw) * kw.beside[dt] + more, jw = sum_time(w, sw, launch);
      for (const Kind& kx : KINDS) {
        if (!fits(x, kx)) continue;
        const i64 tx = tiles_of(x, kx.bm, kx.bn);
        for (int sx = 1; sx <= PARTS && may_cut(x, tx, sx); ++sx) {
          const float nx = (float)(tx * sx), lx = (float)((x.steps + sx - 1) / sx) * kx.beside[dt] + more;
          float time = lx > lw ? lx : lw;
          if (nx + nw > WORKGROUPS) {
            const float even = (nx * lx + nw * lw) / WORKGROUPS + 0.7f * lw;
            time = lx > even ? lx : even;
          }
          if (nx + nw > 256) time *= crowd;
          time += sum_time(x, sx, launch) + jw - (sx > 1 && sw > 1 ? launch : 0.0f);
          if (time < least) {
            least = time;
            px = {kx.tile, sx};
            pw = {kw.tile, sw};
          }
        }
      }
    }
  }
  return true;
}

size_t part_bytes(const Shape& p, int split) {
  return split > 1 ? (size_t)((p.items * split * p.M * p.N * (p.pair ? 8 : 4) + 255) / 256 * 256) : 0;
}
// at most, whatever the choice
size_t most_part_bytes(const Shape& p) {
  GemmPlan g{TILE_MID, 1};
  if (large_plan(p, g)) return part_bytes(p, g.split);
  int most = 1;
  for (const Kind& k : KINDS)
    if (fits(p, k))
      for (int split = PARTS; split > most; --split)
        if (may_cut(p, tiles_of(p, k.bm, k.bn), split)) most = split;
  return part_bytes(p, most);
}

// bytes of LDS: the buffers, or the outputs on their way
template <typename T, int EPI, int BM, int BN, int WM, int NB>
constexpr int lds_bytes() {
  constexpr int loop = NB * (BM + BN) * ROWB, rows = StoreOf<T, EPI, BM, EPI != EPI_PLAIN ? BN / 2 : BN, BM / WM / 16>::BYTES;
  static_assert(loop <= LDS_BYTES, "");
  return loop > rows ? loop : rows;
}
// a product's workgroups on tiles of bm x bn (PAIR: of both products)
unsigned gemm_blocks(const FfnArgs& a, i64 bm, i64 bn) {
  return (unsigned)(((a.N + bn - 1) / bn) * ((a.M + bm - 1) / bm) * a.items * a.split);
}
unsigned join_blocks(const FfnArgs& a) {
  const i64 blocks = (a.items * a.M * a.N + 1023) / 1024;
  return (unsigned)(blocks < 4096 ? blocks : 4096);
}

template <typename T, bool AKC, bool BKC, int EPI, int ACT, int BM, int BN, int WM, int WN, int NB>
void launch_tile(const FfnArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((ffn_gemm_kernel<T, AKC, BKC, EPI, ACT, BM, BN, WM, WN, NB>),
                     dim3(gemm_blocks(a, BM, EPI != EPI_PLAIN ? BN / 2 : BN)), dim3(64 * WM * WN), (lds_bytes<T, EPI, BM, BN, WM, NB>()), s, a);
}

template <typename T, int EPI, bool KC>
Shape shape_of(const FfnArgs& a) {
  return shape_of(a.M, a.N, a.K, a.segs, a.items, EPI != EPI_PLAIN, KC, sizeof(T));
}

template <typename T, bool AKC, bool BKC, int EPI, int ACT>
void launch_gemm(FfnArgs a, float* part, hipStream_t s) {
  const GemmPlan g = gemm_plan(shape_of<T, EPI, AKC>(a));
  a.split = g.split;
  a.part = part;
  if (g.tile == TILE_LARGE) launch_tile<T, AKC, BKC, EPI, ACT, 256, 256, 2, 4, 2>(a, s);
  else if (g.tile == TILE_MID) launch_tile<T, AKC, BKC, EPI, ACT, 128, 128, 2, 2, 2>(a, s);
  else if (g.tile == TILE_NARROW) launch_tile<T, AKC, BKC, EPI, ACT, 128, 64, 2, 2, 3>(a, s);
  else if constexpr (AKC) launch_tile<T, AKC, BKC, EPI, ACT, 32, 64, 2, 2, 6>(a, s);
  if (g.split > 1) hipLaunchKernelGGL((ffn_join_kernel<T, EPI, ACT>), dim3(join_blocks(a)), dim3(256), 0, s, a);
}

// dx and the weights' gradients, neither on the large tile
template <typename T, int BMX, int BNX, int WX, int NBX, int BNW, int NBW>
void launch_grads_tile(const FfnArgs& dx, const FfnArgs& dw, hipStream_t s) {
  constexpr int lx = lds_bytes<T, EPI_PLAIN, BMX, BNX, WX, NBX>(), lw = lds_bytes<T, EPI_PLAIN, 128, BNW, 2, NBW>();
  const unsigned first = gemm_blocks(dx, BMX, BNX);
  hipLaunchKernelGGL((ffn_grads_kernel<T, BMX, BNX, WX, NBX, BNW, NBW>), dim3(first + gemm_blocks(dw, 128, BNW)), dim3(256),
                     lx > lw ? lx : lw, s, dx, dw, first);
}
template <typename T, int BMX, int BNX, int WX, int NBX>
void launch_grads_dx(const FfnArgs& dx, const FfnArgs& dw, bool mid, hipStream_t s) {
  if (mid) launch_grads_tile<T, BMX, BNX, WX, NBX, 128, 2>(dx, dw, s);
  else launch_grads_tile<T, BMX, BNX, WX, NBX, 64, 3>(dx, dw, s);
}
template <typename T>
void launch_grads(FfnArgs dx, FfnArgs dw, const GemmPlan& px, const GemmPlan& pw, float* part, hipStream_t s) {
  dx.split = px.split;
  dx.part = part;
  dw.split = pw.split;
  dw.part = (float*)((char*)part + part_bytes(shape_of<T, EPI_PLAIN, true>(dx), px.split));
  const bool mid = pw.tile == TILE_MID;
  if (px.tile == TILE_MID) launch_grads_dx<T, 128, 128, 2, 2>(dx, dw, mid, s);
  else if (px.tile == TILE_NARROW) launch_grads_dx<T, 128, 64, 2, 3>(dx, dw, mid, s);
  else launch_grads_dx<T, 32, 64, 2, 6>(dx, dw, mid, s);
  const unsigned first = px.split > 1 ? join_blocks(dx) : 0, rest = pw.split > 1 ? join_blocks(dw) : 0;
  if (first + rest) hipLaunchKernelGGL((ffn_join_grads_kernel<T>), dim3(first + rest), dim3(256), 0, s, dx, dw, first);
}

template <typename T, int ACT>
void ffn_fwd(const ssmvjp_ffn_desc& d, const FfnFwdPointers& p, hipStream_t s) {
  FfnArgs a{d.rows, d.hidden, d.dim, {{p.x, d.dim}}, {{p.w_gate, d.dim}, {p.w_up, d.dim}}, 1, d.hidden, {p.h, p.gate, p.up}, nullptr, 1, 1, nullptr};
  launch_gemm<T, true, true, EPI_GLU, ACT>(a, (float*)p.workspace, s);
}

// Whether dgate and dup of bf16 are kept in two parts: where dgate or a weight's gradient has fewer than TWO_PARTS values,
// of products of normal ones, among which few large ones count, or dx, whose values are sums, fewer than a quarter of
// that.  Over 400 drawn sizes the gradients are then at most 1.45 of the error that their own roundings would leave (1.55
// without).  The products of such calls are short: from kept gate and up 48 x 392 -> 8 takes 6.8 us of the GPU in two parts
// and 6.1 in one, 33 x 400 -> 96 8.6 and 7.3, both behind the host's 14 us a call.  Two parts at every size would make the
// gradients' 2.34e-3 of the norm 1.66e-3 for twice the products: 8192 x 4096 -> 12288 5620 us instead of 2815,
// 1024 x 1024 -> 2816 74 instead of 46, 777 x 1000 -> 2712 69 instead of 43.
constexpr i64 TWO_PARTS = 8192;
int grads_parts(const ssmvjp_ffn_desc& d) {
  const bool few = d.rows * d.hidden < TWO_PARTS || d.hidden * d.dim < TWO_PARTS || d.rows * d.dim < TWO_PARTS / 4;
  return d.dtype == SSMVJP_BF16 && few ? 2 : 1;
}
// dgate, dup, and their second parts
size_t grads_bytes(const ssmvjp_ffn_desc& d) {
  return (size_t)((grads_parts(d) * 2 * d.rows * d.hidden * (d.dtype == SSMVJP_BF16 ? 2 : 4) + 255) / 256 * 256);
}

template <typename T, int ACT>
void ffn_bwd(const ssmvjp_ffn_desc& d, const FfnBwdPointers& p, hipStream_t s) {
  const i64 n = d.rows * d.hidden;
  const bool two = grads_parts(d) == 2;
  T *dgate = (T*)p.workspace, *dup = dgate + n, *dgate2 = two ? dup + n : nullptr, *dup2 = two ? dgate2 + n : nullptr;
  float* part = (float*)((char*)p.workspace + grads_bytes(d));
  if (n > 0) {
    if (p.gate) {
      const i64 need = (n * (i64)sizeof(T) + 4095) / 4096, blocks = need < (1 << 22) ? need : 1 << 22;
      const dim3 grid((unsigned)blocks);
      const T *dh = (const T*)p.dh, *gate = (const T*)p.gate, *up = (const T*)p.up;
      if (two) hipLaunchKernelGGL((ffn_grad_kernel<T, ACT, true>), grid, dim3(256), 0, s, dh, gate, up, dgate, dup, n);
      else hipLaunchKernelGGL((ffn_grad_kernel<T, ACT, false>), grid, dim3(256), 0, s, dh, gate, up, dgate, dup, n);
    } else {
      FfnArgs a{d.rows, d.hidden, d.dim, {{p.x, d.dim}}, {{p.w_gate, d.dim}, {p.w_up, d.dim}}, 1, d.hidden, {dgate, dup, dgate2, dup2}, p.dh, 1, 1, nullptr};
      launch_gemm<T, true, true, EPI_GLU_BACK, ACT>(a, part, s);
    }
  }
  const bool want_dx = p.dx && n > 0;
  const FfnArgs x{d.rows, d.dim, d.hidden, {{dgate, d.hidden}, {dup, d.hidden}, {dgate2, d.hidden}, {dup2, d.hidden}},
                  {{p.w_gate, d.dim}, {p.w_up, d.dim}}, two ? 4 : 2, d.dim, {p.dx}, nullptr, 1, 1, nullptr};
  // both weights' gradients are one product
  FfnArgs w{d.hidden, d.dim, d.rows, {}, {{p.x, d.dim}, {p.x, d.dim}}, two ? 2 : 1, d.dim, {}, nullptr, 0, 1, nullptr};
  const auto weight = [&](const T* first, const T* second, void* out) {
    w.A[w.items * w.segs] = {first, d.hidden};
    if (two) w.A[w.items * w.segs + 1] = {second, d.hidden};
    w.C[w.items++] = out;
  };
  if (p.dw_gate) weight(dgate, dgate2, p.dw_gate);
  if (p.dw_up) weight(dup, dup2, p.dw_up);
  if (want_dx && w.items) {
    GemmPlan px, pw;
    if (grads_plan(shape_of<T, EPI_PLAIN, true>(x), shape_of<T, EPI_PLAIN, false>(w), px, pw)) return launch_grads<T>(x, w, px, pw, part, s);
  }
  if (want_dx) launch_gemm<T, true, false, EPI_PLAIN, 0>(x, part, s);
  if (w.items) launch_gemm<T, false, false, EPI_PLAIN, 0>(w, part, s);
}

}  // namespace

size_t ffn_fwd_workspace_bytes(const ssmvjp_ffn_desc& d) {
  const Shape p = shape_of(d.rows, d.hidden, d.dim, 1, 1, true, true, d.dtype == SSMVJP_BF16 ? 2 : 4);
  return part_bytes(p, gemm_plan(p).split);
}

// dgate and dup, then the parts: of the forward's products, and behind those of dx and the weights' gradients
size_t ffn_bwd_workspace_bytes(const ssmvjp_ffn_desc& d) {
  const size_t elem = d.dtype == SSMVJP_BF16 ? 2 : 4, fwd = most_part_bytes(shape_of(d.rows, d.hidden, d.dim, 1, 1, true, true, elem));
  const int parts = grads_parts(d);
  const size_t dx = most_part_bytes(shape_of(d.rows, d.dim, d.hidden, 2 * parts, 1, false, true, elem));
  // one weight's gradient may be asked for without the other
  const size_t one = most_part_bytes(shape_of(d.hidden, d.dim, d.rows, parts, 1, false, false, elem));
  const size_t both = most_part_bytes(shape_of(d.hidden, d.dim, d.rows, parts, 2, false, false, elem));
  const size_t grads = dx + (one > both ? one : both);
  return grads_bytes(d) + (fwd > grads ? fwd : grads);
}

hipError_t launch_ffn_fwd(const ssmvjp_ffn_desc& d, const FfnFwdPointers& p, hipStream_t stream) {
  const bool gelu = d.act == SSMVJP_ACT_GELU;
  if (d.dtype == SSMVJP_BF16) {
    if (gelu) ffn_fwd<bf16, SSMVJP_ACT_GELU>(d, p, stream);
    else ffn_fwd<bf16, SSMVJP_ACT_SILU>(d, p, stream);
  } else {
    if (gelu) ffn_fwd<float, SSMVJP_ACT_GELU>(d, p, stream);
    else ffn_fwd<float, SSMVJP_ACT_SILU>(d, p, stream);
  }
  return hipGetLastError();
}

hipError_t launch_ffn_bwd(const ssmvjp_ffn_desc& d, const FfnBwdPointers& p, hipStream_t stream) {
  const bool gelu = d.act == SSMVJP_ACT_GELU;
  if (d.dtype == SSMVJP_BF16) {
    if (gelu) ffn_bwd<bf16, SSMVJP_ACT_GELU>(d, p, stream);
    else ffn_bwd<bf16, SSMVJP_ACT_SILU>(d, p, stream);
  } else {
    if (gelu) ffn_bwd<float, SSMVJP_ACT_GELU>(d, p, stream);
    else ffn_bwd<float, SSMVJP_ACT_SILU>(d, p, stream);
  }
  return hipGetLastError();
}

}  // namespace ssmvjp
