// linear_scan.hip -- the linear recurrence with one state value per channel:
// whole sequences, their gradients, and one token on a pool of states.
//
//   log form:    a_t = exp(g_t),  u_t = x_t
//   gated form:  L_t = c softplus(decay) sigmoid(r_t), a_t = exp(-L_t),
//                u_t = m_t w_t x_t with m_t = sqrt(1 - a_t^2), w_t = sigmoid(i_t)
//   h_t = a_t h_{t-1} + u_t
// Adjoint, with l_t the gradient of h_t (l_t = dh_t + a_{t+1} l_{t+1}):
//   log form:    dx = l, dg = l a h_{t-1}
//   gated form:  dx = l m w, di = l m w x (1 - w),
//                E = L dJ/dL = l (w x a^2 (L/m) - L a h_{t-1}),
//                dr = E (1 - sigmoid(r)), ddecay = sigmoid(decay)/softplus(decay) sum E
// E is formed with L/m, which stays finite (sqrt(L/2)) where L and m go to zero.
//
// Both directions go over the data once.  A workgroup takes a tile of tokens of
// 64 or 128 channels; its eight waves hold consecutive rows of it in registers.
// A run of tokens acts on the state before it as h -> A h + H (A the product of
// its a), and such pairs combine in order; what a tile needs of the tiles before
// it in its sequence it takes from the pairs that they publish:
//   - every tile publishes its pair as soon as it has it, before it waits;
//   - the last tile of each group of GROUP tiles publishes the state behind it;
//   - a tile combines the state behind the group before its own with the pairs
//     of the tiles before it in its group, always these and in this order, so
//     that results do not depend on which tile ran when.
// Pairs and states are published as single 64- and 32-bit words past the L2s
// (device-scope atomics) over a filling that no published value has, so a value
// that is there is whole and no fence is needed.  The tiles of a channel slab
// are handed out by a counter in the order of the sequence: what a tile waits
// for was handed out before it, to a workgroup that is running.  A counter for
// every slab, since additions to one address take 11.5 ns each: one counter for
// all cost 47 of 118 us of the backward at b=2 T=4096 D=4096.
//
// The bytes are the bound, and in the gated form the coefficients beside them:
// six (backward seven) of an element's instructions are transcendental, each as
// long as four others.  Gated bf16 b=2 T=4096 D=4096: forward 60 us for 271 MB
// (vector units busy 0.59 of it), backward 108 us for 472 MB (0.63), where a copy
// at 5.2 TB/s takes 52 and 91.  Log form, 32771 packed tokens of 2560
// channels: 142 us for 671 MB; 123 where no tile waits, of 256 sequences of 128
// tokens 108.  Tiles of half as many tokens: 170 us, groups of 32 tiles: 150;
// three workgroups per CU of the gated form (80 registers) spill: 93 us.
#include <type_traits>

#include "common.cuh"
#include "delta_seq.cuh"
#include "kernels.h"

namespace ssmvjp {
namespace {

constexpr int NW = 8;         // waves of a workgroup
constexpr int FWD_ROWS = 16;  // rows of a wave: tiles of 128 tokens forward ...
constexpr int BWD_ROWS = 8;   // ... and of 64 backward, which holds more of each
constexpr int GROUP = 16;     // tiles between published states

typedef unsigned long long u64;
constexpr u64 NO_PAIR = ~0ull;
constexpr unsigned NO_STATE = ~0u;
// Polls before a wave gives up and goes on with NaN: seconds, where a wait lasts microseconds.
constexpr int POLLS = 1 << 22;

struct ScanArgs {
  const int* off;         // borders of packed sequences, or NULL
  i64 nseq, T, per, D;    // per: tiles of one sequence (off == NULL)
  i64 ntiles;             // tile slots
  int nslab;              // channel slabs
  bool chain;             // a sequence may have more than one tile
  float c;
  const void *x, *gate, *igate;
  const float *decay, *h0;
  void* h;
  float *h_final, *ckpt;
  // backward
  const float* kept;
  const void* dh;
  const float* dh_final;
  void *dx, *dgate, *digate;
  float *part, *dh0;
  // what tiles tell each other
  u64* pairs;        // [ntiles][D]
  unsigned* states;  // [ntiles / GROUP + 1][D]
  unsigned* tickets; // one every TICKET words
};

constexpr int TICKET = 32;

// Tile slots of N tokens each: a packed sequence s owns those from start / N + s, which never meet the next one's
// (see delta_seq.cuh).  Every border counts as the largest up to it: a tile waits for others, so that each slot has to
// belong to one sequence whatever the borders hold.
struct Span {
  i64 seq, start, end;
};
// the sequence of a packed slot (-1: it lies before all); called by whole waves
template <int N>
__device__ __forceinline__ Span of_slot(const ScanArgs& a, i64 slot, int lane) {
  const auto at = [](int v, int l) { return __builtin_amdgcn_readlane(v, l); };
  int most = 0;  // of the borders before this round's
  for (i64 s0 = 0;; s0 += 64) {
    const i64 i = s0 + lane;
    i64 o = i <= a.nseq ? a.off[i] : 0;
    o = o < 0 ? 0 : o > a.T ? a.T : o;
    int e = (int)o;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int up = __shfl_up(e, d);
      e = lane >= d && up > e ? up : e;
    }
    e = e > most ? e : most;
    // those whose first slot is not behind `slot`; border nseq is none's
    const int n = __popcll(__ballot(i < a.nseq && (i64)e / N + i <= slot));
    if (n < 64) return {s0 + n - 1, n > 0 ? at(e, n > 0 ? n - 1 : 0) : most, at(e, n)};
    most = at(e, 63);
  }
}

struct Tile {
  i64 seq, start, len;  // the sequence
  i64 slot0, slot, j, n;  // its first slot, this one, tile j of n
};

__device__ __forceinline__ i64 uniform(i64 v) {
  return (i64)(((u64)(unsigned)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32) |
               (unsigned)__builtin_amdgcn_readfirstlane((int)v));
}

// tile number `o` in the order of hand-out (REV: from the ends of the sequences); false: a slot without tokens
template <int N, bool REV>
__device__ __forceinline__ bool find_tile(const ScanArgs& a, i64 o, int lane, Tile& t) {
  if (!a.off) {
    const i64 j = o / a.nseq;
    t.seq = o - j * a.nseq;
    t.j = REV ? a.per - 1 - j : j;
    t.n = a.per;
    t.start = t.seq * a.T;
    t.len = a.T;
    t.slot0 = t.seq * a.per;
    t.slot = t.slot0 + t.j;
    return true;
  }
  t.slot = REV ? a.ntiles - 1 - o : o;
  const Span sp = of_slot<N>(a, t.slot, lane);
  t.seq = uniform(sp.seq);
  if (t.seq < 0) return false;
  t.start = uniform(sp.start);
  t.len = uniform(sp.end) - t.start;
  t.slot0 = t.start / N + t.seq;
  t.j = t.slot - t.slot0;
  t.n = (t.len + N - 1) / N;
  return t.j >= 0 && t.j < t.n;
}

__device__ __forceinline__ float sigmoid_hw(float z) { return __builtin_amdgcn_rcpf(1.0f + exp_hw(-z)); }

// per channel: c softplus(decay), and sigmoid(decay) / softplus(decay) (1 where both go to exp(decay)).  The rate stays
// finite with its factor log2(e): it meets the 0 of a shut gate, and that of a = 0 in the gradients.
constexpr float RATE_MAX = 2.3e38f;
__device__ __forceinline__ float decay_rate(float c, float z) {
  const float rate = c * softplus_hw(z);
  return rate > RATE_MAX ? RATE_MAX : rate;
}
__device__ __forceinline__ float decay_slope(float z) { return z < -16.0f ? 1.0f : sigmoid_f(z) / softplus_f(z); }

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float MIN_NORMAL = 1.17549435e-38f;  // the reciprocals take denormals as zeros

struct Token {
  float a, u;       // h = a h + u
  float sr, w, mw;  // gated form: sigmoid(r), w, m w
};

// A state that a channel keeps over thousands of tokens adds up what each a_t near one has lost, and v_exp_f32 may be a
// step beside it.  There a is one rounding of 1 + (e^g - 1), by the series of e^g - 1: final states of thousands of tokens
// come out four times nearer.  Behind g^4 / 24 it leaves out at most 8e-9, an eighth of a step of a.
__device__ __forceinline__ float log_gate(float g) {
  const float p = fmaf(g, fmaf(g, fmaf(g, 1.0f / 24, 1.0f / 6), 0.5f), 1.0f);
  return fabsf(g) < 0.0625f ? fmaf(g, p, 1.0f) : exp_hw(g);
}

// rate2: log2(e) c softplus(decay).  With s = 1 - a, by its series where it is small (up to L^5 / 120, which leaves out
// 4e-8 of it at most), m^2 = 1 - a^2 = s (1 + a) loses nothing where a is near one.
// top: the series' last coefficient, in a register that the caller keeps.
constexpr float Y = LN2;
__device__ __forceinline__ float series_top() {
  float c5 = Y * Y * Y * Y * Y / 120;
  asm volatile("" : "+v"(c5));
  return c5;
}
__device__ __forceinline__ Token gated_token(float x, float r, float i, float rate2, float top) {
  Token t;
  t.sr = sigmoid_hw(r);
  t.w = sigmoid_hw(i);
  const float lc = rate2 * t.sr, e = __builtin_amdgcn_exp2f(-lc);
  constexpr float c2 = -Y * Y / 2, c3 = Y * Y * Y / 6, c4 = -Y * Y * Y * Y / 24;
  const float p = fmaf(lc, fmaf(lc, fmaf(lc, fmaf(lc, top, c4), c3), c2), Y);
  const bool near = lc < 0.125f / Y;
  const float s = near ? lc * p : 1.0f - e;
  t.a = near ? fmaf(-lc, p, 1.0f) : e;
  t.mw = __builtin_amdgcn_sqrtf(fmaf(s, t.a, s)) * t.w;
  t.u = t.mw * x;
  return t;
}

// A h + u.  GROWS: A may have overflowed (log gates above 0); a state of zero stays out of that.
template <bool GROWS>
__device__ __forceinline__ float apply(float A, float h, float u) {
  return GROWS && h == 0.0f ? u : fmaf(A, h, u);
}

// ---------------------------------------------------------------------------
// rows of V channels per lane
// ---------------------------------------------------------------------------
// a lane's values of one row as they lie in memory (two of bf16 in one register)
template <typename T, int V>
struct Raw {
  T v[V];
  __device__ __forceinline__ float get(int i) const { return (float)v[i]; }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = (T)0.0f;
  }
  __device__ __forceinline__ void pin() {}
};
template <>
struct Raw<bf16, 2> {
  unsigned v;
  __device__ __forceinline__ float get(int i) const { return __uint_as_float(i ? v & 0xffff0000u : v << 16); }
  __device__ __forceinline__ void clear() { v = 0u; }
  // from here on the values are taken out of the word again: they are not kept beside it
  __device__ __forceinline__ void pin() { asm volatile("" : "+v"(v)); }
};
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_raw(const T* row, unsigned off) {
  Raw<T, V> r;
  __builtin_memcpy(&r, __builtin_assume_aligned((const char*)row + off * (unsigned)sizeof(T), V * sizeof(T)), V * sizeof(T));
  return r;
}
// the same from row `row` of a workgroup's rows: the row's offset in a scalar register, nothing to add per lane.
// STREAM: past the caches' normal order, for what is read once
template <typename T, int V, bool STREAM>
__device__ __forceinline__ Raw<T, V> load_row(brsrc rs, unsigned off, unsigned row) {
  constexpr int B = V * (int)sizeof(T), AUX = STREAM ? 2 : 0;  // nt
  Raw<T, V> r;
  if constexpr (B == 2) {
    const unsigned short w = __builtin_amdgcn_raw_buffer_load_b16(rs, (int)(off * sizeof(T)), (int)row, AUX);
    __builtin_memcpy(&r, &w, B);
  } else if constexpr (B == 4) {
    const unsigned w = __builtin_amdgcn_raw_buffer_load_b32(rs, (int)(off * sizeof(T)), (int)row, AUX);
    __builtin_memcpy(&r, &w, B);
  } else {
    const auto w = __builtin_amdgcn_raw_buffer_load_b64(rs, (int)(off * sizeof(T)), (int)row, AUX);
    __builtin_memcpy(&r, &w, B);
  }
  return r;
}
// rows of T from element e on; what is read there is the caller's to keep inside
template <typename T>
__device__ __forceinline__ brsrc rows_at(const void* p, i64 e) {
  return make_rsrc((const T*)p + e, 0x7fffffffu);
}
template <int V>
__device__ __forceinline__ void store_raw(bf16* row, unsigned off, const float (&v)[V]) {
  char* p = (char*)row + off * 2u;
  if constexpr (V == 2) *(unsigned*)p = pk_bf16(v[0], v[1]);
  else *(bf16*)p = (bf16)v[0];
}
template <int V>
__device__ __forceinline__ void store_raw(float* row, unsigned off, const float (&v)[V]) {
  char* p = (char*)row + off * 4u;
  if constexpr (V == 2) *(float2*)p = make_float2(v[0], v[1]);
  else *(float*)p = v[0];
}

// ---------------------------------------------------------------------------
// what tiles publish
// ---------------------------------------------------------------------------
__device__ __forceinline__ float plain_nan(float v) { return v == v ? v : __uint_as_float(0x7fc00000u); }

__device__ __forceinline__ void put_pair(u64* p, float A, float H) {
  const u64 v = (u64)__float_as_uint(plain_nan(A)) | ((u64)__float_as_uint(plain_nan(H)) << 32);
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void put_state(unsigned* p, float h) {
  __hip_atomic_store(p, __float_as_uint(plain_nan(h)), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename W, W NONE>
__device__ __forceinline__ W await(const W* p) {
  W v = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (int n = 0; v == NONE && n < POLLS; ++n) {
    __builtin_amdgcn_s_sleep(1);
    v = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  return v;  // NONE is a NaN
}

struct Pair {
  float A, H;
};

// Everything between a workgroup's segments and its sequence's other tiles.  Waves are numbered `w` in the order of
// the recurrence (REV: the last rows first), tiles `k` likewise.
template <int V, bool GROWS>
struct Chain {
  Pair (*seg)[V][64];   // [NW]: the waves' segments
  Pair (*look)[V][64];  // [NW]: what the waves found of the tiles before
  float (*base)[64];    // the state behind the group before

  // the state before this wave's rows.  first: the state before the sequence
  __device__ __forceinline__ void enter(const ScanArgs& a, i64 slot, int step, i64 k, i64 n, int w, int lane, i64 ch0,
                                        unsigned coff, bool mine, const float (&first)[V], float (&h)[V]) {
    // (1) this tile's pair; the last tile's is not needed, and a group's last one publishes a state instead
    const int back = (int)(k % GROUP);
    if (w == 0 && k + 1 < n && back != GROUP - 1) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        Pair t = seg[0][v][lane];
#pragma unroll
        for (int i = 1; i < NW; ++i) {
          const Pair s = seg[i][v][lane];
          t.H = apply<GROWS>(s.A, t.H, s.H);
          t.A *= s.A;
        }
        if (mine) put_pair(a.pairs + slot * a.D + ch0 + coff + v, t.A, t.H);
      }
    }
    // (2) the tiles before it in its group, two per wave; and the state behind the group before
    if (k > 0) {
      Pair f[V];
#pragma unroll
      for (int v = 0; v < V; ++v) f[v] = {1.0f, 0.0f};
      constexpr int EACH = GROUP / NW;
#pragma unroll
      for (int i = 0; i < EACH; ++i) {
        const int b = w * EACH + i;
        if (b < back) {
          const u64* p = a.pairs + (slot - (i64)step * (back - b)) * a.D + ch0 + coff;
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const u64 q = await<u64, NO_PAIR>(p + v);
            const float A = __uint_as_float((unsigned)q);
            f[v].H = apply<GROWS>(A, f[v].H, __uint_as_float((unsigned)(q >> 32)));
            f[v].A *= A;
          }
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) look[w][v][lane] = f[v];
      if (w == NW - 1 && k >= GROUP) {
        const unsigned* p = a.states + (slot - (i64)step * (back + 1)) / GROUP * a.D + ch0 + coff;
#pragma unroll
        for (int v = 0; v < V; ++v) base[v][lane] = __uint_as_float(await<unsigned, NO_STATE>(p + v));
      }
      __syncthreads();
    }
    // (3) in order
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[v] = k >= GROUP ? base[v][lane] : first[v];
      if (k > 0)
        for (int i = 0; i < NW; ++i) h[v] = apply<GROWS>(look[i][v][lane].A, h[v], look[i][v][lane].H);
      for (int i = 0; i < w; ++i) h[v] = apply<GROWS>(seg[i][v][lane].A, h[v], seg[i][v][lane].H);
    }
  }
  // the state behind the last wave's rows, where a group ends
  __device__ __forceinline__ void leave(const ScanArgs& a, i64 slot, i64 k, i64 n, int w, i64 ch0, unsigned coff, bool mine,
                                        const float (&h)[V]) {
    if (w == NW - 1 && k + 1 < n && k % GROUP == GROUP - 1 && mine)
#pragma unroll
      for (int v = 0; v < V; ++v) put_state(a.states + slot / GROUP * a.D + ch0 + coff + v, h[v]);
  }
};

template <int N, bool REV>
__device__ __forceinline__ bool take_tile(const ScanArgs& a, int lane, unsigned* shared, Tile& t, int& slab) {
  unsigned i = blockIdx.x / (unsigned)a.nslab;
  slab = (int)(blockIdx.x - i * (unsigned)a.nslab);
  if (a.chain) {
    // from the filling, ~0, on
    if (threadIdx.x == 0)
      *shared = __hip_atomic_fetch_add(a.tickets + (i64)slab * TICKET, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1u;
    __syncthreads();
    i = (unsigned)__builtin_amdgcn_readfirstlane((int)*shared);
  }
  return find_tile<N, REV>(a, i, lane, t);
}

template <typename T, bool GATED, int V, bool STREAM>
__global__ void __launch_bounds__(64 * NW) scan_fwd_kernel(ScanArgs a) {
  constexpr int R = FWD_ROWS, N = R * NW;
  __shared__ Pair seg[NW][V][64], look[NW][V][64];
  __shared__ float base[V][64];
  __shared__ unsigned number;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Tile t;
  int slab;
  if (!take_tile<N, false>(a, lane, &number, t, slab)) return;
  const i64 ch0 = (i64)slab * 64 * V, t0 = t.j * N + w * R;
  const bool mine = ch0 + lane * V < a.D;
  const unsigned coff = mine ? lane * V : 0;
  const int rows = t0 >= t.len ? 0 : t.len - t0 < R ? (int)(t.len - t0) : R;
  const i64 at = (t.start + t0) * a.D + ch0;

  typedef Raw<T, V> raw;
  raw x[R];
  float ai[R][V], ui[GATED ? R : 1][V];  // h = ai h + ui (log form: ui is x)
  float first[V], rate[V];
  Pair f[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    first[v] = a.h0 ? a.h0[t.seq * a.D + ch0 + coff + v] : 0.0f;
    if constexpr (GATED) rate[v] = a.decay[ch0 + coff + v];
    f[v] = {1.0f, 0.0f};
  }
  auto scan = [&](auto full) {
    raw r[GATED ? R : 1], ig[GATED ? R : 1];
    Raw<float, V> g[GATED ? 1 : R];
    const brsrc bx = rows_at<T>(a.x, at), bg = GATED ? rows_at<T>(a.gate, at) : rows_at<float>(a.gate, at);
    const brsrc bi = rows_at<T>(GATED ? a.igate : a.x, at);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const unsigned row = (unsigned)(full || i < rows ? i : rows - 1) * (unsigned)a.D, o = row * (unsigned)sizeof(T);
      if constexpr (GATED) {
        r[i] = load_row<T, V, STREAM>(bg, coff, o);
        ig[i] = load_row<T, V, STREAM>(bi, coff, o);
      } else {
        g[i] = load_row<float, V, STREAM>(bg, coff, row * 4u);
      }
      x[i] = load_row<T, V, STREAM>(bx, coff, o);
    }
    const float top = GATED ? series_top() : 0.0f;
    if constexpr (GATED)
#pragma unroll
      for (int v = 0; v < V; ++v) rate[v] = LOG2E * decay_rate(a.c, rate[v]);
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float u;
        if constexpr (GATED) {
          const Token k = gated_token(x[i].get(v), r[i].get(v), ig[i].get(v), rate[v], top);
          ai[i][v] = k.a;
          ui[i][v] = u = k.u;
        } else {
          ai[i][v] = log_gate(g[i].v[v]);
          u = x[i].get(v);
        }
        if (full || i < rows) {
          f[v].A *= ai[i][v];
          f[v].H = fmaf(ai[i][v], f[v].H, u);
        }
      }
      x[i].pin();
      // two tokens at a time, in the order of their loads (left to the compiler, which takes a later token's x first, the
      // gated form waits for most of the loads at once: 67 us at b=2 T=4096 D=4096 instead of 62)
      if (GATED && i % 2) __builtin_amdgcn_sched_barrier(0);
    }
  };
  if (rows == R) scan(std::true_type{});
  else if (rows > 0) scan(std::false_type{});
#pragma unroll
  for (int v = 0; v < V; ++v) seg[w][v][lane] = f[v];
  __syncthreads();
  float h[V], last[V];
  Chain<V, !GATED> chain{seg, look, base};
  chain.enter(a, t.slot, 1, t.j, t.n, w, lane, ch0, coff, mine, first, h);
  // the state behind the tile first: the next group waits for it
#pragma unroll
  for (int v = 0; v < V; ++v) last[v] = apply<!GATED>(f[v].A, h[v], f[v].H);
  chain.leave(a, t.slot, t.j, t.n, w, ch0, coff, mine, last);
  if (!mine) return;
  if (a.ckpt && rows > 0 && w * R % DCH == 0) {
    const i64 row = (a.off ? t.start / DCH + t.seq : t.seq * ((a.T + DCH - 1) / DCH)) + t0 / DCH;
#pragma unroll
    for (int v = 0; v < V; ++v) a.ckpt[row * a.D + ch0 + coff + v] = h[v];
  }
  if (a.h_final && w == NW - 1 && t.j == t.n - 1)
#pragma unroll
    for (int v = 0; v < V; ++v) a.h_final[t.seq * a.D + ch0 + coff + v] = last[v];
  if (!a.h) return;
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (i < rows) {
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = fmaf(ai[i][v], h[v], GATED ? ui[GATED ? i : 0][v] : x[i].get(v));
      store_raw((T*)a.h + at + (i64)i * a.D, coff, h);
    }
}

// A wave's rows: forward from the state before the tile (kept by the forward pass), backward from the gradient of the
// state behind it.  b_t = a_t l_t, the gradient that reaches h_{t-1}, obeys b_t = a_t b_{t+1} + a_t dh_t.
template <typename T, bool GATED, int V, bool STREAM>
__global__ void __launch_bounds__(64 * NW) scan_bwd_kernel(ScanArgs a) {
  constexpr int R = BWD_ROWS, N = R * NW;
  static_assert(N == DCH, "a tile of the backward starts at a kept state");
  __shared__ Pair seg[NW][V][64], look[NW][V][64], fseg[NW][V][64];
  __shared__ float base[V][64];
  __shared__ unsigned number;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Tile t;
  int slab;
  if (!take_tile<N, true>(a, lane, &number, t, slab)) {
    // a slot without tokens has no part in the sum over the tokens
    const i64 ch = (i64)slab * 64 * V + threadIdx.x;
    if (GATED && threadIdx.x < 64 * V && ch < a.D) a.part[t.slot * a.D + ch] = 0.0f;
    return;
  }
  const i64 ch0 = (i64)slab * 64 * V, t0 = t.j * N + w * R;
  const bool mine = ch0 + lane * V < a.D;
  const unsigned coff = mine ? lane * V : 0;
  const int rows = t0 >= t.len ? 0 : t.len - t0 < R ? (int)(t.len - t0) : R;
  const i64 at = (t.start + t0) * a.D + ch0;
  typedef Raw<T, V> raw;
  raw x[R], dh[R];
  float ai[R][V];                                                                    // h = ai h + u
  float sr[GATED ? R : 1][V], wi[GATED ? R : 1][V], mw[GATED ? R : 1][V];
  float first[V], rate[V], hin[V];
  Pair f[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    first[v] = a.dh_final ? a.dh_final[t.seq * a.D + ch0 + coff + v] : 0.0f;
    hin[v] = a.kept[t.slot * a.D + ch0 + coff + v];
    if constexpr (GATED) rate[v] = a.decay[ch0 + coff + v];
    f[v] = {1.0f, 0.0f};
  }
  auto load = [&](auto full) {
    raw r[GATED ? R : 1], ig[GATED ? R : 1];
    Raw<float, V> g[GATED ? 1 : R];
    const brsrc bx = rows_at<T>(a.x, at), bg = GATED ? rows_at<T>(a.gate, at) : rows_at<float>(a.gate, at);
    const brsrc bi = rows_at<T>(GATED ? a.igate : a.x, at), bd = rows_at<T>(a.dh, at);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const unsigned row = (unsigned)(full || i < rows ? i : rows - 1) * (unsigned)a.D, o = row * (unsigned)sizeof(T);
      if constexpr (GATED) {
        r[i] = load_row<T, V, STREAM>(bg, coff, o);
        ig[i] = load_row<T, V, STREAM>(bi, coff, o);
      } else {
        g[i] = load_row<float, V, STREAM>(bg, coff, row * 4u);
      }
      x[i] = load_row<T, V, STREAM>(bx, coff, o);
      dh[i] = load_row<T, V, STREAM>(bd, coff, o);
    }
    const float top = GATED ? series_top() : 0.0f;
    if constexpr (GATED)
#pragma unroll
      for (int v = 0; v < V; ++v) rate[v] = LOG2E * decay_rate(a.c, rate[v]);
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float u;
        if constexpr (GATED) {
          const Token k = gated_token(x[i].get(v), r[i].get(v), ig[i].get(v), rate[v], top);
          ai[i][v] = k.a; u = k.u; sr[i][v] = k.sr; wi[i][v] = k.w; mw[i][v] = k.mw;
        } else {
          ai[i][v] = log_gate(g[i].v[v]);
          u = x[i].get(v);
        }
        if (!full && i >= rows) ai[i][v] = 1.0f, u = 0.0f;
        f[v].A *= ai[i][v];
        f[v].H = fmaf(ai[i][v], f[v].H, u);
      }
      if (!full && i >= rows) dh[i].clear();
      x[i].pin();
    }
  };
  if (rows == R) {
    load(std::true_type{});
  } else if (rows > 0) {
    load(std::false_type{});
  } else {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      x[i].clear();
      dh[i].clear();
#pragma unroll
      for (int v = 0; v < V; ++v) {
        ai[i][v] = 1.0f;
        if constexpr (GATED) sr[i][v] = wi[i][v] = mw[i][v] = 0.0f;
      }
    }
  }
  const int wr = NW - 1 - w;  // the waves in the order of the adjoint
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float B = 0.0f;
#pragma unroll
    for (int i = R - 1; i >= 0; --i) B = ai[i][v] * (B + dh[i].get(v));
    fseg[w][v][lane] = f[v];
    seg[wr][v][lane] = {f[v].A, B};
  }
#pragma unroll
  for (int i = 0; i < R; ++i) dh[i].pin();
  __syncthreads();
  float b[V];
  Chain<V, !GATED> chain{seg, look, base};
  const i64 k = t.n - 1 - t.j;
  chain.enter(a, t.slot, -1, k, t.n, wr, lane, ch0, coff, mine, first, b);
  float sum[V], prev[R][V];  // h_{t-1}
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float h = hin[v];
    for (int i = 0; i < w; ++i) h = apply<!GATED>(fseg[i][v][lane].A, h, fseg[i][v][lane].H);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      prev[i][v] = h;
      h = fmaf(ai[i][v], h, GATED ? mw[GATED ? i : 0][v] * x[i].get(v) : x[i].get(v));
    }
    sum[v] = 0.0f;
  }
#pragma unroll
  for (int i = R - 1; i >= 0; --i) {
    float ox[V], og[V], oi[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float l = dh[i].get(v) + b[v], hp = prev[i][v];
      b[v] = ai[i][v] * l;
      if constexpr (GATED) {
        const float La = LN2 * rate[v] * sr[i][v] * ai[i][v], wx = wi[i][v] * x[i].get(v), lm = l * mw[i][v];
        const float w_m = wi[i][v] * (wi[i][v] * __builtin_amdgcn_rcpf(fmaxf(mw[i][v], MIN_NORMAL)));  // w / m, finite
        const float E = l * fmaf(La * w_m, ai[i][v] * x[i].get(v), -La * hp);
        ox[v] = lm;
        oi[v] = lm * (x[i].get(v) - wx);
        og[v] = E * (1.0f - sr[i][v]);
        if (i < rows) sum[v] += E;
      } else {
        ox[v] = l;
        og[v] = b[v] * hp;
      }
    }
    if (i < rows && mine) {
      const i64 e = at + (i64)i * a.D;
      store_raw((T*)a.dx + e, coff, ox);
      if constexpr (GATED) {
        store_raw((T*)a.dgate + e, coff, og);
        store_raw((T*)a.digate + e, coff, oi);
      } else {
        store_raw((float*)a.dgate + e, coff, og);
      }
    }
  }
  chain.leave(a, t.slot, k, t.n, wr, ch0, coff, mine, b);
  if (a.dh0 && w == 0 && t.j == 0 && mine)
#pragma unroll
    for (int v = 0; v < V; ++v) a.dh0[t.seq * a.D + ch0 + coff + v] = b[v];
  if constexpr (GATED) {
    // fseg and look are read no more behind this barrier
    __syncthreads();
    float(*sums)[V][64] = (float(*)[V][64])fseg;
#pragma unroll
    for (int v = 0; v < V; ++v) sums[w][v][lane] = sum[v];
    __syncthreads();
    if (w == 0 && mine)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float s = sums[0][v][lane];
#pragma unroll
        for (int i = 1; i < NW; ++i) s += sums[i][v][lane];
        a.part[t.slot * a.D + ch0 + coff + v] = s;
      }
  }
}

// Before a call whose tiles wait for each other: the filling of what they publish, and the counter.  Rows of ckpt that no
// token has: zeros.  Sequences without tokens, which have no tile: their final state (`to`) is their first (`from`); which
// those are goes by the rule of the tiles (of_slot).  That is the first `first` workgroups', a wave's for INIT_CHANNELS of a
// sequence (behind the filling and 256 a wave, 7 packed sequences of 3001 x 1001 float32 backward take 29.7 us instead
// of 28.8).
constexpr int INIT_CHANNELS = 64;
__global__ void __launch_bounds__(256) scan_init_kernel(u64* pairs, i64 words, DeltaSeqs seqs, i64 D, const float* from, float* to,
                                                        unsigned first, float* clear, i64 nclear) {
  if (blockIdx.x < first) {
    const int lane = threadIdx.x & 63;
    const unsigned per = (unsigned)((D + INIT_CHANNELS - 1) / INIT_CHANNELS);
    const unsigned wave = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (unsigned i = wave; i < (unsigned)seqs.nseq * per; i += first * 4) {
      const unsigned s = i / per;
      if (seqs.off ? !seqs.risen_empty(s, lane) : seqs.T > 0) continue;
      const i64 ch = (i64)(i - s * per) * INIT_CHANNELS + lane;
      if (ch < D) to[s * D + ch] = from ? from[s * D + ch] : 0.0f;
    }
    return;
  }
  const i64 i0 = (i64)(blockIdx.x - first) * 256 + threadIdx.x, step = (i64)(gridDim.x - first) * 256;
  for (i64 i = i0; i < words; i += step) pairs[i] = NO_PAIR;
  for (i64 i = i0; i < nclear; i += step) clear[i] = 0.0f;
}

// ddecay = slope * sum over the tiles: 16 runs of tiles per channel, each in order, then the runs in order
__global__ void __launch_bounds__(1024) decay_sum_kernel(const float* part, i64 n, i64 D, const float* decay, float* out) {
  __shared__ float runs[16][64];
  const i64 ch = (i64)blockIdx.x * 64 + (threadIdx.x & 63), each = (n + 15) / 16;
  const int run = threadIdx.x >> 6;
  float sum = 0.0f;
  if (ch < D)
#pragma unroll 8
    for (i64 i = run * each; i < n && i < (run + 1) * each; ++i) sum += part[i * D + ch];
  runs[run][threadIdx.x & 63] = sum;
  __syncthreads();
  if (run || ch >= D) return;
  for (int i = 1; i < 16; ++i) sum += runs[i][threadIdx.x];
  out[ch] = n > 0 ? sum * decay_slope(decay[ch]) : 0.0f;
}

struct StepArgs {
  i64 nslots, D, nblk;
  float c;
  const void *x, *gate, *igate;
  const float* decay;
  float* state;
  const int* slots;
  void* h;
};

// V channels per thread.  The state of the named slot is on its way while the wave looks through the earlier requests.
// Two trips to memory and the launch are what it takes: 2.8 us for one request of 4096 channels, 6.1 for 256 (17 MB).
template <typename T, bool GATED, int V>
__global__ void __launch_bounds__(256) scan_step_kernel(StepArgs a) {
  const i64 req = blockIdx.x / a.nblk, ch = ((blockIdx.x % a.nblk) * 256 + threadIdx.x) * V;
  const bool mine = ch < a.D;
  const unsigned coff = mine ? (unsigned)ch : 0;
  const i64 e = req * a.D;
  i64 slot = a.slots ? a.slots[req] : req;
  const bool in = slot >= 0 && slot < a.nslots;
  float* p = a.state + (in ? slot : 0) * a.D + coff;
  Raw<T, V> x = load_raw<T, V>((const T*)a.x + e, coff), r, ig;
  Raw<float, V> g;
  if constexpr (GATED) {
    r = load_raw<T, V>((const T*)a.gate + e, coff);
    ig = load_raw<T, V>((const T*)a.igate + e, coff);
  } else {
    g = load_raw<float, V>((const float*)a.gate + e, coff);
  }
  float s[V], o[V];
#pragma unroll
  for (int v = 0; v < V; ++v) s[v] = a.nslots > 0 ? p[v] : 0.0f;
  bool dead = !in;
  if (a.slots && in) {
    bool taken = false;
#pragma unroll 4
    for (i64 j = threadIdx.x & 63; j < req; j += 64) taken |= a.slots[j] == (int)slot;
    dead = __any(taken);
  }
  if (!mine) return;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float ai, u;
    if constexpr (GATED) {
      const Token k = gated_token(x.get(v), r.get(v), ig.get(v), LOG2E * decay_rate(a.c, a.decay[coff + v]), series_top());
      ai = k.a;
      u = k.u;
    } else {
      ai = log_gate(g.v[v]);
      u = x.get(v);
    }
    o[v] = dead ? 0.0f : fmaf(ai, s[v], u);
    if (!dead) p[v] = o[v];
  }
  store_raw((T*)a.h + e, coff, o);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
i64 tile_slots(const ssmvjp_linear_scan_desc& d, int n) {
  return d.packed ? d.seqlen / n + d.batch : d.batch * ((d.seqlen + n - 1) / n);
}
// a sequence may have more than one tile
bool chained(const ssmvjp_linear_scan_desc& d, int n) { return d.seqlen > n; }

i64 round64(i64 n) { return (n + 63) / 64 * 64; }
// words of 8 bytes: the pairs, the states, the counters
i64 chain_words(const ssmvjp_linear_scan_desc& d, int n) {
  if (!chained(d, n)) return 0;
  const i64 slots = tile_slots(d, n);
  return slots * d.dim + ((slots / GROUP + 1) * d.dim + 1) / 2 + (d.dim + 63) / 64 * (TICKET / 2);
}

void set_chain(const ssmvjp_linear_scan_desc& d, int n, void* workspace, ScanArgs& a) {
  a.ntiles = tile_slots(d, n);
  a.per = (d.seqlen + n - 1) / n;
  a.chain = chained(d, n);
  if (!a.chain) return;
  a.pairs = (u64*)workspace;
  a.states = (unsigned*)(a.pairs + a.ntiles * d.dim);
  a.tickets = (unsigned*)(a.pairs + chain_words(d, n) - (d.dim + 63) / 64 * (TICKET / 2));
}

void launch_init(const ScanArgs& a, void* base, i64 words, const float* from, float* to, float* clear, i64 nclear, hipStream_t s) {
  const auto blocks = [](i64 n, i64 each) { return (unsigned)((n + each - 1) / each < 2048 ? (n + each - 1) / each : 2048); };
  const unsigned first = to ? blocks(a.nseq * ((a.D + INIT_CHANNELS - 1) / INIT_CHANNELS), 4) : 0;
  const unsigned grid = first + blocks(words > nclear ? words : nclear, 1024);
  if (grid)
    hipLaunchKernelGGL(scan_init_kernel, dim3(grid), dim3(256), 0, s, (u64*)base, words, DeltaSeqs{a.off, a.nseq, a.T, a.per}, a.D, from,
                       to, first, clear, nclear);
}

template <typename T, bool GATED, int V, bool BWD, bool STREAM>
void launch_tiles(ScanArgs& a, hipStream_t s) {
  a.nslab = (int)((a.D + 64 * V - 1) / (64 * V));
  const dim3 grid((unsigned)(a.ntiles * a.nslab));
  if constexpr (BWD) hipLaunchKernelGGL((scan_bwd_kernel<T, GATED, V, STREAM>), grid, dim3(64 * NW), 0, s, a);
  else hipLaunchKernelGGL((scan_fwd_kernel<T, GATED, V, STREAM>), grid, dim3(64 * NW), 0, s, a);
}

// Inputs of more than this are read with the streaming hint: what was written just before is then out of the caches
// anyway (one sequence of D=4096 gated, backward: 240 -> 228 us for 512 MB read; 63.8 -> 64.5 for 128 MB, 74.1 -> 77.0
// for 93 MB where the states are formed again first and the second pass finds the inputs in the caches).
constexpr i64 STREAM_BYTES = 128 << 20;

// Two channels per lane where every row starts at a multiple of two elements: 4 bytes of bf16 a load.
template <typename T, bool GATED, bool BWD>
void launch_wide(ScanArgs& a, hipStream_t s) {
  const void* big[] = {a.x, a.igate, a.h, a.dh, a.dx, a.digate};
  const void* gates[] = {a.gate, a.dgate};
  bool two = a.D % 2 == 0;
  for (const void* p : big) two &= (uintptr_t)p % (2 * sizeof(T)) == 0;
  for (const void* p : gates) two &= (uintptr_t)p % (2 * (GATED ? sizeof(T) : 4)) == 0;
  const i64 read = (a.off ? a.T : a.nseq * a.T) * a.D * (i64)((GATED ? 3 * sizeof(T) : sizeof(T) + 4) + (BWD ? sizeof(T) : 0));
  const bool stream = read > STREAM_BYTES;
  if (!two) launch_tiles<T, GATED, 1, BWD, false>(a, s);
  else if (stream) launch_tiles<T, GATED, 2, BWD, true>(a, s);
  else launch_tiles<T, GATED, 2, BWD, false>(a, s);
}

template <typename T, bool GATED, int V>
void launch_step_v(StepArgs& a, i64 batch, hipStream_t s) {
  a.nblk = (a.D + 256 * V - 1) / (256 * V);
  hipLaunchKernelGGL((scan_step_kernel<T, GATED, V>), dim3((unsigned)(batch * a.nblk)), dim3(256), 0, s, a);
}
template <typename T, bool GATED>
void launch_step(StepArgs& a, i64 batch, hipStream_t s) {
  const bool two = a.D % 2 == 0 && (uintptr_t)a.x % (2 * sizeof(T)) == 0 && (uintptr_t)a.h % (2 * sizeof(T)) == 0 &&
                   (uintptr_t)a.igate % (2 * sizeof(T)) == 0 && (uintptr_t)a.gate % (2 * (GATED ? sizeof(T) : 4)) == 0;
  if (two) launch_step_v<T, GATED, 2>(a, batch, s);
  else launch_step_v<T, GATED, 1>(a, batch, s);
}

template <bool BWD>
void launch_scan(const ssmvjp_linear_scan_desc& d, ScanArgs& a, hipStream_t s) {
  if (a.ntiles == 0 || d.seqlen == 0 || d.batch == 0) return;
  const bool gated = d.form == SSMVJP_SCAN_GATED;
  if (d.dtype == SSMVJP_BF16) gated ? launch_wide<bf16, true, BWD>(a, s) : launch_wide<bf16, false, BWD>(a, s);
  else gated ? launch_wide<float, true, BWD>(a, s) : launch_wide<float, false, BWD>(a, s);
}

ScanArgs scan_args(const ssmvjp_linear_scan_desc& d, const int* off) {
  ScanArgs a{};
  a.off = d.packed ? off : nullptr;
  a.nseq = d.batch; a.T = d.seqlen; a.D = d.dim; a.c = d.c;
  return a;
}

}  // namespace

int64_t linear_scan_ckpt_rows(const ssmvjp_linear_scan_desc& d) { return tile_slots(d, DCH); }

size_t linear_scan_fwd_workspace_bytes(const ssmvjp_linear_scan_desc& d) {
  return (size_t)(8 * round64(chain_words(d, FWD_ROWS * NW)));
}

// the tiles' words of the forward pass for the states and of the backward, partial sums of ddecay, states
size_t linear_scan_bwd_workspace_bytes(const ssmvjp_linear_scan_desc& d) {
  return (size_t)(8 * (round64(chain_words(d, FWD_ROWS * NW)) + round64(chain_words(d, BWD_ROWS * NW))) +
                  8 * linear_scan_ckpt_rows(d) * d.dim);
}

hipError_t launch_linear_scan_fwd(const ssmvjp_linear_scan_desc& d, const LinearScanPointers& p, hipStream_t stream) {
  constexpr int N = FWD_ROWS * NW;
  ScanArgs a = scan_args(d, p.seq_offsets);
  a.x = p.x; a.gate = p.gate; a.igate = p.input_gate; a.decay = p.decay; a.h0 = p.h0;
  a.h = p.h; a.h_final = p.h_final; a.ckpt = p.ckpt;
  set_chain(d, N, p.workspace, a);
  const bool gaps = d.packed || d.seqlen == 0;  // sequences without tokens, rows of ckpt without one
  launch_init(a, p.workspace, chain_words(d, N), p.h0, gaps ? p.h_final : nullptr, d.packed ? p.ckpt : nullptr,
              d.packed && p.ckpt ? linear_scan_ckpt_rows(d) * d.dim : 0, stream);
  launch_scan<false>(d, a, stream);
  return hipGetLastError();
}

hipError_t launch_linear_scan_bwd(const ssmvjp_linear_scan_desc& d, const LinearScanBwdPointers& p, hipStream_t stream) {
  constexpr int NF = FWD_ROWS * NW, NB = BWD_ROWS * NW;
  const i64 f = round64(chain_words(d, NF)), b = chain_words(d, NB), rows = linear_scan_ckpt_rows(d);
  u64* words = (u64*)p.workspace;
  float* part = (float*)(words + f + round64(b));
  float* states = part + rows * d.dim;
  const bool gated = d.form == SSMVJP_SCAN_GATED;
  if (d.batch > 0) {
    ScanArgs a = scan_args(d, p.seq_offsets);
    a.x = p.x; a.gate = p.gate; a.igate = p.input_gate; a.decay = p.decay; a.h0 = p.h0;
    ScanArgs fwd = a;
    a.kept = p.ckpt ? p.ckpt : states; a.dh = p.dh; a.dh_final = p.dh_final;
    a.dx = p.dx; a.dgate = p.dgate; a.digate = p.dinput_gate; a.part = part; a.dh0 = p.dh0;
    set_chain(d, NB, words + f, a);
    // one launch for what both passes wait on
    launch_init(a, p.ckpt ? words + f : words, p.ckpt ? b : f + b, p.dh_final, d.packed || d.seqlen == 0 ? p.dh0 : nullptr, nullptr, 0,
                stream);
    if (!p.ckpt) {
      fwd.ckpt = states;
      set_chain(d, NF, words, fwd);
      launch_scan<false>(d, fwd, stream);
    }
    launch_scan<true>(d, a, stream);
  }
  if (gated)
    hipLaunchKernelGGL(decay_sum_kernel, dim3((unsigned)((d.dim + 63) / 64)), dim3(1024), 0, stream, part,
                       d.batch > 0 && d.seqlen > 0 ? rows : 0, d.dim, p.decay, p.ddecay);
  return hipGetLastError();
}

hipError_t launch_linear_step(const ssmvjp_linear_step_desc& d, const LinearStepPointers& p, hipStream_t stream) {
  StepArgs a{d.nslots, d.dim, 0, d.c, p.x, p.gate, p.input_gate, p.decay, p.state, p.slots, p.h};
  const bool gated = d.form == SSMVJP_SCAN_GATED;
  if (d.dtype == SSMVJP_BF16) gated ? launch_step<bf16, true>(a, d.batch, stream) : launch_step<bf16, false>(a, d.batch, stream);
  else gated ? launch_step<float, true>(a, d.batch, stream) : launch_step<float, false>(a, d.batch, stream);
  return hipGetLastError();
}

}  // namespace ssmvjp
