// delta_seq.cuh -- the sequences of a gated delta rule call: `nseq` sequences of
// T tokens each, or packed behind one another in T tokens, with the borders in
// device memory.
//
// Borders are clamped to [0, T] and an end before its start is an empty
// sequence, so that no value in device memory can lead to an access outside
// the tensors.  Chunk slots: sequence s owns the slots from start / 64 + s (or
// s * ceil(T / 64) where all have T tokens), which needs no prefix sum: since
// floor((x + n) / 64) + 1 >= floor(x / 64) + ceil(n / 64), the slots of
// successive sequences never meet, and T / 64 + nseq of them are enough.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace ssmvjp {

constexpr int DCH = 64;  // tokens per chunk

struct DeltaSpan {
  i64 start, len, slot0;  // first token, tokens, first chunk slot
};

struct DeltaSeqs {
  const int* off;  // [nseq + 1], or NULL: nseq sequences of T tokens
  i64 nseq, T, per;  // per: chunk slots of one sequence (off == NULL)

  __device__ __forceinline__ i64 border(i64 s) const {
    const i64 o = off[s];
    return o < 0 ? 0 : o > T ? T : o;
  }
  // Where a border below one before it counts as that one (called by whole waves): where sequence s starts, the largest
  // of borders 0 .. s ...
  __device__ __forceinline__ i64 risen(i64 s, int lane) const {
    int most = most_of(s, lane);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int o = __shfl_xor(most, d);
      most = o > most ? o : most;
    }
    return most;
  }
  // ... and whether it has no tokens: its end is not above that
  __device__ __forceinline__ bool risen_empty(i64 s, int lane) const {
    const int end = (int)border(s + 1);
    return __any(most_of(s, lane) >= end);
  }
  // a lane's share of that maximum
  __device__ __forceinline__ int most_of(i64 s, int lane) const {
    int most = 0;
#pragma unroll 4
    for (i64 i = lane; i <= s; i += 64) {
      const int o = (int)border(i);
      most = o > most ? o : most;
    }
    return most;
  }
  __device__ __forceinline__ DeltaSpan span(i64 s) const {
    if (!off) return {s * T, T, s * per};
    const i64 o0 = border(s), o1 = border(s + 1);
    return {o0, o1 > o0 ? o1 - o0 : 0, o0 / DCH + s};
  }
  // the sequence that owns a chunk slot; called by whole waves
  __device__ __forceinline__ i64 of_slot(i64 slot, int lane) const {
    if (!off) return (unsigned)slot / (unsigned)per;
    i64 s = -1;  // the last sequence whose first slot is not behind `slot` (slot 0 is sequence 0's)
    for (i64 s0 = 0; s0 < nseq; s0 += 64) {
      const i64 i = s0 + lane;
      const bool in = i < nseq && border(i) / DCH + i <= slot;
      const int n = __popcll(__ballot(in));
      s += n;
      if (n < 64) break;
    }
    return s < 0 ? 0 : s;
  }
};

// NaN or an infinity
__device__ __forceinline__ bool nonfinite(float v) { return !(fabsf(v) <= 3.402823466e38f); }

inline i64 delta_slots(const ssmvjp_delta_chunk_desc& d) {
  return d.packed ? d.seqlen / DCH + d.batch : d.batch * ((d.seqlen + DCH - 1) / DCH);
}
inline DeltaSeqs delta_seqs(const ssmvjp_delta_chunk_desc& d, const int* off) {
  return {d.packed ? off : nullptr, d.batch, d.seqlen, (d.seqlen + DCH - 1) / DCH};
}

}  // namespace ssmvjp
