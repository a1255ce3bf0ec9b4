// sequences.h -- which rows of a tensor belong to which sequence (gfx950): dense [b, t, d] tensors,
// whole or with a length for each sequence, and packed [n, d] ones with b + 1 offsets.
//
// Rows are numbered as they lie: row s * t + i of a dense tensor, row r of a packed one. Kernels
// cut that axis into tiles whatever the sequences' lengths are, so that a batch of ragged histories
// fills the card as evenly as a dense one; where a sequence starts, the state is cut.
#pragma once

#include "common.h"
#include "host.h"

namespace mips {

struct Sequences {
  int32_t b;
  uint32_t t;           // dense: rows a sequence; packed: 0
  uint32_t n;           // rows
  const void* offsets;  // packed: [b + 1], else NULL
  const void* lengths;  // dense: [b] or NULL
  int32_t wide;         // offsets or lengths are int64
};

struct Rows {
  const void* p;
  int64_t row;    // elements from a row to the next one of its sequence
  int64_t extra;  // dense: sequence stride - t * row stride
};

// Where the offsets are broken (decreasing, negative, past the rows), results are meaningless but
// every access stays in bounds: offsets are clamped to [0, n] and only compared with rows.
__device__ __forceinline__ uint32_t index_at(const void* p, int wide, int64_t i, uint32_t most) {
  const int64_t v = wide ? ((const int64_t*)p)[i] : (int64_t)((const int32_t*)p)[i];
  return v < 0 ? 0u : (v > (int64_t)most ? most : (uint32_t)v);
}

// The first i in [0, b] with offsets[i] >= r, or b + 1: 64 probes a round, by one wave (all lanes).
__device__ __forceinline__ int32_t lower_bound(const Sequences& S, uint32_t r) {
  const int lane = threadIdx.x & 63;
  int32_t lo = 0, hi = S.b + 1;
  while (lo < hi) {
    const int32_t step = (hi - lo + 63) >> 6;
    const int64_t at = lo + (int64_t)lane * step;
    const bool no_less = at >= hi || index_at(S.offsets, S.wide, at, S.n) >= r;
    const uint64_t m = __ballot(no_less);
    const int k = m ? __ffsll((unsigned long long)m) - 1 : 64;  // probes 0 .. k-1 are below r
    if (k == 0) break;  // lo itself
    const int64_t top = lo + (int64_t)k * step;
    lo = lo + (k - 1) * step + 1;
    hi = top < hi ? (int32_t)top : hi;
  }
  return lo;
}

// The rows of sequence s: [*begin, *end) in the numbering above.
__device__ __forceinline__ void sequence_rows(const Sequences& S, int64_t s, uint32_t* begin, uint32_t* end) {
  if (S.t) {
    *begin = (uint32_t)s * S.t;
    *end = *begin + (S.lengths ? index_at(S.lengths, S.wide, s, S.t) : S.t);
  } else {
    *begin = index_at(S.offsets, S.wide, s, S.n);
    *end = index_at(S.offsets, S.wide, s + 1, S.n);
    if (*end < *begin) *end = *begin;
  }
}

// One wave's LDS accesses stay in order; this keeps the compiler from moving them.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Calls f(s, begin, end) for the sequences with rows in [r0, r1), those of a wave together. Dense ones
// come with rows of padding or none too, packed ones only with rows.
template <typename F>
__device__ __forceinline__ void for_sequences(const Sequences& S, uint32_t r0, uint32_t r1, F f) {
  uint32_t begin, end;
  if (S.t) {
    for (uint32_t s = r0 / S.t; s < (uint32_t)S.b && s * S.t < r1; ++s) {
      sequence_rows(S, s, &begin, &end);
      f((int32_t)s, begin, end);
    }
    return;
  }
  const int lane = threadIdx.x & 63;
  int64_t s0 = lower_bound(S, r0);
  s0 = s0 > 0 ? s0 - 1 : 0;
  for (; s0 < S.b; s0 += 64) {
    begin = end = ~0u;
    if (s0 + lane < S.b) sequence_rows(S, s0 + lane, &begin, &end);
    uint64_t m = __ballot(begin < end && begin < r1 && end > r0);
    while (m) {
      const int k = __ffsll((unsigned long long)m) - 1;
      m &= m - 1;
      f((int32_t)(s0 + k), (uint32_t)__shfl((int)begin, k), (uint32_t)__shfl((int)end, k));
    }
    if ((uint32_t)__shfl((int)begin, 63) >= r1) break;  // this one and all behind it
  }
}

// What is kept of a packed row: its sequence << 2, | kFirst and kFinal where it is its sequence's first and
// last one; kPad for a row of no sequence.
constexpr int32_t kFirst = 1, kFinal = 2, kPad = -1;

// ------------------------------------------------------------------------------- host
// Checks a mips_sequences and makes a Sequences of it; MIPS_OK or an error.
int check_sequences(const mips_sequences* q, Sequences* out);
// Checks the rows of one tensor of `dtype` and width d against the sequences.
int check_rows(const mips_rows* r, const Sequences& S, int32_t d, int32_t dtype, Rows* out);
// Whether four neighbouring elements of every row can be loaded at once.
inline bool rows_by_four(const Rows& r, int32_t d, int32_t dtype) {
  return d % 4 == 0 && r.row % 4 == 0 && r.extra % 4 == 0 && aligned(r.p, 4 * elem_bytes(dtype));
}

}  // namespace mips
