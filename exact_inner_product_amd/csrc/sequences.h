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

// What is said about a row of a tile.
constexpr uint32_t kFirst = 1, kFinal = 2;  // of its sequence
constexpr uint32_t kPad = 4;                // of no sequence: nothing is read, zeros are written
constexpr uint32_t kBeyond = 8;             // not this tile's: nothing is read or written
constexpr uint32_t kCut = kFirst | kPad | kBeyond;

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

// Marks the rows [r0, r0 + rows) of a tile, all threads of the workgroup: kind[i], and for first and
// final rows their sequence. empty(s) is called by one thread for every sequence without rows
// that this tile answers for (where it would lie; the last tile for those behind the rows).
// Ends with a barrier. kind has `space` entries; those from `rows` on are kBeyond.
template <int THREADS, typename F>
__device__ __forceinline__ void mark_rows(const Sequences& S, uint32_t r0, uint32_t rows, uint32_t space, bool last,
                                          uint8_t* kind, int32_t* first, int32_t* final, F empty) {
  const uint32_t tid = threadIdx.x;
  if (S.t) {
    for (uint32_t i = tid; i < space; i += THREADS) {
      uint32_t k = kBeyond;
      if (i < rows) {
        const uint32_t r = r0 + i, s = r / S.t, pos = r - s * S.t;
        const uint32_t len = S.lengths ? index_at(S.lengths, S.wide, s, S.t) : S.t;
        k = pos >= len ? kPad : ((pos == 0 ? kFirst : 0u) | (pos + 1 == len ? kFinal : 0u));
        if (pos == 0 && len == 0) empty((int32_t)s);
        first[i] = final[i] = (int32_t)s;
      }
      kind[i] = (uint8_t)k;
    }
    __syncthreads();
    return;
  }
  // the rows from offsets[0] to offsets[b] belong to sequences
  const uint32_t begin = index_at(S.offsets, S.wide, 0, S.n), end = index_at(S.offsets, S.wide, S.b, S.n);
  for (uint32_t i = tid; i < space; i += THREADS) {
    const uint32_t r = r0 + i;
    kind[i] = (uint8_t)(i >= rows ? kBeyond : (r < begin || r >= end ? kPad : 0u));
    first[i] = final[i] = -1;
  }
  __shared__ int32_t from;
  if (tid < 64) {
    const int32_t k = lower_bound(S, r0);
    if (tid == 0) from = k > 0 ? k - 1 : 0;  // the sequence that r0 may lie inside of
  }
  __syncthreads();
  for (int64_t s = (int64_t)from + tid; s < S.b; s += THREADS) {
    const uint32_t o0 = index_at(S.offsets, S.wide, s, S.n), o1 = index_at(S.offsets, S.wide, s + 1, S.n);
    if (o0 >= r0 + rows && !last) break;
    if (o1 <= o0) {
      if (o0 >= r0) empty((int32_t)s);
      continue;
    }
    if (o0 >= r0 && o0 < r0 + rows) first[o0 - r0] = (int32_t)s;
    if (o1 > r0 && o1 <= r0 + rows) final[o1 - 1 - r0] = (int32_t)s;
  }
  __syncthreads();
  for (uint32_t i = tid; i < rows; i += THREADS)
    kind[i] |= (uint8_t)((first[i] >= 0 ? kFirst : 0u) | (final[i] >= 0 ? kFinal : 0u));
  __syncthreads();
}

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
