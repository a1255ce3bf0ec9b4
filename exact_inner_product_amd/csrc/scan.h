// scan.h -- parts shared by the gated recurrence's two directions (scan.hip, scan_grad.hip).
//
//   h_r = a_r h_{r-1} + b_r x_r,   a = sigmoid(forget),  b = sigmoid(-forget) or sigmoid(gate)
//
// is the composition of affine maps of the state, (A, B): h -> A h + B, which is associative. A
// workgroup takes a tile: kTileRows(lanes) rows by up to 128 channels, 4 channels a thread and
// a few rows in a run, all in registers. Runs are joined across the lanes of a wave by shuffles,
// across the waves in LDS, and tiles by a chain through memory (below).
#pragma once

#include "sequences.h"

namespace mips {

constexpr int kTileThreadRows = 4096;  // rows of a tile times lanes a row
constexpr int kTileRowsMost = 1024;

// Lanes a row (4 channels each) and their logarithm: 4, 8, 16 or 32, of widths up to 16, 32, 64, any.
inline int scan_lanes_log2(int32_t d) { return d > 64 ? 5 : d > 32 ? 4 : d > 16 ? 3 : 2; }
inline int tile_rows(int32_t d) { return kTileThreadRows >> scan_lanes_log2(d); }

// How a call's rows are cut. Dense sequences of at most a tile's rows lie whole in tiles of a
// multiple of their length: no state passes between tiles. Else the tiles are chained.
struct Tiling {
  uint32_t rows;      // of a tile
  uint32_t tiles;
  uint32_t columns;   // tiles side by side along the channels
  int lanes_log2;
  bool chained;
};
inline Tiling tiling_of(const Sequences& S, int32_t d) {
  Tiling T;
  T.lanes_log2 = scan_lanes_log2(d);
  T.rows = (uint32_t)tile_rows(d);
  const bool whole = S.t && S.t <= T.rows;
  if (whole) T.rows = T.rows / S.t * S.t;
  T.tiles = S.n ? (S.n + T.rows - 1) / T.rows : 1u;
  T.chained = !whole && T.tiles > 1;
  const uint32_t width = 4u << T.lanes_log2;
  T.columns = ((uint32_t)d + width - 1) / width;
  return T;
}

// ------------------------------------------------------------------------------ gates
// sigmoid(v) and sigmoid(-v), each exact to a few units in the last place (1 - sigmoid(v) would
// not be): with e = exp(-|v|) they are 1 / (1 + e) and e / (1 + e).
__device__ __forceinline__ void sigmoids(float v, float* up, float* down) {
  const float e = __builtin_amdgcn_exp2f(-1.44269504f * fabsf(v));
  const float r = __builtin_amdgcn_rcpf(1.0f + e);
  const float q = e * r;
  *up = v < 0.0f ? q : r;
  *down = v < 0.0f ? r : q;
}

// --------------------------------------------------------------------- affine maps
// A >= 0 or NaN. A map that forgets its argument (a sequence starts inside) has A = kForgets; it
// must not be an ordinary 0, which makes NaN of an argument that is not finite, as the recurrence does.
constexpr float kForgets = -1.0f;

// `later` after `earlier`.
__device__ __forceinline__ void compose(float a0, float b0, float a1, float b1, float* a, float* b) {
  *b = a1 < 0.0f ? b1 : fmaf(a1, b0, b1);
  *a = (a1 < 0.0f || a0 < 0.0f) ? kForgets : a0 * a1;
}
__device__ __forceinline__ float apply(float a, float b, float h) { return a < 0.0f ? b : fmaf(a, h, b); }

// -------------------------------------------------------------------- chain of tiles
// Each tile and channel has a 64-bit word: empty, the tile's own map (A, B), or, once it is known,
// the state behind the tile. It is written and read with relaxed atomics of one word, value and
// meaning together, so nothing else has to be ordered. Tiles are handed out by a counter, in the
// chain's order: what a workgroup waits for belongs to workgroups that run already, each of which writes
// its map before it waits, and the first tile waits for nothing; so every wait ends, whatever the
// order in which the card starts workgroups.
//
// The state before a tile is always the same left fold, h <- A h + B over the maps since the nearest
// known state, which is itself that fold: results do not depend on how far a tile had to look back.
constexpr uint32_t kEmpty = 0xFFFFFFFFu;   // A of a word that is not written yet
constexpr uint32_t kState = 0x80000000u;   // A of a word that holds a state
constexpr int kWindow = 8;                 // words looked at together

__device__ __forceinline__ uint64_t chain_word(uint32_t a, float b) {
  return ((uint64_t)a << 32) | __float_as_uint(b);
}
__device__ __forceinline__ void chain_put(uint64_t* w, uint64_t v) {
  __hip_atomic_store(w, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t chain_get(const uint64_t* w) {
  return __hip_atomic_load(w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t chain_map(float a, float b) {
  // a product of gates has no sign; the sign that a NaN may have is taken away
  return chain_word(a == a ? __float_as_uint(a) : 0x7FC00000u, b);
}

// The state before tile `k` >= 1 of a chain whose words lie `stride` apart.
__device__ __forceinline__ float chain_state(const uint64_t* words, int64_t stride, uint32_t k) {
  uint64_t w[kWindow];
  int64_t at = (int64_t)k - 1;
  int64_t found = -1;
  while (found < 0) {  // tile 0 holds a state: the walk ends there at the latest
    const int64_t low = at - (kWindow - 1) > 0 ? at - (kWindow - 1) : 0;
#pragma unroll
    for (int j = 0; j < kWindow; ++j) w[j] = chain_get(words + (at - j > low ? at - j : low) * stride);
#pragma unroll
    for (int j = 0; j < kWindow; ++j) {
      if (found >= 0) continue;
      const int64_t i = at - j > low ? at - j : low;
      while ((uint32_t)(w[j] >> 32) == kEmpty) {
        __builtin_amdgcn_s_sleep(1);
        w[j] = chain_get(words + i * stride);
      }
      if ((uint32_t)(w[j] >> 32) == kState) found = i;
    }
    if (found < 0) at = low - 1;
  }
  float h = 0.0f;
  if (at == (int64_t)k - 1) {  // the words are at hand
#pragma unroll
    for (int j = kWindow - 1; j >= 0; --j) {
      const int64_t i = at - j;
      if (i < found) continue;
      const uint32_t a = (uint32_t)(w[j] >> 32);
      const float b = __uint_as_float((uint32_t)w[j]);
      h = a == kState ? b : fmaf(__uint_as_float(a), h, b);
    }
    return h;
  }
  for (int64_t i0 = found; i0 < (int64_t)k; i0 += kWindow) {  // none of these is empty any more
#pragma unroll
    for (int j = 0; j < kWindow; ++j) w[j] = chain_get(words + (i0 + j < (int64_t)k ? i0 + j : i0) * stride);
#pragma unroll
    for (int j = 0; j < kWindow; ++j) {
      if (i0 + j >= (int64_t)k) continue;
      const uint32_t a = (uint32_t)(w[j] >> 32);
      const float b = __uint_as_float((uint32_t)w[j]);
      h = a == kState ? b : fmaf(__uint_as_float(a), h, b);
    }
  }
  return h;
}

// Empties the words and sets the counter to 0 (a kernel: a memset node replays wrongly in graphs).
__global__ void chain_clear_kernel(uint64_t* words, uint64_t count, uint32_t* counter);

// Workspace of a chained call: the counter, then the words [tiles][columns * width].
inline size_t chain_bytes(const Tiling& T) {
  return T.chained ? 256 + (size_t)T.tiles * T.columns * (4u << T.lanes_log2) * 8 : 0;
}
int chain_clear(const Tiling& T, void* workspace, hipStream_t s);

// -------------------------------------------------------------------- four channels
template <bool VEC>
__device__ __forceinline__ void load4(const float* p, int live, float* v) {
  typedef float f32x4_t __attribute__((ext_vector_type(4)));
  if constexpr (VEC) {
    const f32x4_t q = *(const f32x4_t*)p;
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = q[c];
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = c < live ? p[c] : 0.0f;
  }
}

// Raw elements of four channels, kept as they are stored.
template <typename T> struct Raw;
template <> struct Raw<float> {
  float v[4];
  __device__ __forceinline__ float at(int c) const { return v[c]; }
};
template <> struct Raw<__bf16> {
  uint32_t v[2];
  __device__ __forceinline__ float at(int c) const {
    return __uint_as_float((c & 1) ? v[c >> 1] & 0xFFFF0000u : v[c >> 1] << 16);
  }
};

template <typename T>
__device__ __forceinline__ void raw_zero(Raw<T>* r) {
#pragma unroll
  for (unsigned c = 0; c < sizeof(r->v) / 4; ++c) r->v[c] = 0;
}
// `live` channels (1 to 4) of a row at p; 4 and aligned with VEC.
template <bool VEC>
__device__ __forceinline__ void raw_load(const float* p, int live, Raw<float>* r) {
  load4<VEC>(p, live, r->v);
}
template <bool VEC>
__device__ __forceinline__ void raw_load(const __bf16* p, int live, Raw<__bf16>* r) {
  typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
  if constexpr (VEC) {
    const u32x2_t q = *(const u32x2_t*)p;
    r->v[0] = q[0];
    r->v[1] = q[1];
  } else {
    const uint16_t* u = (const uint16_t*)p;
    r->v[0] = (uint32_t)u[0] | (live > 1 ? (uint32_t)u[1] << 16 : 0u);
    r->v[1] = (live > 2 ? (uint32_t)u[2] : 0u) | (live > 3 ? (uint32_t)u[3] << 16 : 0u);
  }
}
template <bool VEC>
__device__ __forceinline__ void store4(float* p, int live, const float* v) {
  typedef float f32x4_t __attribute__((ext_vector_type(4)));
  if constexpr (VEC) {
    __builtin_nontemporal_store(f32x4_t{v[0], v[1], v[2], v[3]}, (f32x4_t*)p);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (c < live) p[c] = v[c];
  }
}
template <bool VEC>
__device__ __forceinline__ void store4(__bf16* p, int live, const float* v) {
  typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
  if constexpr (VEC) {
    __builtin_nontemporal_store(bf16x4_t{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]}, (bf16x4_t*)p);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (c < live) p[c] = (__bf16)v[c];
  }
}

}  // namespace mips
