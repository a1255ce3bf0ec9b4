// scan.hip -- the gated linear recurrence over sequences, forward (gfx950). scan.h has the method.
//
// One pass: forget logits, inputs (and gate logits) are read once and the states written once. Bound by
// memory where sequences lie whole in tiles: 4096 x 127 x 128 bf16 take 82 us (5.3 TB/s, the carries
// among them; vector units busy half of the time), and 43 where half of the rows are padding and only last
// states are wanted (vector units and latency). Chained tiles add what they wait for one another: 65,536 x
// 1024 bf16 take 109 (4.0 TB/s), 600,000 x 100 packed f32 with gates 227 (4.5 TB/s). Dense sequences
// just above half a tile leave half of its threads idle: 65 x 128 bf16 take 1.6 times what 127 x 128 do, row for row.
#include <type_traits>

#include "scan.h"

namespace mips {

struct ScanArgs {
  Sequences S;
  Rows x, forget, gate;
  const float* initial;  // [b, d] or NULL
  void* states;          // [n, d] or NULL
  float* last;           // [b, d]
  float* carries;        // [runs of all tiles, d] or NULL: the state before each run
  const int32_t* info;   // packed rows
  uint64_t* words;       // chained calls: of tiles, then of groups
  uint32_t* counters;
  int32_t d;
  int32_t lanes_log2;
  uint32_t rows, tiles, columns;
  uint32_t block0;       // of this launch
  int32_t flat;          // load_flat serves
};

// A padded sequence without rows would begin at row r: its last state is its initial one.
__device__ __forceinline__ void none_last(const ScanArgs& A, uint32_t r, int64_t channel, int live) {
  const int64_t i = (int64_t)(r / A.S.t) * A.d + channel;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (c < live) A.last[i + c] = A.initial ? A.initial[i + c] : 0.0f;
}

// STATES: every state is wanted, and held until the one before the run is known. Else a run keeps its map and, of
// a sequence that goes on from the run before, the map up to its final row: registers for half as
// many waves again, where this is bound by latency (4096 x 127 x 128 bf16 with lengths: 72 us when states were held, 43).
template <typename T, bool GATE, int VEC, bool STATES, bool CHAINED, int THREADS>
__global__ __launch_bounds__(THREADS, STATES || GATE || THREADS > 512 ? 4 : 6) void scan_kernel(ScanArgs A) {
  constexpr int R = kRun<T>;
  extern __shared__ __attribute__((aligned(16))) uint8_t shared[];
  Shared M;
  shared_bytes(THREADS, 4 << A.lanes_log2, CHAINED, &M, shared);
  const int tid = threadIdx.x;
  const uint32_t job = A.block0 + blockIdx.x, column = job % A.columns;
  const uint32_t tile = CHAINED ? chain_ticket(A.counters, column) : job / A.columns;
  const uint32_t r0 = tile * A.rows;
  const uint32_t rows = min(A.rows, A.S.n - r0);
  const int width = 4 << A.lanes_log2;
  const int c0 = column * width;                        // the tile's first channel
  const int lanes = 1 << A.lanes_log2;
  const int ch = (tid & (lanes - 1)) * 4;              // this thread's first channel in the tile
  const int live = min(4, A.d - c0 - ch);               // <= 0: none
  const uint32_t at = (uint32_t)(tid >> A.lanes_log2) * R;  // its first row in the tile
  const int64_t channel = c0 + ch;
  const uint32_t from = live > 0 ? ch : 0;              // lanes without channels load those of the first
  const int some = live > 0 ? live : min(4, A.d - c0);
  const bool wide = A.d >= 4;

  const Marks marks = run_marks<R>(A.S, A.info, r0, rows, at);
  const bool special = __any(marks.any());
  const bool idle = special && __all((marks.bits & ((1u << R) - 1u)) == (1u << R) - 1u);  // a wave of padding

  const uint32_t source = CHAINED ? chain_source(A.S, A.info, r0, A.rows, tile) : 0;

  // the run from a state of 0: P the product of the gates so far, h the state
  constexpr int KEPT = STATES ? R : 1;
  float P[KEPT][4], h[KEPT][4];
  float fP[4], fh[4];    // those of `ends`, the final row that sees the state before the run, without STATES
  int ends = R;
  int cut = R;           // the first row that does not see the state before the run
#pragma unroll
  for (int t = 0; t < KEPT; ++t)
#pragma unroll
    for (int c = 0; c < 4; ++c) P[t][c] = h[t][c] = 0.0f;
  if (idle) {
    cut = 0;
  } else {
    Raw<T> x[R], f[R], g[R];
    if (A.flat) {
      load_flat<VEC>(A.forget, r0, rows, at, c0, from, some, wide, marks, f);
      load_flat<VEC>(A.x, r0, rows, at, c0, from, some, wide, marks, x);
      if (GATE) load_flat<VEC>(A.gate, r0, rows, at, c0, from, some, wide, marks, g);
    } else {
      load_gaps<VEC>(A.S, A.forget, r0, rows, at, c0, from, some, wide, marks, f);
      load_gaps<VEC>(A.S, A.x, r0, rows, at, c0, from, some, wide, marks, x);
      if (GATE) load_gaps<VEC>(A.S, A.gate, r0, rows, at, c0, from, some, wide, marks, g);
    }
    auto run = [&](auto plain) __attribute__((always_inline)) {
      constexpr bool PLAIN = decltype(plain)::value;  // no row of the wave begins or ends a sequence, or is padding
      float p[4], v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        p[c] = 1.0f;
        v[c] = 0.0f;
      }
#pragma unroll
      for (int t = 0; t < R; ++t) {
        const bool has = !PLAIN && marks.wave_has(t);
        if (has && marks.cut(t)) {
          cut = min(cut, t);
          const bool init = A.initial && live > 0 && marks.first(t);
          const float* q = init ? A.initial + row_sequence(A.S, A.info, r0 + at + t) * A.d + channel : nullptr;
#pragma unroll
          for (int c = 0; c < 4; ++c) v[c] = init && c < live ? q[c] : 0.0f;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float a, na, b, nb;
          sigmoids(f[t].at(c), &a, &na);
          b = na;
          if (GATE) sigmoids(g[t].at(c), &b, &nb);
          v[c] = fmaf(a, v[c], b * x[t].at(c));
          p[c] *= a;
          if (has && marks.pad(t)) v[c] = 0.0f;
          if (STATES) {
            P[STATES ? t : 0][c] = p[c];
            h[STATES ? t : 0][c] = v[c];
            here(&P[STATES ? t : 0][c]);
            here(&h[STATES ? t : 0][c]);
          }
        }
        if (!STATES && has && marks.final(t)) {
          if (t < cut) {
            ends = t;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              fP[c] = p[c];
              fh[c] = v[c];
            }
          } else if (live > 0) {
            float* q = A.last + row_sequence(A.S, A.info, r0 + at + t) * A.d + channel;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (c < live) q[c] = v[c];
          }
        }
      }
      if (!STATES) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          P[0][c] = p[c];
          h[0][c] = v[c];
        }
      }
    };
    if (special) run(std::false_type{});
    else run(std::true_type{});
  }

  float ra[4];  // the run's map
#pragma unroll
  for (int c = 0; c < 4; ++c) ra[c] = cut < R ? kForgets : P[KEPT - 1][c];
  half_maps<false>(tid, ra, h[KEPT - 1], lanes, M);
  const int64_t stride = (int64_t)A.columns * width;
  const Chain C{A.words, A.words + A.tiles * stride, stride, (uint32_t)(c0 + (tid & 127))};
  join_halves<THREADS, false, CHAINED>(tid, M, C, tile, source, min(width, A.d - c0), width);
  if (live <= 0) return;
  float state[4];  // before the run
  half_reach(tid, M, lanes, state);

  if (A.carries && at < rows && !idle)
    store4<VEC>(A.carries + ((int64_t)tile * (THREADS >> A.lanes_log2) + (tid >> A.lanes_log2)) * A.d + channel, live, state);
  // sequences without rows that would begin in this run
  auto none_lasts = [&]() __attribute__((always_inline)) {
    if (!A.S.lengths) return;
    for (uint32_t m = run_nones<R>(A.S, r0 + at, marks); m; m &= m - 1) none_last(A, r0 + at + (__ffs(m) - 1), channel, live);
  };
  if (!STATES) {
    if (!special) return;
    if (ends < R) {
      float* p = A.last + row_sequence(A.S, A.info, r0 + at + ends) * A.d + channel;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < live) p[c] = fmaf(fP[c], state[c], fh[c]);
    }
    none_lasts();
    return;
  }
  uint8_t* base = (uint8_t*)((T*)A.states + (int64_t)r0 * A.d + c0);
  uint32_t out = (at * (uint32_t)A.d + ch) * (uint32_t)sizeof(T);
  auto write = [&](auto plain) __attribute__((always_inline)) {
    constexpr bool PLAIN = decltype(plain)::value;
#pragma unroll
    for (int t = 0; t < R; ++t, out += (uint32_t)A.d * sizeof(T)) {
      constexpr int K = STATES;
      float v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = PLAIN || t < cut ? fmaf(P[K * t][c], state[c], h[K * t][c]) : h[K * t][c];
      const bool has = !PLAIN && marks.wave_has(t);
      if (has && marks.beyond(t)) continue;
      store4<VEC>((T*)(base + out), live, v);
      if (!has) continue;
      if (!marks.final(t)) continue;
      float* p = A.last + row_sequence(A.S, A.info, r0 + at + t) * A.d + channel;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < live) p[c] = v[c];
    }
  };
  if (!special) return write(std::true_type{});
  write(std::false_type{});
  none_lasts();
}

struct BeginArgs {
  Sequences S;
  int32_t* info;
  uint32_t described;  // rows of info, to the end of the last tile
  uint64_t* words;
  uint64_t count;
  uint32_t* counters;
  uint32_t columns;
  int32_t d;
  const float* as;
  float* of_none;
};
constexpr uint32_t kDescribed = 256;  // rows that a wave describes, four a lane

// Rows [r0, r0 + kDescribed), below `rows`, of packed sequences, by one wave. A sequence marks its first row in LDS (or the
// first one here), with a number that grows from sequence to sequence: the highest mark up to a row
// is its own sequence's. (A loop over the sequences, each writing its rows, took 28 us where 2147 of up to
// two rows take 6.)
__device__ __forceinline__ void describe(const Sequences& S, uint32_t r0, uint32_t rows, uint32_t first, uint32_t past,
                                         int32_t* mark, int32_t* info) {
  const int lane = threadIdx.x & 63;
  for (uint32_t i = lane; i <= kDescribed; i += 64) mark[i] = 0;
  wave_fence();
  int64_t s0 = lower_bound(S, r0);
  s0 = s0 > 0 ? s0 - 1 : 0;
  for (; s0 < S.b; s0 += 64) {
    uint32_t begin = ~0u, end = ~0u;
    if (s0 + lane < S.b) sequence_rows(S, s0 + lane, &begin, &end);
    if (begin < end && begin <= r0 + kDescribed && end > r0)
      mark[max(begin, r0) - r0] = (int32_t)((uint32_t)(s0 + lane + 1) << 1) | (begin >= r0 ? 1 : 0);
    if ((uint32_t)__shfl((int)begin, 63) > r0 + kDescribed) break;  // this one and all behind it
  }
  wave_fence();
  int32_t m[5], high = 0;
#pragma unroll
  for (int j = 0; j < 5; ++j) m[j] = mark[4 * lane + j];
#pragma unroll
  for (int j = 0; j < 4; ++j) high = max(high, m[j]);
  for (int o = 1; o < 64; o <<= 1) {
    const int32_t v = __shfl_up(high, o);
    if (lane >= o) high = max(high, v);
  }
  high = __shfl_up(high, 1);
  if (lane == 0) high = 0;
  int4 out;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t r = r0 + 4 * lane + j;
    high = max(high, m[j]);
    (&out.x)[j] = r < first || r >= past || !high
                      ? kPad
                      : (int32_t)((uint32_t)((high >> 1) - 1) << 2) | (m[j] & 1 ? kFirst : 0) | (m[j + 1] || r + 1 == past ? kFinal : 0);
  }
  if (r0 + 4 * lane < rows) *(int4*)(info + r0 + 4 * lane) = out;  // (a tile has a multiple of 4 rows)
}

static __global__ __launch_bounds__(256) void scan_begin_kernel(BeginArgs A) {
  __shared__ int32_t marks[4][kDescribed + 1];
  for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < A.count; i += (uint64_t)gridDim.x * 256)
    A.words[i] = ~uint64_t(0);
  if (blockIdx.x == 0 && threadIdx.x < A.columns) A.counters[threadIdx.x * kCounterPitch] = 0;
  if (!A.info) return;
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), waves = (int64_t)gridDim.x * 4;
  const uint32_t first = index_at(A.S.offsets, A.S.wide, 0, A.S.n), past = index_at(A.S.offsets, A.S.wide, A.S.b, A.S.n);
  for (int64_t k = wave; k * kDescribed < A.described; k += waves)
    describe(A.S, (uint32_t)k * kDescribed, A.described, first, past, marks[threadIdx.x >> 6], A.info);
  if (!A.of_none) return;
  const int64_t spans = (A.d + 255) / 256;
  for (int64_t k = wave; k < A.S.b * spans; k += waves) {
    const int64_t s = k / spans;
    uint32_t lo, hi;
    sequence_rows(A.S, s, &lo, &hi);
    if (lo < hi) continue;
    const int c0 = (int)(k - s * spans) * 256;
    for (int c = c0 + lane; c < min(A.d, c0 + 256); c += 64) A.of_none[s * A.d + c] = A.as ? A.as[s * A.d + c] : 0.0f;
  }
}

int scan_begin(const Sequences& S, const Tiling& T, const ScanSpace& W, int32_t d, const float* as, float* of_none,
               hipStream_t s) {
  if (!S.offsets && !T.chained) return MIPS_OK;
  const BeginArgs A{S, W.info, T.tiles * T.rows, W.words, W.count, W.counters, T.columns, d, as, of_none};
  uint64_t blocks = (W.count + 1023) / 1024;
  if (W.info) {
    const uint64_t rows = ((uint64_t)A.described + 4 * kDescribed - 1) / (4 * kDescribed);
    const uint64_t seqs = of_none ? ((uint64_t)S.b * ((d + 255) / 256) + 3) / 4 : 0;
    blocks = blocks > rows ? blocks : rows;
    blocks = blocks > seqs ? blocks : seqs;
  }
  hipLaunchKernelGGL(scan_begin_kernel, dim3((uint32_t)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, A);
  return check_launch();
}

int check_sequences(const mips_sequences* q, Sequences* out) {
  if (!q || q->b < 1) return MIPS_ERR_INVALID_ARG;
  if (q->offsets && q->lengths) return MIPS_ERR_INVALID_ARG;
  if ((q->offsets || q->lengths) && q->index_bits != 32 && q->index_bits != 64) return MIPS_ERR_UNSUPPORTED;
  const int64_t most = MIPS_TOKENS_MAX;
  if (q->offsets) {
    if (q->n < 0 || !aligned(q->offsets, q->index_bits / 8)) return MIPS_ERR_INVALID_ARG;
    if (q->n > most) return MIPS_ERR_UNSUPPORTED;
  } else {
    if (q->t < 1) return MIPS_ERR_INVALID_ARG;
    if (q->lengths && !aligned(q->lengths, q->index_bits / 8)) return MIPS_ERR_INVALID_ARG;
    if (q->t > most || q->b > most / q->t) return MIPS_ERR_UNSUPPORTED;
  }
  if (q->b > MIPS_B_MAX) return MIPS_ERR_UNSUPPORTED;
  out->b = q->b;
  out->t = q->offsets ? 0u : (uint32_t)q->t;
  out->n = q->offsets ? (uint32_t)q->n : (uint32_t)q->b * (uint32_t)q->t;
  out->offsets = q->offsets;
  out->lengths = q->lengths;
  out->wide = q->index_bits == 64;
  return MIPS_OK;
}

int check_rows(const mips_rows* r, const Sequences& S, int32_t d, int32_t dtype, Rows* out) {
  if (!r || (S.n > 0 && !r->data) || !aligned(r->data, elem_bytes(dtype)) || r->row_stride < d) return MIPS_ERR_INVALID_ARG;
  if (r->row_stride > (S.t ? int64_t(1) << 40 : MIPS_PACKED_STRIDE_MAX)) return MIPS_ERR_UNSUPPORTED;
  int64_t extra = 0;
  if (S.t) {
    if (r->seq_stride < d || r->seq_stride > int64_t(1) << 44) return MIPS_ERR_INVALID_ARG;
    extra = S.b > 1 ? r->seq_stride - (int64_t)S.t * r->row_stride : 0;
  }
  *out = Rows{r->data, r->row_stride, extra};
  return MIPS_OK;
}

template <typename T, bool STATES, bool CHAINED, int THREADS>
static void (*scan_variant(bool gate, int vec))(ScanArgs) {
  if (vec == 2) return gate ? scan_kernel<T, true, 2, STATES, CHAINED, THREADS> : scan_kernel<T, false, 2, STATES, CHAINED, THREADS>;
  if constexpr (std::is_same<T, __bf16>::value) {
    if (vec == 1) return gate ? scan_kernel<T, true, 1, STATES, CHAINED, THREADS> : scan_kernel<T, false, 1, STATES, CHAINED, THREADS>;
  }
  return gate ? scan_kernel<T, true, 0, STATES, CHAINED, THREADS> : scan_kernel<T, false, 0, STATES, CHAINED, THREADS>;
}
template <bool STATES>
static void (*scan_kernel_of(int32_t dtype, const Tiling& T, bool gate, int vec))(ScanArgs) {
  if (dtype == MIPS_BF16)
    return T.chained ? scan_variant<__bf16, STATES, true, kTileThreads>(gate, vec)
                     : scan_variant<__bf16, STATES, false, kTileThreads>(gate, vec);
  if (T.threads > kTileThreads) return scan_variant<float, STATES, false, 2 * kTileThreads>(gate, vec);  // never chained
  return T.chained ? scan_variant<float, STATES, true, kTileThreads>(gate, vec)
                   : scan_variant<float, STATES, false, kTileThreads>(gate, vec);
}

}  // namespace mips

using namespace mips;

extern "C" {

int64_t mips_gated_scan_carries(const mips_sequences* seq, int32_t d, int32_t dtype) {
  Sequences S;
  if (check_sequences(seq, &S) != MIPS_OK || d < 1 || d > MIPS_EMBEDDING_D_MAX || (dtype != MIPS_F32 && dtype != MIPS_BF16))
    return -1;
  return scan_runs(scan_tiling(S, d, dtype));
}

size_t mips_gated_scan_workspace_size(const mips_sequences* seq, int32_t d, int32_t dtype) {
  Sequences S;
  if (check_sequences(seq, &S) != MIPS_OK || d < 1 || d > MIPS_EMBEDDING_D_MAX || (dtype != MIPS_F32 && dtype != MIPS_BF16))
    return 0;
  const Tiling T = scan_tiling(S, d, dtype);
  return T.chained || S.offsets ? scan_space(S, T, nullptr).bytes : 0;
}

int mips_gated_scan(const mips_sequences* seq, int32_t d, int32_t dtype, const mips_rows* x, const mips_rows* forget,
                    const mips_rows* gate, const float* initial, void* states, float* last, float* carries,
                    void* workspace, size_t workspace_bytes, void* stream) {
  ScanArgs A{};
  if (const int rc = check_sequences(seq, &A.S)) return rc;
  if (d < 1) return MIPS_ERR_INVALID_ARG;
  if (d > MIPS_EMBEDDING_D_MAX || (dtype != MIPS_F32 && dtype != MIPS_BF16)) return MIPS_ERR_UNSUPPORTED;
  if (const int rc = check_rows(x, A.S, d, dtype, &A.x)) return rc;
  if (const int rc = check_rows(forget, A.S, d, dtype, &A.forget)) return rc;
  if (gate) {
    if (const int rc = check_rows(gate, A.S, d, dtype, &A.gate)) return rc;
  }
  const Tiling T = scan_tiling(A.S, d, dtype);
  if (!last || !aligned(last, 4) || !aligned(initial, 4) || !aligned(states, elem_bytes(dtype)) ||
      !aligned(workspace, 256) || ((T.chained || A.S.offsets) && !workspace) || !aligned(carries, 4))
    return MIPS_ERR_INVALID_ARG;
  const ScanSpace W = scan_space(A.S, T, workspace);
  if ((T.chained || A.S.offsets) && workspace_bytes < W.bytes) return MIPS_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  A.initial = initial;
  A.states = states;
  A.last = last;
  A.carries = carries;
  A.d = d;
  A.lanes_log2 = T.lanes_log2;
  A.rows = T.rows;
  A.tiles = T.tiles;
  A.columns = T.columns;
  A.info = W.info;
  A.words = W.words;
  A.counters = W.counters;
  if (const int rc = scan_begin(A.S, T, W, d, initial, last, s)) return rc;
  const bool by_four = rows_by_four(A.x, d, dtype) && rows_by_four(A.forget, d, dtype) &&
                   (!gate || rows_by_four(A.gate, d, dtype)) && aligned(states, 4 * elem_bytes(dtype)) && aligned(carries, 16);
  A.flat = rows_flat(A.x, T, dtype) && rows_flat(A.forget, T, dtype) && (!gate || rows_flat(A.gate, T, dtype));
  const int vec = rows_vec(by_four, d, dtype);
  void (*kernel)(ScanArgs) = states ? scan_kernel_of<true>(dtype, T, gate, vec) : scan_kernel_of<false>(dtype, T, gate, vec);
  const uint64_t jobs = (uint64_t)T.tiles * T.columns, most = kMaxGridBlocks / 2;  // up to 1024 threads each
  const size_t lds = shared_bytes(T.threads, 4 << T.lanes_log2, T.chained, nullptr, nullptr);
  for (uint64_t j = 0; j < jobs; j += most) {
    A.block0 = (uint32_t)j;
    const uint64_t left = jobs - j;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)(left < most ? left : most)), dim3(T.threads), lds, s, A);
    if (const int rc = check_launch()) return rc;
  }
  return MIPS_OK;
}

}  // extern "C"
