// scan.hip -- the gated linear recurrence over sequences, forward (gfx950). scan.h has the method.
//
// One pass: forget logits, inputs (and gate logits) are read once and the states written once.
#include "scan.h"

namespace mips {

struct ScanArgs {
  Sequences S;
  Rows x, forget, gate;
  const float* initial;  // [b, d] or NULL
  void* states;          // [n, d] or NULL
  float* last;           // [b, d]
  float* carries;        // [the gradient's tiles, d], or NULL: it needs none
  const int32_t* info;   // packed rows
  uint64_t* words;       // chained calls: of tiles, then of groups
  uint32_t* counters;
  int32_t d;
  int32_t lanes_log2;
  uint32_t rows, tiles, columns;
  uint32_t half;         // rows of the gradient's tiles
  uint32_t block0;       // of this launch
  int32_t chained;
  int32_t flat;          // load_flat serves
};

template <typename T, bool GATE, bool VEC, int R, int THREADS>
__global__ __launch_bounds__(THREADS, 4) void scan_kernel(ScanArgs A) {
  constexpr int WAVES = THREADS / 64;
  __shared__ float2 maps[WAVES][128];
  __shared__ __attribute__((aligned(16))) float entry[WAVES][128];  // the state before each wave's rows

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint32_t job = A.block0 + blockIdx.x, column = job % A.columns;
  const uint32_t tile = A.chained ? chain_ticket(A.counters, column) : job / A.columns;
  const uint32_t r0 = tile * A.rows;
  const uint32_t rows = min(A.rows, A.S.n - r0);
  const int width = 4 << A.lanes_log2;
  const int c0 = column * width;                        // the tile's first channel
  const int lanes = 1 << A.lanes_log2;
  const int ch = (lane & (lanes - 1)) * 4;              // this thread's first channel in the tile
  const int live = min(4, A.d - c0 - ch);               // <= 0: none
  const uint32_t at = (uint32_t)(tid >> A.lanes_log2) * R;  // its first row in the tile
  const int64_t channel = c0 + ch;
  const uint32_t from = live > 0 ? ch : 0;              // lanes without channels load those of others
  const int some = live > 0 ? live : 1;

  const Marks marks = run_marks<R>(A.S, A.info, r0, rows, at);
  const bool special = __any(marks.any());
  const bool idle = special && __all((marks.bits & ((1u << R) - 1u)) == (1u << R) - 1u);  // a wave of padding

  const uint32_t source = A.chained ? chain_source(A.S, A.info, r0, A.rows, tile) : 0;

  // the run from a state of 0: P the product of the gates so far, h the state
  float P[R][4], h[R][4];
  int cut = R;  // the first row that does not see the state before the run
  if (idle) {
#pragma unroll
    for (int t = 0; t < R; ++t)
#pragma unroll
      for (int c = 0; c < 4; ++c) P[t][c] = h[t][c] = 0.0f;
    cut = 0;
  } else {
    Raw<T> x[R], f[R], g[R];
    if (A.flat) {
      load_flat<VEC>(A.forget, r0, rows, at, c0, from, some, marks, f);
      load_flat<VEC>(A.x, r0, rows, at, c0, from, some, marks, x);
      if (GATE) load_flat<VEC>(A.gate, r0, rows, at, c0, from, some, marks, g);
    } else {
      load_gaps<VEC>(A.S, A.forget, r0, rows, at, c0, from, some, marks, f);
      load_gaps<VEC>(A.S, A.x, r0, rows, at, c0, from, some, marks, x);
      if (GATE) load_gaps<VEC>(A.S, A.gate, r0, rows, at, c0, from, some, marks, g);
    }
    if (special) {
#pragma unroll
      for (int t = 0; t < R; ++t) {
        if (marks.cut(t)) cut = min(cut, t);
        float init[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (A.initial && live > 0 && marks.first(t)) {
          const float* p = A.initial + row_sequence(A.S, A.info, r0 + at + t) * A.d + channel;
#pragma unroll
          for (int c = 0; c < 4; ++c) init[c] = c < live ? p[c] : 0.0f;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float a, na, b, nb;
          sigmoids(f[t].at(c), &a, &na);
          b = na;
          if (GATE) sigmoids(g[t].at(c), &b, &nb);
          const float prev = marks.cut(t) ? init[c] : (t ? h[t - 1][c] : 0.0f);
          const float v = fmaf(a, prev, b * x[t].at(c));
          h[t][c] = marks.pad(t) ? 0.0f : v;
          P[t][c] = t ? P[t - 1][c] * a : a;
        }
      }
    } else {
#pragma unroll
      for (int t = 0; t < R; ++t)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float a, na, b, nb;
          sigmoids(f[t].at(c), &a, &na);
          b = na;
          if (GATE) sigmoids(g[t].at(c), &b, &nb);
          h[t][c] = t ? fmaf(a, h[t - 1][c], b * x[t].at(c)) : b * x[t].at(c);
          P[t][c] = t ? P[t - 1][c] * a : a;
        }
    }
  }

  // maps of the runs before this one, within the wave and then the tile
  float ra[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) ra[c] = cut < R ? kForgets : P[R - 1][c];
  float ea[4], eb[4], wa[4], wb[4];
  if (special) wave_maps<false, true>(ra, h[R - 1], lane, lanes, ea, eb, wa, wb);
  else wave_maps<false, false>(ra, h[R - 1], lane, lanes, ea, eb, wa, wb);
  if (lane < lanes) {
#pragma unroll
    for (int c = 0; c < 4; ++c) maps[wave][ch + c] = float2{wa[c], wb[c]};
  }
  __syncthreads();
  // one thread a channel takes the state through the waves (all threads doing so for their own
  // wave would be a tenth of the kernel's instructions)
  const int channels = min(width, A.d - c0);
  float v = 0.0f;
  if (A.chained) {
    float a = 1.0f, b = 0.0f;
    if (tid < channels) {
#pragma unroll 4
      for (int w = 0; w < WAVES; ++w) compose(a, b, maps[w][tid].x, maps[w][tid].y, &a, &b);
    }
    const int64_t stride = (int64_t)A.columns * width;
    const Chain C{A.words, A.words + A.tiles * stride, stride, (uint32_t)(c0 + (tid & 127))};
    v = chain_link<THREADS>(C, tile, source, channels, a, b);
  }
  if (tid < channels) {
#pragma unroll 4
    for (int w = 0; w < WAVES; ++w) {
      entry[w][tid] = v;
      v = apply(maps[w][tid].x, maps[w][tid].y, v);
    }
  }
  __syncthreads();
  if (live <= 0) return;
  float state[4];  // before the run
#pragma unroll
  for (int c = 0; c < 4; ++c) state[c] = apply(ea[c], eb[c], entry[wave][ch + c]);

  if (A.carries && at % A.half == 0 && at < rows) {  // where a tile of the gradient begins
    float* p = A.carries + ((int64_t)tile * (A.rows / A.half) + at / A.half) * A.d + channel;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (c < live) p[c] = state[c];
  }
  uint8_t* base = (uint8_t*)((T*)A.states + (int64_t)r0 * A.d + c0);
  uint32_t out = (at * (uint32_t)A.d + ch) * (uint32_t)sizeof(T);
  if (!special) {
    if (!A.states) return;
#pragma unroll
    for (int t = 0; t < R; ++t, out += (uint32_t)A.d * sizeof(T)) {
      float v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = fmaf(P[t][c], state[c], h[t][c]);
      store4<VEC>((T*)(base + out), live, v);
    }
    return;
  }
#pragma unroll
  for (int t = 0; t < R; ++t, out += (uint32_t)A.d * sizeof(T)) {
    if (marks.beyond(t)) continue;
    float v[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = t < cut ? fmaf(P[t][c], state[c], h[t][c]) : h[t][c];
    if (A.states) store4<VEC>((T*)(base + out), live, v);
    const uint32_t r = r0 + at + t;
    // a padded sequence without rows: where its first one would lie
    const bool none = A.S.lengths && marks.pad(t) && r % A.S.t == 0;
    if (!none && !marks.final(t)) continue;
    const int64_t i = row_sequence(A.S, A.info, r) * A.d + channel;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (c < live) A.last[i + c] = !none ? v[c] : (A.initial ? A.initial[i + c] : 0.0f);
  }
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
constexpr uint32_t kDescribed = 256;  // rows that a wave describes

static __global__ __launch_bounds__(256) void scan_begin_kernel(BeginArgs A) {
  for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < A.count; i += (uint64_t)gridDim.x * 256)
    A.words[i] = ~uint64_t(0);
  if (blockIdx.x == 0 && threadIdx.x < A.columns) A.counters[threadIdx.x * kCounterPitch] = 0;
  if (!A.info) return;
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), waves = (int64_t)gridDim.x * 4;
  for (int64_t k = wave; k * kDescribed < A.described; k += waves) {
    const uint32_t r0 = (uint32_t)k * kDescribed, r1 = min(r0 + kDescribed, A.described);
    const uint32_t begin = index_at(A.S.offsets, A.S.wide, 0, A.S.n), end = index_at(A.S.offsets, A.S.wide, A.S.b, A.S.n);
    for (uint32_t r = r0 + lane; r < r1; r += 64)
      if (r < begin || r >= end) A.info[r] = kPad;
    for_sequences(A.S, r0, min(r1, A.S.n), [&](int32_t s, uint32_t lo, uint32_t hi) {
      for (uint32_t r = max(lo, r0) + lane; r < min(hi, r1); r += 64)
        A.info[r] = (int32_t)((uint32_t)s << 2) | (r == lo ? kFirst : 0) | (r + 1 == hi ? kFinal : 0);
    });
  }
  if (!A.of_none) return;
  for (int64_t s0 = wave * 64; s0 < A.S.b; s0 += waves * 64) {
    uint32_t lo = 0, hi = 1;
    if (s0 + lane < A.S.b) sequence_rows(A.S, s0 + lane, &lo, &hi);
    uint64_t m = __ballot(lo == hi);
    while (m) {
      const int64_t s = s0 + __ffsll((unsigned long long)m) - 1;
      m &= m - 1;
      for (int c = lane; c < A.d; c += 64) A.of_none[s * A.d + c] = A.as ? A.as[s * A.d + c] : 0.0f;
    }
  }
}

int scan_begin(const Sequences& S, const Tiling& T, const ScanSpace& W, int32_t d, const float* as, float* of_none,
               hipStream_t s) {
  if (!S.offsets && !T.chained) return MIPS_OK;
  const BeginArgs A{S, W.info, T.tiles * T.rows, W.words, W.count, W.counters, T.columns, d, as, of_none};
  uint64_t blocks = (W.count + 1023) / 1024;
  if (W.info) {
    const uint64_t rows = ((uint64_t)A.described + 4 * kDescribed - 1) / (4 * kDescribed), seqs = ((uint64_t)S.b + 255) / 256;
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

template <typename T, int R, int THREADS>
static void (*scan_variant(bool gate, bool vec))(ScanArgs) {
  return gate ? (vec ? scan_kernel<T, true, true, R, THREADS> : scan_kernel<T, true, false, R, THREADS>)
              : (vec ? scan_kernel<T, false, true, R, THREADS> : scan_kernel<T, false, false, R, THREADS>);
}

// Bytes that both directions of a call need; the tiles of the gradient if they are chained, else 0.
static size_t scan_bytes(const Sequences& S, int32_t d) {
  const size_t f = scan_space(S, forward_tiling(S, d, MIPS_BF16), nullptr).bytes;
  const size_t b = scan_space(S, backward_tiling(S, d), nullptr).bytes;  // and forward in f32
  return f > b ? f : b;
}
static uint32_t scan_carries(const Sequences& S, int32_t d) {
  const Tiling B = backward_tiling(S, d);
  return B.chained ? B.tiles : 0;
}

}  // namespace mips

using namespace mips;

extern "C" {

int64_t mips_gated_scan_carries(const mips_sequences* seq, int32_t d) {
  Sequences S;
  if (check_sequences(seq, &S) != MIPS_OK || d < 1 || d > MIPS_EMBEDDING_D_MAX) return -1;
  return scan_carries(S, d);
}

size_t mips_gated_scan_workspace_size(const mips_sequences* seq, int32_t d) {
  Sequences S;
  if (check_sequences(seq, &S) != MIPS_OK || d < 1 || d > MIPS_EMBEDDING_D_MAX) return 0;
  return scan_bytes(S, d);
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
  const Tiling T = forward_tiling(A.S, d, dtype);
  const bool carried = scan_carries(A.S, d) > 0;
  if (!last || !aligned(last, 4) || !aligned(initial, 4) || !aligned(states, elem_bytes(dtype)) ||
      !aligned(workspace, 256) || ((T.chained || A.S.offsets) && !workspace) || (carried && !carries) || !aligned(carries, 4))
    return MIPS_ERR_INVALID_ARG;
  if ((T.chained || A.S.offsets) && workspace_bytes < scan_bytes(A.S, d)) return MIPS_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  A.initial = initial;
  A.states = states;
  A.last = last;
  A.carries = carried ? carries : nullptr;
  A.half = carried ? backward_tiling(A.S, d).rows : T.rows;
  A.d = d;
  A.lanes_log2 = T.lanes_log2;
  A.rows = T.rows;
  A.tiles = T.tiles;
  A.columns = T.columns;
  A.chained = T.chained;
  const ScanSpace W = scan_space(A.S, T, workspace);
  A.info = W.info;
  A.words = W.words;
  A.counters = W.counters;
  if (const int rc = scan_begin(A.S, T, W, d, initial, last, s)) return rc;
  const bool vec = rows_by_four(A.x, d, dtype) && rows_by_four(A.forget, d, dtype) &&
                   (!gate || rows_by_four(A.gate, d, dtype)) && aligned(states, 4 * elem_bytes(dtype));
  A.flat = rows_flat(A.x, T, dtype) && rows_flat(A.forget, T, dtype) && (!gate || rows_flat(A.gate, T, dtype));
  void (*kernel)(ScanArgs) = nullptr;
  if (dtype == MIPS_BF16) kernel = scan_variant<__bf16, kLongRun, kTileThreads>(gate != nullptr, vec);
  else if (T.threads == kTileThreads) kernel = scan_variant<float, kRun, kTileThreads>(gate != nullptr, vec);
  else kernel = scan_variant<float, kRun, 2 * kTileThreads>(gate != nullptr, vec);
  const uint64_t jobs = (uint64_t)T.tiles * T.columns, most = kMaxGridBlocks / 2;  // up to 1024 threads each
  for (uint64_t j = 0; j < jobs; j += most) {
    A.block0 = (uint32_t)j;
    const uint64_t left = jobs - j;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)(left < most ? left : most)), dim3(T.threads), 0, s, A);
    if (const int rc = check_launch()) return rc;
  }
  return MIPS_OK;
}

}  // extern "C"
