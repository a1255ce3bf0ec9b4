// scan.hip -- the gated linear recurrence over sequences, forward (gfx950). scan.h has the method.
//
// One pass: forget logits, inputs (and gate logits) are read once and the states written once.
#include "scan.h"

namespace mips {

constexpr int kScanThreads = 512;
constexpr int kScanRun = kTileThreadRows / kScanThreads;  // rows of a thread

struct ScanArgs {
  Sequences S;
  Rows x, forget, gate;
  const float* initial;  // [b, d] or NULL
  void* states;          // [n, d] or NULL
  float* last;           // [b, d]
  float* carries;        // [tiles, d], chained calls
  uint64_t* words;       // chained calls
  uint32_t* counter;
  int32_t d;
  int32_t lanes_log2;
  uint32_t rows, tiles, columns;
  uint32_t block0;       // of this launch
  int32_t chained;
};

template <typename T, bool GATE, bool VEC>
__global__ __launch_bounds__(kScanThreads) void scan_kernel(ScanArgs A) {
  constexpr int R = kScanRun, WAVES = kScanThreads / 64;
  __shared__ __attribute__((aligned(8))) uint8_t kind[kTileRowsMost];
  __shared__ int32_t first[kTileRowsMost], final[kTileRowsMost];
  __shared__ float2 maps[WAVES][128];
  __shared__ float before[128];
  __shared__ uint32_t ticket;

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  uint32_t job = A.block0 + blockIdx.x;
  if (A.chained) {
    if (tid == 0) ticket = atomicAdd(A.counter, 1u);
    __syncthreads();
    job = ticket;
  }
  const uint32_t tile = job / A.columns, column = job - tile * A.columns;
  const uint32_t r0 = tile * A.rows;
  const uint32_t rows = min(A.rows, A.S.n - r0);
  const int width = 4 << A.lanes_log2;
  const int c0 = column * width;                        // the tile's first channel
  const int lanes = 1 << A.lanes_log2;
  const int ch = (lane & (lanes - 1)) * 4;              // this thread's first channel in the tile
  const int live = min(4, A.d - c0 - ch);               // <= 0: none
  const uint32_t at = (uint32_t)(tid >> A.lanes_log2) * R;  // its first row in the tile
  const int64_t channel = c0 + ch;

  Raw<T> x[R], f[R], g[R];
  auto load = [&](bool all, uint64_t kinds) __attribute__((always_inline)) {
    // of its run's rows r = r0 + at + t; a run may pass into the next sequences of a dense tensor
    uint32_t s = 0, pos = 0;
    const bool dense = A.S.t != 0;
    if (dense) {
      s = (r0 + at) / A.S.t;
      pos = r0 + at - s * A.S.t;
    }
#pragma unroll
    for (int t = 0; t < R; ++t) {
      raw_zero(&x[t]);
      raw_zero(&f[t]);
      if (GATE) raw_zero(&g[t]);
      const bool want = all ? at + t < rows : ((kinds >> (8 * t)) & (kPad | kBeyond)) == 0;
      if (want && live > 0) {
        const int64_t r = (int64_t)r0 + at + t;
        raw_load<VEC>((const T*)A.x.p + r * A.x.row + s * A.x.extra + channel, live, &x[t]);
        raw_load<VEC>((const T*)A.forget.p + r * A.forget.row + s * A.forget.extra + channel, live, &f[t]);
        if (GATE) raw_load<VEC>((const T*)A.gate.p + r * A.gate.row + s * A.gate.extra + channel, live, &g[t]);
      }
      if (dense && ++pos == A.S.t) {
        pos = 0;
        ++s;
      }
    }
  };
  // rows behind a sequence's length are not read; without lengths nothing has to be known first
  if (!A.S.lengths) load(true, 0);
  const uint32_t space = kTileThreadRows >> A.lanes_log2;
  mark_rows<kScanThreads>(A.S, r0, rows, space, tile + 1 == A.tiles, kind, first, final, [&](int32_t s) {
    for (int c = c0; c < min(A.d, c0 + width); ++c)
      A.last[(int64_t)s * A.d + c] = A.initial ? A.initial[(int64_t)s * A.d + c] : 0.0f;
  });
  const uint64_t kinds = *(const uint64_t*)&kind[at];
  if (A.S.lengths) load(false, kinds);

  // the run from a state of 0: P the product of the gates so far, h the state
  float P[R][4], h[R][4];
  int cut = R;  // the first row that does not see the state before the run
  if (__any(kinds != 0)) {
#pragma unroll
    for (int t = 0; t < R; ++t) {
      const uint32_t k = (uint32_t)(kinds >> (8 * t)) & 255u;
      if (k & kCut) cut = min(cut, t);
      float init[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if ((k & kFirst) && A.initial && live > 0) {
        const float* p = A.initial + (int64_t)first[at + t] * A.d + channel;
#pragma unroll
        for (int c = 0; c < 4; ++c) init[c] = c < live ? p[c] : 0.0f;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float a, na, b, nb;
        sigmoids(f[t].at(c), &a, &na);
        b = na;
        if (GATE) sigmoids(g[t].at(c), &b, &nb);
        const float prev = (k & kCut) ? init[c] : (t ? h[t - 1][c] : 0.0f);
        const float v = fmaf(a, prev, b * x[t].at(c));
        h[t][c] = (k & (kPad | kBeyond)) ? 0.0f : v;
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

  // maps of the runs before this one, within the wave and then the tile
  float ma[4], mb[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    ma[c] = cut < R ? kForgets : P[R - 1][c];
    mb[c] = h[R - 1][c];
  }
  for (int o = lanes; o < 64; o <<= 1) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float pa = __shfl_up(ma[c], o), pb = __shfl_up(mb[c], o);
      if (lane >= o) compose(pa, pb, ma[c], mb[c], &ma[c], &mb[c]);
    }
  }
  if (lane >= 64 - lanes) {
#pragma unroll
    for (int c = 0; c < 4; ++c) maps[wave][ch + c] = float2{ma[c], mb[c]};
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {  // of the runs before it in its wave
    ma[c] = __shfl_up(ma[c], lanes);
    mb[c] = __shfl_up(mb[c], lanes);
    if (lane < lanes) {
      ma[c] = 1.0f;
      mb[c] = 0.0f;
    }
  }
  __syncthreads();
  if (A.chained) {
    if (tid < width && c0 + tid < A.d) {
      float a = 1.0f, b = 0.0f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) compose(a, b, maps[w][tid].x, maps[w][tid].y, &a, &b);
      const int64_t stride = (int64_t)A.columns * width;
      uint64_t* own = A.words + tile * stride + c0 + tid;
      // a tile whose first row goes on with a sequence needs the state before it
      const bool needs = tile > 0 && (kind[0] & kCut) == 0;
      if (!needs || a < 0.0f) chain_put(own, chain_word(kState, b));
      else chain_put(own, chain_map(a, b));
      float state = 0.0f;
      if (needs) {
        state = chain_state(A.words + c0 + tid, stride, tile);
        if (!(a < 0.0f)) chain_put(own, chain_word(kState, fmaf(a, state, b)));
      }
      before[tid] = state;
      A.carries[(int64_t)tile * A.d + c0 + tid] = state;
    }
    __syncthreads();
  }
  float wa[4] = {1.0f, 1.0f, 1.0f, 1.0f}, wb[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int w = 0; w < wave; ++w) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float2 m = maps[w][ch + c];
      compose(wa[c], wb[c], m.x, m.y, &wa[c], &wb[c]);
    }
  }
  float state[4];  // before the run
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float s0 = A.chained ? before[ch + c] : 0.0f;
    state[c] = apply(ma[c], mb[c], apply(wa[c], wb[c], s0));
  }
  if (live <= 0) return;
#pragma unroll
  for (int t = 0; t < R; ++t) {
    const uint32_t k = (uint32_t)(kinds >> (8 * t)) & 255u;
    if (k & kBeyond) continue;
    float v[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = t < cut ? fmaf(P[t][c], state[c], h[t][c]) : h[t][c];
    if (A.states) store4<VEC>((T*)A.states + ((int64_t)r0 + at + t) * A.d + channel, live, v);
    if ((k & (kFinal | kPad)) == kFinal) {
      float* p = A.last + (int64_t)final[at + t] * A.d + channel;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < live) p[c] = v[c];
    }
  }
}

__global__ __launch_bounds__(256) void chain_clear_kernel(uint64_t* words, uint64_t count, uint32_t* counter) {
  for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (uint64_t)gridDim.x * 256)
    words[i] = ~uint64_t(0);
  if (blockIdx.x == 0 && threadIdx.x == 0) *counter = 0;
}

int chain_clear(const Tiling& T, void* workspace, hipStream_t s) {
  const uint64_t count = (uint64_t)T.tiles * T.columns * (4u << T.lanes_log2);
  const uint64_t blocks = (count + 1023) / 1024;
  hipLaunchKernelGGL(chain_clear_kernel, dim3((uint32_t)(blocks < 2048 ? blocks : 2048)), dim3(256), 0, s,
                     (uint64_t*)((uint8_t*)workspace + 256), count, (uint32_t*)workspace);
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
  if (r->row_stride > int64_t(1) << 40) return MIPS_ERR_UNSUPPORTED;
  int64_t extra = 0;
  if (S.t) {
    if (r->seq_stride < d || r->seq_stride > int64_t(1) << 44) return MIPS_ERR_INVALID_ARG;
    extra = S.b > 1 ? r->seq_stride - (int64_t)S.t * r->row_stride : 0;
  }
  *out = Rows{r->data, r->row_stride, extra};
  return MIPS_OK;
}

}  // namespace mips

using namespace mips;

extern "C" {

int64_t mips_gated_scan_carries(const mips_sequences* seq, int32_t d) {
  Sequences S;
  if (check_sequences(seq, &S) != MIPS_OK || d < 1 || d > MIPS_EMBEDDING_D_MAX) return -1;
  const Tiling T = tiling_of(S, d);
  return T.chained ? (int64_t)T.tiles : 0;
}

size_t mips_gated_scan_workspace_size(const mips_sequences* seq, int32_t d) {
  Sequences S;
  if (check_sequences(seq, &S) != MIPS_OK || d < 1 || d > MIPS_EMBEDDING_D_MAX) return 0;
  return 256 + chain_bytes(tiling_of(S, d));
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
  const Tiling T = tiling_of(A.S, d);
  if (!last || !aligned(last, 4) || !aligned(initial, 4) || !aligned(states, elem_bytes(dtype)) ||
      !aligned(workspace, 256) || (T.chained && (!workspace || !carries)) || !aligned(carries, 4))
    return MIPS_ERR_INVALID_ARG;
  if (T.chained && workspace_bytes < 256 + chain_bytes(T)) return MIPS_ERR_WORKSPACE;
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
  A.chained = T.chained;
  if (T.chained) {
    A.counter = (uint32_t*)workspace;
    A.words = (uint64_t*)((uint8_t*)workspace + 256);
    if (const int rc = chain_clear(T, workspace, s)) return rc;
  }
  const bool vec = rows_by_four(A.x, d, dtype) && rows_by_four(A.forget, d, dtype) &&
                   (!gate || rows_by_four(A.gate, d, dtype)) && aligned(states, 4 * elem_bytes(dtype));
  void (*kernel)(ScanArgs) = nullptr;
  if (dtype == MIPS_F32)
    kernel = gate ? (vec ? scan_kernel<float, true, true> : scan_kernel<float, true, false>)
                  : (vec ? scan_kernel<float, false, true> : scan_kernel<float, false, false>);
  else
    kernel = gate ? (vec ? scan_kernel<__bf16, true, true> : scan_kernel<__bf16, true, false>)
                  : (vec ? scan_kernel<__bf16, false, true> : scan_kernel<__bf16, false, false>);
  const uint64_t jobs = (uint64_t)T.tiles * T.columns;
  for (uint64_t j = 0; j < jobs; j += kMaxGridBlocks) {
    A.block0 = (uint32_t)j;
    const uint64_t left = jobs - j;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)(left < (uint64_t)kMaxGridBlocks ? left : kMaxGridBlocks)), dim3(kScanThreads), 0, s, A);
    if (const int rc = check_launch()) return rc;
  }
  return MIPS_OK;
}

}  // extern "C"
