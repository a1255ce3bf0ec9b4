// scan_grad.hip -- the gradient of the gated linear recurrence (gfx950). scan.h has the method.
//
// With G the gradient of the states (and, at a sequence's final row, of the last one),
//   D_r = G_r + a_{r+1} D_{r+1},
//   dx = D b,   dforget = D (h_{r-1} - x) a b, or D h_{r-1} a (1 - a) and dgate = D x b (1 - b),
//   dinitial = a D at the first row.
// What flows backward is u_r = a_r (G_r + u_{r+1}), again a composition of affine maps, from the
// last tile to the first. The states h_{r-1} are not read: they follow from the inputs, which are
// needed anyway, and the state before the run, which the forward call left in binary32 (an eighth of a
// bf16 tensor's rows, and a quarter of its bytes, in full tiles; taking the states from tile to tile here as well, by maps
// as the gradient, was a third more instructions, and they are what bounds this kernel).
//
// A run's rows are gone through twice: forward, for the factor of D in dforget and the run's map of u, and,
// when it is known what flows in from behind, backward for D.
//
// 4096 x 127 x 128 bf16 take 132 us (5.3 TB/s; vector units busy 59% of the time, four waves a SIMD held by
// 128 registers), 105 where half of the rows are padding; chained: 65,536 x 1024 bf16 145 (4.8 TB/s), 600,000
// x 100 packed f32 with gates 367 (4.7 TB/s). With gates bf16 spills 5 to 10 registers a thread in whole tiles, 30
// to 42 chained, f32 36 where rows do not lie by four and tiles are chained: 188 us (5.2 TB/s) for 4096 x 127 x 128 bf16.
#include <type_traits>

#include "scan.h"

namespace mips {

struct ScanGradArgs {
  Sequences S;
  Rows x, forget, gate, grad;
  const float* initial;    // [b, d] or NULL
  const float* grad_last;  // [b, d] or NULL
  const float* carries;    // [runs of all tiles, d]: the state before each run
  void *dx, *dforget, *dgate;
  float* dinitial;         // [b, d] or NULL
  const int32_t* info;     // packed rows
  uint64_t* words;
  uint32_t* counters;
  int32_t d;
  int32_t lanes_log2;
  uint32_t rows, tiles, columns;
  uint32_t block0;
  int32_t flat;
};

template <typename T, bool GATE, int VEC, bool CHAINED, int THREADS>
__global__ __launch_bounds__(THREADS, 4) void scan_grad_kernel(ScanGradArgs A) {
  constexpr int R = kRun<T>;
  extern __shared__ __attribute__((aligned(16))) uint8_t shared[];
  Shared M;
  shared_bytes(THREADS, 4 << A.lanes_log2, CHAINED, &M, shared);
  const int tid = threadIdx.x;
  const uint32_t job = A.block0 + blockIdx.x, column = job % A.columns;
  const uint32_t step = CHAINED ? chain_ticket(A.counters, column) : job / A.columns;
  const uint32_t tile = A.tiles - 1 - step;
  const uint32_t r0 = tile * A.rows;
  const uint32_t rows = min(A.rows, A.S.n - r0);
  const int width = 4 << A.lanes_log2;
  const int c0 = column * width;
  const int lanes = 1 << A.lanes_log2;
  const int ch = (tid & (lanes - 1)) * 4;
  const int live = min(4, A.d - c0 - ch);
  const uint32_t at = (uint32_t)(tid >> A.lanes_log2) * R;
  const int64_t channel = c0 + ch;
  const uint32_t from = live > 0 ? ch : 0;              // lanes without channels load those of the first
  const int some = live > 0 ? live : min(4, A.d - c0);
  const bool wide = A.d >= 4;
  const uint32_t source = CHAINED ? chain_source_back(A.S, A.info, r0 + rows - 1, A.rows, A.tiles, step) : 0;

  const Marks marks = run_marks<R>(A.S, A.info, r0, rows, at);
  const bool special = __any(marks.any());
  const bool idle = special && __all((marks.bits & ((1u << R) - 1u)) == (1u << R) - 1u);  // a wave of padding
  Raw<T> x[R], f[R], g[R], G[R];
  float h[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // the state before the run, then before each row
#pragma unroll
  for (int t = 0; t < R; ++t) x[t] = f[t] = g[t] = G[t] = Raw<T>{};
  if (!idle) {
    if (A.flat) {
      load_flat<VEC>(A.forget, r0, rows, at, c0, from, some, wide, marks, f);
      load_flat<VEC>(A.x, r0, rows, at, c0, from, some, wide, marks, x);
      if (GATE) load_flat<VEC>(A.gate, r0, rows, at, c0, from, some, wide, marks, g);
      if (A.grad.p) load_flat<VEC>(A.grad, r0, rows, at, c0, from, some, wide, marks, G);
    } else {
      load_gaps<VEC>(A.S, A.forget, r0, rows, at, c0, from, some, wide, marks, f);
      load_gaps<VEC>(A.S, A.x, r0, rows, at, c0, from, some, wide, marks, x);
      if (GATE) load_gaps<VEC>(A.S, A.gate, r0, rows, at, c0, from, some, wide, marks, g);
      if (A.grad.p) load_gaps<VEC>(A.S, A.grad, r0, rows, at, c0, from, some, wide, marks, G);
    }
    if (at < rows)
      load4<VEC>(A.carries + ((int64_t)tile * (THREADS >> A.lanes_log2) + (tid >> A.lanes_log2)) * A.d + c0 + from, some, wide, h);
  }

  // [b, d] floats at a row's sequence, for the rows that have one
  auto row4 = [&](const float* p, uint32_t row, float* v) __attribute__((always_inline)) {
    p += row_sequence(A.S, A.info, r0 + row) * A.d + channel;
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = c < live ? p[c] : 0.0f;
  };

  // forward: q, by which D is multiplied for dforget, and the run's map of what flows in from behind, v -> fa v + fb
  // (row t's own, v -> a (G + v), goes inside those before it)
  float q[R][4], fa[4], fb[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    fa[c] = idle ? kForgets : 1.0f;
    fb[c] = 0.0f;
  }
  auto forward = [&](auto plain) __attribute__((always_inline)) {
    constexpr bool PLAIN = decltype(plain)::value;  // no row of the wave begins or ends a sequence, or is padding
    bool ended = false;  // a sequence of the run has: what lies behind belongs to others
#pragma unroll
    for (int t = 0; t < R; ++t) {
      const bool has = !PLAIN && marks.wave_has(t);
      if (has) {
        ended = ended || marks.pad(t);
        if (marks.cut(t)) {
#pragma unroll
          for (int c = 0; c < 4; ++c) h[c] = 0.0f;
          if (A.initial && live > 0 && marks.first(t)) row4(A.initial, at + t, h);
        }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float up, down, b, nb;
        sigmoids(f[t].at(c), &up, &down);
        b = down;
        if (GATE) sigmoids(g[t].at(c), &b, &nb);
        const float xx = x[t].at(c);
        q[t][c] = up * down * (GATE ? h[c] : h[c] - xx);
        here(&q[t][c]);
        h[c] = fmaf(up, h[c], b * xx);
        fa[c] *= up;
        fb[c] = !PLAIN && ended ? fb[c] : fmaf(fa[c], G[t].at(c), fb[c]);
      }
      if (has && !ended && marks.final(t)) {
        ended = true;
        if (A.grad_last && live > 0) {
          float end[4];
          row4(A.grad_last, at + t, end);
#pragma unroll
          for (int c = 0; c < 4; ++c) fb[c] = fmaf(fa[c], end[c], fb[c]);
        }
      }
      if (t & 1) __builtin_amdgcn_sched_barrier(0);  // rows that are computed at once take registers
    }
    if (!PLAIN && ended) {
#pragma unroll
      for (int c = 0; c < 4; ++c) fa[c] = kForgets;
    }
  };
  if (!special) forward(std::true_type{});
  else if (!idle) forward(std::false_type{});
  half_maps<true>(tid, fa, fb, lanes, M);
  const int64_t stride = (int64_t)A.columns * width;
  const Chain C{A.words, A.words + A.tiles * stride, stride, (uint32_t)(c0 + (tid & 127))};
  join_halves<THREADS, true, CHAINED>(tid, M, C, step, source, min(width, A.d - c0), width);
  if (live <= 0) return;
  const int64_t tile0 = (int64_t)r0 * A.d + c0;
  const uint32_t pitch = (uint32_t)A.d * sizeof(T), out0 = at * pitch + ch * (uint32_t)sizeof(T);
  // A padded sequence without rows would begin at row r: its last state is its initial one
  auto none = [&](uint32_t r) __attribute__((always_inline)) {
    const int64_t i = (int64_t)(r / A.S.t) * A.d + channel;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (c < live) A.dinitial[i + c] = A.grad_last ? A.grad_last[i + c] : 0.0f;
  };
  auto nones = [&]() __attribute__((always_inline)) {
    if (!A.S.lengths || !A.dinitial) return;
    for (uint32_t m = run_nones<R>(A.S, r0 + at, marks); m; m &= m - 1) none(r0 + at + (__ffs(m) - 1));
  };
  if (idle) {
    const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
    for (int t = 0; t < R; ++t) {
      if (marks.beyond(t)) continue;
      const uint32_t out = out0 + t * pitch;
      store4<VEC>((T*)((uint8_t*)((T*)A.dx + tile0) + out), live, zero);
      store4<VEC>((T*)((uint8_t*)((T*)A.dforget + tile0) + out), live, zero);
      if (GATE) store4<VEC>((T*)((uint8_t*)((T*)A.dgate + tile0) + out), live, zero);
    }
    nones();
    return;
  }
  float u[4];  // what flows into the run from behind, then into each row
  half_reach(tid, M, lanes, u);
#pragma unroll
  for (int t = 0; t < R; ++t) {
    raw_again(&f[t]);
    raw_again(&G[t]);
    if (GATE) {
      raw_again(&g[t]);
      raw_again(&x[t]);
    }
  }
  auto backward = [&](auto plain) __attribute__((always_inline)) {
    constexpr bool PLAIN = decltype(plain)::value;
#pragma unroll
    for (int t = R - 1; t >= 0; --t) {
      const bool has = !PLAIN && marks.wave_has(t);
      const bool pad = has && marks.pad(t);
      if (has && marks.final(t)) {
#pragma unroll
        for (int c = 0; c < 4; ++c) u[c] = 0.0f;
        if (A.grad_last) row4(A.grad_last, at + t, u);
      }
      float dx[4], df[4], dg[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float D = G[t].at(c) + u[c];
        float up, down, b, nb;
        sigmoids(f[t].at(c), &up, &down);
        b = down;
        if (GATE) {
          sigmoids(g[t].at(c), &b, &nb);
          dg[c] = D * (x[t].at(c) * (b * nb));  // (D x may be past the type's largest value where the product is not)
        }
        dx[c] = D * b;
        df[c] = D * q[t][c];
        u[c] = up * D;
        if (pad) dx[c] = df[c] = dg[c] = u[c] = 0.0f;
      }
      if (t & 1) __builtin_amdgcn_sched_barrier(0);
      if (has && marks.beyond(t)) continue;
      const uint32_t out = out0 + t * pitch;
      store4<VEC>((T*)((uint8_t*)((T*)A.dx + tile0) + out), live, dx);
      store4<VEC>((T*)((uint8_t*)((T*)A.dforget + tile0) + out), live, df);
      if (GATE) store4<VEC>((T*)((uint8_t*)((T*)A.dgate + tile0) + out), live, dg);
      if (!has || !A.dinitial) continue;
      if (!marks.first(t)) continue;
      float* p = A.dinitial + row_sequence(A.S, A.info, r0 + at + t) * A.d + channel;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < live) p[c] = u[c];
    }
  };
  if (!special) return backward(std::true_type{});
  backward(std::false_type{});
  nones();
}

template <typename T, bool CHAINED, int THREADS>
static void (*grad_variant(bool gate, int vec))(ScanGradArgs) {
  if (vec == 2) return gate ? scan_grad_kernel<T, true, 2, CHAINED, THREADS> : scan_grad_kernel<T, false, 2, CHAINED, THREADS>;
  if constexpr (std::is_same<T, __bf16>::value) {
    if (vec == 1) return gate ? scan_grad_kernel<T, true, 1, CHAINED, THREADS> : scan_grad_kernel<T, false, 1, CHAINED, THREADS>;
  }
  return gate ? scan_grad_kernel<T, true, 0, CHAINED, THREADS> : scan_grad_kernel<T, false, 0, CHAINED, THREADS>;
}
static void (*grad_kernel_of(int32_t dtype, const Tiling& T, bool gate, int vec))(ScanGradArgs) {
  if (dtype == MIPS_BF16)
    return T.chained ? grad_variant<__bf16, true, kTileThreads>(gate, vec) : grad_variant<__bf16, false, kTileThreads>(gate, vec);
  if (T.threads > kTileThreads) return grad_variant<float, false, 2 * kTileThreads>(gate, vec);  // never chained
  return T.chained ? grad_variant<float, true, kTileThreads>(gate, vec) : grad_variant<float, false, kTileThreads>(gate, vec);
}

}  // namespace mips

using namespace mips;

extern "C" {

int mips_gated_scan_backward(const mips_sequences* seq, int32_t d, int32_t dtype, const mips_rows* x,
                             const mips_rows* forget, const mips_rows* gate, const float* initial,
                             const mips_rows* grad_states, const float* grad_last, const float* carries,
                             void* grad_x, void* grad_forget, void* grad_gate, float* grad_initial,
                             void* workspace, size_t workspace_bytes, void* stream) {
  ScanGradArgs A{};
  if (const int rc = check_sequences(seq, &A.S)) return rc;
  if (d < 1) return MIPS_ERR_INVALID_ARG;
  if (d > MIPS_EMBEDDING_D_MAX || (dtype != MIPS_F32 && dtype != MIPS_BF16)) return MIPS_ERR_UNSUPPORTED;
  if (const int rc = check_rows(x, A.S, d, dtype, &A.x)) return rc;
  if (const int rc = check_rows(forget, A.S, d, dtype, &A.forget)) return rc;
  if (gate) {
    if (const int rc = check_rows(gate, A.S, d, dtype, &A.gate)) return rc;
  }
  if (grad_states) {
    if (const int rc = check_rows(grad_states, A.S, d, dtype, &A.grad)) return rc;
  }
  const Tiling T = scan_tiling(A.S, d, dtype);
  const int E = elem_bytes(dtype);
  if ((!grad_states && !grad_last) || (A.S.n > 0 && (!grad_x || !grad_forget || (gate && !grad_gate))) ||
      !aligned(grad_x, E) || !aligned(grad_forget, E) || !aligned(grad_gate, E) || !aligned(initial, 4) ||
      !aligned(grad_last, 4) || !aligned(grad_initial, 4) || !aligned(carries, 4) || !aligned(workspace, 256) ||
      !carries || ((T.chained || A.S.offsets) && !workspace))
    return MIPS_ERR_INVALID_ARG;
  const ScanSpace W = scan_space(A.S, T, workspace);
  if ((T.chained || A.S.offsets) && workspace_bytes < W.bytes) return MIPS_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  A.initial = initial;
  A.grad_last = grad_last;
  A.carries = carries;
  A.dx = grad_x;
  A.dforget = grad_forget;
  A.dgate = grad_gate;
  A.dinitial = grad_initial;
  A.d = d;
  A.lanes_log2 = T.lanes_log2;
  A.rows = T.rows;
  A.tiles = T.tiles;
  A.columns = T.columns;
  A.info = W.info;
  A.words = W.words;
  A.counters = W.counters;
  if (const int rc = scan_begin(A.S, T, W, d, grad_last, grad_initial, s)) return rc;
  const uintptr_t V = 4 * E;
  const bool by_four = rows_by_four(A.x, d, dtype) && rows_by_four(A.forget, d, dtype) &&
                   (!gate || rows_by_four(A.gate, d, dtype)) && (!A.grad.p || rows_by_four(A.grad, d, dtype)) &&
                   aligned(carries, 16) && aligned(grad_x, V) && aligned(grad_forget, V) && aligned(grad_gate, V);
  A.flat = rows_flat(A.x, T, dtype) && rows_flat(A.forget, T, dtype) && (!gate || rows_flat(A.gate, T, dtype)) &&
           (!A.grad.p || rows_flat(A.grad, T, dtype));
  void (*kernel)(ScanGradArgs) = grad_kernel_of(dtype, T, gate, rows_vec(by_four, d, dtype));
  const uint64_t jobs = (uint64_t)T.tiles * T.columns, most = kMaxGridBlocks / 2;
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
