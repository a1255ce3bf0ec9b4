// scan_grad.hip -- the gradient of the gated linear recurrence (gfx950). scan.h has the method.
//
// With G the gradient of the states (and, at a sequence's final row, of the last one),
//   D_r = G_r + a_{r+1} D_{r+1},
//   dx = D b,   dforget = D (h_{r-1} - x) a b, or D h_{r-1} a (1 - a) and dgate = D x b (1 - b),
//   dinitial = a D at the first row.
// What flows backward is u_r = a_r (G_r + u_{r+1}), again a composition of affine maps, from the
// last tile to the first. The states h_{r-1} are not read: they follow from the inputs, which are
// needed anyway, and the state before the tile, which the forward call left in binary32.
#include <type_traits>

#include "scan.h"

namespace mips {

struct ScanGradArgs {
  Sequences S;
  Rows x, forget, gate, grad;
  const float* initial;    // [b, d] or NULL
  const float* grad_last;  // [b, d] or NULL
  const float* carries;    // [tiles, d], chained calls
  void *dx, *dforget, *dgate;
  float* dinitial;         // [b, d] or NULL
  const int32_t* info;     // packed rows
  uint64_t* words;
  uint32_t* counters;
  int32_t d;
  int32_t lanes_log2;
  uint32_t rows, tiles, columns;
  uint32_t block0;
  int32_t chained, flat;
};

template <typename T, bool GATE, bool VEC, int THREADS>
__global__ __launch_bounds__(THREADS, 4) void scan_grad_kernel(ScanGradArgs A) {
  constexpr int R = kRun, WAVES = THREADS / 64;
  __shared__ float2 maps[WAVES][128];   // of the state, forward
  __shared__ float2 flows[WAVES][128];  // of the gradient, backward
  __shared__ __attribute__((aligned(16))) float entry[WAVES][128], leave[WAVES][128];  // what each wave's rows start from

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint32_t job = A.block0 + blockIdx.x, column = job % A.columns;
  const uint32_t step = A.chained ? chain_ticket(A.counters, column) : job / A.columns;
  const uint32_t tile = A.tiles - 1 - step;
  const uint32_t r0 = tile * A.rows;
  const uint32_t rows = min(A.rows, A.S.n - r0);
  const int width = 4 << A.lanes_log2;
  const int c0 = column * width;
  const int lanes = 1 << A.lanes_log2;
  const int ch = (lane & (lanes - 1)) * 4;
  const int live = min(4, A.d - c0 - ch);
  const uint32_t at = (uint32_t)(tid >> A.lanes_log2) * R;
  const int64_t channel = c0 + ch;
  const uint32_t from = live > 0 ? ch : 0;
  const int some = live > 0 ? live : 1;
  const uint32_t mine = tid - 128;  // the channel that this thread takes the state of through the waves
  const float state_in = A.chained && mine < (uint32_t)min(width, A.d - c0) ? A.carries[(int64_t)tile * A.d + c0 + mine] : 0.0f;
  const uint32_t source = A.chained ? chain_source_back(A.S, A.info, r0 + rows - 1, A.rows, A.tiles, step) : 0;

  const Marks marks = run_marks<R>(A.S, A.info, r0, rows, at);
  const bool special = __any(marks.any());
  const bool idle = special && __all((marks.bits & ((1u << R) - 1u)) == (1u << R) - 1u);  // a wave of padding
  Raw<T> x[R], f[R], g[R], G[R];
  if (!A.grad.p || idle) {
#pragma unroll
    for (int t = 0; t < R; ++t) G[t] = Raw<T>{};
  }
  if (idle) {
#pragma unroll
    for (int t = 0; t < R; ++t) {
      x[t] = f[t] = Raw<T>{};
      if (GATE) g[t] = Raw<T>{};
    }
  } else {
    if (A.flat) {
      load_flat<VEC>(A.forget, r0, rows, at, c0, from, some, marks, f);
      load_flat<VEC>(A.x, r0, rows, at, c0, from, some, marks, x);
      if (GATE) load_flat<VEC>(A.gate, r0, rows, at, c0, from, some, marks, g);
      if (A.grad.p) load_flat<VEC>(A.grad, r0, rows, at, c0, from, some, marks, G);
    } else {
      load_gaps<VEC>(A.S, A.forget, r0, rows, at, c0, from, some, marks, f);
      load_gaps<VEC>(A.S, A.x, r0, rows, at, c0, from, some, marks, x);
      if (GATE) load_gaps<VEC>(A.S, A.gate, r0, rows, at, c0, from, some, marks, g);
      if (A.grad.p) load_gaps<VEC>(A.S, A.grad, r0, rows, at, c0, from, some, marks, G);
    }
  }

  // [b, d] floats at a row's sequence, for the rows that have one
  auto row4 = [&](const float* p, uint32_t row, float* v) __attribute__((always_inline)) {
    p += row_sequence(A.S, A.info, r0 + row) * A.d + channel;
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = c < live ? p[c] : 0.0f;
  };

  // maps of the run, both taken along with its rows: the state's, h -> ma h + mb, and the gradient's,
  // where row t's map of what flows in from behind, v -> a (G + v), goes inside those before it
  float a[R][4], na[R][4];
  float ea[4], eb[4], la[4], lb[4];  // what reaches the run of what reaches the wave
  {
    float ma[4], mb[4], fa[4], fb[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      ma[c] = fa[c] = 1.0f;
      mb[c] = fb[c] = 0.0f;
    }
    if (special) {
#pragma unroll
      for (int t = 0; t < R; ++t) {
        const bool pad = marks.pad(t);
        float init[4] = {0.0f, 0.0f, 0.0f, 0.0f}, end[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (A.initial && live > 0 && marks.first(t)) row4(A.initial, at + t, init);
        if (A.grad_last && live > 0 && marks.final(t)) row4(A.grad_last, at + t, end);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float b, nb;
          sigmoids(f[t].at(c), &a[t][c], &na[t][c]);
          b = na[t][c];
          if (GATE) sigmoids(g[t].at(c), &b, &nb);
          const float u = b * x[t].at(c);
          if (marks.cut(t)) {
            ma[c] = kForgets;
            mb[c] = pad ? 0.0f : fmaf(a[t][c], init[c], u);
          } else {
            mb[c] = fmaf(a[t][c], mb[c], u);
            ma[c] = ma[c] < 0.0f ? kForgets : ma[c] * a[t][c];
          }
          if (!(fa[c] < 0.0f)) {  // no sequence of the run has ended yet
            const float p = fa[c] * a[t][c];
            if (pad) {
              fa[c] = kForgets;
            } else if (marks.final(t)) {
              fb[c] = fmaf(p, G[t].at(c) + end[c], fb[c]);
              fa[c] = kForgets;
            } else {
              fb[c] = fmaf(p, G[t].at(c), fb[c]);
              fa[c] = p;
            }
          }
        }
      }
    } else {
#pragma unroll
      for (int t = 0; t < R; ++t)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float b, nb;
          sigmoids(f[t].at(c), &a[t][c], &na[t][c]);
          b = na[t][c];
          if (GATE) sigmoids(g[t].at(c), &b, &nb);
          mb[c] = fmaf(a[t][c], mb[c], b * x[t].at(c));
          ma[c] *= a[t][c];
          fb[c] = fmaf(ma[c], G[t].at(c), fb[c]);
        }
#pragma unroll
      for (int c = 0; c < 4; ++c) fa[c] = ma[c];
    }
    auto exchange = [&](auto cuts) __attribute__((always_inline)) {
      constexpr bool CUTS = decltype(cuts)::value;
      float wa[4], wb[4];
      wave_maps<false, CUTS>(ma, mb, lane, lanes, ea, eb, wa, wb);
      if (lane < lanes) {
#pragma unroll
        for (int c = 0; c < 4; ++c) maps[wave][ch + c] = float2{wa[c], wb[c]};
      }
      wave_maps<true, CUTS>(fa, fb, lane, lanes, la, lb, wa, wb);
      if (lane < lanes) {
#pragma unroll
        for (int c = 0; c < 4; ++c) flows[wave][ch + c] = float2{wa[c], wb[c]};
      }
    };
    if (special) exchange(std::true_type{});
    else exchange(std::false_type{});
  }
  __syncthreads();
  // one thread a channel takes the gradient backward through the waves, another the state forward
  const int channels = min(width, A.d - c0);
  float v = 0.0f;
  if (A.chained) {
    float ta = 1.0f, tb = 0.0f;
    if (tid < channels) {
#pragma unroll 4
      for (int w = WAVES - 1; w >= 0; --w) compose(ta, tb, flows[w][tid].x, flows[w][tid].y, &ta, &tb);
    }
    const int64_t stride = (int64_t)A.columns * width;
    const Chain C{A.words, A.words + A.tiles * stride, stride, (uint32_t)(c0 + (tid & 127))};
    v = chain_link<THREADS>(C, step, source, channels, ta, tb);
  }
  if (tid < channels) {
#pragma unroll 4
    for (int w = WAVES - 1; w >= 0; --w) {
      leave[w][tid] = v;
      v = apply(flows[w][tid].x, flows[w][tid].y, v);
    }
  } else if (tid >= 128 && tid - 128 < channels) {
    v = state_in;
#pragma unroll 4
    for (int w = 0; w < WAVES; ++w) {
      entry[w][tid - 128] = v;
      v = apply(maps[w][tid - 128].x, maps[w][tid - 128].y, v);
    }
  }
  __syncthreads();
  if (live <= 0) return;
  float h[4], u[4];  // the state before the run, the gradient that flows into it from behind
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    h[c] = apply(ea[c], eb[c], entry[wave][ch + c]);
    u[c] = apply(la[c], lb[c], leave[wave][ch + c]);
  }
  if (GATE) {
#pragma unroll
    for (int t = 0; t < R; ++t) raw_again(&g[t]);
  }
  const int64_t tile0 = (int64_t)r0 * A.d + c0;
  const uint32_t pitch = (uint32_t)A.d * sizeof(T), out0 = at * pitch + ch * (uint32_t)sizeof(T);
  auto gradients = [&](auto plain) __attribute__((always_inline)) {
    constexpr bool PLAIN = decltype(plain)::value;  // no row of the wave begins or ends a sequence, or is padding
    // backward first: D is used up, and what flows on, v = a D, takes the place of G
    float v[R][4];
#pragma unroll
    for (int t = R - 1; t >= 0; --t) {
      const bool pad = !PLAIN && marks.pad(t);
      if (!PLAIN && marks.final(t)) {
#pragma unroll
        for (int c = 0; c < 4; ++c) u[c] = 0.0f;
        if (A.grad_last) row4(A.grad_last, at + t, u);
      }
      float dx[4], dg[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float D = G[t].at(c) + u[c];
        float b = na[t][c], nb;
        if (GATE) {
          sigmoids(g[t].at(c), &b, &nb);
          dg[c] = pad ? 0.0f : D * x[t].at(c) * b * nb;
        }
        dx[c] = pad ? 0.0f : D * b;
        u[c] = pad ? 0.0f : a[t][c] * D;
        v[t][c] = u[c];
      }
      if (!PLAIN && marks.beyond(t)) continue;
      const uint32_t out = out0 + t * pitch;
      store4<VEC>((T*)((uint8_t*)((T*)A.dx + tile0) + out), live, dx);
      if (GATE) store4<VEC>((T*)((uint8_t*)((T*)A.dgate + tile0) + out), live, dg);
      if (PLAIN || !A.dinitial) continue;
      const uint32_t r = r0 + at + t;
      // a padded sequence without rows, where its first one would lie: its last state is the initial one
      const bool none = A.S.lengths && pad && r % A.S.t == 0;
      if (!none && !marks.first(t)) continue;
      const int64_t i = row_sequence(A.S, A.info, r) * A.d + channel;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < live) A.dinitial[i + c] = !none ? u[c] : (A.grad_last ? A.grad_last[i + c] : 0.0f);
    }
    if (GATE) {
#pragma unroll
      for (int t = 0; t < R; ++t) raw_again(&g[t]);
    }
#pragma unroll
    for (int t = 0; t < R; ++t) {
      if (!PLAIN && marks.cut(t)) {
#pragma unroll
        for (int c = 0; c < 4; ++c) h[c] = 0.0f;
        if (A.initial && marks.first(t)) row4(A.initial, at + t, h);
      }
      float df[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float xx = x[t].at(c);
        df[c] = !PLAIN && marks.pad(t) ? 0.0f : v[t][c] * na[t][c] * (GATE ? h[c] : h[c] - xx);
        float b = na[t][c], nb;
        if (GATE) sigmoids(g[t].at(c), &b, &nb);
        h[c] = fmaf(a[t][c], h[c], b * xx);
      }
      if (PLAIN || !marks.beyond(t)) store4<VEC>((T*)((uint8_t*)((T*)A.dforget + tile0) + out0 + t * pitch), live, df);
    }
  };
  if (special) gradients(std::false_type{});
  else gradients(std::true_type{});
}

template <int THREADS>
static void (*grad_variant(int32_t dtype, bool gate, bool vec))(ScanGradArgs) {
  if (dtype == MIPS_F32)
    return gate ? (vec ? scan_grad_kernel<float, true, true, THREADS> : scan_grad_kernel<float, true, false, THREADS>)
                : (vec ? scan_grad_kernel<float, false, true, THREADS> : scan_grad_kernel<float, false, false, THREADS>);
  return gate ? (vec ? scan_grad_kernel<__bf16, true, true, THREADS> : scan_grad_kernel<__bf16, true, false, THREADS>)
              : (vec ? scan_grad_kernel<__bf16, false, true, THREADS> : scan_grad_kernel<__bf16, false, false, THREADS>);
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
  const Tiling T = backward_tiling(A.S, d);
  const int E = elem_bytes(dtype);
  if ((!grad_states && !grad_last) || (A.S.n > 0 && (!grad_x || !grad_forget || (gate && !grad_gate))) ||
      !aligned(grad_x, E) || !aligned(grad_forget, E) || !aligned(grad_gate, E) || !aligned(initial, 4) ||
      !aligned(grad_last, 4) || !aligned(grad_initial, 4) || !aligned(carries, 4) || !aligned(workspace, 256) ||
      (T.chained && !carries) || ((T.chained || A.S.offsets) && !workspace))
    return MIPS_ERR_INVALID_ARG;
  if ((T.chained || A.S.offsets) && workspace_bytes < scan_space(A.S, T, workspace).bytes) return MIPS_ERR_WORKSPACE;
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
  A.chained = T.chained;
  const ScanSpace W = scan_space(A.S, T, workspace);
  A.info = W.info;
  A.words = W.words;
  A.counters = W.counters;
  if (const int rc = scan_begin(A.S, T, W, d, grad_last, grad_initial, s)) return rc;
  const uintptr_t V = 4 * E;
  const bool vec = rows_by_four(A.x, d, dtype) && rows_by_four(A.forget, d, dtype) &&
                   (!gate || rows_by_four(A.gate, d, dtype)) && (!A.grad.p || rows_by_four(A.grad, d, dtype)) &&
                   aligned(grad_x, V) && aligned(grad_forget, V) && aligned(grad_gate, V);
  A.flat = rows_flat(A.x, T, dtype) && rows_flat(A.forget, T, dtype) && (!gate || rows_flat(A.gate, T, dtype)) &&
           (!A.grad.p || rows_flat(A.grad, T, dtype));
  void (*kernel)(ScanGradArgs) = T.threads == 1024 ? grad_variant<1024>(dtype, gate != nullptr, vec)
                                                   : grad_variant<512>(dtype, gate != nullptr, vec);
  const uint64_t jobs = (uint64_t)T.tiles * T.columns, most = kMaxGridBlocks / 2;
  for (uint64_t j = 0; j < jobs; j += most) {
    A.block0 = (uint32_t)j;
    const uint64_t left = jobs - j;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)(left < most ? left : most)), dim3(T.threads), 0, s, A);
    if (const int rc = check_launch()) return rc;
  }
  return MIPS_OK;
}

}  // extern "C"
