// scan_grad.hip -- the gradient of the gated linear recurrence (gfx950). scan.h has the method.
//
// With G the gradient of the states (and, at a sequence's final row, of the last one),
//   D_r = G_r + a_{r+1} D_{r+1},
//   dx = D b,   dforget = D (h_{r-1} - x) a b, or D h_{r-1} a (1 - a) and dgate = D x b (1 - b),
//   dinitial = a D at the first row.
// What flows backward is u_r = a_r (G_r + u_{r+1}), again a composition of affine maps, from the
// last tile to the first. The states h_{r-1} are not read: they follow from the inputs, which are
// needed anyway, and the state before the tile, which the forward call left in binary32.
#include "scan.h"

namespace mips {

constexpr int kGradThreads = 1024;
constexpr int kGradRun = kTileThreadRows / kGradThreads;

struct ScanGradArgs {
  Sequences S;
  Rows x, forget, gate, grad;
  const float* initial;    // [b, d] or NULL
  const float* grad_last;  // [b, d] or NULL
  const float* carries;    // [tiles, d], chained calls
  void *dx, *dforget, *dgate;
  float* dinitial;         // [b, d] or NULL
  uint64_t* words;
  uint32_t* counter;
  int32_t d;
  int32_t lanes_log2;
  uint32_t rows, tiles, columns;
  uint32_t block0;
  int32_t chained;
};

template <typename T, bool GATE, bool VEC>
__global__ __launch_bounds__(kGradThreads) void scan_grad_kernel(ScanGradArgs A) {
  constexpr int R = kGradRun, WAVES = kGradThreads / 64;
  __shared__ __attribute__((aligned(8))) uint8_t kind[kTileRowsMost];
  __shared__ int32_t first[kTileRowsMost], final[kTileRowsMost];
  __shared__ float2 maps[WAVES][128];   // of the state, forward
  __shared__ float2 flows[WAVES][128];  // of the gradient, backward
  __shared__ float before[128], behind[128];
  __shared__ uint32_t ticket;

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  uint32_t job = A.block0 + blockIdx.x;
  if (A.chained) {
    if (tid == 0) ticket = atomicAdd(A.counter, 1u);
    __syncthreads();
    job = ticket;
  }
  const uint32_t step = job / A.columns, column = job - step * A.columns;
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
  const bool owner = tid < width && c0 + tid < A.d;  // of a channel's state and gradient between tiles
  float state_in = 0.0f;
  if (A.chained && owner) state_in = A.carries[(int64_t)tile * A.d + c0 + tid];

  Raw<T> x[R], f[R], g[R], G[R];
  auto load = [&](bool all, uint32_t kinds) __attribute__((always_inline)) {
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
      raw_zero(&G[t]);
      const bool want = all ? at + t < rows : ((kinds >> (8 * t)) & (kPad | kBeyond)) == 0;
      if (want && live > 0) {
        const int64_t r = (int64_t)r0 + at + t;
        raw_load<VEC>((const T*)A.x.p + r * A.x.row + s * A.x.extra + channel, live, &x[t]);
        raw_load<VEC>((const T*)A.forget.p + r * A.forget.row + s * A.forget.extra + channel, live, &f[t]);
        if (GATE) raw_load<VEC>((const T*)A.gate.p + r * A.gate.row + s * A.gate.extra + channel, live, &g[t]);
        if (A.grad.p) raw_load<VEC>((const T*)A.grad.p + r * A.grad.row + s * A.grad.extra + channel, live, &G[t]);
      }
      if (dense && ++pos == A.S.t) {
        pos = 0;
        ++s;
      }
    }
  };
  if (!A.S.lengths) load(true, 0);
  const uint32_t space = kTileThreadRows >> A.lanes_log2;
  mark_rows<kGradThreads>(A.S, r0, rows, space, tile + 1 == A.tiles, kind, first, final, [&](int32_t s) {
    // the last state of a sequence without rows is its initial one
    if (!A.dinitial) return;
    for (int c = c0; c < min(A.d, c0 + width); ++c)
      A.dinitial[(int64_t)s * A.d + c] = A.grad_last ? A.grad_last[(int64_t)s * A.d + c] : 0.0f;
  });
  const uint32_t kinds = *(const uint32_t*)&kind[at];
  if (A.S.lengths) load(false, kinds);
  const bool special = __any(kinds != 0);

  // [b, d] floats at a row's sequence, for the rows that have one
  auto row4 = [&](const float* p, int32_t s, float* v) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = c < live ? p[(int64_t)s * A.d + channel + c] : 0.0f;
  };
  auto kind_at = [&](int t) __attribute__((always_inline)) { return (kinds >> (8 * t)) & 255u; };

  // maps of the run: the state's from its first row to its last, the gradient's the other way
  float a[R][4], ma[4], mb[4], fa[4], fb[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    ma[c] = 1.0f;
    mb[c] = 0.0f;
  }
#pragma unroll
  for (int t = 0; t < R; ++t) {
    const uint32_t k = special ? kind_at(t) : 0u;
    float init[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if ((k & kFirst) && A.initial && live > 0) row4(A.initial, first[at + t], init);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float na, b, nb;
      sigmoids(f[t].at(c), &a[t][c], &na);
      b = na;
      if (GATE) sigmoids(g[t].at(c), &b, &nb);
      const float u = b * x[t].at(c);
      if (k & kCut) {
        ma[c] = kForgets;
        mb[c] = (k & kFirst) ? fmaf(a[t][c], init[c], u) : 0.0f;
      } else {
        mb[c] = fmaf(a[t][c], mb[c], u);
        ma[c] = ma[c] < 0.0f ? kForgets : ma[c] * a[t][c];
      }
    }
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    fa[c] = 1.0f;
    fb[c] = 0.0f;
  }
#pragma unroll
  for (int t = R - 1; t >= 0; --t) {
    const uint32_t k = special ? kind_at(t) : 0u;
    const bool pad = (k & (kPad | kBeyond)) != 0;
    float end[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if ((k & kFinal) && !pad && A.grad_last && live > 0) row4(A.grad_last, final[at + t], end);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (pad || (k & kFinal)) {
        fa[c] = kForgets;
        fb[c] = pad ? 0.0f : a[t][c] * (G[t].at(c) + end[c]);
      } else {
        fb[c] = a[t][c] * (G[t].at(c) + fb[c]);
        fa[c] = fa[c] < 0.0f ? kForgets : fa[c] * a[t][c];
      }
    }
  }
  for (int o = lanes; o < 64; o <<= 1) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float pa = __shfl_up(ma[c], o), pb = __shfl_up(mb[c], o);
      const float qa = __shfl_down(fa[c], o), qb = __shfl_down(fb[c], o);
      if (lane >= o) compose(pa, pb, ma[c], mb[c], &ma[c], &mb[c]);
      if (lane + o < 64) compose(qa, qb, fa[c], fb[c], &fa[c], &fb[c]);
    }
  }
  if (lane >= 64 - lanes) {
#pragma unroll
    for (int c = 0; c < 4; ++c) maps[wave][ch + c] = float2{ma[c], mb[c]};
  }
  if (lane < lanes) {
#pragma unroll
    for (int c = 0; c < 4; ++c) flows[wave][ch + c] = float2{fa[c], fb[c]};
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    ma[c] = __shfl_up(ma[c], lanes);
    mb[c] = __shfl_up(mb[c], lanes);
    fa[c] = __shfl_down(fa[c], lanes);
    fb[c] = __shfl_down(fb[c], lanes);
    if (lane < lanes) {
      ma[c] = 1.0f;
      mb[c] = 0.0f;
    }
    if (lane >= 64 - lanes) {
      fa[c] = 1.0f;
      fb[c] = 0.0f;
    }
  }
  if (owner) before[tid] = state_in;
  __syncthreads();
  if (A.chained) {
    if (owner) {
      float fa1 = 1.0f, fb1 = 0.0f;
#pragma unroll
      for (int w = WAVES - 1; w >= 0; --w) compose(fa1, fb1, flows[w][tid].x, flows[w][tid].y, &fa1, &fb1);
      const int64_t stride = (int64_t)A.columns * width;
      uint64_t* own = A.words + step * stride + c0 + tid;
      // a tile whose last row is not the end of its sequence needs the gradient from behind it
      const bool needs = step > 0 && (kind[rows - 1] & (kFinal | kPad)) == 0;
      if (!needs || fa1 < 0.0f) chain_put(own, chain_word(kState, fb1));
      else chain_put(own, chain_map(fa1, fb1));
      float flow = 0.0f;
      if (needs) {
        flow = chain_state(A.words + c0 + tid, stride, step);
        if (!(fa1 < 0.0f)) chain_put(own, chain_word(kState, fmaf(fa1, flow, fb1)));
      }
      behind[tid] = flow;
    }
    __syncthreads();
  }
  float h[4], u[4];  // the state before the run, the gradient that flows into it from behind
  {
    float wa[4] = {1.0f, 1.0f, 1.0f, 1.0f}, wb[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int w = 0; w < wave; ++w) {
#pragma unroll
      for (int c = 0; c < 4; ++c) compose(wa[c], wb[c], maps[w][ch + c].x, maps[w][ch + c].y, &wa[c], &wb[c]);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) h[c] = apply(ma[c], mb[c], apply(wa[c], wb[c], before[ch + c]));
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      wa[c] = 1.0f;
      wb[c] = 0.0f;
    }
    for (int w = WAVES - 1; w > wave; --w) {
#pragma unroll
      for (int c = 0; c < 4; ++c) compose(wa[c], wb[c], flows[w][ch + c].x, flows[w][ch + c].y, &wa[c], &wb[c]);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
      u[c] = apply(fa[c], fb[c], apply(wa[c], wb[c], A.chained ? behind[ch + c] : 0.0f));
  }
  if (live <= 0) return;

  float prev[R][4];  // the state before each row
#pragma unroll
  for (int t = 0; t < R; ++t) {
    const uint32_t k = special ? kind_at(t) : 0u;
    if (k & kCut) {
#pragma unroll
      for (int c = 0; c < 4; ++c) h[c] = 0.0f;
      if ((k & kFirst) && A.initial) row4(A.initial, first[at + t], h);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      prev[t][c] = h[c];
      float up, na, b, nb;
      sigmoids(f[t].at(c), &up, &na);
      b = na;
      if (GATE) sigmoids(g[t].at(c), &b, &nb);
      h[c] = fmaf(a[t][c], h[c], b * x[t].at(c));
    }
  }
#pragma unroll
  for (int t = R - 1; t >= 0; --t) {
    const uint32_t k = special ? kind_at(t) : 0u;
    if (k & kBeyond) continue;
    const bool pad = (k & kPad) != 0;
    const int64_t out = ((int64_t)r0 + at + t) * A.d + channel;
    if (k & kFinal) {
#pragma unroll
      for (int c = 0; c < 4; ++c) u[c] = 0.0f;
      if (A.grad_last && !pad) row4(A.grad_last, final[at + t], u);
    }
    float dx[4], df[4], dg[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float up, na, b, nb;
      sigmoids(f[t].at(c), &up, &na);
      const float D = G[t].at(c) + u[c], aa = a[t][c], xx = x[t].at(c);
      if (GATE) {
        sigmoids(g[t].at(c), &b, &nb);
        df[c] = D * prev[t][c] * aa * na;
        dg[c] = D * xx * b * nb;
      } else {
        b = na;
        df[c] = D * (prev[t][c] - xx) * aa * na;
      }
      dx[c] = D * b;
      u[c] = aa * D;
      if (pad) dx[c] = df[c] = dg[c] = u[c] = 0.0f;
    }
    store4<VEC>((T*)A.dx + out, live, dx);
    store4<VEC>((T*)A.dforget + out, live, df);
    if (GATE) store4<VEC>((T*)A.dgate + out, live, dg);
    if ((k & (kFirst | kPad)) == kFirst && A.dinitial) {
      float* p = A.dinitial + (int64_t)first[at + t] * A.d + channel;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < live) p[c] = u[c];
    }
  }
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
  const Tiling T = tiling_of(A.S, d);
  const int E = elem_bytes(dtype);
  if ((!grad_states && !grad_last) || (A.S.n > 0 && (!grad_x || !grad_forget || (gate && !grad_gate))) ||
      !aligned(grad_x, E) || !aligned(grad_forget, E) || !aligned(grad_gate, E) || !aligned(initial, 4) ||
      !aligned(grad_last, 4) || !aligned(grad_initial, 4) || !aligned(carries, 4) || !aligned(workspace, 256) ||
      (T.chained && (!workspace || !carries)))
    return MIPS_ERR_INVALID_ARG;
  if (T.chained && workspace_bytes < 256 + chain_bytes(T)) return MIPS_ERR_WORKSPACE;
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
  if (T.chained) {
    A.counter = (uint32_t*)workspace;
    A.words = (uint64_t*)((uint8_t*)workspace + 256);
    if (const int rc = chain_clear(T, workspace, s)) return rc;
  }
  const uintptr_t V = 4 * E;
  const bool vec = rows_by_four(A.x, d, dtype) && rows_by_four(A.forget, d, dtype) &&
                   (!gate || rows_by_four(A.gate, d, dtype)) && (!A.grad.p || rows_by_four(A.grad, d, dtype)) &&
                   aligned(grad_x, V) && aligned(grad_forget, V) && aligned(grad_gate, V);
  void (*kernel)(ScanGradArgs) = nullptr;
  if (dtype == MIPS_F32)
    kernel = gate ? (vec ? scan_grad_kernel<float, true, true> : scan_grad_kernel<float, true, false>)
                  : (vec ? scan_grad_kernel<float, false, true> : scan_grad_kernel<float, false, false>);
  else
    kernel = gate ? (vec ? scan_grad_kernel<__bf16, true, true> : scan_grad_kernel<__bf16, true, false>)
                  : (vec ? scan_grad_kernel<__bf16, false, true> : scan_grad_kernel<__bf16, false, false>);
  const uint64_t jobs = (uint64_t)T.tiles * T.columns;
  for (uint64_t j = 0; j < jobs; j += kMaxGridBlocks / 2) {
    A.block0 = (uint32_t)j;
    const uint64_t left = jobs - j, most = kMaxGridBlocks / 2;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)(left < most ? left : most)), dim3(kGradThreads), 0, s, A);
    if (const int rc = check_launch()) return rc;
  }
  return MIPS_OK;
}

}  // extern "C"
