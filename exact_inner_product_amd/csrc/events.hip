// events.hip -- the gated recurrence for single events against a table of states (gfx950).
//
// For events e in order: row = rows[e], h = a_e state[row] + b_e x_e, state[row] = h, out[e] = h.
// A row that several events name gets them one after another: the first of them does the work
// of all, so that no two workgroups touch one row. To find out, every workgroup looks through all
// events' rows once (4 or 8 bytes each, from the caches) against a small hash table of its own.
//
// Bound by latency: ids, the look through them while the first events' rows arrive, one round of
// arithmetic. In graphs 16 events of any size take 4.4 us, 4096 x 128 bf16 of a million rows with gates 7.2 (8
// MB), 65,536 without 77, mostly looking, and 58 if half of them are padding. Events of one row are a trip to
// memory each: 13,236 of 1265 rows take 31 us, 65,536 of which 30% name one row 6.8 ms.
#include <numeric>
#include <utility>

#include "scan.h"

namespace mips {

constexpr int kEventsMost = 128;       // events of a workgroup
constexpr uint32_t kPlaces = 1024;     // of the workgroup's rows, by their hash
constexpr int kLook = 16;              // events that a thread looks at together
constexpr uint32_t kHitsMost = 1024;   // later events of a workgroup's rows that it takes at once
static_assert(kHitsMost >= (uint32_t)kEventsMost, "a workgroup's events lie in its first window");

struct EventArgs {
  const void *x, *forget, *gate;
  int64_t x_stride, forget_stride, gate_stride;
  const float* state;
  float* out;       // [rows, d], may be `state`
  int64_t state_stride, out_stride;
  int64_t table;    // rows of it
  const void* ids;
  int32_t wide;
  int32_t b, d;
  int32_t own;      // events of a workgroup
  int32_t lanes_log2;
  void* h;          // [b, d]
};

__device__ __forceinline__ int64_t event_row(const EventArgs& A, int64_t e) {
  return A.wide ? ((const int64_t*)A.ids)[e] : (int64_t)((const int32_t*)A.ids)[e];
}
__device__ __forceinline__ uint32_t row_hash(int64_t row) {
  return ((uint32_t)row * 2654435761u + (uint32_t)(row >> 32) * 40503u) >> (32 - 10);
}

// Rows outside the table are not entered in the hash table: nothing is found for them. All events are looked through
// once: those before the workgroup's own say which of its rows another one has, those behind are sorted by row and
// event. Where these are too many, as they are with a row of a thousand events, they are taken in windows of as
// many events as there is room for, those of rows that another workgroup has left out.
template <typename T, bool GATE, bool VEC, int THREADS>
__global__ __launch_bounds__(THREADS) void events_kernel(EventArgs A) {
  __shared__ int64_t own[kEventsMost];
  __shared__ uint32_t taken[kEventsMost];  // its row is another event's: of this workgroup or of one before
  __shared__ uint32_t later[kEventsMost];  // events of its row behind it, of those found
  __shared__ uint32_t start[kEventsMost];  // of them in `order`
  __shared__ uint32_t places[kPlaces];     // own event + 1, the first of its row here, or 0
  __shared__ __attribute__((aligned(16))) uint32_t hits[kHitsMost + 4];  // own event << 16 | event, as found
  __shared__ uint32_t nhits;
  __shared__ uint16_t order[kHitsMost];    // events by row, then as they come
  const int tid = threadIdx.x;
  const int32_t e0 = (int32_t)blockIdx.x * A.own;
  const int count = min(A.own, A.b - e0);
  for (int i = tid; i < (int)kPlaces; i += THREADS) places[i] = 0;
  if (tid == 0) nhits = 0;
  if (tid < count) {
    own[tid] = event_row(A, e0 + tid);
    taken[tid] = later[tid] = 0;
  }
  __syncthreads();
  auto inside = [&](int64_t row) __attribute__((always_inline)) { return (uint64_t)row < (uint64_t)A.table; };
  if (tid < count && inside(own[tid])) {
    // at most kEventsMost of kPlaces are taken: the search for a free one ends, and those below
    for (uint32_t v = row_hash(own[tid]);; v = (v + 1) & (kPlaces - 1)) {
      const uint32_t p = atomicCAS(&places[v], 0u, (uint32_t)tid + 1u);
      if (p == 0u) break;
      if (own[p - 1] != own[tid]) continue;
      const uint32_t was = atomicMin(&places[v], (uint32_t)tid + 1u);  // (a place stays its row's)
      taken[max(was, (uint32_t)tid + 1u) - 1] = 1;
      break;
    }
  }
  // what the group's first event reads is on its way while its row is looked for
  const int lanes = 1 << A.lanes_log2, lane = tid & (lanes - 1), mine = tid >> A.lanes_log2;
  float h[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  Raw<T> x{}, f{}, g{};
  const bool wide = A.d >= 4;
  auto inputs = [&](int32_t e, int c0, int live) __attribute__((always_inline)) {
    raw_load<VEC>((const T*)A.x + e * A.x_stride + c0, live, wide, &x);
    raw_load<VEC>((const T*)A.forget + e * A.forget_stride + c0, live, wide, &f);
    if (GATE) raw_load<VEC>((const T*)A.gate + e * A.gate_stride + c0, live, wide, &g);
  };
  auto fetch = [&](int i, int c0, int live) __attribute__((always_inline)) {
    load4<VEC>(A.state + own[i] * A.state_stride + c0, live, wide, h);
    inputs(e0 + i, c0, live);
  };
  if (mine < count && lane * 4 < A.d && inside(own[mine])) fetch(mine, lane * 4, min(4, A.d - lane * 4));
  __syncthreads();

  // calls found(i, e) for events e of [from, to) with the row of own event i, its first here; many loads at
  // once: one after another they would be most of the call
  auto look = [&](int32_t from, int32_t to, auto found) __attribute__((always_inline)) {
    for (int32_t first = from + tid; first < to; first += THREADS * kLook) {
      int64_t rows[kLook];
#pragma unroll
      for (int u = 0; u < kLook; ++u) rows[u] = event_row(A, min(first + u * THREADS, to - 1));
#pragma unroll
      for (int u = 0; u < kLook; ++u) {
        const int32_t e = first + u * THREADS;
        if (e >= to) break;
        for (uint32_t v = row_hash(rows[u]), p; (p = places[v]) != 0u; v = (v + 1) & (kPlaces - 1)) {
          const int i = (int)p - 1;
          if (own[i] == rows[u]) found(i, e);  // (and on to a free place: leaving here took 90 us for 77, 65,536 events)
        }
      }
    }
  };
  auto hit = [&](int i, int32_t e) __attribute__((always_inline)) {
    atomicAdd(&later[i], 1u);
    const uint32_t k = atomicAdd(&nhits, 1u);
    if (k < kHitsMost) hits[k] = (uint32_t)i << 16 | (uint32_t)e;
  };
  look(0, A.b, [&](int i, int32_t e) __attribute__((always_inline)) {
    if (e < e0) taken[i] = 1;  // every writer writes the same
    else if (e > e0 + i) hit(i, e);
  });
  __syncthreads();
  const bool whole = nhits <= kHitsMost;
  for (int32_t w0 = e0;; w0 += kHitsMost) {
    if (!whole) {
      __syncthreads();  // nothing of the window before is read any more
      if (tid < count) later[tid] = 0;
      if (tid == 0) nhits = 0;
      __syncthreads();
      look(w0, min(w0 + (int32_t)kHitsMost, A.b), [&](int i, int32_t e) __attribute__((always_inline)) {
        if (e > e0 + i && !taken[i]) hit(i, e);
      });
      __syncthreads();
    }
    const uint32_t n = nhits;
    if (n) {
      if (tid < 4) hits[n + tid] = 0xFFFFFFFFu;
      __syncthreads();
      for (uint32_t k = tid; k < n; k += THREADS) {
        const uint32_t v = hits[k], row = v & 0xFFFF0000u;
        uint32_t at = 0, begin = 0;
        for (uint32_t j = 0; j < n; j += 4) {
          const uint4 q = *(const uint4*)(hits + j);
          at += (q.x < v) + (q.y < v) + (q.z < v) + (q.w < v);
          begin += (q.x < row) + (q.y < row) + (q.z < row) + (q.w < row);
        }
        order[at] = (uint16_t)v;
        start[v >> 16] = begin;  // the same from each of the row's
      }
      __syncthreads();
    }

    const bool first = w0 == e0;
    for (int i = mine; i < count; i += THREADS >> A.lanes_log2) {
      const bool none = !inside(own[i]);
      if (none ? !first : taken[i] || !(first || later[i])) continue;
      for (int c0 = lane * 4; c0 < A.d; c0 += lanes * 4) {
        const int live = min(4, A.d - c0);
        if (none) {
          const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          store4<2 * VEC>((T*)A.h + (int64_t)(e0 + i) * A.d + c0, live, zero);
          continue;
        }
        uint32_t left = later[i];
        const uint16_t* next = order + (left ? start[i] : 0);
        int32_t e = e0 + i;
        if (!first) {  // goes on from the window before, whose state this lane wrote
          e = *next++;
          --left;
          load4<VEC>(A.out + own[i] * A.out_stride + c0, live, wide, h);
          inputs(e, c0, live);
        } else if (i != mine || c0 != lane * 4) {
          fetch(i, c0, live);
        }
        for (;;) {
          // the next one's inputs are on their way while this one is applied
          const Raw<T> x0 = x, f0 = f, g0 = g;
          const int32_t then = left ? *next++ : 0;
          if (left) inputs(then, c0, live);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float a, na, b, nb;
            sigmoids(f0.at(c), &a, &na);
            b = na;
            if (GATE) sigmoids(g0.at(c), &b, &nb);
            h[c] = fmaf(a, h[c], b * x0.at(c));
          }
          store4<2 * VEC>((T*)A.h + (int64_t)e * A.d + c0, live, h);
          if (!left) break;
          --left;
          e = then;
        }
        store4<2 * VEC>(A.out + own[i] * A.out_stride + c0, live, h);
      }
    }
    if (whole || w0 + (int32_t)kHitsMost >= A.b) break;
  }
}

template <typename T, int THREADS>
static void (*events_variant(bool gate, bool vec))(EventArgs) {
  return gate ? (vec ? events_kernel<T, true, true, THREADS> : events_kernel<T, true, false, THREADS>)
              : (vec ? events_kernel<T, false, true, THREADS> : events_kernel<T, false, false, THREADS>);
}

// Whether rows of two tables may share elements: their extents meet, and so do their columns, as they lie
// in rows of the strides' common divisor (one tensor's columns, whichever of its rows each table has).
static bool tables_overlap(const float* p, int64_t p_stride, const float* q, int64_t q_stride, int64_t rows, int32_t d) {
  if (p > q) {
    std::swap(p, q);
    std::swap(p_stride, q_stride);
  }
  const uint64_t apart = ((uint64_t)q - (uint64_t)p) / 4;
  if (apart >= (uint64_t)(rows - 1) * p_stride + d) return false;
  const uint64_t pitch = std::gcd(p_stride, q_stride), in = apart % pitch;
  return in < (uint64_t)d || in + d > pitch;
}

}  // namespace mips

using namespace mips;

extern "C" int mips_gated_step(const void* x, int64_t x_stride, const void* forget, int64_t forget_stride,
                               const void* gate, int64_t gate_stride, int32_t dtype, int32_t b, int32_t d,
                               const float* state, int64_t state_stride, float* out_state, int64_t out_stride,
                               int64_t rows, const void* ids, int32_t id_bits, void* out, void* stream) {
  if (b < 0 || d < 1 || rows < 1 || x_stride < d || forget_stride < d || (gate && gate_stride < d) ||
      state_stride < d || out_stride < d)
    return MIPS_ERR_INVALID_ARG;
  if ((dtype != MIPS_F32 && dtype != MIPS_BF16) || (id_bits != 32 && id_bits != 64) || d > MIPS_EMBEDDING_D_MAX ||
      b > MIPS_EVENTS_MAX)
    return MIPS_ERR_UNSUPPORTED;
  if (b == 0) return MIPS_OK;
  const int E = elem_bytes(dtype);
  if (!x || !forget || !state || !out_state || !ids || !out || !aligned(x, E) || !aligned(forget, E) || !aligned(gate, E) ||
      !aligned(out, E) || !aligned(state, 4) || !aligned(out_state, 4) || !aligned(ids, id_bits / 8) ||
      (out_state == state ? out_stride != state_stride : tables_overlap(state, state_stride, out_state, out_stride, rows, d)))
    return MIPS_ERR_INVALID_ARG;
  EventArgs A{x, forget, gate, x_stride, forget_stride, gate_stride, state, out_state, state_stride, out_stride,
              rows, ids, id_bits == 64, b, d, 0, 0, out};
  A.lanes_log2 = d > 128 ? 6 : d > 64 ? 5 : d > 32 ? 4 : d > 16 ? 3 : 2;
  // Large workgroups where there are many events: each looks through all of them. A workgroup's events
  // are one round of its threads (more, one after another, are so many trips to memory) as long as that
  // leaves no more workgroups than run at once, and fewer where it leaves units idle (7851 events x 16 of
  // 4300 rows: 39 us with 128 a workgroup, 16 with 16; 20 with 8, whose 982 workgroups look through more).
  const int threads = b > 1024 ? 1024 : 256;
  int own = threads >> A.lanes_log2;
  while (own < kEventsMost && b / own > 512) own *= 2;
  while (own > 1 && b / own < 256) own /= 2;
  A.own = own < kEventsMost ? own : kEventsMost;
  const int64_t strides = x_stride | forget_stride | (gate ? gate_stride : 0);
  const bool vec = d % 4 == 0 && strides % 4 == 0 && state_stride % 4 == 0 && aligned(x, 4 * E) && aligned(forget, 4 * E) &&
                   aligned(gate, 4 * E) && aligned(out, 4 * E) && aligned(state, 16) && out_stride % 4 == 0 &&
                   aligned(out_state, 16);
  void (*kernel)(EventArgs) = nullptr;
  if (dtype == MIPS_F32) kernel = threads == 1024 ? events_variant<float, 1024>(gate, vec) : events_variant<float, 256>(gate, vec);
  else kernel = threads == 1024 ? events_variant<__bf16, 1024>(gate, vec) : events_variant<__bf16, 256>(gate, vec);
  hipLaunchKernelGGL(kernel, dim3((b + A.own - 1) / A.own), dim3(threads), 0, (hipStream_t)stream, A);
  return check_launch();
}
