// events.hip -- the gated recurrence for single events against a table of states (gfx950).
//
// For events e in order: row = rows[e], h = a_e state[row] + b_e x_e, state[row] = h, out[e] = h.
// A row that several events name gets them one after another: the first of them does the work
// of all, so that no two workgroups touch one row. To find out, every workgroup looks through all
// events' rows once (4 or 8 bytes each, from the caches) against a small hash table of its own.
//
// Bound by latency: ids, the look through them while the first events' rows arrive, one round of
// arithmetic. 4096 events x 128 bf16 of a million rows with gates take 6.5 us in a graph (8 MB), 16 of
// any 4.4; 65,536 take 90, mostly looking. Events of one row are a trip to memory each: 13,236 of 1265 rows 46.
#include <numeric>
#include <utility>

#include "scan.h"

namespace mips {

constexpr int kEventsMost = 128;       // events of a workgroup
constexpr uint32_t kPlaces = 1024;     // of the workgroup's rows, by their hash
constexpr int kLook = 16;              // events that a thread looks at together
constexpr uint32_t kHitsMost = 1024;   // later events of a workgroup's rows that are kept in LDS

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

// The first event after e, below b, whose row is `row`, or b: all lanes of a group together. `hits` are the
// workgroup's later events (their own event << 16 | event), in any order, if they are all there.
__device__ __forceinline__ int32_t next_event(const EventArgs& A, const uint32_t* hits, uint32_t nhits, int i,
                                              int64_t row, int32_t e, int lanes, int lane) {
  if (nhits <= kHitsMost) {
    uint32_t best = 0xFFFFFFFFu;
    for (uint32_t k = lane; k < nhits; k += lanes) {
      const uint32_t v = hits[k];
      if ((int)(v >> 16) == i && (int32_t)(v & 0xFFFFu) > e) best = min(best, v & 0xFFFFu);
    }
    for (int o = lanes >> 1; o >= 1; o >>= 1) best = min(best, (uint32_t)__shfl_xor((int)best, o));
    return best == 0xFFFFFFFFu ? A.b : (int32_t)best;
  }
  const int shift = (threadIdx.x & 63) & ~(lanes - 1);
  const uint64_t group = (lanes == 64 ? ~uint64_t(0) : (uint64_t(1) << lanes) - 1) << shift;
  for (int32_t at = e + 1; at < A.b; at += lanes) {
    const bool same = at + lane < A.b && event_row(A, at + lane) == row;
    const uint64_t m = __ballot(same) & group;  // this group's lanes are here together
    if (m) return at + (__ffsll((unsigned long long)m) - 1 - shift);
  }
  return A.b;
}

template <typename T, bool GATE, bool VEC, int THREADS>
__global__ __launch_bounds__(THREADS) void events_kernel(EventArgs A) {
  __shared__ int64_t own[kEventsMost];
  __shared__ uint32_t earlier[kEventsMost], later[kEventsMost];
  __shared__ uint32_t places[kPlaces];  // own event + 1, or 0
  __shared__ uint32_t hits[kHitsMost], nhits;
  const int tid = threadIdx.x;
  const int32_t e0 = (int32_t)blockIdx.x * A.own;
  const int count = min(A.own, A.b - e0);
  for (int i = tid; i < (int)kPlaces; i += THREADS) places[i] = 0;
  if (tid == 0) nhits = 0;
  if (tid < count) {
    own[tid] = event_row(A, e0 + tid);
    earlier[tid] = later[tid] = 0;
  }
  __syncthreads();
  if (tid < count) {
    // at most kEventsMost of kPlaces are taken: the search for a free one ends, and those below
    uint32_t v = row_hash(own[tid]);
    while (atomicCAS(&places[v], 0u, (uint32_t)tid + 1u) != 0u) v = (v + 1) & (kPlaces - 1);
  }
  __syncthreads();
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
  if (mine < count && lane * 4 < A.d && own[mine] >= 0 && own[mine] < A.table) fetch(mine, lane * 4, min(4, A.d - lane * 4));

  // many loads at once: one after another they would be most of the call
  for (int32_t first = tid; first < A.b; first += THREADS * kLook) {
    int64_t rows[kLook];
#pragma unroll
    for (int u = 0; u < kLook; ++u) rows[u] = event_row(A, min(first + u * THREADS, A.b - 1));
#pragma unroll
    for (int u = 0; u < kLook; ++u) {
      const int32_t e = first + u * THREADS;
      if (e >= A.b) break;
      for (uint32_t v = row_hash(rows[u]), p; (p = places[v]) != 0u; v = (v + 1) & (kPlaces - 1)) {
        const int i = (int)p - 1;
        if (own[i] != rows[u]) continue;
        if (e < e0 + i) {
          earlier[i] = 1;  // every writer writes the same
        } else if (e > e0 + i) {
          later[i] = 1;
          const uint32_t k = atomicAdd(&nhits, 1u);
          if (k < kHitsMost) hits[k] = (uint32_t)i << 16 | (uint32_t)e;
        }
      }
    }
  }
  __syncthreads();

  for (int i = tid >> A.lanes_log2; i < count; i += THREADS >> A.lanes_log2) {
    const int64_t row = own[i];
    const bool inside = row >= 0 && row < A.table;
    if (inside && earlier[i]) continue;
    for (int base = 0; base < A.d; base += lanes * 4) {
      const int c0 = base + lane * 4, live = min(4, A.d - c0);  // live <= 0: only looks for events
      if (!inside) {
        const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (live > 0) store4<2 * VEC>((T*)A.h + (int64_t)(e0 + i) * A.d + c0, live, zero);
        continue;
      }
      if ((i != mine || base) && live > 0) fetch(i, c0, live);
      for (int32_t e = e0 + i; e < A.b;) {
        // the next one's inputs are on their way while this one is applied
        const int32_t then = later[i] ? next_event(A, hits, nhits, i, row, e, lanes, lane) : A.b;
        const Raw<T> x0 = x, f0 = f, g0 = g;
        if (then < A.b && live > 0) inputs(then, c0, live);
        if (live > 0) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float a, na, b, nb;
            sigmoids(f0.at(c), &a, &na);
            b = na;
            if (GATE) sigmoids(g0.at(c), &b, &nb);
            h[c] = fmaf(a, h[c], b * x0.at(c));
          }
          store4<2 * VEC>((T*)A.h + (int64_t)e * A.d + c0, live, h);
        }
        e = then;
      }
      if (live > 0) store4<2 * VEC>(A.out + row * A.out_stride + c0, live, h);
    }
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
