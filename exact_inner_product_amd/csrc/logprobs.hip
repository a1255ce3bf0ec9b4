// logprobs.hip -- log probabilities of given items under a softmax over an item table, with
// the log-sum-exp, the entropy and the most likely alternatives (gfx950): the entry point and
// the passes behind the statistics pass of softmax.h.
//
// Alternatives. The statistics pass leaves the largest logit of each run of tiles per query. The
// k best items lie in the k best runs, ordered by (largest logit descending, run ascending): for
// an item outside them, each of those k runs holds an item with a larger logit, or with an equal
// one and a lower id. The same holds for groups of runs. So the finish pass picks the k best
// groups, among their runs the k best, scores those runs' rows again with the same matrix
// instructions (bitwise the same scores) and picks the k best rows: exact, with ties by the
// lowest id, at the cost of k runs of rows a query instead of a second pass over the table. Logits of
// NaN, -inf and down to kLeastLogit are no candidates, neither as a run's maximum nor as a row.
#include "host.h"
#include "softmax_api.h"

namespace mips {

constexpr int kGroupThreads = 256;
constexpr int64_t kTopDirect = 2048;   // runs that the finish pass reads without groups
constexpr int64_t kTopGroups = 16384;  // groups that it reads, at most
constexpr int64_t kKeyBytes = 32 * 1024;  // keys of the rescored rows, at most
constexpr size_t kBmaxBytes = size_t(1) << 30;  // run maxima of one batch of queries, at most

// The largest value of each group of `per` runs, for 32 queries at a time: one thread per
// (query column, group), reading 128-byte rows of the maxima (50 x 10M: 10 MB of maxima in 7.5 us).
__global__ __launch_bounds__(kGroupThreads) void group_max_kernel(const float* __restrict__ bmax, int64_t nruns,
                                                                  int per, int64_t ngroups, int64_t gblocks,
                                                                  float* __restrict__ gmax) {
  const int64_t f = blockIdx.x / gblocks;
  const int64_t g = (blockIdx.x % gblocks) * (kGroupThreads / kFrag) + (threadIdx.x >> 5);
  if (g >= ngroups) return;
  const int64_t t0 = g * per, t1 = min(nruns, t0 + per);
  const float* p = bmax + f * nruns * kFrag + (threadIdx.x & 31);
  float m = -INFINITY;
#pragma unroll 8
  for (int64_t t = t0; t < t1; ++t) m = fmaxf(m, p[t * kFrag]);
  gmax[(f * ngroups + g) * kFrag + (threadIdx.x & 31)] = m;
}

struct FinishArgs {
  Table items, queries;
  bool packed_f32;           // items hold dims 8c + 2t + h (a packed f32 corpus)
  int b;
  const float* bias;
  const uint32_t* exclude;
  int64_t exclude_words;
  float scale;
  int nslices;
  const float4* part;
  const void* ids;           // [b, g]
  int id_bits, g, k;
  const float *bmax, *gmax;  // gmax NULL: no groups
  int64_t nruns, ngroups;
  int per_log, rm_log;       // runs of a group, 32-row blocks of a run: powers of two
  float *logprobs, *lse, *entropy, *alt_logprobs;
  int32_t* alt_ids;
};

// Chunks 0 .. NCH - 1 of 32 item rows, lane (l, h) loading its half h of each chunk of row l.
template <bool ROWS, int NCH>
__device__ __forceinline__ void load_chunks(const Table& items, int64_t row, u32x4_t (&a)[NCH]) {
  const int h = (threadIdx.x & 63) >> 5;
  if constexpr (ROWS) {
    const uint8_t* p = items.p + row * items.stride_b + 16 * h;
    const int left = items.row_b - 16 * h;  // chunks at or past the row's end are zero
#pragma unroll
    for (int c = 0; c < NCH; ++c) a[c] = 32 * c < left ? *(const u32x4_t*)(p + 32 * c) : u32x4_t{0u, 0u, 0u, 0u};
  } else {
    const uint8_t* p = items.p + (row >> 5) * (NCH * (int64_t)kChunkBytes) + ((row & 31) + 32 * h) * 16;
#pragma unroll
    for (int c = 0; c < NCH; ++c) a[c] = *(const u32x4_t*)(p + c * kChunkBytes);
  }
}

// The scores of 32 item rows with 32 query columns, of which the diagonal is taken: lane (l, h)
// gives its halves of row l and of column l's query, and gets the score of row l with it if
// diagonal() holds, else nothing. The accumulation of the statistics pass, chunk by chunk, so
// bitwise its scores.
__device__ __forceinline__ bool diagonal() { return (((threadIdx.x >> 2) & 1) ^ ((threadIdx.x >> 5) & 1)) == 0; }
template <int CT, int NCH>
__device__ __forceinline__ float score_rows(const u32x4_t (&a)[NCH], const u32x4_t (&q)[NCH]) {
  const int lane = threadIdx.x & 63;
  f32x16_t acc = {};
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    if constexpr (CT == MIPS_BF16) {
      acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a[c]),
                                                    __builtin_bit_cast(bf16x8_t, q[c]), acc, 0, 0, 0);
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[c][t]), __uint_as_float(q[c][t]), acc, 0, 0, 0);
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) s = acc_row(i, lane) == (lane & 31) ? acc[i] : s;
  return s;
}

__device__ __forceinline__ float logit(const FinishArgs& A, float s, float bias) {
  const float l = __fmul_rn(s, A.scale);
  return A.bias ? __fadd_rn(l, bias) : l;
}

// Of a query that is left without an item (lse -inf, by bitmap or biases) every item's is -inf.
__device__ __forceinline__ float log_prob(float l, float lse) { return lse == -INFINITY ? -INFINITY : l - lse; }

__device__ __forceinline__ bool excluded(const FinishArgs& A, int q, int64_t row) {
  if (!A.exclude) return false;
  return (A.exclude[(int64_t)q * A.exclude_words + (row >> 5)] >> (row & 31)) & 1u;
}

// The lane's halves of a query's chunks, in the order of the item rows'.
template <int NCH>
__device__ __forceinline__ void query_chunks(const FinishArgs& A, int64_t b, u32x4_t (&q)[NCH]) {
  const int h = (threadIdx.x & 63) >> 5;
  const uint8_t* row = A.queries.p + b * A.queries.stride_b;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    q[c] = u32x4_t{0u, 0u, 0u, 0u};
    if (A.packed_f32) {
      const uint32_t* r = (const uint32_t*)row + 8 * c + h;
#pragma unroll
      for (int e = 0; e < 4; ++e) q[c][e] = r[2 * e];
    } else if (32 * c + 16 * h < A.queries.row_b) {
      q[c] = *(const u32x4_t*)(row + 32 * c + 16 * h);
    }
  }
}

// Statistics of a query over some items; join() adds those of others.
struct Stats {
  float m = kMasked, z = 0.0f, x = 0.0f;
  __device__ __forceinline__ void join(float m2, float z2, float x2) {
    const float mn = m2 > m ? m2 : m;
    const float g0 = __builtin_amdgcn_exp2f(m - mn), g1 = __builtin_amdgcn_exp2f(m2 - mn);
    // an empty side has no sums (or only NaN); its reference is no number to multiply with
    x = (m > kEmpty ? g0 * (x + (m - mn) * z) : 0.0f) + (m2 > kEmpty ? g1 * (x2 + (m2 - mn) * z2) : 0.0f);
    z = (m > kEmpty ? g0 * z : z) + (m2 > kEmpty ? g1 * z2 : z2);
    m = mn;
  }
  __device__ __forceinline__ void join_lanes(int n) {  // over the first n (rounded up to 2^i) lanes
    for (int o = 1; o < n; o <<= 1) {
      const float m2 = __shfl_xor(m, o, kWave), z2 = __shfl_xor(z, o, kWave), x2 = __shfl_xor(x, o, kWave);
      join(m2, z2, x2);
    }
  }
  __device__ __forceinline__ bool empty() const { return m <= kEmpty && z == 0.0f; }
  __device__ __forceinline__ float lse() const { return empty() ? -INFINITY : m * kLn2 + logf(z); }
  __device__ __forceinline__ float entropy() const {
    const float h = kLn2 * (log2f(z) - x / z);
    return empty() ? 0.0f : (h < 0.0f ? 0.0f : h);
  }
};

__device__ __forceinline__ void read_ids(const FinishArgs& A, int64_t at, bool& pad, int64_t& row) {
  const int64_t id = A.id_bits == 32 ? (int64_t)((const int32_t*)A.ids)[at] : ((const int64_t*)A.ids)[at];
  pad = id < 0 || id >= A.items.n;
  row = pad ? 0 : id;
}

// Without alternatives: one workgroup per 32 queries. Eight threads a query join the slices'
// statistics; then each wave scores 32 (query, id) pairs at a time, pair i's item as row i and
// its query as column i of one matrix product, whose diagonal holds the scores. Bound by latency:
// 4.7 us for 4096 queries of one id each.
template <int CT, bool ROWS, int NCH>
__global__ __launch_bounds__(256) void pairs_kernel(FinishArgs A) {
  __shared__ float s_lse[kFrag];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int b0 = blockIdx.x * kFrag, nb = min(kFrag, A.b - b0);
  {
    const int q = t >> 3, sub = t & 7;
    Stats S;
    if (q < nb)
#pragma unroll 4
      for (int s = sub; s < A.nslices; s += 8) {
        const float4 p = A.part[(int64_t)s * A.b + b0 + q];
        S.join(p.x, p.y, p.z);
      }
    S.join_lanes(8);
    if (sub == 0 && q < nb) {
      const float lse = S.lse();
      A.lse[b0 + q] = lse;
      s_lse[q] = lse;
      if (A.entropy) A.entropy[b0 + q] = S.entropy();
    }
  }
  __syncthreads();
  for (int p0 = wave * kFrag; p0 < nb * A.g; p0 += 4 * kFrag) {
    const int p = min(p0 + (lane & 31), nb * A.g - 1);  // this lane's pair
    const int64_t at = (int64_t)b0 * A.g + p;
    bool pad;
    int64_t row;
    read_ids(A, at, pad, row);
    const int bl = p / A.g;
    u32x4_t a[NCH], q[NCH];
    load_chunks<ROWS, NCH>(A.items, row, a);
    query_chunks<NCH>(A, b0 + bl, q);
    const float s = score_rows<CT, NCH>(a, q);
    if (diagonal() && p0 + (lane & 31) < nb * A.g)
      A.logprobs[at] = pad ? 0.0f
                           : (excluded(A, b0 + bl, row) ? -INFINITY
                                                        : log_prob(logit(A, s, A.bias ? A.bias[row] : 0.0f), s_lse[bl]));
  }
}

// With alternatives: one workgroup per query joins the slices' statistics, scores the given ids
// and picks the alternatives. Bound by latency, a chain of dependent reads and picks with one
// workgroup a query: 19 us at 16 x 1M x 128 with 20 alternatives, 46 us at 50 x 10M x 128, where 26
// of them score the 80 blocks of 32 rows again (a 1024-thread workgroup and more blocks in flight
// were not faster), 7.4 us over 400 items.
constexpr int kFinThreads = 512;
constexpr int kFinWaves = kFinThreads / kWave;
constexpr int kIdsKept = 128;  // given ids that are read ahead
constexpr int kKept = 4;       // keys that a thread keeps in registers
constexpr int kPickCap = 256;  // candidates of a pick that are ranked by counting

template <int CT, bool ROWS, int NCH>
__global__ __launch_bounds__(kFinThreads) void finish_kernel(FinishArgs A) {
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];  // keys of the rescored rows
  __shared__ float4 red[kFinWaves];
  __shared__ uint64_t found[kPickCap];
  __shared__ __attribute__((aligned(16))) uint32_t maxima[kFinThreads];
  __shared__ uint64_t best[MIPS_ALTERNATIVES_MAX];
  __shared__ int64_t list[MIPS_ALTERNATIVES_MAX];
  __shared__ int32_t s_ids[kIdsKept];
  __shared__ uint32_t cnt;
  const int b = blockIdx.x, t = threadIdx.x, lane = t & 63, wave = t >> 6;

  // everything that the first steps read is asked for at once
  auto run_key = [&](float v, int64_t i) __attribute__((always_inline)) {
    return v == -INFINITY ? 0ull : composite(score_key(v), (uint32_t)i);
  };
  const int64_t f = b / kFrag;
  const int col = b % kFrag;
  const float* bm = A.bmax + f * A.nruns * kFrag + col;
  const float* top = A.gmax ? A.gmax + f * A.ngroups * kFrag + col : bm;  // the first pick's values
  const int64_t ntop = A.gmax ? A.ngroups : A.nruns;
  auto top_key = [&](int64_t i) __attribute__((always_inline)) { return run_key(top[i * kFrag], i); };
  // The min(k, candidates) best of n distinct keys, sorted, in best[]; keys of 0 are no
  // candidates. Returns their number. Each thread takes the largest of its keys; the k-th
  // largest score among those of 64 groups of threads (k > 32: 256 pairs) is a bound that k keys
  // reach, and few others do when the best keys are spread over the threads. Every wave finds it
  // by itself, bit by bit, from all of them. The keys that reach it are ranked by counting the larger
  // ones. Where more than kPickCap reach it, the bound is found among all keys, bit by bit over
  // their 64 bits.
  // A thread's first kKept keys stay in registers, loaded by keep().
  auto keep = [&](auto get, int64_t n, uint64_t (&kept)[kKept]) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < kKept; ++u) {
      const int64_t i = t + u * kFinThreads;
      kept[u] = i < n ? get(i) : 0ull;
    }
  };
  auto pick = [&](auto get, int64_t n, const uint64_t (&kept)[kKept]) __attribute__((always_inline)) {
    uint64_t mine = 0ull;
#pragma unroll
    for (int u = 0; u < kKept; ++u) mine = kept[u] > mine ? kept[u] : mine;
#pragma unroll 4
    for (int64_t i = t + kKept * kFinThreads; i < n; i += kFinThreads) {
      const uint64_t key = get(i);
      mine = key > mine ? key : mine;
    }
    maxima[t] = (uint32_t)(mine >> 32);
    if (t == 0) cnt = 0u;
    __syncthreads();
    uint4 m4 = *(const uint4*)(maxima + 4 * lane);
    {
      const uint4 o = *(const uint4*)(maxima + 256 + 4 * lane);
      m4 = make_uint4(max(m4.x, o.x), max(m4.y, o.y), max(m4.z, o.z), max(m4.w, o.w));
    }
    uint32_t bound = 0u;
    if (A.k <= 32) {  // 64 groups of threads bound few more candidates than 256, and are quicker
      const uint32_t m1 = max(max(m4.x, m4.y), max(m4.z, m4.w));
#pragma unroll
      for (int bit = 31; bit >= 0; --bit) {
        const uint32_t c = bound | (1u << bit);
        bound = __popcll(__ballot(m1 >= c)) >= A.k ? c : bound;
      }
    } else {
#pragma unroll 1
      for (int bit = 31; bit >= 0; --bit) {
        const uint32_t c = bound | (1u << bit);
        const int above = __popcll(__ballot(m4.x >= c)) + __popcll(__ballot(m4.y >= c)) +
                          __popcll(__ballot(m4.z >= c)) + __popcll(__ballot(m4.w >= c));
        bound = above >= A.k ? c : bound;
      }
    }
    uint64_t least = bound == 0u ? 1ull : (uint64_t)bound << 32;
    auto collect = [&]() __attribute__((always_inline)) {
      auto take = [&](uint64_t key) __attribute__((always_inline)) {
        if (key >= least) {
          const uint32_t slot = atomicAdd(&cnt, 1u);
          if (slot < (uint32_t)kPickCap) found[slot] = key;
        }
      };
#pragma unroll
      for (int u = 0; u < kKept; ++u) take(kept[u]);
#pragma unroll 4
      for (int64_t i = t + kKept * kFinThreads; i < n; i += kFinThreads) take(get(i));
      __syncthreads();
    };
    collect();
    if (cnt > (uint32_t)kPickCap) {
      uint64_t bound64 = 0ull;
      for (int bit = 63; bit >= 0; --bit) {
        const uint64_t c = bound64 | (1ull << bit);
        uint32_t above = 0u;
        for (int64_t i = t; i < n; i += kFinThreads) above += get(i) >= c ? 1u : 0u;
        __syncthreads();
        if (t == 0) cnt = 0u;
        __syncthreads();
        atomicAdd(&cnt, above);
        __syncthreads();
        bound64 = cnt >= (uint32_t)A.k ? c : bound64;
      }
      least = bound64;  // (more than kPickCap >= k candidates: it is one of them)
      __syncthreads();
      if (t == 0) cnt = 0u;
      __syncthreads();
      collect();
    }
    const int c = (int)cnt;
    const int r = min(c, A.k);
    if (c <= kWave) {
      if (wave == 0) {
        const uint64_t key = lane < c ? found[lane] : 0ull;
        int rank = 0;
        for (int j = 0; j < c; ++j) {
          const uint64_t other = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(key >> 32), j) << 32) |
                                 (uint32_t)__builtin_amdgcn_readlane((int)key, j);
          rank += other > key ? 1 : 0;
        }
        if (lane < c && rank < r) best[rank] = key;
      }
    } else if (t < c) {
      const uint64_t key = found[t];
      int rank = 0;
#pragma unroll 8
      for (int j = 0; j < c; ++j) rank += found[j] > key ? 1 : 0;
      if (rank < r) best[rank] = key;
    }
    __syncthreads();
    return r;
  };
  uint64_t kept[kKept];
  keep(top_key, ntop, kept);
  const int ng = (A.g + kFrag - 1) / kFrag;  // blocks of given ids
  for (int i = t; i < min(A.g, kIdsKept); i += kFinThreads) {
    bool pad;
    int64_t row;
    read_ids(A, (int64_t)b * A.g + i, pad, row);
    s_ids[i] = pad ? -1 : (int32_t)row;
  }
  u32x4_t q[NCH];  // the query in every column
  query_chunks<NCH>(A, b, q);
  Stats st;
  for (int s = t; s < A.nslices; s += kFinThreads) {
    const float4 p = A.part[(int64_t)s * A.b + b];
    st.join(p.x, p.y, p.z);
  }
  st.join_lanes(min(kWave, A.nslices));
  if (lane == 0) red[wave] = make_float4(st.m, st.z, st.x, 0.0f);
  __syncthreads();
  st.m = red[0].x, st.z = red[0].y, st.x = red[0].z;
  for (int w = 1; w < min(kFinWaves, (A.nslices + kWave - 1) / kWave); ++w) st.join(red[w].x, red[w].y, red[w].z);
  const float lse = st.lse();
  if (t == 0) {
    A.lse[b] = lse;
    if (A.entropy) A.entropy[b] = st.entropy();
  }

  int r = pick(top_key, ntop, kept);
  if (A.gmax) {
    if (t < r) list[t] = (int64_t)composite_id(best[t]) << A.per_log;
    __syncthreads();
    auto key = [&](int64_t i) __attribute__((always_inline)) {
      const int64_t u = list[i >> A.per_log] + (i & ((1 << A.per_log) - 1));
      return u < A.nruns ? run_key(bm[u * kFrag], u) : 0ull;
    };
    const int64_t n = (int64_t)r << A.per_log;
    keep(key, n, kept);
    r = pick(key, n, kept);
  }
  if (t < r) list[t] = (int64_t)composite_id(best[t]) << A.rm_log;  // first 32-row block of the run
  __syncthreads();
  // The rows of the runs and the given ids, 32 a wave at a time; each wave's next block is on
  // its way while this one is scored.
  uint64_t* keys = (uint64_t*)dyn;
  const int nb = r << A.rm_log;
  auto row_of = [&](int i) __attribute__((always_inline)) -> int64_t {  // -1: padding
    if (i < nb) return (list[i >> A.rm_log] + (i & ((1 << A.rm_log) - 1))) * kFrag + (lane & 31);
    const int g = (i - nb) * kFrag + (lane & 31);
    if (g >= A.g) return -1;
    if (g < kIdsKept) return s_ids[g];
    bool pad;
    int64_t row;
    read_ids(A, (int64_t)b * A.g + g, pad, row);
    return pad ? -1 : row;
  };
  struct Block {
    u32x4_t chunks[NCH];
    int64_t row;
    uint32_t word;
    float bias;
  };
  auto fetch = [&](int i, Block& x) __attribute__((always_inline)) {
    if (i >= nb + ng) return;
    x.row = row_of(i);
    const int64_t at = max<int64_t>(0, min<int64_t>(x.row, A.items.n - 1));
    load_chunks<ROWS, NCH>(A.items, at, x.chunks);
    x.word = A.exclude ? A.exclude[(int64_t)b * A.exclude_words + (at >> 5)] : 0u;
    x.bias = A.bias ? A.bias[at] : 0.0f;
  };
  auto score = [&](int i, Block& x) __attribute__((always_inline)) {
    if (i >= nb + ng) return;
    const bool live = x.row >= 0 && x.row < A.items.n;
    const bool out = live && ((x.word >> (x.row & 31)) & 1u);
    const float l = logit(A, score_rows<CT, NCH>(x.chunks, q), x.bias);
    if (!diagonal()) return;
    if (i < nb) {
      keys[i * kFrag + (lane & 31)] = live && !out && l > kLeastLogit ? composite(score_key(l), (uint32_t)x.row) : 0ull;
    } else {
      const int g = (i - nb) * kFrag + (lane & 31);
      if (g < A.g) A.logprobs[(int64_t)b * A.g + g] = !live ? 0.0f : (out ? -INFINITY : log_prob(l, lse));
    }
  };
  Block x0, x1;
  fetch(wave, x0);
#pragma unroll 1
  for (int i = wave; i < nb + ng; i += 2 * kFinWaves) {
    fetch(i + kFinWaves, x1);
    score(i, x0);
    fetch(i + 2 * kFinWaves, x0);
    score(i + kFinWaves, x1);
  }
  __syncthreads();
  auto row_key = [&](int64_t i) __attribute__((always_inline)) { return keys[i]; };
  keep(row_key, (int64_t)nb * kFrag, kept);
  r = pick(row_key, (int64_t)nb * kFrag, kept);
  for (int i = t; i < A.k; i += kFinThreads) {
    const int64_t at = (int64_t)b * A.k + i;
    A.alt_ids[at] = i < r ? (int32_t)composite_id(best[i]) : -1;
    A.alt_logprobs[at] = i < r ? key_score((uint32_t)(best[i] >> 32)) - lse : -INFINITY;
  }
}

// ------------------------------------------------------------------------- the host side
static int width_of(int dtype, int row_b) {  // the kernels' width for rows of row_b bytes
  const int d = row_b / elem_bytes(dtype);
  for (int w = 16; w <= (dtype == MIPS_F32 ? 128 : 256); w *= 2)
    if (d <= w) return w;
  return 0;
}

struct StatsPlan {
  int width, nqf, nqblk, nslices, qbatch;
  int64_t ntiles, nruns, ngroups;
  int per, run_log;
  size_t part, bmax, gmax, bytes;
};

// Query fragments a workgroup holds and slices of the items: the pair with the least estimated
// time, rounds of workgroups (one a compute unit) times the time of one: its query tile, then
// the tiles of a wave, each against every fragment, at no less than the time its bytes take at
// the memory's rate. In microseconds, as measured at the widths 64 to 128: a fragment's fill
// 0.3, a tile and fragment 0.45 (f32: twice the products' time), start and end 4. A training
// call with 1, 2, 4 or 8 fragments fixed: 1000 x 1000 x 64 f32 52.7, 54.7, 60.5, 69.6 us (1 is
// chosen); 4096 x 8192 x 128 bf16 124.7, 112.3, 108.0, 106.7 (8); 4096 x 250,000 x 128 bf16
// 1527 (2), 1440 (4), 1395 (8).
static StatsPlan stats_plan(int b, int64_t n, int d, int dtype, int k) {
  StatsPlan P{};
  P.width = width_of(dtype, d * elem_bytes(dtype));
  const int rm = stats_rm(dtype, P.width);
  P.ntiles = (n + kFrag * rm - 1) / (kFrag * rm);
  const int cus = device_cu_count();
  P.ngroups = 0;
  P.per = 0;
  P.run_log = 0;
  P.qbatch = b;
  if (k > 0) {
    // Runs of up to 4 tiles, as long as a wave has 16 runs and the k runs' keys fit 32 KiB: at
    // 50 x 10M x 128 with 20 alternatives a call takes 578 us with runs of one tile, 550 of two,
    // 523 of four and 524 of eight.
    while (P.run_log < 2 && (P.ntiles >> (P.run_log + 1)) >= (int64_t)cus * kStatsWaves * 16 &&
           ((int64_t)k * rm << (P.run_log + 1)) * kFrag * 8 <= kKeyBytes)
      ++P.run_log;
  }
  P.nruns = (P.ntiles + (1 << P.run_log) - 1) >> P.run_log;
  if (k > 0) {
    // queries of one batch: their run maxima stay within kBmaxBytes
    const int64_t q = (int64_t)(kBmaxBytes / (size_t)(P.nruns * 4)) / kFrag * kFrag;
    if (q < b) P.qbatch = (int)(q < kFrag ? kFrag : q);
    if (P.nruns > kTopDirect) {
      // groups of about sqrt(runs / k): as many group maxima to read as runs of k groups
      P.per = 32;
      while ((int64_t)P.per * P.per * k < P.nruns || (P.nruns + P.per - 1) / P.per > kTopGroups) P.per *= 2;
      P.ngroups = (P.nruns + P.per - 1) / P.per;
    }
  }
  const double tile_us = dtype == MIPS_F32 ? 0.45 * rm * (0.5 + P.width / 32.0) : 0.45 * rm * (0.5 + P.width / 256.0);
  const double tile_bytes = (double)rm * block_bytes(dtype, P.width);
  double best = 1e30;
  for (int nqf = 1; nqf <= 8; nqf *= 2) {
    if (!stats_fits(dtype, P.width, nqf)) break;
    const int nqblk = (P.qbatch + kFrag * nqf - 1) / (kFrag * nqf);
    const int frags = nqblk == 1 ? (P.qbatch + kFrag - 1) / kFrag : nqf;
    // slices of at least one run a wave; a multiple of 8 (XCDs) where there are that many
    int64_t s = cus / nqblk;
    const int64_t most = (P.nruns + kStatsWaves - 1) / kStatsWaves;
    if (s > most) s = most;
    if (s >= 8) s = s / 8 * 8;
    if (s < 1) s = 1;
    const int64_t per = (P.ntiles + s * kStatsWaves - 1) / (s * kStatsWaves);
    const int64_t rounds = (nqblk * s + cus - 1) / cus;
    const double mem = (double)kStatsWaves * tile_bytes / (5.0e6 / cus);  // us: a round of tiles of one unit
    const double t = (double)rounds * (4.0 + 0.3 * frags + (double)per * (frags * tile_us > mem ? frags * tile_us : mem));
    if (t < best) {
      best = t;
      P.nqf = nqf;
      P.nqblk = nqblk;
      P.nslices = (int)s;
    }
    if (nqblk == 1) break;
  }
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t p = at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  const size_t q32 = (size_t)((P.qbatch + kFrag - 1) / kFrag) * kFrag;
  P.part = take((size_t)P.nslices * P.qbatch * sizeof(float4));
  if (k > 0) {
    P.bmax = take(q32 * P.nruns * 4);
    if (P.ngroups) P.gmax = take(q32 * P.ngroups * 4);
  }
  P.bytes = at;
  return P;
}

static int stats_dispatch(int dtype, int width, int nqf, bool rows, const StatsArgs& A, int grid, hipStream_t s) {
  if (dtype == MIPS_F32) {
    switch (width) {
      case 16: return launch_stats<MIPS_F32, 16>(nqf, rows, A, grid, s);
      case 32: return launch_stats<MIPS_F32, 32>(nqf, rows, A, grid, s);
      case 64: return launch_stats<MIPS_F32, 64>(nqf, rows, A, grid, s);
      case 128: return launch_stats<MIPS_F32, 128>(nqf, rows, A, grid, s);
    }
  } else {
    switch (width) {
      case 16: return launch_stats<MIPS_BF16, 16>(nqf, rows, A, grid, s);
      case 32: return launch_stats<MIPS_BF16, 32>(nqf, rows, A, grid, s);
      case 64: return launch_stats<MIPS_BF16, 64>(nqf, rows, A, grid, s);
      case 128: return launch_stats<MIPS_BF16, 128>(nqf, rows, A, grid, s);
      case 256: return launch_stats<MIPS_BF16, 256>(nqf, rows, A, grid, s);
    }
  }
  return MIPS_ERR_UNSUPPORTED;
}

template <int CT, bool ROWS, int NCH>
static int launch_finish_one(const FinishArgs& A, int b, hipStream_t s) {
  if (A.k == 0)
    hipLaunchKernelGGL((pairs_kernel<CT, ROWS, NCH>), dim3((b + kFrag - 1) / kFrag), dim3(256), 0, s, A);
  else
    hipLaunchKernelGGL((finish_kernel<CT, ROWS, NCH>), dim3(b), dim3(kFinThreads),
                       ((size_t)A.k << A.rm_log) * kFrag * 8, s, A);
  return check_launch();
}

template <int CT, bool ROWS>
static int launch_finish(const FinishArgs& A, int width, int b, hipStream_t s) {
  switch (chunks_per_block(CT, width)) {
    case 1: if constexpr (CT == MIPS_BF16) return launch_finish_one<CT, ROWS, 1>(A, b, s); break;
    case 2: return launch_finish_one<CT, ROWS, 2>(A, b, s);
    case 4: return launch_finish_one<CT, ROWS, 4>(A, b, s);
    case 8: return launch_finish_one<CT, ROWS, 8>(A, b, s);
    case 16: return launch_finish_one<CT, ROWS, 16>(A, b, s);
  }
  return MIPS_ERR_UNSUPPORTED;
}

// Sizes that both entry points share; MIPS_OK or a status.
static int check_sizes(int b, int64_t n, int d, int dtype, int layout) {
  if (b < 1 || n < 1 || d < 1) return MIPS_ERR_INVALID_ARG;
  if (dtype != MIPS_F32 && dtype != MIPS_BF16) return MIPS_ERR_UNSUPPORTED;
  if (layout != MIPS_ROWS && layout != MIPS_PACKED) return MIPS_ERR_INVALID_ARG;
  if (n > (int64_t(1) << 31) - 64 || b > MIPS_B_MAX) return MIPS_ERR_UNSUPPORTED;
  const int row_b = d * elem_bytes(dtype);
  if (width_of(dtype, row_b) == 0 || row_b % 16 != 0) return MIPS_ERR_UNSUPPORTED;
  if (layout == MIPS_PACKED && !corpus_d_supported(dtype, d)) return MIPS_ERR_UNSUPPORTED;
  return MIPS_OK;
}

// A row-major operand: 16-byte aligned rows at most 2^25 bytes apart.
static bool rows_ok(const void* p, int64_t stride, int d, int dtype) {
  const int64_t sb = stride * elem_bytes(dtype);
  return aligned(p, 16) && stride >= d && sb % 16 == 0 && sb <= (int64_t(1) << 25);
}

}  // namespace mips

extern "C" {

size_t mips_logprobs_workspace_size(int32_t b, int64_t n, int32_t d, int32_t dtype, int32_t k) {
  using namespace mips;
  if (k < 0 || k > MIPS_ALTERNATIVES_MAX || check_sizes(b, n, d, dtype, MIPS_ROWS) != MIPS_OK) return 0;
  return stats_plan(b, n, d, dtype, k).bytes;
}

int mips_logprobs(const void* queries, int64_t query_stride, int32_t b, const void* items,
                  int32_t layout, int64_t item_stride, int64_t n, int32_t d, int32_t dtype,
                  const float* bias, const uint32_t* exclude, int64_t exclude_row_words,
                  float scale, const void* ids, int32_t id_bits, int32_t g, int32_t k,
                  float* out_logprobs, float* out_lse, float* out_entropy, int32_t* out_alt_ids,
                  float* out_alt_logprobs, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace mips;
  if (const int rc = check_sizes(b, n, d, dtype, layout)) return rc;
  if (g < 0 || k < 0 || !(scale >= MIPS_SCALE_MIN && scale <= MIPS_SCALE_MAX)) return MIPS_ERR_INVALID_ARG;
  if (k > MIPS_ALTERNATIVES_MAX || (g > 0 && id_bits != 32 && id_bits != 64)) return MIPS_ERR_UNSUPPORTED;
  const int64_t words = (n + 31) / 32;
  if (!queries || !items || !out_lse || !workspace || (g > 0 && (!ids || !out_logprobs)) ||
      (k > 0 && (!out_alt_ids || !out_alt_logprobs)))
    return MIPS_ERR_INVALID_ARG;
  if (!rows_ok(queries, query_stride, d, dtype) || !aligned(items, 16) ||
      (layout == MIPS_ROWS && !rows_ok(items, item_stride, d, dtype)))
    return MIPS_ERR_INVALID_ARG;
  if (exclude_row_words < 0 || (exclude_row_words > 0 && (!exclude || exclude_row_words < words)))
    return MIPS_ERR_INVALID_ARG;
  if (!aligned(workspace, 256) || (bias && !aligned(bias, 4)) || (exclude && !aligned(exclude, 4)) ||
      !aligned(out_lse, 4) || (out_entropy && !aligned(out_entropy, 4)) ||
      (g > 0 && (!aligned(ids, id_bits / 8) || !aligned(out_logprobs, 4))) ||
      (k > 0 && (!aligned(out_alt_ids, 4) || !aligned(out_alt_logprobs, 4))))
    return MIPS_ERR_INVALID_ARG;
  const StatsPlan P = stats_plan(b, n, d, dtype, k);
  if (workspace_bytes < P.bytes) return MIPS_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  uint8_t* ws = (uint8_t*)workspace;
  const int E = elem_bytes(dtype), row_b = d * E;
  const bool rows = layout == MIPS_ROWS;
  for (int q0 = 0; q0 < b; q0 += P.qbatch) {
    const int nb = b - q0 < P.qbatch ? b - q0 : P.qbatch;
    StatsArgs A{};
    A.items = Table{(const uint8_t*)items, rows ? item_stride * E : 0, n, row_b};
    A.queries = Table{(const uint8_t*)queries + q0 * query_stride * E, query_stride * E, nb, row_b};
    A.b = nb;
    A.bias = bias;
    A.exclude = exclude ? exclude + q0 * exclude_row_words : nullptr;
    A.exclude_words = exclude_row_words;
    A.scale = scale;
    A.scx = bias ? kLog2e : scale * kLog2e;
    A.vmask = kMasked / A.scx;
    A.nqblk = (nb + kFrag * P.nqf - 1) / (kFrag * P.nqf);
    A.ent = out_entropy != nullptr;
    A.nslices = P.nslices;
    A.nruns = P.nruns;
    A.run_log = P.run_log;
    A.part = (float4*)(ws + P.part);
    A.bmax = k > 0 ? (float*)(ws + P.bmax) : nullptr;
    if (const int rc = stats_dispatch(dtype, P.width, P.nqf, rows, A, A.nqblk * P.nslices, s)) return rc;
    if (P.ngroups) {
      const int64_t gblocks = (P.ngroups + 7) / 8;
      const int64_t nf = (nb + kFrag - 1) / kFrag;
      hipLaunchKernelGGL(group_max_kernel, dim3((unsigned)(gblocks * nf)), dim3(kGroupThreads), 0, s, A.bmax, P.nruns,
                         P.per, P.ngroups, gblocks, (float*)(ws + P.gmax));
      if (const int rc = check_launch()) return rc;
    }
    FinishArgs F{};
    F.items = A.items;
    F.queries = A.queries;
    F.packed_f32 = !rows && dtype == MIPS_F32;
    F.b = nb;
    F.bias = bias;
    F.exclude = A.exclude;
    F.exclude_words = exclude_row_words;
    F.scale = scale;
    F.nslices = P.nslices;
    F.part = A.part;
    F.ids = g > 0 ? (const uint8_t*)ids + (int64_t)q0 * g * (id_bits / 8) : nullptr;
    F.id_bits = id_bits;
    F.g = g;
    F.k = k;
    F.bmax = A.bmax;
    F.gmax = P.ngroups ? (float*)(ws + P.gmax) : nullptr;
    F.nruns = P.nruns;
    F.ngroups = P.ngroups;
    while (1 << F.per_log < P.per) ++F.per_log;
    F.rm_log = (stats_rm(dtype, P.width) == 2 ? 1 : 0) + P.run_log;
    F.logprobs = g > 0 ? out_logprobs + (int64_t)q0 * g : nullptr;
    F.lse = out_lse + q0;
    F.entropy = out_entropy ? out_entropy + q0 : nullptr;
    F.alt_ids = k > 0 ? out_alt_ids + (int64_t)q0 * k : nullptr;
    F.alt_logprobs = k > 0 ? out_alt_logprobs + (int64_t)q0 * k : nullptr;
    int rc;
    if (dtype == MIPS_F32) rc = rows ? launch_finish<MIPS_F32, true>(F, P.width, nb, s) : launch_finish<MIPS_F32, false>(F, P.width, nb, s);
    else rc = rows ? launch_finish<MIPS_BF16, true>(F, P.width, nb, s) : launch_finish<MIPS_BF16, false>(F, P.width, nb, s);
    if (rc) return rc;
  }
  return MIPS_OK;
}

}  // extern "C"
