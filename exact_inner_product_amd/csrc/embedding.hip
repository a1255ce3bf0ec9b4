// embedding.hip -- embedding lookup with scaling and its gradient by sorted tokens (gfx950).
//
// Lookup:   out[t] = scale * table[id_t], a zero row where id_t is outside [0, rows).
// Gradient: out[v] = scale * sum over the tokens t with id_t = v of grad[t].
//
// Both move rows and compute next to nothing, so both are bound by memory traffic (and, for
// few tokens, by launches). The gradient's sum is a segmented sum over the tokens sorted by
// id: no atomics on floats, so that the same call gives the same bits, and a hot id's
// thousands of tokens are split over many groups of lanes.
#include <type_traits>

#include "common.h"
#include "host.h"

namespace mips {

// ------------------------------------------------------------- 16-byte vectors of rows
// A unit is up to 16 bytes of one row: 4 floats, 8 bf16, or (rows that are not 16-byte
// multiples or not aligned) a single element.
template <int DT, bool VEC>
struct Unit {
  static constexpr int N = VEC ? (DT == MIPS_F32 ? 4 : 8) : 1;
  template <bool NT = false>  // NT: past the caches, for what is not used again soon
  static __device__ __forceinline__ void load(const void* p, int64_t i, float (&v)[N]) {
    if constexpr (DT == MIPS_F32) {
      if constexpr (VEC) {
        const u32x4_t* q = (const u32x4_t*)((const float*)p + i);
        const u32x4_t x = NT ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(x[j]);
      } else {
        v[0] = ((const float*)p)[i];
      }
    } else {
      if constexpr (VEC) {
        const u32x4_t* q = (const u32x4_t*)((const uint16_t*)p + i);
        const u32x4_t x = NT ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[2 * j] = __uint_as_float(x[j] << 16);
          v[2 * j + 1] = __uint_as_float(x[j] & 0xFFFF0000u);
        }
      } else {
        v[0] = bf16_to_f32(((const uint16_t*)p)[i]);
      }
    }
  }
  template <bool NT = false>
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&v)[N]) {
    if constexpr (DT == MIPS_F32) {
      typedef float f32x4_t __attribute__((ext_vector_type(4)));
      if constexpr (VEC && NT)
        __builtin_nontemporal_store(f32x4_t{v[0], v[1], v[2], v[3]}, (f32x4_t*)((float*)p + i));
      else if constexpr (VEC)
        *(float4*)((float*)p + i) = make_float4(v[0], v[1], v[2], v[3]);
      else
        ((float*)p)[i] = v[0];
    } else {
      // the one rounding to bf16, to nearest even (the compiler's conversion keeps NaN)
      if constexpr (VEC) {
        bf16x8_t o;
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = (__bf16)v[j];
        if constexpr (NT) __builtin_nontemporal_store(o, (bf16x8_t*)((uint16_t*)p + i));
        else *(bf16x8_t*)((uint16_t*)p + i) = o;
      } else {
        ((__bf16*)p)[i] = (__bf16)v[0];
      }
    }
  }
};

template <typename IdT>
__device__ __forceinline__ int64_t id_at(const void* ids, int64_t t) {
  return (int64_t)((const IdT*)ids)[t];
}

// ------------------------------------------------------------------------------ lookup
constexpr int kLookupRows = 4;  // rows in flight per group of lanes

struct LookupArgs {
  const void* table;
  int64_t rows, row_stride;
  const void* ids;
  int64_t t;
  float scale;
  void* out;
  int d, nunit, tpr_log;  // units per row; log2 of the lanes that share a row
};

// 2^tpr_log lanes share a row and take its units in turn; each group moves kLookupRows
// rows, all of their loads issued before the first store, which keeps several row fetches in
// flight per lane (random rows of a large table miss every cache). Rows are stored past the
// caches, which leaves those to the table's hot rows: 520,192 Zipf rows of 128 bf16 (133 MB
// written) 30 us, 48 with ordinary stores; by 50 rows it is the launch, 2.4 us.
template <int DT, bool VEC, typename IdT>
__global__ __launch_bounds__(256) void lookup_kernel(LookupArgs A) {
  using U = Unit<DT, VEC>;
  const int tpr = 1 << A.tpr_log;
  const int sub = threadIdx.x & (tpr - 1);
  const int groups = 256 >> A.tpr_log;
  const int64_t t0 = (int64_t)blockIdx.x * groups * kLookupRows + (threadIdx.x >> A.tpr_log);
  int64_t row[kLookupRows];
#pragma unroll
  for (int u = 0; u < kLookupRows; ++u) {
    const int64_t t = t0 + u * groups;
    row[u] = t < A.t ? id_at<IdT>(A.ids, t) : -1;
    if (row[u] < 0 || row[u] >= A.rows) row[u] = -1;
  }
  for (int j = sub; j < A.nunit; j += tpr) {
    float v[kLookupRows][U::N];
#pragma unroll
    for (int u = 0; u < kLookupRows; ++u) {
#pragma unroll
      for (int e = 0; e < U::N; ++e) v[u][e] = 0.0f;
      if (row[u] >= 0) U::load(A.table, row[u] * A.row_stride + (int64_t)j * U::N, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kLookupRows; ++u) {
      const int64_t t = t0 + u * groups;
      if (t >= A.t) continue;
      if (row[u] >= 0) {
#pragma unroll
        for (int e = 0; e < U::N; ++e) v[u][e] *= A.scale;
      }
      U::template store<true>(A.out, t * A.d + (int64_t)j * U::N, v[u]);
    }
  }
}

static int log2_lanes(int nunit) {  // lanes that share a row: the least power of two >= nunit, at most 64
  int l = 0;
  while ((1 << l) < nunit && l < 6) ++l;
  return l;
}

template <int DT, bool VEC>
static int launch_lookup(LookupArgs A, int id_bits, hipStream_t s) {
  A.nunit = A.d / Unit<DT, VEC>::N;
  A.tpr_log = log2_lanes(A.nunit);
  const int64_t per = (256 >> A.tpr_log) * kLookupRows;
  const int E = elem_bytes(DT), I = id_bits / 8;
  const int64_t total = A.t;
  for (int64_t t0 = 0; t0 < total; t0 += per * kMaxGridBlocks) {
    LookupArgs P = A;
    P.t = total - t0 < per * kMaxGridBlocks ? total - t0 : per * kMaxGridBlocks;
    P.ids = (const uint8_t*)A.ids + t0 * I;
    P.out = (uint8_t*)A.out + t0 * A.d * E;
    const dim3 grid((unsigned)((P.t + per - 1) / per));
    if (id_bits == 32)
      hipLaunchKernelGGL((lookup_kernel<DT, VEC, int32_t>), grid, dim3(256), 0, s, P);
    else
      hipLaunchKernelGGL((lookup_kernel<DT, VEC, int64_t>), grid, dim3(256), 0, s, P);
    if (const int rc = check_launch()) return rc;
  }
  return MIPS_OK;
}

// ------------------------------------------------------------------ sorting the tokens
// The (id, token) pairs sorted by id, equal ids in token order: the order of the segmented
// sum, and so its rounding, follows from the ids and sizes alone. Ids outside [0, rows) take the key
// `rows` and sort behind every row.
//
// (Few tokens are not sorted as a whole: see small_kernel.) A least-significant-digit radix sort
// of 8-bit digits over at most kSortBlocks contiguous ranges of tokens, two kernels a digit:
// the ranges' digit counts, then every range adds up all counts for its own offsets and
// scatters. Inside a range each wave has a contiguous part: it counts its digits, and with the
// waves' offsets known ranks 64 keys at a time by ballots, which keeps the sort stable. The
// kernels are bound by latency (520,192 tokens of 1M rows, three digits: 8 us a count, 18.5 us a
// scatter); the output's zeros are written beside all of them, a share each, which hides 256 MB.
constexpr int kSortBlocks = 256;
constexpr int kSortTile = 4096;  // tokens of a range: a multiple of this
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / kWave;

__device__ __forceinline__ uint32_t key_of(int64_t id, int64_t rows) {
  return (id < 0 || id >= rows) ? (uint32_t)rows : (uint32_t)id;
}

// Writes zeros to the dense gradient, rows [first, last): workgroup w of nblocks, of any size,
// clears its share. Run in workgroups of their own beside the sort's.
struct ZeroArgs {
  void* p;
  int64_t first, last, stride_b;  // rows, and bytes between them
  int64_t row_b;                  // bytes of a row
  int nblocks;                    // workgroups that clear (0: accumulate into what is there)
};

__device__ __forceinline__ void zero_rows(const ZeroArgs& Z, int w) {
  const u32x4_t z = {0u, 0u, 0u, 0u};
  uint8_t* base = (uint8_t*)Z.p + Z.first * Z.stride_b;
  const int64_t rows = Z.last - Z.first, nt = blockDim.x;
  if (Z.stride_b == Z.row_b && ((uintptr_t)base & 15) == 0) {
    const int64_t total = rows * Z.row_b, n16 = total / 16;
    u32x4_t* p = (u32x4_t*)base;
    for (int64_t i = (int64_t)w * nt + threadIdx.x; i < n16; i += (int64_t)Z.nblocks * nt) __builtin_nontemporal_store(z, p + i);
    if (w == 0 && threadIdx.x < (total & 15) / 2) ((uint16_t*)base)[n16 * 8 + threadIdx.x] = 0;
  } else {
    for (int64_t r = w; r < rows; r += Z.nblocks) {
      uint16_t* p = (uint16_t*)(base + r * Z.stride_b);
      for (int64_t j = threadIdx.x; j < Z.row_b / 2; j += nt) p[j] = 0;
    }
  }
}

// The part [i / n, (i + 1) / n) of the rows (multiples of 8, so that parts keep an alignment of
// 16 bytes), in workgroups of nt threads: 64 bytes a thread at least, at most 1024 of them.
static ZeroArgs zero_part(const ZeroArgs& Z, int i, int n, int nt) {
  ZeroArgs P = Z;
  P.first = i == 0 ? 0 : Z.last * i / n / 8 * 8;
  P.last = i == n - 1 ? Z.last : Z.last * (i + 1) / n / 8 * 8;
  if (Z.nblocks == 0 || P.last <= P.first) {
    P.nblocks = 0;
    return P;
  }
  const int64_t want = ((P.last - P.first) * Z.row_b + nt * 64 - 1) / (nt * 64);
  P.nblocks = (int)(want < 1024 ? want : 1024);
  return P;
}

struct SortArgs {
  const void* ids;          // first pass: the ids; NULL afterwards
  int64_t t, rows;
  int64_t per;              // tokens per range
  int nb;                   // ranges
  int shift;
  const uint32_t *keys_in, *toks_in;
  uint32_t *keys_out, *toks_out;
  uint32_t* counts;         // [nb][256]
  ZeroArgs Z;
};

// Lanes of the wave whose `bits` low bits of dig agree with this lane's, among those that are on.
__device__ __forceinline__ uint64_t same_digit(uint32_t dig, int bits, bool on) {
  uint64_t same = __ballot(on);
  for (int bit = 0; bit < bits; ++bit) {
    const uint64_t m = __ballot((dig >> bit) & 1u);
    same &= ((dig >> bit) & 1u) ? m : ~m;
  }
  return same;
}

// The place of this lane's key: the wave's next place of its digit (`off`, in LDS, this wave's
// alone) plus its rank among the lanes with the same digit. Moves the wave's places on.
__device__ __forceinline__ uint32_t take_place(uint32_t* off, uint32_t dig, int bits, bool on) {
  const uint64_t same = same_digit(dig, bits, on);
  const uint32_t rank = (uint32_t)__popcll(same & ((1ull << (threadIdx.x & 63)) - 1ull));
  const uint32_t p = on ? off[dig] + rank : 0u;
  // one wave's LDS accesses stay in order; the fences keep the compiler from reordering them
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  if (on && rank == 0u) off[dig] += (uint32_t)__popcll(same);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  return p;
}

template <typename IdT>
__device__ __forceinline__ uint32_t sort_key(const SortArgs& A, int64_t i) {
  return A.ids ? key_of(id_at<IdT>(A.ids, i), A.rows) : A.keys_in[i];
}

template <typename IdT>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs A) {
  if ((int)blockIdx.x >= A.nb) {
    zero_rows(A.Z, (int)blockIdx.x - A.nb);
    return;
  }
  __shared__ uint32_t hist[4][256];  // four copies: fewer lanes meet in one counter
  hist[threadIdx.x >> 8][threadIdx.x & 255] = 0u;
  __syncthreads();
  const int64_t i0 = blockIdx.x * A.per, i1 = min(A.t, i0 + A.per);
#pragma unroll 4
  for (int64_t i = i0 + threadIdx.x; i < i1; i += kSortThreads)
    atomicAdd(&hist[threadIdx.x >> 8][(sort_key<IdT>(A, i) >> A.shift) & 255u], 1u);
  __syncthreads();
  const int t = threadIdx.x;
  if (t < 256) A.counts[blockIdx.x * 256 + t] = hist[0][t] + hist[1][t] + hist[2][t] + hist[3][t];
}

template <typename IdT>
__global__ __launch_bounds__(kSortThreads) void sort_scatter_kernel(SortArgs A) {
  if ((int)blockIdx.x >= A.nb) {
    zero_rows(A.Z, (int)blockIdx.x - A.nb);
    return;
  }
  __shared__ uint32_t off[kSortWaves][256];  // a wave's keys per digit, then its next place of each
  __shared__ uint32_t part[2][4][256];
  __shared__ uint32_t wsum[4];
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int64_t i0 = blockIdx.x * A.per, i1 = min(A.t, i0 + A.per);
  const int64_t w0 = i0 + wave * (A.per / kSortWaves), w1 = min(i1, w0 + A.per / kSortWaves);
#pragma unroll
  for (int w = 0; w < kSortWaves / 4; ++w) off[4 * w + (t >> 8)][t & 255] = 0u;
  // digit t & 255: tokens of the ranges before this one and of all ranges, a quarter of the
  // ranges a thread
  uint32_t before = 0u, all = 0u;
#pragma unroll 16
  for (int b = t >> 8; b < A.nb; b += 4) {
    const uint32_t c = A.counts[b * 256 + (t & 255)];
    all += c;
    before += b < (int)blockIdx.x ? c : 0u;
  }
  part[0][t >> 8][t & 255] = before;
  part[1][t >> 8][t & 255] = all;
  __syncthreads();
#pragma unroll 4
  for (int64_t i = w0 + lane; i < w1; i += kWave) atomicAdd(&off[wave][(sort_key<IdT>(A, i) >> A.shift) & 255u], 1u);
  uint32_t incl = 0u;
  if (t < 256) {  // prefix over the digits
    before = part[0][0][t] + part[0][1][t] + part[0][2][t] + part[0][3][t];
    all = part[1][0][t] + part[1][1][t] + part[1][2][t] + part[1][3][t];
    incl = all;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const uint32_t u = __shfl_up(incl, o, kWave);
      if (lane >= o) incl += u;
    }
    if (lane == kWave - 1) wsum[wave] = incl;
  }
  __syncthreads();
  if (t < 256) {
    uint32_t p = incl - all + before;
    for (int w = 0; w < wave; ++w) p += wsum[w];
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = off[w][t];
      off[w][t] = p;
      p += c;
    }
  }
  __syncthreads();
  for (int64_t s0 = w0; s0 < w1; s0 += kWave) {  // wave-uniform
    const int64_t i = s0 + lane;
    const bool on = i < w1;
    const uint32_t key = on ? sort_key<IdT>(A, i) : 0u;
    const uint32_t tok = !on ? 0u : (A.ids ? (uint32_t)i : A.toks_in[i]);
    const uint32_t dig = (key >> A.shift) & 255u;
    const uint32_t p = take_place(off[wave], dig, 8, on);
    if (on) {
      A.keys_out[p] = key;
      A.toks_out[p] = tok;
    }
  }
}

// --------------------------------------------------------------------- segmented sum
// A group of 2^tpr_log lanes sums `chunk` consecutive sorted tokens. A segment (one id's
// tokens) that lies inside a chunk is written to its row at once. A segment that crosses
// chunks leaves one f32 partial row per chunk: slot 2c for the chunk's first segment where it
// began before the chunk, slot 2c + 1 for its last where it goes on behind it. join_kernel
// adds those rows. Bound by the gradient's bytes in random order: 133 MB in 39 us (read past the
// caches, 133 us a call; 138 through them), the join 14 us.
struct SegArgs {
  const void* grad;
  int64_t grad_stride;
  const uint32_t *keys, *toks;
  int64_t t, rows;
  int d, nunit, tpr_log, chunk;
  float scale;
  int accumulate;
  void* out;
  int64_t out_stride;
  float* part;  // [2 * nchunk][d]
  int64_t nchunk;
};

constexpr int kSegBatch = 4;  // row fetches in flight per lane

template <int DT, int OUT, bool VEC>
__device__ __forceinline__ void write_row(const SegArgs& A, uint32_t key, int64_t j,
                                          float (&a)[Unit<DT, VEC>::N]) {
  constexpr int N = Unit<DT, VEC>::N;
  const int64_t at = (int64_t)key * A.out_stride + j;
#pragma unroll
  for (int e = 0; e < N; ++e) a[e] *= A.scale;
  if constexpr (OUT == DT) {
    if (A.accumulate) {
      float o[N];
      Unit<DT, VEC>::load(A.out, at, o);
#pragma unroll
      for (int e = 0; e < N; ++e) a[e] += o[e];
    }
    Unit<DT, VEC>::store(A.out, at, a);
  } else {  // bf16 gradients into an f32 table: 8 elements, two 16-byte stores
    float* p = (float*)A.out + at;
#pragma unroll
    for (int e = 0; e < N; ++e) p[e] = A.accumulate ? p[e] + a[e] : a[e];
  }
}

template <int DT, int OUT, bool VEC>
__global__ __launch_bounds__(256) void segment_kernel(SegArgs A) {
  using U = Unit<DT, VEC>;
  constexpr int N = U::N;
  const int tpr = 1 << A.tpr_log;
  const int sub = threadIdx.x & (tpr - 1);
  const int64_t c = (int64_t)blockIdx.x * (256 >> A.tpr_log) + (threadIdx.x >> A.tpr_log);
  if (c >= A.nchunk) return;
  const int64_t i0 = c * A.chunk, i1 = min(A.t, i0 + A.chunk);
  const uint32_t none = (uint32_t)A.rows;
  const uint32_t prev = i0 > 0 ? A.keys[i0 - 1] : 0xFFFFFFFFu;  // keys are at most 2^31
  const uint32_t next = i1 < A.t ? A.keys[i1] : 0xFFFFFFFFu;
  for (int u = sub; u < A.nunit; u += tpr) {
    const int64_t j = (int64_t)u * N;
    float a[N] = {};
    uint32_t cur = A.keys[i0];
    bool began = cur != prev;  // the current segment began in this chunk
    auto close = [&](bool ends) __attribute__((always_inline)) {
      if (cur != none) {
        if (began && ends) {
          write_row<DT, OUT, VEC>(A, cur, j, a);
        } else {
          float* p = A.part + (2 * c + (began ? 1 : 0)) * A.d + j;
#pragma unroll
          for (int e = 0; e < N; ++e) p[e] = a[e];
        }
      }
#pragma unroll
      for (int e = 0; e < N; ++e) a[e] = 0.0f;
    };
    for (int64_t i = i0; i < i1; i += kSegBatch) {
      uint32_t k[kSegBatch];
      float v[kSegBatch][N];
#pragma unroll
      for (int b = 0; b < kSegBatch; ++b) {
        const int64_t ib = i + b < i1 ? i + b : i1 - 1;
        k[b] = A.keys[ib];
        U::template load<true>(A.grad, (int64_t)A.toks[ib] * A.grad_stride + j, v[b]);
      }
#pragma unroll
      for (int b = 0; b < kSegBatch; ++b) {
        if (i + b >= i1) break;
        if (k[b] != cur) {
          close(true);
          cur = k[b];
          began = true;
        }
#pragma unroll
        for (int e = 0; e < N; ++e) a[e] += v[b][e];
      }
    }
    // the last segment; one that both entered and leaves the chunk takes the chunk's slot 2c
    if (cur != next) close(true);
    else close(false);
  }
}

// Adds the partial rows of the segments that cross chunks. A group of 2^tpr_log lanes looks at
// one chunk: a segment that began in it and goes on over at most kJoinShort chunks is added up
// by the group, chunk after chunk. Longer ones (hot ids) are left to the whole workgroup, one
// after the other: the groups take chunks in turn, then their sums are joined in LDS, in a fixed
// order.
constexpr int kJoinShort = 16;

template <int DT, int OUT, bool VEC>
__global__ __launch_bounds__(256) void join_kernel(SegArgs A) {
  constexpr int N = Unit<DT, VEC>::N;
  __shared__ float red[256 * N];
  __shared__ int64_t long_c[256], long_end[256];
  __shared__ int nlong;
  const int tpr = 1 << A.tpr_log;
  const int sub = threadIdx.x & (tpr - 1), g = threadIdx.x >> A.tpr_log, ng = 256 >> A.tpr_log;
  if (threadIdx.x == 0) nlong = 0;
  __syncthreads();
  auto add_rows = [&](int64_t c, int64_t from, int64_t to, int step, int64_t j, float (&a)[N]) __attribute__((always_inline)) {
#pragma unroll 4
    for (int64_t q = from; q <= to; q += step) {
      const float* p = A.part + (2 * q + (q == c ? 1 : 0)) * A.d + j;
#pragma unroll
      for (int e = 0; e < N; ++e) a[e] += p[e];
    }
  };
  const int64_t c = (int64_t)blockIdx.x * ng + g;
  const int64_t last = (c + 1) * A.chunk - 1;  // the chunk's last token
  if (last + 1 < A.t) {
    const uint32_t key = A.keys[last], first = A.keys[c * A.chunk];
    const bool earlier = first == key && c > 0 && A.keys[c * A.chunk - 1] == key;
    if (key != (uint32_t)A.rows && A.keys[last + 1] == key && !earlier) {
      // end of the segment: the first token with a larger key, near by or by bisection
      int64_t lo = last + 1, hi = min(A.t, last + 1 + (int64_t)kJoinShort * A.chunk);
      if (hi < A.t && A.keys[hi - 1] == key) {
        lo = hi;
        hi = A.t;
      }
      while (lo < hi) {
        const int64_t m = (lo + hi) >> 1;
        if (A.keys[m] > key) hi = m;
        else lo = m + 1;
      }
      const int64_t end = (lo - 1) / A.chunk;  // chunk of the segment's last token
      if (end - c <= kJoinShort) {
        for (int u = sub; u < A.nunit; u += tpr) {
          float a[N] = {};
          add_rows(c, c, end, 1, (int64_t)u * N, a);
          write_row<DT, OUT, VEC>(A, key, (int64_t)u * N, a);
        }
      } else if (sub == 0) {
        const int at = atomicAdd(&nlong, 1);  // (their order changes no sum)
        long_c[at] = c;
        long_end[at] = end;
      }
    }
  }
  __syncthreads();
  for (int s = 0; s < nlong; ++s) {
    const int64_t lc = long_c[s], le = long_end[s];
    const uint32_t key = A.keys[(lc + 1) * A.chunk];
    for (int u0 = 0; u0 < A.nunit; u0 += tpr) {
      const int u = u0 + sub;
      float a[N] = {};
      if (u < A.nunit) add_rows(lc, lc + g, le, ng, (int64_t)u * N, a);
#pragma unroll
      for (int e = 0; e < N; ++e) red[threadIdx.x * N + e] = a[e];
      __syncthreads();
      for (int h = ng >> 1; h >= 1; h >>= 1) {
        if (g < h) {
#pragma unroll
          for (int e = 0; e < N; ++e) red[threadIdx.x * N + e] += red[(threadIdx.x + h * tpr) * N + e];
        }
        __syncthreads();
      }
      if (g == 0 && u < A.nunit) {
#pragma unroll
        for (int e = 0; e < N; ++e) a[e] = red[threadIdx.x * N + e];
        write_row<DT, OUT, VEC>(A, key, (int64_t)u * N, a);
      }
      __syncthreads();
    }
  }
}

// ------------------------------------------------------------------------- few tokens
// One launch: a workgroup owns 2^rlog rows of the output. Its waves look through all ids, a
// quarter each, and keep the tokens of its rows in token order; a counting sort in LDS by row
// (stable, as above) puts a row's tokens in a run; groups of 2^tpr_log lanes sum a row each and
// write it, zeros where it has no token. A row with many tokens is summed by all groups of the
// workgroup in turns and joined in a fixed order. Every workgroup reads the ids; small_pays() says
// when that costs less than the launches it saves. Bound by latency: 8191 tokens of 65,536 x 64 f32
// take 15.4 us, sorted 50.
constexpr int kSmallMax = 16384;
constexpr int kSmallRows = 1024;   // rows of a workgroup, at most
constexpr int kSmallHot = 32;      // tokens of a row that one group sums by itself, at most
constexpr int kSmallBatch = 16;    // id loads in flight a lane
constexpr int kSmallSum = 8;       // row loads in flight a lane
constexpr int kLdsBytes = 160 * 1024;

struct SmallArgs {
  SegArgs G;        // grad, rows, d, units, scale, output
  const void* ids;
  int rlog;
};

// LDS: the waves' tokens (and later the groups' sums, 256 units), and the sorted tokens.
__host__ __device__ constexpr int small_list(int t) {
  return (t + 255) / 256 * 256 * 4 > 8192 ? (t + 255) / 256 * 256 * 4 : 8192;
}
__host__ __device__ constexpr int small_lds(int t) { return small_list(t) + (t + 1) / 2 * 4; }
constexpr int kSmallStatic = 22 * 1024;  // the rest of it

// Workgroups that run at once: as many a compute unit as its LDS holds, at most 4.
static int64_t small_resident(int t) {
  const int fit = kLdsBytes / (small_lds(t) + kSmallStatic);
  return (int64_t)device_cu_count() * (fit > 4 ? 4 : (fit < 1 ? 1 : fit));
}

// Whether the gradient takes one launch. Each round of workgroups reads all ids, so the tokens
// times the rounds decide (all at once on one card, sorted against one launch, in microseconds):
// 8000 tokens of 1M x 128 rows in bf16, 2 rounds, 69 : 50; 16,000 of 262,144, 1 round, 51 : 36;
// 4000 of 4M x 64, 6 rounds, 109 : 101; 8000 of 4M x 64, 8 rounds, 114 : 131; 16,000 of 1M x 128,
// 4 rounds, 71 : 104.
constexpr int64_t kSmallRounds = 32768;
static bool small_pays(int64_t t, int64_t rows) {
  if (t > kSmallMax) return false;
  const int64_t most = small_resident((int)t);
  const int64_t rounds = ((rows + kSmallRows - 1) / kSmallRows + most - 1) / most;
  return t * rounds <= kSmallRounds;
}

template <int DT, int OUT, bool VEC, typename IdT>
__global__ __launch_bounds__(256) void small_kernel(SmallArgs P) {
  const SegArgs& A = P.G;
  using U = Unit<DT, VEC>;
  constexpr int N = U::N;
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  __shared__ uint32_t off[4][kSmallRows];
  __shared__ uint32_t start[kSmallRows + 1];
  __shared__ uint32_t wsum[4];
  __shared__ uint16_t hot[kSmallMax / kSmallHot];
  __shared__ uint32_t nhot;
  float* red = (float*)dyn;  // (the lists have been used by then)
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int n = (int)A.t, quarter = (n + 255) / 256 * 64, R = 1 << P.rlog;
  const int64_t row0 = (int64_t)blockIdx.x << P.rlog;
  const int64_t nrow = min<int64_t>(R, A.rows - row0);
  uint32_t* list = (uint32_t*)dyn + wave * quarter;          // row within the workgroup << 14 | token
  uint16_t* sorted = (uint16_t*)(dyn + small_list(n));
  for (int i = t; i < 4 * R; i += 256) off[i >> P.rlog][i & (R - 1)] = 0u;
  if (t == 0) nhot = 0u;
  __syncthreads();

  int m = 0;  // tokens kept by this wave
  for (int i0 = wave * quarter; i0 < (wave + 1) * quarter; i0 += kWave * kSmallBatch) {
    IdT id[kSmallBatch];
#pragma unroll
    for (int u = 0; u < kSmallBatch; ++u) {
      const int i = i0 + u * kWave + lane;
      id[u] = i < n && i < (wave + 1) * quarter ? ((const IdT*)P.ids)[i] : (IdT)-1;
    }
#pragma unroll
    for (int u = 0; u < kSmallBatch; ++u) {
      const uint64_t r = (uint64_t)(int64_t)id[u] - (uint64_t)row0;  // (ids before row0 wrap to the far end)
      const bool on = id[u] >= 0 && r < (uint64_t)nrow;
      const uint64_t mask = __ballot(on);
      if (on) {
        list[m + __popcll(mask & ((1ull << lane) - 1ull))] = (uint32_t)r << 14 | (uint32_t)(i0 + u * kWave + lane);
        atomicAdd(&off[wave][r], 1u);
      }
      m += __popcll(mask);
    }
  }
  __syncthreads();
  // first places: rows 4 t .. 4 t + 3 of thread t, then the waves within a row
  uint32_t cnt[4], all = 0u;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int r = 4 * t + e;
    cnt[e] = r < R ? off[0][r] + off[1][r] + off[2][r] + off[3][r] : 0u;
    all += cnt[e];
  }
  uint32_t incl = all;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const uint32_t x = __shfl_up(incl, o, kWave);
    if (lane >= o) incl += x;
  }
  if (lane == kWave - 1) wsum[wave] = incl;
  __syncthreads();
  uint32_t p = incl - all;
  for (int w = 0; w < wave; ++w) p += wsum[w];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int r = 4 * t + e;
    if (r < R) {
      start[r] = p;
      if (r == R - 1) start[R] = p + cnt[e];
      uint32_t q = p;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t c = off[w][r];
        off[w][r] = q;
        q += c;
      }
      if (cnt[e] > (uint32_t)kSmallHot) hot[atomicAdd(&nhot, 1u)] = (uint16_t)r;  // (their order changes no sum)
    }
    p += cnt[e];
  }
  __syncthreads();
  for (int i0 = 0; i0 < m; i0 += kWave) {  // wave-uniform
    const bool on = i0 + lane < m;
    const uint32_t x = on ? list[i0 + lane] : 0u;
    const uint32_t to = take_place(off[wave], x >> 14, P.rlog, on);
    if (on) sorted[to] = (uint16_t)(x & 16383u);
  }
  __syncthreads();

  const int tpr = 1 << A.tpr_log;
  const int sub = t & (tpr - 1), g = t >> A.tpr_log, ng = 256 >> A.tpr_log;
  // adds tokens from, from + step, .. below `to` of the sorted list
  auto add_tokens = [&](uint32_t from, uint32_t to, uint32_t step, int64_t j, float (&a)[N]) __attribute__((always_inline)) {
    for (uint32_t i = from; i < to; i += kSmallSum * step) {
      float v[kSmallSum][N];
#pragma unroll
      for (int b = 0; b < kSmallSum; ++b)
        if (i + b * step < to) U::load(A.grad, (int64_t)sorted[i + b * step] * A.grad_stride + j, v[b]);
#pragma unroll
      for (int b = 0; b < kSmallSum; ++b)
        if (i + b * step < to)
#pragma unroll
          for (int e = 0; e < N; ++e) a[e] += v[b][e];
    }
  };
  for (int r = g; r < nrow; r += ng) {
    const uint32_t from = start[r], to = start[r + 1];
    if (to - from > (uint32_t)kSmallHot || (to == from && A.accumulate)) continue;
    for (int u = sub; u < A.nunit; u += tpr) {
      float a[N] = {};
      add_tokens(from, to, 1, (int64_t)u * N, a);
      write_row<DT, OUT, VEC>(A, (uint32_t)(row0 + r), (int64_t)u * N, a);
    }
  }
  for (uint32_t s = 0; s < nhot; ++s) {
    const uint32_t r = hot[s];
    for (int u0 = 0; u0 < A.nunit; u0 += tpr) {
      const int u = u0 + sub;
      float a[N] = {};
      if (u < A.nunit) add_tokens(start[r] + g, start[r + 1], ng, (int64_t)u * N, a);
      __syncthreads();
#pragma unroll
      for (int e = 0; e < N; ++e) red[t * N + e] = a[e];
      __syncthreads();
      for (int h = ng >> 1; h >= 1; h >>= 1) {
        if (g < h) {
#pragma unroll
          for (int e = 0; e < N; ++e) red[t * N + e] += red[(t + h * tpr) * N + e];
        }
        __syncthreads();
      }
      if (g == 0 && u < A.nunit) {
#pragma unroll
        for (int e = 0; e < N; ++e) a[e] = red[t * N + e];
        write_row<DT, OUT, VEC>(A, (uint32_t)(row0 + r), (int64_t)u * N, a);
      }
    }
  }
}

template <int DT, int OUT, bool VEC>
static int launch_small(SegArgs G, const void* ids, int id_bits, hipStream_t s) {
  G.nunit = G.d / Unit<DT, VEC>::N;
  G.tpr_log = log2_lanes(G.nunit);
  // rows of a workgroup: so many that all workgroups run at once, but at most kSmallRows
  SmallArgs P{G, ids, 0};
  const int64_t most = small_resident((int)G.t);
  while (P.rlog < 10 && ((G.rows - 1) >> P.rlog) + 1 > most) ++P.rlog;
  static_assert(kSmallRows == 1 << 10, "rlog is at most 10");
  static const hipError_t attr[2] = {
      hipFuncSetAttribute((const void*)small_kernel<DT, OUT, VEC, int32_t>, hipFuncAttributeMaxDynamicSharedMemorySize,
                          small_lds(kSmallMax)),
      hipFuncSetAttribute((const void*)small_kernel<DT, OUT, VEC, int64_t>, hipFuncAttributeMaxDynamicSharedMemorySize,
                          small_lds(kSmallMax))};
  (void)attr;
  const dim3 grid((unsigned)((G.rows + (1 << P.rlog) - 1) >> P.rlog));
  const size_t lds = small_lds((int)G.t);
  if (id_bits == 32) hipLaunchKernelGGL((small_kernel<DT, OUT, VEC, int32_t>), grid, dim3(256), lds, s, P);
  else hipLaunchKernelGGL((small_kernel<DT, OUT, VEC, int64_t>), grid, dim3(256), lds, s, P);
  return check_launch();
}

// Sorted tokens per group: enough groups to fill the chip (about 16 waves a compute unit) before
// a group takes more than 8 tokens, at most 64. A call of 520,192 tokens of 128 bf16 with chunks of
// 8, 16, 32, 64, 128 takes 151, 141, 134, 141, 161 us (32 is chosen); 30,000 of 64 f32 with 8, 16,
// 32, 64 56.5, 58.3, 60.0, 69.7 (8).
static int seg_chunk(int64_t t, int tpr_log) {
  const int64_t groups = (int64_t)4096 * 64 >> tpr_log;
  int c = 8;
  while (c < 64 && t / c > groups) c *= 2;
  return c;
}

template <int DT, int OUT, bool VEC>
static int launch_segments(SegArgs A, hipStream_t s) {
  A.nunit = A.d / Unit<DT, VEC>::N;
  A.tpr_log = log2_lanes(A.nunit);
  A.chunk = seg_chunk(A.t, A.tpr_log);
  A.nchunk = (A.t + A.chunk - 1) / A.chunk;
  const int groups = 256 >> A.tpr_log;
  hipLaunchKernelGGL((segment_kernel<DT, OUT, VEC>), dim3((unsigned)((A.nchunk + groups - 1) / groups)),
                     dim3(256), 0, s, A);
  if (const int rc = check_launch()) return rc;
  if (A.nchunk > 1) {
    hipLaunchKernelGGL((join_kernel<DT, OUT, VEC>), dim3((unsigned)((A.nchunk - 1 + groups - 1) / groups)), dim3(256),
                       0, s, A);
    return check_launch();
  }
  return MIPS_OK;
}

struct GradPlan {
  int64_t per;
  int nb, passes;
  size_t keys[2], toks[2], counts, part, bytes;
};

static GradPlan grad_plan(int64_t t, int64_t rows, int d) {
  GradPlan P{};
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t p = at;
    at += (n + 255) / 256 * 256;
    return p;
  };
  int bits = 1;  // keys 0 .. rows
  while ((int64_t(1) << bits) <= rows) ++bits;
  if (small_pays(t, rows)) {
    P.bytes = 256;
    return P;
  }
  P.passes = (bits + 7) / 8;
  P.nb = (int)((t + kSortTile - 1) / kSortTile < kSortBlocks ? (t + kSortTile - 1) / kSortTile : kSortBlocks);
  if (P.nb < 1) P.nb = 1;
  P.per = (t + P.nb - 1) / P.nb;
  P.per = (P.per + kSortTile - 1) / kSortTile * kSortTile;
  P.nb = (int)((t + P.per - 1) / P.per);
  P.keys[0] = take((size_t)t * 4);
  P.toks[0] = take((size_t)t * 4);
  P.keys[1] = take((size_t)t * 4);
  P.toks[1] = take((size_t)t * 4);
  P.counts = take((size_t)P.nb * 256 * 4);
  // partial rows: two per chunk (rows in 16-byte units share the fewest lanes, and so have
  // the smallest chunks)
  const int chunk = seg_chunk(t, log2_lanes(d / 8));
  P.part = take((size_t)((t + chunk - 1) / chunk) * 2 * (size_t)d * 4);
  P.bytes = at;
  return P;
}

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 64;

static bool dtype_ok(int dt) { return dt == MIPS_F32 || dt == MIPS_BF16; }

}  // namespace mips

extern "C" {

int mips_embedding_lookup(const void* table, int32_t dtype, int64_t rows, int32_t d,
                          int64_t row_stride, const void* ids, int32_t id_bits, int64_t t,
                          float scale, void* out, void* stream) {
  using namespace mips;
  if (t < 0 || rows < 1 || d < 1 || row_stride < d) return MIPS_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || (id_bits != 32 && id_bits != 64) || d > MIPS_EMBEDDING_D_MAX)
    return MIPS_ERR_UNSUPPORTED;
  if (t == 0) return MIPS_OK;
  const int E = elem_bytes(dtype);
  if (!table || !ids || !out || !aligned(table, E) || !aligned(out, E) || !aligned(ids, id_bits / 8))
    return MIPS_ERR_INVALID_ARG;
  LookupArgs A{table, rows, row_stride, ids, t, scale, out, d, 0, 0};
  hipStream_t s = (hipStream_t)stream;
  const bool vec = aligned(table, 16) && aligned(out, 16) && (row_stride * E) % 16 == 0 && (d * E) % 16 == 0;
  if (dtype == MIPS_F32) return vec ? launch_lookup<MIPS_F32, true>(A, id_bits, s) : launch_lookup<MIPS_F32, false>(A, id_bits, s);
  return vec ? launch_lookup<MIPS_BF16, true>(A, id_bits, s) : launch_lookup<MIPS_BF16, false>(A, id_bits, s);
}

size_t mips_embedding_grad_workspace_size(int64_t t, int64_t rows, int32_t d) {
  if (t < 0 || t > MIPS_TOKENS_MAX || rows < 1 || rows > mips::kMaxRows || d < 1 || d > MIPS_EMBEDDING_D_MAX)
    return 0;
  return mips::grad_plan(t, rows, d).bytes;
}

int mips_embedding_grad(const void* grad, int32_t grad_dtype, int64_t t, int32_t d,
                        int64_t grad_stride, const void* ids, int32_t id_bits, int64_t rows,
                        float scale, int32_t accumulate, void* out, int32_t out_dtype,
                        int64_t out_stride, void* workspace, size_t workspace_bytes,
                        void* stream) {
  using namespace mips;
  if (t < 0 || rows < 1 || d < 1 || grad_stride < d || out_stride < d) return MIPS_ERR_INVALID_ARG;
  if (!dtype_ok(grad_dtype) || (out_dtype != grad_dtype && out_dtype != MIPS_F32) ||
      (id_bits != 32 && id_bits != 64) || d > MIPS_EMBEDDING_D_MAX || t > MIPS_TOKENS_MAX ||
      rows > kMaxRows)
    return MIPS_ERR_UNSUPPORTED;
  const int E = elem_bytes(grad_dtype), O = elem_bytes(out_dtype);
  if (!out || !aligned(out, O)) return MIPS_ERR_INVALID_ARG;
  if (t > 0 && (!grad || !ids || !aligned(grad, E) || !aligned(ids, id_bits / 8) || !workspace ||
                !aligned(workspace, 256)))
    return MIPS_ERR_INVALID_ARG;
  hipStream_t s = (hipStream_t)stream;
  const GradPlan P = grad_plan(t, rows, d);
  if (t > 0 && workspace_bytes < P.bytes) return MIPS_ERR_WORKSPACE;
  uint8_t* ws = (uint8_t*)workspace;
  SegArgs G{grad, grad_stride, nullptr, nullptr, t, rows, d, 0, 0, 0, scale, accumulate, out, out_stride, nullptr, 0};
  const bool vec = aligned(grad, 16) && aligned(out, 16) && (grad_stride * E) % 16 == 0 &&
                   (out_stride * O) % 16 == 0 && (d * E) % 16 == 0;
  // the launcher of the operands' types and units: of few tokens, or of sorted ones
  auto dispatch = [&](auto small) {
    auto go = [&](auto dt, auto ot, auto v) {
      constexpr int DT = decltype(dt)::value, OT = decltype(ot)::value;
      constexpr bool V = decltype(v)::value;
      if constexpr (decltype(small)::value) return launch_small<DT, OT, V>(G, ids, id_bits, s);
      else return launch_segments<DT, OT, V>(G, s);
    };
    using F32 = std::integral_constant<int, MIPS_F32>;
    using B16 = std::integral_constant<int, MIPS_BF16>;
    if (grad_dtype == MIPS_F32) return vec ? go(F32{}, F32{}, std::true_type{}) : go(F32{}, F32{}, std::false_type{});
    if (out_dtype == MIPS_BF16) return vec ? go(B16{}, B16{}, std::true_type{}) : go(B16{}, B16{}, std::false_type{});
    return vec ? go(B16{}, F32{}, std::true_type{}) : go(B16{}, F32{}, std::false_type{});
  };
  if (small_pays(t, rows)) return t == 0 && accumulate ? MIPS_OK : dispatch(std::true_type{});

  const ZeroArgs Z{out, 0, rows, out_stride * O, (int64_t)d * O, accumulate ? 0 : 1};
  int src = 0;
  {
    for (int p = 0; p < P.passes; ++p) {
      const int in = (p + 1) & 1, to = p & 1;  // pass 0 reads the ids and writes buffer 0
      SortArgs S{p == 0 ? ids : nullptr, t, rows, P.per, P.nb, 8 * p,
                 (const uint32_t*)(ws + P.keys[in]), (const uint32_t*)(ws + P.toks[in]),
                 (uint32_t*)(ws + P.keys[to]), (uint32_t*)(ws + P.toks[to]),
                 (uint32_t*)(ws + P.counts), zero_part(Z, 2 * p, 2 * P.passes, kSortThreads)};
      const dim3 gc(P.nb + S.Z.nblocks);
      if (id_bits == 32) hipLaunchKernelGGL(sort_count_kernel<int32_t>, gc, dim3(kSortThreads), 0, s, S);
      else hipLaunchKernelGGL(sort_count_kernel<int64_t>, gc, dim3(kSortThreads), 0, s, S);
      if (const int rc = check_launch()) return rc;
      S.Z = zero_part(Z, 2 * p + 1, 2 * P.passes, kSortThreads);
      const dim3 gs(P.nb + S.Z.nblocks);
      if (id_bits == 32) hipLaunchKernelGGL(sort_scatter_kernel<int32_t>, gs, dim3(kSortThreads), 0, s, S);
      else hipLaunchKernelGGL(sort_scatter_kernel<int64_t>, gs, dim3(kSortThreads), 0, s, S);
      if (const int rc = check_launch()) return rc;
      src = to;
    }
  }
  G.keys = (const uint32_t*)(ws + P.keys[src]);
  G.toks = (const uint32_t*)(ws + P.toks[src]);
  G.part = (float*)(ws + P.part);
  return dispatch(std::false_type{});
}

}  // extern "C"
