// pool.hip -- the mean of a sequence's rows, L2-normalised, and its gradient (gfx950).
//
//   m = sum of the rows / their number (0 without rows),  n = sqrt(max(sum m^2, 1e-12)),  u = m / n
//   dm = (g - u (u . g)) / n, or g / n where the sum is below 1e-12;  each row's gradient dm / number
//
// Bound by reading the rows, and by writing their gradients: 4096 x 127 x 128 bf16 with lengths take 16 us
// (67 MB, 4.2 TB/s) and 27 us (133 MB, 4.9 TB/s); short calls by latency, 16 x 50 x 64 5 us.
// (Normalisation as the index's: sum over all channels, 1e-12 under the root:
// recsys_two_tower_model.py:69, 73-76, 1287-1306.)
#include "sequences.h"

namespace mips {

constexpr int kPoolThreads = 256;  // four waves, each on its own
constexpr int kPoolWaves = kPoolThreads / 64;
constexpr float kPoolEps = 1e-12f;
constexpr int kAhead = 8;  // rows that a lane loads together

struct PoolArgs {
  Sequences S;
  Rows x;           // forward: the rows
  int32_t d;
  int32_t lanes;    // of a row, 8 channels each, 1 to 64
  int32_t normalize;
  uint32_t chunk;   // rows of a wave
  uint32_t chunks;
  float* part;      // [chunks][2][d]: sums of the sequence that a chunk goes on with, of the one it leaves open
  void* vectors;    // [b, d]
  float* mean;      // [b, d]
  float* norm;      // [b]
  const void* grad; // backward: [b, d], grad_stride apart
  int64_t grad_stride;
  int32_t grad_aligned;
  void* dx;         // [n, d]
};

// Eight channels of a row, 16-byte loads with VEC (bf16: one, f32: two). Without, the same from any
// address of an element; `live` < 8 only where d is.
template <typename T, bool VEC>
__device__ __forceinline__ void row8(const T* p, int live, float* v) {
  typedef T v8_t __attribute__((ext_vector_type(8), aligned(16)));
  if constexpr (VEC) {
    const v8_t q = *(const v8_t*)p;
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = (float)q[c];
  } else {
    typedef T u8_t __attribute__((ext_vector_type(8), aligned(sizeof(T))));
    u8_t q = (T)0.0f;
    if (live == 8) {
      q = *(const u8_t*)p;
    } else {
#pragma unroll
      for (int c = 0; c < 7; ++c)
        if (c < live) q[c] = p[c];
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = (float)q[c];
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void put8(T* p, int live, const float* v) {
  typedef T v8_t __attribute__((ext_vector_type(8), aligned(16)));
  if constexpr (VEC) {
    v8_t q;
#pragma unroll
    for (int c = 0; c < 8; ++c) q[c] = (T)v[c];
    __builtin_nontemporal_store(q, (v8_t*)p);
  } else {
    typedef T u8_t __attribute__((ext_vector_type(8), aligned(sizeof(T))));
    u8_t q;
#pragma unroll
    for (int c = 0; c < 8; ++c) q[c] = (T)v[c];
    if (live == 8) {
      *(u8_t*)p = q;
    } else {
#pragma unroll
      for (int c = 0; c < 7; ++c)
        if (c < live) p[c] = q[c];
    }
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// sum m^2 -> the norm (NaN stays NaN).
__device__ __forceinline__ float pool_norm(const PoolArgs& A, float square) {
  if (!A.normalize) return 1.0f;
  return sqrtf(square < kPoolEps ? kPoolEps : square);
}

// The eight channels of a row that a lane has in the span from c0: *live of them (0: none), from *c. Where
// the last lane's would pass the end of a row of eight or more, it takes the last eight, the first `skip`
// of which are its neighbour's too: both compute and write the same. (24 x 23,696 x 100 bf16 with lengths: 16 us,
// its gradient 19; 71 and 83 where elements move one by one.)
__device__ __forceinline__ void span8(int32_t d, int at, int* c, int* live, int* skip) {
  const int left = d - at;
  *c = left < 8 && d >= 8 ? d - 8 : at;
  *live = left <= 0 ? 0 : (d < 8 ? d : 8);
  *skip = at - *c;
}

// One wave a chunk: the sums of its sequences; those that lie whole in it are finished.
template <typename T, bool VEC>
__global__ __launch_bounds__(kPoolThreads) void pool_kernel(PoolArgs A) {
  const uint32_t chunk = blockIdx.x * kPoolWaves + (threadIdx.x >> 6);
  if (chunk >= A.chunks) return;
  const uint32_t r0 = chunk * A.chunk, r1 = min(r0 + A.chunk, A.S.n);
  const int lane = threadIdx.x & 63, lanes = A.lanes, slots = 64 / lanes, slot = lane / lanes;
  const int at = (lane & (lanes - 1)) * 8;
  for_sequences(A.S, r0, r1, [&](int32_t s, uint32_t begin, uint32_t end) {
    const uint32_t lo = max(begin, r0), hi = min(end, r1);
    const bool whole = begin >= r0 && end <= r1;
    const float inv = end > begin ? 1.0f / (float)(end - begin) : 0.0f;
    float square = 0.0f, sum[8];
    for (int c0 = 0; c0 < A.d; c0 += lanes * 8) {
      int c, live, skip;
      span8(A.d, c0 + at, &c, &live, &skip);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
      if (live > 0) {
        const T* p = (const T*)A.x.p + (A.S.t ? s * A.x.extra : 0) + c;
        uint32_t r = lo + slot;
        for (; r + (kAhead - 1) * slots < hi; r += kAhead * slots) {
          float v[kAhead][8];
#pragma unroll
          for (int k = 0; k < kAhead; ++k) row8<T, VEC>(p + (int64_t)(r + k * slots) * A.x.row, live, v[k]);
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[e] += ((v[0][e] + v[1][e]) + (v[2][e] + v[3][e])) + ((v[4][e] + v[5][e]) + (v[6][e] + v[7][e]));
        }
        for (; r < hi; r += slots) {
          float v[8];
          row8<T, VEC>(p + (int64_t)r * A.x.row, live, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[e] += v[e];
        }
      }
      for (int o = lanes; o < 64; o <<= 1) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += __shfl_xor(sum[e], o);
      }
      if (slot || live <= 0) continue;
      if (!whole) {
        float* q = A.part + ((int64_t)chunk * 2 + (begin < r0 ? 0 : 1)) * A.d + c;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < live) q[e] = sum[e];
        continue;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum[e] *= inv;
        if (e >= skip) square = fmaf(sum[e], sum[e], square);
      }
      float* q = A.mean + (int64_t)s * A.d + c;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < live) q[e] = sum[e];
    }
    if (!whole) return;
    const float n = pool_norm(A, wave_sum(square));
    if (lane == 0) A.norm[s] = n;
    if (slot) return;
    for (int c0 = 0; c0 < A.d; c0 += lanes * 8) {
      int c, live, skip;
      span8(A.d, c0 + at, &c, &live, &skip);
      if (live <= 0) continue;
      if (A.d > lanes * 8) {  // several spans: this lane wrote them above
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = e < live ? A.mean[(int64_t)s * A.d + c + e] : 0.0f;
      }
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = sum[e] / n;
      put8<T, VEC>((T*)A.vectors + (int64_t)s * A.d + c, live, v);
    }
  });
}

// One workgroup a sequence: those that lie in several chunks, and packed ones without rows. W channels' parts
// are added by several threads, eight in flight each, and joined in their order. (W = 4 where d allows it:
// 8 sequences of 94 parts of 1024 channels take 19 us with 1, 12 with 4.)
template <typename T, int kJoinThreads, int W>
__global__ __launch_bounds__(kJoinThreads) void pool_join_kernel(PoolArgs A) {
  typedef float v_t __attribute__((ext_vector_type(W)));
  __shared__ float red[kJoinThreads / 64];
  __shared__ v_t part[kJoinThreads];
  const int tid = threadIdx.x;
  const int64_t s = blockIdx.x;
  uint32_t begin, end;
  sequence_rows(A.S, s, &begin, &end);
  const uint32_t k0 = begin / A.chunk, k1 = end > begin ? (end - 1) / A.chunk : k0;
  if (k0 == k1 && (end > begin || A.S.t)) return;
  const float inv = end > begin ? 1.0f / (float)(end - begin) : 0.0f;
  int span = 16;  // threads side by side
  while (span < kJoinThreads && span * W < A.d) span *= 2;
  const int slices = kJoinThreads / span, slice = tid / span;
  const uint32_t parts = end > begin ? k1 - k0 + 1 : 0u, each = (parts + slices - 1) / slices;
  float square = 0.0f;
  for (int c0 = 0; c0 < A.d; c0 += span * W) {
    const int c = c0 + (tid & (span - 1)) * W;
    v_t sum = 0.0f;
    if (c < A.d) {
      const uint32_t lo = slice * each, hi = min(lo + each, parts);
      // the first chunk left the sequence open, the others went on with it
      auto at = [&](uint32_t j) { return *(const v_t*)(A.part + ((int64_t)(k0 + j) * 2 + (j == 0 ? 1 : 0)) * A.d + c); };
      uint32_t j = lo;
      for (; j + 8 <= hi; j += 8)
        sum += ((at(j) + at(j + 1)) + (at(j + 2) + at(j + 3))) + ((at(j + 4) + at(j + 5)) + (at(j + 6) + at(j + 7)));
      for (; j < hi; ++j) sum += at(j);
    }
    __syncthreads();
    part[tid] = sum;
    __syncthreads();
    if (slice == 0 && c < A.d) {
      for (int q = 1; q < slices; ++q) sum += part[q * span + tid];
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const float m = sum[e] * inv;
        A.mean[s * A.d + c + e] = m;
        square = fmaf(m, m, square);
      }
    }
  }
  square = wave_sum(square);
  if ((tid & 63) == 0) red[tid >> 6] = square;
  __syncthreads();
  square = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 64; ++w) square += red[w];
  const float n = pool_norm(A, square);
  if (tid == 0) A.norm[s] = n;
  if (slice) return;
  for (int c0 = tid * W; c0 < A.d; c0 += span * W)  // this thread wrote these
#pragma unroll
    for (int e = 0; e < W; ++e) ((T*)A.vectors)[s * A.d + c0 + e] = (T)(A.mean[s * A.d + c0 + e] / n);
}

// One wave a chunk of rows, each sequence's row of gradients computed again for every chunk.
template <typename T, bool VEC>
__global__ __launch_bounds__(kPoolThreads) void pool_grad_kernel(PoolArgs A) {
  const uint32_t chunk = blockIdx.x * kPoolWaves + (threadIdx.x >> 6);
  if (chunk >= A.chunks) return;
  const uint32_t r0 = chunk * A.chunk, r1 = min(r0 + A.chunk, A.S.n);
  const int lane = threadIdx.x & 63, lanes = A.lanes, slots = 64 / lanes, slot = lane / lanes;
  const int at = (lane & (lanes - 1)) * 8;
  // rows [lo, hi) of dx as v, channels c ..
  auto fill = [&](uint32_t lo, uint32_t hi, int c, int live, const float* v) {
    for (uint32_t r = lo + slot; r < hi; r += slots) put8<T, VEC>((T*)A.dx + (int64_t)r * A.d + c, live, v);
  };
  auto zeros = [&](uint32_t lo, uint32_t hi) {
    const float v[8] = {};
    for (int c0 = at; c0 < A.d; c0 += lanes * 8) {
      int c, live, skip;
      span8(A.d, c0, &c, &live, &skip);
      fill(lo, hi, c, live, v);
    }
  };
  for_sequences(A.S, r0, r1, [&](int32_t s, uint32_t begin, uint32_t end) {
    if (A.S.t) zeros(max(end, r0), min(begin + A.S.t, r1));
    if (end <= r0) return;
    const float* m = A.mean + (int64_t)s * A.d;
    const T* g = (const T*)A.grad + s * A.grad_stride;
    const float n = A.norm[s], inv = 1.0f / (float)(end - begin);
    // u (u . g) = m (m . g) / n^2, away where the root is that of 1e-12
    auto along = [&](float dot, float square) { return A.normalize && !(square < kPoolEps) ? dot / n / n : 0.0f; };
    const uint32_t lo = max(begin, r0), hi = min(end, r1);
    auto read = [&](int c, int live, float* mv, float* gv) {
      if (A.normalize) {
        row8<float, VEC>(m + c, live, mv);
      } else {  // the gradient does not depend on the mean, which need not be finite
#pragma unroll
        for (int e = 0; e < 8; ++e) mv[e] = 0.0f;
      }
      if (VEC && A.grad_aligned) row8<T, VEC>(g + c, live, gv);
      else row8<T, false>(g + c, live, gv);
    };
    if (A.d <= lanes * 8) {  // one span: a lane's channels of m and g are read once
      int c, live, skip;
      span8(A.d, at, &c, &live, &skip);
      float mv[8], gv[8], dot = 0.0f, square = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) mv[e] = gv[e] = 0.0f;
      if (live > 0) read(c, live, mv, gv);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e < skip) continue;
        dot = fmaf(mv[e], gv[e], dot);
        square = fmaf(mv[e], mv[e], square);
      }
      for (int o = 1; o < lanes; o <<= 1) {
        dot += __shfl_xor(dot, o);
        square += __shfl_xor(square, o);
      }
      if (live <= 0) return;
      const float t = along(dot, square);
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (gv[e] - mv[e] * t) / n * inv;
      fill(lo, hi, c, live, v);
      return;
    }
    // several spans: their channels are read again for the results
    float mv[8], gv[8], dot = 0.0f, square = 0.0f;
    for (int c0 = at; c0 < A.d && A.normalize; c0 += lanes * 8) {
      int c, live, skip;
      span8(A.d, c0, &c, &live, &skip);
      read(c, live, mv, gv);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e < skip) continue;
        dot = fmaf(mv[e], gv[e], dot);
        square = fmaf(mv[e], mv[e], square);
      }
    }
    const float t = along(wave_sum(dot), wave_sum(square));
    for (int c0 = at; c0 < A.d; c0 += lanes * 8) {
      int c, live, skip;
      span8(A.d, c0, &c, &live, &skip);
      read(c, live, mv, gv);
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (gv[e] - mv[e] * t) / n * inv;
      fill(lo, hi, c, live, v);
    }
  });
  if (!A.S.t) {  // packed rows of no sequence
    zeros(r0, min(r1, index_at(A.S.offsets, A.S.wide, 0, A.S.n)));
    zeros(max(r0, index_at(A.S.offsets, A.S.wide, A.S.b, A.S.n)), r1);
  }
}

// Whether every sequence is pooled whole by one wave: short dense ones, longer ones where there are waves
// enough without cutting them.
static bool pool_whole(const Sequences& S, int32_t d) {
  return S.t && S.t <= 256 && (S.b >= 1024 || (int64_t)S.t * d <= 8192);
}
// Rows of a wave. Sequences are few microseconds of latency each, so few go to one wave where they are
// short (2147 packed ones of up to two rows: 16 a wave take 20 us, 4 take 8). Cut ones: as many rows as leave
// 4096 waves, but few parts to join, fewer where rows are wide.
static uint32_t pool_chunk(const Sequences& S, int32_t d) {
  if (pool_whole(S, d)) {
    const uint32_t rows = S.n / 8192;
    return rows < 32 ? (rows > S.t ? rows / S.t * S.t : S.t) : (S.t >= 32 ? S.t : 32 / S.t * S.t);
  }
  const uint32_t mean = S.n / S.b, wide = d > 512 ? 16 : 8192 / d;
  uint32_t least = mean < 4 ? 4 : (mean > 64 ? 64 : mean);
  if (wide < least) least = wide > 16 ? wide : (least < 16 ? least : 16);
  const uint32_t rows = S.n / 4096;
  return rows < least ? least : (rows > 1024 ? 1024 : rows);
}
template <typename T>
static void (*join_kernel_of(bool few, int32_t d))(PoolArgs) {
  if (d % 4) return few ? pool_join_kernel<T, 128, 1> : pool_join_kernel<T, 1024, 1>;
  return few ? pool_join_kernel<T, 128, 4> : pool_join_kernel<T, 1024, 4>;
}
static int pool_lanes(int32_t d) {
  int lanes = 1;
  while (lanes < 64 && lanes * 8 < d) lanes *= 2;
  return lanes;
}
static size_t pool_bytes(const Sequences& S, int32_t d) {
  if (pool_whole(S, d)) return 0;
  const uint32_t chunk = pool_chunk(S, d);
  return 256 + ((size_t)S.n + chunk - 1) / chunk * 2 * d * sizeof(float);
}

}  // namespace mips

using namespace mips;

extern "C" {

size_t mips_pool_workspace_size(const mips_sequences* seq, int32_t d) {
  Sequences S;
  if (check_sequences(seq, &S) != MIPS_OK || d < 1 || d > MIPS_EMBEDDING_D_MAX) return 0;
  return pool_bytes(S, d);
}

int mips_pool_normalize(const mips_sequences* seq, int32_t d, int32_t dtype, const mips_rows* x, int32_t normalize,
                        void* vectors, float* mean, float* norm, void* workspace, size_t workspace_bytes,
                        void* stream) {
  PoolArgs A{};
  if (const int rc = check_sequences(seq, &A.S)) return rc;
  if (d < 1) return MIPS_ERR_INVALID_ARG;
  if (d > MIPS_EMBEDDING_D_MAX || (dtype != MIPS_F32 && dtype != MIPS_BF16)) return MIPS_ERR_UNSUPPORTED;
  if (const int rc = check_rows(x, A.S, d, dtype, &A.x)) return rc;
  const int E = elem_bytes(dtype);
  const bool joins = !pool_whole(A.S, d);
  if (!vectors || !mean || !norm || !aligned(vectors, E) || !aligned(mean, 4) || !aligned(norm, 4) ||
      !aligned(workspace, 256) || (joins && !workspace))
    return MIPS_ERR_INVALID_ARG;
  if (joins && workspace_bytes < pool_bytes(A.S, d)) return MIPS_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  A.d = d;
  A.lanes = pool_lanes(d);
  A.normalize = normalize != 0;
  A.chunk = pool_chunk(A.S, d);
  A.chunks = (uint32_t)(((uint64_t)A.S.n + A.chunk - 1) / A.chunk);
  A.part = (float*)workspace;
  A.vectors = vectors;
  A.mean = mean;
  A.norm = norm;
  const int64_t step = 16 / E;
  const bool vec = d % 8 == 0 && A.x.row % step == 0 && A.x.extra % step == 0 && aligned(A.x.p, 16) && aligned(vectors, 16);
  if (A.chunks) {
    const dim3 grid((A.chunks + kPoolWaves - 1) / kPoolWaves);
    if (dtype == MIPS_F32)
      hipLaunchKernelGGL((vec ? pool_kernel<float, true> : pool_kernel<float, false>), grid, dim3(kPoolThreads), 0, s, A);
    else
      hipLaunchKernelGGL((vec ? pool_kernel<__bf16, true> : pool_kernel<__bf16, false>), grid, dim3(kPoolThreads), 0, s, A);
    if (const int rc = check_launch()) return rc;
  }
  if (joins) {
    // (sequences of few parts leave most of 1024 threads idle: 4000 of 15 rows: 21 us, with 128 5)
    const bool few = A.chunks < 32u * (uint32_t)A.S.b;
    void (*join)(PoolArgs) = dtype == MIPS_F32 ? join_kernel_of<float>(few, d) : join_kernel_of<__bf16>(few, d);
    hipLaunchKernelGGL(join, dim3(A.S.b), dim3(few ? 128 : 1024), 0, s, A);
    return check_launch();
  }
  return MIPS_OK;
}

int mips_pool_normalize_backward(const mips_sequences* seq, int32_t d, int32_t dtype, const void* grad,
                                 int64_t grad_stride, int32_t normalize, const float* mean, const float* norm,
                                 void* grad_x, void* stream) {
  PoolArgs A{};
  if (const int rc = check_sequences(seq, &A.S)) return rc;
  if (d < 1 || grad_stride < d) return MIPS_ERR_INVALID_ARG;
  if (d > MIPS_EMBEDDING_D_MAX || (dtype != MIPS_F32 && dtype != MIPS_BF16)) return MIPS_ERR_UNSUPPORTED;
  const int E = elem_bytes(dtype);
  if (!grad || !mean || !norm || (A.S.n > 0 && !grad_x) || !aligned(grad, E) || !aligned(mean, 4) || !aligned(norm, 4) ||
      !aligned(grad_x, E))
    return MIPS_ERR_INVALID_ARG;
  if (A.S.n == 0) return MIPS_OK;
  A.d = d;
  A.lanes = pool_lanes(d);
  A.normalize = normalize != 0;
  A.mean = (float*)mean;
  A.norm = (float*)norm;
  A.grad = grad;
  A.grad_stride = grad_stride;
  A.dx = grad_x;
  // rows that share one row's gradient: 64 where that leaves 8192 waves (4096 x 127 x 128 bf16: 34 us with 32)
  A.chunk = A.S.n / 8192 < 4 ? 4 : (A.S.n / 8192 > 64 ? 64 : A.S.n / 8192);
  A.grad_aligned = grad_stride * E % 16 == 0 && aligned(grad, 16);
  while (A.chunk < 1024 && A.S.n / A.chunk > 65536) A.chunk *= 2;
  A.chunks = (uint32_t)(((uint64_t)A.S.n + A.chunk - 1) / A.chunk);
  const bool vec = d % 8 == 0 && aligned(grad_x, 16) && aligned(mean, 16);
  const dim3 grid((A.chunks + kPoolWaves - 1) / kPoolWaves);
  hipStream_t s = (hipStream_t)stream;
  if (dtype == MIPS_F32)
    hipLaunchKernelGGL((vec ? pool_grad_kernel<float, true> : pool_grad_kernel<float, false>), grid, dim3(kPoolThreads), 0, s, A);
  else
    hipLaunchKernelGGL((vec ? pool_grad_kernel<__bf16, true> : pool_grad_kernel<__bf16, false>), grid, dim3(kPoolThreads), 0, s, A);
  return check_launch();
}

}  // extern "C"
