// gradnorm.hip -- the global norm of a model's gradients and clipping by it (gfx950).
//
//   norm = sqrt(sum over all tensors of sum x^2),  coef = min(1, max_norm / (norm + 1e-6)),
//   x <- coef * x;  coef = 1 where max_norm is infinite.
//
// Both passes are bound by memory traffic: x is read for the norm, and read and written for
// the scaling (a set of tensors that fits the caches is read from memory once). Squares are
// summed in binary64, so that no value's square over- or underflows and the order of a sum
// hardly shows: a conversion and a fused multiply-add an element, less than half of what the
// vector units do in the time the loads take. Sums are joined in a fixed order, with no
// atomics. 1.03 GB of f32: the norm 171 us (6.0 TB/s), the scaling 341 us (6.0 TB/s read and
// written; 400 us with ordinary loads and stores: what is read or written for the last time goes past
// the caches). 48 small tensors: 5 + 5.5 us, the call is its launches.
#include "common.h"
#include "host.h"

namespace mips {

constexpr int kNormGroup = 64;      // tensors per launch (their table is a kernel argument)
constexpr int kNormChunk = 16384;   // elements a workgroup takes at a time
constexpr int kNormBlocks = 1024;   // workgroups of a launch, at most
constexpr int kNormPartials = 2048; // partial sums of a call: about this many, over all launches

struct NormTensor {
  const void* x;
  void* out;
  int64_t n;
};

struct NormArgs {
  NormTensor t[kNormGroup];
  uint32_t chunk0[kNormGroup + 1];  // first chunk of each tensor; the last entry: all chunks
  uint64_t bf16;                    // bit i: tensor i is bf16
  int nt;
  double* part;       // this launch's partial sums, one per workgroup
  const double* all;  // every launch's (scaling pass)
  int nall;
  float max_norm;
  float* norm;        // written by workgroup 0 of the first scaling launch, or NULL
};

__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, kWave);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  const double r = (red[0] + red[1]) + (red[2] + red[3]);
  __syncthreads();
  return r;
}

// The tensor of chunk c (uniform over the workgroup: the search runs on the scalar unit).
__device__ __forceinline__ int tensor_of(const NormArgs& A, uint32_t c) {
  int lo = 0, hi = A.nt - 1;
  while (lo < hi) {
    const int m = (lo + hi + 1) >> 1;
    if (A.chunk0[m] <= c) lo = m;
    else hi = m - 1;
  }
  return lo;
}

// Calls f(values, count, element index) for this thread's elements of [i0, i1) of x: 16-byte
// loads where x is aligned, four of them in flight per thread. LAST: x is not read again.
template <bool BF16, bool LAST, typename F>
__device__ __forceinline__ void for_units(const void* x, int64_t i0, int64_t i1, bool vec, F f) {
  constexpr int N = BF16 ? 8 : 4;
  constexpr int kBatch = 4;
  int64_t done = i0;
  if (vec) {
    const int64_t nv = (i1 - i0) / N;
    const u32x4_t* p = (const u32x4_t*)((const uint8_t*)x + i0 * (16 / N));
    for (int64_t b = threadIdx.x; b < nv; b += 256 * kBatch) {
      u32x4_t v[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        v[u] = b + u * 256 < nv ? (LAST ? __builtin_nontemporal_load(p + b + u * 256) : p[b + u * 256])
                                : u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (b + u * 256 >= nv) break;
        float y[N];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (BF16) {
            y[2 * e] = __uint_as_float(v[u][e] << 16);
            y[2 * e + 1] = __uint_as_float(v[u][e] & 0xFFFF0000u);
          } else {
            y[e] = __uint_as_float(v[u][e]);
          }
        }
        f(y, N, i0 + (b + u * 256) * N);
      }
    }
    done = i0 + nv * N;
  }
  for (int64_t i = done + threadIdx.x; i < i1; i += 256) {
    float y[N];
    y[0] = BF16 ? bf16_to_f32(((const uint16_t*)x)[i]) : ((const float*)x)[i];
    f(y, 1, i);
  }
}

__global__ __launch_bounds__(256) void norm_kernel(NormArgs A) {
  __shared__ double red[4];
  double s = 0.0;
  const uint32_t total = A.chunk0[A.nt];
  for (uint32_t c = blockIdx.x; c < total; c += gridDim.x) {
    const int i = tensor_of(A, c);
    const NormTensor T = A.t[i];
    const int64_t i0 = (int64_t)(c - A.chunk0[i]) * kNormChunk;
    const int64_t i1 = min(T.n, i0 + kNormChunk);
    const bool vec = ((uintptr_t)T.x & 15) == 0;
    auto add = [&](const float* y, int n, int64_t) __attribute__((always_inline)) {
      for (int e = 0; e < n; ++e) s = fma((double)y[e], (double)y[e], s);
    };
    if ((A.bf16 >> i) & 1u) for_units<true, false>(T.x, i0, i1, vec, add);
    else for_units<false, false>(T.x, i0, i1, vec, add);
  }
  s = block_sum(s, red);
  if (threadIdx.x == 0) A.part[blockIdx.x] = s;
}

// Every workgroup adds up the call's partial sums itself (at most a few thousand, from the
// caches), which costs less than a launch of one workgroup in between would. Chunks are taken
// from the last to the first: what the norm pass read last is still in the caches.
__global__ __launch_bounds__(256) void clip_kernel(NormArgs A) {
  __shared__ double red[4];
  double s = 0.0;
  for (int i = threadIdx.x; i < A.nall; i += 256) s += A.all[i];
  const double norm = sqrt(block_sum(s, red));
  // coef in binary32 as the values it scales; a NaN norm gives a NaN coef, an infinite one 0. Without
  // a bound on the norm it is 1, whatever the norm is (inf / inf would be NaN)
  const float q = isinf(A.max_norm) ? 1.0f : (float)((double)A.max_norm / (norm + 1e-6));
  const float coef = q < 1.0f ? q : (q != q ? q : 1.0f);
  if (A.norm && blockIdx.x == 0 && threadIdx.x == 0) *A.norm = (float)norm;
  const uint32_t total = A.chunk0[A.nt];
  for (uint32_t k = blockIdx.x; k < total; k += gridDim.x) {
    const uint32_t c = total - 1u - k;
    const int i = tensor_of(A, c);
    const NormTensor T = A.t[i];
    if (coef == 1.0f && T.out == T.x) continue;  // nothing to change
    const int64_t i0 = (int64_t)(c - A.chunk0[i]) * kNormChunk;
    const int64_t i1 = min(T.n, i0 + kNormChunk);
    const bool vec = (((uintptr_t)T.x | (uintptr_t)T.out) & 15) == 0;
    if ((A.bf16 >> i) & 1u) {
      for_units<true, true>(T.x, i0, i1, vec, [&](const float* y, int n, int64_t at) __attribute__((always_inline)) {
        __bf16* o = (__bf16*)T.out + at;
        if (n == 8) {
          bf16x8_t v;
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = (__bf16)(y[e] * coef);  // rounded to nearest even
          __builtin_nontemporal_store(v, (bf16x8_t*)o);
        } else {
          o[0] = (__bf16)(y[0] * coef);
        }
      });
    } else {
      for_units<false, true>(T.x, i0, i1, vec, [&](const float* y, int n, int64_t at) __attribute__((always_inline)) {
        float* o = (float*)T.out + at;
        typedef float f32x4_t __attribute__((ext_vector_type(4)));
        if (n == 4) __builtin_nontemporal_store(f32x4_t{y[0] * coef, y[1] * coef, y[2] * coef, y[3] * coef}, (f32x4_t*)o);
        else o[0] = y[0] * coef;
      });
    }
  }
}

// Workgroups of a launch: one per chunk, at most kNormBlocks, and so that all launches of the
// call together leave about kNormPartials partial sums.
static int norm_blocks(uint32_t chunks, int groups) {
  int most = kNormPartials / groups;
  most = most > kNormBlocks ? kNormBlocks : (most < 16 ? 16 : most);
  return (int)(chunks < (uint32_t)most ? chunks : (uint32_t)most);
}

}  // namespace mips

extern "C" {

size_t mips_clip_workspace_size(int32_t ntensors) {
  if (ntensors < 1) return 0;
  const size_t groups = ((size_t)ntensors + mips::kNormGroup - 1) / mips::kNormGroup;
  const size_t per = groups * 16 > mips::kNormPartials ? 16 : mips::kNormPartials / groups;
  return groups * (per < mips::kNormBlocks ? per : mips::kNormBlocks) * sizeof(double) + 256;
}

int mips_clip_grad_norm(const void* const* tensors, void* const* outs, const int64_t* counts,
                        const int32_t* dtypes, int32_t ntensors, float max_norm, float* out_norm,
                        void* workspace, size_t workspace_bytes, void* stream) {
  using namespace mips;
  if (!tensors || !outs || !counts || !dtypes || ntensors < 1 || !out_norm || !aligned(out_norm, 4) ||
      !workspace || !aligned(workspace, 256) || !(max_norm >= 0.0f))
    return MIPS_ERR_INVALID_ARG;
  for (int i = 0; i < ntensors; ++i) {
    if (dtypes[i] != MIPS_F32 && dtypes[i] != MIPS_BF16) return MIPS_ERR_UNSUPPORTED;
    if (counts[i] < 0 || counts[i] > (int64_t(1) << 38)) return MIPS_ERR_INVALID_ARG;
    const int E = elem_bytes(dtypes[i]);
    if (counts[i] > 0 && (!tensors[i] || !outs[i] || !aligned(tensors[i], E) || !aligned(outs[i], E)))
      return MIPS_ERR_INVALID_ARG;
  }
  if (workspace_bytes < mips_clip_workspace_size(ntensors)) return MIPS_ERR_WORKSPACE;
  const int groups = (ntensors + kNormGroup - 1) / kNormGroup;
  hipStream_t s = (hipStream_t)stream;
  double* part = (double*)workspace;
  int nall = 0;
  for (int pass = 0; pass < 2; ++pass) {
    for (int g = 0; g < groups; ++g) {
      // the scaling pass starts with the group that the norm pass read last
      const int gi = pass == 0 ? g : groups - 1 - g;
      NormArgs A{};
      const int i0 = gi * kNormGroup;
      A.nt = ntensors - i0 < kNormGroup ? ntensors - i0 : kNormGroup;
      uint64_t at = 0;  // at most 2^24 chunks a tensor, 2^30 a launch
      for (int i = 0; i < A.nt; ++i) {
        A.t[i] = NormTensor{tensors[i0 + i], outs[i0 + i], counts[i0 + i]};
        if (dtypes[i0 + i] == MIPS_BF16) A.bf16 |= uint64_t(1) << i;
        A.chunk0[i] = (uint32_t)at;
        at += (uint64_t)((counts[i0 + i] + kNormChunk - 1) / kNormChunk);
      }
      A.chunk0[A.nt] = (uint32_t)at;
      int nb = norm_blocks((uint32_t)at, groups);
      A.max_norm = max_norm;
      if (pass == 0) {
        if (nb < 1) nb = 1;  // empty tensors: one partial sum of zero
        A.part = part + nall;
        nall += nb;
        hipLaunchKernelGGL(norm_kernel, dim3(nb), dim3(256), 0, s, A);
      } else {
        A.all = part;
        A.nall = nall;
        A.norm = g == 0 ? out_norm : nullptr;
        const uint32_t most = 2048;
        nb = (int)(at < most ? (at < 1 ? 1 : at) : most);
        hipLaunchKernelGGL(clip_kernel, dim3(nb), dim3(256), 0, s, A);
      }
      if (const int rc = check_launch()) return rc;
    }
  }
  return MIPS_OK;
}

}  // extern "C"
