// logprobs_grad.hip -- the gradient of mips_logprobs (gfx950): the entry point, the terms of
// each query and the joining of split sums, around the passes of softmax_grad.h.
#include "host.h"
#include "softmax_api.h"

namespace mips {

struct TermsArgs {
  const float *lse, *entropy, *grad_logprobs, *grad_entropy;
  const void* ids;
  int id_bits, b, bpad, g;
  int64_t n;
  const uint32_t* exclude;
  int64_t exclude_words;
  int extra;             // see QueryTerms
  float *add, *coef, *hent, *sign, *gval;
  uint32_t* neg;
  int32_t* tgt;
};

// The target of query b at ids[at] and its gradient. One outside [0, n) is padding, and an excluded
// one, or any of a query that is left without an item, has a constant log probability: none of them has
// a gradient.
__device__ __forceinline__ int32_t read_target(const TermsArgs& A, int b, int64_t at, float& v) {
  v = 0.0f;
  if (b >= A.b || A.lse[b] == -INFINITY) return kNoTarget;
  const int64_t id = A.id_bits == 32 ? (int64_t)((const int32_t*)A.ids)[at] : ((const int64_t*)A.ids)[at];
  if (id < 0 || id >= A.n) return kNoTarget;
  if (A.exclude && ((A.exclude[(int64_t)b * A.exclude_words + (id >> 5)] >> (id & 31)) & 1u)) return kNoTarget;
  v = A.grad_logprobs[at];
  return (int32_t)id;
}

// Query b's terms, given the sum of its targets' gradients.
__device__ __forceinline__ float write_terms(const TermsArgs& A, int b, float sum) {
  float add = kMasked, coef = 0.0f, hent = 0.0f;
  if (b < A.b && A.lse[b] != -INFINITY) {
    coef = -sum;
    if (A.grad_entropy) {
      const float h = A.grad_entropy[b];
      coef = -fmaf(h, A.entropy[b], sum);
      hent = -h * kLn2;
    }
    add = -A.lse[b] * kLog2e;
    if (!A.extra) add = coef == 0.0f ? kMasked : add + log2f(fabsf(coef));
  }
  A.add[b] = add;
  A.coef[b] = coef;
  A.hent[b] = hent;
  A.sign[b] = coef < 0.0f ? -1.0f : 1.0f;
  return coef;
}

// The terms of QueryTerms (bound by launch and latency: 4 us for 4096 queries). With one target at
// most, a thread a query, 64 of them a wave.
__global__ __launch_bounds__(256) void terms_kernel(TermsArgs A) {
  const int b = blockIdx.x * 256 + threadIdx.x;
  if (b >= A.bpad) return;
  float v = 0.0f;
  if (A.g > 0) {
    A.tgt[b] = read_target(A, b, b, v);
    A.gval[b] = v;
  }
  const float coef = write_terms(A, b, v);
  const uint64_t neg = __ballot(coef < 0.0f);  // (bpad is a multiple of 64: whole waves get here)
  if ((threadIdx.x & 31) == 0) A.neg[b >> 5] = (uint32_t)(neg >> (threadIdx.x & 32));
}

// With more, a lane a target: a wave sorts a query's targets by their ranks, for the queries' pass to
// walk through (4096 queries of 8 targets: 5.8 us). A workgroup takes 32 queries, so that it has a
// whole word of signs.
constexpr int kSortedThreads = 1024;
__global__ __launch_bounds__(kSortedThreads) void sorted_terms_kernel(TermsArgs A) {
  __shared__ int negative[kFrag];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int i = wave; i < kFrag; i += kSortedThreads / kWave) {
    const int b = blockIdx.x * kFrag + i;
    const int64_t at = (int64_t)b * A.g;
    float v = 0.0f;
    const int32_t t = lane < A.g ? read_target(A, b, at + lane, v) : kNoTarget;
    int rank = 0;
    for (int j = 0; j < A.g; ++j) {
      const int32_t o = __builtin_amdgcn_readlane(t, j);
      rank += o < t || (o == t && j < lane) ? 1 : 0;
    }
    if (lane < A.g) {
      A.tgt[at + rank] = t;
      A.gval[at + rank] = v;
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, kWave);
    if (lane == 0) negative[i] = write_terms(A, b, v) < 0.0f;
  }
  __syncthreads();
  const uint32_t neg = (uint32_t)__ballot(lane < kFrag && negative[lane % kFrag]);
  if (threadIdx.x == 0) A.neg[blockIdx.x] = neg;
}
static_assert(MIPS_TARGETS_MAX <= kWave, "a lane for each target of a query");

struct JoinArgs {
  const float* part;  // [nsplit][rows][d]
  int nsplit;
  int64_t rows;
  int d;
  float scale;
  const float* sign;  // a factor per row, or NULL
  void* out;          // [rows, d]
  int ways_log;       // 2^ways_log threads share four columns of a row
};

// Four columns of a row: the splits' sums, the scale and the one rounding to
// the operands' type. Way w of the threads that share them adds splits w, w + ways, ..; the ways are
// joined in a fixed order in LDS. Of many splits it is bound by the latency of the loads: 256
// splits of 160 x 128 sums take 23.8 us by one way, 14.0, 9.4 and 8.0 by 2, 4 and 8 (and 8.0 by 16);
// of few by their bytes, whatever the ways: 16 of 4096 x 128, 33 MB, 5.7 us.
template <int DT>
__global__ __launch_bounds__(256) void join_rows_kernel(JoinArgs A) {
  __shared__ float4 red[256];
  const int per = A.d / 4, ways = 1 << A.ways_log, wide = 256 >> A.ways_log;
  const int t = threadIdx.x, way = t >> (8 - A.ways_log), e = t & (wide - 1);
  const int64_t i = (int64_t)blockIdx.x * wide + e;
  const bool on = i < A.rows * per;
  const int64_t row = on ? i / per : 0;
  const int c = on ? (int)(i % per) * 4 : 0;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int s = on ? way : A.nsplit; s < A.nsplit; s += ways) {
    const float4 p = *(const float4*)(A.part + ((int64_t)s * A.rows + row) * A.d + c);
    v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
  }
  red[t] = v;
  __syncthreads();
  if (way != 0 || !on) return;
  for (int w = 1; w < ways; ++w) {
    const float4 p = red[w * wide + e];
    v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
  }
  if (A.sign) {
    const float k = A.sign[row];
    v.x *= k, v.y *= k, v.z *= k, v.w *= k;
  }
  v.x *= A.scale, v.y *= A.scale, v.z *= A.scale, v.w *= A.scale;
  if (DT == MIPS_F32) {
    *(float4*)((float*)A.out + row * A.d + c) = v;
  } else {
    __bf16* o = (__bf16*)A.out + row * A.d + c;
    typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
    *(bf16x4_t*)o = bf16x4_t{(__bf16)v.x, (__bf16)v.y, (__bf16)v.z, (__bf16)v.w};
  }
}

__global__ __launch_bounds__(256) void join_bias_kernel(const float* part, int nsplit, int64_t n, float* out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float v = 0.0f;
  for (int s = 0; s < nsplit; ++s) v += part[(int64_t)s * n + i];
  out[i] = v;
}

// ------------------------------------------------------------------------- the host side
static int grad_width(int dtype, int d) {
  for (int w = 32; w <= (dtype == MIPS_F32 ? 128 : 256); w *= 2)
    if (d <= w) return w;
  return 0;
}

struct SplitPlan {
  int nown, nsplit;
  int64_t ntiles;
};

// Splits of the streamed rows: the number that minimises rounds of workgroups times tiles of a
// split, plus the traffic of the partial sums it takes. Rates as measured for one workgroup's products
// (bf16 4e12, f32 0.3e12 flop/s) and for the partial rows' write and read (4e12 bytes/s): they
// only weigh the two against each other. Both passes of a call with fixed splits, in microseconds:
// 4096 x 8192 x 128 bf16, items' pass in 1, 2, 4, 8: 193, 140, 115, 107 (8 chosen), queries'
// in 8, 16, 32: 113, 107, 118 (16); 1000 x 1000 x 64 f32, items' in 1, 4, 8, 16: 131, 68, 57, 54 (16);
// 4096 x 250,000 x 128 bf16, items' in 1, 2: 1398, 1483 (1), queries' in 8, 16: 1613, 1398 (16).
constexpr int kMostSplits = 512;  // a workgroup for each place of the chip, for a single own tile
static SplitPlan split_plan(int dtype, int width, int d, int64_t own, int64_t streamed, bool direct) {
  SplitPlan P{};
  const int per = grad_own(dtype, width);
  P.nown = (int)((own + per - 1) / per);
  P.ntiles = (streamed + kGradTile - 1) / kGradTile;
  const double tile_s = 4.0 * kGradTile * per * width / (dtype == MIPS_BF16 ? 4e12 : 0.3e12);
  const double part_s = 8.0 * (double)own * d / 4e12;
  const int cus = device_cu_count() * grad_per_unit(dtype, width);
  double best = 1e30;
  P.nsplit = 1;
  // (with four rounds or more the last one's idle units cost little: no split)
  const int most = P.nown >= 4 * cus ? 1 : kMostSplits;
  for (int s = 1; s <= most && s <= P.ntiles; ++s) {
    const int64_t rounds = ((int64_t)P.nown * s + cus - 1) / cus;
    const double t = (double)rounds * (double)((P.ntiles + s - 1) / s) * tile_s + (s > 1 || !direct ? s * part_s : 0.0);
    if (t < best) {
      best = t;
      P.nsplit = s;
    }
  }
  return P;
}

struct BackwardPlan {
  int width, bpad;
  SplitPlan q, i;
  size_t add, coef, hent, sign, neg, gval, tgt, part, bias_part, bytes;
};

static BackwardPlan backward_plan(int b, int64_t n, int d, int dtype, int g) {
  BackwardPlan P{};
  P.width = grad_width(dtype, d);
  P.bpad = (b + kGradTile - 1) / kGradTile * kGradTile;
  P.q = split_plan(dtype, P.width, d, b, n, false);
  P.i = split_plan(dtype, P.width, d, n, b, true);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t p = at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  P.add = take((size_t)P.bpad * 4);
  P.coef = take((size_t)P.bpad * 4);
  P.hent = take((size_t)P.bpad * 4);
  P.sign = take((size_t)P.bpad * 4);
  P.neg = take((size_t)P.bpad / 8);
  P.gval = take((size_t)P.bpad * g * 4);
  P.tgt = take((size_t)P.bpad * g * 4);
  // the two passes run one after the other and share the partial sums' room
  const size_t pq = (size_t)P.q.nsplit * b * d * 4, pi = P.i.nsplit > 1 ? (size_t)P.i.nsplit * n * d * 4 : 0;
  P.part = take(pq > pi ? pq : pi);
  P.bias_part = take((size_t)P.i.nsplit * n * 4);
  P.bytes = at;
  return P;
}

static int grad_dispatch(int dtype, int width, bool items, bool extra, const GradArgs& A, hipStream_t s) {
  if (dtype == MIPS_F32) {
    switch (width) {
      case 32: return launch_grad<MIPS_F32, 32>(items, extra, A, s);
      case 64: return launch_grad<MIPS_F32, 64>(items, extra, A, s);
      case 128: return launch_grad<MIPS_F32, 128>(items, extra, A, s);
    }
  } else {
    switch (width) {
      case 32: return launch_grad<MIPS_BF16, 32>(items, extra, A, s);
      case 64: return launch_grad<MIPS_BF16, 64>(items, extra, A, s);
      case 128: return launch_grad<MIPS_BF16, 128>(items, extra, A, s);
      case 256: return launch_grad<MIPS_BF16, 256>(items, extra, A, s);
    }
  }
  return MIPS_ERR_UNSUPPORTED;
}

static int launch_join(JoinArgs J, int dtype, hipStream_t s) {
  J.ways_log = 0;
  while (J.ways_log < 3 && 32 << J.ways_log <= J.nsplit) ++J.ways_log;  // at least 16 splits a way
  const int64_t work = J.rows * (J.d / 4), wide = 256 >> J.ways_log;
  const dim3 grid((unsigned)((work + wide - 1) / wide));
  if (dtype == MIPS_F32) hipLaunchKernelGGL(join_rows_kernel<MIPS_F32>, grid, dim3(256), 0, s, J);
  else hipLaunchKernelGGL(join_rows_kernel<MIPS_BF16>, grid, dim3(256), 0, s, J);
  return check_launch();
}

static int backward_sizes(int b, int64_t n, int d, int dtype, int g) {
  if (b < 1 || n < 1 || d < 1 || g < 0) return MIPS_ERR_INVALID_ARG;
  if (dtype != MIPS_F32 && dtype != MIPS_BF16) return MIPS_ERR_UNSUPPORTED;
  if (n > (int64_t(1) << 30) || b > MIPS_B_MAX || g > MIPS_TARGETS_MAX) return MIPS_ERR_UNSUPPORTED;
  if (grad_width(dtype, d) == 0 || (d * elem_bytes(dtype)) % 16 != 0) return MIPS_ERR_UNSUPPORTED;
  return MIPS_OK;
}

static bool grad_rows_ok(const void* p, int64_t stride, int d, int dtype) {
  return aligned(p, 16) && stride >= d && (stride * elem_bytes(dtype)) % 16 == 0 && stride <= (int64_t(1) << 31);
}

}  // namespace mips

extern "C" {

size_t mips_logprobs_backward_workspace_size(int32_t b, int64_t n, int32_t d, int32_t dtype, int32_t g) {
  using namespace mips;
  return backward_sizes(b, n, d, dtype, g) == MIPS_OK ? backward_plan(b, n, d, dtype, g).bytes : 0;
}

int mips_logprobs_backward(const void* queries, int64_t query_stride, int32_t b, const void* items,
                           int64_t item_stride, int64_t n, int32_t d, int32_t dtype,
                           const float* bias, const uint32_t* exclude, int64_t exclude_row_words,
                           float scale, const void* ids, int32_t id_bits, int32_t g,
                           const float* lse, const float* entropy, const float* grad_logprobs,
                           const float* grad_entropy, void* grad_queries, void* grad_items,
                           float* grad_bias, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace mips;
  if (const int rc = backward_sizes(b, n, d, dtype, g)) return rc;
  if (!(scale >= MIPS_SCALE_MIN && scale <= MIPS_SCALE_MAX)) return MIPS_ERR_INVALID_ARG;
  if (g > 0 && id_bits != 32 && id_bits != 64) return MIPS_ERR_UNSUPPORTED;
  if (!queries || !items || !lse || !workspace || (g > 0 && (!ids || !grad_logprobs)) || (grad_entropy && !entropy) ||
      (!grad_queries && !grad_items && !grad_bias))
    return MIPS_ERR_INVALID_ARG;
  if (!grad_rows_ok(queries, query_stride, d, dtype) || !grad_rows_ok(items, item_stride, d, dtype) ||
      (grad_queries && !aligned(grad_queries, 16)) || (grad_items && !aligned(grad_items, 16)) ||
      !aligned(workspace, 256))
    return MIPS_ERR_INVALID_ARG;
  if (exclude_row_words < 0 || (exclude_row_words > 0 && (!exclude || exclude_row_words < (n + 31) / 32)))
    return MIPS_ERR_INVALID_ARG;
  if ((g > 0 && !aligned(ids, id_bits / 8)) || (bias && !aligned(bias, 4)) || (exclude && !aligned(exclude, 4)) ||
      !aligned(lse, 4) || (entropy && !aligned(entropy, 4)) || (grad_logprobs && !aligned(grad_logprobs, 4)) ||
      (grad_entropy && !aligned(grad_entropy, 4)) || (grad_bias && !aligned(grad_bias, 4)))
    return MIPS_ERR_INVALID_ARG;
  const BackwardPlan P = backward_plan(b, n, d, dtype, g);
  if (workspace_bytes < P.bytes) return MIPS_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  uint8_t* ws = (uint8_t*)workspace;
  const int E = elem_bytes(dtype);

  const bool extra = grad_entropy || grad_bias || exclude_row_words > 0;
  TermsArgs T{lse, entropy, grad_logprobs, grad_entropy, ids, id_bits, b, P.bpad, g, n, exclude, exclude_row_words,
              extra, (float*)(ws + P.add), (float*)(ws + P.coef), (float*)(ws + P.hent), (float*)(ws + P.sign),
              (float*)(ws + P.gval), (uint32_t*)(ws + P.neg), (int32_t*)(ws + P.tgt)};
  if (g <= 1) hipLaunchKernelGGL(terms_kernel, dim3((P.bpad + 255) / 256), dim3(256), 0, s, T);
  else hipLaunchKernelGGL(sorted_terms_kernel, dim3(P.bpad / kFrag), dim3(kSortedThreads), 0, s, T);
  if (const int rc = check_launch()) return rc;

  const Table tq{(const uint8_t*)queries, query_stride * E, b, d * E};
  const Table ti{(const uint8_t*)items, item_stride * E, n, d * E};
  GradArgs A{};
  A.q = QueryTerms{T.add, T.coef, T.hent, T.neg, T.tgt, T.gval, g};
  A.bias = bias;
  A.exclude = exclude;
  A.exclude_words = exclude_row_words;
  A.scale = scale;
  A.scx = scale * kLog2e;
  A.inv_scx = 1.0f / A.scx;

  if (grad_items || grad_bias) {
    A.own = ti;
    A.str = tq;
    A.nown = P.i.nown;
    A.nsplit = P.i.nsplit;
    A.ntiles = P.i.ntiles;
    A.out = grad_items;
    A.part = (float*)(ws + P.part);
    A.bias_part = grad_bias ? (float*)(ws + P.bias_part) : nullptr;
    if (const int rc = grad_dispatch(dtype, P.width, true, extra, A, s)) return rc;
    if (grad_items && P.i.nsplit > 1) {
      const JoinArgs J{A.part, P.i.nsplit, n, d, scale, nullptr, grad_items, 0};
      if (const int rc = launch_join(J, dtype, s)) return rc;
    }
    if (grad_bias) {
      hipLaunchKernelGGL(join_bias_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, A.bias_part, P.i.nsplit,
                         n, grad_bias);
      if (const int rc = check_launch()) return rc;
    }
  }
  if (grad_queries) {
    A.own = tq;
    A.str = ti;
    A.nown = P.q.nown;
    A.nsplit = P.q.nsplit;
    A.ntiles = P.q.ntiles;
    A.out = nullptr;
    A.part = (float*)(ws + P.part);
    A.bias_part = nullptr;
    if (const int rc = grad_dispatch(dtype, P.width, false, extra, A, s)) return rc;
    const JoinArgs J{A.part, P.q.nsplit, b, d, scale, extra ? nullptr : T.sign, grad_queries, 0};
    if (const int rc = launch_join(J, dtype, s)) return rc;
  }
  return MIPS_OK;
}

}  // extern "C"
