// dropout.hip -- dropout from a counter-based generator; the mask is never stored (gfx950).
//
// Eight neighbouring elements share one block of Philox4x32-10 (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011), 16 bits each. The counter is the
// elements' place and the call's offset, the key the seed, so that the gradient finds the mask again.
//
// Bound by memory: 520,192 x 128 bf16 take 44 us (6.0 TB/s), with a residual 76 (5.3); the ten rounds'
// multiplications, five an element, hide behind it.
#include "common.h"
#include "host.h"

namespace mips {

struct DropArgs {
  const void* x;
  const void* residual;  // or NULL
  void* out;
  int64_t n;
  uint64_t seed, offset;
  const uint64_t* counter;  // added to the offset, or NULL
  uint32_t cut;             // kept: 16 random bits at least this
  float scale;
};

__device__ __forceinline__ u32x4_t philox(uint64_t index, uint64_t offset, uint64_t seed) {
  uint32_t c0 = (uint32_t)index, c1 = (uint32_t)(index >> 32), c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p = (uint64_t)c0 * 0xD2511F53u, q = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(q >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)q;
    c2 = (uint32_t)(p >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)p;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4_t{c0, c1, c2, c3};
}

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__bf16 v) { return (float)v; }

template <typename T, bool VEC>
__global__ __launch_bounds__(256) void dropout_kernel(DropArgs A) {
  typedef T v8_t __attribute__((ext_vector_type(8), aligned(16)));
  const uint64_t offset = A.offset + (A.counter ? *A.counter : 0);
  const int64_t blocks = (A.n + 7) / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < blocks; i += (int64_t)gridDim.x * 256) {
    const T* x = (const T*)A.x + i * 8;
    const T* y = (const T*)A.residual + i * 8;
    T* o = (T*)A.out + i * 8;
    const bool whole = VEC && i * 8 + 8 <= A.n;
    const int live = (int)min((int64_t)8, A.n - i * 8);
    float v[8], res[8];
    if (whole) {
      const v8_t q = *(const v8_t*)x;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = widen(q[e]);
      if (A.residual) {
        const v8_t w = *(const v8_t*)y;
#pragma unroll
        for (int e = 0; e < 8; ++e) res[e] = widen(w[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = e < live ? widen(x[e]) : 0.0f;
        if (A.residual) res[e] = e < live ? widen(y[e]) : 0.0f;
      }
    }
    const u32x4_t r = philox((uint64_t)i, offset, A.seed);
    v8_t q;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t bits = (e & 1) ? r[e >> 1] >> 16 : r[e >> 1] & 0xFFFFu;
      // one rounding, of the sum: the product's own would show where the two cancel
      if (A.residual) v[e] = bits >= A.cut ? fmaf(v[e], A.scale, res[e]) : res[e];
      else v[e] = bits >= A.cut ? v[e] * A.scale : 0.0f;
      q[e] = (T)v[e];
    }
    if (whole) {
      *(v8_t*)o = q;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < live) o[e] = q[e];
    }
  }
}

}  // namespace mips

using namespace mips;

extern "C" int mips_dropout(const void* x, int32_t dtype, int64_t n, double p, uint64_t seed, uint64_t offset,
                            const uint64_t* counter, const void* residual, void* out, void* stream) {
  if (n < 0 || !(p >= 0.0 && p <= 1.0)) return MIPS_ERR_INVALID_ARG;
  if ((dtype != MIPS_F32 && dtype != MIPS_BF16) || n > int64_t(1) << 40) return MIPS_ERR_UNSUPPORTED;
  if (n == 0) return MIPS_OK;
  const int E = elem_bytes(dtype);
  if (!x || !out || !aligned(x, E) || !aligned(residual, E) || !aligned(out, E) || !aligned(counter, 8)) return MIPS_ERR_INVALID_ARG;
  DropArgs A{x, residual, out, n, seed, offset, counter, 0, 0.0f};
  A.cut = (uint32_t)(p * 65536.0 + 0.5);
  A.scale = A.cut < 65536u ? (float)(65536.0 / (65536u - A.cut)) : 0.0f;
  const bool vec = aligned(x, 16) && aligned(residual, 16) && aligned(out, 16);
  const int64_t blocks = (n + 2047) / 2048;
  const dim3 grid((uint32_t)(blocks < 8192 ? blocks : 8192));
  hipStream_t s = (hipStream_t)stream;
  if (dtype == MIPS_F32)
    hipLaunchKernelGGL((vec ? dropout_kernel<float, true> : dropout_kernel<float, false>), grid, dim3(256), 0, s, A);
  else
    hipLaunchKernelGGL((vec ? dropout_kernel<__bf16, true> : dropout_kernel<__bf16, false>), grid, dim3(256), 0, s, A);
  return check_launch();
}
