// softmax.h -- the fused score and softmax-statistics pass for gfx950; included only by
// softmax_inst.hip.
#pragma once

#include <utility>

#include "host.h"
#include "softmax_api.h"

namespace mips {

template <int N, typename F>
__device__ __forceinline__ void unroll_for(F&& f) {
  if constexpr (N > 0) {
    unroll_for<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, bytes, 0x00020000);
}

// One 16-byte chunk of both operands: a 32x32x16 bf16 product, or four 32x32x2 f32 ones.
template <int CT>
__device__ __forceinline__ void mfma_chunk(f32x16_t& acc, u32x4_t a, u32x4_t b) {
  if constexpr (CT == MIPS_BF16) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                  __builtin_bit_cast(bf16x8_t, b), acc, 0, 0, 0);
  } else {
#pragma unroll
    for (int t = 0; t < 4; ++t)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[t]), __uint_as_float(b[t]), acc, 0, 0, 0);
  }
}

// Sets the bits of the 16 rows that accumulator registers 0..15 of this lane hold: bit i is
// row 8 (i >> 2) + 4 (lane >> 5) + (i & 3) of the block's word.
__device__ __forceinline__ uint32_t lane_bits(uint32_t w, int lane) {
  const uint32_t wl = w >> (4 * (lane >> 5));
  return (wl & 0xFu) | ((wl >> 4) & 0xF0u) | ((wl >> 8) & 0xF00u) | ((wl >> 12) & 0xF000u);
}

// Per query: the running reference m, the sum of e_j = 2^(y_j - m) and the sum of
// e_j (y_j - m), y = l * log2(e), over the items of a slice.
//
// One workgroup = 8 waves (two per SIMD) = one slice of the items x one block of 32 NQF
// queries. The query block sits in LDS as MFMA operands; each wave streams its own tiles of RM
// 32-row item blocks from memory into registers, NS - 1 stages ahead, and multiplies each tile
// with every query fragment. An accumulator register holds one item's score for the lane's
// own query column (lane & 31), so the statistics of a column are per lane, with no
// exchange between lanes until the end of the slice. They live in LDS between tiles (three
// values per fragment and lane), which lets the fragment loop stay a loop: kept in registers,
// they would have to be unrolled over fragments, ring stages and both epilogues, far past
// the instruction cache.
//
// What bounds it: with few queries the items' bytes; with many its instructions. Per 32 x 32 tile
// of scores at a width of 128 in bf16, 8 products of 32 cycles and about 70 vector instructions
// (for each register half a maximum, a multiply-add, an exp2 of 8 cycles and an addition).
// Measured: 1M x 128 bf16 by 16 queries 50 us (5.1 TB/s); 10M x 128 by 50 queries 440 us
// (5.8 TB/s), 475-495 with the entropy and the run maxima and 5% excluded; 250,000 x 128 by 4096
// queries 306 us (0.86 PFLOP/s, the matrix pipes busy 45% and the vector units 58% of the cycles).
// Without the tile's maximum, testing the sums instead, the last fell to 291 us, but packed
// corpora and small batches lost more (10M x 128 by 256 queries 960 -> 1037 us).
template <int CT, int D, int NQF, bool ROWS, int MODE>
__global__ __launch_bounds__(kStatsThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void stats_kernel(
    StatsArgs A) {
  constexpr int E = elem_bytes(CT);
  constexpr int NCH = chunks_per_block(CT, D);
  constexpr int RM = stats_rm(CT, D);
  constexpr int NS = stats_ns(CT, D);
  constexpr int64_t BLK = block_bytes(CT, D);
  constexpr int QB = kFrag * NQF;
  constexpr bool ENT = MODE != STATS_LSE, BM = MODE == STATS_ALT;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // Workgroup -> (slice, query block): consecutive workgroups go to different XCDs, and the
  // query blocks of one slice share an XCD (and its L2).
  int slice, qblk;
  {
    const int w = blockIdx.x;
    if (A.nslices % 8 == 0) {
      const int xcd = w & 7, idx = w >> 3;
      slice = (idx / A.nqblk) * 8 + xcd;
      qblk = idx % A.nqblk;
    } else {
      slice = w / A.nqblk;
      qblk = w % A.nqblk;
    }
  }
  const int qbase = qblk * QB;
  const int nq = min(QB, A.b - qbase);           // live columns
  const int nfr = (nq + kFrag - 1) / kFrag;      // live fragments

  // Query tile: slot s of chunk c of fragment f holds query 32f + (s & 31), bytes
  // 32c + 16 (s >> 5) .. of its row; for a packed f32 corpus, dims 8c + 2t + (s >> 5).
  {
    u32x4_t* dst = (u32x4_t*)lds;
    for (int i = threadIdx.x; i < nfr * NCH * 64; i += kStatsThreads) {
      const int s = i & 63, c = (i >> 6) % NCH, f = (i >> 6) / NCH;
      const int q = f * kFrag + (s & 31);
      u32x4_t v = {0u, 0u, 0u, 0u};
      if (q < nq) {
        const uint8_t* row = A.queries.p + (int64_t)(qbase + q) * A.queries.stride_b;
        if constexpr (CT == MIPS_F32 && !ROWS) {
          const uint32_t* r = (const uint32_t*)row + 8 * c + (s >> 5);
#pragma unroll
          for (int t = 0; t < 4; ++t) v[t] = r[2 * t];
        } else {
          const int off = 32 * c + 16 * (s >> 5);
          if (off < A.queries.row_b) v = *(const u32x4_t*)(row + off);
        }
      }
      dst[i] = v;
    }
  }
  constexpr int SV = stats_values(MODE);
  float* st = (float*)(lds + (size_t)QB * D * E) + (size_t)wave * NQF * SV * kWave + lane;
  auto clear = [&]() __attribute__((always_inline)) {
    for (int f = 0; f < NQF; ++f) {
      st[(SV * f + 0) * kWave] = kMasked;
      st[(SV * f + 1) * kWave] = 0.0f;
      st[(SV * f + 2) * kWave] = 0.0f;
    }
  };
  clear();
  __syncthreads();
  // A logit of -inf has e = 0 and would make e t a NaN in the entropy's sum. Biases are bounded from
  // below as they are loaded, so what is left are rows of infinities: a wave that finds such a NaN at
  // its end takes its tiles again with every logit bounded, in the branch of the masks. (A call of
  // 4096 x 250,000 x 128 with the entropy: 338 us without any of this, 345 so, 363 with each tile's sum
  // tested.)
  bool bounded = false;

  // Tiles go in runs of 2^run_log consecutive ones, a wave's runs kStatsWaves apart: the run
  // is the unit of the maxima. Tile i of this wave, of `count`:
  const int run = 1 << A.run_log;
  const int64_t r_begin = (int64_t)slice * A.nruns / A.nslices, r_end = (int64_t)(slice + 1) * A.nruns / A.nslices;
  const int64_t count = (r_end - r_begin - wave + kStatsWaves - 1) / kStatsWaves * run;
  auto tile_of = [&](int64_t i) __attribute__((always_inline)) {
    return ((r_begin + wave + (i >> A.run_log) * kStatsWaves) << A.run_log) + (i & (run - 1));
  };
  const int64_t nblocks = (A.items.n + kFrag - 1) / kFrag;

  // A stage's loads are unconditional (blocks past the end read the last block again and are
  // masked out), so that the compiler's wait counts stay exact. Lane r < RM also loads the
  // exclusion word of block r.
  auto load_stage = [&](u32x4_t (&a)[RM][NCH], uint32_t& xraw, int64_t tile) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < RM; ++r) {
      const int64_t fr = min<int64_t>(tile * RM + r, nblocks - 1);
      if constexpr (ROWS) {
        const int64_t rows = min<int64_t>(kFrag, A.items.n - fr * kFrag);
        const __amdgpu_buffer_rsrc_t rs =
            rows_rsrc(A.items.p + fr * kFrag * A.items.stride_b, (int)((rows - 1) * A.items.stride_b) + A.items.row_b);
        const int base = (lane & 31) * (int)A.items.stride_b + 16 * (lane >> 5);
        const int left = A.items.row_b - 16 * (lane >> 5);  // chunks at or past the row's end read zeros
#pragma unroll
        for (int c = 0; c < NCH; ++c)
          a[r][c] = __builtin_bit_cast(
              u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, 32 * c < left ? base + 32 * c : 0x7FFFFFF0, 0, 0));
      } else {
        const __amdgpu_buffer_rsrc_t rs = rows_rsrc(A.items.p + fr * BLK, (int)BLK);
#pragma unroll
        for (int c = 0; c < NCH; ++c)
          a[r][c] = __builtin_bit_cast(
              u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, lane * 16, c * kChunkBytes, 0));
      }
    }
    const int64_t fr = min<int64_t>(tile * RM + (lane < RM ? lane : RM - 1), nblocks - 1);
    const uint32_t* wp = (A.exclude && A.exclude_words == 0) ? A.exclude + fr : (const uint32_t*)A.items.p;
    xraw = *wp;
  };

  // Operand chunks of the products to come, kLook ahead; a chunk is replaced as soon as its
  // products have been issued.
  constexpr int kLook = NCH < 8 ? NCH : (NCH == 8 ? 8 : 4);
  u32x4_t bq[kLook];
  // Behind chunk c of fragment f: its chunk c + kLook, or those of the fragment that follows.
  auto refill = [&](int c, int f, int follow) __attribute__((always_inline)) {
    const int cc = c + kLook;
    bq[c % kLook] = ((const u32x4_t*)(lds + (size_t)(cc < NCH ? f : follow) * BLK) + lane)[(cc % NCH) * 64];
  };
  auto compute_stage = [&](const u32x4_t (&a)[RM][NCH], uint32_t xraw, int64_t i_tile) __attribute__((always_inline)) {
    const int64_t tile = tile_of(i_tile);
    // words of the tile's blocks, rows past n set; uniform
    uint32_t word[RM], any = 0u;
#pragma unroll
    for (int r = 0; r < RM; ++r) {
      const int64_t left = A.items.n - (tile * RM + r) * kFrag;
      uint32_t w = (A.exclude && A.exclude_words == 0) ? (uint32_t)__builtin_amdgcn_readlane((int)xraw, r) : 0u;
      if (left < kFrag) w |= left <= 0 ? ~0u : ~0u << left;
      word[r] = w;
      any |= w;
    }
    if (ENT && bounded) any = ~0u;
    // the tile's biases: rows 8q + 4 (lane >> 5) + (0..3) for q = 0..3 (rows past n read 0 and
    // are masked); kept for all fragments where the registers allow it
    constexpr bool kKeepBias = RM == 1 && NCH <= 8;
    float bv[RM][16];
    auto load_bias = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int r = 0; r < RM; ++r) {
        const int64_t blk = min<int64_t>(tile * RM + r, nblocks - 1);
        const __amdgpu_buffer_rsrc_t rs =
            rows_rsrc(A.bias + blk * kFrag, (int)min<int64_t>(kFrag, A.items.n - blk * kFrag) * 4);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const u32x4_t v = __builtin_bit_cast(
              u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, (lane >> 5) * 16 + q * 32, 0, 0));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = __uint_as_float(v[e]);
            bv[r][4 * q + e] = ENT && x < A.vmask ? A.vmask : x;  // (one that masks, for the entropy: see bounded)
          }
        }
      }
    };
    if (kKeepBias && A.bias) load_bias();
    // One fragment: `cur` holds its scores, `nxt` receives those of the next one, whose products
    // run while this one's exponentials are taken.
    auto fragment = [&](f32x16_t (&cur)[RM], f32x16_t (&nxt)[RM], int f) __attribute__((always_inline)) {
      if (A.bias) {
        if (!kKeepBias) load_bias();
#pragma unroll
        for (int r = 0; r < RM; ++r)
#pragma unroll
          for (int i = 0; i < 16; ++i) cur[r][i] = __fadd_rn(__fmul_rn(cur[r][i], A.scale), bv[r][i]);
      }
      if (any != 0u) {
        // Register i holds row 8 (i >> 2) + (i & 3) in lanes 0-31 and that row + 4 in lanes
        // 32-63: a wave-uniform lane mask, built on the scalar unit, applied by one select.
#pragma unroll
        for (int r = 0; r < RM; ++r) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int b0 = 8 * (i >> 2) + (i & 3);
            const uint64_t lanes = (((word[r] >> b0) & 1u) ? 0x00000000FFFFFFFFull : 0ull) |
                                   (((word[r] >> (b0 + 4)) & 1u) ? 0xFFFFFFFF00000000ull : 0ull);
            cur[r][i] = __builtin_amdgcn_inverse_ballot_w64(lanes) ? A.vmask : cur[r][i];
          }
        }
        if (ENT && bounded) {
#pragma unroll
          for (int r = 0; r < RM; ++r)
#pragma unroll
            for (int i = 0; i < 16; ++i) cur[r][i] = cur[r][i] < A.vmask ? A.vmask : cur[r][i];
        }
      }
      if (A.exclude_words != 0) {  // this column's own words
        const int q = min(qbase + f * kFrag + (lane & 31), A.b - 1);
#pragma unroll
        for (int r = 0; r < RM; ++r) {
          const uint32_t bits =
              lane_bits(A.exclude[(int64_t)q * A.exclude_words + min<int64_t>(tile * RM + r, nblocks - 1)], lane);
#pragma unroll
          for (int i = 0; i < 16; ++i) cur[r][i] = ((bits >> i) & 1u) ? A.vmask : cur[r][i];
        }
      }
      float m = st[(SV * f + 0) * kWave], z = st[(SV * f + 1) * kWave], x = st[(SV * f + 2) * kWave];
      float vm = cur[0][0];
#pragma unroll
      for (int r = 0; r < RM; ++r)
#pragma unroll
        for (int i = 0; i < 16; ++i) vm = fmaxf(vm, cur[r][i]);
      if constexpr (BM) {
        const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(vm), __float_as_uint(vm), false, false);
        const float v2 = fmaxf(__uint_as_float(sw[0]), __uint_as_float(sw[1]));  // both halves' rows
        // the run's maximum so far, stored behind its last tile
        const int in_run = (int)(i_tile & (run - 1));
        const float v3 = in_run == 0 ? v2 : fmaxf(v2, st[(SV * f + 3) * kWave]);
        st[(SV * f + 3) * kWave] = v3;
        const float l0 = A.bias ? v3 : v3 * A.scale, l = l0 > kLeastLogit ? l0 : -INFINITY;
        // the store is unconditional, out of the buffer's range where nothing is to be stored (the
        // upper lanes, the earlier tiles): one that may or may not be issued makes the compiler's
        // wait counts for the item loads behind it inexact
        const __amdgpu_buffer_rsrc_t rs = rows_rsrc(
            A.bmax + ((int64_t)(qbase / kFrag + f) * A.nruns + (tile >> A.run_log)) * kFrag, kFrag * 4);
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(l), rs, in_run == run - 1 ? lane * 4 : 1024, 0, 0);
      }
      const float mn = vm * A.scx;
      if (__builtin_expect(__ballot(mn > m + kSlack) != 0ull, 0)) {
        if (mn > m) {
          const float g = __builtin_amdgcn_exp2f(m - mn);
          // (a sum over masked values alone is dropped here, infinite or not; NaN came from an eligible
          // item, in a tile that held nothing else, and stays)
          const float kept = z == z ? 0.0f : z;
          x = g > 0.0f ? g * (x - (mn - m) * z) : kept;
          z = g > 0.0f ? g * z : kept;
          m = mn;
        }
      }
      // Each chunk's products for the next fragment (after the last one: of the first again, unused,
      // which cost nothing beside the exponentials; a branch would part the two), then its share of
      // this one's exponentials. The barriers keep the compiler from parting the two again.
      float z0 = 0.0f, z1 = 0.0f, x0 = 0.0f, x1 = 0.0f;
      const int g = f + 1 < nfr ? f + 1 : 0, follow = f + 2 < nfr ? f + 2 : 0;
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        if constexpr (NQF > 1) {
#pragma unroll
          for (int r = 0; r < RM; ++r) {
            if (c == 0) nxt[r] = f32x16_t{};
            mfma_chunk<CT>(nxt[r], a[r][c], bq[c % kLook]);
          }
          refill(c, g, follow);
        }
#pragma unroll
        for (int k = c * 16 * RM / NCH; k < (c + 1) * 16 * RM / NCH; ++k) {
          const float t = fmaf(cur[k >> 4][k & 15], A.scx, -m);
          float e = __builtin_amdgcn_exp2f(t);
          if constexpr (NQF > 1) asm volatile("" : "+v"(e));  // computed here, under these products
          if (k & 1) {
            z1 += e;
            if constexpr (ENT) x1 = fmaf(e, t, x1);
          } else {
            z0 += e;
            if constexpr (ENT) x0 = fmaf(e, t, x0);
          }
        }
        if constexpr (NQF > 1) __builtin_amdgcn_sched_barrier(0);
      }
      st[(SV * f + 0) * kWave] = m;
      st[(SV * f + 1) * kWave] = z + (z0 + z1);
      if constexpr (ENT) st[(SV * f + 2) * kWave] = x + (x0 + x1);
    };
    f32x16_t acc0[RM], acc1[RM];
#pragma unroll
    for (int r = 0; r < RM; ++r) acc0[r] = f32x16_t{};
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
#pragma unroll
      for (int r = 0; r < RM; ++r) mfma_chunk<CT>(acc0[r], a[r][c], bq[c % kLook]);
      refill(c, 0, nfr > 1 ? 1 : 0);
    }
    if constexpr (NQF > 1) {
      for (int f = 0; f < nfr; f += 2) {
        fragment(acc0, acc1, f);
        if (f + 1 < nfr) fragment(acc1, acc0, f + 1);
      }
    } else {
      fragment(acc0, acc1, 0);
    }
  };

  u32x4_t a[NS][RM][NCH];
  uint32_t xw[NS];
  while (count > 0) {
    int64_t i = 0;
#pragma unroll
    for (int c = 0; c < kLook; ++c) bq[c] = ((const u32x4_t*)lds + lane)[c * 64];
    unroll_for<NS - 1>([&](auto uc) __attribute__((always_inline)) {
      constexpr int u = decltype(uc)::value;
      load_stage(a[u], xw[u], tile_of(i + u));
    });
    auto step = [&](auto uc) __attribute__((always_inline)) {
      constexpr int u = decltype(uc)::value;
      constexpr int ld = (u + NS - 1) % NS;
      load_stage(a[ld], xw[ld], tile_of(i + u + NS - 1));
      compute_stage(a[u], xw[u], i + u);
      return i + u + 1 >= count;
    };
    if constexpr (NS == 3) {
      while (!(step(std::integral_constant<int, 0>{}) || step(std::integral_constant<int, 1>{}) ||
               step(std::integral_constant<int, 2>{})))
        i += NS;
    } else {
      while (!(step(std::integral_constant<int, 0>{}) || step(std::integral_constant<int, 1>{})))
        i += NS;
    }
    if (!ENT || bounded) break;
    for (int f = 0; f < nfr; ++f) {
      const float z = st[(SV * f + 1) * kWave], x = st[(SV * f + 2) * kWave];
      bounded |= __ballot(x != x && z == z) != 0ull;
    }
    if (!bounded) break;
    clear();
  }
  __syncthreads();

  // The column's statistics over the 8 waves and the two halves of each.
  const float* all = (const float*)(lds + (size_t)QB * D * E);
  for (int q = threadIdx.x; q < nq; q += kStatsThreads) {
    const int f = q / kFrag, l = q % kFrag;
    auto at = [&](int w, int k) { return all[((w >> 1) * NQF * SV + SV * f + k) * kWave + l + 32 * (w & 1)]; };
    float m = kMasked;
    for (int w = 0; w < 2 * kStatsWaves; ++w) m = fmaxf(m, at(w, 0));
    float z = 0.0f, x = 0.0f;
    for (int w = 0; w < 2 * kStatsWaves; ++w) {
      const float mw = at(w, 0), zw = at(w, 1), g = __builtin_amdgcn_exp2f(mw - m);
      if (mw > kEmpty) {
        z = fmaf(g, zw, z);
        x = fmaf(g, at(w, 2) + (mw - m) * zw, x);
      } else if (zw != zw) {
        z = zw;  // only NaN was seen
      }
    }
    A.part[(int64_t)slice * A.b + qbase + q] = make_float4(m, z, x, 0.0f);
  }
}

template <int CT, int D, int NQF, bool ROWS, int MODE>
static int launch_stats_two(const StatsArgs& A, int grid, hipStream_t s) {
  constexpr int lds = stats_lds(CT, D, NQF, MODE);
  static const hipError_t attr = hipFuncSetAttribute((const void*)stats_kernel<CT, D, NQF, ROWS, MODE>,
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  (void)attr;
  hipLaunchKernelGGL((stats_kernel<CT, D, NQF, ROWS, MODE>), dim3(grid), dim3(kStatsThreads), lds, s, A);
  return check_launch();
}

template <int CT, int D, int NQF, bool ROWS>
static int launch_stats_one(const StatsArgs& A, int grid, hipStream_t s) {
  if (A.bmax) return launch_stats_two<CT, D, NQF, ROWS, STATS_ALT>(A, grid, s);
  return A.ent ? launch_stats_two<CT, D, NQF, ROWS, STATS_ENT>(A, grid, s)
               : launch_stats_two<CT, D, NQF, ROWS, STATS_LSE>(A, grid, s);
}

template <int CT, int D>
int launch_stats(int nqf, bool rows, const StatsArgs& A, int grid, hipStream_t s) {
  switch (nqf) {
    case 1: return rows ? launch_stats_one<CT, D, 1, true>(A, grid, s) : launch_stats_one<CT, D, 1, false>(A, grid, s);
    case 2: return rows ? launch_stats_one<CT, D, 2, true>(A, grid, s) : launch_stats_one<CT, D, 2, false>(A, grid, s);
    case 4: return rows ? launch_stats_one<CT, D, 4, true>(A, grid, s) : launch_stats_one<CT, D, 4, false>(A, grid, s);
    case 8:
      if constexpr (stats_fits(CT, D, 8))
        return rows ? launch_stats_one<CT, D, 8, true>(A, grid, s) : launch_stats_one<CT, D, 8, false>(A, grid, s);
      break;
  }
  return MIPS_ERR_UNSUPPORTED;
}

}  // namespace mips
