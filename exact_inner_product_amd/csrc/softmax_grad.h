// softmax_grad.h -- the backward pass of the softmax over an item table for gfx950; included
// only by softmax_inst.hip.
//
// With p_bj = exp(l_bj - lse_b), g the gradients of the targets' log probabilities and h_b that
// of the entropy,
//   w_bj = sum_i g_bi [id_bi = j] - p_bj (sum_i g_bi + h_b (log p_bj + H_b))
//   dq_b = scale sum_j w_bj c_j,   dc_j = scale sum_b w_bj q_b,   dbias_j = sum_b w_bj.
// Both sums are one kernel with the roles changed: it owns rows X (items for dc, queries for
// dq), streams rows Y, computes a tile of scores, turns them into weights in registers and
// multiplies the weights with Y again. The scores are computed once for each sum, and never
// written.
#pragma once

#include "host.h"
#include "softmax.h"
#include "softmax_api.h"

namespace mips {

typedef short i16x4_t __attribute__((ext_vector_type(4)));

// Streamed rows in LDS: 16-byte slot s of row j is kept at slot s ^ swz(j). Eight consecutive
// rows' equal slots (the operand of the scores, one row a lane) then lie in eight different
// 16-byte columns, and four consecutive rows' equal slot pairs (the transposed read of the
// second product) in four different 32-byte ones: both read without bank conflicts.
__device__ __forceinline__ int swz(int j) { return ((j & 3) << 1) | ((j >> 2) & 1); }

// One workgroup = grad_waves waves of 32 own rows each, one split of the streamed rows. A wave
// holds its rows as MFMA operands in registers, and the 32 x D sums. Per 32 streamed rows:
//  1. scores, transposed: the streamed rows as the first operand, the own rows as the second,
//     so that a lane holds 16 scores of its own row (column lane & 31);
//  2. weights, in place;
//  3. sums += weights x streamed rows. The accumulator layout of step 1 is an operand layout of
//     step 3 with the streamed rows in another order, so the weights stay in their lanes; the
//     other operand takes the streamed rows in the same order, transposed by the LDS read
//     (bf16), or element by element (f32).
// In bf16 the weights are rounded to bf16 for step 3, to nearest: an independent relative error
// of at most 2^-8 each, under sums that are rounded to bf16 themselves. Sums are in binary32.
//
// Tiles of 64 streamed rows are double-buffered: the next tile's rows are loaded to registers
// before this tile's products and stored to the other buffer after them, with one barrier a
// tile.
template <int CT, int D, bool ITEMS, bool EXTRA>
__global__ __launch_bounds__(64 * grad_waves(CT, D))
__attribute__((amdgpu_waves_per_eu(grad_waves(CT, D) / 4, grad_waves(CT, D) / 4))) void grad_kernel(GradArgs A) {
  constexpr int E = elem_bytes(CT);
  constexpr int NCH = chunks_per_block(CT, D);  // 32-byte steps of a row
  constexpr int NT = 64 * grad_waves(CT, D);
  constexpr int RB = grad_row_bytes(CT, D);
  constexpr int SL = RB / 16;                   // slots of a row in LDS
  constexpr int NLD = kGradTile * SL / NT;      // slots each thread moves per tile
  constexpr int DT = (D + 31) / 32;             // 32-column tiles of the sums
  constexpr int JB = kGradTile / 32;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  // [2] tiles | [2][64] lse2 or bias | [2][64] coef | [2][64] hent | [2][64] words | [2][64][g] targets
  float* va = (float*)(lds + 2 * kGradTile * RB);
  float* vb = va + 2 * kGradTile;
  float* vc = vb + 2 * kGradTile;
  int32_t* vt = (int32_t*)(vc + 2 * kGradTile + 2 * kGradTile);

  const int lane = threadIdx.x & 63, h = lane >> 5, col = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // Workgroup -> (split, own tile): the own tiles of one split share an XCD, and its L2 the
  // streamed rows, where there are enough splits; else the other way round it makes no
  // difference.
  int split, tile_own;
  {
    const int w = blockIdx.x;
    if (A.nsplit % 8 == 0) {
      const int xcd = w & 7, idx = w >> 3;
      split = (idx / A.nown) * 8 + xcd;
      tile_own = idx % A.nown;
    } else {
      split = w / A.nown;
      tile_own = w % A.nown;
    }
  }
  const int64_t own0 = (int64_t)tile_own * grad_own(CT, D) + wave * 32;
  const int64_t own = own0 + col;                       // this lane's own row
  const bool live = own < A.own.n;
  const int64_t own_c = live ? own : A.own.n - 1;

  u32x4_t x[NCH];  // own rows: lane (col, h) holds bytes 32c + 16h .. of row col
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int off = 32 * c + 16 * h;
    x[c] = u32x4_t{0u, 0u, 0u, 0u};
    if (live && off < A.own.row_b) x[c] = *(const u32x4_t*)(A.own.p + own_c * A.own.stride_b + off);
  }
  f32x16_t sum[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) sum[d] = f32x16_t{};
  float dbias = 0.0f;

  // the lane's own terms
  float my_lse2 = 1e30f, my_coef = 0.0f, my_hent = 0.0f, my_bias = 0.0f;
  if constexpr (!ITEMS) {
    my_lse2 = A.q.lse2[own_c];
    my_coef = live ? A.q.coef[own_c] : 0.0f;
    if (EXTRA) my_hent = live ? A.q.hent[own_c] : 0.0f;
  } else if (EXTRA) {
    if (A.bias) my_bias = A.bias[own_c];
  }

  const int64_t t_begin = (int64_t)split * A.ntiles / A.nsplit, t_end = (int64_t)(split + 1) * A.ntiles / A.nsplit;

  // ---- staging
  u32x4_t ld[NLD];
  float la = 0.0f, lb = 0.0f, lc = 0.0f;
  int32_t lt = -1;
  uint32_t lw[NLD];
  const bool shared_mask = A.exclude != nullptr && A.exclude_words == 0;
  auto stage_load = [&](int64_t tile) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NLD; ++i) {
      const int e = i * NT + threadIdx.x, j = e / SL, s = e % SL;
      const int64_t r = tile * kGradTile + j;
      ld[i] = u32x4_t{0u, 0u, 0u, 0u};
      if (r < A.str.n && 16 * s < A.str.row_b) ld[i] = *(const u32x4_t*)(A.str.p + r * A.str.stride_b + 16 * s);
      if (!ITEMS && EXTRA && shared_mask) lw[i] = r < A.str.n ? A.exclude[r >> 5] : 0u;
    }
    if (threadIdx.x < kGradTile) {
      const int64_t r = tile * kGradTile + threadIdx.x;
      if constexpr (ITEMS) {  // padded arrays: every row of a tile has its terms
        la = A.q.lse2[r];
        lb = A.q.coef[r];
        if (EXTRA) lc = A.q.hent[r];
      } else if (EXTRA) {
        la = A.bias && r < A.str.n ? A.bias[r] : 0.0f;
      }
    }
    if constexpr (ITEMS) {
      if ((int)threadIdx.x < kGradTile * A.q.g) lt = A.q.tgt[tile * kGradTile * A.q.g + threadIdx.x];
    }
  };
  auto stage_store = [&](int64_t tile, int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NLD; ++i) {
      const int e = i * NT + threadIdx.x, j = e / SL, s = e % SL;
      u32x4_t v = ld[i];
      // an excluded item's row may hold anything: it takes no part in the sums
      if (!ITEMS && EXTRA && shared_mask && ((lw[i] >> (j & 31)) & 1u)) v = u32x4_t{0u, 0u, 0u, 0u};
      *(u32x4_t*)(lds + (size_t)buf * kGradTile * RB + j * RB + ((s ^ (swz(j) & (SL - 1))) << 4)) = v;
    }
    if (threadIdx.x < kGradTile) {
      if (ITEMS || EXTRA) va[buf * kGradTile + threadIdx.x] = la;
      if (ITEMS) vb[buf * kGradTile + threadIdx.x] = lb;
      if (ITEMS && EXTRA) vc[buf * kGradTile + threadIdx.x] = lc;
    }
    if constexpr (ITEMS) {
      if ((int)threadIdx.x < kGradTile * A.q.g) vt[buf * kGradTile * A.q.g + threadIdx.x] = lt;
      for (int i = NT + threadIdx.x; i < kGradTile * A.q.g; i += NT)
        vt[buf * kGradTile * A.q.g + i] = A.q.tgt[tile * kGradTile * A.q.g + i];
    }
  };

  // lane-constant parts of the LDS addresses
  int sbase[4];  // scores: slot 2c + h of row col, for c = 0..3 (mod 4)
#pragma unroll
  for (int c = 0; c < 4; ++c) sbase[c] = col * RB + (((2 * c + h) ^ swz(col)) << 4);
  const int tl = lane & 15, tg = (lane >> 4) & 1;
  int tbase[2];  // transposed reads: row 4h + (tl >> 2), columns 16 tg + 4 (tl & 3) of an even or odd column tile
#pragma unroll
  for (int o = 0; o < 2; ++o)
    tbase[o] = (4 * h + (tl >> 2)) * RB + (((4 * o + 2 * tg + ((tl & 3) >> 1)) ^ (((tl >> 2) << 1) | h)) << 4) + 8 * (tl & 1);

  auto compute = [&](int64_t tile, int buf) __attribute__((always_inline)) {
    const uint8_t* y = lds + (size_t)buf * kGradTile * RB;
#pragma unroll 1
    for (int jb = 0; jb < JB; ++jb) {
      // masks: bit i of `bits` <=> register i's pair takes no part
      uint32_t bits = 0u;
      bool masked = false;  // uniform
      if constexpr (!ITEMS) {
        const int64_t left = A.str.n - (tile * kGradTile + jb * 32);
        uint32_t w = 0u;
        if (left < 32) w = left <= 0 ? ~0u : ~0u << left;
        if (EXTRA && A.exclude && left > 0) {
          const int64_t blk = tile * JB + jb;
          if (A.exclude_words == 0) {
            w |= (uint32_t)__builtin_amdgcn_readfirstlane((int)A.exclude[blk]);
            masked = w != 0u;
          } else {
            w |= A.exclude[own_c * A.exclude_words + blk];
            masked = true;
          }
        } else {
          masked = w != 0u;
        }
        if (masked) bits = lane_bits(w, lane);
      } else if (EXTRA) {
        if (A.exclude && A.exclude_words != 0) {  // each query's own word of this wave's block of items
          masked = true;
          const int64_t blk = min(own0, A.own.n - 1) >> 5;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int64_t r = min<int64_t>(tile * kGradTile + jb * 32 + acc_row(i, lane), A.str.n - 1);
            bits |= ((A.exclude[r * A.exclude_words + blk] >> col) & 1u) << i;
          }
        }
      }

      f32x16_t s = {};
#pragma unroll
      for (int c = 0; c < NCH; ++c)
        mfma_chunk<CT>(s, *(const u32x4_t*)(y + jb * 32 * RB + sbase[c & 3] + (c >> 2) * 128), x[c]);

      // weights
      float w[16];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int at = buf * kGradTile + jb * 32 + 8 * q + 4 * h;  // registers 4q .. 4q + 3
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = a, c = a;
        if (ITEMS || (EXTRA && A.bias)) a = *(const float4*)(va + at);
        if (ITEMS) b = *(const float4*)(vb + at);
        if (ITEMS && EXTRA) c = *(const float4*)(vc + at);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 4 * q + e;
          const float ae = e == 0 ? a.x : (e == 1 ? a.y : (e == 2 ? a.z : a.w));
          const float be = e == 0 ? b.x : (e == 1 ? b.y : (e == 2 ? b.z : b.w));
          const float ce = e == 0 ? c.x : (e == 1 ? c.y : (e == 2 ? c.z : c.w));
          const float lse2 = ITEMS ? ae : my_lse2;
          float v = s[i];
          if (EXTRA && A.bias) v = __fadd_rn(__fmul_rn(v, A.scale), ITEMS ? my_bias : ae);
          const float t = fmaf(v, A.scx, -lse2);
          const float p = __builtin_amdgcn_exp2f(t);
          float k = ITEMS ? be : my_coef;
          if (EXTRA && A.use_hent) k += (p > 0.0f ? t : 0.0f) * (ITEMS ? ce : my_hent);
          w[i] = p * k;
        }
      }
      if (masked) {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = ((bits >> i) & 1u) ? 0.0f : w[i];
      }
      if constexpr (ITEMS) {
        // targets among this wave's items: rare, so one ballot a target column
        for (int g = 0; g < A.q.g; ++g) {
          const int32_t tgt = vt[(buf * kGradTile + jb * 32 + col) * A.q.g + g];
          if (__ballot(tgt >= own0 && tgt < own0 + 32) != 0ull) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int j = jb * 32 + acc_row(i, lane);
              if (vt[(buf * kGradTile + j) * A.q.g + g] == (int32_t)own)
                w[i] += A.q.gval[(tile * kGradTile + j) * A.q.g + g];
            }
          }
        }
        if (EXTRA && A.bias_part) {
#pragma unroll
          for (int i = 0; i < 16; ++i) dbias += w[i];
        }
      }

      // sums += w^T Y
      if constexpr (CT == MIPS_BF16) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          bf16x8_t wa;
#pragma unroll
          for (int e = 0; e < 8; ++e) wa[e] = (__bf16)w[8 * kb + e];
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            typedef __attribute__((address_space(3))) i16x4_t lds_i16x4;
            const uint8_t* p = y + (jb * 32 + 16 * kb) * RB + tbase[d & 1] + (d >> 1) * 128;
            const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p);
            const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + 8 * RB));
            const bf16x8_t yb = __builtin_bit_cast(
                bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            sum[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wa, yb, sum[d], 0, 0, 0);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = jb * 32 + 8 * (i >> 2) + (i & 3);  // + 4h: swz of row j + 4h is swz(j) ^ h
          const uint8_t* row = y + (j + 4 * h) * RB;
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            const int slot = (8 * d + (col >> 2)) ^ (swz(j) ^ h);
            sum[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(w[i], *(const float*)(row + (slot << 4) + 4 * (col & 3)),
                                                          sum[d], 0, 0, 0);
          }
        }
      }
    }
  };

  if (t_begin < t_end) {
    stage_load(t_begin);
    stage_store(t_begin, 0);
    __syncthreads();
    int buf = 0;
    for (int64_t t = t_begin; t < t_end; ++t) {
      const bool more = t + 1 < t_end;
      if (more) stage_load(t + 1);
      compute(t, buf);
      if (more) stage_store(t + 1, buf ^ 1);
      __syncthreads();
      buf ^= 1;
    }
  }

  // rows acc_row(i, lane) of the wave's tile, column 32 d + col
  const int d_live = A.own.row_b / E;
  uint32_t dead = 0u;  // excluded items have no gradient
  if (ITEMS && EXTRA && shared_mask && own0 < A.own.n) dead = A.exclude[own0 >> 5];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = acc_row(i, lane);
    const int64_t row = own0 + r;
    if (row >= A.own.n) continue;
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const int c = 32 * d + col;
      if (c >= d_live) continue;
      const float v = ((dead >> r) & 1u) ? 0.0f : sum[d][i];
      if (A.nsplit > 1 || !ITEMS)
        A.part[((int64_t)split * A.own.n + row) * d_live + c] = v;
      else if (A.out == nullptr)
        continue;  // only the bias' gradient was asked for
      else if (CT == MIPS_F32)
        ((float*)A.out)[row * d_live + c] = v * A.scale;
      else
        ((__bf16*)A.out)[row * d_live + c] = (__bf16)(v * A.scale);
    }
  }
  if constexpr (ITEMS && EXTRA) {
    if (A.bias_part) {
      dbias += __shfl_xor(dbias, 32, kWave);
      if (h == 0 && live) A.bias_part[(int64_t)split * A.own.n + own] = ((dead >> col) & 1u) ? 0.0f : dbias;
    }
  }
}

template <int CT, int D, bool ITEMS, bool EXTRA>
static int launch_grad_one(const GradArgs& A, hipStream_t s) {
  static const hipError_t attr = hipFuncSetAttribute((const void*)grad_kernel<CT, D, ITEMS, EXTRA>,
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
  (void)attr;
  hipLaunchKernelGGL((grad_kernel<CT, D, ITEMS, EXTRA>), dim3((unsigned)(A.nown * A.nsplit)),
                     dim3(64 * grad_waves(CT, D)), grad_lds(CT, D, ITEMS ? A.q.g : 0), s, A);
  return check_launch();
}

template <int CT, int D>
int launch_grad(bool items, bool extra, const GradArgs& A, hipStream_t s) {
  if (items) return extra ? launch_grad_one<CT, D, true, true>(A, s) : launch_grad_one<CT, D, true, false>(A, s);
  return extra ? launch_grad_one<CT, D, false, true>(A, s) : launch_grad_one<CT, D, false, false>(A, s);
}

}  // namespace mips
