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

// Lane l of four neighbours gives v[0..3] of column l and gets columns 0..3 of v[l]. All lanes of the
// wave take part.
__device__ __forceinline__ void quad_transpose(float (&v)[4], int lane) {
  auto from = [](float x, auto perm) __attribute__((always_inline)) {
    constexpr int ctrl = decltype(perm)::value;
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), ctrl, 0xF, 0xF, true));
  };
  constexpr std::integral_constant<int, 0xB1> next{};  // of lane l ^ 1
  constexpr std::integral_constant<int, 0x4E> over{};  // of lane l ^ 2
  const bool odd = lane & 1, high = lane & 2;
#pragma unroll
  for (int e = 0; e < 4; e += 2) {  // rows e and e + 1: columns of this lane and the next
    const float got = from(odd ? v[e] : v[e + 1], next);
    const float a = odd ? got : v[e], b = odd ? v[e + 1] : got;
    v[e] = a, v[e + 1] = b;
  }
  const float g0 = from(high ? v[0] : v[2], over), g1 = from(high ? v[1] : v[3], over);
  const float a = high ? v[2] : v[0], b = high ? v[3] : v[1];
  v[0] = high ? g0 : a, v[1] = high ? g1 : b;
  v[2] = high ? a : g0, v[3] = high ? b : g1;
}

// Streamed rows in LDS: 16-byte slot s of row j is kept at slot s ^ swz(j). Eight consecutive
// rows' equal slots (the operand of the scores, one row a lane) then lie in eight different
// 16-byte columns, and four consecutive rows' equal slot pairs (the transposed read of the
// second product) in four different 32-byte ones: both read at 128 bytes a cycle, half of what LDS
// can do. Four swizzle bits reach all of it (64 of 145 LDS cycles per 32 x 32 block gone), but need
// more address arithmetic, and the pass, bound by its matrix and vector instructions, was no
// faster: 592 + 491 us against 583 + 486 (items + queries, 4096 x 250,000 x 128).
__device__ __forceinline__ int swz(int j) { return ((j & 3) << 1) | ((j >> 2) & 1); }

// One workgroup = grad_waves waves of 32 own rows each, one split of the streamed rows. A wave
// holds its rows as MFMA operands in registers, and the 32 x D sums. Per 32 streamed rows:
//  1. scores, transposed: the streamed rows as the first operand, the own rows as the second,
//     so that a lane holds 16 scores of its own row (column lane & 31). The streamed rows'
//     addends come in as one more chunk, split into three bf16 parts (24 bits): read from LDS
//     per row instead, they would take four 16-byte reads a lane, as much as half of all
//     operand reads, and the pass was bound by LDS with them;
//  2. weights, in place: a fused multiply-add, an exp2 and half a conversion a score;
//  3. sums += weights x streamed rows. The accumulator layout of step 1 is an operand layout of
//     step 3 with the streamed rows in another order, so the weights stay in their lanes; the
//     other operand takes the streamed rows in the same order, transposed by the LDS read
//     (bf16), or element by element (f32).
// In bf16 the weights are rounded to bf16 for step 3, to nearest: an independent relative error
// of at most 2^-8 each, under sums that are rounded to bf16 themselves. The targets' weights g - p G
// are not: with nearly all of the probability a target has a weight of nearly 0, of which the rounding
// of p G leaves nothing, and with little its weight is most of its item's gradient, whose error the
// rounding would double. So step 3 takes - p G of a target as of any other row, and g and what the
// rounding left are added as one more product in binary32, of one row each (4096 targets among
// 250,000 items: 0.4% of the blocks hold one). Sums are in binary32.
//
// What bounds it: matrix and vector instructions together, which share a SIMD's issue. Per 32 x 32
// block of a width of 128 in bf16, 17 products of 32 cycles and about 70 vector instructions, 16 of
// them exp2 (8 cycles each): at 4096 x 250,000 x 128 the queries' pass takes 485 us (1.08 PFLOP/s of
// its two products) with the matrix pipes busy 54% and the vector units 41% of the cycles; the items'
// pass 568 us (45% and 38%; it also looks for signs, and for targets by their ids). In f32 the products
// bound it (32 x 32 x 2, 64 cycles each). A small batch is latency: 1000 x 1000 x 64 in f32 takes
// 14 + 13.5 us, 4096 x 8192 x 128 in bf16 34 + 34 us, of which targets are about a tenth (12% of the
// blocks hold one).
//
// Step 1 of the next 32 rows is interleaved with step 2 of these, chunk by chunk, so that the
// matrix pipe works under the exponentials. Tiles of 64 streamed rows go through three LDS
// buffers: the tile after the next is on its way from memory, the next is written at the start
// of a tile, and one barrier in the middle of the tile makes it readable before its first
// scores are due at the end.
template <int CT, int D, bool ITEMS, bool EXTRA>
__global__ __launch_bounds__(64 * grad_waves(CT, D))
__attribute__((amdgpu_waves_per_eu(grad_wps(CT, D), grad_wps(CT, D)))) void grad_kernel(GradArgs A) {
  constexpr int E = elem_bytes(CT);
  constexpr int NCH = chunks_per_block(CT, D);  // 32-byte steps of a row
  constexpr int NT = 64 * grad_waves(CT, D);
  constexpr int RB = grad_row_bytes(CT, D);
  constexpr int SL = RB / 16;                   // slots of a row in LDS
  constexpr int NLD = kGradTile * SL / NT;      // slots each thread moves per tile
  constexpr int DT = (D + 31) / 32;             // 32-column tiles of the sums
  constexpr int kLook = NCH < 4 ? NCH : 4;      // operand chunks read ahead
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  // per buffer: rows | addend chunks | coef | hent | signs | targets
  uint8_t* vadd = lds + kGradBufs * kGradTile * RB;
  float* vcoef = (float*)(vadd + kGradBufs * kGradTile * 16);
  float* vhent = vcoef + kGradBufs * kGradTile;
  uint32_t* vneg = (uint32_t*)(vhent + kGradBufs * kGradTile);  // [3][2], 16 words kept
  int32_t* vtgt = (int32_t*)(vneg + 16);

  const int lane = threadIdx.x & 63, h = lane >> 5, col = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // Workgroup -> (split, own tile): consecutive workgroups go to different XCDs; the own tiles
  // of one split share an XCD, and its L2 the streamed rows, where the splits allow it.
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
  // the addend chunk's partner: ones for its three parts (f32: for its one), in the first half
  const u32x4_t ones = h != 0 ? u32x4_t{0u, 0u, 0u, 0u}
                              : (CT == MIPS_BF16 ? u32x4_t{0x3F803F80u, 0x00003F80u, 0u, 0u}
                                                 : u32x4_t{0x3F800000u, 0u, 0u, 0u});
  f32x16_t sum[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) sum[d] = f32x16_t{};
  float dbias = 0.0f;

  // the lane's own terms
  const float masked_add = kMasked * A.inv_scx;
  float my_add = 0.0f, my_coef = 0.0f, my_hent = 0.0f;
  bool flip = false;  // this query's sums are of -w: its coefficient is negative (plain)
  if constexpr (!ITEMS) {
    my_add = live ? A.q.add[own_c] : kMasked;
    if (!EXTRA) flip = (A.q.neg[own_c >> 5] >> (own_c & 31)) & 1u;
    if (EXTRA) my_coef = live ? A.q.coef[own_c] : 0.0f;
    if (EXTRA) my_hent = live ? A.q.hent[own_c] : 0.0f;
  } else {
    if (A.bias) my_add = A.bias[own_c] * kLog2e;
  }

  const int64_t t_begin = (int64_t)split * A.ntiles / A.nsplit, t_end = (int64_t)(split + 1) * A.ntiles / A.nsplit;

  // Queries' pass: the next target of the lane's query with its gradient, and the one after it, which
  // is on its way when it is needed. Targets and blocks come in the rows' order, so that one comparison
  // a block finds the few that hold a target.
  int32_t target = kNoTarget, target2 = kNoTarget;
  float target_grad = 0.0f, target_grad2 = 0.0f;
  int64_t target_at = own_c * A.q.g, target_end = target_at + A.q.g;  // of the one after
  auto next_target = [&]() __attribute__((always_inline)) {
    target = target2, target_grad = target_grad2, target2 = kNoTarget;
    if (++target_at < target_end) {
      target2 = A.q.tgt[target_at];
      target_grad2 = flip ? -A.q.gval[target_at] : A.q.gval[target_at];
    }
  };
  if (!ITEMS && live) {
    int passed = 0;
#pragma unroll 8
    for (int g = 0; g < A.q.g; ++g) passed += A.q.tgt[own_c * A.q.g + g] < t_begin * kGradTile ? 1 : 0;
    target_at += passed - 1;
    next_target();
    next_target();
  }

  // ---- staging
  u32x4_t ld[NLD];
  float la = 0.0f, lb = 0.0f, lc = 0.0f;
  int32_t lt = kNoTarget;
  uint32_t lw[NLD], law = 0u, ln = 0u;
  const bool shared_mask = A.exclude != nullptr && A.exclude_words == 0;
  auto stage_load = [&](int64_t tile) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NLD; ++i) {
      const int e = i * NT + threadIdx.x, j = e / SL, s = e % SL;
      // Padding queries, of weight 0, hold the last one's row: zeros would make NaN of the score
      // with an item's row of infinities.
      const int64_t r = ITEMS ? min((int)tile * kGradTile + j, (int)A.str.n - 1) : tile * kGradTile + j;
      ld[i] = u32x4_t{0u, 0u, 0u, 0u};
      if ((ITEMS || r < A.str.n) && 16 * s < A.str.row_b) ld[i] = *(const u32x4_t*)(A.str.p + r * A.str.stride_b + 16 * s);
      if (!ITEMS && shared_mask) lw[i] = r < A.str.n ? A.exclude[r >> 5] : 0u;
    }
    if (threadIdx.x < kGradTile) {
      const int64_t r = tile * kGradTile + threadIdx.x;
      if constexpr (ITEMS) {  // padded arrays: every row of a tile has its terms
        la = A.q.add[r] * A.inv_scx;
        if (EXTRA) lb = A.q.coef[r];
        if (EXTRA) lc = A.q.hent[r];
      } else {
        la = r >= A.str.n ? masked_add : (A.bias ? A.bias[r] * kLog2e * A.inv_scx : 0.0f);
        // a bias that masks its item (-inf, the lowest float) stays finite: -inf would make NaN of
        // its parts and of its product with the zeros beside the ones (a NaN bias stays NaN)
        la = la < masked_add ? masked_add : la;
        law = shared_mask && r < A.str.n ? A.exclude[r >> 5] >> (r & 31) : 0u;
      }
    }
    if constexpr (ITEMS) {
      if ((int)threadIdx.x < kGradTile * A.q.g) lt = A.q.tgt[tile * kGradTile * A.q.g + threadIdx.x];
      if (!EXTRA && threadIdx.x < kGradTile / 32) ln = A.q.neg[tile * (kGradTile / 32) + threadIdx.x];
    }
  };
  auto stage_store = [&](int64_t tile, int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NLD; ++i) {
      const int e = i * NT + threadIdx.x, j = e / SL, s = e % SL;
      u32x4_t v = ld[i];
      // an excluded item's row may hold anything: it takes no part in the sums
      if (!ITEMS && shared_mask && ((lw[i] >> (j & 31)) & 1u)) v = u32x4_t{0u, 0u, 0u, 0u};
      *(u32x4_t*)(lds + (size_t)buf * kGradTile * RB + j * RB + ((s ^ (swz(j) & (SL - 1))) << 4)) = v;
    }
    if (threadIdx.x < kGradTile) {
      const float a = (!ITEMS && (law & 1u)) ? masked_add : la;
      u32x4_t v = {__float_as_uint(a), 0u, 0u, 0u};
      if constexpr (CT == MIPS_BF16) {
        const __bf16 p0 = (__bf16)a, p1 = (__bf16)(a - (float)p0), p2 = (__bf16)(a - (float)p0 - (float)p1);
        v = u32x4_t{(uint32_t)__builtin_bit_cast(uint16_t, p0) | ((uint32_t)__builtin_bit_cast(uint16_t, p1) << 16),
                    (uint32_t)__builtin_bit_cast(uint16_t, p2), 0u, 0u};
      }
      *(u32x4_t*)(vadd + (buf * kGradTile + threadIdx.x) * 16) = v;
      if (ITEMS && EXTRA) {
        vcoef[buf * kGradTile + threadIdx.x] = lb;
        vhent[buf * kGradTile + threadIdx.x] = lc;
      }
    }
    if constexpr (ITEMS) {
      if (!EXTRA && threadIdx.x < kGradTile / 32) vneg[buf * (kGradTile / 32) + threadIdx.x] = ln;
      if ((int)threadIdx.x < kGradTile * A.q.g) vtgt[buf * kGradTile * A.q.g + threadIdx.x] = lt;
      for (int i = NT + threadIdx.x; i < kGradTile * A.q.g; i += NT)
        vtgt[buf * kGradTile * A.q.g + i] = A.q.tgt[tile * kGradTile * A.q.g + i];
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

  // Operand chunks of a block's scores: chunk NCH is the addends'.
  u32x4_t yq[kLook];
  auto read_chunk = [&](int buf, int jb, int c) __attribute__((always_inline)) {
    if (c == NCH) return *(const u32x4_t*)(vadd + (buf * kGradTile + jb * 32 + col) * 16);
    return *(const u32x4_t*)(lds + (size_t)buf * kGradTile * RB + jb * 32 * RB + sbase[c & 3] + (c >> 2) * 128);
  };
  auto read_first = [&](int buf, int jb) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < kLook; ++c) yq[c] = read_chunk(buf, jb, c);
  };
  // Chunk c's products for block jb, and the read of chunk c + kLook.
  auto score_chunk = [&](f32x16_t& s, int buf, int jb, int c) __attribute__((always_inline)) {
    if (c == 0) s = f32x16_t{};
    if (c < NCH) {
      mfma_chunk<CT>(s, yq[c % kLook], x[c < NCH ? c : 0]);
    } else if constexpr (CT == MIPS_BF16) {
      mfma_chunk<CT>(s, yq[c % kLook], ones);
    } else {
      s = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(yq[c % kLook][0]), __uint_as_float(ones[0]), s, 0, 0, 0);
    }
    if (c + kLook <= NCH) yq[c % kLook] = read_chunk(buf, jb, c + kLook);
  };

  // Steps 2 and 3 of block jb of tile `tile` (buffer buf), whose scores are in `s`, with step 1
  // of block nj of buffer nbuf into `nxt` between; then `between`, the first chunk reads of the
  // block after that, and the sums.
  auto block = [&](f32x16_t& s, f32x16_t& nxt, int64_t tile, int buf, int jb, int nbuf, int nj,
                   auto between) __attribute__((always_inline)) {
    uint32_t bits = 0u;  // bit i: register i's pair takes no part
    if constexpr (EXTRA) {
      if (A.exclude && A.exclude_words != 0) {
        if constexpr (!ITEMS) {  // this query's own word of the block of items
          if (tile * kGradTile + jb * 32 < A.str.n)
            bits = lane_bits(A.exclude[own_c * A.exclude_words + tile * (kGradTile / 32) + jb], lane);
        } else {                 // each query's own word of this wave's block of items
          const int64_t blk = min(own0, A.own.n - 1) >> 5;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int64_t r = min<int64_t>(tile * kGradTile + jb * 32 + acc_row(i, lane), A.str.n - 1);
            bits |= ((A.exclude[r * A.exclude_words + blk] >> col) & 1u) << i;
          }
        }
      }
    }
    // the block's first targets and signs, read ahead of the products
    int32_t tgt0 = kNoTarget;
    uint32_t negw = 0u;
    if constexpr (ITEMS) {
      if (A.q.g > 0) tgt0 = vtgt[(buf * kGradTile + jb * 32 + col) * A.q.g];
      if (!EXTRA) negw = vneg[buf * (kGradTile / 32) + jb];
    }
    float w[16];
    float ck[16], hk[16];
    if constexpr (EXTRA && ITEMS) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // registers 4q .. 4q + 3: rows 8q + 4h ..
        const float4 a = *(const float4*)(vcoef + buf * kGradTile + jb * 32 + 8 * q + 4 * h);
        const float4 b = *(const float4*)(vhent + buf * kGradTile + jb * 32 + 8 * q + 4 * h);
        ck[4 * q] = a.x, ck[4 * q + 1] = a.y, ck[4 * q + 2] = a.z, ck[4 * q + 3] = a.w;
        hk[4 * q] = b.x, hk[4 * q + 1] = b.y, hk[4 * q + 2] = b.z, hk[4 * q + 3] = b.w;
      }
    }
#pragma unroll
    for (int c = 0; c <= NCH; ++c) {
      score_chunk(nxt, nbuf, nj, c);
#pragma unroll
      for (int i = c * 16 / (NCH + 1); i < (c + 1) * 16 / (NCH + 1); ++i) {
        const float t = fmaf(s[i], A.scx, my_add);
        w[i] = __builtin_amdgcn_exp2f(t);
        if constexpr (EXTRA) {
          // 0 log 0 = 0: log2 p of a masked item may be -inf, but below -126 its p is 0
          const float k = fmaf(fmaxf(t, -200.0f), ITEMS ? hk[i] : my_hent, ITEMS ? ck[i] : my_coef);
          w[i] = ((bits >> i) & 1u) ? 0.0f : w[i] * k;
        }
        asm volatile("" : "+v"(w[i]));  // computed here, under these products
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // the streamed rows as the sums' operand: lane (column, h) holds rows 4h + (0..3) and
    // 8 + 4h + (0..3) of half kb; the first half's are read ahead of what comes between
    const uint8_t* y = lds + (size_t)buf * kGradTile * RB + jb * 32 * RB;
    auto read_columns = [&](int kb, int d) __attribute__((always_inline)) {
      typedef __attribute__((address_space(3))) i16x4_t lds_i16x4;
      const uint8_t* p = y + 16 * kb * RB + tbase[d & 1] + (d >> 1) * 128;
      const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p);
      const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + 8 * RB));
      return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    constexpr int kAhead = CT == MIPS_BF16 ? (DT < 4 ? DT : 4) : 1;
    bf16x8_t ahead[kAhead];
    if constexpr (CT == MIPS_BF16) {
#pragma unroll
      for (int d = 0; d < kAhead; ++d) ahead[d] = read_columns(0, d);
    }
    // A target, own row `own_r` and streamed row `str_r` of the block (both uniform): its gradient v
    // and, in bf16, what the rounding of its weight will leave go to the sums as a multiple of the
    // streamed row, in binary32. The weight is register 4 (str_r >> 3) + (str_r & 3) of lane own_r of
    // half (str_r >> 2) & 1, the sums' row the register of the same form of own_r, in one half's lanes.
    auto add_target = [&](int own_r, int str_r, float v) __attribute__((always_inline)) {
      const int at = 4 * (str_r >> 3) + (str_r & 3), holder = own_r + 32 * ((str_r >> 2) & 1);
      if constexpr (CT == MIPS_BF16) {
        float x = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) x = i == at ? w[i] : x;
        const float rounded = (float)(__bf16)x;
        v += __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x - rounded), holder));
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = i == at && lane == holder ? rounded : w[i];  // (an id given twice)
      }
      float row[DT];
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const int byte = (32 * d + col) * E;
        const uint8_t* q = y + str_r * RB + (((byte >> 4) ^ (swz(str_r) & (SL - 1))) << 4) + (byte & 15);
        if constexpr (CT == MIPS_BF16) row[d] = bf16_to_f32(*(const uint16_t*)q);
        else row[d] = *(const float*)q;
      }
      const float k = own_r == lane ? v : 0.0f;
#pragma unroll
      for (int d = 0; d < DT; ++d) sum[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(k, row[d], sum[d], 0, 0, 0);
    };
    if constexpr (ITEMS) {
      if constexpr (!EXTRA) {
        // the queries whose coefficient is negative (none, or all, in most losses)
        const uint32_t neg = (uint32_t)__builtin_amdgcn_readfirstlane((int)negw);
        if (neg != 0u) {
          const uint32_t nb = lane_bits(neg, lane);
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = ((nb >> i) & 1u) ? -w[i] : w[i];
        }
      }
      if (EXTRA && A.bias_part) {
#pragma unroll
        for (int i = 0; i < 16; ++i) dbias += w[i];
      }
      // targets among this wave's items: rare, so one ballot a target column, and the pairs it
      // finds one by one
      for (int g = 0; g < A.q.g; ++g) {
        const int32_t tgt = g == 0 ? tgt0 : vtgt[(buf * kGradTile + jb * 32 + col) * A.q.g + g];
        uint32_t hits = (uint32_t)__ballot(tgt >= own0 && tgt < own0 + 32);
        while (hits != 0u) {
          const int j = __builtin_ctz(hits);
          hits &= hits - 1u;
          const int r = __builtin_amdgcn_readlane(tgt, j) - (int)own0;
          const float v = A.q.gval[(tile * kGradTile + jb * 32 + j) * A.q.g + g];
          add_target(r, j, v);
          if (EXTRA && A.bias_part) dbias += lane == r ? v : 0.0f;
        }
      }
    } else {
      // targets of this wave's queries among the block's items, as rare
      const int32_t first = (int32_t)(tile * kGradTile) + jb * 32;
      uint32_t hits = (uint32_t)__ballot(target < first + 32);
      while (hits != 0u) {
        const int r = __builtin_ctz(hits);
        const int j = __builtin_amdgcn_readlane(target, r) - first;
        add_target(r, j, __int_as_float(__builtin_amdgcn_readlane(__float_as_int(target_grad), r)));
        if (col == r) next_target();
        hits = (uint32_t)__ballot(target < first + 32);
      }
    }
    between();
    // sums += w^T Y
    if constexpr (CT == MIPS_BF16) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        bf16x8_t wa;
#pragma unroll
        for (int e = 0; e < 8; ++e) wa[e] = (__bf16)w[8 * kb + e];
#pragma unroll
        for (int d = 0; d < DT; ++d)
          sum[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              wa, kb == 0 && d < kAhead ? ahead[d < kAhead ? d : 0] : read_columns(kb, d), sum[d], 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int j = 8 * (i >> 2) + (i & 3);  // + 4h: swz of row j + 4h is swz(j) ^ h
        const uint8_t* row = y + (j + 4 * h) * RB;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const int slot = (8 * d + (col >> 2)) ^ (swz(j) ^ h);
          sum[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(w[i], *(const float*)(row + (slot << 4) + 4 * (col & 3)),
                                                        sum[d], 0, 0, 0);
        }
      }
    }
  };

  static_assert(kGradTile == 64 && kGradBufs == 3, "the loop below takes two blocks a tile, three buffers");
  if (t_begin < t_end) {
    f32x16_t s0, s1;
    stage_load(t_begin);
    stage_store(t_begin, 0);
    if (t_begin + 1 < t_end) stage_load(t_begin + 1);
    __syncthreads();
    read_first(0, 0);
#pragma unroll
    for (int c = 0; c <= NCH; ++c) score_chunk(s0, 0, 0, c);
    read_first(0, 1);
    int buf = 0;
    for (int64_t t = t_begin; t < t_end; ++t) {
      const int nbuf = buf == 2 ? 0 : buf + 1;
      // (written last two tiles ago and read until one tile ago: everybody has passed the
      // barrier of the last tile since)
      if (t + 1 < t_end) stage_store(t + 1, nbuf);
      if (t + 2 < t_end) stage_load(t + 2);
      block(s0, s1, t, buf, 0, buf, 1, [&]() __attribute__((always_inline)) {
        __syncthreads();  // the next tile is readable
        read_first(nbuf, 0);
      });
      // (after the last tile: scores of what the buffer holds, unused)
      block(s1, s0, t, buf, 1, nbuf, 0, [&]() __attribute__((always_inline)) { read_first(nbuf, 1); });
      buf = nbuf;
    }
  }

  // A lane holds rows acc_row(i, lane) of column 32 d + col. Four registers of four neighbouring
  // lanes are transposed, so that lane l stores four columns of row l & 3 at once (items' pass of
  // 452 x 860,000 x 16: 177 us, with a store per column 206).
  const int d_live = A.own.row_b / E;
  uint32_t dead = 0u;  // excluded items have no gradient
  if (ITEMS && shared_mask && own0 < A.own.n) dead = A.exclude[own0 >> 5];
  const bool direct = ITEMS && A.nsplit == 1;
  if (!direct || A.out != nullptr) {  // (else only the bias' gradient was asked for)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = 8 * q + 4 * h + (col & 3);
      const int64_t row = own0 + r;
      const bool none = (dead >> r) & 1u;
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const int c = 32 * d + (col & ~3);
        const bool on = row < A.own.n && c < d_live;
        float v[4] = {sum[d][4 * q], sum[d][4 * q + 1], sum[d][4 * q + 2], sum[d][4 * q + 3]};
        quad_transpose(v, lane);
        if (!on) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = none ? 0.0f : v[e];
        if (!direct) {
          *(float4*)(A.part + ((int64_t)split * A.own.n + row) * d_live + c) = make_float4(v[0], v[1], v[2], v[3]);
        } else if constexpr (CT == MIPS_F32) {
          typedef float f32x4_t __attribute__((ext_vector_type(4)));
          __builtin_nontemporal_store(f32x4_t{v[0] * A.scale, v[1] * A.scale, v[2] * A.scale, v[3] * A.scale},
                                      (f32x4_t*)((float*)A.out + row * d_live + c));
        } else {
          typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
          __builtin_nontemporal_store(bf16x4_t{(__bf16)(v[0] * A.scale), (__bf16)(v[1] * A.scale),
                                               (__bf16)(v[2] * A.scale), (__bf16)(v[3] * A.scale)},
                                      (bf16x4_t*)((__bf16*)A.out + row * d_live + c));
        }
      }
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
