// softmax_api.h -- softmax over an item table: shared constants, operand loads and argument
// blocks of its kernels, and the launchers that each per-(type, width) translation unit
// instantiates.
//
// With s_bj = q_b . c_j accumulated in binary32, a logit is
//   l_bj = fl(fl(s_bj * scale) + bias_j)          (no bias: fl(s_bj * scale))
// and every kernel works with p_bj = exp(l_bj - lse_b), lse_b = log sum_j exp(l_bj) over the
// eligible items j.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"

namespace mips {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// Masked logits are a large negative finite value (in log2 units), so that the running sums
// need no special case: exp2 of it is 0 and 0 times it is 0. A maximum at or below kEmpty means
// that no eligible item has been seen; what was summed until then is dropped.
constexpr float kMasked = -1e30f;
constexpr float kEmpty = -0.9e30f;
// The same bound for a logit. One that is not above it (NaN and -inf among them) is no alternative:
// in a run's maximum and in the row's own key alike, so that what is listed does not depend on
// which rows happen to be scored again.
constexpr float kLeastLogit = kEmpty * kLn2;

// The exponents' reference is not the exact running maximum: it follows when a value exceeds it
// by kSlack (log2 units), so that the rescaling branch is taken a few times per slice instead
// of every few tiles. Sums of 2^31 terms of 2^16 stay far inside binary32.
constexpr float kSlack = 16.0f;

// An item table (or a batch of queries): rows of row_b bytes every stride_b bytes (ROWS; both
// multiples of 16, 16-byte aligned), or the fragment-tiled layout of a packed corpus.
struct Table {
  const uint8_t* p;
  int64_t stride_b;
  int64_t n;
  int row_b;
};

// What the statistics pass computes: the sum, the entropy's sum too, or both and tile maxima.
enum { STATS_LSE = 0, STATS_ENT = 1, STATS_ALT = 2 };

struct StatsArgs {
  Table items, queries;
  int b;
  const float* bias;         // [n] or NULL
  const uint32_t* exclude;   // bitmap or NULL
  int64_t exclude_words;     // words per query; 0: one bitmap for the batch
  float scale;
  float scx;                 // log2 units per unit of a score (no bias) or of a logit
  float vmask;               // a masked score or logit: kMasked / scx
  int nqblk, nslices;
  int64_t nruns;             // runs of 2^run_log tiles
  int run_log;
  int ent;                   // whether the entropy's sums are wanted
  float4* part;              // [nslices][b]: reference, sum, sum of e * exponent
  float* bmax;               // [ceil(b/32)][nruns][32] largest logit of each run, or NULL
};

// 32-row blocks per tile of the pass: 8 KiB of items a wave and stage, at most 2 (more
// accumulators than that spill).
__host__ __device__ constexpr int stats_rm(int ct, int d) {
  const int r = 8192 / (int)block_bytes(ct, d);
  return r < 1 ? 1 : (r > 2 ? 2 : r);
}
// Stages in the register ring (one in use, the others in flight).
__host__ __device__ constexpr int stats_ns(int ct, int d) {
  return stats_rm(ct, d) * block_bytes(ct, d) > 8192 ? 2 : 3;
}
constexpr int kStatsThreads = 512;
constexpr int kStatsWaves = 8;
// Values kept per wave, query fragment and lane: reference, sum, the entropy's sum, and the run's
// maximum where it is wanted.
__host__ __device__ constexpr int stats_values(int mode) { return mode == STATS_ALT ? 4 : 3; }
// LDS of a workgroup of 32 * nqf queries: the query tile and those values.
__host__ __device__ constexpr int stats_lds(int ct, int d, int nqf, int mode = STATS_ALT) {
  return kFrag * nqf * d * elem_bytes(ct) + kStatsWaves * nqf * stats_values(mode) * kWave * 4;
}
__host__ __device__ constexpr bool stats_fits(int ct, int d, int nqf) {
  return stats_lds(ct, d, nqf) <= 160 * 1024;
}

template <int CT, int D>
int launch_stats(int nqf, bool rows, const StatsArgs& A, int grid, hipStream_t s);

}  // namespace mips

// ---------------------------------------------------------------------- the backward pass
namespace mips {

// What a score's weight needs besides the score, s in its own units and everything else in
// log2 units:  w = 2^(s scx + add_b + add_j), with the signs applied where they are uniform.
//  plain: add_b = log2 |coef_b| - lse_b log2 e, so that w = p |coef_b|, coef_b = - sum_i g_bi;
//  extra (entropy gradient, bitmaps per query, bias gradient): add_b = - lse_b log2 e and
//         w = p (coef_b + hent_b log2 p), coef_b with the entropy's share, hent_b = - h_b ln 2.
// add_j = bias_j log2 e. The streamed rows' addend is divided by scx and enters the scores'
// products as one more 16-byte chunk, against a chunk of ones. Queries are padded to a multiple
// of kGradTile with addends of kMasked.
constexpr int32_t kNoTarget = 0x7FFFFFFF;
struct QueryTerms {
  const float* add;      // add_b
  const float* coef;
  const float* hent;     // 0 without an entropy gradient
  const uint32_t* neg;   // bit b & 31 of word b >> 5: coef_b < 0 (plain)
  const int32_t* tgt;    // [b][g], ascending for each query; kNoTarget: none
  const float* gval;     // [b][g]
  int g;
};

struct GradArgs {
  Table own, str;            // the rows whose gradient is computed, and the rows summed over
  QueryTerms q;
  const float* bias;
  const uint32_t* exclude;
  int64_t exclude_words;
  float scale, scx, inv_scx;
  int nown, nsplit;          // own tiles and splits of the streamed rows
  int64_t ntiles;            // tiles of streamed rows
  void* out;                 // [own.n, d] of the operands' type; nsplit == 1
  float* part;               // [nsplit][own.n][d], otherwise
  float* bias_part;          // items' pass: [nsplit][own.n] gradient of the bias, or NULL
};

constexpr int kGradTile = 64;  // streamed rows per tile
constexpr int kGradBufs = 3;   // tiles in LDS: this one, the next, and the one being written

// Waves per SIMD: two where the sums and operands fit 256 registers.
__host__ __device__ constexpr int grad_wps(int ct, int d) { return d * elem_bytes(ct) > 256 ? 1 : 2; }
// Waves of a workgroup: in bf16 eight, which share each tile of streamed rows (four, in two
// workgroups a unit, moved twice the rows through LDS: 506 us against 456 for the queries of
// 4096 x 250,000 x 128 at the time); in f32, bound by its products, four: twice the workgroups for small
// batches (1000 x 1000 x 64: 15.5 us against 20.8).
__host__ __device__ constexpr int grad_waves(int ct, int d) { return ct == MIPS_BF16 && grad_wps(ct, d) == 2 ? 8 : 4; }
// Workgroups that run on a compute unit at once.
__host__ __device__ constexpr int grad_per_unit(int ct, int d) { return 4 * grad_wps(ct, d) / grad_waves(ct, d); }
__host__ __device__ constexpr int grad_own(int ct, int d) { return 32 * grad_waves(ct, d); }
// LDS of a workgroup, per tile: the rows (at least 128 bytes each), their addends as a 16-byte
// chunk, two more values a row and g targets; and 64 bytes of signs.
__host__ __device__ constexpr int grad_row_bytes(int ct, int d) { return d * elem_bytes(ct) < 128 ? 128 : d * elem_bytes(ct); }
__host__ __device__ constexpr int grad_lds(int ct, int d, int g) {
  return kGradBufs * kGradTile * (grad_row_bytes(ct, d) + 16 + 8 + 4 * g) + 64;
}

template <int CT, int D>
int launch_grad(bool items, bool extra, const GradArgs& A, hipStream_t s);

}  // namespace mips
