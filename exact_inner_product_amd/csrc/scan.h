// scan.h -- parts shared by the gated recurrence's two directions (scan.hip, scan_grad.hip).
//
//   h_r = a_r h_{r-1} + b_r x_r,   a = sigmoid(forget),  b = sigmoid(-forget) or sigmoid(gate)
//
// is the composition of affine maps of the state, (A, B): h -> A h + B, which is associative. A
// workgroup takes a tile: 512 threads, 4 channels and a run of rows each, all in registers, so
// 128 rows by 128 channels in bf16. Runs are joined across the halves of a wave and its waves in LDS, tiles
// by a chain through memory (below). Each tensor moves once; a thread alone down a channel would move
// them as often, but 4096 x 128 channels are too few threads to fill the memory's queues.
#pragma once

#include "sequences.h"

// Products and sums are joined where fmaf says so and nowhere else: the variants for aligned and other
// rows, compiled apart, give the same bits.
#pragma clang fp contract(off)

namespace mips {

constexpr int kTileThreads = 512;
// Rows of a thread, a run: of what it holds of each, eight fit in its registers in bf16 and four in f32.
template <typename T> constexpr int kRun = sizeof(T) == 2 ? 8 : 4;

// Lanes a row (4 channels each): 4, 8, 16 or 32, of widths up to 16, 32, 64, any.
inline int scan_lanes_log2(int32_t d) { return d > 64 ? 5 : d > 32 ? 4 : d > 16 ? 3 : 2; }

// How a call's rows are cut. Dense sequences that fit in a tile lie whole in tiles of a multiple of
// their length: no state passes between tiles. Else the tiles are chained.
struct Tiling {
  uint32_t rows;      // of a tile
  uint32_t tiles;
  uint32_t columns;   // tiles side by side along the channels
  int lanes_log2;
  int threads;        // of a workgroup: 512 or 1024
  bool chained;
};
inline Tiling tiling_of(const Sequences& S, int32_t d, int run, int threads) {
  Tiling T;
  T.lanes_log2 = scan_lanes_log2(d);
  T.threads = threads;
  T.rows = (uint32_t)(threads * run) >> T.lanes_log2;
  const bool whole = S.t && S.t <= T.rows;
  if (whole) T.rows = T.rows / S.t * S.t;
  T.tiles = S.n ? (S.n + T.rows - 1) / T.rows : 1u;
  T.chained = !whole && T.tiles > 1;
  const uint32_t width = 4u << T.lanes_log2;
  T.columns = ((uint32_t)d + width - 1) / width;
  return T;
}
inline Tiling scan_tiling(const Sequences& S, int32_t d, int32_t dtype) {
  if (dtype == MIPS_BF16) return tiling_of(S, d, kRun<__bf16>, kTileThreads);
  // f32: twice the threads where that makes sequences lie whole in a tile
  const Tiling T = tiling_of(S, d, kRun<float>, kTileThreads), W = tiling_of(S, d, kRun<float>, 2 * kTileThreads);
  return T.chained && S.t && !W.chained ? W : T;
}
// Runs of all tiles.
inline int64_t scan_runs(const Tiling& T) { return (int64_t)T.tiles * (T.threads >> T.lanes_log2); }

// ------------------------------------------------------------------------------ gates
// sigmoid(v) and sigmoid(-v) (1 - sigmoid(v) would lose the small one): with e = exp(-v) they are 1 / (1 + e) and
// e / (1 + e), which is 1 to binary32 for e above 2^24, also where e is infinite and its product with 0 no
// number. The product with log2 e is rounded, which is |v| units in the last place of e at most: the
// smaller of the two is off by up to (2 |v| + 8) 2^-24 of its value. Values below 2^-126 may be 0, and
// sigmoid(-inf) is: an input that it gates leaves nothing, whatever finite value it holds. A NaN stays one.
__device__ __forceinline__ void sigmoids(float v, float* up, float* down) {
  const float e = __builtin_amdgcn_exp2f(-1.44269504f * v);
  const float r = __builtin_amdgcn_rcpf(1.0f + e);
  *up = r;
  *down = e > 0x1p24f ? 1.0f : e * r;
}

// --------------------------------------------------------------------- affine maps
// A >= 0 or NaN. A map that forgets its argument (a sequence starts inside) has A = kForgets; it
// must not be an ordinary 0, which makes NaN of an argument that is not finite, as the recurrence does.
constexpr float kForgets = -1.0f;

// `later` after `earlier`.
__device__ __forceinline__ void compose(float a0, float b0, float a1, float b1, float* a, float* b) {
  *b = a1 < 0.0f ? b1 : fmaf(a1, b0, b1);
  *a = (a1 < 0.0f || a0 < 0.0f) ? kForgets : a0 * a1;
}
__device__ __forceinline__ float apply(float a, float b, float h) { return a < 0.0f ? b : fmaf(a, h, b); }

// -------------------------------------------------------------------- chain of tiles
// Each tile and channel has a 64-bit word: empty, or the tile's map (A, B), a constant one where the
// state is cut inside. So has each group of kGroup tiles, written by its last tile; when that knows the
// state behind the group, it is written over the group's map, as a constant. Words are written and read with
// relaxed atomics, value and meaning together, so nothing else has to be ordered.
//
// Tiles are handed out by a counter, one a column of channels, in the chain's order: what a workgroup waits for
// are words of tiles handed out before its own, to workgroups that run already. The first of the
// unfinished tiles finds all it waits for, so every wait ends, whatever the order in which the card
// starts workgroups. A tile's word is written before anything is waited for, a group's after a wait
// for its tiles' words alone: no wait follows from another along the chain.
//
// The state before a tile is always the same fold, h <- A h + B over groups and then over tiles of its
// own group: constants only cut it short. Results do not depend on what was known when.
constexpr uint32_t kEmpty = 0xFFFFFFFFu;     // A of a word that is not written yet
constexpr uint32_t kConstant = 0x80000000u;  // A of a constant map
constexpr uint32_t kGroup = 16;

struct Chain {
  uint64_t* tiles;   // the same for all threads, as the rest but `channel`: scalar registers
  uint64_t* groups;
  int64_t stride;    // from a tile's words to the next one's
  uint32_t channel;
};

__device__ __forceinline__ void chain_put(uint64_t* w, float a, float b) {
  // a product of gates has no sign; the sign that a NaN may have is taken away
  const uint32_t m = a < 0.0f ? kConstant : (a == a ? __float_as_uint(a) : 0x7FC00000u);
  __hip_atomic_store(w, ((uint64_t)m << 32) | __float_as_uint(b), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t chain_get(const uint64_t* w) {
  return __hip_atomic_load(w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Workspace: the columns' counters (an atomic a tile on one address takes 12 ns, so they lie apart); of packed
// rows, what is known of each (to the end of the last tile); of chained tiles the words of tiles and of
// groups, [columns * width] each.
constexpr int kCounterPitch = 64;
struct ScanSpace {
  uint32_t* counters;
  int32_t* info;
  uint64_t* words;
  uint64_t count;  // of words
  size_t bytes;
};
inline ScanSpace scan_space(const Sequences& S, const Tiling& T, void* workspace) {
  ScanSpace W;
  uint8_t* p = (uint8_t*)workspace;
  W.counters = (uint32_t*)p;
  p += (size_t)T.columns * kCounterPitch * 4;
  W.info = S.offsets ? (int32_t*)p : nullptr;
  if (S.offsets) p += ((size_t)T.tiles * T.rows * 4 + 255) / 256 * 256;
  W.words = (uint64_t*)p;
  W.count = T.chained ? (uint64_t)(T.tiles + (T.tiles + kGroup - 1) / kGroup) * T.columns * (4u << T.lanes_log2) : 0;
  W.bytes = (size_t)(p - (uint8_t*)workspace) + W.count * 8;
  return W;
}
// The launch before a scan of packed or chained rows: empties the words, sets the counters to 0 (a
// kernel: a memset node replays wrongly in graphs), describes packed rows, and writes rows of
// `of_none` ([b, d]; NULL: not wanted) for packed sequences without rows: those of `as`, or 0.
int scan_begin(const Sequences& S, const Tiling& T, const ScanSpace& W, int32_t d, const float* as, float* of_none,
               hipStream_t s);

// What the threads of a workgroup share, each row `width` long.
struct Shared {
  float2* maps;      // [halves]: maps of half waves
  float* reach;      // [halves]: what reaches them
  float2* parts;     // [parts]: maps of four halves in a row
  float4* inner;     // [threads][2], fewer than 32 lanes a row only
  float* state;      // chained tiles only: what reaches the tile
  float2* before;    // [parts], chained tiles only: maps of some of the group's tiles
  uint64_t* groups;  // [kGroup], chained tiles only: words of the groups before
};
constexpr int kPart = 4;  // halves of a part
__host__ __device__ inline size_t shared_bytes(int threads, int width, bool chained, Shared* s, uint8_t* p) {
  const size_t halves = threads / 32, parts = halves / kPart, w = width;
  const size_t o1 = halves * w * 8, o2 = o1 + halves * w * 4, o3 = o2 + parts * w * 8;
  const size_t o4 = o3 + (width < 128 ? (size_t)threads * 32 : 0), o5 = o4 + (chained ? w * 8 : 0);
  const size_t o6 = o5 + (chained ? parts * w * 8 : 0), o7 = o6 + (chained ? kGroup * w * 8 : 0);
  if (s)
    *s = Shared{(float2*)p, (float*)(p + o1), (float2*)(p + o2), (float4*)(p + o3), (float*)(p + o4), (float2*)(p + o5), (uint64_t*)(p + o6)};
  return o7;
}

// The tile of a workgroup in its column. (Workgroups that stay and take one tile after another, with
// the next one asked for ahead, make those behind it wait until they come to it: twice the time.)
__device__ __forceinline__ uint32_t chain_ticket(uint32_t* counters, uint32_t column) {
  __shared__ uint32_t ticket;
  if (threadIdx.x == 0) ticket = atomicAdd(counters + column * kCounterPitch, 1u);
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(ticket);
}

// -------------------------------------------------------------- runs of half a wave
// The maps that threads of a channel take states through are those of half waves: with 32 lanes a row of
// one run. With fewer, the runs of a half are joined by shuffles first; what a run gets of what reaches its half
// waits in LDS meanwhile (registers are short), as it is needed only again behind the chain.
//
// Writes the half's map of this lane's four channels. BACK: the argument comes from the last run.
template <bool BACK>
__device__ __forceinline__ void half_maps(int tid, const float* ra, const float* rb, int lanes, const Shared& M) {
  const int in = tid & 31;
  float4* p = (float4*)(M.maps + (tid >> 5) * lanes * 4 + (tid & (lanes - 1)) * 4);
  if (lanes == 32) {
    p[0] = float4{ra[0], rb[0], ra[1], rb[1]};
    p[1] = float4{ra[2], rb[2], ra[3], rb[3]};
    return;
  }
  float xa[4], xb[4], ea[4], eb[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    xa[c] = ra[c];
    xb[c] = rb[c];
  }
  for (int o = lanes; o < 32; o <<= 1) {
    const bool has = BACK ? in + o < 32 : in >= o;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float pa = BACK ? __shfl_down(xa[c], o, 32) : __shfl_up(xa[c], o, 32);
      const float pb = BACK ? __shfl_down(xb[c], o, 32) : __shfl_up(xb[c], o, 32);
      if (has) compose(pa, pb, xa[c], xb[c], &xa[c], &xb[c]);
    }
  }
  const bool edge = BACK ? in + lanes >= 32 : in < lanes;  // nothing of the half before it
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float pa = BACK ? __shfl_down(xa[c], lanes, 32) : __shfl_up(xa[c], lanes, 32);
    const float pb = BACK ? __shfl_down(xb[c], lanes, 32) : __shfl_up(xb[c], lanes, 32);
    ea[c] = edge ? 1.0f : pa;
    eb[c] = edge ? 0.0f : pb;
  }
  M.inner[tid * 2] = float4{ea[0], ea[1], ea[2], ea[3]};
  M.inner[tid * 2 + 1] = float4{eb[0], eb[1], eb[2], eb[3]};
  if (BACK ? in < lanes : in + lanes >= 32) {
    p[0] = float4{xa[0], xb[0], xa[1], xb[1]};
    p[1] = float4{xa[2], xb[2], xa[3], xb[3]};
  }
}
// What reaches this lane's run, of what reaches its half.
__device__ __forceinline__ void half_reach(int tid, const Shared& M, int lanes, float* v) {
  const float4 r = *(const float4*)(M.reach + (tid >> 5) * lanes * 4 + (tid & (lanes - 1)) * 4);
  v[0] = r.x;
  v[1] = r.y;
  v[2] = r.z;
  v[3] = r.w;
  if (lanes == 32) return;
  const float4 a = M.inner[tid * 2], b = M.inner[tid * 2 + 1];
  v[0] = apply(a.x, b.x, v[0]);
  v[1] = apply(a.y, b.y, v[1]);
  v[2] = apply(a.z, b.z, v[2]);
  v[3] = apply(a.w, b.w, v[3]);
}

__device__ __forceinline__ float word_a(uint64_t w) {
  const uint32_t m = (uint32_t)(w >> 32);
  return m == kConstant ? kForgets : __uint_as_float(m);
}
__device__ __forceinline__ float word_b(uint64_t w) { return __uint_as_float((uint32_t)w); }

// From the maps of half waves to what reaches each, all threads of a workgroup together; begins and ends with
// a barrier. Threads of a channel share it in parts: a part composes four halves, or four tiles.
//
// Chained: tile k's state is found from tile `source` on, one that is constant because the sequence begins
// there; k itself if the tile needs no state, and its map is then taken as constant. Words of the
// group's tiles and of the kGroup groups before it are asked for at once, so that a link costs one trip
// to memory where nothing is late.
template <int THREADS, bool BACK, bool CHAINED>
__device__ __forceinline__ void join_halves(int tid, const Shared& M, const Chain& C, uint32_t k, uint32_t source,
                                            int channels, int width) {
  constexpr int HALVES = THREADS / 32, PARTS = HALVES / kPart, EACH = kGroup / PARTS;
  const int i = tid & 127, part = tid >> 7;
  const bool has = i < channels, owner = tid < channels;
  const float2* maps = M.maps + (BACK ? HALVES - 1 - part * kPart : part * kPart) * width + i;
  const int next = BACK ? -width : width;
  __syncthreads();
  float a = 1.0f, b = 0.0f;
  if (has) {
#pragma unroll
    for (int w = 0; w < kPart; ++w) compose(a, b, maps[w * next].x, maps[w * next].y, &a, &b);
    M.parts[part * width + i] = float2{a, b};
  }
  __syncthreads();
  float v = 0.0f;  // what reaches the tile
  if (CHAINED) {
    const bool needs = source < k;
    const uint32_t group = k / kGroup, begin = group * kGroup, before = k - begin;
    const bool closes = before == kGroup - 1;
    uint64_t* own = C.groups + group * C.stride + C.channel;
    if (owner) {
#pragma unroll
      for (int p = 1; p < PARTS; ++p) compose(a, b, M.parts[p * width + i].x, M.parts[p * width + i].y, &a, &b);
      if (!needs) a = kForgets;
      chain_put(C.tiles + k * C.stride + C.channel, a, b);
    }
    if (needs || closes) {
      const uint32_t low = source > begin && !closes ? source - begin : 0u;  // tiles low .. before - 1 of the group
      const uint32_t depth = needs ? group - min(source / kGroup, group) : 0u;  // groups before it
      const uint32_t asked = min(depth, kGroup);                                // at once, the nearest first
      if (has) {
        uint64_t tw[EACH], gw[EACH];
#pragma unroll
        for (int j = 0; j < EACH; ++j) {
          const uint32_t t = part * EACH + j;
          if (t >= low && t < before) tw[j] = chain_get(C.tiles + (begin + t) * C.stride + C.channel);
          if (t < asked) gw[j] = chain_get(C.groups + (group - 1 - t) * C.stride + C.channel);
        }
        float ta = 1.0f, tb = 0.0f;
#pragma unroll
        for (int j = 0; j < EACH; ++j) {
          const uint32_t t = part * EACH + j;
          if (t < low || t >= before) continue;
          while ((uint32_t)(tw[j] >> 32) == kEmpty) {
            __builtin_amdgcn_s_sleep(1);
            tw[j] = chain_get(C.tiles + (begin + t) * C.stride + C.channel);
          }
          compose(ta, tb, word_a(tw[j]), word_b(tw[j]), &ta, &tb);
        }
        M.before[part * width + i] = float2{ta, tb};
#pragma unroll
        for (int j = 0; j < EACH; ++j)
          if (part * EACH + j < asked) M.groups[(part * EACH + j) * width + i] = gw[j];  // empty or not
      }
      __syncthreads();
      if (owner) {
        float ga = 1.0f, gb = 0.0f, va, vb;  // of the group's tiles before this one, and with it
#pragma unroll
        for (int p = 0; p < PARTS; ++p) compose(ga, gb, M.before[p * width + i].x, M.before[p * width + i].y, &ga, &gb);
        compose(ga, gb, a, b, &va, &vb);
        if (closes) chain_put(own, va, vb);
        if (needs) {
          // back to the nearest constant (the source's group is one), and forward again
          uint32_t t = 0;
          for (; t < asked; ++t) {
            uint64_t w = M.groups[t * width + i];
            if ((uint32_t)(w >> 32) == kEmpty) {
              do {
                __builtin_amdgcn_s_sleep(1);
                w = chain_get(C.groups + (group - 1 - t) * C.stride + C.channel);
              } while ((uint32_t)(w >> 32) == kEmpty);
              M.groups[t * width + i] = w;
            }
            if ((uint32_t)(w >> 32) == kConstant) {
              ++t;
              break;
            }
          }
          if (t == asked && asked < depth && (uint32_t)(M.groups[(t - 1) * width + i] >> 32) != kConstant) {
            // further back than the words at hand
            uint32_t from = group - asked;
            uint64_t w;
            do {
              --from;
              do w = chain_get(C.groups + from * C.stride + C.channel);
              while ((uint32_t)(w >> 32) == kEmpty);
            } while (from > group - depth && (uint32_t)(w >> 32) != kConstant);
            for (; from < group - asked; ++from) {
              w = chain_get(C.groups + from * C.stride + C.channel);
              v = apply(word_a(w), word_b(w), v);
            }
          }
          for (; t > 0; --t) {
            const uint64_t w = M.groups[(t - 1) * width + i];
            v = apply(word_a(w), word_b(w), v);
          }
          if (closes && !(va < 0.0f)) chain_put(own, kForgets, apply(va, vb, v));
          v = apply(ga, gb, v);
        }
      }
    }
    if (owner) M.state[i] = v;
    __syncthreads();
    if (has) v = M.state[i];
  }
  if (has) {
    for (int p = 0; p < part; ++p) v = apply(M.parts[p * width + i].x, M.parts[p * width + i].y, v);
    float* reach = M.reach + (BACK ? HALVES - 1 - part * kPart : part * kPart) * width + i;
#pragma unroll
    for (int w = 0; w < kPart; ++w) {
      reach[w * next] = v;
      v = apply(maps[w * next].x, maps[w * next].y, v);
    }
  }
  __syncthreads();
}

// -------------------------------------------------------------------- four channels
// Of a row of at least four channels (`wide`) the last `live` ones, fewer than four, are loaded with those before
// them and moved down: loads of four, whatever the alignment (the card takes any), in every lane.
template <int VEC>
__device__ __forceinline__ void load4(const float* p, int live, bool wide, float* v) {
  typedef float f32x4_t __attribute__((ext_vector_type(4)));
  if constexpr (VEC) {
    const f32x4_t q = *(const f32x4_t*)p;
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = q[c];
  } else if (wide) {
    typedef float f32x4u_t __attribute__((ext_vector_type(4), aligned(4)));
    const int back = 4 - live;
    const f32x4u_t q = *(const f32x4u_t*)(p - back);
    const float r0 = back & 1 ? q[1] : q[0], r1 = back & 1 ? q[2] : q[1], r2 = back & 1 ? q[3] : q[2];
    v[0] = back & 2 ? r2 : r0;
    v[1] = back & 2 ? q[3] : r1;
    v[2] = r2;
    v[3] = q[3];
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = c < live ? p[c] : 0.0f;
  }
}

// Raw elements of four channels, kept as they are stored.
template <typename T> struct Raw;
template <> struct Raw<float> {
  float v[4];
  __device__ __forceinline__ float at(int c) const { return v[c]; }
};
template <> struct Raw<__bf16> {
  uint32_t v[2];
  __device__ __forceinline__ float at(int c) const {
    return __uint_as_float((c & 1) ? v[c >> 1] & 0xFFFF0000u : v[c >> 1] << 16);
  }
};

// Has v computed here, not where it is used, with all it comes from in registers until then.
__device__ __forceinline__ void here(float* v) { asm volatile("" : "+v"(*v)); }
// Makes the compiler forget what it has computed from r, so that it does so again where it is needed
// rather than keep it in registers.
template <typename T>
__device__ __forceinline__ void raw_again(Raw<T>* r) {
#pragma unroll
  for (unsigned c = 0; c < sizeof(r->v) / 4; ++c) asm volatile("" : "+v"(r->v[c]));
}
// `live` channels (1 to 4) of a row at p; 4 and aligned with VEC. Others hold anything.
template <int VEC>
__device__ __forceinline__ void raw_load(const float* p, int live, bool wide, Raw<float>* r) {
  load4<VEC>(p, live, wide, r->v);
}
template <int VEC>
__device__ __forceinline__ void raw_load(const __bf16* p, int live, bool wide, Raw<__bf16>* r) {
  typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
  if constexpr (VEC) {
    const u32x2_t q = *(const u32x2_t*)p;
    r->v[0] = q[0];
    r->v[1] = q[1];
  } else if (wide) {
    uint64_t q;
    __builtin_memcpy(&q, p - (4 - live), 8);
    q >>= 16 * (4 - live);
    r->v[0] = (uint32_t)q;
    r->v[1] = (uint32_t)(q >> 32);
  } else {
    const uint16_t* u = (const uint16_t*)p;
    r->v[0] = (uint32_t)u[0] | (live > 1 ? (uint32_t)u[1] << 16 : 0u);
    r->v[1] = live > 2 ? (uint32_t)u[2] : 0u;
  }
}
// Rows of a run that are not inner ones of a sequence, a bit each, 8 a kind, in one register.
struct Marks {
  uint32_t bits;
  __device__ __forceinline__ bool any() const { return bits != 0; }
  __device__ __forceinline__ bool pad(int t) const { return (bits >> t) & 1u; }            // of no sequence: 0
  __device__ __forceinline__ bool beyond(int t) const { return (bits >> (8 + t)) & 1u; }   // and not this tile's
  __device__ __forceinline__ bool cut(int t) const { return (bits >> (16 + t)) & 1u; }     // pad, or a first row
  __device__ __forceinline__ bool final(int t) const { return (bits >> (24 + t)) & 1u; }
  __device__ __forceinline__ bool first(int t) const { return cut(t) && !pad(t); }
  // Whether a lane of the wave has one at row t: what few rows need is done for those.
  __device__ __forceinline__ bool wave_has(int t) const { return __any((bits >> t) & 0x01010101u); }
};
// The sequence of a row that has one.
__device__ __forceinline__ int64_t row_sequence(const Sequences& S, const int32_t* packed, uint32_t r) {
  return S.t ? r / S.t : (uint32_t)packed[r] >> 2;
}
template <int R>
__device__ __forceinline__ Marks run_marks(const Sequences& S, const int32_t* packed, uint32_t r0, uint32_t rows,
                                           uint32_t at) {
  const uint32_t r = r0 + at;
  uint32_t pad = 0, cut = 0, final = 0;
  const uint32_t here = at < rows ? min(rows - at, (uint32_t)R) : 0u;
  const uint32_t beyond = ((1u << R) - 1u) & ~((1u << here) - 1u);
  if (!S.t) {
#pragma unroll
    for (int t = 0; t < R; t += 4) {
      const i32x4_t v = *(const i32x4_t*)(packed + r + t);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        pad |= (uint32_t)((uint32_t)v[e] >= (uint32_t)S.b << 2) << (t + e);
        cut |= (uint32_t)(v[e] & kFirst) << (t + e);
        final |= (uint32_t)(v[e] & kFinal) >> 1 << (t + e);
      }
    }
  } else {
    uint32_t s = r / S.t, pos = r - s * S.t;
    if (!S.lengths) {
      if (pos > 0 && pos + R < S.t && !beyond) return Marks{0u};
#pragma unroll
      for (int t = 0; t < R; ++t) {
        cut |= (uint32_t)(pos == 0) << t;
        pos = pos + 1 == S.t ? 0 : pos + 1;
        final |= (uint32_t)(pos == 0) << t;
      }
    } else if (S.t >= (uint32_t)R) {  // rows of at most two sequences
      auto below = [](uint32_t n) { return (1u << min(n, (uint32_t)R)) - 1u; };
      if (here) {
        const uint32_t split = S.t - pos, len = index_at(S.lengths, S.wide, s, S.t);
        const uint32_t some = len > pos ? len - pos : 0u;  // rows of the first one, at most split
        cut = pos == 0;
        pad = below(split) & ~below(some);
        final = some && some <= (uint32_t)R ? 1u << (some - 1) : 0u;
        if (split < here) {
          const uint32_t more = split + index_at(S.lengths, S.wide, s + 1, S.t);
          cut |= 1u << split;
          pad |= below(R) & ~below(more);
          if (more > split && more <= (uint32_t)R) final |= 1u << (more - 1);
        }
      }
    } else {
      uint32_t len = 0;
      for (uint32_t t = 0; t < here; ++t) {
        if (t == 0 || pos == 0) len = index_at(S.lengths, S.wide, s, S.t);
        cut |= (uint32_t)(pos == 0) << t;
        pad |= (uint32_t)(pos >= len) << t;
        final |= (uint32_t)(pos + 1 == len) << t;
        if (++pos == S.t) {
          pos = 0;
          ++s;
        }
      }
    }
  }
  pad |= beyond;
  final &= ~pad;
  return Marks{pad | beyond << 8 | (cut | pad) << 16 | final << 24};
}

// Padded sequences: a run's rows, from row r on, where sequences without rows would begin. A bit each.
template <int R>
__device__ __forceinline__ uint32_t run_nones(const Sequences& S, uint32_t r, const Marks& marks) {
  uint32_t first = 0;
  const uint32_t pos = r % S.t;
  for (uint32_t t = pos ? S.t - pos : 0u; t < (uint32_t)R; t += S.t) first |= 1u << t;
  return first & marks.bits & ~(marks.bits >> 8);
}

// The tile where the sequence of row r0 begins, the first of tile k, in whose chain k's state is then found;
// k itself if no sequence goes on from the tile before.
__device__ __forceinline__ uint32_t chain_source(const Sequences& S, const int32_t* packed, uint32_t r0, uint32_t rows, uint32_t k) {
  if (k == 0) return 0;
  uint32_t begin, end;
  int64_t s;
  if (S.t) {
    s = r0 / S.t;
  } else {
    const uint32_t v = (uint32_t)packed[r0];
    if (v >= (uint32_t)S.b << 2) return k;  // padding
    s = v >> 2;
  }
  sequence_rows(S, s, &begin, &end);
  return begin < r0 && r0 < end ? begin / rows : k;
}
// Backward: the step of the tile where the sequence of row r, the last of step k's tile, ends. Step 0 is the last tile.
__device__ __forceinline__ uint32_t chain_source_back(const Sequences& S, const int32_t* packed, uint32_t r, uint32_t rows,
                                                      uint32_t tiles, uint32_t k) {
  if (k == 0) return 0;
  uint32_t begin, end;
  int64_t s;
  if (S.t) {
    s = r / S.t;
  } else {
    const uint32_t v = (uint32_t)packed[r];
    if (v >= (uint32_t)S.b << 2) return k;
    s = v >> 2;
  }
  sequence_rows(S, s, &begin, &end);
  return begin <= r && r + 1 < end ? tiles - 1 - (end - 1) / rows : k;
}

// A run of a tensor: rows `row` .. of the tile [r0, r0 + rows), channels `channel` .. of those from c0
// on. There is no branch around a load: for rows beyond the tile and padding one is loaded that is
// there (the run's first, or the tile's last), and not looked at.
//
// Sequences without gaps between them, tiles below 2^31 bytes: a scalar address and 32-bit offsets.
template <int VEC, typename T, int R>
__device__ __forceinline__ void load_flat(const Rows& src, uint32_t r0, uint32_t rows, uint32_t row, int c0,
                                          uint32_t channel, int live, bool wide, Marks skip, Raw<T> (&out)[R]) {
  const uint8_t* base = (const uint8_t*)((const T*)src.p + (int64_t)r0 * src.row + c0);
  const uint32_t bytes = (uint32_t)src.row * sizeof(T);
  const uint32_t first = (row < rows ? row : rows - 1) * bytes + channel * (uint32_t)sizeof(T);
  uint32_t at = first;
#pragma unroll
  for (int t = 0; t < R; ++t) {
    raw_load<VEC>((const T*)(base + (skip.pad(t) ? first : at)), live, wide, &out[t]);
    at += bytes;
  }
}
inline bool rows_flat(const Rows& r, const Tiling& T, int32_t dtype) {
  return r.extra == 0 && (int64_t)T.rows * r.row * elem_bytes(dtype) < int64_t(1) << 31;
}
// Any others, dense ones (packed rows have no gaps and a bounded stride).
template <int VEC, typename T, int R>
__device__ __forceinline__ void load_gaps(const Sequences& S, const Rows& src, uint32_t r0, uint32_t rows, uint32_t row,
                                          int c0, uint32_t channel, int live, bool wide, Marks skip, Raw<T> (&out)[R]) {
  const uint32_t r = r0 + (row < rows ? row : rows - 1), s = r / S.t;
  const T* p = (const T*)src.p + (int64_t)r * src.row + (int64_t)s * src.extra + c0 + channel;
  const T* first = p;
  uint32_t left = (s + 1) * S.t - r;  // rows of this sequence
#pragma unroll
  for (int t = 0; t < R; ++t) {
    raw_load<VEC>(skip.pad(t) ? first : p, live, wide, &out[t]);
    if (row + t + 1 < rows) {
      p += src.row;
      if (--left == 0) {
        p += src.extra;
        left = S.t;
      }
    }
  }
}

// Past the caches with VEC 2 (4096 x 127 x 128 bf16: 86 -> 82 us, its gradient 142 -> 131).
template <int VEC>
__device__ __forceinline__ void store4(float* p, int live, const float* v) {
  typedef float f32x4_t __attribute__((ext_vector_type(4)));
  if constexpr (VEC) {
    const f32x4_t q{v[0], v[1], v[2], v[3]};
    if (VEC > 1) __builtin_nontemporal_store(q, (f32x4_t*)p);
    else *(f32x4_t*)p = q;
  } else if (live == 4) {
    __builtin_memcpy(p, v, 16);
  } else {
#pragma unroll
    for (int c = 0; c < 3; ++c)
      if (c < live) p[c] = v[c];
  }
}
template <int VEC>
__device__ __forceinline__ void store4(__bf16* p, int live, const float* v) {
  typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
  const bf16x4_t q{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
  if constexpr (VEC) {
    if (VEC > 1) __builtin_nontemporal_store(q, (bf16x4_t*)p);
    else *(bf16x4_t*)p = q;
  } else if (live == 4) {
    __builtin_memcpy(p, &q, 8);
  } else {
#pragma unroll
    for (int c = 0; c < 3; ++c)
      if (c < live) p[c] = q[c];
  }
}
// A kernel's VEC: 0 where some rows do not lie by four. Else 2, but 1 for rows of less than 64 bytes, whose
// lines would go to memory in pieces (32,768 x 127 x 16 bf16, gradient: 389 us with 2, 169 with 1, 232 with
// 0). There is no 1 for floats: rows of less than 16 are too narrow for more kernels.
inline int rows_vec(bool by_four, int32_t d, int32_t dtype) {
  if (!by_four || d * elem_bytes(dtype) >= 64) return by_four ? 2 : 0;
  return dtype == MIPS_BF16 ? 1 : 0;
}

}  // namespace mips
