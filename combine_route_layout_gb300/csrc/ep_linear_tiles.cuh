// Tiles of 256 features by up to 256 rows that a pair of CTAs shares, for the products
// of bf16 operands: which tiles there are, the parts that their contractions are cut
// into, and what becomes of a tile's sums. The kernel's parameters Q hold its LinearParams
// `p`, the output (`out`, `features` long, `f_tiles` tiles of them), the tiles' `cap` and
// a dense product's `plan`, and the contraction's `terms`, Q::kDepth of them a stage.
// The products of block-quantised operands have tiles and sums of their own; they share
// what comes with parts (splits_for, tickets, add_parts), the tiles' table (take_tile, of
// barriers B with tile_full, tile_empty and tiles), the epilogue's meeting and the maps.
#pragma once

#include <cuda.h>

#include "ep_launch.cuh"
#include "ep_linear.cuh"
#include "ep_mma.cuh"

namespace ep {
namespace {

constexpr int kMaxRows = 256;                    // rows of a tile (f32 outputs: half)
constexpr int kMinCap = 64;
constexpr int kMaxSplits = 8;
// Stages of a contraction that is cut, and of a part of it, at least. Joining
// costs as much as sixteen stages, few parts or many (16 stages in two parts:
// 9.3 us for 7.3; 32 stages in four parts 10.5 and 8.8, in two 11.3 and 10.4: 1024
// x 1024 or 2048 x 256 f32, 16 x 2048 x 2048). dW's parts of a tile are 128 KB (32
// stages of 8 tiles in two parts 19.2 us for 15.7, with tiles of 256 rows).
constexpr int kWorth = 24, kLeast = 7, kWorthGrad = 48, kLeastGrad = 16;
constexpr int kEpilogueWarps = 8;                // two to each quarter of the TMEM lanes
constexpr int kThreads = (4 + kEpilogueWarps) * 32;
constexpr int kGroupBytes = 16;                  // what the plan keeps of a group

enum Mode { kForward = 0, kInputGrad = 1, kWeightGrad = 2 };

// What every CTA finds out about the call from the groups' counts.
struct Plan {
  int tiles;
  int cap;           // most rows of a tile
  int splits;        // parts that a tile's contraction is cut into
  int size;          // dense: rows of a tile
};

// Count this part in; what the CTA's threads wrote before the barrier ahead of
// this call is visible to the one that counts last, and theirs to it.
__device__ __forceinline__ unsigned int ticket_take(unsigned int* ticket) {
  unsigned int before;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(ticket) : "memory");
  return before;
}

// n / d for 0 <= n, 0 < d below 2^31, in two float steps. The compiler's integer
// division is longer, and a tile's place takes ten of them one after another.
__device__ __forceinline__ int quotient(int n, int d) {
  const float r = __fdividef(1.0f, (float)d);
  int q = (int)((float)n * r);              // off by 2^-21 of itself at most
  int left = n - q * d;
  const int more = (int)floorf((float)left * r);   // off by one at most
  q += more;
  left -= more * d;
  if (left < 0) --q;
  if (left >= d) ++q;
  return q;
}

// A part of the contraction of one tile.
struct Tile {
  int g;
  int64_t begin;     // first pool row of the group
  int r0, rows;      // rows of the tile within the group (dW: of the weight rows)
  int f0;            // first feature
  int n;             // MMA's N
  int terms;         // length of the contraction
  int kb0, kb1;      // this part's stages; none: kb0 >= kb1
  int part, parts;   // its place among the tile's parts that have any
};

constexpr int kSlots = 4;     // tiles that are worked out ahead

// Rows of a tile of a group of `count` rows: as few tiles as `cap` rows (a
// power of two) allow, of about equal size, in whole steps of 32.
__host__ __device__ __forceinline__ int tile_rows(int count, int cap, int (*div)(int, int)) {
  const int tiles = div(count + cap - 1, cap);
  return tiles ? (div(count + tiles - 1, tiles) + 31) / 32 * 32 : 32;
}

// Parts that contractions of `blocks` stages are cut into where `tiles` tiles
// leave pairs idle, from `worth` stages on; a part has at least `least` of them.
__host__ __device__ __forceinline__ int splits_for(int pairs, int tiles, int blocks, int worth,
                                                   int least) {
  if (blocks < worth) return 1;
  int n = tiles > 0 && tiles < pairs ? pairs / tiles : 1;
  if (n > kMaxSplits) n = kMaxSplits;
  if (n > blocks / least) n = blocks / least;
  return n < 1 ? 1 : n;
}

__device__ __forceinline__ int tiles_in(int count, int cap) {
  const int size = tile_rows(count, cap, quotient);
  return quotient(count + size - 1, size);
}

// Tiles are numbered in int32: segments that overlap may have more, and are refused then.
constexpr int kMostTiles = (1 << 30) - 1;
__device__ __forceinline__ int add_tiles(int a, int b) { return min(a + b, kMostTiles); }

// Unit u of the plan: part u % splits of tile u / splits.
template <int MODE, typename Q>
__device__ __forceinline__ Tile tile_at(const Q& q, const Plan& plan, const int* first,
                                        const int* begins, const int* counts, const int* sizes,
                                        int u) {
  Tile w;
  int t = plan.splits == 1 ? u : quotient(u, plan.splits);
  w.part = u - t * plan.splits;
  int lo = 0, hi = q.p.s.G - 1;          // the last group that starts at or before t
  if constexpr (MODE == kWeightGrad) {
    const int per = q.f_tiles * q.r_tiles;
    lo = quotient(t, per);
    t -= lo * per;
  } else {
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= t) lo = mid; else hi = mid - 1;
    }
    t -= first[lo];
  }
  w.g = lo;
  w.begin = begins[lo];
  const int count = counts[lo];
  if constexpr (MODE == kWeightGrad) {
    const int r = quotient(t, q.f_tiles);
    w.r0 = r * plan.cap;
    w.f0 = (t - r * q.f_tiles) * 256;
    w.rows = min(plan.cap, q.p.Nw - w.r0);
    w.n = w.rows > 128 ? 256 : 128;
    w.terms = count;
  } else {
    // 8 row tiles at a time pass over all features, so that tiles that run
    // together share operands in L2
    const int size = sizes[lo];
    const int tiles = quotient(count + size - 1, size);
    const int band = quotient(t, 8 * q.f_tiles);
    const int in = min(8, tiles - band * 8);
    t -= band * 8 * q.f_tiles;
    const int f = quotient(t, in);
    w.r0 = (band * 8 + t - f * in) * size;
    w.f0 = f * 256;
    w.rows = min(size, count - w.r0);
    w.n = (w.rows + 31) / 32 * 32;
    w.terms = q.terms;
  }
  const int blocks = (w.terms + Q::kDepth - 1) / Q::kDepth;
  w.parts = 1;
  w.kb0 = 0;
  w.kb1 = blocks;
  if (plan.splits > 1) {
    const int each = quotient(blocks + plan.splits - 1, plan.splits);
    w.parts = blocks ? quotient(blocks + each - 1, each) : 1;
    w.kb0 = w.part * each;
    w.kb1 = min(blocks, w.kb0 + each);
  }
  return w;
}

// The groups' segments, the size of the tiles and the first tile of each
// group. All threads of the CTA. (A dense product's plan comes from the host.)
//
// Where the tiles of 256 rows are fewer than half the pairs, tiles of 128 and
// then 64 rows use more of the SMs at the cost of reading the weights more
// often; what is still idle then takes parts of the tiles' contractions, whose
// f32 sums the last part to finish adds up. 1024 x 7168 x 256: 43.7 us as 4
// tiles of 256 rows, 27.5 us as 16 tiles of 64 rows in 4 parts each (as measured
// when it was built; 14.1 us now).
template <int MODE, typename Q>
__device__ Plan plan_tiles(const Q& q, int* first, int* begins, int* counts, int* sizes) {
  const int base_cap = q.cap;
  __shared__ int sums[3][kThreads / 32];
  if (!q.p.s.begin) {
    if (threadIdx.x == 0) {
      first[0] = begins[0] = 0;
      counts[0] = (int)q.p.s.dense_rows;
      sizes[0] = q.plan.size;
    }
    __syncthreads();
    return q.plan;
  }
  const int G = q.p.s.G, pairs = gridDim.x >> 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (G + kThreads - 1) / kThreads;
  const int g0 = threadIdx.x * per, g1 = min(G, g0 + per);
  Plan plan;
  plan.cap = base_cap;
  int n0 = 0, n1 = 0, n2 = 0;            // tiles of cap, cap / 2, cap / 4 rows; dW: largest count
  for (int g = g0; g < g1; ++g) {
    int64_t b, c;
    segment_of(q.p.s, g, b, c);
    begins[g] = (int)b;
    counts[g] = (int)c;
    if constexpr (MODE == kWeightGrad) {
      n0 = max(n0, (int)c);
    } else {
      n0 = add_tiles(n0, tiles_in((int)c, base_cap) * q.f_tiles);
      n1 = add_tiles(n1, tiles_in((int)c, base_cap / 2) * q.f_tiles);
      n2 = add_tiles(n2, tiles_in((int)c, base_cap / 4) * q.f_tiles);
    }
  }
  int s0 = n0, s1 = n1, s2 = n2;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const int x = __shfl_xor_sync(kFull, s0, o);
    s0 = MODE == kWeightGrad ? max(s0, x) : add_tiles(s0, x);
    if (MODE != kWeightGrad) {
      s1 = add_tiles(s1, __shfl_xor_sync(kFull, s1, o));
      s2 = add_tiles(s2, __shfl_xor_sync(kFull, s2, o));
    }
  }
  if (lane == 0) {
    sums[0][warp] = s0;
    sums[1][warp] = s1;
    sums[2][warp] = s2;
  }
  __syncthreads();
  if constexpr (MODE == kWeightGrad) {
    int most = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) most = max(most, sums[0][w]);
    plan.tiles = G * q.f_tiles * q.r_tiles;
    plan.splits = splits_for(pairs, plan.tiles, (most + Q::kDepth - 1) / Q::kDepth, kWorthGrad,
                             kLeastGrad);
    return plan;
  }
  s0 = s1 = s2 = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    s0 = add_tiles(s0, sums[0][w]);
    s1 = add_tiles(s1, sums[1][w]);
    s2 = add_tiles(s2, sums[2][w]);
  }
  int level = 0, mine = n0;
  plan.tiles = s0;
  if (2 * s0 <= pairs) {
    level = 1;
    mine = n1;
    plan.tiles = s1;
    if (2 * s1 <= pairs && base_cap / 2 > kMinCap) {
      level = 2;
      mine = n2;
      plan.tiles = s2;
    }
  }
  plan.cap = base_cap >> level;
  plan.splits = splits_for(pairs, plan.tiles,
                           (q.terms + Q::kDepth - 1) / Q::kDepth, kWorth, kLeast);
  // tiles before this thread's groups: an exclusive scan over the threads
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += v;
  }
  int before = incl - mine;
  for (int w = 0; w < warp; ++w) before += sums[level][w];
  for (int g = g0; g < g1; ++g) {
    first[g] = before;
    sizes[g] = tile_rows(counts[g], plan.cap, quotient);
    before += quotient(counts[g] + sizes[g] - 1, sizes[g]) * q.f_tiles;
  }
  if (plan.tiles >= kMostTiles) {
    plan.tiles = 0;
    if (threadIdx.x == 0) atomicOr(q.p.s.err, kErrSegment);
  }
  __syncthreads();
  return plan;
}

// Accesses that a predicate turns off: no branch keeps one column's from the
// next one's. (With a test on each column the compiler makes branches, and
// 8192 x 1024 x 8192 takes 237 us instead of 102.)
__device__ __forceinline__ void put(float* at, float v, bool on) {
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n @p st.global.f32 [%0], %1;\n}" ::"l"(at),
               "f"(v), "r"((uint32_t)on)
               : "memory");
}
__device__ __forceinline__ void put(__nv_bfloat16* at, float v, bool on) {
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n @p st.global.b16 [%0], %1;\n}" ::"l"(at),
               "h"(__bfloat16_as_ushort(__float2bfloat16_rn(v))), "r"((uint32_t)on)
               : "memory");
}
__device__ __forceinline__ void put2(__nv_bfloat16* at, float lo, float hi, bool on) {
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n @p st.global.b32 [%0], %1;\n}" ::"l"(at),
               "r"(cvt_bf16x2(lo, hi)), "r"((uint32_t)on)
               : "memory");
}
__device__ __forceinline__ float get(const float* at, bool on) {
  float v;
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n mov.b32 %0, 0;\n @p ld.global.f32 %0, [%1];\n}"
               : "=f"(v)
               : "l"(at), "r"((uint32_t)on)
               : "memory");
  return v;
}
__device__ __forceinline__ float get(const __nv_bfloat16* at, bool on) {
  unsigned short v;
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n mov.b16 %0, 0;\n @p ld.global.b16 %0, [%1];\n}"
               : "=h"(v)
               : "l"(at), "r"((uint32_t)on)
               : "memory");
  return __bfloat162float(__ushort_as_bfloat16(v));
}
// Another CTA's sum, from L2.
__device__ __forceinline__ float get_part(const float* at, bool on) {
  float v;
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n mov.b32 %0, 0;\n @p ld.global.cg.f32 %0, [%1];\n}"
               : "=f"(v)
               : "l"(at), "r"((uint32_t)on)
               : "memory");
  return v;
}

// The sums of a tile's parts (at most MOST), `next` floats apart, of a lane's 32
// columns (`left` of them exist), added in the parts' order. AT columns of all
// parts are asked for at once, as many as 64 registers hold: each such round
// waits for L2 once, the parts one after another would wait for it each (1024 x
// 7168 x 256, 4 parts: 15.0 us; with 8 columns a round 17.5).
template <int MOST, int AT>
__device__ __forceinline__ void add_most_parts(const float* at, int next, int parts, int left,
                                               float (&r)[32]) {
#pragma unroll
  for (int h = 0; h < 32; h += AT) {
#pragma unroll
    for (int c = 0; c < AT; ++c) r[h + c] = 0.0f;
    if (h >= left) continue;
    float v[MOST][AT];
#pragma unroll
    for (int i = 0; i < MOST; ++i)
#pragma unroll
      for (int c = 0; c < AT; ++c)
        v[i][c] = get_part(at + i * next + (h + c) * 256, i < parts && h + c < left);
#pragma unroll
    for (int i = 0; i < MOST; ++i)
#pragma unroll
      for (int c = 0; c < AT; ++c) r[h + c] += v[i][c];
  }
}

__device__ __forceinline__ void add_parts(const float* at, int next, int parts, int left,
                                          float (&r)[32]) {
  if (parts <= 2) {
    add_most_parts<2, 32>(at, next, parts, left, r);
  } else if (parts <= 4) {
    add_most_parts<4, 16>(at, next, parts, left, r);
  } else {
    add_most_parts<kMaxSplits, 8>(at, next, parts, left, r);
  }
}

// Tile number i of this pair, as the scheduling warp left it: for one thread,
// and for a warp.
template <typename B>
__device__ __forceinline__ bool take_tile(B* bar, int i, Tile& w) {
  const int slot = i % kSlots;
  if (!mbar_wait_soon(&bar->tile_full[slot], (i / kSlots) & 1)) return false;
  w = bar->tiles[slot];
  mbar_arrive(&bar->tile_empty[slot]);
  return true;
}

template <typename B>
__device__ __forceinline__ bool warp_take_tile(B* bar, int i, Tile& w, int lane) {
  const int slot = i % kSlots;
  if (!warp_wait(&bar->tile_full[slot], (i / kSlots) & 1)) return false;
  w = bar->tiles[slot];
  __syncwarp();
  if (lane == 0) mbar_arrive(&bar->tile_empty[slot]);
  return true;
}

// The epilogue's warps meet; false if one of them does not come.
template <typename B>
__device__ __forceinline__ bool epilogue_meet(B* bar, int lane, uint32_t& phase) {
  __syncwarp();
  if (lane == 0) mbar_arrive(&bar->joined);
  const bool ok = warp_wait(&bar->joined, phase);
  phase ^= 1;
  return ok;
}

// A lane's feature of `left` rows, one store each.
template <typename T>
__device__ __forceinline__ void store_each(T* at, int64_t ld, int left, const float (&v)[32]) {
  if (left >= 32) {
#pragma unroll
    for (int c = 0; c < 32; ++c, at += ld) put(at, v[c], true);
  } else {
#pragma unroll
    for (int c = 0; c < 32; ++c, at += ld) put(at, v[c], c < left);
  }
}

// The same two features at a time: lanes 2 i and 2 i + 1 exchange a value of
// every two rows, so that each stores both features of one of them. Half the
// stores, each of four whole sectors. Needs rows and tensor on 4-byte
// boundaries (an even `ld`).
__device__ __forceinline__ void store_pairs(__nv_bfloat16* rows, int64_t ld, int feature,
                                            int features, int left, const float (&v)[32]) {
  const int odd = feature & 1;
  __nv_bfloat16* at = rows + (feature - odd) + odd * ld;
  const int mine = feature - odd < features ? left - odd : 0;   // `features` is even with ld
  const bool all = left >= 32 && mine > 0;
#pragma unroll
  for (int c = 0; c < 32; c += 2, at += 2 * ld) {
    const float other = __shfl_xor_sync(kFull, odd ? v[c] : v[c + 1], 1);
    put2(at, odd ? other : v[c], odd ? v[c + 1] : other, all || c < mine);
  }
}
__device__ __forceinline__ void store_pairs(float* rows, int64_t ld, int feature, int features,
                                            int left, const float (&v)[32]) {
  store_each(rows + feature, ld, feature < features ? left : 0, v);
}

// The epilogue of 32 columns (rows of the output) of a warp's 32 lanes
// (features), T the output's type. The residual's loads come first.
template <int MODE, int ACT, typename T, typename Q>
__device__ __forceinline__ void epilogue(const Q& q, const Tile& w, int cta, int lane,
                                         int quad, int c0, const float (&r)[32], float b) {
  const auto& p = q.p;
  const int f = quad * 32 + lane;          // lane of the accumulator
  const int left = w.rows - c0;            // columns that exist
  const int64_t row0 = (MODE == kWeightGrad ? (int64_t)w.g * p.Nw : w.begin) + w.r0 + c0;
  if (MODE == kForward && ACT == EP_ACT_SWIGLU) {
    // even lanes hold a feature's gate, odd lanes its up value; a pair of
    // lanes exchanges two columns so that each finishes one of them
    const int out = w.f0 / 2 + cta * 64 + f / 2;
    const int odd = lane & 1;
    const int mine = out < p.N ? left - odd : 0;   // this lane's columns are 0, 2, ... below it
    const int64_t row = row0 + odd;
    T* y = static_cast<T*>(p.y) + row * p.N + out;
    const T* res = static_cast<const T*>(p.residual) + row * p.N + out;
    __nv_bfloat16* z = p.z + row * p.Nw + out;
    float add[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) add[i] = 0.0f;
    if (p.residual) {
#pragma unroll
      for (int i = 0; i < 16; ++i) add[i] = get(res + (int64_t)(2 * i) * p.N, 2 * i < mine);
    }
    const int kept = p.z ? mine : 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float v0 = r[2 * i] + b, v1 = r[2 * i + 1] + b;
      const float other = __shfl_xor_sync(kFull, odd ? v0 : v1, 1);
      const float gate = odd ? other : v0, up = odd ? v1 : other;
      put(y, silu_of(gate) * up + add[i], 2 * i < mine);
      put(z, gate, 2 * i < kept);
      put(z + p.N, up, 2 * i < kept);
      y += 2 * (int64_t)p.N;
      z += 2 * (int64_t)p.Nw;
    }
    return;
  }
  const int feature = w.f0 + cta * 128 + f;
  const int mine = feature < q.features ? left : 0;
  const int64_t ld = q.features;           // the output's rows are its features
  float v[32];
  if (MODE == kForward) {
    const T* res = static_cast<const T*>(p.residual) + row0 * ld + feature;
#pragma unroll
    for (int c = 0; c < 32; ++c) v[c] = r[c] + b;
    if (p.z) {
      __nv_bfloat16* z = p.z + row0 * ld;
      if (q.pairs_z) {
        store_pairs(z, ld, feature, q.features, left, v);
      } else {
        store_each(z + feature, ld, mine, v);
      }
    }
#pragma unroll
    for (int c = 0; c < 32; ++c) v[c] = act_of(ACT, v[c]);
    if (p.residual) {
#pragma unroll
      for (int c = 0; c < 32; ++c) v[c] += get(res + (int64_t)c * ld, c < mine);
    }
  } else {
#pragma unroll
    for (int c = 0; c < 32; ++c) v[c] = r[c];
  }
  T* y = static_cast<T*>(q.out) + row0 * ld;
  if (q.pairs_out) {
    store_pairs(y, ld, feature, q.features, left, v);
  } else {
    store_each(y + feature, ld, mine, v);
  }
}

// ---------------------------------------------------------------------- host

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                            const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                            const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline Encode encoder() {
  static Encode fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<Encode>(p);
  }();
  return fn;
}

// A map of bf16 (of E4M3 with `size` 1) with 128-byte swizzle; zeros beyond the
// tensor's edges. Strides count elements.
inline bool make_map(CUtensorMap* m, const void* base, int rank, const int64_t* dims,
                     const int64_t* strides, const int* box, int size = 2) {
  Encode fn = encoder();
  if (!fn) return false;
  cuuint64_t d[4], s[4];
  cuuint32_t b[4], one[4] = {1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = (cuuint64_t)(dims[i] > 0 ? dims[i] : 1);
    b[i] = (cuuint32_t)box[i];
    if (i) s[i - 1] = (cuuint64_t)strides[i] * size;
  }
  return fn(m, size == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<void*>(base), d, s, b,
            one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline int grid_of(int sms, int64_t tiles) {
  const int64_t most = sms / 2 < kLinearMaxPairs ? sms / 2 : kLinearMaxPairs;
  const int64_t pairs = tiles < most ? tiles : most;
  return (int)(2 * (pairs < 1 ? 1 : pairs));
}

inline int host_quotient(int n, int d) { return n / d; }

// plan_tiles for a dense product, whose rows the host knows.
inline Plan dense_plan(int64_t rows64, int base_cap, int f_tiles, int blocks, int pairs) {
  const int rows = (int)rows64;
  Plan plan;
  plan.cap = base_cap;
  for (int level = 0;; ++level) {
    const int size = tile_rows(rows, base_cap >> level, host_quotient);
    plan.cap = base_cap >> level;
    plan.tiles = (rows + size - 1) / size * f_tiles;
    plan.size = size;
    if (2 * plan.tiles > pairs || plan.cap <= kMinCap) break;
  }
  plan.splits = splits_for(pairs, plan.tiles, blocks, kWorth, kLeast);
  return plan;
}

// Upper bound of the units of all groups (their counts are on the device).
inline int64_t most_units(const LinearSegs& s, int f_tiles, int stages) {
  const int64_t rows = s.begin ? s.pool : s.dense_rows;
  const int64_t parts = stages / kLeast;
  return (rows / kMinCap + s.G) * f_tiles * (parts < 1 ? 1 : parts < kMaxSplits ? parts : kMaxSplits);
}

}  // namespace
}  // namespace ep
