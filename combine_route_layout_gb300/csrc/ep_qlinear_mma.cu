// The products of block-quantised operands on the tensor cores: z = x W^T and
// dx = dz' W, with the forward's bias, activation and residual in the epilogue.
//
// A stage is 128 bytes of each operand row, which of E4M3 are 128 terms: exactly one
// scale block. The tensor core adds up one stage at a time, into two accumulators in
// turn, and the epilogue's warps take each such sum out of tensor memory and add it,
// times its scales, to f32 sums of the tile in their registers, while the next one is
// made:
//     sum[row][feature] += stage[row][feature] (sx[row][block] sw[feature block][block])
// Rows are on the M side, 128 of them to a CTA, features on the N side, 256 (or 128
// where those leave half of the pairs idle): a lane is a row, whose scale is one
// register, and the weights' scale is one for all of a warp's columns (two with SwiGLU),
// so that the epilogue reads no shared memory. (Features on the M side, as in the bf16
// products, take the rows' scales from there, eight 16-byte loads a warp and stage:
// under the tensor core's own reads each takes 100 cycles, and 8192^3 961 us.)
//
// A sum changes hands twice a stage (512 cycles of the tensor core), and every look at a
// shared-memory barrier takes 200 to 250 cycles then. So each CTA makes its own
// products, and its epilogue hands an accumulator back by a hardware barrier. CTAs work
// by themselves: neighbours take the halves of a tile of 256 rows, and each loads all of
// its weights, which the second has from L2. (Each loading half for both of a cluster
// takes 2 % less for the 128 experts below, but needs loads into another CTA's
// shared memory, which no kernel here has.) Groups
// of at most 128 rows have tiles of twice the features instead, half of them each
// CTA's, so that experts with a handful of rows keep all SMs reading weights (256 experts
// x 32 rows, above: 306 us when it came in, 502 with such rows in one CTA of a pair).
// SwiGLU: half of the tile's columns are gates, half the same features' up values; a
// thread has both. W is read as it is for dx too: MN-major, a box of 128 terms x 128
// features.
//
// Roles by warp: 0 TMA, 1 MMA, 2 looks for complete sums and tells the epilogue by
// another hardware barrier (18 us of 8192^3 when it came in, 533 then), 3 works
// out the tiles (one thread each, but for 1 and 2, which wait as warps), 4-11 epilogue:
// TMEM lanes go by warp % 4, columns by halves. 128 sums a thread: the other warps give
// registers up for them (16 warps with 64 sums each: 870 us).
//
// Bound by that loop, at the full clock: 128 experts x 973 rows, 4096 to 2 x 2048 with
// SwiGLU, bias and pre-activations, 2.59 ms, 1.61 PFLOP/s, 1000 to 1100 cycles a stage; 256
// experts x 32 rows, 7168 to 2 x 512, 295 to 301 us, 96 % of the copy's bandwidth; 256
// experts x 1024 rows, 7168 to 2 x 2048, 7.4 ms, 2.07 PFLOP/s; 8192^3 535 us, 2.05.
#include <atomic>
#include <climits>
#include <cstring>
#include <type_traits>

#include "ep_linear_tiles.cuh"
#include "ep_qlinear.cuh"

namespace ep {
namespace {

constexpr int kDepth = 128;                      // terms per stage: 128 bytes
constexpr int kTileRows = 256;                   // of both neighbours
constexpr int kStageA = 128 * kDepth;            // bytes of a CTA's rows
constexpr int kRingBytes = 4 * (kStageA + 256 * kDepth);
constexpr int kMaxStages = 6;                    // of 128 features
constexpr int kTmemColumns = 512;                // two accumulators
constexpr int kTurnRows = 8, kTurnPitch = 33;    // words: rows that are stored by column
constexpr int kTurnWords = 2 * kTurnRows * kTurnPitch;   // of a warp: gates and up
constexpr int kTurnBytes = kEpilogueWarps * kTurnWords * 4;
constexpr int kHandover = 32 * (1 + kEpilogueWarps);     // threads of the hardware barriers
// Registers of a thread at the start, of the first four warps and of the epilogue's
// (at an earlier step 8192^3 took 535 us so, 614 to 687 with 216 for the epilogue, 580
// with 232).
constexpr int kRegisters = 168, kRegistersLess = 56, kRegistersMore = 224;
static_assert(kThreads * kRegisters >= 128 * kRegistersLess + kEpilogueWarps * 32 * kRegistersMore,
              "registers for the epilogue");

// How far an f32's exponent is from `least` on, zeros and negative distances beyond any: with
// exponents below `most` alone if less than key_range(least, most).
__device__ __forceinline__ uint32_t scale_key(float v, uint32_t least) {
  return 2u * __float_as_uint(v) - 2u * (least << 23);
}
constexpr uint32_t key_range(uint32_t least, uint32_t most) { return 2u * ((most - least) << 23); }

struct QPlan {
  int tiles, splits;
  int width;         // columns of a CTA's tile: 256 or 128
  int size;          // dense: rows of a tile
};

struct MmaParams {
  QLinearParams p;
  void* out;               // y or dx
  int outs;                // length of its rows
  int stages;              // of a contraction
  int vec;                 // rows and tensors allow 32-byte accesses
  int pairs;               // of multiprocessors: the grid has fewer where units are
  QPlan plan;              // of a dense product
  // scale of (pool row, block) and of (group, feature block, block)
  const float* row_scale;
  int row_ld;
  int64_t group_ld;
  int feature_ld, block_ld;
  int feature_blocks;
  int up;                  // from a gate's scales to its up rows'
};

struct Barriers {
  uint64_t full[kMaxStages];  // a stage's operands have landed
  uint64_t empty[kMaxStages]; // the products have read this stage
  uint64_t acc_full[2];       // a stage's sum is complete
  uint64_t tile_full[kSlots], tile_empty[kSlots];
  uint64_t joined;            // the epilogue's warps meet
  Tile tiles[kSlots];
  uint32_t failed;            // a sum's warp gave up: sums are not to be had
  uint32_t met;               // sums for which the MMA warp has the accumulator back
  uint32_t tmem;
  uint32_t last;              // this CTA's part of a tile was the last
};

// Wait until the MMA warp has the accumulator of sum n back, for whoever is not told by
// the sum itself. That warp's waits and the epilogue's give up after a second each, at
// most five one after another; this one's limit is beyond them.
constexpr uint64_t kMetNs = 16 * kMbarWaitNs;
__device__ __forceinline__ void wait_met(const Barriers* bar, int n) {
  const volatile uint32_t* met = &bar->met;
  const uint64_t t0 = globaltimer_ns();
  while (*met <= (uint32_t)n && globaltimer_ns() - t0 < kMetNs) __nanosleep(200);
  __syncwarp();
}

// Results of a row that a CTA's tile has.
__host__ __device__ __forceinline__ int results_in(int width, bool gated) { return gated ? width / 2 : width; }

// Whether a group's tiles are all rows by twice the features.
__host__ __device__ __forceinline__ bool few_rows(int count) { return count <= kTileRows / 2; }

// Tiles beside each other for `outs` results of a row of a group.
__host__ __device__ __forceinline__ int tiles_beside(int outs, int width, bool gated, int count,
                                                     int (*div)(int, int)) {
  const int each = results_in(width, gated) * (few_rows(count) ? 2 : 1);
  return div(outs + each - 1, each);
}

// The groups' segments, the rows of the tiles and the first tile of each group. All
// threads of the CTA. (A dense product's plan comes from the host.)
template <bool GATED>
__device__ QPlan plan_qtiles(const MmaParams& q, int* first, int* begins, int* counts, int* sizes) {
  __shared__ int sums[2][kThreads / 32];
  if (!q.p.s.begin) {
    if (threadIdx.x == 0) {
      first[0] = begins[0] = 0;
      counts[0] = (int)q.p.s.dense_rows;
      sizes[0] = q.plan.size;
    }
    __syncthreads();
    return q.plan;
  }
  const int G = q.p.s.G, pairs = q.pairs;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (G + kThreads - 1) / kThreads;
  const int g0 = threadIdx.x * per, g1 = min(G, g0 + per);
  int n0 = 0, n1 = 0;                    // tiles of 256 and 128 columns
  for (int g = g0; g < g1; ++g) {
    int64_t b, c;
    segment_of(q.p.s, g, b, c);
    begins[g] = (int)b;
    counts[g] = (int)c;
    const int above = tiles_in((int)c, kTileRows);
    n0 = add_tiles(n0, above * tiles_beside(q.outs, 256, GATED, (int)c, quotient));
    n1 = add_tiles(n1, above * tiles_beside(q.outs, 128, GATED, (int)c, quotient));
  }
  int i0 = n0, i1 = n1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v0 = __shfl_up_sync(kFull, i0, o), v1 = __shfl_up_sync(kFull, i1, o);
    if (lane >= o) {
      i0 = add_tiles(i0, v0);
      i1 = add_tiles(i1, v1);
    }
  }
  if (lane == 31) {
    sums[0][warp] = i0;
    sums[1][warp] = i1;
  }
  __syncthreads();
  int all0 = 0, all1 = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    all0 = add_tiles(all0, sums[0][w]);
    all1 = add_tiles(all1, sums[1][w]);
  }
  QPlan plan;
  const int narrow = 2 * all0 <= pairs;
  plan.width = narrow ? 128 : 256;
  plan.tiles = narrow ? all1 : all0;
  int before = narrow ? i1 - n1 : i0 - n0;
  for (int w = 0; w < warp; ++w) before += sums[narrow][w];
  // no more units than the grid has pairs: each has one place for sums of parts
  plan.splits = plan.width == 128 ? splits_for(gridDim.x >> 1, plan.tiles, q.stages, kWorth, kLeast) : 1;
  plan.size = 0;
  for (int g = g0; g < g1; ++g) {
    first[g] = before;
    sizes[g] = tile_rows(counts[g], kTileRows, quotient);
    before += quotient(counts[g] + sizes[g] - 1, sizes[g]) * tiles_beside(q.outs, plan.width, GATED, counts[g], quotient);
  }
  if (plan.tiles >= kMostTiles) {
    plan.tiles = 0;
    if (threadIdx.x == 0) atomicOr(q.p.s.err, kErrSegment);
  }
  __syncthreads();
  return plan;
}

// Unit u of the plan: part u % splits of tile u / splits. f0 counts results of a row.
template <bool GATED>
__device__ __forceinline__ Tile qtile_at(const MmaParams& q, const QPlan& plan, const int* first,
                                         const int* begins, const int* counts, const int* sizes, int u) {
  Tile w;
  int t = plan.splits == 1 ? u : quotient(u, plan.splits);
  w.part = u - t * plan.splits;
  int lo = 0, hi = q.p.s.G - 1;          // the last group that starts at or before t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= t) lo = mid; else hi = mid - 1;
  }
  t -= first[lo];
  w.g = lo;
  w.begin = begins[lo];
  const int count = counts[lo];
  // 8 row tiles at a time pass over all features, so that tiles that run together
  // share operands in L2
  const int size = sizes[lo];
  const int tiles = quotient(count + size - 1, size);
  const int f_tiles = tiles_beside(q.outs, plan.width, GATED, count, quotient);
  const int band = quotient(t, 8 * f_tiles);
  const int in = min(8, tiles - band * 8);
  t -= band * 8 * f_tiles;
  const int f = quotient(t, in);
  w.r0 = (band * 8 + t - f * in) * size;
  w.rows = min(size, count - w.r0);
  // rows of the even CTA, the others are the odd one's; or all are both's
  w.n = few_rows(count) ? w.rows : (w.rows + 63) / 64 * 32;
  w.terms = few_rows(count) ? results_in(plan.width, GATED) : 0;   // to the odd CTA's features
  w.f0 = f * results_in(plan.width, GATED) * (few_rows(count) ? 2 : 1);
  w.parts = 1;
  w.kb0 = 0;
  w.kb1 = q.stages;
  if (plan.splits > 1) {
    const int each = quotient(q.stages + plan.splits - 1, plan.splits);
    w.parts = quotient(q.stages + each - 1, each);
    w.kb0 = w.part * each;
    w.kb1 = min(q.stages, w.kb0 + each);
  }
  return w;
}

// A CTA's part of a tile: how many rows, the first of them, the first feature.
struct Share {
  int rows;
  int64_t row0;
  int f0;
};
__device__ __forceinline__ Share share_of(const MmaParams& q, const Tile& w, int cta) {
  Share s;
  const bool few = w.terms > 0;
  s.f0 = w.f0 + cta * w.terms;
  s.rows = s.f0 >= q.outs ? 0 : few || !cta ? min(w.rows, w.n) : w.rows - w.n;
  s.row0 = w.begin + w.r0 + (few ? 0 : cta * w.n);
  return s;
}

__device__ __forceinline__ void store_v8(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void load_v8(const void* p, uint32_t (&v)[8]) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "l"(p)
               : "memory");
}

// 32 neighbouring values of a row, 32 bytes at a time: whole sectors of a lane's own.
__device__ __forceinline__ void store_row(__nv_bfloat16* at, const float (&v)[32]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = cvt_bf16x2(v[16 * h + 2 * i], v[16 * h + 2 * i + 1]);
    store_v8(at + 16 * h, u);
  }
}
__device__ __forceinline__ void store_row(float* at, const float (&v)[32]) {
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(v[8 * h + i]);
    store_v8(at + 8 * h, u);
  }
}
__device__ __forceinline__ void add_row(const __nv_bfloat16* at, float (&v)[32]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t u[8];
    load_v8(at + 16 * h, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[16 * h + 2 * i] += bf16_lo(u[i]);
      v[16 * h + 2 * i + 1] += bf16_hi(u[i]);
    }
  }
}
__device__ __forceinline__ void add_row(const float* at, float (&v)[32]) {
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    uint32_t u[8];
    load_v8(at + 8 * h, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[8 * h + i] += __uint_as_float(u[i]);
  }
}

// The epilogue of 32 columns of a warp's rows: `z` (and `up`, with SwiGLU) is a lane's
// row, T the output's type. Whole aligned pieces go out as they are; others are turned
// round, kTurnRows rows at a time, so that a warp stores 32 neighbours of a row.
template <int MODE, int ACT, typename T>
__device__ __forceinline__ void finish(const MmaParams& q, float* room, int g, int64_t row0, int rows,
                                       int col, int lane, float (&z)[32], float (&up)[32]) {
  constexpr bool kGated = MODE == kForward && ACT == EP_ACT_SWIGLU;
  const QLinearParams& p = q.p;
  const float* bias = MODE == kForward && p.bias ? p.bias + (int64_t)g * p.Nw + col : nullptr;
  T* y = static_cast<T*>(q.out) + row0 * q.outs + col;
  const T* res = MODE == kForward && p.residual ? static_cast<const T*>(p.residual) + row0 * q.outs + col : nullptr;
  __nv_bfloat16* zp = MODE == kForward && p.z ? p.z + row0 * p.Nw + col : nullptr;
  if (q.vec && col + 32 <= q.outs) {
    if (lane >= rows) return;
    if (bias) {
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        z[c] += bias[c];
        if (kGated) up[c] += bias[p.N + c];
      }
    }
    if (zp) {
      store_row(zp + (int64_t)lane * p.Nw, z);
      if (kGated) store_row(zp + (int64_t)lane * p.Nw + p.N, up);
    }
    if (MODE == kForward) {
#pragma unroll
      for (int c = 0; c < 32; ++c) z[c] = kGated ? silu_of(z[c]) * up[c] : act_of(ACT, z[c]);
    }
    if (res) add_row(res + (int64_t)lane * q.outs, z);
    store_row(y + (int64_t)lane * q.outs, z);
    return;
  }
  const bool in = col + lane < q.outs;
  const float b = bias && in ? bias[lane] : 0.0f, b_up = kGated && bias && in ? bias[p.N + lane] : 0.0f;
  for (int r0 = 0; r0 < 32; r0 += kTurnRows) {
    if (r0 >= rows) break;
    float add[kTurnRows];                // all of the residual's loads ahead of the stores
#pragma unroll
    for (int r = 0; r < kTurnRows; ++r) add[r] = res ? get(res + (int64_t)(r0 + r) * q.outs + lane, in && r0 + r < rows) : 0.0f;
    __syncwarp();
    if (lane / kTurnRows == r0 / kTurnRows) {
      float* to = room + (lane % kTurnRows) * kTurnPitch;
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        to[c] = z[c];
        if (kGated) to[kTurnRows * kTurnPitch + c] = up[c];
      }
    }
    __syncwarp();
    float v[kTurnRows], u[kTurnRows];
#pragma unroll
    for (int r = 0; r < kTurnRows; ++r) {
      v[r] = room[r * kTurnPitch + lane] + b;
      u[r] = kGated ? room[(kTurnRows + r) * kTurnPitch + lane] + b_up : 0.0f;
    }
    if (zp) {
#pragma unroll
      for (int r = 0; r < kTurnRows; ++r) {
        put(zp + (int64_t)(r0 + r) * p.Nw + lane, v[r], in && r0 + r < rows);
        if (kGated) put(zp + (int64_t)(r0 + r) * p.Nw + p.N + lane, u[r], in && r0 + r < rows);
      }
    }
#pragma unroll
    for (int r = 0; r < kTurnRows; ++r) {
      if (MODE == kForward) v[r] = kGated ? silu_of(v[r]) * u[r] : act_of(ACT, v[r]);
      put(y + (int64_t)(r0 + r) * q.outs + lane, v[r] + add[r], in && r0 + r < rows);
    }
  }
  __syncwarp();
}

struct Maps {
  CUtensorMap rows[3];     // boxes of 128, 64 and 32 rows
  CUtensorMap w[2];        // boxes of 128 and 64 features (dx: 128 features of 128 and 64 terms)
};

template <int MODE, int ACT, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    product8_kernel(const __grid_constant__ Maps maps, MmaParams q) {
  constexpr bool kGated = MODE == kForward && ACT == EP_ACT_SWIGLU;
  constexpr int kScaleGroup = kGated ? 4 : 2;   // stages whose scales are fetched at once: registers allow no more
  extern __shared__ uint8_t raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
  float* rooms = reinterpret_cast<float*>(ring + kRingBytes);    // [epilogue warp][kTurnWords]
  Barriers* bar = reinterpret_cast<Barriers*>(ring + kRingBytes + kTurnBytes);
  int* first = reinterpret_cast<int*>(bar + 1);
  int* begins = first + q.p.s.G;
  int* counts = begins + q.p.s.G;
  int* sizes = counts + q.p.s.G;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cta = blockIdx.x & 1;
  int32_t* timeout = q.p.s.err;

  // one thread a barrier
  if (threadIdx.x < kMaxStages) {
    mbar_init(&bar->full[threadIdx.x], 1);
    mbar_init(&bar->empty[threadIdx.x], 1);
  } else if (threadIdx.x < kMaxStages + 2) {
    mbar_init(&bar->acc_full[threadIdx.x - kMaxStages], 1);
  }
  if (threadIdx.x >= 32 && threadIdx.x < 32 + kSlots) {
    // producer, MMA, sums, the epilogue's warps
    mbar_init(&bar->tile_full[threadIdx.x - 32], 1);
    mbar_init(&bar->tile_empty[threadIdx.x - 32], 3 + kEpilogueWarps);
  } else if (threadIdx.x == 32 + kSlots) {
    mbar_init(&bar->joined, kEpilogueWarps);
    bar->failed = bar->met = 0;
  }
  if (threadIdx.x < 64) mbar_init_fence();
  if (threadIdx.x == 64) {
    tma_prefetch_map(&maps.rows[0]);
    tma_prefetch_map(&maps.w[0]);
  }
  __syncthreads();                       // the barriers are ready
  if (warp == 1) tmem_alloc_own(&bar->tmem, kTmemColumns);
  begin_overlapped();
  const QPlan plan = plan_qtiles<kGated>(q, first, begins, counts, sizes);
  const int units = plan.tiles * plan.splits;
  const int half_bytes = plan.width / 2 * kDepth;         // of the weights, of each CTA
  const int stage_bytes = kStageA + 2 * half_bytes;
  const int stages = min(kMaxStages, kRingBytes / stage_bytes);
  tc_fence_before();
  __syncthreads();                       // the TMEM address is there
  tc_fence_after();
  const uint32_t tmem = bar->tmem;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int mine = pair < units ? (units - 1 - pair) / pairs + 1 : 0;   // this pair's units

  if (warp < 4) {
    registers_less<kRegistersLess>();
    if (warp == 0 && elect_one()) {
      // ---------------------------------------------- producer: one thread
      int it = 0, s = 0;                      // stages written so far, the ring's place
      uint32_t phase = 1;                     // the first pass over the ring waits for nothing
      const uint32_t full0 = smem_addr(&bar->full[0]), ring0 = smem_addr(ring);
      bool ok = true;
      for (int i = 0; i < mine && ok; ++i) {
        Tile w;
        ok = take_tile(bar, i, w);
        if (!ok) break;
        const Share mine_of = share_of(q, w, cta);
        if (mine_of.rows <= 0) continue;
        const int row = (int)mine_of.row0, f = mine_of.f0;
        const int box = w.n > 64 ? 0 : w.n > 32 ? 1 : 2;
        const uint32_t bytes = (kStageA >> box) + 2 * half_bytes;
        const bool wide = plan.width == 256;
        const CUtensorMap* map_w = &maps.w[wide ? 0 : 1];
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (it >= stages) {
            ok = mbar_wait_soon(&bar->empty[s], phase);
            if (!ok) break;
          }
          const uint32_t on = full0 + s * 8, a = ring0 + s * stage_bytes, b = a + kStageA;
          mbar_arrive_expect_tx(&bar->full[s], bytes);
          const int d = kb * kDepth;
          const int second = MODE == kInputGrad && kb >= q.p.Nb;  // up's half of the terms
          // half h of the weights: 128 bytes by width / 2
          const auto half_at = [&](int h, int (&c)[3]) {
            if (MODE == kInputGrad) {
              c[0] = f + (wide ? h * 128 : 0);
              c[1] = d - second * q.p.Nb * kDepth + (wide ? 0 : h * 64);
              c[2] = second;
            } else {
              c[0] = d;
              c[1] = kGated ? f : f + h * (plan.width / 2);
              c[2] = kGated ? h : 0;
            }
          };
          int c[3];
          half_at(0, c);
          tma_own_4d(b, map_w, c[0], c[1], c[2], w.g, on);
          half_at(1, c);
          tma_own_4d(b + half_bytes, map_w, c[0], c[1], c[2], w.g, on);
          tma_own_2d(a, &maps.rows[box], d, row, on);
          ++it;
          if (++s == stages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      // the products' arrivals, before this CTA may leave
      for (int i = 0; i < stages && i < it && ok; ++i) {
        s = s == 0 ? stages - 1 : s - 1;
        ok = mbar_wait_soon(&bar->empty[s], ((it - 1 - i) / stages) & 1);
      }
      if (!ok) {
        atomicOr(timeout, kErrLinearTimeout);
        // copies in flight must land before the CTAs leave
        for (int i = 0; i < stages && i < it; ++i)
          (void)mbar_wait(&bar->full[(it - 1 - i) % stages], ((it - 1 - i) / stages) & 1);
      }
    } else if (warp == 1) {
      // ---------------------------------------------- MMA: one lane issues, the warp waits.
      // After a wait that gave up it issues nothing, but meets the epilogue as often
      // as ever, and so do the epilogue's warps: the hardware barriers have no limit.
      // `met` says how far it has come, sums or none.
      constexpr bool kMnB = MODE == kInputGrad;
      constexpr uint32_t kStepA = 32 >> 4, kStepB = (kMnB ? 4096 : 32) >> 4;
      const uint32_t stage_units = (uint32_t)stage_bytes >> 4;
      const uint64_t op_a = smem_operand(smem_addr(ring), 16);
      const uint64_t op_b = smem_operand(smem_addr(ring) + kStageA, kMnB ? 128 * kDepth : 16);
      const uint32_t a0 = (uint32_t)op_a, a_high = (uint32_t)(op_a >> 32);
      const uint32_t b0 = (uint32_t)op_b, b_high = (uint32_t)(op_b >> 32);
      const uint32_t empty0 = smem_addr(&bar->empty[0]), sum0 = smem_addr(&bar->acc_full[0]);
      const uint32_t full0 = smem_addr(&bar->full[0]);
      const uint32_t form = mma8_form(plan.width, kMnB);
      int n_acc = 0, issued = 0;             // sums met for, sums that are made
      uint32_t s = 0, phase = 0;             // the ring's place
      bool ok = true, ready = false;         // ready: that place was seen to be full
      for (int i = 0; i < mine; ++i) {
        Tile w;
        if (ok) ok = warp_take_tile(bar, i, w, lane);
        if (!ok) w = qtile_at<kGated>(q, plan, first, begins, counts, sizes, pair + i * pairs);
        if (share_of(q, w, cta).rows <= 0) continue;
        for (int kb = w.kb0; kb < w.kb1; ++kb, ++n_acc) {
          if (ok && !__all_sync(kFull, ready)) ok = warp_wait(&bar->full[s], phase);
          if (n_acc >= 2) named_sync(1 + (n_acc & 1), kHandover);
          if (ok) {
            tc_fence_after();
            if (lane == 0) {
              mma8_stage<kStepA, kStepB>(tmem + (n_acc & 1) * 256, a0 + s * stage_units, a_high,
                                         b0 + s * stage_units, b_high, form);
              mma8_commit(sum0 + (n_acc & 1) * 8);
              mma8_commit(empty0 + s * 8);
            }
            __syncwarp();
            issued = n_acc + 1;
            if (++s == (uint32_t)stages) {
              s = 0;
              phase ^= 1;
            }
            ready = mbar_test(full0 + s * 8, phase);       // its answer comes under the MMAs
          }
          if (lane == 0) *const_cast<volatile uint32_t*>(&bar->met) = n_acc + 1;
        }
      }
      for (int last = n_acc < 2 ? 0 : n_acc - 2; last < n_acc; ++last) named_sync(1 + (last & 1), kHandover);
      // no sum may be on its way when the CTA gives its tensor memory back: the epilogue,
      // if told of sums that nobody had seen, is no witness
      if (issued > 0) ok = warp_wait(&bar->acc_full[(issued - 1) & 1], ((issued - 1) >> 1) & 1) && ok;
      if (!ok && lane == 0) atomicOr(timeout, kErrLinearTimeout);
    } else if (warp == 2) {
      // ---------------------------------------------- sums: looks for each and tells the epilogue.
      // After a wait that gave up it tells it of all sums, as the others meet as often as
      // ever, but of none before the MMA warp has come to it: told of the next but one too
      // early, a warp would count twice in a meeting that another has not come to yet.
      int n_acc = 0;
      bool ok = true;
      for (int i = 0; i < mine; ++i) {
        Tile w;
        if (ok) ok = warp_take_tile(bar, i, w, lane);
        if (!ok) w = qtile_at<kGated>(q, plan, first, begins, counts, sizes, pair + i * pairs);
        if (share_of(q, w, cta).rows <= 0) continue;
        for (int kb = w.kb0; kb < w.kb1; ++kb, ++n_acc) {
          if (ok) ok = warp_wait(&bar->acc_full[n_acc & 1], (n_acc >> 1) & 1);
          if (!ok) {
            if (lane == 0) bar->failed = 1;
            wait_met(bar, n_acc);
          }
          tc_fence_after();
          tc_fence_before();
          __syncwarp();
          named_arrive(3 + (n_acc & 1), kHandover);
        }
      }
      if (!ok && lane == 0) atomicOr(timeout, kErrLinearTimeout);
    } else if (warp == 3 && elect_one()) {
      // ---------------------------------------------- works out the tiles, ahead of all roles
      bool ok = true;
      for (int i = 0; i < mine; ++i) {
        const int slot = i % kSlots;
        if (i >= kSlots) {
          ok = mbar_wait_soon(&bar->tile_empty[slot], (i / kSlots - 1) & 1);
          if (!ok) break;
        }
        bar->tiles[slot] = qtile_at<kGated>(q, plan, first, begins, counts, sizes, pair + i * pairs);
        mbar_arrive(&bar->tile_full[slot]);
      }
      if (!ok) atomicOr(timeout, kErrLinearTimeout);
    }
  } else {
    registers_more<kRegistersMore>();
    // ------------------------------------------------ epilogue
    // Blocks of 32 columns: four (256 columns) or two of this warp's half; with SwiGLU
    // blocks 0 and 2 are gates, 1 and 3 the same features' up values.
    const int quad = warp & 3, turn = (warp - 4) >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const int sub = plan.width / 128;                     // half as many blocks
    float* room = rooms + (warp - 4) * kTurnWords;
    int n_acc = 0;
    uint32_t meeting = 0;
    bool ok = true;
    for (int i = 0; i < mine; ++i) {
      const int u = pair + i * pairs;
      Tile w;
      if (ok) ok = warp_take_tile(bar, i, w, lane);
      if (!ok) w = qtile_at<kGated>(q, plan, first, begins, counts, sizes, u);
      const Share share = share_of(q, w, cta);
      if (share.rows <= 0 || w.kb0 >= w.kb1) continue;
      const int mine_rows = share.rows - quad * 32;       // from this warp's on
      const int64_t row0 = share.row0 + quad * 32;
      const int col0 = share.f0 + turn * (kGated ? plan.width / 4 : plan.width / 2);
      // this lane's scales and its features', kScaleGroup stages ahead
      const float* row_scales = q.row_scale + (row0 + min(lane, max(mine_rows, 1) - 1)) * q.row_ld;
      const float* w_scales = q.p.ws + w.g * q.group_ld +
                              (int64_t)min(col0 / 128, q.feature_blocks - 1) * q.feature_ld;
      float by[kScaleGroup], by_up[kScaleGroup], next[kScaleGroup], next_w[kScaleGroup], next_up[kScaleGroup];
      auto fetch = [&](int kb) {
#pragma unroll
        for (int j = 0; j < kScaleGroup; ++j) {
          next[j] = next_w[j] = next_up[j] = 0.0f;
          if (mine_rows > 0 && kb + j < w.kb1) {
            next[j] = row_scales[kb + j];
            next_w[j] = w_scales[(int64_t)(kb + j) * q.block_ld];
            if (kGated) next_up[j] = w_scales[q.up + (int64_t)(kb + j) * q.block_ld];
          }
        }
      };
      // Scales whose product is no normal number stay apart: order_scales. Whether a group of
      // stages may have such is a look at the products, or, with gates, which have twice
      // as many, at scales beyond 2^-63 to 2^63: the rows' each time, the weights' here.
      uint32_t key_w = 0;
      constexpr uint32_t kLow = kGated ? 64 : 1, kHigh = kGated ? 190 : 255;
      if (kGated) {
        for (int kb = w.kb0 + lane; kb < w.kb1; kb += 32) {
          const float* of_w = w_scales + (int64_t)kb * q.block_ld;
          key_w = max(key_w, max(scale_key(of_w[0], kLow), scale_key(of_w[q.up], kLow)));
        }
      }
      fetch(w.kb0);
      float sum[4][32];
#pragma unroll
      for (int h = 0; h < 4; ++h)
#pragma unroll
        for (int c = 0; c < 32; ++c) sum[h][c] = 0.0f;
      int left = 0;                                       // scales that are there
      bool outside = false;                               // some of a group's may be such
      int known = 0;                                      // where they may: 1 none has, 2 some have
      for (int kb = w.kb0; kb < w.kb1; ++kb, ++n_acc, --left) {
        if (left == 0) {
          uint32_t key = key_w;
#pragma unroll
          for (int j = 0; j < kScaleGroup; ++j) {
            by[j] = next[j] * next_w[j];
            by_up[j] = next[j] * next_up[j];
            key = max(key, scale_key(kGated ? next[j] : by[j], kLow));
          }
          outside = __any_sync(kFull, key >= key_range(kLow, kHigh));
          known = 0;
          left = kScaleGroup;
          fetch(kb + kScaleGroup);
        }
        __syncwarp();
        named_sync(3 + (n_acc & 1), kHandover);
        tc_fence_after();
        const float scale = by[0], scale_up = by_up[0];
#pragma unroll
        for (int j = 0; j + 1 < kScaleGroup; ++j) {
          by[j] = by[j + 1];
          by_up[j] = by_up[j + 1];
        }
        const uint32_t at = lanes + (n_acc & 1) * 256 + turn * (kGated ? plan.width / 4 : plan.width / 2);
        __syncwarp();
        if (mine_rows > 0 && ok) {
          // 16 columns' loads are on their way under the arithmetic of the 16 before:
          // tensor memory gives 64 bytes a cycle to each quarter of the SM
          float r[2][16];
          const auto column_of = [&](int c) {             // of piece c of 16 columns
            return kGated ? (c >> 1 & 1) * (plan.width / 2) + (c >> 2) * 32 + (c & 1) * 16 : c * 16;
          };
          bool apart = false;
          if (__builtin_expect(outside, 0)) {
            if (known == 0) {                             // zeros, or products that are normal all the same
              bool any = false;
              for (int j = 0; j < left && kb + j < w.kb1; ++j) {
                const float row = row_scales[kb + j], *of_w = w_scales + (int64_t)(kb + j) * q.block_ld;
                any |= scales_apart(row, of_w[0], row * of_w[0]);
                if (kGated) any |= scales_apart(row, of_w[q.up], row * of_w[q.up]);
              }
              known = __any_sync(kFull, any) ? 2 : 1;
            }
            apart = known == 2;
          }
          const auto add = [&](auto which, float first, float first_up, float second, float second_up) {
            constexpr bool APART = decltype(which)::value;
            tmem_begin16(at, r[0]);
            tmem_wait16(r[0]);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              if (c >= 4 && sub == 1) continue;
              const bool more = c != 7 && (c != 3 || sub == 2);
              if (more) tmem_begin16(at + column_of(c + 1), r[(c + 1) & 1]);
              const bool is_up = kGated && (c >> 1 & 1);
              const float by_c = is_up ? second_up : second;
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const float v = APART ? r[c & 1][k] * (is_up ? first_up : first) : r[c & 1][k];
                sum[c / 2][(c & 1) * 16 + k] = fmaf(v, by_c, sum[c / 2][(c & 1) * 16 + k]);
              }
              if (more) tmem_wait16(r[(c + 1) & 1]);
            }
          };
          if (__builtin_expect(!apart, 1)) {
            add(std::false_type(), 1.0f, 1.0f, scale, scale_up);
          } else {
            const float row = row_scales[kb], *of_w = w_scales + (int64_t)kb * q.block_ld;
            float first, second, first_up = 1.0f, second_up = 0.0f;
            order_scales(row, of_w[0], first, second);
            if (kGated) order_scales(row, of_w[q.up], first_up, second_up);
            add(std::true_type(), first, first_up, second, second_up);
          }
        }
        tc_fence_before();
        __syncwarp();
        named_arrive(1 + (n_acc & 1), kHandover);
      }
      if (*const_cast<volatile uint32_t*>(&bar->failed)) ok = false;
      if (!ok) continue;
      // the values of this part: the tile's result, or sums for the part that finishes
      // last, which then adds all of them in their order
      if (w.parts == 1) {
        if (mine_rows <= 0) continue;
#pragma unroll
        for (int h = 0; h < 4; h += kGated ? 2 : 1) {
          const int col = col0 + (kGated ? h / 2 : h) * 32;
          if (h >= 2 * sub || col >= q.outs) continue;
          finish<MODE, ACT, T>(q, room, w.g, row0, mine_rows, col, lane, sum[h], sum[(h + 1) & 3]);
        }
        continue;
      }
      // this lane's place in the pair's (a pair has one unit where there are parts, of
      // tiles of 128 columns)
      float* sums = q.p.partial + ((int64_t)pair * 128 * 256 + cta * 128 + quad * 32 + lane);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int column = (kGated ? h * 64 : h * 32) + turn * (kGated ? 32 : 64);
#pragma unroll
        for (int c = 0; c < 32; ++c) put(sums + (column + c) * 256, sum[h][c], lane < mine_rows);
      }
      ok = epilogue_meet(bar, lane, meeting);
      if (!ok) continue;
      if (threadIdx.x == 128) {
        unsigned int* ticket = q.p.tickets + quotient(u, plan.splits) * 2 + cta;
        const bool last = ticket_take(ticket) == (unsigned)w.parts - 1;
        if (last) *ticket = 0u;
        bar->last = last;
      }
      ok = epilogue_meet(bar, lane, meeting);
      if (!ok || !bar->last || mine_rows <= 0) continue;
      const float* parts = sums - (int64_t)w.part * 128 * 256;
      const int there = lane < mine_rows ? 32 : 0;        // a lane without a row reads nothing
#pragma unroll 1
      for (int h = 0; h < (kGated ? 1 : 2); ++h) {
        const int col = col0 + h * 32;
        if (col >= q.outs) continue;
        const int column = h * 32 + turn * (kGated ? 32 : 64);
        float z[32], up[32];
        add_parts(parts + column * 256, 128 * 256, w.parts, there, z);
        if (kGated) add_parts(parts + (column + 64) * 256, 128 * 256, w.parts, there, up);
        finish<MODE, ACT, T>(q, room, w.g, row0, mine_rows, col, lane, z, up);
      }
    }
    if (!ok && lane == 0) atomicOr(timeout, kErrLinearTimeout);
  }
  __syncwarp();
  __syncthreads();
  if (warp == 1) tmem_free_own(tmem, kTmemColumns);
}

// ---------------------------------------------------------------------- host

template <int MODE, int ACT, typename T>
cudaError_t launch_tiles(const Maps& maps, MmaParams& q, int grid, cudaStream_t st) {
  const auto whole = [](const void* p) { return (uintptr_t)p % 32 == 0; };
  q.vec = q.outs % 16 == 0 && whole(q.out) && whole(q.p.residual) && whole(q.p.z);
  constexpr size_t kOther = 1024 + kRingBytes + kTurnBytes + sizeof(Barriers);
  constexpr size_t kMost = kOther + EP_MAX_EXPERTS * kGroupBytes;
  static_assert(kMost <= 227 * 1024 - 512, "shared memory");
  static std::atomic<uint64_t> raised{0};
  const auto kernel = product8_kernel<MODE, ACT, T>;
  // the epilogue's warps ask for registers that the block has to have been launched
  // with, or they would wait for ever
  static std::atomic<int> checked{0};
  if (!checked.load(std::memory_order_relaxed)) {
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, kernel);
    if (e != cudaSuccess) return e;
    if (a.numRegs < kRegisters) return cudaErrorInvalidKernelImage;
    checked.store(1, std::memory_order_relaxed);
  }
  const cudaError_t e = raise_shared_limit(kernel, kMost, &raised);
  if (e != cudaSuccess) return e;
  return launch_overlapped(kernel, dim3((unsigned)grid), kThreads, kOther + (size_t)q.p.s.G * kGroupBytes, st,
                           maps, q);
}

template <typename T>
cudaError_t launch_forward(const Maps& m, MmaParams& q, int grid, cudaStream_t st) {
  switch (q.p.act) {
    case EP_ACT_RELU: return launch_tiles<kForward, EP_ACT_RELU, T>(m, q, grid, st);
    case EP_ACT_SILU: return launch_tiles<kForward, EP_ACT_SILU, T>(m, q, grid, st);
    case EP_ACT_GELU: return launch_tiles<kForward, EP_ACT_GELU, T>(m, q, grid, st);
    case EP_ACT_SWIGLU: return launch_tiles<kForward, EP_ACT_SWIGLU, T>(m, q, grid, st);
    default: return launch_tiles<kForward, EP_ACT_NONE, T>(m, q, grid, st);
  }
}

// What both products set: the grid, and a dense product's plan.
int plan_grid(MmaParams& q, bool gated, int sms) {
  const LinearSegs& s = q.p.s;
  const int64_t rows = s.begin ? s.pool : s.dense_rows;
  const int each = results_in(128, gated), parts = q.stages / kLeast;
  const int64_t most = (rows / kTileRows + s.G) * ((q.outs + each - 1) / each) *
                       (parts < 1 ? 1 : parts < kMaxSplits ? parts : kMaxSplits);
  const int grid = grid_of(sms, most), pairs = grid_of(sms, INT_MAX) / 2;
  q.pairs = pairs;
  QPlan& plan = q.plan;
  const int dense = (int)s.dense_rows;
  plan.size = tile_rows(dense, kTileRows, host_quotient);
  const int above = (dense + plan.size - 1) / plan.size;
  plan.width = 256;
  plan.tiles = above * tiles_beside(q.outs, 256, gated, dense, host_quotient);
  if (2 * plan.tiles <= pairs) {
    plan.width = 128;
    plan.tiles = above * tiles_beside(q.outs, 128, gated, dense, host_quotient);
  }
  plan.splits = plan.width == 128 ? splits_for(grid / 2, plan.tiles, q.stages, kWorth, kLeast) : 1;
  return grid;
}

// Maps of both operands: rows of codes in boxes of 128, 64 and 32 rows; W [G][parts][N][K]
// in boxes of 128 bytes by 128 or 64 rows.
bool make_maps(Maps* m, const QLinearParams& p, const uint8_t* rows, int64_t cols) {
  const int64_t count = p.s.begin ? p.s.pool : p.s.dense_rows;
  const int64_t row_dims[2] = {cols, count}, row_strides[2] = {1, cols};
  const int64_t dims[4] = {p.K, p.N, p.Nw / p.N, p.s.G};
  const int64_t strides[4] = {1, p.K, (int64_t)p.N * p.K, (int64_t)p.Nw * p.K};
  bool ok = true;
  for (int i = 0; i < 3; ++i) {
    const int box[2] = {kDepth, 128 >> i};
    ok = ok && make_map(&m->rows[i], rows, 2, row_dims, row_strides, box, 1);
  }
  for (int i = 0; i < 2; ++i) {
    const int box[4] = {kDepth, 128 >> i, 1, 1};
    ok = ok && make_map(&m->w[i], p.w, 4, dims, strides, box, 1);
  }
  return ok;
}

}  // namespace

cudaError_t launch_qlinear_forward(const QLinearParams& p, int sms, cudaStream_t st) {
  MmaParams q;
  q.p = p;
  q.out = p.y;
  q.outs = p.N;
  q.stages = p.Kb;
  q.row_scale = p.xs;
  q.row_ld = p.Kb;
  q.group_ld = (int64_t)p.Sw * p.Kb;
  q.feature_ld = p.Kb;
  q.block_ld = 1;
  q.feature_blocks = p.Nb;
  q.up = p.Nb * p.Kb;
  Maps m;
  if (!make_maps(&m, p, p.x, p.K)) return cudaErrorInvalidValue;
  const int grid = plan_grid(q, p.act == EP_ACT_SWIGLU, sms);
  return p.y_f32 ? launch_forward<float>(m, q, grid, st) : launch_forward<__nv_bfloat16>(m, q, grid, st);
}

cudaError_t launch_qlinear_input_grad(const QLinearParams& p, int sms, cudaStream_t st) {
  MmaParams q;
  q.p = p;
  q.out = p.dx;
  q.outs = p.K;
  q.stages = p.Sw;
  q.row_scale = p.dzs;
  q.row_ld = p.Sw;
  q.group_ld = (int64_t)p.Sw * p.Kb;
  q.feature_ld = 1;
  q.block_ld = p.Kb;
  q.feature_blocks = p.Kb;
  q.up = 0;
  Maps m;
  if (!make_maps(&m, p, p.dz8, (int64_t)p.Sw * kDepth)) return cudaErrorInvalidValue;
  const int grid = plan_grid(q, false, sms);
  return launch_tiles<kInputGrad, EP_ACT_NONE, __nv_bfloat16>(m, q, grid, st);
}

}  // namespace ep
