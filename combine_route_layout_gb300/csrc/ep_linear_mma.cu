// The three products of an expert layer on the tensor cores: z = x W^T,
// dx = dz W, dW = dz^T x, with the forward's bias, activation and residual in
// the epilogue.
//
// Every output is computed transposed: the tensor core's M side is the
// output's contiguous axis (features), its N side the rows (tokens, or dW's
// rows). That way the weights always fill M = 256, a tile takes as many rows
// as an expert has (N in steps of 32, so ragged experts waste no arithmetic
// and few-row experts cost weight traffic alone), a lane of the accumulator is
// one feature (one bias value per thread) and a warp stores 32 consecutive
// features of a row.
//
// A pair of CTAs (two SMs) shares one tile of 256 features x up to 256 rows:
// each stages its 128 features and its half of the rows, 64 terms at a time,
// by TMA with 128-byte swizzle into a ring of stages; one thread of the even
// CTA issues the MMAs, the accumulators (two, so that a tile's epilogue runs
// under the next one's products) stay in TMEM. Grid: one CTA per SM, each pair
// walks the tiles of all groups. A pair reads 64 KB a stage for 8.4 MFLOP; tiles
// of one CTA alone would read half as much again.
//
// Roles by warp: 0 TMA, 1 MMA, 2 clears the tails of dW's contractions, 3 works
// out the tiles, 4-11 epilogue (TMEM lanes go by warp % 4; the two warps of a
// quarter take every other 32 columns). TMA, MMA and tiles are one thread each,
// whose loop must take less than a stage's products, 512 cycles: it takes about
// 280, and an epilogue's warps beside it slow it down.
//
// What bounds it. Long products run at the tensor core's rate in cycles (512 a
// stage) and at the power limit in time: 32768 x 4096 x 4096 dense 1.73 PFLOP/s at
// 1.6 GHz (the library's product 1.77); 128 experts of 973 rows, 4096 x 4096,
// SwiGLU with pre-activation, 1.42-1.47 at 1.3 GHz, where the experts' weights
// come from HBM as well. From idle clocks: 8192^3 1.9 PFLOP/s. Few rows an expert:
// HBM (256 experts x 32 rows, 7168 x 1024: 6.5 TB/s). Small products: set-up and
// pipeline latency (about 6 us, part of it under the kernel before) and the stages
// of a tile one after another.
#include <atomic>
#include <climits>
#include <cstring>

#include "ep_linear_tiles.cuh"

namespace ep {
namespace {

constexpr int kDepth = 64;                       // terms per stage: 128 bytes of bf16
constexpr int kStageA = 128 * kDepth * 2;        // bytes of a CTA's 128 features
constexpr int kStageB = 128 * kDepth * 2;        // bytes of a CTA's half of the rows
// The ring holds 6 stages of 256 rows, 8 of 128 or 9 of 64: products of few rows
// wait for their loads' latency, and more of them are on their way (1024 x 7168 x
// 256: 14.1 us, 15.1 with 6; dW of 4096 rows, 2048 x 1024: 19.8 and 22.2).
constexpr int kRingBytes = 6 * (kStageA + kStageB);
constexpr int kMaxStages = 9;
// f32 outputs: the tensor core cuts off what its accumulator cannot hold, an
// error that grows with the number of steps to the power 3/2 (7168 terms: 8e-6 of
// the result); sums of 512 terms are added up in registers instead, which
// leaves 4.5e-7.
constexpr int kChunk32 = 8;                      // stages of such a sum
constexpr int kLongStages = kLongTerms / kDepth; // bf16 outputs: stages of a sum
constexpr int kTmemColumns = 512;                // two accumulators

struct MmaParams {
  static constexpr int kDepth = ep::kDepth;
  LinearParams p;
  void* out;         // y, dx or dW
  int features;      // length of the output's contiguous axis (weight rows or K)
  int f_tiles;       // 256-feature tiles
  int r_tiles;       // dW: tiles of `cap` rows of each group (else by the group's count)
  int cap;           // most rows of a tile
  int terms;         // of a contraction (dW: the group's rows)
  int a_blocks;      // MN-major operands: the map cuts rows into blocks of 64
  int b_blocks;      // elements, so that one box takes two of them
  int pairs_out, pairs_z;   // bf16 outputs whose rows allow two features a store
  Plan plan;         // of a dense product
  float* partial;    // sums of parts and of long contractions: [pair][column][256 features]
  unsigned int* tickets;   // parts that are done: [tile][2], zero between calls
};

struct Barriers {
  uint64_t full[kMaxStages];  // both CTAs' operands have landed (even CTA's)
  uint64_t empty[kMaxStages]; // this CTA's stage may be written again
  uint64_t landed;            // dW: this CTA's last block has landed; its tail is to be cleared
  uint64_t acc_full[2];       // the MMAs of a sum are complete
  uint64_t acc_empty[2];      // even CTA's: both CTAs' epilogues are done
  uint64_t tile_full[kSlots], tile_empty[kSlots];
  uint64_t joined;            // the epilogue's warps meet
  Tile tiles[kSlots];
  uint32_t tmem;
  uint32_t last;              // this CTA's part of a tile was the last
};

// Whether stage kb is dW's last and ends inside a 16-term step.
template <int MODE>
__device__ __forceinline__ bool has_tail(const Tile& w, int kb) {
  const int valid = w.terms - kb * kDepth;
  return MODE == kWeightGrad && valid < kDepth && (valid & 15);
}

// An accumulator's sum is there (a thread of the even CTA passes the news on), and
// has been read. What these barriers guard lies in tensor memory alone, and the
// tensor core's own fences order it with the arrivals and waits between them, which
// need cluster scope, since they meet threads of both CTAs, and no release: one
// costs 0.4 to 0.5 us each time (1024 x 7168 x 256: 15.7 us for 13.8).
__device__ __forceinline__ bool accumulator_ready(Barriers* bar, int acc, int n_acc, int cta) {
  if (!warp_wait_cluster(&bar->acc_full[acc], (n_acc >> 1) & 1)) return false;
  tc_fence_after();
  if (cta == 0 && threadIdx.x == 128) {
    tc_fence_before();
    mbar_signal_at(in_cta(&bar->acc_full[acc], 1));
  }
  __syncwarp();
  return true;
}

__device__ __forceinline__ void accumulator_free(Barriers* bar, int acc, int lane) {
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_signal_at(in_cta(&bar->acc_empty[acc], 0));
}

// Maps of the two operands. A K-major operand's rows come in boxes of 128, 64,
// 32 or 16 rows, the smallest that holds a CTA's half of the tile: one TMA
// instruction each (with boxes of 16 rows alone, seven for 112 rows, ragged
// experts' products took 3.82 ms where full tiles take 3.1).
struct Maps {
  CUtensorMap a;
  CUtensorMap b[4];
};

template <int MODE, int ACT, typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ Maps maps, MmaParams q) {
  constexpr bool kGated = MODE == kForward && ACT == EP_ACT_SWIGLU;
  constexpr bool kChunked = sizeof(T) == 4;
  extern __shared__ uint8_t raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
  Barriers* bar = reinterpret_cast<Barriers*>(ring + kRingBytes);
  int* first = reinterpret_cast<int*>(bar + 1);
  int* begins = first + q.p.s.G;
  int* counts = begins + q.p.s.G;
  int* sizes = counts + q.p.s.G;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t cta = cluster_rank();
  int32_t* timeout = q.p.s.err;

  // one thread a barrier
  if (threadIdx.x < kMaxStages) {
    mbar_init(&bar->full[threadIdx.x], 2);       // each CTA's producer
    mbar_init(&bar->empty[threadIdx.x], 1);
  } else if (threadIdx.x < kMaxStages + 2) {
    mbar_init(&bar->acc_full[threadIdx.x - kMaxStages], 1);
    mbar_init(&bar->acc_empty[threadIdx.x - kMaxStages], 2 * kEpilogueWarps);  // of both CTAs
  }
  if (threadIdx.x >= 32 && threadIdx.x < 32 + kSlots) {
    // producer, the epilogue's warps, MMA (even CTA), tails (dW)
    mbar_init(&bar->tile_full[threadIdx.x - 32], 1);
    mbar_init(&bar->tile_empty[threadIdx.x - 32],
              1 + kEpilogueWarps + (cta == 0 ? 1 : 0) + (MODE == kWeightGrad ? 1 : 0));
  } else if (threadIdx.x == 32 + kSlots) {
    mbar_init(&bar->landed, 1);
    mbar_init(&bar->joined, kEpilogueWarps);
  }
  if (threadIdx.x < 64) mbar_init_fence();
  if (threadIdx.x == 64) {
    tma_prefetch_map(&maps.a);
    tma_prefetch_map(&maps.b[0]);
  }
  __syncthreads();
  cluster_arrive();                      // the barriers are ready; the wait is below
  if (warp == 1) tmem_alloc(&bar->tmem, kTmemColumns);
  begin_overlapped();
  const Plan plan = plan_tiles<MODE>(q, first, begins, counts, sizes);
  const int units = plan.tiles * plan.splits;
  const int stage_bytes = kStageA + plan.cap / 2 * kDepth * 2;
  const int stages = min(kMaxStages, kRingBytes / stage_bytes);
  // dW: the last stage of a contraction, whose tail has to be cleared, has a
  // place beside the ring, so that the time this takes passes under the others
  const int tail_place = stages - 1, ring_stages = MODE == kWeightGrad ? tail_place : stages;
  tc_fence_before();
  __syncthreads();                       // the TMEM address is there
  tc_fence_after();
  cluster_wait();
  const uint32_t tmem = bar->tmem;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int mine = pair < units ? (units - 1 - pair) / pairs + 1 : 0;   // this pair's units

  if (warp == 0 && elect_one()) {
    // ------------------------------------------------ producer: one thread
    int it = 0, s = 0, tails = 0;           // stages written so far, the ring's place
    uint32_t phase = 1;                     // the first pass over the ring waits for nothing
    const uint32_t full0 = in_cta(&bar->full[0], 0), empty0 = in_cta(&bar->empty[0], 1);
    const uint32_t ring0 = smem_addr(ring), own0 = smem_addr(&bar->empty[0]);
    bool ok = true, ready = false;          // ready: the place was seen to be free
    for (int i = 0; i < mine && ok; ++i) {
      Tile w;
      ok = take_tile(bar, i, w);
      if (!ok) break;
      const int half = w.n / 2;
      const int fc = w.f0 + (int)cta * 128;                     // this CTA's features
      const int rc = w.r0 + (int)cta * half;                    // this CTA's rows
      const int box = MODE == kWeightGrad ? 0 : half > 64 ? 0 : half > 32 ? 1 : half > 16 ? 2 : 3;
      const uint32_t bytes = kStageA + (MODE != kWeightGrad || q.b_blocks ? kStageB >> box
                                                                          : half / 64 * 8192);
      const CUtensorMap* map_b = &maps.b[box];
      // stage kb's operands into place `to`, their bytes on barrier `on`
      auto load = [&](int kb, int to, uint32_t on) {
        const uint32_t a = ring0 + to * stage_bytes, b = a + kStageA;
        const int d = kb * kDepth;
        const int row = (int)w.begin + d;                       // dW: contraction row
        if (MODE == kForward) {
          if (kGated) {
            tma_load_4d(a, &maps.a, d, 0, fc / 2, w.g, on);
          } else {
            tma_load_3d(a, &maps.a, d, fc, w.g, on);
          }
        } else if (MODE == kInputGrad) {
          if (q.a_blocks) {
            tma_load_4d(a, &maps.a, 0, d, fc / 64, w.g, on);
          } else {
            tma_load_3d(a, &maps.a, fc, d, w.g, on);
            tma_load_3d(a + 8192, &maps.a, fc + 64, d, w.g, on);
          }
        } else if (q.a_blocks) {
          tma_load_3d(a, &maps.a, 0, row, fc / 64, on);
        } else {
          tma_load_2d(a, &maps.a, fc, row, on);
          tma_load_2d(a + 8192, &maps.a, fc + 64, row, on);
        }
        if (MODE != kWeightGrad) {
          tma_load_2d(b, map_b, d, (int)w.begin + rc, on);
        } else if (q.b_blocks) {
          tma_load_3d(b, map_b, 0, row, rc / 64, on);
        } else {
          tma_load_2d(b, map_b, rc, row, on);
          if (half == 128) tma_load_2d(b + 8192, map_b, rc + 64, row, on);
        }
      };
      const bool tail = has_tail<MODE>(w, w.kb1 - 1);
      const int end = w.kb1 - (tail ? 1 : 0);
      // once the ring is full of this tile's stages, the place of the last
      // tile's tail is free or soon will be
      const int tail_at = min(w.kb0 + ring_stages, end);
      for (int kb = w.kb0; kb < w.kb1; ++kb) {
        if (tail && kb == tail_at) {
          if (tails > 0) {
            ok = mbar_wait_soon(&bar->empty[tail_place], (tails - 1) & 1);
            if (!ok) break;
            if (cta == 0) mbar_signal_at(empty0 + tail_place * 8);
          }
          ++tails;
          mbar_arrive_expect_tx(&bar->landed, bytes);
          load(w.kb1 - 1, tail_place, smem_addr(&bar->landed));
        }
        if (kb == end) break;
        if (it >= ring_stages) {
          if (!ready) ok = mbar_wait_soon(&bar->empty[s], phase);
          if (!ok) break;
          if (cta == 0) mbar_signal_at(empty0 + s * 8);
        }
        const int to = s;
        ++it;
        if (++s == ring_stages) {
          s = 0;
          phase ^= 1;
        }
        ready = it >= ring_stages && mbar_test(own0 + s * 8, phase);   // its answer comes under the loads
        mbar_signal_expect_tx_at(full0 + to * 8, bytes);
        load(kb, to, full0 + to * 8);
      }
    }
    if (!ok) {
      atomicOr(timeout, kErrLinearTimeout);
      // copies in flight must land before the CTAs leave
      for (int i = 0; i < ring_stages && i < it; ++i) {
        s = s == 0 ? ring_stages - 1 : s - 1;
        (void)mbar_wait(&bar->full[s], ((it - 1 - i) / ring_stages) & 1);
      }
      if (tails > 0) (void)mbar_wait(&bar->landed, (tails - 1) & 1);
    }
  } else if (warp == 1 && cta == 0 && elect_one()) {
    // ------------------------------------------------ MMA: one thread of the even CTA
    // operands of stage 0; a stage is stage_bytes on, 16 terms are 32 bytes of
    // a row (K-major) or 16 rows (MN-major) on
    constexpr bool kMnA = MODE != kForward, kMnB = MODE == kWeightGrad;
    constexpr uint32_t kStepA = (kMnA ? 2048 : 32) >> 4, kStepB = (kMnB ? 2048 : 32) >> 4;
    const uint32_t stage_units = (uint32_t)stage_bytes >> 4;
    const uint64_t op_a = smem_operand(smem_addr(ring), kMnA ? 8192 : 16);
    const uint64_t op_b = smem_operand(smem_addr(ring) + kStageA, kMnB ? 8192 : 16);
    const uint32_t a0 = (uint32_t)op_a, a_high = (uint32_t)(op_a >> 32);
    const uint32_t b0 = (uint32_t)op_b, b_high = (uint32_t)(op_b >> 32);
    const uint32_t full0 = smem_addr(&bar->full[0]), empty0 = smem_addr(&bar->empty[0]);
    int n_acc = 0, tails = 0;
    uint32_t s = 0, phase = 0;             // the ring's place
    bool ok = true, ready = false;         // ready: that place was seen to be full
    for (int i = 0; i < mine && ok; ++i) {
      Tile w;
      ok = take_tile(bar, i, w);
      if (!ok) break;
      const uint32_t form = mma_form(w.n, kMnA, kMnB);
      const int full_end = min(w.kb1, w.terms / kDepth);   // stages of 64 terms end here
      for (int kb = w.kb0; kb < w.kb1 && ok; ++n_acc) {    // an accumulator's sum
        const int stop = min(w.kb1, kb + (kChunked ? kChunk32 : kLongStages));
        if (n_acc >= 2) {
          ok = mbar_wait_soon_cluster(&bar->acc_empty[n_acc & 1], ((n_acc >> 1) - 1) & 1);
          if (!ok) break;
          tc_fence_after();
        }
        const uint32_t d = tmem + (n_acc & 1) * 256;
        bool accumulate = false;
        for (const int run = min(stop, full_end); kb < run; ++kb) {
          if (!ready) ok = mbar_wait_soon(&bar->full[s], phase);
          if (!ok) break;
          tc_fence_after();
          const uint32_t at = s;
          if (++s == ring_stages) {
            s = 0;
            phase ^= 1;
          }
          ready = mbar_test(full0 + s * 8, phase);         // its answer comes under the MMAs
          mma_stage<kStepA, kStepB>(d, a0 + at * stage_units, a_high, b0 + at * stage_units, b_high,
                                    form, accumulate);
          mma_commit(empty0 + at * 8);
          accumulate = true;
        }
        if (ok && kb < stop) {             // the last stage, of fewer terms
          uint32_t at = s;
          if (has_tail<MODE>(w, kb)) {     // in a place of its own, whose rows both CTAs cleared
            at = tail_place;
            ok = mbar_wait_cluster(&bar->full[tail_place], tails++ & 1);
          } else {
            if (!ready) ok = mbar_wait_soon(&bar->full[s], phase);
            if (++s == ring_stages) {
              s = 0;
              phase ^= 1;
            }
            ready = false;
          }
          if (!ok) break;
          tc_fence_after();
          const uint32_t a = a0 + at * stage_units, b = b0 + at * stage_units;
          const int steps = (w.terms - kb * kDepth + 15) / 16;
          for (int step = 0; step < steps; ++step)
            mma_step(d, a + step * kStepA, a_high, b + step * kStepB, b_high, form,
                     accumulate || step > 0);
          mma_commit(empty0 + at * 8);
          ++kb;
        }
        if (ok) mma_commit(smem_addr(&bar->acc_full[n_acc & 1]));
      }
    }
    if (!ok) atomicOr(timeout, kErrLinearTimeout);
  } else if (MODE == kWeightGrad && warp == 2) {
    // ------------------------------------------------ clears the rows past a segment's last
    // that the last 16-term step of its last stage would take in: they belong
    // to somebody else, and may hold anything
    uint32_t tails = 0;
    bool ok = true;
    for (int i = 0; i < mine && ok; ++i) {
      Tile w;
      ok = warp_take_tile(bar, i, w, lane);
      if (!ok) break;
      if (w.kb0 >= w.kb1 || !has_tail<MODE>(w, w.kb1 - 1)) continue;
      ok = warp_wait(&bar->landed, tails++ & 1);
      if (!ok) break;
      const int valid = w.terms - (w.kb1 - 1) * kDepth, more = (valid + 15) / 16 * 16 - valid;
      uint8_t* stage = ring + tail_place * stage_bytes;
      for (int row = valid + (lane >> 3); row < valid + more; row += 4)
#pragma unroll
        for (int part = 0; part < 4; ++part)                    // 16-byte pieces of a and b
          if (part * 8192 < stage_bytes)
            reinterpret_cast<uint4*>(stage + part * 8192 + row * 128)[lane & 7] = make_uint4(0, 0, 0, 0);
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive_at(in_cta(&bar->full[tail_place], 0));
    }
    if (!ok && lane == 0) atomicOr(timeout, kErrLinearTimeout);
  } else if (warp == 3 && elect_one()) {
    // ------------------------------------------------ works out the tiles, ahead of all roles:
    // a tile's place takes over a thousand cycles of dependent arithmetic
    bool ok = true;
    for (int i = 0; i < mine; ++i) {
      const int slot = i % kSlots;
      if (i >= kSlots) {
        ok = mbar_wait_soon(&bar->tile_empty[slot], (i / kSlots - 1) & 1);
        if (!ok) break;
      }
      bar->tiles[slot] = tile_at<MODE>(q, plan, first, begins, counts, sizes, pair + i * pairs);
      mbar_arrive(&bar->tile_full[slot]);
    }
    if (!ok) atomicOr(timeout, kErrLinearTimeout);
  } else if (warp >= 4) {
    // ------------------------------------------------ epilogue
    // 64 columns of the tile belong to the warp pair of a quarter: 32 to this
    // warp (T f32: at most two such blocks, whose sums it keeps)
    const int quad = warp & 3, turn = (warp - 4) >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    constexpr int kBlocks = kChunked ? kMaxRows / 2 / 64 : 1;
    int n_acc = 0;
    uint32_t meeting = 0;
    bool ok = true;
    for (int i = 0; i < mine && ok; ++i) {
      const int u = pair + i * pairs;
      Tile w;
      ok = warp_take_tile(bar, i, w, lane);
      if (!ok) break;
      const bool whole = w.parts == 1;
      if (w.kb0 >= w.kb1 && (MODE != kWeightGrad || w.part > 0 || w.terms > 0)) continue;
      float b = 0.0f;
      if (MODE == kForward && q.p.bias) {
        const int f = (int)cta * 128 + quad * 32 + lane;
        const float* bias = q.p.bias + (int64_t)w.g * q.p.Nw;
        if (kGated) {
          const int out = w.f0 / 2 + f / 2;
          if (out < q.p.N) b = bias[(f & 1 ? q.p.N : 0) + out];
        } else if (w.f0 + f < q.features) {
          b = bias[w.f0 + f];
        }
      }
      // this lane's column in the pair's place (a pair has one unit where there are parts)
      float* sums = q.partial + ((int64_t)pair * plan.cap * 256 + cta * 128 + quad * 32 + lane);
      const bool none = w.kb0 >= w.kb1;    // a group with no rows: its weight gradient is zero
      float keep[kBlocks][32];
      if (kChunked && !none) {             // the sums of the part's chunks, in their order
        const int chunks = (w.kb1 - w.kb0 + kChunk32 - 1) / kChunk32;
        for (int chunk = 0; chunk < chunks; ++chunk, ++n_acc) {
          const int acc = n_acc & 1;
          ok = accumulator_ready(bar, acc, n_acc, (int)cta);
          if (!ok) break;
#pragma unroll
          for (int h = 0; h < kBlocks; ++h) {
            const int c0 = turn * 32 + h * 64;
            if (c0 >= w.rows) continue;
            float r[32];
            tmem_load32(lanes + acc * 256 + c0, r);
#pragma unroll
            for (int c = 0; c < 32; ++c) keep[h][c] = chunk ? keep[h][c] + r[c] : r[c];
          }
          accumulator_free(bar, acc, lane);
        }
      }
      bool kept = false;                   // sums of a long contraction wait in the pair's place
      if (!kChunked && !none) {
        for (int kb = w.kb0 + kLongStages; kb < w.kb1; kb += kLongStages, ++n_acc, kept = true) {
          ok = accumulator_ready(bar, n_acc & 1, n_acc, (int)cta);
          if (!ok) break;
          for (int c0 = turn * 32; c0 < w.rows; c0 += 64) {
            float r[32];
            __syncwarp();
            tmem_load32(lanes + (n_acc & 1) * 256 + c0, r);
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              r[c] += get(sums + (c0 + c) * 256, kept && c0 + c < w.rows);
              put(sums + (c0 + c) * 256, r[c], c0 + c < w.rows);
            }
          }
          accumulator_free(bar, n_acc & 1, lane);
        }
        if (ok) ok = accumulator_ready(bar, n_acc & 1, n_acc, (int)cta);
      }
      if (!ok) break;
      // first the values of this part: the tile's result, or sums for the part
      // that finishes last, which then adds all of them in their order
      const float* parts_of = nullptr;
      while (true) {
        const bool result = whole || parts_of;
#pragma unroll
        for (int h = 0; h < (kChunked ? kBlocks : 1); ++h)
          for (int c0 = turn * 32 + h * 64; c0 < w.rows; c0 += kChunked ? w.rows : 64) {
            float r[32];
            if (parts_of) {
              add_parts(parts_of + c0 * 256, plan.cap * 256, w.parts, w.rows - c0, r);
            } else if (none) {
#pragma unroll
              for (int c = 0; c < 32; ++c) r[c] = 0.0f;
            } else if (kChunked) {
#pragma unroll
              for (int c = 0; c < 32; ++c) r[c] = keep[h][c];
            } else {
              __syncwarp();
              tmem_load32(lanes + (n_acc & 1) * 256 + c0, r);
              if (kept) {
#pragma unroll
                for (int c = 0; c < 32; ++c) r[c] += get(sums + (c0 + c) * 256, c0 + c < w.rows);
              }
            }
            if (result) {
              epilogue<MODE, ACT, T>(q, w, (int)cta, lane, quad, c0, r, b);
            } else {
#pragma unroll
              for (int c = 0; c < 32; ++c) put(sums + (c0 + c) * 256, r[c], c0 + c < w.rows);
            }
          }
        if (!kChunked && !none && !parts_of) {
          accumulator_free(bar, n_acc & 1, lane);
          ++n_acc;
        }
        if (result) break;
        ok = epilogue_meet(bar, lane, meeting);
        if (!ok) break;
        if (threadIdx.x == 128) {
          unsigned int* ticket = q.tickets + quotient(u, plan.splits) * 2 + cta;
          const bool last = ticket_take(ticket) == (unsigned)w.parts - 1;
          if (last) *ticket = 0u;
          bar->last = last;
        }
        ok = epilogue_meet(bar, lane, meeting);
        if (!ok || !bar->last) break;
        parts_of = sums - (int64_t)w.part * plan.cap * 256;
      }
    }
    if (!ok && lane == 0) atomicOr(timeout, kErrLinearTimeout);
  }
  __syncwarp();
  __syncthreads();
  cluster_arrive();   // the other CTA may still arrive on this one's barriers
  cluster_wait();
  if (warp == 1) tmem_free(tmem, kTmemColumns);
}

// ---------------------------------------------------------------------- host

bool map_rows(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t ld, int box_rows) {
  const int64_t dims[2] = {cols, rows}, strides[2] = {1, ld};
  const int box[2] = {kDepth, box_rows};
  return make_map(m, base, 2, dims, strides, box);
}

// Rows of a K-major operand, in boxes of 128, 64, 32 and 16 rows.
bool map_k_major(CUtensorMap (&m)[4], const void* base, int64_t cols, int64_t rows, int64_t ld) {
  bool ok = true;
  for (int i = 0; i < 4; ++i) ok = ok && map_rows(&m[i], base, cols, rows, ld, 128 >> i);
  return ok;
}

// An MN-major operand of `groups` matrices [rows][cols]: a stage's 64 rows by
// 128 columns, as two 64-column parts. Where rows are whole blocks of 64
// elements (`blocks`), one box takes both parts.
bool map_mn_major(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t ld,
                  int groups, int blocks) {
  if (blocks) {
    const int64_t dims[4] = {64, rows, (cols + 63) / 64, groups};
    const int64_t strides[4] = {1, ld, 64, rows * ld};
    const int box[4] = {64, kDepth, 2, 1};
    return make_map(m, base, groups ? 4 : 3, dims, strides, box);
  }
  const int64_t dims[3] = {cols, rows, groups}, strides[3] = {1, ld, rows * ld};
  const int box[3] = {64, kDepth, 1};
  return make_map(m, base, groups ? 3 : 2, dims, strides, box);
}

template <int MODE, int ACT, typename T>
cudaError_t launch_tiles(const Maps& maps, MmaParams& q, int grid, cudaStream_t st) {
  q.pairs_out = q.features % 2 == 0 && (uintptr_t)q.out % 4 == 0;
  q.pairs_z = q.features % 2 == 0 && (uintptr_t)q.p.z % 4 == 0;
  const size_t smem = 1024 + kRingBytes + sizeof(Barriers) + (size_t)q.p.s.G * kGroupBytes;
  static std::atomic<uint64_t> raised{0};
  const cudaError_t e = raise_shared_limit(
      product_kernel<MODE, ACT, T>, 1024 + kRingBytes + sizeof(Barriers) + EP_MAX_EXPERTS * kGroupBytes, &raised);
  if (e != cudaSuccess) return e;
  return launch_overlapped(product_kernel<MODE, ACT, T>, dim3((unsigned)grid), kThreads, smem, st, maps, q);
}

Plan dense_grad_plan(int64_t rows, int cap, int tiles, int pairs) {
  return Plan{tiles, cap, splits_for(pairs, tiles, (int)((rows + kDepth - 1) / kDepth), kWorthGrad, kLeastGrad), 0};
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

}  // namespace

cudaError_t launch_linear_forward(const LinearParams& p, int sms, cudaStream_t st) {
  const bool gated = p.act == EP_ACT_SWIGLU;
  const int64_t rows = p.s.begin ? p.s.pool : p.s.dense_rows;
  MmaParams q;
  q.p = p;
  q.partial = p.partial;
  q.tickets = p.tickets;
  q.out = p.y;
  q.features = p.Nw;
  q.f_tiles = (p.Nw + 255) / 256;
  q.r_tiles = 0;
  q.cap = p.y_f32 ? kMaxRows / 2 : kMaxRows;
  q.terms = p.K;
  Maps m;
  bool ok;
  if (gated) {   // gate and up rows of a feature next to each other
    const int64_t dims[4] = {p.K, 2, p.N, p.s.G};
    const int64_t strides[4] = {1, (int64_t)p.N * p.K, p.K, (int64_t)p.Nw * p.K};
    const int box[4] = {kDepth, 2, 64, 1};
    ok = make_map(&m.a, p.w, 4, dims, strides, box);
  } else {
    const int64_t dims[3] = {p.K, p.Nw, p.s.G}, strides[3] = {1, p.K, (int64_t)p.Nw * p.K};
    const int box[3] = {kDepth, 128, 1};
    ok = make_map(&m.a, p.w, 3, dims, strides, box);
  }
  if (!ok || !map_k_major(m.b, p.x, p.K, rows, p.K)) return cudaErrorInvalidValue;
  q.a_blocks = q.b_blocks = 0;
  const int grid = grid_of(sms, most_units(p.s, q.f_tiles, p.K / kDepth));
  q.plan = dense_plan(p.s.dense_rows, q.cap, q.f_tiles,
                      (p.K + kDepth - 1) / kDepth, grid / 2);
  return p.y_f32 ? launch_forward<float>(m, q, grid, st)
                 : launch_forward<__nv_bfloat16>(m, q, grid, st);
}

cudaError_t launch_linear_input_grad(const LinearParams& p, int sms, cudaStream_t st) {
  const int64_t rows = p.s.begin ? p.s.pool : p.s.dense_rows;
  MmaParams q;
  q.p = p;
  q.partial = p.partial;
  q.tickets = p.tickets;
  q.out = p.dx;
  q.features = p.K;
  q.f_tiles = (p.K + 255) / 256;
  q.r_tiles = 0;
  q.cap = kMaxRows;
  q.terms = p.Nw;
  q.a_blocks = p.K % 64 == 0;
  q.b_blocks = 0;
  Maps m;
  if (!map_mn_major(&m.a, p.w, p.K, p.Nw, p.K, p.s.G, q.a_blocks) ||
      !map_k_major(m.b, p.dz, p.Nw, rows, p.ldz))
    return cudaErrorInvalidValue;
  const int grid = grid_of(sms, most_units(p.s, q.f_tiles, p.Nw / kDepth));
  q.plan = dense_plan(p.s.dense_rows, q.cap, q.f_tiles, (p.Nw + kDepth - 1) / kDepth, grid / 2);
  return launch_tiles<kInputGrad, EP_ACT_NONE, __nv_bfloat16>(m, q, grid, st);
}

cudaError_t launch_linear_weight_grad(const LinearParams& p, int sms, cudaStream_t st) {
  const int64_t rows = p.s.begin ? p.s.pool : p.s.dense_rows;
  MmaParams q;
  q.p = p;
  q.partial = p.partial;
  q.tickets = p.tickets;
  q.out = p.dw;
  q.features = p.K;
  q.f_tiles = (p.K + 255) / 256;
  // tiles of 128 rows where those of 256 leave half of the pairs idle, so that a
  // part of a tile never has more (4096 rows, 1024 x 512: 15.7 us for 24.2; 16384
  // rows, 512 x 256: 24.2 for 35.2)
  const int64_t wide = (int64_t)p.s.G * q.f_tiles * ((p.Nw + kMaxRows - 1) / kMaxRows);
  const int cap = p.dw_f32 || 2 * wide <= grid_of(sms, INT_MAX) / 2 ? kMaxRows / 2 : kMaxRows;
  q.cap = cap;
  q.terms = 0;
  q.r_tiles = (p.Nw + cap - 1) / cap;
  q.a_blocks = p.K % 64 == 0;
  // columns past Nw give rows of dW that are not stored; tiles of 128 rows
  // have one 64-column part to a CTA
  q.b_blocks = p.ldz % 64 == 0 && cap == kMaxRows;
  Maps m;
  if (!map_mn_major(&m.a, p.x, p.K, rows, p.K, 0, q.a_blocks) ||
      !map_mn_major(&m.b[0], p.dz, p.Nw, rows, p.ldz, 0, q.b_blocks))
    return cudaErrorInvalidValue;
  for (int i = 1; i < 4; ++i) m.b[i] = m.b[0];
  const int64_t units = (int64_t)p.s.G * q.f_tiles * q.r_tiles * kMaxSplits;
  const int grid = grid_of(sms, units);
  q.plan = dense_grad_plan(p.s.dense_rows, cap, q.f_tiles * q.r_tiles, grid / 2);
  return p.dw_f32 ? launch_tiles<kWeightGrad, EP_ACT_NONE, float>(m, q, grid, st)
                  : launch_tiles<kWeightGrad, EP_ACT_NONE, __nv_bfloat16>(m, q, grid, st);
}

}  // namespace ep
