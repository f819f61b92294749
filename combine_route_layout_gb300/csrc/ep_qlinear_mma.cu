// The products of block-quantised operands on the tensor cores: z = x W^T and
// dx = dz' W, with the forward's bias, activation and residual in the epilogue.
//
// Tiles, pairs of CTAs, the ring of stages and the parts of contractions are those of
// the bf16 products (ep_linear_mma.cu): outputs are computed transposed, features on
// the tensor core's M side, rows on its N side. A stage is 128 bytes of each operand
// row, which of E4M3 are 128 terms: exactly one scale block. So the tensor core adds
// up one stage at a time, into the two accumulators in turn, and the epilogue's warps
// take each such sum out of TMEM and add it, times its scales, to f32 sums of the tile
// in their registers, while the next stage's is made:
//     sum[feature][row] += stage[feature][row] (sx[row][block] sw[feature block][block])
// The transposed form has one weight scale for all of a CTA's features (two with
// SwiGLU: gate on even lanes, up on odd ones); a warp of its own fetches the scales of
// the rows, as the quantiser lays them out, and leaves the products of both in shared
// memory, kSlots stages ahead, from where the epilogue reads four rows' at once for
// all lanes. W is read as it is for dx too: MN-major, a box of 128 terms x 128
// features.
//
// Registers: 128 sums a thread of the epilogue; the other warps give theirs up.
#include <atomic>
#include <climits>
#include <cstring>

#include "ep_linear_tiles.cuh"
#include "ep_qlinear.cuh"

namespace ep {
namespace {

constexpr int kDepth = 128;                      // terms per stage: 128 bytes
constexpr int kStageA = 128 * kDepth;            // bytes of a CTA's 128 features
constexpr int kStageB = 128 * kDepth;            // bytes of a CTA's half of the rows
constexpr int kRingBytes = 5 * (kStageA + kStageB);
constexpr int kMaxStages = 8;
constexpr int kScaleBytes = 8 * kMaxRows * 4;    // 8 stages' scales are there ahead (gated: 4)
constexpr int kMaxScaleSlots = 8;
constexpr int kPitch = 36;                       // words of a row of 32 that warps turn round
constexpr int kTurnBytes = kEpilogueWarps * 32 * kPitch * 4;
constexpr int kTmemColumns = 512;                // two accumulators
// Registers of a thread at the start, of the first four warps and of the epilogue's.
constexpr int kRegisters = 168, kRegistersLess = 88, kRegistersMore = 208;
static_assert(kThreads * kRegisters >= 128 * kRegistersLess + kEpilogueWarps * 32 * kRegistersMore,
              "registers for the epilogue");

struct MmaParams {
  static constexpr int kDepth = ep::kDepth;
  QLinearParams p;
  void* out;               // y or dx
  int features;            // length of the output's contiguous axis (weight rows or K)
  int f_tiles, cap, terms;
  int pairs_out, pairs_z;  // bf16 outputs whose rows allow two features a store
  Plan plan;               // of a dense product
  // scale of (pool row, block) and of (group, feature block, block)
  const float* row_scale;
  int row_ld;
  int64_t group_ld;
  int feature_ld, block_ld;
  int feature_blocks;
  int up;                  // from a gate's scales to its up rows'
};

struct Barriers {
  uint64_t full[kMaxStages];  // both CTAs' operands have landed (even CTA's)
  uint64_t empty[kMaxStages]; // the MMAs have read this stage
  uint64_t acc_full[2];       // a stage's sum is complete
  uint64_t acc_empty[2];      // even CTA's: both CTAs' epilogues have read it
  uint64_t scale_full[kMaxScaleSlots], scale_empty[kMaxScaleSlots];
  uint64_t tile_full[kSlots], tile_empty[kSlots];
  uint64_t joined;            // the epilogue's warps meet
  Tile tiles[kSlots];
  uint32_t tmem;
  uint32_t last;              // this CTA's part of a tile was the last
};

// Two sums of f32 at once: acc += a b.
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ void floats_of(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

// A stage's sum is there, on both CTAs by the tensor core's own arrival, and has been
// read. What these barriers guard lies in tensor memory alone: see ep_linear_mma.cu.
__device__ __forceinline__ bool sum_ready(Barriers* bar, int n_acc) {
  if (!warp_wait_cluster(&bar->acc_full[n_acc & 1], (n_acc >> 1) & 1)) return false;
  tc_fence_after();
  return true;
}
__device__ __forceinline__ void sum_free(Barriers* bar, int n_acc, int lane) {
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_signal_at(in_cta(&bar->acc_empty[n_acc & 1], 0));
}

// A block of 32 features by 32 rows, from the order in which the tensor memory gives
// pairs of rows to a feature of a lane and all its rows, by way of shared memory: the
// pitch keeps both ways free of conflicts.
__device__ __forceinline__ void turn_round(float* at, int lane, const uint64_t (&sum)[4][4], float (&r)[32]) {
  float* to = at + (lane & 3) * 2 * kPitch + (lane >> 2);
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      floats_of(sum[j][i], lo, hi);
      to[8 * i * kPitch + 8 * j] = lo;
      to[(8 * i + 1) * kPitch + 8 * j] = hi;
    }
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 32; ++c) r[c] = at[c * kPitch + lane];
  __syncwarp();
}

struct Maps {
  CUtensorMap a;
  CUtensorMap b[4];        // boxes of 128, 64, 32 and 16 rows
};

template <int MODE, int ACT, typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    product8_kernel(const __grid_constant__ Maps maps, MmaParams q) {
  constexpr bool kGated = MODE == kForward && ACT == EP_ACT_SWIGLU;
  constexpr int kBlocks = kMaxRows / 64;         // of 32 columns, of a warp
  constexpr int kScaleSlots = kGated ? 4 : 8, kScaleRow = kGated ? 2 * kMaxRows : kMaxRows;
  constexpr int kScaleAhead = kGated ? 2 : 4;    // stages whose scales are fetched at once
  extern __shared__ uint8_t raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
  float* scales = reinterpret_cast<float*>(ring + kRingBytes);   // [slot][gate, up][row]
  float* turned = scales + kScaleBytes / 4;                      // [epilogue warp][row][feature]
  Barriers* bar = reinterpret_cast<Barriers*>(ring + kRingBytes + kScaleBytes + kTurnBytes);
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
    // producer, scales, the epilogue's warps, MMA (even CTA)
    mbar_init(&bar->tile_full[threadIdx.x - 32], 1);
    mbar_init(&bar->tile_empty[threadIdx.x - 32], 2 + kEpilogueWarps + (cta == 0 ? 1 : 0));
  } else if (threadIdx.x >= 40 && threadIdx.x < 40 + kMaxScaleSlots) {
    mbar_init(&bar->scale_full[threadIdx.x - 40], 1);
    mbar_init(&bar->scale_empty[threadIdx.x - 40], kEpilogueWarps);
  } else if (threadIdx.x == 32 + kSlots) {
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
  const int stage_bytes = kStageA + plan.cap / 2 * kDepth;
  const int stages = min(kMaxStages, kRingBytes / stage_bytes);
  tc_fence_before();
  __syncthreads();                       // the TMEM address is there
  tc_fence_after();
  cluster_wait();
  const uint32_t tmem = bar->tmem;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int mine = pair < units ? (units - 1 - pair) / pairs + 1 : 0;   // this pair's units

  if (warp < 4) {
    registers_less<kRegistersLess>();
    if (warp == 0 && elect_one()) {
      // ---------------------------------------------- producer: one thread
      int it = 0, s = 0;                      // stages written so far, the ring's place
      uint32_t phase = 1;                     // the first pass over the ring waits for nothing
      const uint32_t full0 = in_cta(&bar->full[0], 0);
      const uint32_t ring0 = smem_addr(ring);
      bool ok = true;
      for (int i = 0; i < mine && ok; ++i) {
        Tile w;
        ok = take_tile(bar, i, w);
        if (!ok) break;
        const int half = w.n / 2;
        const int fc = w.f0 + (int)cta * 128;                     // this CTA's features
        const int row = (int)w.begin + w.r0 + (int)cta * half;    // this CTA's rows
        const int box = half > 64 ? 0 : half > 32 ? 1 : half > 16 ? 2 : 3;
        const uint32_t bytes = kStageA + (kStageB >> box);
        const CUtensorMap* map_b = &maps.b[box];
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (it >= stages) {
            ok = mbar_wait_soon(&bar->empty[s], phase);
            if (!ok) break;
          }
          const uint32_t on = full0 + s * 8, a = ring0 + s * stage_bytes;
          mbar_signal_expect_tx_at(on, bytes);
          const int d = kb * kDepth;
          if (MODE == kInputGrad) {
            const int second = kb >= q.p.Nb;                      // up's half of the terms
            tma_load_4d(a, &maps.a, fc, d - second * q.p.Nb * kDepth, second, w.g, on);
          } else if (kGated) {
            tma_load_4d(a, &maps.a, d, 0, fc / 2, w.g, on);
          } else {
            tma_load_3d(a, &maps.a, d, fc, w.g, on);
          }
          tma_load_2d(a + kStageA, map_b, d, row, on);
          ++it;
          if (++s == stages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      // the MMAs' arrivals are this CTA's to wait for, the other's too
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
    } else if (warp == 1 && cta == 0 && elect_one()) {
      // ---------------------------------------------- MMA: one thread of the even CTA
      // operands of stage 0; a stage is stage_bytes on
      constexpr bool kMnA = MODE == kInputGrad;
      constexpr uint32_t kStepA = (kMnA ? 4096 : 32) >> 4, kStepB = 32 >> 4;
      const uint32_t stage_units = (uint32_t)stage_bytes >> 4;
      const uint64_t op_a = smem_operand(smem_addr(ring), 16);
      const uint64_t op_b = smem_operand(smem_addr(ring) + kStageA, 16);
      const uint32_t a0 = (uint32_t)op_a, a_high = (uint32_t)(op_a >> 32);
      const uint32_t b0 = (uint32_t)op_b, b_high = (uint32_t)(op_b >> 32);
      const uint32_t empty0 = smem_addr(&bar->empty[0]), sum0 = smem_addr(&bar->acc_full[0]);
      int n_acc = 0;
      uint32_t s = 0, phase = 0;             // the ring's place
      bool ok = true;
      for (int i = 0; i < mine && ok; ++i) {
        Tile w;
        ok = take_tile(bar, i, w);
        if (!ok) break;
        const uint32_t form = mma8_form(w.n, kMnA);
        for (int kb = w.kb0; kb < w.kb1; ++kb, ++n_acc) {
          if (n_acc >= 2) {
            ok = mbar_wait_soon_cluster(&bar->acc_empty[n_acc & 1], ((n_acc >> 1) - 1) & 1);
            if (!ok) break;
            tc_fence_after();
          }
          ok = mbar_wait_soon(&bar->full[s], phase);
          if (!ok) break;
          tc_fence_after();
          mma8_stage<kStepA, kStepB>(tmem + (n_acc & 1) * 256, a0 + s * stage_units, a_high,
                                     b0 + s * stage_units, b_high, form);
          mma_commit_both(empty0 + s * 8);
          mma_commit_both(sum0 + (n_acc & 1) * 8);
          if (++s == (uint32_t)stages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      // the other CTA's last arrivals here
      for (int last = n_acc - 2; last < n_acc && ok; ++last)
        if (last >= 0) ok = mbar_wait_soon_cluster(&bar->acc_empty[last & 1], (last >> 1) & 1);
      if (!ok) atomicOr(timeout, kErrLinearTimeout);
      tc_fence_after();
    } else if (warp == 2) {
      // ---------------------------------------------- scales
      int n_scale = 0;
      bool ok = true;
      for (int i = 0; i < mine && ok; ++i) {
        Tile w;
        ok = warp_take_tile(bar, i, w, lane);
        if (!ok) break;
        const float* rows = q.row_scale + (w.begin + w.r0 + lane) * q.row_ld;
        const int fc = kGated ? w.f0 / 2 + (int)cta * 64 : w.f0 + (int)cta * 128;
        const float* features = q.p.ws + w.g * q.group_ld + (int64_t)min(fc / 128, q.feature_blocks - 1) * q.feature_ld;
        for (int kb0 = w.kb0; kb0 < w.kb1 && ok; kb0 += kScaleAhead) {
          float v[kScaleAhead][kMaxRows / 32], gate[kScaleAhead], up[kScaleAhead];
#pragma unroll
          for (int u = 0; u < kScaleAhead; ++u) {
            const int kb = kb0 + u;
            const bool there = kb < w.kb1;
#pragma unroll
            for (int j = 0; j < kMaxRows / 32; ++j) {
              v[u][j] = 0.0f;
              if (there && lane + 32 * j < w.rows) v[u][j] = rows[(int64_t)(32 * j) * q.row_ld + kb];
            }
            gate[u] = up[u] = 0.0f;
            if (there) {
              gate[u] = features[(int64_t)kb * q.block_ld];
              if (kGated) up[u] = features[q.up + (int64_t)kb * q.block_ld];
            }
          }
#pragma unroll
          for (int u = 0; u < kScaleAhead; ++u) {
            if (kb0 + u >= w.kb1 || !ok) continue;
            const int slot = n_scale % kScaleSlots;
            if (n_scale >= kScaleSlots) ok = warp_wait(&bar->scale_empty[slot], (n_scale / kScaleSlots - 1) & 1);
            if (!ok) continue;
            // the order in which the epilogue's threads take a block of 32 rows
            float* to = scales + slot * kScaleRow + (lane & 7) / 2 * 8 + lane / 8 * 2 + (lane & 1);
#pragma unroll
            for (int j = 0; j < kMaxRows / 32; ++j) {
              if (32 * j >= w.n) continue;
              to[32 * j] = v[u][j] * gate[u];
              if (kGated) to[kMaxRows + 32 * j] = v[u][j] * up[u];
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar->scale_full[slot]);
            ++n_scale;
          }
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
        bar->tiles[slot] = tile_at<MODE>(q, plan, first, begins, counts, sizes, pair + i * pairs);
        mbar_arrive(&bar->tile_full[slot]);
      }
      if (!ok) atomicOr(timeout, kErrLinearTimeout);
    }
  } else {
    registers_more<kRegistersMore>();
    // ------------------------------------------------ epilogue
    // 64 columns of the tile belong to the warp pair of a quarter: 32 to this warp
    const int quad = warp & 3, turn = (warp - 4) >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    // a thread's sums are of the features lane / 4 + 8 j: gates, or up's
    const float* my_scales = scales + (kGated && (lane & 4) ? kMaxRows : 0) + turn * 32 + (lane & 3) * 8;
    float* turn_at = turned + (warp - 4) * 32 * kPitch;
    int n_acc = 0;                         // sums, and their scales
    uint32_t meeting = 0;
    bool ok = true;
    for (int i = 0; i < mine && ok; ++i) {
      const int u = pair + i * pairs;
      Tile w;
      ok = warp_take_tile(bar, i, w, lane);
      if (!ok) break;
      if (w.kb0 >= w.kb1) continue;
      const bool whole = w.parts == 1;
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
      const int blocks = (w.n - turn * 32 + 63) / 64;   // of this warp (none below 1)
      uint64_t sum[kBlocks][4][4];                      // [..][lane / 4 + 8 j][8 i + 2 (lane % 4), + 1]
#pragma unroll
      for (int h = 0; h < kBlocks; ++h)
#pragma unroll
        for (int c = 0; c < 16; ++c) sum[h][c / 4][c % 4] = 0;   // two f32 zeros
      for (int kb = w.kb0; kb < w.kb1; ++kb, ++n_acc) {
        const int slot = n_acc % kScaleSlots;
        ok = warp_wait(&bar->scale_full[slot], (n_acc / kScaleSlots) & 1) && sum_ready(bar, n_acc);
        if (!ok) break;
        const float* scale = my_scales + slot * kScaleRow;
        if (blocks < 1) sum_free(bar, n_acc, lane);
#pragma unroll
        for (int h = 0; h < kBlocks; ++h) {
          if (h >= blocks) continue;
          const ulonglong2 by0 = *reinterpret_cast<const ulonglong2*>(scale + h * 64);
          const ulonglong2 by1 = *reinterpret_cast<const ulonglong2*>(scale + h * 64 + 4);
          float r[4][8];
          tmem_load_pairs(lanes + (n_acc & 1) * 256 + turn * 32 + h * 64, r);
          if (h == blocks - 1) sum_free(bar, n_acc, lane);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            fma2(sum[h][j][0], pair_of(r[j][0], r[j][1]), by0.x);
            fma2(sum[h][j][1], pair_of(r[j][2], r[j][3]), by0.y);
            fma2(sum[h][j][2], pair_of(r[j][4], r[j][5]), by1.x);
            fma2(sum[h][j][3], pair_of(r[j][6], r[j][7]), by1.y);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->scale_empty[slot]);
      }
      if (!ok) break;
      // the values of this part: the tile's result, or sums for the part that finishes
      // last, which then adds all of them in their order
      if (whole) {
#pragma unroll
        for (int h = 0; h < kBlocks; ++h) {
          const int c0 = turn * 32 + h * 64;
          if (c0 >= w.rows) continue;
          float r[32];
          turn_round(turn_at, lane, sum[h], r);
          epilogue<MODE, ACT, T>(q, w, (int)cta, lane, quad, c0, r, b);
        }
        continue;
      }
      // this lane's column in the pair's place (a pair has one unit where there are parts)
      float* sums = q.p.partial + ((int64_t)pair * plan.cap * 256 + cta * 128 + quad * 32 + lane);
      const int c0 = turn * 32;                         // parts are of tiles of at most 64 rows
      float r[32];
      turn_round(turn_at, lane, sum[0], r);
#pragma unroll
      for (int c = 0; c < 32; ++c) put(sums + (c0 + c) * 256, r[c], c0 + c < w.rows);
      ok = epilogue_meet(bar, lane, meeting);
      if (!ok) break;
      if (threadIdx.x == 128) {
        unsigned int* ticket = q.p.tickets + quotient(u, plan.splits) * 2 + cta;
        const bool last = ticket_take(ticket) == (unsigned)w.parts - 1;
        if (last) *ticket = 0u;
        bar->last = last;
      }
      ok = epilogue_meet(bar, lane, meeting);
      if (!ok) break;
      if (!bar->last || c0 >= w.rows) continue;
      add_parts(sums - (int64_t)w.part * plan.cap * 256 + c0 * 256, plan.cap * 256, w.parts, w.rows - c0, r);
      epilogue<MODE, ACT, T>(q, w, (int)cta, lane, quad, c0, r, b);
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

// Rows of a K-major operand, in boxes of 128, 64, 32 and 16 rows.
bool map_rows8(CUtensorMap (&m)[4], const void* base, int64_t cols, int64_t rows) {
  const int64_t dims[2] = {cols, rows}, strides[2] = {1, cols};
  bool ok = true;
  for (int i = 0; i < 4; ++i) {
    const int box[2] = {kDepth, 128 >> i};
    ok = ok && make_map(&m[i], base, 2, dims, strides, box, 1);
  }
  return ok;
}

template <int MODE, int ACT, typename T>
cudaError_t launch_tiles(const Maps& maps, MmaParams& q, int grid, cudaStream_t st) {
  q.pairs_out = q.features % 2 == 0 && (uintptr_t)q.out % 4 == 0;
  q.pairs_z = q.features % 2 == 0 && (uintptr_t)q.p.z % 4 == 0;
  constexpr size_t kFixed = 1024 + kRingBytes + kScaleBytes + kTurnBytes + sizeof(Barriers);
  static_assert(kFixed + EP_MAX_EXPERTS * kGroupBytes <= 227 * 1024, "shared memory");
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
  const cudaError_t e = raise_shared_limit(kernel, kFixed + EP_MAX_EXPERTS * kGroupBytes, &raised);
  if (e != cudaSuccess) return e;
  return launch_overlapped(kernel, dim3((unsigned)grid), kThreads, kFixed + (size_t)q.p.s.G * kGroupBytes,
                           st, maps, q);
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
int plan_grid(MmaParams& q, int sms) {
  q.f_tiles = (q.features + 255) / 256;
  q.cap = kMaxRows;
  const int stages = (q.terms + kDepth - 1) / kDepth;
  const int grid = grid_of(sms, most_units(q.p.s, q.f_tiles, stages));
  q.plan = dense_plan(q.p.s.dense_rows, q.cap, q.f_tiles, stages, grid / 2);
  return grid;
}

}  // namespace

cudaError_t launch_qlinear_forward(const QLinearParams& p, int sms, cudaStream_t st) {
  const int64_t rows = p.s.begin ? p.s.pool : p.s.dense_rows;
  MmaParams q;
  q.p = p;
  q.out = p.y;
  q.features = p.Nw;
  q.terms = p.K;
  q.row_scale = p.xs;
  q.row_ld = p.Kb;
  q.group_ld = (int64_t)p.Sw * p.Kb;
  q.feature_ld = p.Kb;
  q.block_ld = 1;
  q.feature_blocks = p.Nb;
  q.up = p.Nb * p.Kb;
  Maps m;
  bool ok;
  if (p.act == EP_ACT_SWIGLU) {   // gate and up rows of a feature next to each other
    const int64_t dims[4] = {p.K, 2, p.N, p.s.G};
    const int64_t strides[4] = {1, (int64_t)p.N * p.K, p.K, (int64_t)p.Nw * p.K};
    const int box[4] = {kDepth, 2, 64, 1};
    ok = make_map(&m.a, p.w, 4, dims, strides, box, 1);
  } else {
    const int64_t dims[3] = {p.K, p.Nw, p.s.G}, strides[3] = {1, p.K, (int64_t)p.Nw * p.K};
    const int box[3] = {kDepth, 128, 1};
    ok = make_map(&m.a, p.w, 3, dims, strides, box, 1);
  }
  if (!ok || !map_rows8(m.b, p.x, p.K, rows)) return cudaErrorInvalidValue;
  const int grid = plan_grid(q, sms);
  return p.y_f32 ? launch_forward<float>(m, q, grid, st) : launch_forward<__nv_bfloat16>(m, q, grid, st);
}

cudaError_t launch_qlinear_input_grad(const QLinearParams& p, int sms, cudaStream_t st) {
  const int64_t rows = p.s.begin ? p.s.pool : p.s.dense_rows;
  const int parts = p.Sw / p.Nb;
  MmaParams q;
  q.p = p;
  q.out = p.dx;
  q.features = p.K;
  q.terms = p.Sw * kDepth;
  q.row_scale = p.dzs;
  q.row_ld = p.Sw;
  q.group_ld = (int64_t)p.Sw * p.Kb;
  q.feature_ld = 1;
  q.block_ld = p.Kb;
  q.feature_blocks = p.Kb;
  q.up = 0;
  Maps m;
  const int64_t dims[4] = {p.K, p.N, parts, p.s.G};
  const int64_t strides[4] = {1, p.K, (int64_t)p.N * p.K, (int64_t)p.Nw * p.K};
  const int box[4] = {128, kDepth, 1, 1};
  if (!make_map(&m.a, p.w, 4, dims, strides, box, 1) || !map_rows8(m.b, p.dz8, q.terms, rows))
    return cudaErrorInvalidValue;
  const int grid = plan_grid(q, sms);
  return launch_tiles<kInputGrad, EP_ACT_NONE, __nv_bfloat16>(m, q, grid, st);
}

}  // namespace ep
