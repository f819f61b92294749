// Tensor-core (tcgen05, TMEM), tiled-TMA and cluster primitives for sm_103a
// as inline PTX, for kernels whose CTA pairs share one matrix tile. Waits are
// bounded as in ep_bulk.cuh.
#pragma once

#include "ep_bulk.cuh"

namespace ep {

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n .reg .pred p;\n"
      " elect.sync _|p, 0xFFFFFFFF;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// A barrier of the cluster's CTAs that orders no memory of theirs.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// The address of this CTA's `p` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
  return r;
}

__device__ __forceinline__ void mbar_arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

// The relaxed forms order no other access of this thread: enough where what
// the barrier guards is moved by TMA and read by the tensor core alone. A
// release at cluster scope costs about half a microsecond, on every stage.
// Enough too where it guards tensor memory: tc_fence_before() ahead of the arrival
// and tc_fence_after() behind the wait, at cluster scope both, order that.
__device__ __forceinline__ void mbar_signal_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

__device__ __forceinline__ void mbar_signal_expect_tx_at(uint32_t cluster_addr, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(
                   cluster_addr),
               "r"(bytes)
               : "memory");
}

__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done != 0;
}

// mbar_wait for a barrier that the other CTA of the cluster arrives on too.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 0; i < kMbarMaxPolls; ++i) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if (globaltimer_ns() - t0 > kMbarWaitNs) return false;
  }
  return false;
}

// Whether the phase is complete, without waiting. `bar`: shared-memory address.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

// mbar_wait without a look at the clock on the first polls.
__device__ __forceinline__ bool mbar_wait_soon(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait(bar, parity);
}

// The same for a barrier that the other CTA of the cluster arrives on too.
__device__ __forceinline__ bool mbar_wait_soon_cluster(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait_cluster(bar, parity)) return true;
  return mbar_wait_cluster(bar, parity);
}

// The same for a whole warp, which agrees on the answer: a lane alone that gave
// up would leave the others in their next warp-wide step.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xFFFFFFFFu, mbar_wait_soon(bar, parity));
}
__device__ __forceinline__ bool warp_wait_cluster(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xFFFFFFFFu, mbar_wait_soon_cluster(bar, parity));
}

__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Tiled TMA loads into this CTA's shared memory; the bytes complete on the
// barrier at `bar`, which may be the other CTA's of the pair. The innermost
// coordinate is a multiple of 16 bytes.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* map, int c0, int c1,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* map, int c0, int c1, int c2,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* map, int c0, int c1, int c2,
                                            int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_prefetch_map(const void* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ------------------------------------------------------------------- tcgen05

// Both CTAs of the pair call these with one whole warp each.
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_addr(dst)),
               "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}

__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Shared-memory operand with 128-byte swizzle (rows of 128 bytes, groups of 8
// rows 1024 bytes apart). K-major: a row is one index, 64 terms. MN-major: a
// row is one term, 64 indices; the next 64 indices lie `next` bytes on.
__device__ __forceinline__ uint64_t smem_operand(uint32_t addr, uint32_t next) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(next >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// Both operands bf16, f32 accumulator, M = 256 over the CTA pair.
__device__ __forceinline__ uint32_t mma_form(uint32_t n, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn_major << 15) |
         ((uint32_t)b_mn_major << 16) | ((n >> 3) << 17) | ((256u >> 4) << 24);
}

// Four products of 16 terms each, a stage: d += a b, or d = a b + ... unless
// `accumulate`. The operands' steps, A_STEP and B_STEP (in 16-byte units), change
// their descriptors' low words alone. One statement: the thread that issues has
// to stay ahead of the tensor core.
template <uint32_t A_STEP, uint32_t B_STEP>
__device__ __forceinline__ void mma_stage(uint32_t d, uint32_t a, uint32_t a_high, uint32_t b,
                                          uint32_t b_high, uint32_t form, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p, t;\n .reg .b32 x, y;\n .reg .b64 a, b;\n"
      " setp.ne.u32 p, %6, 0;\n setp.eq.u32 t, 0, 0;\n"
      " mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n"
      " add.u32 x, %1, %7;\n add.u32 y, %3, %8;\n mov.b64 a, {x, %2};\n mov.b64 b, {y, %4};\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, t;\n"
      " add.u32 x, %1, %9;\n add.u32 y, %3, %10;\n mov.b64 a, {x, %2};\n mov.b64 b, {y, %4};\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, t;\n"
      " add.u32 x, %1, %11;\n add.u32 y, %3, %12;\n mov.b64 a, {x, %2};\n mov.b64 b, {y, %4};\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, t;\n}" ::"r"(d),
      "r"(a), "r"(a_high), "r"(b), "r"(b_high), "r"(form), "r"((uint32_t)accumulate), "n"(A_STEP),
      "n"(B_STEP), "n"(2 * A_STEP), "n"(2 * B_STEP), "n"(3 * A_STEP), "n"(3 * B_STEP)
      : "memory");
}

// One product of 16 terms.
__device__ __forceinline__ void mma_step(uint32_t d, uint32_t a, uint32_t a_high, uint32_t b,
                                         uint32_t b_high, uint32_t form, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n"
      " setp.ne.u32 p, %6, 0;\n mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n}" ::"r"(d),
      "r"(a), "r"(a_high), "r"(b), "r"(b_high), "r"(form), "r"((uint32_t)accumulate)
      : "memory");
}

// Arrive on this CTA's barrier once the MMAs issued so far are complete.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
               : "memory");
}

// 32 columns of this warp's 32 lanes: register c holds column c of the lane.
__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"  // one statement: no register is read before the wait
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int c = 0; c < 32; ++c) v[c] = __uint_as_float(r[c]);
}

}  // namespace ep
