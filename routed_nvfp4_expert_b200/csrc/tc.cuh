// tcgen05 (5th-generation tensor core, TMEM accumulators) and TMA tensor-copy
// helpers for sm_100a, as inline PTX.
#pragma once

#include <cuda.h>

#include "tma.cuh"

namespace rnx {

// ---------------------------------------------------------------- TMEM
// Allocation is warp-wide; the base address is written to shared memory.
RNX_DEVICE void tmem_alloc(uint32_t* smem_dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_dst)),
               "r"(ncols)
               : "memory");
}
RNX_DEVICE void tmem_relinquish() { asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory"); }
RNX_DEVICE void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
RNX_DEVICE void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
RNX_DEVICE void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// One lane of a converged warp (the others get false). Keeping the whole warp
// in a role's loop and issuing tcgen05 / TMA instructions from the elected
// lane keeps the loop state warp-uniform (uniform registers), which is what
// lets one thread issue MMAs back to back.
RNX_DEVICE bool elect_one() {
  uint32_t pred = 0;
  asm volatile(
      "{\n\t.reg .b32 r;\n\t.reg .pred p;\n\t"
      "elect.sync r|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(pred));
  return pred != 0;
}

// ---------------------------------------------------------------- descriptors
// Shared-memory matrix descriptor, K-major, 128-byte swizzle: rows of 128 B,
// 8-row groups 1024 B apart (SBO), LBO unused (16 B), descriptor version 1.
// The buffer must be 1024-byte aligned (base offset 0).
RNX_DEVICE uint64_t sdesc_k_sw128(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)1 << 16;                // leading byte offset: 16 B
  d |= (uint64_t)(1024 >> 4) << 32;      // stride byte offset: 1024 B
  d |= (uint64_t)1 << 46;                // version (sm_100)
  d |= (uint64_t)2 << 61;                // layout: SWIZZLE_128B
  return d;
}

// Shared-memory matrix descriptor, MN-major, 128-byte swizzle: a block is 64
// consecutive elements of the M (or N) index (128 B) by any number of k rows
// 128 B apart, 8-row groups 1024 B apart (SBO); the next 64 elements of the M
// (or N) index start block_bytes later (LBO). K = 16 of one MMA spans 2048 B.
RNX_DEVICE uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t block_bytes) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(block_bytes >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// Descriptor of a 512-byte scale-factor atom (32 rows of 16 B, no swizzle)
// as the source of tcgen05.cp .32x128b.
RNX_DEVICE uint64_t sdesc_sf_atom(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(128 >> 4) << 32;       // 8-row groups 128 B apart
  d |= (uint64_t)1 << 46;
  return d;                               // layout: SWIZZLE_NONE
}

// Instruction descriptor of kind::mxf4nvf4 with block16 (E4M3) scales:
// A, B = E2M1, K-major; M, N the tile shape; scale factor ids 0.
__host__ __device__ constexpr uint32_t idesc_mxf4nvf4(int M, int N) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Instruction descriptor of kind::f16 with bf16 A/B, fp32 accumulate, K-major.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// The same with A and / or B MN-major.
__host__ __device__ constexpr uint32_t idesc_bf16_major(int M, int N, bool a_mn, bool b_mn) {
  return idesc_bf16(M, N) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16);
}

// ---------------------------------------------------------------- MMA (one CTA)
RNX_DEVICE void mma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrive on `bar` once every tcgen05 operation this thread issued so far is done.
RNX_DEVICE void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// Each thread of the warp reads 32 consecutive 32-bit columns of its TMEM lane
// into r[0..31] (r must index registers: constant offsets into local arrays).
RNX_DEVICE void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// 16 consecutive columns.
RNX_DEVICE void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
RNX_DEVICE void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------------------- TMA tensor copies
// 2D tiled load of the box at element coordinates (x, y) into shared memory,
// completion counted as bytes on `bar`. x times the element size must be a
// multiple of 16 bytes.
RNX_DEVICE void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

// 2D tiled store of the box at (x, y) from shared memory (the layout the
// tensor map's swizzle describes), tracked by the thread's bulk async-group.
// Rows or columns outside the tensor are not written.
RNX_DEVICE void tma_store_2d(const CUtensorMap* map, int x, int y, const void* src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x), "r"(y),
               "r"(smem_u32(src))
               : "memory");
}

// ---------------------------------------------------------------- CTA pairs (cta_group::2)
// A cluster of two CTAs runs one MMA of M = 256: each CTA holds 128 rows of
// A, half of the N rows of B and its own scale atoms; the even CTA issues the
// MMAs and the scale copies for both.

RNX_DEVICE uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Every thread of both CTAs: arrive (release) and wait (acquire).
RNX_DEVICE void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// shared::cluster address of the same shared-memory offset in CTA `rank`.
RNX_DEVICE uint32_t mapa_shared(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// Arrive on a barrier of this or the peer CTA (a shared::cluster address)
// with CTA-scope release. Used for "accumulator drained" signals, which order
// only this thread's completed tcgen05.ld (tcgen05.wait::ld, then
// tcgen05.fence::before_thread_sync) before the peer's MMAs; no data passes
// through memory. A cluster-scope release would first wait for every global
// load and store this thread has in flight, about 1-4 us under load.
RNX_DEVICE void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// The same without ordering memory: every thread of the cluster has arrived.
// In two halves, so that a thread does not wait where it arrives.
RNX_DEVICE void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
RNX_DEVICE void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
RNX_DEVICE void cluster_sync_relaxed() {
  cluster_arrive_relaxed();
  cluster_wait();
}

// One word into a CTA of the cluster, visible there behind a cluster_sync_all.
RNX_DEVICE void st_cluster(uint32_t cluster_addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}

// fp32 from a CTA of the cluster (shared::cluster address).
RNX_DEVICE float4 ld_cluster_f4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}
RNX_DEVICE float ld_cluster_f1(uint32_t cluster_addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// Store one word into a CTA of the cluster; its 4 bytes are counted on the
// barrier (shared::cluster addresses of the same CTA).
RNX_DEVICE void st_async(uint32_t cluster_addr, uint32_t v, uint32_t bar_cluster) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(cluster_addr), "r"(v),
               "r"(bar_cluster)
               : "memory");
}

RNX_DEVICE bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Bounded wait (cluster-scope acquire) for a barrier that peer CTAs arrive on.
// limit_ns 0: one try.
RNX_DEVICE bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, unsigned long long limit_ns = kWaitLimitNs) {
  if (limit_ns == 0) return mbar_try_wait_cluster(bar, parity);
  unsigned long long t0 = globaltimer_ns();
  for (uint32_t i = 0;; ++i) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if ((i & 255u) == 255u && globaltimer_ns() - t0 > limit_ns) return false;
  }
}

RNX_DEVICE void tmem_alloc_pair(uint32_t* smem_dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_dst)),
               "r"(ncols)
               : "memory");
}
RNX_DEVICE void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
RNX_DEVICE void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

RNX_DEVICE void mma_mxf4nvf4_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                  uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.block16 [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
      : "memory");
}

// bf16 operands, M = 256 over the pair.
RNX_DEVICE void mma_bf16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Scale-atom copy issued by the even CTA: each CTA's atom at this shared
// offset goes to the same TMEM columns of that CTA.
RNX_DEVICE void tmem_cp_sf_pair(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

// Arrive on `bar` (same shared offset) in every CTA of cta_mask once the
// pair's tcgen05 operations issued so far are done.
RNX_DEVICE void mma_commit_pair_mc(uint64_t* bar, uint16_t cta_mask) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                   smem_u32(bar)),
               "h"(cta_mask)
               : "memory");
}

// 2D tiled load into this CTA's shared memory whose completion is counted on
// the barrier at shared::cluster address `bar_cluster` (the even CTA's).
RNX_DEVICE void tma_load_2d_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(bar_cluster)
      : "memory");
}

// ---------------------------------------------------------------- a pair that stops early
// A wait that runs out stops both CTAs of a pair, and their producers may stop
// at different steps: a step that only some of them issued would leave its
// copies on the way, to either CTA, with a barrier that never completes. So each
// producer leaves its count of issued steps in its own CTA, and once everything
// has stopped the even CTA collects them, counts the missing bytes as if they had
// come and waits for the rest; only then do the CTAs leave.

// By one lane, before the pair's closing cluster_sync_all: the abort flag of both.
RNX_DEVICE void stop_pair(uint32_t* status, volatile int* abort_flag) {
  set_status(status, kDevErrTimeout);
  const uint32_t at = smem_u32(const_cast<int*>(abort_flag));
  st_cluster(mapa_shared(at, 0), 1u);
  st_cluster(mapa_shared(at, 1), 1u);
}

// By all threads of both CTAs behind that barrier, when no producer issues any
// more, every MMA is done and the flag is set. issued: steps by PRODUCERS
// producers, the even CTA's first (each CTA has set its own), whose first announces
// a step's bytes; bytes: of a step by each producer. No producer is ahead of
// another by more than the ring, since a slot is freed by the products of a step
// that all issued.
template <int PRODUCERS, int STAGES>
RNX_DEVICE void pair_drain(uint32_t rank, uint64_t* full_bar, volatile int* issued, const uint32_t (&bytes)[PRODUCERS],
                           uint32_t* status) {
  const int lane = threadIdx.x & 31;
  constexpr int kMine = PRODUCERS / 2;
  if (rank == 1 && threadIdx.x < kMine)
    st_cluster(mapa_shared(smem_u32(const_cast<int*>(issued + kMine + threadIdx.x)), 0), (uint32_t)issued[kMine + threadIdx.x]);
  __syncwarp();
  cluster_sync_all();
  if (rank == 0 && threadIdx.x < 32) {
    int first = issued[0], last = issued[0];
    uint32_t all = bytes[0];
    for (int i = 1; i < PRODUCERS; ++i) first = min(first, issued[i]), last = max(last, issued[i]), all += bytes[i];
    if (lane == 0) {
      for (int step = first; step < last; ++step) {
        uint64_t* bar = &full_bar[step % STAGES];
        if (issued[0] <= step) mbar_arrive_expect_tx(bar, all);
        for (int i = 0; i < PRODUCERS; ++i)
          if (issued[i] <= step) mbar_complete_tx(bar, bytes[i]);
      }
    }
    __syncwarp();
    for (int step = max(0, last - STAGES); step < last; ++step)
      if (!mbar_wait(&full_bar[step % STAGES], (uint32_t)(step / STAGES) & 1u) && lane == 0)
        set_status(status, kDevErrTimeout);
    __syncwarp();
  }
  cluster_sync_all();
}

}  // namespace rnx
