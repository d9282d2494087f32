// Helpers of the CTA-pair tensor-core kernels (sm_100a): two CTAs of a cluster
// on neighbouring SMs run one tcgen05.mma of M = 256 (cta_group::2).  Each CTA
// holds 128 rows of A and half of B's rows in its own shared memory, at the
// same offsets, and 128 rows of D in its own tensor memory; the leader (rank
// 0) issues for both.  Barriers that the leader waits on live in its shared
// memory and the other CTA arrives on them remotely; a commit signals the
// barrier at the same offset in both CTAs.
#pragma once

#include "tc_common.cuh"

namespace mbok {

__device__ __forceinline__ uint32_t pair_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}

// The leader's copy of this CTA's shared-memory object `p` (cluster address).
__device__ __forceinline__ uint32_t pair_leader(const void* p) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, 0;\n" : "=r"(a) : "r"(tc_smem(p)));
  return a;
}

// Arrive on a barrier of either CTA.  What such an arrival announces is shared
// or tensor memory of this CTA that the tensor cores will access, ordered
// before it by fence.proxy.async or tcgen05.fence; no thread of the other CTA
// reads this thread's writes, so the arrival needs no cluster-scope release
// (which took 0.6 us each: it waits for all of the thread's memory operations).
__device__ __forceinline__ void pair_arrive(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];\n" ::"r"(cluster_addr) : "memory");
}

// A TMA load into this CTA's shared memory that completes on a barrier of
// either CTA (cluster address).
__device__ __forceinline__ void pair_tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];\n" ::"r"(tc_smem(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// As tc_wait, ordered after arrivals from either CTA.  A try may suspend the warp
// for up to 20 us: many warps wait long, and their polling took issue slots from
// the unpack (32 tokens, 11008 x 2 x 4096: 51 -> 49 us).
constexpr unsigned kPairTryNs = 20000;
__device__ __forceinline__ bool pair_wait(uint64_t* bar, unsigned parity, unsigned long long limit = kTcWaitNs) {
  const uint32_t a = tc_smem(bar);
  unsigned long long t0 = 0;
  for (unsigned it = 1;; ++it) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(a), "r"(parity), "r"(kPairTryNs)
        : "memory");
    if (done) return true;
    if ((it & 7u) == 0) {
      const unsigned long long t = tc_ns();
      if (t0 == 0) t0 = t;
      else if (t - t0 > limit) return false;
    }
  }
}

// One lane of a converged warp.  The issuing loops below run in whole warps and
// elect a lane only around the instructions themselves: that keeps their
// operands in uniform registers.  Issued from inside an `if (lane == 0)` loop a
// tcgen05.mma took 130 to 190 cycles, more than most of them run.
__device__ __forceinline__ bool elect_lane() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e != 0;
}

__device__ __forceinline__ void pair_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// Tensor memory for both CTAs: one whole warp of each CTA runs these.
__device__ __forceinline__ void pair_alloc(uint32_t* slot, unsigned cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(tc_smem(slot)), "r"(cols));
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::);
}
__device__ __forceinline__ void pair_dealloc(uint32_t tmem, unsigned cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(cols));
}

__device__ __forceinline__ void pair_mma(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}

// Arrives on `bar` in both CTAs once the MMAs issued so far are done.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(
          tc_smem(bar)),
      "h"(uint16_t(3))
      : "memory");
}

// Matrix descriptor, M- or N-major with 128-byte swizzle: blocks of 64
// elements along M (or N) `block_bytes` apart; within a block one 128-byte
// line per k, groups of 8 lines 1024 bytes apart.
__device__ __forceinline__ uint64_t tc_desc_sw128_mn(uint32_t saddr, uint32_t block_bytes) {
  uint64_t d = 0;
  d |= uint64_t((saddr >> 4) & 0x3FFF);
  d |= uint64_t(block_bytes >> 4) << 16;       // leading byte offset
  d |= uint64_t(1024 >> 4) << 32;              // stride byte offset
  d |= uint64_t(1) << 46;
  d |= uint64_t(2) << 61;
  return d;
}

// Instruction descriptor of kind::f16: D f32, A and B both bf16 or both f16,
// M = m, N = n, each operand K-major or (a_mn, b_mn) M-/N-major.
inline uint32_t tc_idesc_f16(int m, int n, bool bf16, bool a_mn, bool b_mn) {
  const uint32_t t = bf16 ? 1u : 0u;
  return (1u << 4) | (t << 7) | (t << 10) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) |
         (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}

// Drains for a CTA whose wait gave up: both phases of every barrier that a
// copy or an MMA in flight completes, bounded.
__device__ __forceinline__ void tc_drain_barriers(uint64_t* bars, int n) {
  for (int i = 0; i < n; ++i) {
    (void)tc_wait(&bars[i], 0u, kTcDrainNs);
    (void)tc_wait(&bars[i], 1u, kTcDrainNs);
  }
}

// Host: a two-dimensional tensor map; false if the driver refuses it.
inline bool make_map(CUtensorMap* m, CUtensorMapDataType type, const void* base, uint64_t inner, uint64_t outer,
                     uint64_t stride_bytes, uint32_t box_inner, uint32_t box_outer, bool swizzle128) {
  const EncodeTiledFn enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {stride_bytes};
  const cuuint32_t box[2] = {box_inner, box_outer};
  const cuuint32_t ones[2] = {1, 1};
  return enc(m, type, 2, const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
             swizzle128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace mbok
