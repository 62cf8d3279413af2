// What the kernels on pairs of SMs share (tc_pair.cu: one weight; experts_tc.cu:
// the products grouped by expert): the inline PTX of a cluster of two CTAs
// with tcgen05.mma.cta_group::2, the walk over a cluster's tiles, and how many
// clusters are resident at once.
#pragma once

#include <mutex>
#include <vector>

#include "common.cuh"
#include "tc_ptx.cuh"

namespace w4a16 {
namespace pair {

using namespace tc;

constexpr int kCols = 128;                       // weight columns per CTA (256 per pair)
constexpr int kStageK = 64;                      // k per atom
constexpr int kCodeAtomBytes = kCols * kStageK / 2;  // 4 KiB: 8 strips x 512 B
constexpr int kAtomCols = kStageK / 2;           // tensor-memory columns of one atom of A
constexpr int kSmemLimit = 227 * 1024;
constexpr int kBarBytes = 1024;

// Stage s of a cluster's sequence as (its tile's index in the sequence,
// stage kb of that tile), stepped forward without a division.
struct SeqPos {
  int kb, tile;
  __device__ __forceinline__ void step(int d, int nk) {
    kb += d;
    while (kb >= nk) {
      kb -= nk;
      ++tile;
    }
  }
};

// ------------------------------------------------------------------ cluster PTX

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Every thread of both CTAs arrives, then waits for all of them.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The address in CTA `rank`'s shared memory of this CTA's shared address `a`.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t a, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}

// Arrive on an mbarrier in either CTA of the pair (`cluster_bar` from
// cluster_addr), with the default release semantics of mbarrier.arrive.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// Bounded wait (as mbar_wait) that polls with test_wait instead of suspending
// in try_wait: for barriers completed by the other CTA (its arrivals, or the
// pair's multicast commits), where a thread suspended in try_wait was measured
// to resume about 0.45 us after the phase completed.
__device__ __forceinline__ bool mbar_wait_poll(uint32_t bar, uint32_t parity,
                                               volatile int* abort_flag, int code, int* err) {
  if (mbar_test(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  for (uint32_t i = 1;; ++i) {
    if (mbar_test(bar, parity)) return true;
    if ((i & 63u) == 0) {
      if (*abort_flag) return false;
      if (globaltimer() - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        atomicOr(err, code);
        return false;
      }
    }
  }
}

// Tensor memory of the pair: one warp of each CTA allocates (and frees)
// together; every tcgen05 instruction of the kernel uses cta_group::2.
__device__ __forceinline__ void pair_tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void pair_tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
// D (256 x N over the pair, fp32 in tensor memory) (+)= A (256 x 16 in tensor
// memory: each CTA's 128 rows at the same address) * B (16 x N: each CTA's
// N/2 columns at the same shared address).
__device__ __forceinline__ void pair_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                                uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive once on the mbarrier at shared address `bar` of BOTH CTAs when every
// MMA this thread issued before has completed.
__device__ __forceinline__ void pair_commit_both(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

// Clusters of a kernel and launch shape that are resident at once
// (cudaOccupancyMaxActiveClusters, kept per kernel, device and shared-memory
// size). A cluster's two CTAs sit on the two SMs of one TPC within one GPC,
// so GPCs with an odd number of usable SMs leave an SM out and the count can
// be below SMs / 2; a persistent grid larger than it would run its last
// clusters after the others, each with its whole share of the tiles.
inline cudaError_t max_active_clusters(const void* kernel, const cudaLaunchConfig_t& cfg, int* out) {
  struct Entry {
    const void* kernel;
    int device;
    size_t smem;
    int clusters;
  };
  static std::mutex mu;
  static std::vector<Entry> known;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(mu);
    for (const Entry& k : known)
      if (k.kernel == kernel && k.device == dev && k.smem == cfg.dynamicSmemBytes) {
        *out = k.clusters;
        return cudaSuccess;
      }
  }
  int n = 0;
  e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
  if (e != cudaSuccess) return e;
  if (n < 1) return cudaErrorInvalidConfiguration;
  std::lock_guard<std::mutex> lock(mu);
  known.push_back({kernel, dev, cfg.dynamicSmemBytes, n});
  *out = n;
  return cudaSuccess;
}

}  // namespace pair
}  // namespace w4a16
