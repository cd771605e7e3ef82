// cluster.cuh -- inline-PTX wrappers for thread-block clusters: ranks, the cluster
// barrier, mbarriers that other blocks of the cluster complete, and stores and minima into
// their shared memory.
#pragma once
#include "ptx.cuh"

namespace moe {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Count bytes to come in the current phase without arriving.
__device__ __forceinline__ void mbar_add_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
// As mbar_wait for a barrier that other CTAs of the cluster complete: what they
// wrote before is visible afterwards.
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity) {
  uint64_t t0 = 0;
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kSuspendNs)
        : "memory");
    if (ok) return true;
    if (t0 == 0) t0 = globaltimer();
    else if (globaltimer() - t0 > kWaitLimitNs) return false;
  }
}
// Store two floats at this CTA's shared address `dst` in the CTA of rank `cta`, and
// count the 8 bytes on that CTA's mbarrier at this CTA's address `bar`.
__device__ __forceinline__ void st_async_f32x2(uint32_t dst, uint32_t bar, uint32_t cta, float a,
                                               float b) {
  uint32_t rdst, rbar;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(rdst) : "r"(dst), "r"(cta));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(rbar) : "r"(bar), "r"(cta));
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
          rdst),
      "f"(a), "f"(b), "r"(rbar)
      : "memory");
}
// Lower the int at this CTA's shared address `dst` in the CTA of rank `cta` to v.
__device__ __forceinline__ void red_min_cluster(uint32_t dst, uint32_t cta, int v) {
  uint32_t rdst;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(rdst) : "r"(dst), "r"(cta));
  asm volatile("red.relaxed.cluster.shared::cluster.min.s32 [%0], %1;" ::"r"(rdst), "r"(v)
               : "memory");
}

}  // namespace moe
