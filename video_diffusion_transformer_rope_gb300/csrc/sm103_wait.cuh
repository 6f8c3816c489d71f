// Bounded waits of whole warps on mbarriers, shared by the tile kernels (attn_tiles_sm103.cu, weigh_tiles_sm103.cu): every
// one gives up after kWaitLimitNs, raises its block's abort flag (a word of shared memory) and records its site.
#pragma once
#include "sm103_ptx.cuh"

namespace vdx {

constexpr int kSiteDrain = 42;      // of a copy or product in flight on the way out

__device__ __forceinline__ int ld_shared_flag(uint32_t addr) {
  int v;
  asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_flag(uint32_t addr) {
  asm volatile("st.volatile.shared.b32 [%0], %1;" ::"r"(addr), "r"(1) : "memory");
}

// Latch a wait that gave up, and the first site that did, beside whatever else has been reported.
__device__ __forceinline__ void report_timeout(int site) {
  if ((atomicOr(&g_error_word, 1u) & 1u) == 0) atomicOr(&g_error_word, static_cast<unsigned>(site & 0xff) << 8);
}

// mbar_try_wait that pairs with another CTA's cluster-scope release: what that CTA wrote by plain stores (or
// read) before it arrived lies before what follows here.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// The rest of a warp's wait for a barrier phase whose first look (mbar_try_wait, which itself blocks for
// a while) failed.  Kept out of line: a dozen inlined copies would spread the roles' loops over so
// much code that they miss the instruction caches.  The warp gives up as one, when the CTA's abort
// flag is raised or after kWaitLimitNs, and then raises the flag and records the site.
template <bool kCluster>
__device__ __noinline__ bool wait_more(uint32_t bar, uint32_t parity, uint32_t abort_flag, int site) {
  const unsigned long long t0 = global_timer_ns();
  while (true) {
    if (__all_sync(0xffffffffu, kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, ld_shared_flag(abort_flag) != 0)) return false;
    if (__any_sync(0xffffffffu, global_timer_ns() - t0 > kWaitLimitNs)) {
      st_shared_flag(abort_flag);
      if ((threadIdx.x & 31) == 0) report_timeout(site);
      return false;
    }
  }
}
// kCluster: for what the other CTA did by plain accesses.  Waits for copies, products and tensor memory need
// CTA scope only (the copies' bytes, the commits and the tcgen05 fences order those).
template <bool kCluster = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint32_t abort_flag, int site) {
  if (__all_sync(0xffffffffu, kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity))) return true;
  return wait_more<kCluster>(bar, parity, abort_flag, site);
}
// The softmax warps' form: their registers are past what a function call leaves room for.
__device__ __forceinline__ bool warp_wait_inline(uint32_t bar, uint32_t parity, uint32_t abort_flag, int site) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const unsigned long long t0 = global_timer_ns();
  while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
    if (__any_sync(0xffffffffu, ld_shared_flag(abort_flag) != 0 || global_timer_ns() - t0 > kWaitLimitNs)) {
      st_shared_flag(abort_flag);
      if ((threadIdx.x & 31) == 0) report_timeout(site);
      return false;
    }
  }
  return true;
}

// Bounded wait on the way out, whatever the abort flag says: copies and MMAs in flight finish
// before shared or tensor memory is released.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return;
  const unsigned long long t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      report_timeout(kSiteDrain);
      return;
    }
  }
}

}  // namespace vdx
