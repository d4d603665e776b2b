// Shared-memory rings fed by bulk copies: mbarrier and copy instructions, the
// bounded waits, and the device-side error word that they set. Included once
// per translation unit, which has its own error word.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "tw.h"

namespace tw {
namespace {

// Device-side error word of the kernels of this translation unit (bit 0:
// consumer wait, bit 1: producer wait, bit 2: final drain, bit 3: a row index
// outside the expert rows).
__device__ unsigned int g_device_error = 0;

constexpr int kMaxStages = 32;
constexpr unsigned long long kWaitLimitNs = 2000000000ull;  // give up after 2 s
constexpr uint32_t kWaitLimitPolls = 1u << 26;
constexpr unsigned long long kDrainLimitNs = 200000000ull;  // 0.2 s per stage
// ------------------------------------------------------------------ PTX helpers

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count)
               : "memory");
}

__device__ __forceinline__ void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)),
               "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done != 0;
}

__device__ __forceinline__ unsigned long long global_timer_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

__device__ __forceinline__ uint64_t l2_evict_first_policy() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

__device__ __forceinline__ uint64_t l2_evict_normal_policy() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// 1-D TMA bulk copy global -> shared, completing `bytes` on the mbarrier.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar,
                                          uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1], %2, [%3], %4;" ::"r"(smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

__device__ __forceinline__ uint32_t sm_id() {
  uint32_t id;
  asm volatile("mov.u32 %0, %%smid;" : "=r"(id));
  return id;
}

// Wait for the phase of the given parity of *bar to complete. Bounded: gives
// up after limit_ns (kWaitLimitNs in the kernels) or kWaitLimitPolls polls,
// then sets *abort and the device error word. Returns false at once while
// *abort is set.
__device__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned code,
                           unsigned long long limit_ns = kWaitLimitNs) {
  if (*abort) return false;
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_timer_ns();
  for (uint32_t i = 1; i < kWaitLimitPolls; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 0u) {
      if (*abort) return false;
      if (global_timer_ns() - t0 > limit_ns) break;
    }
  }
  *abort = 1;
  atomicOr(&g_device_error, code);
  return false;
}

// Bounded wait that ignores the abort flag (used to drain in-flight copies).
__device__ bool drain_phase(uint64_t* bar, uint32_t parity) {
  const unsigned long long t0 = global_timer_ns();
  for (uint32_t i = 0; i < kWaitLimitPolls; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 255u && global_timer_ns() - t0 > kDrainLimitNs) break;
  }
  atomicOr(&g_device_error, 4u);
  return false;
}

// Waits (bounded) until every bulk copy a producer issued into its ring of
// `stages` stages has landed: `issued` items went out in order, item i on
// stage i % stages in phase i / stages, so the last item of each stage
// completes after all earlier ones there. The producer owns this drain, on
// the normal path too (where it returns as the consumers' waits complete),
// so no CTA exits with copies into its shared memory in flight, even if a
// consumer gives up a wait after the producer has left its issue loop.
__device__ void drain_ring(uint64_t* full, int stages, long long issued) {
  const long long last = issued - 1;
  for (int st = 0; st < stages && st <= last; ++st) {
    const long long it_last = last - ((last - st) % stages);
    drain_phase(&full[st], static_cast<uint32_t>((it_last / stages) & 1));
  }
}

int read_ring_error(int reset, unsigned* code) {
  if (cudaMemcpyFromSymbol(code, g_device_error, sizeof(*code)) != cudaSuccess) return TW_ERR_CUDA;
  if (reset && *code) {
    const unsigned zero = 0;
    if (cudaMemcpyToSymbol(g_device_error, &zero, sizeof(zero)) != cudaSuccess) return TW_ERR_CUDA;
  }
  return TW_OK;
}

}  // namespace
}  // namespace tw
