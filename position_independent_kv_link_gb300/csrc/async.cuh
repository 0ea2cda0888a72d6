// Barriers in shared memory with bounded waits, bulk copies and the cluster's barrier, for the kernels of the decode-step calls.
#pragma once
#include <atomic>

#include "batch_internal.cuh"

namespace pic {

constexpr unsigned long long kWaitLimit = 4000000000ull;   // SM cycles, about 2 s

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// the same, but suspended for up to 20 us before it answers
__device__ __forceinline__ bool mbar_try_long(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}
// false (and the timeout flag) after kWaitLimit, or when the CTA has given up (`abort`: its word in shared memory)
static __device__ __noinline__ bool mbar_wait_on(uint32_t bar, uint32_t parity, volatile unsigned* abort, unsigned* flag) {
  const unsigned long long t0 = clock64();
  for (;;) {
    if (mbar_try_long(bar, parity)) return true;
    if (*abort) return false;
    if (clock64() - t0 > kWaitLimit) {
      atomicOr(flag, kBatchTimeout);
      *abort = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile unsigned* abort, unsigned* flag) {
  return mbar_try(bar, parity) || mbar_try_long(bar, parity) || mbar_wait_on(bar, parity, abort, flag);
}
// for the whole warp: the same answer in every lane
static __device__ __noinline__ bool warp_wait_on(uint32_t bar, uint32_t parity, volatile unsigned* abort, unsigned* flag) {
  return __all_sync(0xffffffffu, mbar_try_long(bar, parity) || mbar_wait_on(bar, parity, abort, flag));
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile unsigned* abort, unsigned* flag) {
  return __all_sync(0xffffffffu, mbar_try(bar, parity)) || warp_wait_on(bar, parity, abort, flag);
}
// waits on when the CTA has given up
__device__ __forceinline__ void mbar_settle(uint32_t bar, uint32_t parity, unsigned* flag) {
  unsigned none = 0;
  if (!mbar_try(bar, parity)) mbar_wait_on(bar, parity, &none, flag);
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The two halves of pdl_enter (pic_internal.h): the next kernel's CTAs come once all of this one's have called pdl_leave or have ended.
// CTAs that come while others still work take the places that happen to be free, and then share their own work out unevenly (4-bit
// gemm, one row of 128256 x 4096 again and again: 62 us for 55), so that long kernels call it late or not at all.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_leave() { asm volatile("griddepcontrol.launch_dependents;"); }

// ------------------------------------------------------------------ host
constexpr int kKnownDevices = 64;

inline int device_sms(int dev) {   // asked for once per device
  static std::atomic<int> sms[kKnownDevices];
  const bool known = dev >= 0 && dev < kKnownDevices;
  int n = known ? sms[dev].load() : 0;
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 152;
  if (known) sms[dev].store(n);
  return n;
}

// The dynamic shared memory that a kernel may have, set once per device.
template <auto kernel>
struct SharedMemory {
  std::atomic<bool> set[kKnownDevices] = {};
  cudaError_t allow(int dev, int bytes) {
    const bool known = dev >= 0 && dev < kKnownDevices;
    if (known && set[dev].load()) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && known) set[dev].store(true);
    return e;
  }
};

// How many clusters of c <= 8 CTAs of a kernel the device runs at once, asked for once per device (and amount of shared memory: the
// kernels here use about the same in every launch).
template <auto kernel>
struct ClusterRoom {
  std::atomic<int> known[kKnownDevices][9] = {};
  int clusters(int dev, int c, cudaLaunchConfig_t cfg, cudaLaunchAttribute* at, int sms) {
    const bool keep = dev >= 0 && dev < kKnownDevices;
    int n = keep ? known[dev][c].load() : 0;
    if (n > 0) return n;
    cfg.gridDim = dim3((unsigned)(c * sms));
    at[0].val.clusterDim.x = c;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      return 0;
    }
    if (keep) known[dev][c].store(n);
    return n;
  }
};

}  // namespace pic
