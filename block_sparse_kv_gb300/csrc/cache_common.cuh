// Device helpers of the cache operators (4-bit cache, token scores, eviction) that go beyond the ones
// every kernel shares.
#pragma once

#include "common.cuh"

namespace bskv {
namespace dev {

// n / d for 0 <= n < 2^31 by one multiplication: with 2^(s-1) < d <= 2^s and m = ceil(2^(31+s) / d),
// n m / 2^(31+s) is n / d plus less than 2^31 2^s / 2^(31+s) / d, so it has the same integer part.
struct FastDiv {
  uint32_t d, m, shift;  // m = 0: d = 1
  FastDiv() = default;
  explicit FastDiv(int32_t divisor) : d(uint32_t(divisor)), m(0), shift(0) {
    if (d <= 1) return;
    uint32_t s = 1;
    while ((uint64_t(1) << s) < d) ++s;
    m = uint32_t(((uint64_t(1) << (31 + s)) + d - 1) / d);
    shift = s - 1;
  }
  __device__ __forceinline__ int div(int n) const { return m ? int(__umulhi(uint32_t(n), m) >> shift) : n; }
  __device__ __forceinline__ int divmod(int n, int& rest) const {
    const int q = div(n);
    rest = n - q * int(d);
    return q;
  }
};

// ---- overlapping launches --------------------------------------------------------------

// Lets a kernel launched to start early begin once every CTA of this one got here or ended.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// Waits until the kernel before this one has ended and its writes are visible.
__device__ __forceinline__ void wait_for_prior_grid() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---- thread-block clusters ------------------------------------------------------------

// The halves of a cluster barrier: what was written before the arrival is visible after the wait.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ int2 ld_cluster_v2(uint32_t addr) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

// ---- copies and tensor memory ---------------------------------------------------------

// cp_async_16 to an address of the shared window.
__device__ __forceinline__ void cp_async_16_at(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns: thread i of the warp gets lane (base + i).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
}  // namespace dev
}  // namespace bskv
