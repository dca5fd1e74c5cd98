// linear_ptx.cuh -- inline-PTX wrappers the linear-layer kernels need beyond sm100_ptx.cuh:
// TMA loads of weight tiles (2-D) and token views (4-D), short TMEM loads, suspended waits.
// No cluster multicast.
#pragma once

#include <cuda_fp16.h>

#include "sm100_ptx.cuh"

namespace tara {

// Tile loads into this CTA's shared memory, counted on an mbarrier of the pair's even CTA.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map,
                                                 uint32_t bar_cluster, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar_cluster)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d_pair(uint32_t dst, const CUtensorMap* map,
                                                 uint32_t bar_cluster, int x, int y, int z,
                                                 int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar_cluster)
      : "memory");
}

// 32 lanes x 8 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

constexpr uint64_t kLinWaitNs = 2000000000ull;    // 2 s per wait; a normal wait is microseconds
constexpr uint32_t kLinIdleNs = 1000000u;           // 1 ms between looks at the clock
constexpr uint64_t kLinDrainNs = 200000000ull;    // 0.2 s to let in-flight MMAs land
// A CTA that gives up leaves its pair's ring at once; the other starves from then on, gives up a
// whole wait later, drains, and only then arrives on the first one's exit barrier, in shared memory
// that has to be there still.  So the wait before the exit outlasts all of that.
constexpr uint64_t kLinExitNs = 6000000000ull;
static_assert(kLinExitNs >= 2 * (kLinWaitNs + kLinDrainNs), "the peer's last wait ends first");

// One try of up to `hint_ns`: the thread is suspended by the hardware, not polling, until the
// phase completes or the hint runs out.
__device__ __forceinline__ bool mbar_try_wait_for(uint32_t bar, uint32_t parity,
                                                  uint32_t hint_ns) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(hint_ns)
      : "memory");
  return ok != 0;
}

// Bounded wait as mbar_wait, suspended between looks at the clock: waits here last up to a
// tile's products (tens of microseconds), and ten polling warps an SM cost issue slots and
// power.
__device__ __forceinline__ bool mbar_wait_idle(uint64_t* bar, uint32_t parity,
                                               volatile int* abort) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait_for(a, parity, kLinIdleNs)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait_for(a, parity, kLinIdleNs)) {
    if (*abort) return false;
    if (global_timer_ns() - t0 > kLinWaitNs) {
      *abort = 1;
      return false;
    }
  }
  return true;
}

// Bounded wait of a whole warp: true only when every lane saw the phase complete.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity,
                                               volatile int* abort) {
  const bool ok = mbar_wait_idle(bar, parity, abort);
  return __all_sync(0xffffffffu, ok);
}

template <bool kBF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  return kBF16 ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
}
template <bool kBF16>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
  if (kBF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// 8 consecutive 16-bit values as fp32.
template <bool kBF16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = unpack16<kBF16>(w[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
__device__ __forceinline__ uint4 ldg16(const void* base, long long i) {   // i: 16-bit elements
  return __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i));
}

}  // namespace tara
