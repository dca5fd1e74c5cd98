// linear_skinny.cuh -- the 16-bit linear layer and Q/K/V projection for few rows.
//
// Bound by reading W once (2*C*K bytes; at one row an operation a byte, at 128 rows half the
// tensor rate of the measured ridge).  So the roles are swapped: 128 rows of W are the M = 128
// operand of tcgen05.mma, kT tokens (16 to 128) the N operand, and no lane of the tensor core
// multiplies padding when there is one token.  K is split over the CTAs of a cluster, so that C/128
// tiles still fill the device; each keeps a ring of 16 KB weight tiles in flight (up to three CTAs an
// SM, so that one streams while another starts or ends).
// The partial sums meet in the CTAs' shared memory: CTA r of a cluster of S takes tokens r, r + S,
// ..., reads the S partials of each through distributed shared memory in rank order (the same
// bits every time, no atomics, no workspace that two captured graphs could share) and finishes
// it: a warp a token, 4 columns a lane, so a head's norm is a shuffle sum and every access to y
// and the residual covers 256 consecutive bytes.
#pragma once

#include "linear_pair.cuh"

namespace tara {

constexpr int kSkinnyThreads = 192;   // warp 0 loads, warp 1 issues MMAs, warps 2-5 read TMEM

template <int kT>
struct SkinnyLin {
  static constexpr int kWBytes = 128 * 128;
  static constexpr int kXBytes = kT * 128;
  static constexpr int kStageBytes = kWBytes + kXBytes;
  static constexpr int kCtas = kT <= 64 ? 3 : (kT == 128 ? 2 : 1);        // an SM
  static constexpr int kStages = (kCtas == 3 ? 73728 : 196608 / kCtas) / kStageBytes;   // 3 or 4
  static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + (2 * kStages + 1) * 8 + 16;
  static constexpr uint32_t kTmemCols = kT < 32 ? 32 : kT;
  static_assert(kT * 128 * 4 <= kStages * kStageBytes, "the partial sums reuse the ring");
  static_assert(kCtas * (kSmemBytes + 1024) <= 233472, "shared memory of an SM");
};

struct SkinnyArgs {
  LinearArgs lin;      // N: rows of one branch
  HeadArgs head;
  int rows;            // rows of x one blockIdx.z covers (all branches, or one)
  int splits;          // CTAs of a cluster
};

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint64_t* bar,
                                            int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint64_t* bar,
                                            int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// 4 consecutive 16-bit values <-> fp32.
template <bool kBF16>
__device__ __forceinline__ float4 load4(const void* p, long long i) {
  const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
  const float2 lo = unpack16<kBF16>(w.x), hi = unpack16<kBF16>(w.y);
  return make_float4(lo.x, lo.y, hi.x, hi.y);
}

// One token's 4 columns from column c of the output (all lanes of the warp together cover 128
// columns): bias, then act/gate/residual or the head's norm and rotation, then the store.
template <bool kBF16, bool kQkv>
__device__ __forceinline__ void skinny_finish(const LinearArgs& a, const HeadArgs& head, float4 s,
                                              int b, int n, int c) {
  const bool ok = c < a.C;
  const int part = ok ? c / a.part_cols : 0;
  const int pc = ok ? c - part * a.part_cols : 0;
  float f[4] = {s.x, s.y, s.z, s.w};
  if (a.bias && ok) {
    const float4 t = load4<kBF16>(a.bias, c);
    f[0] += t.x; f[1] += t.y; f[2] += t.z; f[3] += t.w;
  }
  if (!kQkv) {
    activate_any(f, a.act);
    if (a.gate && ok) {
      const float4 t = load4<kBF16>(a.gate, b * a.gate_b + c);
      f[0] *= t.x; f[1] *= t.y; f[2] *= t.z; f[3] *= t.w;
    }
    if (a.residual.ptr && ok) {
      const float4 t = load4<kBF16>(a.residual.ptr, row_offset(a.residual, b, n, c));
      f[0] += t.x; f[1] += t.y; f[2] += t.z; f[3] += t.w;
    }
  } else {
    // a head lies across 16 lanes (D = 64) or the warp (D = 128)
    const int lane = threadIdx.x & 31;
    const int lanes = head.D / 4, l = lane & (lanes - 1);
    const int h = pc / head.D, d = pc - h * head.D;
    const bool turned_part = ok && part < 2;
    if (head.norm) {
      float ss = f[0] * f[0] + f[1] * f[1] + f[2] * f[2] + f[3] * f[3];
      for (int o = lanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (turned_part) {
        const float r = __frsqrt_rn(fmaf(ss, head.inv_d, head.eps));
        float4 t = make_float4(1.f, 1.f, 1.f, 1.f);
        if (head.weight[part]) t = load4<kBF16>(head.weight[part], h * head.weight_h + d);
        f[0] *= r * t.x; f[1] *= r * t.y; f[2] *= r * t.z; f[3] *= r * t.w;
      }
    }
    if (head.table) {
      const float* cs = head.table + b * head.table_b + (long long)n * head.rot;
      const bool turned = turned_part && d < head.rot;
      if (head.halves) {
        const int half = head.rot / 8;                   // lanes of one half of the pairs
        const int partner = (lane - l) + (l < half ? l + half : (l < 2 * half ? l - half : l));
        float g[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = __shfl_sync(0xffffffffu, f[i], partner);
        if (turned) {
          const bool low = l < half;
          const float4* c4 = reinterpret_cast<const float4*>(cs + 8 * (low ? l : l - half));
          const float4 t0 = __ldg(c4), t1 = __ldg(c4 + 1);
          const float sign = low ? -1.f : 1.f;
          f[0] = fmaf(f[0], t0.x, g[0] * (sign * t0.y));
          f[1] = fmaf(f[1], t0.z, g[1] * (sign * t0.w));
          f[2] = fmaf(f[2], t1.x, g[2] * (sign * t1.y));
          f[3] = fmaf(f[3], t1.z, g[3] * (sign * t1.w));
        }
      } else if (turned) {
        const float4 t = __ldg(reinterpret_cast<const float4*>(cs + d));
        const float x0 = f[0], y0 = f[1], x1 = f[2], y1 = f[3];
        f[0] = fmaf(x0, t.x, -y0 * t.y);
        f[1] = fmaf(x0, t.y, y0 * t.x);
        f[2] = fmaf(x1, t.z, -y1 * t.w);
        f[3] = fmaf(x1, t.w, y1 * t.z);
      }
    }
  }
  if (ok) {
    const RowView& y = a.y[part];
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(const_cast<void*>(y.ptr)) +
                              row_offset(y, b, n, pc)) =
        make_uint2(pack16<kBF16>(f[0], f[1]), pack16<kBF16>(f[2], f[3]));
  }
}

template <bool kBF16, int kT, bool kQkv>
__global__ void __launch_bounds__(kSkinnyThreads, SkinnyLin<kT>::kCtas)
linear_skinny_kernel(const __grid_constant__ PairLinMaps maps,
                     const __grid_constant__ SkinnyArgs args) {
  using S = SkinnyLin<kT>;
  constexpr int NS = S::kStages;
  const LinearArgs& a = args.lin;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* part = reinterpret_cast<float*>(smem);        // [token][128 columns], over the ring
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + NS * S::kStageBytes);
  uint64_t* empty = full + NS;
  uint64_t* acc_full = empty + NS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = args.splits;
  const int rank = (int)cluster_ctarank();
  const int c0 = (int)(blockIdx.x / (unsigned)splits) * 128;
  const int t0 = (int)blockIdx.y * kT;                 // first row of this token tile
  const int z = (int)blockIdx.z;                       // branch of x (0 when they run on)
  const int k_steps = (a.K + 63) / 64;
  const int k_begin = (int)((long long)k_steps * rank / splits);
  const int k_end = (int)((long long)k_steps * (rank + 1) / splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, S::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // an earlier kernel gave up: skip the work (every CTA still meets its cluster below)
  const bool skip = *reinterpret_cast<volatile int*>(a.status) != 0;

  if (warp == 0) {
    if (lane == 0 && !skip) {
      tma_prefetch_desc(&maps.w);
      tma_prefetch_desc(&maps.x);
      const int xD = a.x.D;
      int h = 0, d = k_begin * 64;
      if (d >= xD) {
        h = d / xD;
        d -= h * xD;
      }
      int slot = 0;
      uint32_t phase = 0;
      for (int k = k_begin; k < k_end; ++k) {
        if (!mbar_wait_idle(&empty[slot], phase ^ 1u, abort_flag)) break;
        mbar_arrive_expect_tx(&full[slot], S::kStageBytes);
        const uint32_t dst = smem_u32(smem) + (uint32_t)slot * S::kStageBytes;
        tma_load_2d(dst, &maps.w, &full[slot], k * 64, c0);
        tma_load_4d(dst + S::kWBytes, &maps.x, &full[slot], d, t0, h, z);
        if ((d += 64) >= xD) {
          d = 0;
          ++h;
        }
        if (++slot == NS) {
          slot = 0;
          phase ^= 1u;
        }
      }
      // copies already issued land within microseconds: give them 1 ms before this CTA's shared
      // memory can be released
      if (*abort_flag)
        for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    }
  } else if (warp == 1) {
    if (lane == 0 && !skip) {
      constexpr uint32_t idesc = make_idesc_f16(128, kT, kBF16, false);
      const uint64_t wd0 = make_sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t xd0 = make_sdesc_sw128(smem_u32(smem + S::kWBytes), 16, 1024);
      int slot = 0;
      uint32_t phase = 0;
      for (int k = k_begin; k < k_end; ++k) {
        if (!mbar_wait_idle(&full[slot], phase, abort_flag)) break;
        tc_fence_after();
        const uint64_t off = (uint64_t)((slot * S::kStageBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_ss(tmem, wd0 + off + (uint64_t)(kk * 2), xd0 + off + (uint64_t)(kk * 2), idesc,
                  (k > k_begin || kk > 0) ? 1u : 0u);
        umma_commit(&empty[slot]);
        if (++slot == NS) {
          slot = 0;
          phase ^= 1u;
        }
      }
      // also after a wait that gave up: the products issued so far complete before the exit
      umma_commit(acc_full);
      volatile int no_abort = 0;
      if (*abort_flag) mbar_wait(acc_full, 0, &no_abort, kLinDrainNs);
    }
  } else if (!skip) {
    if (mbar_wait_warp(acc_full, 0, abort_flag)) {
      tc_fence_after();
      const int q = warp & 3;                          // TMEM lane quarter
      const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16);
      float* col = part + q * 32 + lane;
#pragma unroll 1
      for (int t = 0; t < kT; t += 16) {
        uint32_t v[16];
        tmem_ld8(acc + t, v);
        tmem_ld8(acc + t + 8, v + 8);
        tmem_ld_wait();
        reg_fence<16>(v);
#pragma unroll
        for (int i = 0; i < 16; ++i) col[(t + i) * 128] = __uint_as_float(v[i]);
      }
      tc_fence_before();
    }
  }

  // every CTA of the cluster has its partial sums in shared memory
  __syncthreads();
  cluster_sync_all();
  if (!skip && !*abort_flag) {
    const int tokens = min(kT, args.rows - t0);
    const uint32_t mine = smem_u32(part) + (uint32_t)lane * 16u;
    const bool run_on = args.rows != a.N;              // rows go through all branches
    // two tokens at a time, all their partial sums in flight together
    const int step = splits * (kSkinnyThreads / 32);
    for (int t = rank + splits * warp; t < tokens; t += 2 * step) {
      const bool two = t + step < tokens;
      float4 v[2][8];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        if (r < splits) {
          const uint32_t peer = mapa_shared(mine, (uint32_t)r);
          v[0][r] = ld_cluster_f4(peer + (uint32_t)t * 512u);
          if (two) v[1][r] = ld_cluster_f4(peer + (uint32_t)(t + step) * 512u);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (i == 1 && !two) break;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < splits) {
            s.x += v[i][r].x; s.y += v[i][r].y; s.z += v[i][r].z; s.w += v[i][r].w;
          }
        const int row = t0 + t + i * step;
        const int b = run_on ? row / a.N : z;
        skinny_finish<kBF16, kQkv>(a, args.head, s, b, run_on ? row - b * a.N : row, c0 + 4 * lane);
      }
    }
  }
  // no CTA leaves while its partial sums may still be read
  cluster_sync_all();
  if (threadIdx.x == 0 && *abort_flag) atomicExch(a.status, 1);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
}

}  // namespace tara
