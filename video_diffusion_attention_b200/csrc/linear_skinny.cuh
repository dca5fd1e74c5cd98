// linear_skinny.cuh -- the 16-bit linear layer and Q/K/V projection for few rows.
//
// Bound by reading W once (2*C*K bytes; at one row an operation a byte, at 128 rows half the
// tensor rate of the measured ridge).  So the roles are swapped: 128 rows of W are the M = 128
// operand of tcgen05.mma, kT tokens (16 to 256) the N operand, and no lane of the tensor core
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

__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// 4 consecutive 16-bit values <-> fp32.
template <bool kBF16>
__device__ __forceinline__ float4 load4(const void* p, long long i) {
  const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
  const float2 lo = unpack16<kBF16>(w.x), hi = unpack16<kBF16>(w.y);
  return make_float4(lo.x, lo.y, hi.x, hi.y);
}

// What one lane needs to finish its 4 columns of any token (all lanes of a warp together cover the
// CTA's 128 columns): parameters in registers, addresses as base and strides.  Gathered while the
// products run; computed per token it made each take 800 cycles.
struct SkinnyLane {
  bool ok;                  // the columns exist and are to be stored
  int part, l, d;           // output part; lane and column within the head (projection)
  float4 bias, gain;        // gain: gate (when shared by the branches) or norm weight
  uint16_t* y;
  const uint16_t* residual;
  const uint16_t* gate;     // per branch
  long long y_b, y_n, r_b, r_n, gate_b;
};

template <bool kBF16, bool kQkv>
__device__ __forceinline__ SkinnyLane skinny_lane(const LinearArgs& a, const HeadArgs& head, int c) {
  SkinnyLane s;
  s.ok = c < a.C;
  const int cc = s.ok ? c : 0;
  s.part = cc < a.part_cols ? 0 : cc / a.part_cols;
  const int pc = cc - s.part * a.part_cols;
  s.bias = a.bias ? load4<kBF16>(a.bias, cc) : make_float4(0.f, 0.f, 0.f, 0.f);
  s.gain = make_float4(1.f, 1.f, 1.f, 1.f);
  s.gate = s.residual = nullptr;
  s.r_b = s.r_n = s.gate_b = 0;
  s.l = s.d = 0;
  if (kQkv) {
    const int h = pc / head.D;
    s.d = pc - h * head.D;
    s.l = (threadIdx.x & 31) & (head.D / 4 - 1);
    if (s.part < 2 && head.norm && head.weight[s.part] != nullptr)
      s.gain = load4<kBF16>(head.weight[s.part], h * head.weight_h + s.d);
  } else {
    if (a.gate) {
      if (a.gate_b == 0)
        s.gain = load4<kBF16>(a.gate, cc);
      else
        s.gate = static_cast<const uint16_t*>(a.gate) + cc;
      s.gate_b = a.gate_b;
    }
    if (a.residual.ptr) {
      s.residual = static_cast<const uint16_t*>(a.residual.ptr) + row_offset(a.residual, 0, 0, cc);
      s.r_b = a.residual.b;
      s.r_n = a.residual.n;
    }
  }
  const RowView& y = a.y[s.part];
  s.y = static_cast<uint16_t*>(const_cast<void*>(y.ptr)) + row_offset(y, 0, 0, pc);
  s.y_b = y.b;
  s.y_n = y.n;
  return s;
}

// One token's 4 columns: bias, then act/gate/residual or the head's norm and rotation, the store.
template <bool kBF16, bool kQkv>
__device__ __forceinline__ void skinny_finish(const HeadArgs& head, int act, const SkinnyLane& t,
                                              float4 s, int b, int n) {
  float f[4] = {s.x + t.bias.x, s.y + t.bias.y, s.z + t.bias.z, s.w + t.bias.w};
  if (!kQkv) {
    activate_any(f, act);
    float4 g = t.gain;
    if (t.gate) g = load4<kBF16>(t.gate, b * t.gate_b);
    f[0] *= g.x; f[1] *= g.y; f[2] *= g.z; f[3] *= g.w;
    if (t.residual) {
      const float4 r = load4<kBF16>(t.residual, b * t.r_b + n * t.r_n);
      f[0] += r.x; f[1] += r.y; f[2] += r.z; f[3] += r.w;
    }
  } else {
    // a head lies across 16 lanes (D = 64) or the warp (D = 128)
    const bool turned_part = t.ok && t.part < 2;
    if (head.norm) {
      float ss = f[0] * f[0] + f[1] * f[1] + f[2] * f[2] + f[3] * f[3];
      for (int o = head.D / 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (turned_part) {
        const float r = __frsqrt_rn(fmaf(ss, head.inv_d, head.eps));
        f[0] *= r * t.gain.x; f[1] *= r * t.gain.y; f[2] *= r * t.gain.z; f[3] *= r * t.gain.w;
      }
    }
    if (head.table) {
      const float* cs = head.table + b * head.table_b + (long long)n * head.rot;
      const bool turned = turned_part && t.d < head.rot;
      if (head.halves) {
        const int half = head.rot / 8;                   // lanes of one half of the pairs
        const int first = (int)(threadIdx.x & 31) - t.l;
        const int partner = first + (t.l < half ? t.l + half : (t.l < 2 * half ? t.l - half : t.l));
        float g[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = __shfl_sync(0xffffffffu, f[i], partner);
        if (turned) {
          const bool low = t.l < half;
          const float4* c4 = reinterpret_cast<const float4*>(cs + 8 * (low ? t.l : t.l - half));
          const float4 t0 = __ldg(c4), t1 = __ldg(c4 + 1);
          const float sign = low ? -1.f : 1.f;
          f[0] = fmaf(f[0], t0.x, g[0] * (sign * t0.y));
          f[1] = fmaf(f[1], t0.z, g[1] * (sign * t0.w));
          f[2] = fmaf(f[2], t1.x, g[2] * (sign * t1.y));
          f[3] = fmaf(f[3], t1.z, g[3] * (sign * t1.w));
        }
      } else if (turned) {
        const float4 t4 = __ldg(reinterpret_cast<const float4*>(cs + t.d));
        const float x0 = f[0], y0 = f[1], x1 = f[2], y1 = f[3];
        f[0] = fmaf(x0, t4.x, -y0 * t4.y);
        f[1] = fmaf(x0, t4.y, y0 * t4.x);
        f[2] = fmaf(x1, t4.z, -y1 * t4.w);
        f[3] = fmaf(x1, t4.w, y1 * t4.z);
      }
    }
  }
  if (t.ok)
    *reinterpret_cast<uint2*>(t.y + b * t.y_b + n * t.y_n) =
        make_uint2(pack16<kBF16>(f[0], f[1]), pack16<kBF16>(f[2], f[3]));
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
  volatile int* skip_flag = abort_flag + 1;            // rank 0's holds for the whole cluster

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
  SkinnyLane mine = skinny_lane<kBF16, kQkv>(a, args.head, c0 + 4 * lane);
  const int N = a.N, rows = args.rows, act = a.act;

  // Whether an earlier kernel gave up, read once a cluster: the word may change while this kernel
  // runs, and warps or CTAs that read it by themselves could take different ways (a CTA would
  // leave with its copies in flight, or sum partial sums nobody wrote).  All of them load and
  // multiply; the flag only withholds the stores, so its latency is hidden.
  if (rank == 0 && threadIdx.x == 64) *skip_flag = *reinterpret_cast<volatile int*>(a.status);

  if (warp == 0) {
    if (lane == 0) {
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
    if (lane == 0) {
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
  } else {
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
  if (splits > 1) cluster_sync_all();
  if (!*abort_flag) {
    const int skip =
        ld_cluster_s32(mapa_shared(smem_u32(const_cast<const int*>(skip_flag)), 0));
    const int tokens = min(kT, rows - t0);
    const int step = splits * (kSkinnyThreads / 32);
    const int first = rank + splits * warp;
    float4* sums = reinterpret_cast<float4*>(part) + lane;     // token t: sums[t * 32]
    // a warp's tokens: the sums over the cluster, into this CTA's own place for the token (which
    // no other CTA reads); the partial sums of one token, or of two where a warp has several, in
    // flight together
    constexpr int kAhead = kT >= 128 ? 2 : 1;
    if (splits > 1) {
      const uint32_t here = smem_u32(sums);
      for (int t = first; t < tokens; t += kAhead * step) {
        float4 v[kAhead][8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          if (r < splits) {
            const uint32_t peer = mapa_shared(here, (uint32_t)r);
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
              if (t + i * step < tokens) v[i][r] = ld_cluster_f4(peer + (uint32_t)(t + i * step) * 512u);
          }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (t + i * step >= tokens) break;
          float4 s = v[i][0];
#pragma unroll
          for (int r = 1; r < 8; ++r)
            if (r < splits) {
              s.x += v[i][r].x; s.y += v[i][r].y; s.z += v[i][r].z; s.w += v[i][r].w;
            }
          sums[(t + i * step) * 32] = s;
        }
      }
    }
    // then each token by itself
    mine.ok = mine.ok && skip == 0;
    const bool run_on = rows != N;                     // rows go through all branches
#pragma unroll kAhead
    for (int t = first; t < tokens; t += step) {
      const int row = t0 + t;
      const int b = run_on ? row / N : z;
      skinny_finish<kBF16, kQkv>(args.head, act, mine, sums[t * 32], b, run_on ? row - b * N : row);
    }
  }
  // no CTA leaves while its partial sums may still be read
  if (splits > 1)
    cluster_sync_all();
  else
    __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) atomicExch(a.status, 1);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
}

}  // namespace tara
