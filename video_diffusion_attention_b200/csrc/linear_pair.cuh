// linear_pair.cuh -- the 16-bit linear layer and Q/K/V projection on SM pairs.
//
//   y = residual + gate * act(x W^T + bias)        or        [q | k | v] = x W^T + bias
//                                                            with q, k normalised and rotated
//
// Tensor-bound: 2*M*K*C operations against (M*K + C*K + M*C) 16-bit words.  One persistent
// cluster of two CTAs per SM pair walks output tiles of 256 rows x BN columns.  Each CTA holds
// 128 rows of x (its half of the M = 256 operand) and BN/2 rows of W (half of the N operand),
// so every operand byte is loaded into one SM only; the even CTA's MMA warp issues
// tcgen05.mma.cta_group::2 on a ring of 64-column K steps.  Accumulators are double-buffered in
// tensor memory, so the epilogue of a tile runs under the next tile's products.
//
// Epilogue: 8 warps, thread = row (32x32b TMEM loads), 128 columns a warp and tile: at BN = 256
// the two warpgroups take the two column halves of every tile, at BN = 128 they take turns.  A
// warp therefore always holds whole heads (128 = one head of 128 or two of 64) and the norm of a
// head is a sum inside one thread.  Bias, gate and norm weights of the warp's columns are
// staged in shared memory as fp32; the residual is read with coalesced 16-byte loads (issued
// before the wait for the accumulators) and turned to row order through the same swizzled
// buffer the output leaves from by TMA store, which clips at the view's last row.
#pragma once

#include "linear_common.cuh"
#include "linear_ptx.cuh"

namespace tara {

constexpr int kPairLinThreads = 320;   // warp 0 loads, warp 1 issues MMAs, warps 2-9 epilogue

template <int BN>
struct PairLin {
  static constexpr int kABytes = 128 * 128;              // 128 rows x 64 columns
  static constexpr int kBBytes = (BN / 2) * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = BN == 256 ? 5 : 7;
  static constexpr int kOutBytes = 8 * 4096;             // per warp: 32 rows x 64 columns
  static constexpr int kVecBytes = 8 * 2 * 128 * 4;      // per warp: two fp32 vectors
  static constexpr int kBarCount = 2 * kStages + 4 + 2;
  static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kOutBytes + kVecBytes +
                                    kBarCount * 8 + 16;
  static constexpr uint32_t kTmemCols = 2 * BN;
  static_assert(kSmemBytes <= 232448, "dynamic shared memory above the 227 KB per-CTA limit");
};

// Norm and rotation of the projection's q and k (kQkv kernels).
struct HeadArgs {
  const void* weight[2];   // q, k; nullptr: 1
  long long weight_h;      // elements between heads' weights
  const float* table;
  long long table_b;
  int D, rot, halves, norm;
  float eps, inv_d;
};

struct PairLinMaps {
  CUtensorMap x, w, y[3];
};

struct PairLinArgs {
  LinearArgs lin;
  HeadArgs head;
  int m_tiles, n_tiles;    // 256-row tiles of one branch, BN-column tiles
  int group;               // row tiles walked together (L2 reuse of W)
};

template <bool kBF16, int BN, bool kQkv>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairLinThreads, 1)
linear_pair_kernel(const __grid_constant__ PairLinMaps maps,
                   const __grid_constant__ PairLinArgs args) {
  using S = PairLin<BN>;
  constexpr int NS = S::kStages;
  const LinearArgs& a = args.lin;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_out = smem + NS * S::kStageBytes;
  float* s_vec = reinterpret_cast<float*>(s_out + S::kOutBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_out + S::kOutBytes + S::kVecBytes);
  uint64_t* full = bars;                 // even CTA: both CTAs' parts of a stage landed
  uint64_t* empty = full + NS;           // both CTAs (2-SM commit): the stage was read
  uint64_t* acc_full = empty + NS;       // [2] both CTAs (2-SM commit): accumulators complete
  uint64_t* acc_empty = acc_full + 2;    // [2] even CTA: epilogue warps have read them
  uint64_t* drain = acc_empty + 2;       // even CTA: every MMA has completed
  uint64_t* exit_bar = drain + 1;        // the peer is done with this CTA's memory
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(exit_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int k_steps = (a.K + 63) / 64;
  const int rows_t = a.B * args.m_tiles;               // row tiles of all branches
  const int n_tiles_total = rows_t * args.n_tiles;
  const int n_clusters = (int)(gridDim.x >> 1);
  const int first = (int)(blockIdx.x >> 1);

  // Tile t: row tiles go in groups; inside a group the rows vary fastest, so the clusters that
  // run together share a few row tiles of x and a few column tiles of W.
  auto decode = [&](int t, int& b, int& m0, int& c0) {
    const int span = args.group * args.n_tiles;
    const int g = t / span, r = t - g * span;
    const int rows = min(args.group, rows_t - g * args.group);
    const int mt = g * args.group + r % rows;
    c0 = (r / rows) * BN;
    b = mt / args.m_tiles;
    m0 = (mt - b * args.m_tiles) * 256;
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      // warps of both CTAs that read buffer i of a tile: both warpgroups at BN = 256, one at 128
      mbar_init(&acc_empty[i], BN == 256 ? 16 : 8);
    }
    mbar_init(drain, 1);
    mbar_init(exit_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  cluster_sync_all();
  // one decision for both CTAs: skip all work if an earlier kernel gave up
  if (threadIdx.x == 0 && leader) {
    const int st = *reinterpret_cast<volatile int*>(a.status) != 0 ? 1 : 0;
    const uint32_t peer_flag = mapa_shared(smem_u32((const void*)abort_flag), 1);
    *abort_flag = st;
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer_flag), "r"(st) : "memory");
  }
  cluster_sync_all();
  if (*abort_flag) return;

  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, S::kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------ TMA producer (both CTAs) -------------------------
      tma_prefetch_desc(&maps.x);
      tma_prefetch_desc(&maps.w);
      bool ok = true;
      int it = 0;
      const int xD = a.x.D;
      for (int t = first; ok && t < n_tiles_total; t += n_clusters) {
        int b, m0, c0;
        decode(t, b, m0, c0);
        const int row = m0 + (int)rank * 128;
        const int wrow = c0 + (int)rank * (BN / 2);
        int h = 0, d = 0;      // column of x: (head, column of the head)
        for (int k = 0; k < k_steps; ++k, ++it) {
          const int slot = it % NS;
          if (!(ok = mbar_wait(&empty[slot], ((uint32_t)(it / NS) & 1u) ^ 1u, abort_flag,
                               kLinWaitNs)))
            break;
          if (leader) mbar_arrive_expect_tx(&full[slot], 2 * S::kStageBytes);
          const uint32_t full_l = mapa_shared(smem_u32(&full[slot]), 0);
          const uint32_t dst = smem_u32(smem + slot * S::kStageBytes);
          tma_load_4d_pair(dst, &maps.x, full_l, d, row, h, b);
          tma_load_2d_pair(dst + S::kABytes, &maps.w, full_l, k * 64, wrow);
          if ((d += 64) >= xD) {
            d = 0;
            ++h;
          }
        }
      }
      if (*abort_flag && it > 0) {
        // copies already issued land within microseconds; their completion is counted in the
        // even CTA, so give them 1 ms before this CTA's shared memory can be released
        for (int w = 0; w < 1000; ++w) __nanosleep(1000);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ------------------------------ MMA issuer (even CTA) ----------------------------
      constexpr uint32_t idesc = make_idesc_f16(256, BN, kBF16, false);
      const uint64_t ad0 = make_sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t bd0 = make_sdesc_sw128(smem_u32(smem + S::kABytes), 16, 1024);
      bool ok = true;
      int it = 0, n = 0;
      for (int t = first; ok && t < n_tiles_total; t += n_clusters, ++n) {
        const int buf = n & 1;
        if (n >= 2 && !(ok = mbar_wait(&acc_empty[buf], ((uint32_t)(n >> 1) & 1u) ^ 1u, abort_flag,
                                       kLinWaitNs)))
          break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(buf * BN);
        for (int k = 0; k < k_steps; ++k, ++it) {
          const int slot = it % NS;
          if (!(ok = mbar_wait(&full[slot], (uint32_t)(it / NS) & 1u, abort_flag, kLinWaitNs)))
            break;
          tc_fence_after();
          const uint64_t off = (uint64_t)((slot * S::kStageBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_ss_pair(d, ad0 + off + kk * 2, bd0 + off + kk * 2, idesc, (k > 0 || kk > 0) ? 1u : 0u);
          umma_commit_pair(&empty[slot]);
        }
        if (ok) umma_commit_pair(&acc_full[buf]);
      }
      // every MMA this thread issued completes before either CTA releases its memory
      umma_commit_pair(drain);
      volatile int no_abort = 0;
      mbar_wait(drain, 0, &no_abort, kLinDrainNs);
    }
  } else {
    // ------------------------------ epilogue warps (both CTAs) -------------------------
    const int wq = warp & 3;                 // TMEM lane quarter
    const int grp = (warp - 2) >> 2;         // warpgroup: column half (256) or tile parity (128)
    const int ew = warp - 2;
    const uint32_t out = smem_u32(s_out + ew * 4096);
    const uint32_t own = out + (uint32_t)(lane * 128);       // this thread's row of the buffer
    const uint32_t sw = (uint32_t)(lane & 7);
    float* vec0 = s_vec + ew * 256;          // bias
    float* vec1 = vec0 + 128;                // gate, or the norm's weight
    const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
    bool ok = true;
    int n = 0;
    for (int t = first; ok && t < n_tiles_total; t += n_clusters, ++n) {
      if (BN == 128 && (n & 1) != grp) continue;
      const int buf = n & 1;
      int b, m0, c0;
      decode(t, b, m0, c0);
      if (BN == 256) c0 += grp * 128;
      const int r0 = m0 + (int)rank * 128 + wq * 32;         // the warp's first row
      const bool rows_ok = r0 < a.N;
      const uint32_t acc = tmem + lane_base + (uint32_t)(buf * BN + (BN == 256 ? grp * 128 : 0));

      // ---- per-column vectors of the warp's 128 columns: 4 a lane, zero past the last column
      __syncwarp();
      {
        const int c = c0 + 4 * lane;
        float4 v0 = make_float4(0.f, 0.f, 0.f, 0.f), v1 = make_float4(1.f, 1.f, 1.f, 1.f);
        if (c < a.C) {
          auto load4 = [](const void* p, long long i) {
            const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
            const float2 lo = unpack16<kBF16>(w.x), hi = unpack16<kBF16>(w.y);
            return make_float4(lo.x, lo.y, hi.x, hi.y);
          };
          if (a.bias) v0 = load4(a.bias, c);
          if (kQkv) {
            const int part = c / a.part_cols;
            if (part < 2 && args.head.weight[part] != nullptr) {
              const int pc = c - part * a.part_cols, h = pc / args.head.D;
              v1 = load4(args.head.weight[part], h * args.head.weight_h + (pc - h * args.head.D));
            }
          } else if (a.gate) {
            v1 = load4(a.gate, b * a.gate_b + c);
          }
        }
        reinterpret_cast<float4*>(vec0)[lane] = v0;
        reinterpret_cast<float4*>(vec1)[lane] = v1;
      }
      __syncwarp();

      // ---- residual of the first 64 columns, in flight while the products run: 16 bytes a lane,
      // 8 lanes a row, 4 rows a load
      uint4 res[8];
      auto load_residual = [&](int chunk) {
        const int c = c0 + chunk * 64 + (lane & 7) * 8;
        const bool c_ok = c < a.C;
        const uint16_t* p = static_cast<const uint16_t*>(a.residual.ptr) +
                            row_offset(a.residual, b, 0, c_ok ? c : 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int row = r0 + i * 4 + (lane >> 3);
          res[i] = make_uint4(0u, 0u, 0u, 0u);
          if (c_ok && row < a.N)
            res[i] = *reinterpret_cast<const uint4*>(p + (long long)row * a.residual.n);
        }
      };
      if (!kQkv && a.residual.ptr) load_residual(0);

      if (!(ok = mbar_wait_warp(&acc_full[buf], (uint32_t)(n >> 1) & 1u, abort_flag))) break;
      tc_fence_after();

      float rstd[2] = {1.f, 1.f};            // of the warp's one or two heads
      int hcols = 128;                       // columns of a head
      if (kQkv) {
        hcols = args.head.D;
        if (args.head.norm && c0 < 2 * a.part_cols) {
#pragma unroll 1
          for (int h = 0; h < 128 / hcols; ++h) {
            float ss = 0.f;
#pragma unroll 1
            for (int p = 0; p < hcols; p += 32) {
              uint32_t v[32];
              tmem_ld32(acc + h * hcols + p, v);
              tmem_ld_wait();
              reg_fence<32>(v);
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float x = __uint_as_float(v[i]) + vec0[h * hcols + p + i];
                ss = fmaf(x, x, ss);
              }
            }
            rstd[h] = __frsqrt_rn(fmaf(ss, args.head.inv_d, args.head.eps));
          }
        }
      }

#pragma unroll 1
      for (int chunk = 0; chunk < 2; ++chunk) {
        const int cc = c0 + chunk * 64;      // first column of the chunk
        // the buffer's last store has read it
        if (lane == 0) bulk_wait_read();
        __syncwarp();
        if (!kQkv && a.residual.ptr) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t row = (uint32_t)(i * 4 + (lane >> 3));
            st_shared_v4(out + row * 128 + ((((uint32_t)lane & 7u) ^ (row & 7u)) << 4), res[i].x,
                         res[i].y, res[i].z, res[i].w);
          }
          __syncwarp();
          if (chunk == 0) load_residual(1);
        }
        // which output the chunk belongs to: parts begin at multiples of 64 columns
        const int part = cc / a.part_cols;
        const bool turn = kQkv && part < 2 && args.head.table != nullptr;
#pragma unroll 1
        for (int p = 0; p < 64; p += 32) {
          const int col = chunk * 64 + p;    // within the warp's 128 columns
          uint32_t v[32];
          tmem_ld32(acc + col, v);
          if (!kQkv) {
            tmem_ld_wait();
            reg_fence<32>(v);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float f[8];
              const uint32_t slot16 = own + ((((uint32_t)(p / 8 + q)) ^ sw) << 4);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                f[i] = apply_act(__uint_as_float(v[q * 8 + i]) + vec0[col + q * 8 + i], a.act);
              if (a.gate) {
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] *= vec1[col + q * 8 + i];
              }
              if (a.residual.ptr) {
                const uint4 rw = ld_shared_v4(slot16);
                const uint32_t w[4] = {rw.x, rw.y, rw.z, rw.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float2 rf = unpack16<kBF16>(w[i]);
                  f[2 * i] += rf.x;
                  f[2 * i + 1] += rf.y;
                }
              }
              st_shared_v4(slot16, pack16<kBF16>(f[0], f[1]), pack16<kBF16>(f[2], f[3]),
                           pack16<kBF16>(f[4], f[5]), pack16<kBF16>(f[6], f[7]));
            }
          } else {
            const int h = col / hcols;                       // head within the warp's columns
            const int d0 = col - h * hcols;                  // first column within the head
            const bool normed = part < 2 && args.head.norm;
            const float r = normed ? rstd[h] : 1.f;
            const int half = args.head.rot / 2;
            uint32_t u[32];                                  // the pairs' other columns (halves)
            if (turn && args.head.halves) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int d = d0 + q * 8;
                const int other = d < half ? d + half : (d < 2 * half ? d - half : d);
                tmem_ld8(acc + h * hcols + other, u + q * 8);
              }
            }
            tmem_ld_wait();
            reg_fence<32>(v);
            if (turn && args.head.halves) reg_fence<32>(u);
            const long long row = min(r0 + lane, a.N - 1);
            const float* cs = turn ? args.head.table + b * args.head.table_b + row * args.head.rot
                                   : nullptr;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float f[8];
              const int d = d0 + q * 8;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                f[i] = __uint_as_float(v[q * 8 + i]) + vec0[col + q * 8 + i];
                if (normed) f[i] *= r * vec1[col + q * 8 + i];
              }
              if (turn && d < args.head.rot) {
                if (args.head.halves) {
                  const int other = d < half ? d + half : d - half;
                  const float4* c4 = reinterpret_cast<const float4*>(cs + 2 * (d < half ? d : d - half));
                  const float sign = d < half ? -1.f : 1.f;
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const float4 t4 = c4[i];
                    const int o = h * hcols + other + 2 * i;
                    float g0 = __uint_as_float(u[q * 8 + 2 * i]) + vec0[o];
                    float g1 = __uint_as_float(u[q * 8 + 2 * i + 1]) + vec0[o + 1];
                    if (normed) {
                      g0 *= r * vec1[o];
                      g1 *= r * vec1[o + 1];
                    }
                    f[2 * i] = fmaf(f[2 * i], t4.x, sign * g0 * t4.y);
                    f[2 * i + 1] = fmaf(f[2 * i + 1], t4.z, sign * g1 * t4.w);
                  }
                } else {
                  const float4* c4 = reinterpret_cast<const float4*>(cs + d);
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    const float4 t4 = c4[i];
                    const float x0 = f[4 * i], y0 = f[4 * i + 1], x1 = f[4 * i + 2], y1 = f[4 * i + 3];
                    f[4 * i] = fmaf(x0, t4.x, -y0 * t4.y);
                    f[4 * i + 1] = fmaf(x0, t4.y, y0 * t4.x);
                    f[4 * i + 2] = fmaf(x1, t4.z, -y1 * t4.w);
                    f[4 * i + 3] = fmaf(x1, t4.w, y1 * t4.z);
                  }
                }
              }
              st_shared_v4(own + ((((uint32_t)(p / 8 + q)) ^ sw) << 4), pack16<kBF16>(f[0], f[1]),
                           pack16<kBF16>(f[2], f[3]), pack16<kBF16>(f[4], f[5]),
                           pack16<kBF16>(f[6], f[7]));
            }
          }
        }
        if (chunk == 1) {
          // the accumulators are read: the MMA warp may start the tile after next in them
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&acc_empty[buf]), 0));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && rows_ok && cc < a.C) {
          const int pc = cc - part * a.part_cols;
          const int yD = a.y[part].D;
          const int h = pc / yD;
          tma_store_4d(&maps.y[part], out, pc - h * yD, r0, h, b);
          bulk_commit();
        }
      }
    }
    if (lane == 0) bulk_wait_all();
    tc_fence_before();
  }

  __syncthreads();
  // neither CTA of the pair leaves (and frees its shared and tensor memory) before the other
  // is done with the pair's barriers and operands; bounded
  if (threadIdx.x == 0) {
    mbar_arrive_cluster(mapa_shared(smem_u32(exit_bar), rank ^ 1u));
    volatile int no_abort = 0;
    mbar_wait(exit_bar, 0, &no_abort, kLinWaitNs);
    if (*abort_flag) atomicExch(a.status, 1);
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, S::kTmemCols);
  }
}

}  // namespace tara
