// linear_pair.cuh -- the 16-bit linear layer and Q/K/V projection on SM pairs.
//
//   y = residual + gate * act(x W^T + bias)        or        [q | k | v] = x W^T + bias
//                                                            with q, k normalised and rotated
//
// Tensor-bound: 2*M*K*C operations against (M*K + C*K + M*C) 16-bit words.  One persistent
// cluster of two CTAs per SM pair walks output tiles of 256*kSubs rows x BN columns.  Each CTA
// holds 128 rows of x per sub-tile (its half of an M = 256 operand) and BN/2 rows of W (half of
// the N operand), so every operand byte is loaded into one SM only; the even CTA's MMA warp
// issues tcgen05.mma.cta_group::2 on a ring of 64-column K steps.  The two accumulators in
// tensor memory are the two sub-tiles of a tile (kSubs = 2), or take turns over tiles, the
// epilogue of one tile running under the next tile's products (kSubs = 1).
//
// Epilogue: 8 warps, thread = row (32x32b TMEM loads), 128 columns a warp and accumulator: at
// BN = 256 the two warpgroups take the two column halves of every accumulator, at BN = 128 they
// take turns.  A warp therefore always holds whole heads (128 = one head of 128 or two of 64)
// and the norm of a head is a sum inside one thread.  Columns go in pieces of four blocks of
// eight; whatever is per row and column (residual, (cos, sin) pairs, the output) crosses between
// the row-per-thread order of the accumulators and coalesced global accesses through 4 KB of
// swizzled shared memory per warp, and is loaded one piece ahead.  (Row-per-thread accesses to
// the table made the projection's epilogue 15,700 cycles a unit of 128 x 256; TMA stores from
// one buffer made the plain one 5,300, waiting for each store to read it.)  Bias, gate and norm
// weights are the same for all lanes and come through L1.
#pragma once

#include "linear_common.cuh"
#include "linear_ptx.cuh"

namespace tara {

constexpr int kPairLinThreads = 320;   // warp 0 loads, warp 1 issues MMAs, warps 2-9 epilogue

template <int BN, int kSubs>
struct PairLin {
  static constexpr int kABytes = kSubs * 128 * 128;      // kSubs x 128 rows x 64 columns
  static constexpr int kBBytes = (BN / 2) * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = 196608 / kStageBytes;   // 4, 6 or 8 stages
  static constexpr int kOutBytes = 8 * 4096;             // 4 KB of staging per warp
  static constexpr int kBarCount = 2 * kStages + 4 + 2;
  static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kOutBytes + kBarCount * 8 + 16;
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
  CUtensorMap x, w;
};

struct PairLinArgs {
  LinearArgs lin;
  HeadArgs head;
  int m_tiles, n_tiles;    // row tiles of one branch, column tiles
  int group;               // row tiles walked together (L2 reuse of W)
};

// ---- staging: 32 rows x 64 bytes (a piece of the output or the residual) or 32 rows x 128 bytes
// (16 (cos, sin) pairs), 16-byte chunks swizzled so that both a row per thread and whole rows by
// neighbouring lanes are free of bank conflicts
__device__ __forceinline__ uint32_t stage64(uint32_t buf, int row, int chunk) {
  return buf + (uint32_t)(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
}
__device__ __forceinline__ uint32_t stage128(uint32_t buf, int row, int chunk) {
  return buf + (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4));
}

// What one warp works on: 32 rows from r0 of branch b, 128 columns from c0, their accumulators.
struct PairWarp {
  uint32_t acc;      // tensor memory: lane quarter and first column
  uint32_t buf;      // staging
  int b, r0, c0, lane;
};

// 32 columns of the residual: 4 lanes a row, 8 rows a load.
__device__ __forceinline__ void pair_load_residual(const LinearArgs& a, const PairWarp& w, int cc,
                                                   uint4 (&res)[4]) {
  const int c = cc + (w.lane & 3) * 8;
  const int row = w.r0 + (w.lane >> 2);
  const bool c_ok = c < a.C;
  const uint16_t* p = static_cast<const uint16_t*>(a.residual.ptr) +
                      row_offset(a.residual, w.b, row, c_ok ? c : 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    res[i] = make_uint4(0u, 0u, 0u, 0u);
    if (c_ok && row + i * 8 < a.N)
      res[i] = *reinterpret_cast<const uint4*>(p + (long long)(i * 8) * a.residual.n);
  }
}

// The staged piece -> y: blocks of eight columns from column `col` (of the output's row) of this
// lane's chunk; `ok`: the chunk is inside the output.
__device__ __forceinline__ void pair_store(const LinearArgs& a, const RowView& y, const PairWarp& w,
                                           int col, bool ok) {
  const int row = w.lane >> 2;
  uint16_t* p = static_cast<uint16_t*>(const_cast<void*>(y.ptr)) +
                row_offset(y, w.b, w.r0 + row, col);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 v = ld_shared_v4(stage64(w.buf, row + i * 8, w.lane & 3));
    if (ok && w.r0 + row + i * 8 < a.N)
      *reinterpret_cast<uint4*>(p + (long long)(i * 8) * y.n) = v;
  }
}

// residual + gate * act(accumulator + bias) of the warp's 128 columns.  `res`: the first piece
// of the residual.
template <bool kBF16>
__device__ __forceinline__ void pair_linear(const LinearArgs& a, const PairWarp& w, uint4 (&res)[4]) {
  const bool with_res = a.residual.ptr != nullptr;
#pragma unroll 1
  for (int p = 0; p < 128; p += 32) {
    const int cc = w.c0 + p;
    if (cc >= a.C) break;
    uint32_t v[32];
    tmem_ld32(w.acc + p, v);
    uint4 bias[4], gate[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = cc + q * 8;
      bias[q] = gate[q] = make_uint4(0u, 0u, 0u, 0u);
      if (a.bias && c < a.C) bias[q] = ldg16(a.bias, c);
      if (a.gate && c < a.C) gate[q] = ldg16(a.gate, w.b * a.gate_b + c);
    }
    if (with_res) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        st_shared_v4(stage64(w.buf, i * 8 + (w.lane >> 2), w.lane & 3), res[i].x, res[i].y, res[i].z,
                     res[i].w);
      __syncwarp();
      if (p < 96) pair_load_residual(a, w, cc + 32, res);
    }
    tmem_ld_wait();
    reg_fence<32>(v);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t slot = stage64(w.buf, w.lane, q);
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[q * 8 + i]);
      if (a.bias) {
        float t[8];
        unpack8<kBF16>(bias[q], t);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] += t[i];
      }
      activate_all(f, a.act);
      if (a.gate) {
        float t[8];
        unpack8<kBF16>(gate[q], t);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= t[i];
      }
      if (with_res) {
        float t[8];
        unpack8<kBF16>(ld_shared_v4(slot), t);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] += t[i];
      }
      st_shared_v4(slot, pack16<kBF16>(f[0], f[1]), pack16<kBF16>(f[2], f[3]),
                   pack16<kBF16>(f[4], f[5]), pack16<kBF16>(f[6], f[7]));
    }
    __syncwarp();
    const int part = cc / a.part_cols;     // parts begin at multiples of 64 columns
    const int chunk_col = cc + (w.lane & 3) * 8;
    pair_store(a, a.y[part], w, chunk_col < a.C ? chunk_col - part * a.part_cols : 0,
               chunk_col < a.C);
    __syncwarp();
  }
}

// Bias of 8 columns from column c (zeros without one).
template <bool kBF16>
__device__ __forceinline__ void pair_bias8(const LinearArgs& a, int c, float (&f)[8]) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (a.bias) v = ldg16(a.bias, c);
  unpack8<kBF16>(v, f);
}

// 16 (cos, sin) pairs, number 16 * piece on, of the warp's rows: 8 lanes a row, 4 rows a load.
__device__ __forceinline__ void pair_load_table(const LinearArgs& a, const HeadArgs& head,
                                                const PairWarp& w, int piece, uint4 (&cs)[8]) {
  const int f = piece * 32 + (w.lane & 7) * 4;
  const int row = w.r0 + (w.lane >> 3);
  const float* p = head.table + w.b * head.table_b + (long long)row * head.rot + f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    cs[i] = make_uint4(0u, 0u, 0u, 0u);
    if (f < head.rot && row + i * 4 < a.N)
      cs[i] = __ldg(reinterpret_cast<const uint4*>(p + (long long)(i * 4) * head.rot));
  }
}

// Bias, norm and rotation of the heads in the warp's 128 columns.  `cs`: the first piece of the
// table.
template <bool kBF16>
__device__ __forceinline__ void pair_heads(const LinearArgs& a, const HeadArgs& head,
                                           const PairWarp& w, uint4 (&cs)[8]) {
  const int D = head.D;
  const int half = head.rot / 2;
#pragma unroll 1
  for (int hd = 0; hd < 128; hd += D) {
    const int c_h = w.c0 + hd;                         // the head's first column
    if (c_h >= a.C) break;
    const int part = c_h / a.part_cols;
    const int pc_h = c_h - part * a.part_cols;
    const bool turn = part < 2 && head.table != nullptr;
    const bool normed = part < 2 && head.norm;
    const uint32_t acc = w.acc + hd;

    float r = 1.f;
    if (normed) {
      float ss[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int d = 0; d < D; d += 32) {
        uint32_t v[32];
        tmem_ld32(acc + d, v);
        float t[4][8];
#pragma unroll
        for (int q = 0; q < 4; ++q) pair_bias8<kBF16>(a, c_h + d + q * 8, t[q]);
        tmem_ld_wait();
        reg_fence<32>(v);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float x = __uint_as_float(v[i]) + t[i >> 3][i & 7];
          ss[i & 3] = fmaf(x, x, ss[i & 3]);
        }
      }
      r = __frsqrt_rn(fmaf((ss[0] + ss[1]) + (ss[2] + ss[3]), head.inv_d, head.eps));
    }
    const void* weight = normed ? head.weight[part] : nullptr;
    const long long w_h = pc_h / D * head.weight_h;

    // Pieces.  Half-split pairs: blocks [j, j + 8), [j + 8, j + 16) of the low columns and their
    // partners in the high ones, both halves of 16 pairs (then the columns behind R, 32 a piece);
    // otherwise 32 neighbouring columns.  Piece i turns by the pairs from 16 i.
    const bool split = turn && head.halves;
    const int turning = turn ? (head.rot + 31) / 32 : 0;
    const int pieces = split ? turning + (D - head.rot + 31) / 32 : D / 32;
#pragma unroll 1
    for (int i = 0; i < pieces; ++i) {
      const bool pairs = split && i < turning;
      const int first = pairs ? 16 * i : (split ? head.rot + 32 * (i - turning) : 32 * i);
      const int limit = pairs ? half : D;              // blocks from here on do not exist
      // first column of block q within the head
      auto block = [&](int q) {
        return pairs ? first + (q & 1) * 8 + (q >> 1) * half : first + q * 8;
      };
      auto exists = [&](int q) { return (pairs ? first + (q & 1) * 8 : first + q * 8) < limit; };
      uint32_t v[32];
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_ld8(acc + (exists(q) ? block(q) : 0), v + q * 8);
      float t[32];
      const bool turned = turn && i < turning;
      if (turned) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          st_shared_v4(stage128(w.buf, j * 4 + (w.lane >> 3), w.lane & 7), cs[j].x, cs[j].y, cs[j].z,
                       cs[j].w);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint4 c4 = ld_shared_v4(stage128(w.buf, w.lane, j));
          t[4 * j] = __uint_as_float(c4.x);
          t[4 * j + 1] = __uint_as_float(c4.y);
          t[4 * j + 2] = __uint_as_float(c4.z);
          t[4 * j + 3] = __uint_as_float(c4.w);
        }
        __syncwarp();
        // the next piece's pairs: this head's, or the next head's first
        pair_load_table(a, head, w, i + 1 < turning ? i + 1 : 0, cs);
      }
      float f[4][8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int d = exists(q) ? block(q) : 0;
        pair_bias8<kBF16>(a, c_h + d, f[q]);
        if (q == 0) {
          tmem_ld_wait();
          reg_fence<32>(v);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) f[q][j] += __uint_as_float(v[q * 8 + j]);
        if (normed) {
          float g[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
          if (weight) unpack8<kBF16>(ldg16(weight, w_h + d), g);
#pragma unroll
          for (int j = 0; j < 8; ++j) f[q][j] *= r * g[j];
        }
      }
      if (pairs) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float c = t[16 * q + 2 * j], s = t[16 * q + 2 * j + 1];
            const float x = f[q][j], y = f[q + 2][j];
            f[q][j] = fmaf(x, c, -y * s);
            f[q + 2][j] = fmaf(x, s, y * c);
          }
      } else if (turned) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (first + q * 8 >= head.rot) break;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float c = t[8 * q + 2 * j], s = t[8 * q + 2 * j + 1];
            const float x = f[q][2 * j], y = f[q][2 * j + 1];
            f[q][2 * j] = fmaf(x, c, -y * s);
            f[q][2 * j + 1] = fmaf(x, s, y * c);
          }
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
        st_shared_v4(stage64(w.buf, w.lane, q), pack16<kBF16>(f[q][0], f[q][1]),
                     pack16<kBF16>(f[q][2], f[q][3]), pack16<kBF16>(f[q][4], f[q][5]),
                     pack16<kBF16>(f[q][6], f[q][7]));
      __syncwarp();
      const int q = w.lane & 3;
      pair_store(a, a.y[part], w, pc_h + (exists(q) ? block(q) : 0), exists(q));
      __syncwarp();
    }
  }
}

template <bool kBF16, int BN, int kSubs, bool kQkv>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairLinThreads, 1)
linear_pair_kernel(const __grid_constant__ PairLinMaps maps,
                   const __grid_constant__ PairLinArgs args) {
  using S = PairLin<BN, kSubs>;
  constexpr int NS = S::kStages;
  const LinearArgs& a = args.lin;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_out = smem + NS * S::kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_out + S::kOutBytes);
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
    m0 = (mt - b * args.m_tiles) * (256 * kSubs);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      // warps of both CTAs that read accumulator i: both warpgroups at BN = 256, one at 128
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
      int slot = 0;
      uint32_t phase = 0;    // ring position: slot s of round r completes phase r of its barriers
      bool issued = false;
      const uint32_t full_l = mapa_shared(smem_u32(full), 0);
      const int xD = a.x.D;
      for (int t = first; ok && t < n_tiles_total; t += n_clusters) {
        int b, m0, c0;
        decode(t, b, m0, c0);
        const int row = m0 + (int)rank * 128;
        const int wrow = c0 + (int)rank * (BN / 2);
        // a second sub-tile wholly behind the last row is neither loaded nor multiplied
        const int subs = kSubs == 2 && m0 + 256 < a.N ? 2 : 1;
        const uint32_t bytes = 2u * (uint32_t)(subs * 16384 + S::kBBytes);
        int h = 0, d = 0;      // column of x: (head, column of the head)
        for (int k = 0; k < k_steps; ++k) {
          if (!(ok = mbar_wait_idle(&empty[slot], phase ^ 1u, abort_flag))) break;
          if (leader) mbar_arrive_expect_tx(&full[slot], bytes);
          const uint32_t bar = full_l + (uint32_t)slot * 8u;
          const uint32_t dst = smem_u32(smem) + (uint32_t)slot * S::kStageBytes;
          for (int u = 0; u < subs; ++u)
            tma_load_4d_pair(dst + u * 16384, &maps.x, bar, d, row + u * 256, h, b);
          tma_load_2d_pair(dst + S::kABytes, &maps.w, bar, k * 64, wrow);
          issued = true;
          if (++slot == NS) {
            slot = 0;
            phase ^= 1u;
          }
          if ((d += 64) >= xD) {
            d = 0;
            ++h;
          }
        }
      }
      if (*abort_flag && issued) {
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
      int slot = 0;
      uint32_t phase = 0;
      uint32_t unit = 0;     // accumulators started so far: unit u lives in half u & 1 of TMEM
      for (int t = first; ok && t < n_tiles_total; t += n_clusters, unit += kSubs) {
        int b, m0, c0;
        decode(t, b, m0, c0);
        const int subs = kSubs == 2 && m0 + 256 < a.N ? 2 : 1;
        // One K step of sub-tile u from ring slot s.
        auto multiply = [&](int u, int s, bool start) {
          const uint64_t off = (uint64_t)((s * S::kStageBytes) >> 4);
          const uint32_t d = tmem + ((unit + (uint32_t)u) & 1u) * BN;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_ss_pair(d, ad0 + off + (uint64_t)(u * (16384 >> 4) + kk * 2), bd0 + off + (uint64_t)(kk * 2),
                         idesc, (!start || kk > 0) ? 1u : 0u);
        };
        // The epilogue has read what accumulator u held two units ago (every phase is waited
        // for, also that of a sub-tile that is not multiplied).
        auto accumulator_free = [&](int u) {
          const uint32_t n = unit + (uint32_t)u;
          const bool done = n < 2 || mbar_wait_idle(&acc_empty[n & 1u], ((n >> 1) & 1u) ^ 1u, abort_flag);
          tc_fence_after();
          return done;
        };
        auto advance = [&]() {
          if (++slot == NS) {
            slot = 0;
            phase ^= 1u;
          }
        };
        if (!(ok = accumulator_free(0))) break;
        int k = 0;
        if (kSubs == 2) {
          // the second accumulator is still being read out: the first runs ahead through the
          // stages of the ring, then the second catches up and releases them
          const int lead = min(NS, k_steps);
          const int slot0 = slot;
          for (; ok && k < lead; ++k) {
            if (!(ok = mbar_wait_idle(&full[slot], phase, abort_flag))) break;
            tc_fence_after();
            multiply(0, slot, k == 0);
            advance();
          }
          if (!ok || !(ok = accumulator_free(1))) break;
          for (int i = 0; i < lead; ++i) {
            const int s = slot0 + i < NS ? slot0 + i : slot0 + i - NS;
            if (subs == 2) multiply(1, s, i == 0);
            umma_commit_pair(&empty[s]);
          }
        }
        for (; k < k_steps; ++k) {
          if (!(ok = mbar_wait_idle(&full[slot], phase, abort_flag))) break;
          tc_fence_after();
          multiply(0, slot, k == 0);
          if (kSubs == 2 && subs == 2) multiply(1, slot, false);
          umma_commit_pair(&empty[slot]);
          advance();
        }
        if (ok)
          for (int u = 0; u < kSubs; ++u) umma_commit_pair(&acc_full[(unit + (uint32_t)u) & 1u]);
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
    const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
    PairWarp w;
    w.buf = smem_u32(s_out + ew * 4096);
    w.lane = lane;
    bool ok = true;
    uint32_t unit = 0;
    for (int t = first; ok && t < n_tiles_total; t += n_clusters) {
      int m0;
      decode(t, w.b, m0, w.c0);
      if (BN == 256) w.c0 += grp * 128;
#pragma unroll 1
      for (int u = 0; u < kSubs; ++u, ++unit) {
        const uint32_t half = unit & 1u;
        if (BN == 128 && half != (uint32_t)grp) continue;
        w.r0 = m0 + u * 256 + (int)rank * 128 + wq * 32;
        w.acc = tmem + lane_base + half * BN + (BN == 256 ? grp * 128 : 0);
        const bool live = w.r0 < a.N && w.c0 < a.C;
        // the first piece of what comes from memory, in flight while the products run
        uint4 ahead[kQkv ? 8 : 4];
        if (live) {
          if constexpr (kQkv) {
            if (args.head.table) pair_load_table(a, args.head, w, 0, ahead);
          } else {
            if (a.residual.ptr) pair_load_residual(a, w, w.c0, ahead);
          }
        }
        if (!(ok = mbar_wait_warp(&acc_full[half], (unit >> 1) & 1u, abort_flag))) break;
        tc_fence_after();
        if (live) {
          if constexpr (kQkv)
            pair_heads<kBF16>(a, args.head, w, ahead);
          else
            pair_linear<kBF16>(a, w, ahead);
        }
        // the accumulator is read: the MMA warp may start the unit after next in it
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&acc_empty[half]), 0));
      }
    }
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
