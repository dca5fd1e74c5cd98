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

#include <type_traits>

#include "linear_common.cuh"
#include "linear_ptx.cuh"

namespace tara {

// Warp 0 loads, warp 1 issues MMAs, warps 4-11 are the epilogue (warps 2 and 3 complete the
// control warpgroup).  The launch gives every thread kPairLinRegs registers; the control
// warpgroup lowers its share and the two epilogue warpgroups raise theirs.  The sum must equal
// the launch pool, or the raise would wait for registers that never come; the host refuses to
// launch when ptxas gave the kernel another count.
constexpr int kPairLinThreads = 384;
constexpr int kPairLinRegs = 168;
constexpr int kPairLinControlRegs = 88;
constexpr int kPairLinEpilogueRegs = 208;
static_assert(128 * kPairLinControlRegs + 256 * kPairLinEpilogueRegs == kPairLinThreads * kPairLinRegs,
              "register split must use the launch pool exactly");

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
  int bn;                  // columns of a tile: BN, or less (a multiple of 16) where one head and
                           // one part make up the output's row
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
  uint32_t release;  // shared::cluster address of the accumulator's acc_empty barrier
  int b, r0, c0, lane;
  int c_end;         // the tile's columns end here
};

// The warp has read its part of the accumulator: the MMA warp may start the unit after next in it.
__device__ __forceinline__ void pair_release(const PairWarp& w) {
  tc_fence_before();
  __syncwarp();
  if (w.lane == 0) mbar_arrive_cluster(w.release);
}

// Everything the linear epilogue of one accumulator reads of the kernel's arguments, gathered in
// registers before the products are complete: behind the barriers and shared-memory accesses,
// which are opaque to the compiler, arguments would be fetched again each time.  Its loops stay
// rolled: with all 128 columns in registers and every piece unrolled a unit took 6,600 cycles,
// as it stands 3,200 to 4,500 (of which the stores, at the rate L1 passes them on, 1,500).
struct PairLinearAhead {
  uint16_t* y[2];            // this lane's chunk of each 64 columns' first piece, first row
  const uint16_t* r[2];      // the same of the residual
  long long y_n[2], r_n;     // row strides
  const uint16_t *bias, *gate;
  int cols, rows;            // columns and rows of the warp's part that exist
  bool with_res;
  uint4 res[4];              // the next piece of the residual
};

// 32 columns of the residual from this lane's chunk at `src`: 4 lanes a row, 8 rows a load.
__device__ __forceinline__ void pair_load_residual(const PairLinearAhead& ah, int lane,
                                                   const uint16_t* src, int cols, uint4 (&res)[4]) {
  const int row = lane >> 2;
  const bool c_ok = (lane & 3) * 8 < cols;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    res[i] = make_uint4(0u, 0u, 0u, 0u);
    if (c_ok && row + i * 8 < ah.rows)
      res[i] = *reinterpret_cast<const uint4*>(src + (long long)(i * 8) * ah.r_n);
  }
}

__device__ __forceinline__ void pair_linear_ahead(const LinearArgs& a, const PairWarp& w,
                                                  PairLinearAhead& ah) {
  ah.cols = min(128, w.c_end - w.c0);
  ah.rows = min(32, a.N - w.r0);
  ah.bias = a.bias ? static_cast<const uint16_t*>(a.bias) + w.c0 : nullptr;
  ah.gate = a.gate ? static_cast<const uint16_t*>(a.gate) + w.b * a.gate_b + w.c0 : nullptr;
  ah.with_res = a.residual.ptr != nullptr;
  ah.r_n = a.residual.n;
  const int row = w.r0 + (w.lane >> 2);
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    // heads and parts begin at multiples of 64 columns (or there is one of each)
    const int c = min(w.c0 + p * 64, a.C - 8);
    const int part = c < a.part_cols ? 0 : c / a.part_cols;
    const RowView& y = a.y[part];
    ah.y[p] = static_cast<uint16_t*>(const_cast<void*>(y.ptr)) +
              row_offset(y, w.b, row, c - part * a.part_cols) + (w.lane & 3) * 8;
    ah.y_n[p] = y.n;
    ah.r[p] = nullptr;
    if (ah.with_res)
      ah.r[p] = static_cast<const uint16_t*>(a.residual.ptr) + row_offset(a.residual, w.b, row, c) +
                (w.lane & 3) * 8;
  }
  if (ah.with_res) pair_load_residual(ah, w.lane, ah.r[0], ah.cols, ah.res);
}

// residual + gate * act(accumulator + bias) of the warp's 128 columns, 32 at a time.
template <bool kBF16, int kAct>
__device__ __forceinline__ void pair_linear(const PairWarp& w, PairLinearAhead& ah) {
#pragma unroll 1
  for (int p = 0; p < 4; ++p) {
    const int left = ah.cols - p * 32;
    if (left <= 0) break;
    uint32_t v[32];
    tmem_ld32(w.acc + p * 32, v);
    if (ah.with_res) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        st_shared_v4(stage64(w.buf, i * 8 + (w.lane >> 2), w.lane & 3), ah.res[i].x, ah.res[i].y,
                     ah.res[i].z, ah.res[i].w);
      __syncwarp();
      if (left > 32)
        pair_load_residual(ah, w.lane, (p >= 1 ? ah.r[1] : ah.r[0]) + (p == 1 ? 0 : 32), left - 32,
                           ah.res);
    }
    tmem_ld_wait();
    reg_fence<32>(v);
    float f[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
    // blocks of eight columns behind the last one keep what they have; they are not stored
    if (ah.bias) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float t[8];
        unpack8<kBF16>(ldg16(ah.bias, min(p * 32 + q * 8, ah.cols - 8)), t);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[q * 8 + i] += t[i];
      }
    }
    if (kAct != 0) activate<kAct>(f);
    if (ah.gate) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float t[8];
        unpack8<kBF16>(ldg16(ah.gate, min(p * 32 + q * 8, ah.cols - 8)), t);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[q * 8 + i] *= t[i];
      }
    }
    if (ah.with_res) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float t[8];
        unpack8<kBF16>(ld_shared_v4(stage64(w.buf, w.lane, q)), t);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[q * 8 + i] += t[i];
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      st_shared_v4(stage64(w.buf, w.lane, q), pack16<kBF16>(f[q * 8], f[q * 8 + 1]),
                   pack16<kBF16>(f[q * 8 + 2], f[q * 8 + 3]),
                   pack16<kBF16>(f[q * 8 + 4], f[q * 8 + 5]),
                   pack16<kBF16>(f[q * 8 + 6], f[q * 8 + 7]));
    if (p == 3 || left <= 32) pair_release(w);       // the last columns are in registers
    else __syncwarp();
    uint16_t* dst = ((p & 2) ? ah.y[1] : ah.y[0]) + (p & 1) * 32;
    const long long stride = (p & 2) ? ah.y_n[1] : ah.y_n[0];
    const int row = w.lane >> 2;
    const bool ok = (w.lane & 3) * 8 < left;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 o = ld_shared_v4(stage64(w.buf, row + i * 8, w.lane & 3));
      if (ok && row + i * 8 < ah.rows)
        *reinterpret_cast<uint4*>(dst + (long long)(i * 8) * stride) = o;
    }
    __syncwarp();
  }
}

// The same for the projection's epilogue.
struct PairHeadsAhead {
  const uint16_t *q_weight, *k_weight;   // nullptr: 1
  const uint16_t* bias;      // at the warp's first column
  const float* table;        // this lane's 16 bytes of the warp's first row (nullptr: no rotation)
  long long weight_h;
  int cols, rows, D, rot, halves, norm;
  float eps, inv_d;
  uint4 cs[8];               // the next piece of the table
};

// 16 (cos, sin) pairs, number 16 * piece on, of the warp's rows: 8 lanes a row, 4 rows a load.
__device__ __forceinline__ void pair_load_table(const PairHeadsAhead& ah, int lane, int piece,
                                                uint4 (&cs)[8]) {
  const bool f_ok = piece * 32 + (lane & 7) * 4 < ah.rot;
  const float* p = ah.table + piece * 32;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    cs[i] = make_uint4(0u, 0u, 0u, 0u);
    if (f_ok && (lane >> 3) + i * 4 < ah.rows)
      cs[i] = __ldg(reinterpret_cast<const uint4*>(p + i * 4 * ah.rot));
  }
}

__device__ __forceinline__ void pair_heads_ahead(const LinearArgs& a, const HeadArgs& head,
                                                 const PairWarp& w, PairHeadsAhead& ah) {
  ah.q_weight = static_cast<const uint16_t*>(head.weight[0]);
  ah.k_weight = static_cast<const uint16_t*>(head.weight[1]);
  ah.weight_h = head.weight_h;
  ah.bias = a.bias ? static_cast<const uint16_t*>(a.bias) + w.c0 : nullptr;
  ah.cols = min(128, w.c_end - w.c0);
  ah.rows = min(32, a.N - w.r0);
  ah.D = head.D;
  ah.rot = head.rot;
  ah.halves = head.halves;
  ah.norm = head.norm;
  ah.eps = head.eps;
  ah.inv_d = head.inv_d;
  ah.table = nullptr;
  if (head.table) {
    ah.table = head.table + w.b * head.table_b +
               (long long)(w.r0 + (w.lane >> 3)) * head.rot + (w.lane & 7) * 4;
    pair_load_table(ah, w.lane, 0, ah.cs);
  }
}

// Bias and norm weight of 8 columns of a head, loaded before the accumulators are waited for.
struct PairParams8 {
  uint4 bias, weight;
};
__device__ __forceinline__ PairParams8 pair_params8(const uint16_t* bias, const uint16_t* weight,
                                                    int d) {
  PairParams8 p;
  p.bias = bias ? ldg16(bias, d) : make_uint4(0u, 0u, 0u, 0u);
  p.weight = weight ? ldg16(weight, d) : make_uint4(0u, 0u, 0u, 0u);
  return p;
}

// 8 accumulators: bias, norm (r: its factor) and weight.
template <bool kBF16>
__device__ __forceinline__ void pair_finish8(const uint32_t* v, const PairParams8& p, bool bias,
                                             bool weight, float r, float* f) {
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(v[j]);
  if (bias) {
    float t[8];
    unpack8<kBF16>(p.bias, t);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] += t[j];
  }
  if (weight) {
    float t[8];
    unpack8<kBF16>(p.weight, t);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= r * t[j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= r;
  }
}

template <bool kBF16>
__device__ __forceinline__ void pair_stage8(uint32_t addr, const float* f) {
  st_shared_v4(addr, pack16<kBF16>(f[0], f[1]), pack16<kBF16>(f[2], f[3]),
               pack16<kBF16>(f[4], f[5]), pack16<kBF16>(f[6], f[7]));
}

// Bias, norm and rotation of the heads in the warp's 128 columns.
template <bool kBF16>
__device__ __forceinline__ void pair_heads(const LinearArgs& a, const PairWarp& w,
                                           PairHeadsAhead& ah) {
  const int D = ah.D;
  const int half = ah.rot / 2;
#pragma unroll 1
  for (int hd = 0; hd < 128; hd += D) {
    if (hd >= ah.cols) break;
    const int c_h = w.c0 + hd;                         // the head's first column
    const int part = c_h < a.part_cols ? 0 : c_h / a.part_cols;
    const int pc_h = c_h - part * a.part_cols;
    const bool turn = part < 2 && ah.table != nullptr;
    const bool normed = part < 2 && ah.norm;
    const uint16_t* bias = ah.bias ? ah.bias + hd : nullptr;
    const int h = part < 2 && ah.weight_h ? pc_h / D : 0;
    const uint16_t* weight = !normed ? nullptr : (part == 0 ? ah.q_weight : ah.k_weight);
    if (weight) weight += h * ah.weight_h;
    const uint32_t acc = w.acc + hd;
    const RowView& y = a.y[part];                      // a head's columns lie in one row of y
    uint16_t* out = static_cast<uint16_t*>(const_cast<void*>(y.ptr)) +
                    row_offset(y, w.b, w.r0 + (w.lane >> 2), pc_h);
    const long long out_n = y.n;

    float r = 1.f;
    if (normed) {
      float ss[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int d = 0; d < D; d += 32) {
        uint32_t v[32];
        tmem_ld32(acc + d, v);
        tmem_ld_wait();
        reg_fence<32>(v);
        if (bias) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float t[8];
            unpack8<kBF16>(ldg16(bias, d + q * 8), t);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              v[q * 8 + i] = __float_as_uint(__uint_as_float(v[q * 8 + i]) + t[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float x = __uint_as_float(v[i]);
          ss[i & 3] = fmaf(x, x, ss[i & 3]);
        }
      }
      r = __frsqrt_rn(fmaf((ss[0] + ss[1]) + (ss[2] + ss[3]), ah.inv_d, ah.eps));
    }

    // Pieces of four blocks of eight columns.  Half-split pairs: two low blocks and their
    // partners in the high half, 16 pairs (then the columns behind R, 32 a piece); otherwise 32
    // neighbouring columns.  Piece i turns by the pairs from 16 i, which lie in the staging
    // buffer, 128 bytes a row; a thread overwrites the part of its own row that it has read with
    // its output, block b at chunk 2b (pairs: low blocks at 0 and 4, high ones at 2 and 6).
    const bool split = turn && ah.halves;
    const int turning = turn ? (ah.rot + 31) / 32 : 0;
    const int pieces = split ? turning + (D - ah.rot + 31) / 32 : D / 32;
#pragma unroll 1
    for (int i = 0; i < pieces; ++i) {
      const bool pairs = split && i < turning;
      const bool turned = turn && i < turning;
      const int first = pairs ? 16 * i : (split ? ah.rot + 32 * (i - turning) : 32 * i);
      const int last = pairs ? half : D;               // blocks from here on do not exist
      if (turned) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          st_shared_v4(stage128(w.buf, j * 4 + (w.lane >> 3), w.lane & 7), ah.cs[j].x, ah.cs[j].y,
                       ah.cs[j].z, ah.cs[j].w);
        __syncwarp();
        // the next piece's pairs: this head's, or the next head's first
        pair_load_table(ah, w.lane, i + 1 < turning ? i + 1 : 0, ah.cs);
      }
      if (pairs) {
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {
          const int d = first + q * 8;
          if (d >= last) break;
          uint32_t v[16];
          tmem_ld8(acc + d, v);
          tmem_ld8(acc + d + half, v + 8);
          const PairParams8 lo = pair_params8(bias, weight, d);
          const PairParams8 hi = pair_params8(bias, weight, d + half);
          float t[16];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 c4 = ld_shared_v4(stage128(w.buf, w.lane, 4 * q + j));
            t[4 * j] = __uint_as_float(c4.x);
            t[4 * j + 1] = __uint_as_float(c4.y);
            t[4 * j + 2] = __uint_as_float(c4.z);
            t[4 * j + 3] = __uint_as_float(c4.w);
          }
          tmem_ld_wait();
          reg_fence<16>(v);
          float f[16];
          pair_finish8<kBF16>(v, lo, bias != nullptr, weight != nullptr, r, f);
          pair_finish8<kBF16>(v + 8, hi, bias != nullptr, weight != nullptr, r, f + 8);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float x = f[j], z = f[j + 8], c = t[2 * j], s = t[2 * j + 1];
            f[j] = fmaf(x, c, -z * s);
            f[j + 8] = fmaf(x, s, z * c);
          }
          pair_stage8<kBF16>(stage128(w.buf, w.lane, 4 * q), f);
          pair_stage8<kBF16>(stage128(w.buf, w.lane, 4 * q + 2), f + 8);
        }
      } else {
#pragma unroll 1
        for (int q = 0; q < 4; q += 2) {
          const int d = first + q * 8;
          if (d >= last) break;
          const bool two = d + 8 < last;                 // only behind R can a block be alone
          uint32_t v[16];
          tmem_ld8(acc + d, v);
          tmem_ld8(acc + (two ? d + 8 : d), v + 8);
          const PairParams8 lo = pair_params8(bias, weight, d);
          const PairParams8 hi = pair_params8(bias, weight, two ? d + 8 : d);
          float t[16];
          if (turned) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint4 c4 = ld_shared_v4(stage128(w.buf, w.lane, 2 * q + j));
              t[4 * j] = __uint_as_float(c4.x);
              t[4 * j + 1] = __uint_as_float(c4.y);
              t[4 * j + 2] = __uint_as_float(c4.z);
              t[4 * j + 3] = __uint_as_float(c4.w);
            }
          }
          tmem_ld_wait();
          reg_fence<16>(v);
          float f[16];
          pair_finish8<kBF16>(v, lo, bias != nullptr, weight != nullptr, r, f);
          pair_finish8<kBF16>(v + 8, hi, bias != nullptr, weight != nullptr, r, f + 8);
          if (turned) {
            // R is a multiple of 8: a block turns as a whole or not at all
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if (d + (j & 4 ? 8 : 0) >= ah.rot) break;
              const float x = f[2 * j], z = f[2 * j + 1], c = t[2 * j], s = t[2 * j + 1];
              f[2 * j] = fmaf(x, c, -z * s);
              f[2 * j + 1] = fmaf(x, s, z * c);
            }
          }
          pair_stage8<kBF16>(stage128(w.buf, w.lane, 2 * q), f);
          pair_stage8<kBF16>(stage128(w.buf, w.lane, 2 * q + 2), f + 8);
        }
      }
      __syncwarp();
      // 4 lanes a row, one block each
      const int q = w.lane & 3;
      const int d = pairs ? first + (q & 1) * 8 + (q >> 1) * half : first + q * 8;
      const bool ok = (pairs ? first + (q & 1) * 8 : d) < last;
      const int chunk = pairs ? (q & 1) * 4 + (q >> 1) * 2 : 2 * q;
      const int row = w.lane >> 2;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 o = ld_shared_v4(stage128(w.buf, row + j * 8, chunk));
        if (ok && row + j * 8 < ah.rows)
          *reinterpret_cast<uint4*>(out + d + (long long)(j * 8) * out_n) = o;
      }
      __syncwarp();
    }
  }
}

// kEpi: an activation (numbering of tara_act), or kEpiHeads for the projection.
constexpr int kEpiHeads = 4;

template <bool kBF16, int BN, int kSubs, int kEpi>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairLinThreads, 1)
linear_pair_kernel(const __grid_constant__ PairLinMaps maps,
                   const __grid_constant__ PairLinArgs args) {
  using S = PairLin<BN, kSubs>;
  constexpr int NS = S::kStages;
  constexpr bool kQkv = kEpi == kEpiHeads;
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
    c0 = (r / rows) * args.bn;
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

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kPairLinControlRegs) : "memory");
    if (warp == 0 && lane == 0) {
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
        const int wrow = c0 + (int)rank * (args.bn / 2);
        // a second sub-tile wholly behind the last row is neither loaded nor multiplied
        const int subs = kSubs == 2 && m0 + 256 < a.N ? 2 : 1;
        const uint32_t bytes = 2u * (uint32_t)(subs * 16384 + args.bn * 64);
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
    } else if (warp == 1 && lane == 0 && leader) {
      // ------------------------------ MMA issuer (even CTA) ----------------------------
      const uint32_t idesc = make_idesc_f16(256, args.bn, kBF16, false);
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
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kPairLinEpilogueRegs) : "memory");
    // ------------------------------ epilogue warps (both CTAs) -------------------------
    const int wq = warp & 3;                 // TMEM lane quarter
    const int grp = (warp - 4) >> 2;         // warpgroup: column half (256) or tile parity (128)
    const int ew = warp - 4;
    const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
    PairWarp w;
    w.buf = smem_u32(s_out + ew * 4096);
    const uint32_t acc_empty_l = mapa_shared(smem_u32(acc_empty), 0);
    w.lane = lane;
    bool ok = true;
    uint32_t unit = 0;
    for (int t = first; ok && t < n_tiles_total; t += n_clusters) {
      int m0;
      decode(t, w.b, m0, w.c0);
      w.c_end = min(a.C, w.c0 + args.bn);
      if (BN == 256) w.c0 += grp * 128;
#pragma unroll 1
      for (int u = 0; u < kSubs; ++u, ++unit) {
        const uint32_t half = unit & 1u;
        if (BN == 128 && half != (uint32_t)grp) continue;
        w.r0 = m0 + u * 256 + (int)rank * 128 + wq * 32;
        w.acc = tmem + lane_base + half * BN + (BN == 256 ? grp * 128 : 0);
        const bool live = w.r0 < a.N && w.c0 < w.c_end;
        w.release = acc_empty_l + half * 8u;
        // the first piece of what comes from memory, in flight while the products run
        typename std::conditional<kQkv, PairHeadsAhead, PairLinearAhead>::type ahead;
        if (live) {
          if constexpr (kQkv)
            pair_heads_ahead(a, args.head, w, ahead);
          else
            pair_linear_ahead(a, w, ahead);
        }
        if (!(ok = mbar_wait_warp(&acc_full[half], (unit >> 1) & 1u, abort_flag))) break;
        tc_fence_after();
        if constexpr (kQkv) {
          if (live) pair_heads<kBF16>(a, w, ahead);
          pair_release(w);
        } else if (live) {
          pair_linear<kBF16, kQkv ? 0 : kEpi>(w, ahead);   // releases the accumulator
        } else {
          pair_release(w);
        }
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
    mbar_wait(exit_bar, 0, &no_abort, kLinExitNs);
    if (*abort_flag) atomicExch(a.status, 1);
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, S::kTmemCols);
  }
}

}  // namespace tara
