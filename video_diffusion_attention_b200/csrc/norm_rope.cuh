// norm_rope.cuh -- rotary tables over several axes, and the per-head norm of Q and K with the
// rotation in the same pass.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sm100_ptx.cuh"

namespace tara {

// ---------------------------------------------------------------------------------------
// 8 elements of one row, as fp32: consecutive, or two groups of 4
// ---------------------------------------------------------------------------------------
template <typename T>
struct Vec8;

template <>
struct Vec8<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    v = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void load(const __nv_bfloat16* p, const __nv_bfloat16* q) {
    const uint2 a = *reinterpret_cast<const uint2*>(p), b = *reinterpret_cast<const uint2*>(q);
    v = make_uint4(a.x, a.y, b.x, b.y);
  }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) = pack(f);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, __nv_bfloat16* q, const float (&f)[8]) {
    const uint4 v = pack(f);
    *reinterpret_cast<uint2*>(p) = make_uint2(v.x, v.y);
    *reinterpret_cast<uint2*>(q) = make_uint2(v.z, v.w);
  }
};

template <>
struct Vec8<__half> {
  uint4 v;
  __device__ __forceinline__ void load(const __half* p) {
    v = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void load(const __half* p, const __half* q) {
    const uint2 a = *reinterpret_cast<const uint2*>(p), b = *reinterpret_cast<const uint2*>(q);
    v = make_uint4(a.x, a.y, b.x, b.y);
  }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ void store(__half* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) = pack(f);
  }
  static __device__ __forceinline__ void store(__half* p, __half* q, const float (&f)[8]) {
    const uint4 v = pack(f);
    *reinterpret_cast<uint2*>(p) = make_uint2(v.x, v.y);
    *reinterpret_cast<uint2*>(q) = make_uint2(v.z, v.w);
  }
};

template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) { load(p, p + 4); }
  __device__ __forceinline__ void load(const float* p, const float* q) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(q);
  }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&f)[8]) {
    store(p, p + 4, f);
  }
  static __device__ __forceinline__ void store(float* p, float* q, const float (&f)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(q) = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// ---------------------------------------------------------------------------------------
// rope_table_kernel
// ---------------------------------------------------------------------------------------
constexpr int kRopeMaxPairs = 128;
constexpr int kRopeThreads = 256;

// Per pair: its axis and its frequency in quarter turns per unit of position
// (theta^(-2i/d) * 2/pi), both computed by the host in double precision.
struct RopeFreqs {
  double quarter_turns[kRopeMaxPairs];
  uint8_t axis[kRopeMaxPairs];
  int n_pairs, n_axes;
};

// Angle p * f quarter turns -> the nearest whole number of quarter turns (its low bits) and the
// remainder in radians, |remainder| <= pi/4.  Adding 1.5 * 2^52 rounds to a whole number whose
// low bits are those of the sum; the fma forms the remainder without a second rounding of the
// product, so the phase of far positions survives (|p * f| < 2^31).
__device__ __forceinline__ float quarter_turn_remainder(double p, double f, int& quarter) {
  const double magic = 6755399441055744.0;
  const double m = fma(p, f, magic);
  quarter = __double2loint(m);
  return (float)(fma(p, f, -(m - magic)) * 1.5707963267948966);
}

// sin and cos of two angles |x| <= pi/4 by their Taylor series to x^9 and x^10 (the first terms
// left out are below 2e-9 and 2e-10), two lanes at once in packed fp32.  The angle is rounded to
// fp32 by a choice: carrying its low part through both series would add to what the kernel is
// bound by, its instructions, for a largest error of 3e-8 instead of the 7.2e-8 measured (root mean
// square 1.6e-8; correct rounding has 1.4e-8).
__device__ __forceinline__ void sin_cos_small2(float x0, float x1, float2 (&sc)[2]) {
  auto both = [](float c) { return f32x2_pack(c, c); };
  const uint64_t x = f32x2_pack(x0, x1);
  const uint64_t zero = both(0.f);
  const uint64_t y = f32x2_fma(x, x, zero);
  uint64_t s = f32x2_fma(y, both(1.f / 362880.f), both(-1.f / 5040.f));
  s = f32x2_fma(y, s, both(1.f / 120.f));
  s = f32x2_fma(y, s, both(-1.f / 6.f));
  s = f32x2_fma(f32x2_fma(x, y, zero), s, x);
  uint64_t c = f32x2_fma(y, both(-1.f / 3628800.f), both(1.f / 40320.f));
  c = f32x2_fma(y, c, both(-1.f / 720.f));
  c = f32x2_fma(y, c, both(1.f / 24.f));
  c = f32x2_fma(y, c, both(-0.5f));
  c = f32x2_fma(y, c, both(1.f));
  f32x2_unpack(s, sc[0].x, sc[1].x);
  f32x2_unpack(c, sc[0].y, sc[1].y);
}

// (cos, sin) of an angle from its whole quarter turns and (sin, cos) of its remainder.
__device__ __forceinline__ float2 turn_quarters(float2 sc, int q) {
  const float a = (q & 1) ? sc.x : sc.y, b = (q & 1) ? sc.y : sc.x;
  const uint32_t flip_cos = (uint32_t)(q + 1) << 30 & 0x80000000u;    // quarters 1 and 2
  const uint32_t flip_sin = (uint32_t)q << 30 & 0x80000000u;          // quarters 2 and 3
  return make_float2(__uint_as_float(__float_as_uint(a) ^ flip_cos),
                     __uint_as_float(__float_as_uint(b) ^ flip_sin));
}

// Bound by instruction issue (about 73 warp instructions for two pairs; issue 61% busy at 107,126
// x 64 pairs, where the table, 8 bytes a pair, still fits L2).  A thread keeps two neighbouring
// pairs (one 16-byte store) and
// walks rows with the stride of the grid, the next kRopeBatch positions in flight, so that pair
// index, axis and frequency are set up once.  The frequencies pass through shared memory: read
// by thread index from the kernel's arguments they are fetched one address at a time, which with
// 8 rows a thread took half of the time.
constexpr int kRopeBatch = 4;
constexpr int kRopeCtas = 5;      // CTAs that run together on an SM

__global__ void __launch_bounds__(kRopeThreads, kRopeCtas)
rope_table_kernel(const float* __restrict__ pos, long long n_rows,
                  const __grid_constant__ RopeFreqs fr, float4* __restrict__ table) {
  __shared__ double s_freq[kRopeMaxPairs];
  __shared__ uint8_t s_axis[kRopeMaxPairs];
  for (int i = threadIdx.x; i < fr.n_pairs; i += kRopeThreads) {
    s_freq[i] = fr.quarter_turns[i];
    s_axis[i] = fr.axis[i];
  }
  __syncthreads();
  const int row_units = fr.n_pairs / 2;                   // 16-byte units of a row
  const int rows_step = kRopeThreads / row_units;         // rows of one step of a CTA
  const int r = threadIdx.x / row_units, u = threadIdx.x - r * row_units;
  if (r >= rows_step) return;
  const double f0 = s_freq[2 * u], f1 = s_freq[2 * u + 1];
  const long long stride = (long long)gridDim.x * rows_step;
  const long long row0 = (long long)blockIdx.x * rows_step + r;
  // pointers and a count of the rows ahead instead of 64-bit row numbers in the loop
  const long long pos_step = stride * fr.n_axes, out_step = stride * row_units;
  const float* p0 = pos + row0 * fr.n_axes + s_axis[2 * u];
  const int to1 = (int)s_axis[2 * u + 1] - (int)s_axis[2 * u];
  float4* out = table + row0 * row_units + u;
  long long left = row0 < n_rows ? (n_rows - row0 + stride - 1) / stride : 0;
  float x[kRopeBatch], y[kRopeBatch];
  auto fetch = [&](long long rows) {
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) {
      if (i < rows) {
        x[i] = __ldg(p0);
        y[i] = __ldg(p0 + to1);
      }
      p0 += pos_step;
    }
  };
  fetch(left);
  for (; left > 0; left -= kRopeBatch) {
    float nx[kRopeBatch], ny[kRopeBatch];
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) {
      nx[i] = x[i];
      ny[i] = y[i];
    }
    fetch(left - kRopeBatch);
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) {
      if (i >= left) break;
      int q0, q1;
      const float a0 = quarter_turn_remainder((double)nx[i], f0, q0);
      const float a1 = quarter_turn_remainder((double)ny[i], f1, q1);
      float2 sc[2];
      sin_cos_small2(a0, a1, sc);
      const float2 t0 = turn_quarters(sc[0], q0), t1 = turn_quarters(sc[1], q1);
      *out = make_float4(t0.x, t0.y, t1.x, t1.y);
      out += out_step;
    }
  }
}

// ---------------------------------------------------------------------------------------
// norm_rope_kernel: a row of one head lies across LANES lanes, 8 elements a lane
// ---------------------------------------------------------------------------------------
// HBM-bound: every element of q and k is read and written once, ~10 operations each (56 heads x
// 107,126 x 128 bf16: 960 to 990 us, 6.3 to 6.46 TB/s of a copy's 6.56; walking pointers and packed
// fp32 took the last 4% off).  A warp
// keeps 32/LANES tokens and walks heads, so a token's (cos, sin) pairs are read once for all
// the heads of a CTA and stay in registers, and kBatch heads' loads are in flight per lane.
//
// Which 8 columns a lane holds: with interleaved pairs 8 consecutive ones.  With half-split
// pairs lane l < R/8 holds [4l, 4l + 4) and [R/2 + 4l, R/2 + 4l + 4), so that both columns of a
// pair are in one lane and no exchange between lanes is needed (two 8-byte accesses instead of
// one of 16 bytes; exchanging the halves by shuffles measured 1,189 us where this took 1,076);
// the lanes behind hold the columns that do not turn, 8 consecutive ones each.
struct NormRopeTensor {
  const void* in;
  void* out;
  const void* weight;
  long long in_b, in_h, in_n, out_b, out_h, out_n;   // strides, elements
};

struct NormRopeArgs {
  NormRopeTensor t[2];     // q, k
  const float* table;
  long long table_b;       // floats between branches' tables
  long long weight_h;      // elements between heads' weights (0: shared)
  int H, N, D, rot;
  int norm;
  float eps, inv_d;
  int heads_per_cta, chunks;   // blockIdx.y = tensor * chunks + chunk of heads_per_cta heads
};

constexpr int kNormRopeThreads = 256;

__device__ __forceinline__ uint64_t both2(float c) { return f32x2_pack(c, c); }

template <typename T, int LANES, bool kHalves>
__global__ void __launch_bounds__(kNormRopeThreads)
norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int kRows = 32 / LANES;                       // token rows per warp
  constexpr int kBatch = sizeof(T) == 2 ? 4 : 2;          // heads in flight
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane % LANES;
  const long long n =
      ((long long)blockIdx.x * (kNormRopeThreads / 32) + warp) * kRows + lane / LANES;
  const bool live = n < a.N && 8 * l < a.D;
  const int b = blockIdx.z;
  const bool turned = a.table != nullptr && 8 * l < a.rot;
  // columns [c0, c0 + 4) and [c1, c1 + 4); pairs [c0 / 2, ...) or [4l, ...)
  const int c0 = kHalves && turned ? 4 * l : 8 * l;
  const int c1 = kHalves && turned ? a.rot / 2 + 4 * l : 8 * l + 4;

  // the row's (cos, sin) pairs this lane needs, read once and used for every head
  float cs[8];
  if (live && turned) {
    const float4* src =
        reinterpret_cast<const float4*>(a.table + b * a.table_b + n * a.rot + 8 * l);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 v = src[i];
      cs[4 * i] = v.x; cs[4 * i + 1] = v.y; cs[4 * i + 2] = v.z; cs[4 * i + 3] = v.w;
    }
  }

  const int which = blockIdx.y / a.chunks;
  const NormRopeTensor& t = a.t[which];
  const int h0 = (blockIdx.y - which * a.chunks) * a.heads_per_cta;
  const int h1 = min(h0 + a.heads_per_cta, a.H);
  // strides and pointers in registers: the loop walks them from head to head
  const long long in_h = t.in_h, out_h = t.out_h, weight_h = a.weight_h;
  const T* in = static_cast<const T*>(t.in) + b * t.in_b + n * t.in_n + h0 * in_h;
  T* out = static_cast<T*>(t.out) + b * t.out_b + n * t.out_n + h0 * out_h;
  auto load8 = [&](Vec8<T>& v, const T* row) {
    if (kHalves)
      v.load(row + c0, row + c1);
    else
      v.load(row + c0);
  };
  const bool norm = a.norm;
  const T* weight = static_cast<const T*>(t.weight);
  const bool weighted = norm && weight != nullptr && live;
  // the weights as packed pairs; those of each head are loaded in the loop
  uint64_t w[4] = {both2(1.f), both2(1.f), both2(1.f), both2(1.f)};
  auto load_weight = [&](const T* p) {
    Vec8<T> wv;
    float f[8];
    load8(wv, p);
    wv.unpack(f);
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = f32x2_pack(f[2 * j], f[2 * j + 1]);
  };
  const bool per_head = weighted && weight_h != 0;
  if (weighted && !per_head) load_weight(weight);
  const float eps = a.eps, inv_d = a.inv_d;

  for (int left = h1 - h0, h = h0; left > 0; left -= kBatch, h += kBatch) {
    Vec8<T> v[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (live && i < left) load8(v[i], in);
      in += in_h;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (i >= left) break;                               // the same for the whole warp
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (live) v[i].unpack(x);
      if (norm) {
        uint64_t p[4], ss = 0;                            // (0, 0)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          p[j] = f32x2_pack(x[2 * j], x[2 * j + 1]);
          ss = f32x2_fma(p[j], p[j], ss);
        }
        float s0, s1;
        f32x2_unpack(ss, s0, s1);
        s0 += s1;
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) s0 += __shfl_xor_sync(0xffffffffu, s0, o);
        const float r = __frsqrt_rn(fmaf(s0, inv_d, eps));
        if (per_head) load_weight(weight + (h + i) * weight_h);
        const uint64_t rr = both2(r), zero = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          f32x2_unpack(f32x2_fma(p[j], f32x2_fma(rr, w[j], zero), zero), x[2 * j], x[2 * j + 1]);
      }
      if (turned) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // pair j: columns j of both groups, or neighbours
          float& p = x[kHalves ? j : 2 * j];
          float& q = x[kHalves ? j + 4 : 2 * j + 1];
          const float u = p, z = q, c = cs[2 * j], sn = cs[2 * j + 1];
          p = fmaf(u, c, -z * sn);
          q = fmaf(u, sn, z * c);
        }
      }
      if (live) {
        if (kHalves)
          Vec8<T>::store(out + c0, out + c1, x);
        else
          Vec8<T>::store(out + c0, x);
      }
      out += out_h;
    }
  }
}

}  // namespace tara
