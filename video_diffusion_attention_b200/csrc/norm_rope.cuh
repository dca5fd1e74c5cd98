// norm_rope.cuh -- rotary tables over several axes, and the per-head norm of Q and K with the
// rotation in the same pass.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace tara {

// ---------------------------------------------------------------------------------------
// 8 consecutive elements of one row, as fp32
// ---------------------------------------------------------------------------------------
template <typename T>
struct Vec8;

template <>
struct Vec8<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    v = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <>
struct Vec8<__half> {
  uint4 v;
  __device__ __forceinline__ void load(const __half* p) {
    v = *reinterpret_cast<const uint4*>(p);
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
  static __device__ __forceinline__ void store(__half* p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// ---------------------------------------------------------------------------------------
// rope_table_kernel: one thread per (row, pair)
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

// cos and sin of `turns` quarter turns.  The whole quarter turns come off in double precision,
// so the fp32 part sees at most an eighth of a turn either way and keeps an absolute error near
// 2^-26 however far the position is.
__device__ __forceinline__ float2 cos_sin_quarter_turns(double turns) {
  const double whole = rint(turns);
  float s, c;
  sincospif(0.5f * (float)(turns - whole), &s, &c);
  const int q = (int)((long long)whole & 3);
  const float a = (q & 1) ? s : c, b = (q & 1) ? c : s;
  return make_float2((q == 1 || q == 2) ? -a : a, (q >= 2) ? -b : b);
}

__global__ void __launch_bounds__(kRopeThreads)
rope_table_kernel(const float* __restrict__ pos, long long n_rows,
                  const __grid_constant__ RopeFreqs fr, float2* __restrict__ table) {
  const long long total = n_rows * fr.n_pairs;
  const long long i = (long long)blockIdx.x * kRopeThreads + threadIdx.x;
  if (i >= total) return;
  const long long row = i / fr.n_pairs;
  const int j = (int)(i - row * fr.n_pairs);
  const double p = (double)pos[row * fr.n_axes + fr.axis[j]];
  table[i] = cos_sin_quarter_turns(p * fr.quarter_turns[j]);
}

// ---------------------------------------------------------------------------------------
// norm_rope_kernel: a row of one head lies across LANES lanes, 8 elements a lane
// ---------------------------------------------------------------------------------------
// HBM-bound: every element of q and k is read and written once, ~10 operations each.  A warp
// keeps 32/LANES tokens and walks heads, so a token's (cos, sin) pairs are read once for all
// the heads of a CTA and stay in registers, and kBatch heads' loads are in flight per lane.
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
  const int half = a.rot / 16;                            // lanes of one half (kHalves)

  // the row's (cos, sin) pairs this lane needs, read once and used for every head
  float cs[kHalves ? 16 : 8];
  if (live && turned) {
    const int pair0 = kHalves ? 8 * (l < half ? l : l - half) : 4 * l;
    const float4* src = reinterpret_cast<const float4*>(a.table + b * a.table_b +
                                                        n * a.rot + 2 * pair0);
#pragma unroll
    for (int i = 0; i < (kHalves ? 4 : 2); ++i) {
      const float4 v = src[i];
      cs[4 * i] = v.x; cs[4 * i + 1] = v.y; cs[4 * i + 2] = v.z; cs[4 * i + 3] = v.w;
    }
  }
  // the other half of each pair lies rot/16 lanes away in the same row
  const int partner = (lane - l) + (l < half ? l + half : (l < 2 * half ? l - half : l));
  const float sign = l < half ? -1.f : 1.f;

  const int which = blockIdx.y / a.chunks;
  const NormRopeTensor& t = a.t[which];
  const int h0 = (blockIdx.y - which * a.chunks) * a.heads_per_cta;
  const int h1 = min(h0 + a.heads_per_cta, a.H);
  const T* in = static_cast<const T*>(t.in) + b * t.in_b + n * t.in_n + 8 * l;
  T* out = static_cast<T*>(t.out) + b * t.out_b + n * t.out_n + 8 * l;
  const T* weight = static_cast<const T*>(t.weight) + 8 * l;
  const bool weighted = a.norm && t.weight != nullptr && live;
  float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
  if (weighted) {
    Vec8<T> wv;
    wv.load(weight);
    wv.unpack(w);
  }

  for (int h = h0; h < h1; h += kBatch) {
    Vec8<T> v[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (live && h + i < h1) v[i].load(in + (h + i) * t.in_h);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (h + i >= h1) break;                             // the same for the whole warp
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (live) v[i].unpack(x);
      if (a.norm) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = __frsqrt_rn(fmaf(ss, a.inv_d, a.eps));
        if (a.weight_h != 0 && weighted) {
          Vec8<T> wv;
          wv.load(weight + (h + i) * a.weight_h);
          wv.unpack(w);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= r * w[j];
      }
      if (a.table != nullptr) {
        if (kHalves) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float y = __shfl_sync(0xffffffffu, x[j], partner);
            if (turned) x[j] = fmaf(x[j], cs[2 * j], sign * y * cs[2 * j + 1]);
          }
        } else if (turned) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float u = x[2 * j], z = x[2 * j + 1], c = cs[2 * j], sn = cs[2 * j + 1];
            x[2 * j] = fmaf(u, c, -z * sn);
            x[2 * j + 1] = fmaf(u, sn, z * c);
          }
        }
      }
      if (live) Vec8<T>::store(out + (h + i) * t.out_h, x);
    }
  }
}

}  // namespace tara
