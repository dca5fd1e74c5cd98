// linear_simt.cuh -- the fp32 linear layer on CUDA cores, any strides and sizes: products and
// sums in fp32 (the tensor cores have no such type).
//
// linear_simt_kernel: a CTA of 256 threads computes kM x kM outputs, kM/16 x kM/16 a thread, and
// walks K in steps of kK through two shared-memory buffers; the next step's global loads are in
// flight while the current one is multiplied.  Bound by the FMA rate at kM = 128 (kK = 16), where
// a thread does 32 packed FMAs on four 16-byte shared loads; kM = 32 is for outputs that would
// otherwise leave SMs idle, bound by the latency of a step, hence kK = 64.
// linear_simt_rows_kernel: at most 8 rows.  Bound by reading W, so a warp takes kRowsCols rows of
// W, a lane every 32nd element, and the sums meet in a shuffle tree.
#pragma once

#include "linear_common.cuh"
#include "sm100_ptx.cuh"

namespace tara {

constexpr int kSimtLinThreads = 256;

// The activations once more for single fp32 results, by CUDA's own functions (erfc, not 1 + erf,
// which is 0 from v = -5.5 on, where v Phi(v) is -1e-7).
__device__ __forceinline__ float simt_activate(float v, int act) {
  if (act == 1) return 0.5f * v * erfcf(v * -0.70710678118654752f);
  if (act == 2) return v / (1.0f + expf(-1.5957691216f * (v + 0.044715f * v * v * v)));
  if (act == 3) return v / (1.0f + expf(-v));
  return v;
}

// act(acc + bias) * gate + residual -> y, one element.
__device__ __forceinline__ void simt_finish(const LinearArgs& a, int b, long long n, int c,
                                            float acc) {
  float v = acc;
  if (a.bias) v += static_cast<const float*>(a.bias)[c];
  v = simt_activate(v, a.act);
  if (a.gate) v *= static_cast<const float*>(a.gate)[b * a.gate_b + c];
  if (a.residual.ptr)
    v += static_cast<const float*>(a.residual.ptr)[row_offset(a.residual, b, n, c)];
  const int part = c < a.part_cols ? 0 : c / a.part_cols;
  const RowView& y = a.y[part];
  static_cast<float*>(const_cast<void*>(y.ptr))[row_offset(y, b, n, c - part * a.part_cols)] = v;
}

template <int kM, int kK>
__global__ void __launch_bounds__(kSimtLinThreads)
linear_simt_kernel(const __grid_constant__ LinearArgs a) {
  constexpr int kT = kM / 16;                      // outputs of a thread, each way
  constexpr int kRowStep = kSimtLinThreads / kK;   // loads: kK elements of a row, then the next row
  constexpr int kLoads = kM / kRowStep;
  constexpr int kPitch = kM + (kT < 4 ? 2 : 4);
  __shared__ __align__(16) float sx[2][kK][kPitch];
  __shared__ __align__(16) float sw[2][kK][kPitch];
  const int tid = threadIdx.x;
  const int b = blockIdx.z;
  const long long n0 = (long long)blockIdx.x * kM;
  const int c0 = blockIdx.y * kM;
  // a thread's outputs: groups of up to 4 neighbouring rows and columns, 64 apart
  constexpr int kG = kT < 4 ? kT : 4;
  const int ty = (tid >> 4) * kG, tx = (tid & 15) * kG;
  const float* x = static_cast<const float*>(a.x.ptr);
  const float* w = static_cast<const float*>(a.w);
  const int lr = tid / kK, lk = tid % kK;

  // row offsets of this thread's loads; the column of x moves through the heads with k
  int h = lk < a.x.D ? 0 : lk / a.x.D, d = lk - h * a.x.D, k = lk;
  float rx[kLoads], rw[kLoads];
  auto load = [&]() {
    const bool k_ok = k < a.K;
    const long long xk = b * a.x.b + h * a.x.h + d;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const long long n = n0 + lr + kRowStep * i;
      const int c = c0 + lr + kRowStep * i;
      rx[i] = k_ok && n < a.N ? x[xk + n * a.x.n] : 0.f;
      rw[i] = k_ok && c < a.C ? w[(long long)c * a.K + k] : 0.f;
    }
    k += kK;
    d += kK;
    while (d >= a.x.D && h * (long long)a.x.D < a.K) {
      d -= a.x.D;
      ++h;
    }
  };
  uint64_t acc[kT][kT / 2] = {};                   // packed column pairs
  load();
  int buf = 0;
  for (int k0 = 0; k0 < a.K; k0 += kK, buf ^= 1) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      sx[buf][lk][lr + kRowStep * i] = rx[i];
      sw[buf][lk][lr + kRowStep * i] = rw[i];
    }
    __syncthreads();                               // also: the other buffer's readers are done
    if (k0 + kK < a.K) load();
#pragma unroll
    for (int kk = 0; kk < kK; ++kk) {
      float xv[kT];
      uint64_t wv[kT / 2];
#pragma unroll
      for (int i = 0; i < kT; i += kG) {
        const float* px = &sx[buf][kk][ty + (i / kG) * 64];
        const float* pw = &sw[buf][kk][tx + (i / kG) * 64];
        if constexpr (kG == 4) {
          const float4 t = *reinterpret_cast<const float4*>(px);
          xv[i] = t.x; xv[i + 1] = t.y; xv[i + 2] = t.z; xv[i + 3] = t.w;
          const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(pw);
          wv[i / 2] = u.x; wv[i / 2 + 1] = u.y;
        } else {
          const float2 t = *reinterpret_cast<const float2*>(px);
          xv[i] = t.x; xv[i + 1] = t.y;
          wv[i / 2] = *reinterpret_cast<const uint64_t*>(pw);
        }
      }
#pragma unroll
      for (int i = 0; i < kT; ++i) {
        const uint64_t xx = f32x2_pack(xv[i], xv[i]);
#pragma unroll
        for (int j = 0; j < kT / 2; ++j) acc[i][j] = f32x2_fma(xx, wv[j], acc[i][j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kT; ++i) {
    const long long n = n0 + ty + (i / kG) * 64 + i % kG;
    if (n >= a.N) continue;
#pragma unroll
    for (int j = 0; j < kT; j += 2) {
      const int c = c0 + tx + (j / kG) * 64 + j % kG;
      float lo, hi;
      f32x2_unpack(acc[i][j / 2], lo, hi);
      if (c < a.C) simt_finish(a, b, n, c, lo);
      if (c + 1 < a.C) simt_finish(a, b, n, c + 1, hi);
    }
  }
}

constexpr int kSimtRows = 8;
constexpr int kRowsCols = 2;

// kRows: rows of a branch, rounded up to a power of two (the rows behind the last repeat it).
template <int kRows>
__global__ void __launch_bounds__(kSimtLinThreads)
linear_simt_rows_kernel(const __grid_constant__ LinearArgs a) {
  const int lane = threadIdx.x & 31;
  const int c0 = (int)(blockIdx.x * (kSimtLinThreads / 32) + (threadIdx.x >> 5)) * kRowsCols;
  const int b = blockIdx.y;
  if (c0 >= a.C) return;
  const float* x = static_cast<const float*>(a.x.ptr) + b * a.x.b;
  const float* w0 = static_cast<const float*>(a.w) + (long long)c0 * a.K;
  const float* w1 = c0 + 1 < a.C ? w0 + a.K : w0;
  float acc[kRows][kRowsCols] = {};
#pragma unroll 4
  for (int k = lane; k < a.K; k += 32) {
    const int h = k < a.x.D ? 0 : k / a.x.D;
    const float* xk = x + h * a.x.h + (k - h * a.x.D);
    const float u0 = w0[k], u1 = w1[k];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float xv = xk[min(i, a.N - 1) * a.x.n];
      acc[i][0] = fmaf(xv, u0, acc[i][0]);
      acc[i][1] = fmaf(xv, u1, acc[i][1]);
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i)
#pragma unroll
    for (int j = 0; j < kRowsCols; ++j)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[i][j] += __shfl_xor_sync(0xffffffffu, acc[i][j], o);
  // lane i * kRowsCols + j finishes output (i, j)
  float mine = 0.f;
#pragma unroll
  for (int i = 0; i < kRows; ++i)
#pragma unroll
    for (int j = 0; j < kRowsCols; ++j)
      if (lane == i * kRowsCols + j) mine = acc[i][j];
  const int i = lane / kRowsCols, c = c0 + lane % kRowsCols;
  if (i < a.N && i < kRows && c < a.C) simt_finish(a, b, i, c, mine);
}

}  // namespace tara
