// linear_simt.cuh -- the linear layer on CUDA cores, any strides and sizes.
//
// A CTA of 256 threads computes 64 rows x 64 columns, 4 x 4 per thread, walking K in steps of
// 16 through shared memory.
#pragma once

#include "linear_common.cuh"

namespace tara {

constexpr int kSimtLinThreads = 256;
constexpr int kSimtLinTile = 64;
constexpr int kSimtLinK = 16;

template <typename T>
__global__ void __launch_bounds__(kSimtLinThreads)
linear_simt_kernel(const __grid_constant__ LinearArgs a) {
  __shared__ float sx[kSimtLinK][kSimtLinTile + 4];
  __shared__ float sw[kSimtLinK][kSimtLinTile + 4];
  const int tid = threadIdx.x;
  const int b = blockIdx.z;
  const long long n0 = (long long)blockIdx.x * kSimtLinTile;
  const int c0 = blockIdx.y * kSimtLinTile;
  const int tr = (tid >> 4) * 4, tc = (tid & 15) * 4;
  float acc[4][4] = {};
  const T* x = static_cast<const T*>(a.x.ptr);
  const T* w = static_cast<const T*>(a.w);

  for (int k0 = 0; k0 < a.K; k0 += kSimtLinK) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = tid + i * kSimtLinThreads;
      const int r = e >> 4, kk = e & 15, k = k0 + kk;
      sx[kk][r] = (n0 + r < a.N && k < a.K) ? to_f32(x[row_offset(a.x, b, n0 + r, k)]) : 0.f;
      sw[kk][r] = (c0 + r < a.C && k < a.K) ? to_f32(w[(long long)(c0 + r) * a.K + k]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < kSimtLinK; ++kk) {
      const float4 xv = *reinterpret_cast<const float4*>(&sx[kk][tr]);
      const float4 wv = *reinterpret_cast<const float4*>(&sw[kk][tc]);
      const float xr[4] = {xv.x, xv.y, xv.z, xv.w}, wr[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xr[i], wr[j], acc[i][j]);
    }
    __syncthreads();
  }

#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long n = n0 + tr + i;
    if (n >= a.N) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + tc + j;
      if (c >= a.C) continue;
      float one[1] = {acc[i][j]};
      if (a.bias) one[0] += to_f32(static_cast<const T*>(a.bias)[c]);
      activate_all(one, a.act);
      float v = one[0];
      if (a.gate) v *= to_f32(static_cast<const T*>(a.gate)[b * a.gate_b + c]);
      if (a.residual.ptr)
        v += to_f32(static_cast<const T*>(a.residual.ptr)[row_offset(a.residual, b, n, c)]);
      const int part = c / a.part_cols;
      const RowView& y = a.y[part];
      static_cast<T*>(const_cast<void*>(y.ptr))[row_offset(y, b, n, c - part * a.part_cols)] =
          from_f32<T>(v);
    }
  }
}

}  // namespace tara
