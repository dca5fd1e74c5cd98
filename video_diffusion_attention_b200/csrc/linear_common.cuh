// linear_common.cuh -- arguments and epilogue arithmetic shared by the linear-layer kernels:
//   y = residual + gate * act(x W^T + bias)
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace tara {

// A strided [B][H][N][D] view whose rows are indexed by column c = h * D + d.
struct RowView {
  const void* ptr;
  long long b, h, n;    // strides, elements
  int D;
};

__device__ __forceinline__ long long row_offset(const RowView& v, int b, long long n, int col) {
  const int h = col < v.D ? 0 : col / v.D;   // token-major rows need no division
  return b * v.b + h * v.h + n * v.n + (col - h * v.D);
}

struct LinearArgs {
  RowView x, residual;      // residual.ptr == nullptr: none
  RowView y[3];             // y[col / part_cols], column col % part_cols
  int part_cols;            // C for one output; H*D for q, k, v
  const void *w, *bias, *gate;
  long long gate_b;         // elements between branches' gates
  int act;
  int B, N, K, C;           // N tokens a branch, K input columns, C output columns
  int* status;
};

// v/2 (1 + erf(v / sqrt 2)) as v Phi(v), with Phi from erfc(x) = t exp(-x^2 + P(t)),
// t = 1 / (1 + x/2), x = |v| / sqrt 2: the form of Numerical Recipes' erfcc, P a polynomial of
// degree 9 in t fitted to ln(erfc(x) exp(x^2) / t) on 0 <= x <= 10 by Lawson's iteration (largest
// error 4.5e-8), in log2 units here.  The tail keeps its relative accuracy, and a branch-free
// 16 operations replace a call of erff: with 1,024 input columns erff bounded the kernel.
__device__ __forceinline__ float gelu_erf(float v) {
  const float a = fabsf(v);
  const float t = __fdividef(1.0f, fmaf(a, 0.35355339059f, 1.0f));
  float p = 0.20514240860939026f;
  p = fmaf(p, t, -0.96092289686203f);
  p = fmaf(p, t, 1.6192750930786133f);
  p = fmaf(p, t, -0.9395431876182556f);
  p = fmaf(p, t, -0.1684969663619995f);
  p = fmaf(p, t, 0.02914106659591198f);
  p = fmaf(p, t, 0.040909137576818466f);
  p = fmaf(p, t, 0.5596213340759277f);
  p = fmaf(p, t, 1.440520167350769f);
  p = fmaf(p, t, -1.8256460428237915f);
  const float half_erfc = 0.5f * t * exp2f(fmaf(-0.72134752044448170f * v, v, p));
  return v * (v < 0.0f ? half_erfc : 1.0f - half_erfc);
}

// Activations on the fp32 accumulator (numbering of tara_act).
template <int kAct>
__device__ __forceinline__ float activate(float v) {
  if (kAct == 1) return gelu_erf(v);
  if (kAct == 2) {
    // v/2 (1 + tanh u) = v / (1 + exp(-2u))
    const float u = 0.79788456080286536f * (v + 0.044715f * v * v * v);
    return __fdividef(v, 1.0f + __expf(-2.0f * u));
  }
  if (kAct == 3) return __fdividef(v, 1.0f + __expf(-v));
  return v;
}
// In place on a thread's values; the branch on the activation is taken once.
template <int kN>
__device__ __forceinline__ void activate_all(float (&f)[kN], int act) {
  if (act == 0) return;
  if (act == 1) {
#pragma unroll
    for (int i = 0; i < kN; ++i) f[i] = activate<1>(f[i]);
  } else if (act == 2) {
#pragma unroll
    for (int i = 0; i < kN; ++i) f[i] = activate<2>(f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) f[i] = activate<3>(f[i]);
  }
}

}  // namespace tara
