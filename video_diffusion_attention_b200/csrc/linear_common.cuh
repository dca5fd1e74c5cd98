// linear_common.cuh -- arguments and epilogue arithmetic shared by the linear-layer kernels:
//   y = residual + gate * act(x W^T + bias)
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sm100_ptx.cuh"

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

// Activations on the fp32 accumulators (numbering of tara_act), two elements at a time in packed
// fp32.  What bounds them in the epilogue is the special-function unit, 16 results a cycle and SM:
// two reciprocals are taken as one, of the product (1.5 operations an element instead of 2; what
// goes into the product is bounded, so that it stays finite and an infinity or NaN stays in its
// own element), and the polynomial runs on packed FMAs.
__device__ __forceinline__ uint64_t both(float c) { return f32x2_pack(c, c); }
__device__ __forceinline__ uint64_t f32x2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (v0, v1) <- v 2^x / (1 + 2^x).  x is cut off above 60, where the factor is 1 to fp32, so that the
// product of two denominators stays finite; below, 2^x runs down to 0 and the result with it,
// however large |v| is.  (A NaN in x counts as 60: it stays in its own v.)
__device__ __forceinline__ void logistic_pair(float& v0, float& v1, uint64_t x) {
  float x0, x1, d0, d1;
  f32x2_unpack(x, x0, x1);
  const uint64_t e = f32x2_pack(ex2_approx(fminf(x0, 60.f)), ex2_approx(fminf(x1, 60.f)));
  f32x2_unpack(f32x2_add(e, both(1.f)), d0, d1);
  const uint64_t factor = f32x2_mul(f32x2_mul(e, f32x2_pack(d1, d0)), both(rcp_approx(d0 * d1)));
  f32x2_unpack(f32x2_mul(f32x2_pack(v0, v1), factor), v0, v1);
}

template <int kAct>
__device__ __forceinline__ void activate_pair(float& v0, float& v1) {
  const uint64_t v = f32x2_pack(v0, v1);
  if (kAct == 1) {
    // v/2 (1 + erf(v / sqrt 2)) = v Phi(v), with Phi from erfc(x) = t exp(-x^2 + P(t)),
    // t = 1 / (1 + x/2), x = |v| / sqrt 2: the form of Numerical Recipes' erfcc, P a polynomial
    // of degree 9 in t fitted to ln(erfc(x) exp(x^2) / t) on 0 <= x <= 10 by Lawson's iteration,
    // in log2 units here (largest error of the logarithm, coefficients as stored: 7.9e-8).  The
    // tail keeps its relative accuracy: in fp32 within 9e-6 down to v = -12.8.
    float d0, d1, e0, e1;
    f32x2_unpack(f32x2_fma(f32x2_pack(fminf(fabsf(v0), 64.f), fminf(fabsf(v1), 64.f)),
                           both(0.35355339059f), both(1.f)), d0, d1);
    const float r = rcp_approx(d0 * d1);
    const uint64_t t = f32x2_pack(r * d1, r * d0);
    uint64_t p = f32x2_fma(t, both(0.20514240860939026f), both(-0.96092289686203f));
    p = f32x2_fma(p, t, both(1.6192750930786133f));
    p = f32x2_fma(p, t, both(-0.9395431876182556f));
    p = f32x2_fma(p, t, both(-0.1684969663619995f));
    p = f32x2_fma(p, t, both(0.02914106659591198f));
    p = f32x2_fma(p, t, both(0.040909137576818466f));
    p = f32x2_fma(p, t, both(0.5596213340759277f));
    p = f32x2_fma(p, t, both(1.440520167350769f));
    p = f32x2_fma(p, t, both(-1.8256460428237915f));
    f32x2_unpack(f32x2_fma(f32x2_mul(v, v), both(-0.72134752044448170f), p), e0, e1);
    float h0, h1;                                  // erfc / 2
    f32x2_unpack(f32x2_mul(f32x2_mul(t, both(0.5f)), f32x2_pack(ex2_approx(e0), ex2_approx(e1))),
                 h0, h1);
    v0 *= v0 < 0.f ? h0 : 1.f - h0;
    v1 *= v1 < 0.f ? h1 : 1.f - h1;
  } else if (kAct == 2) {
    // v/2 (1 + tanh u) = v / (1 + exp(-2u)), u = sqrt(2/pi) (v + 0.044715 v^3)
    const uint64_t s = f32x2_fma(f32x2_mul(v, v), both(0.10294324f), both(2.30220819814f));
    logistic_pair(v0, v1, f32x2_mul(v, s));
  } else if (kAct == 3) {
    logistic_pair(v0, v1, f32x2_mul(v, both(1.44269504089f)));
  }
}

// In place on a thread's values.
template <int kAct, int kN>
__device__ __forceinline__ void activate(float (&f)[kN]) {
  static_assert(kN % 2 == 0, "pairs");
#pragma unroll
  for (int i = 0; i < kN; i += 2) activate_pair<kAct>(f[i], f[i + 1]);
}
template <int kN>
__device__ __forceinline__ void activate_any(float (&f)[kN], int act) {
  if (act == 1) activate<1>(f);
  else if (act == 2) activate<2>(f);
  else if (act == 3) activate<3>(f);
}

}  // namespace tara
