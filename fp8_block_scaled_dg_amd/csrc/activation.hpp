// activation.hpp -- the activations of the GEMM epilogue and their derivatives, in fp32.
//
//   relu(x)      = max(x, 0)                      relu'(x) = x > 0
//   silu(x)      = x s(x), s(x) = 1 / (1 + e^-x)  silu'(x) = s (1 + x (1 - s))
//   gelu(x)      = x Phi(x), Phi the normal distribution function
//                                                 gelu'(x) = Phi(x) + x e^(-x^2/2) / sqrt(2 pi)
//   gelu_tanh(x) = x (1 + tanh u) / 2 = x s(2u), u = sqrt(2/pi) (x + 0.044715 x^3)
//                                                 x' = s + x s (1 - s) 2 u'
// Phi is formed as Phi(-z) = t P(t) e^(-z^2/2) for z = |x|, t = 1 / (1 + 0.2687 z): 2 t P(t)
// approximates e^(y^2) erfc(y), y = z / sqrt 2, with a polynomial of degree 8 fitted by
// reweighted least squares; its fp32 coefficients are within 4.9e-8 relative over y in [0, 12].
// Both tails of gelu then keep a relative accuracy of 7e-7 for |x| < 3 and 8.2e-6 for |x| < 13
// (the rounding of x^2 in the exponent), with exp2 and reciprocal rounded to nearest; the
// hardware's 1 ulp adds 1e-7 each. 1 + erf(x / sqrt 2) would cancel to a few bits at x = -5,
// which a block scaled by its own largest value would show. A NaN passes through all of them.
//
// The backward kernel is as much bound by this arithmetic as by memory, so powers are single
// v_exp_f32 on an argument scaled by log2 e (the library expf spends 12 more instructions on
// the last bit and on results below 2^-126, which become zero here).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/dg.h"

namespace dg {

constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + e^-x): the 1-ulp hardware reciprocal; 0 when e^-x overflows
__device__ __forceinline__ float act_sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

// e^(-z^2/2), z = |x|
__device__ __forceinline__ float act_bell(float z) {
  return __builtin_amdgcn_exp2f(-0.5f * kLog2e * z * z);
}

// t P(t) + add = Phi(-z) e^(z^2/2) + add, z = |x|
__device__ __forceinline__ float act_tail(float z, float add) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.26870056986808777f, z, 1.f));
  float p = 0.02952457405626774f;
  p = __builtin_fmaf(p, t, -0.1313483715057373f);
  p = __builtin_fmaf(p, t, 0.1823785901069641f);
  p = __builtin_fmaf(p, t, -0.08126617223024368f);
  p = __builtin_fmaf(p, t, 0.11540254950523376f);
  p = __builtin_fmaf(p, t, 0.06914930045604706f);
  p = __builtin_fmaf(p, t, 0.1020011231303215f);
  p = __builtin_fmaf(p, t, 0.1069524958729744f);
  p = __builtin_fmaf(p, t, 0.10720593482255936f);
  return __builtin_fmaf(p, t, add);
}

__device__ __forceinline__ float act_gelu_tanh_u(float x) {  // 2u
  return 1.5957691216057308f * __builtin_fmaf(0.044715f * x * x, x, x);
}

template <int N>
__device__ __forceinline__ void act_apply(float (&v)[N], int act) {
  if (act == DG_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = v[i] <= 0.f ? 0.f : v[i];
  } else if (act == DG_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= act_sigmoid(v[i]);
  } else if (act == DG_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float z = fabsf(v[i]), q = act_tail(z, 0.f) * act_bell(z);
      v[i] *= v[i] > 0.f ? 1.f - q : q;
    }
  } else if (act == DG_ACT_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= act_sigmoid(act_gelu_tanh_u(v[i]));
  }
}

// d[i] *= act'(x[i])
template <int N>
__device__ __forceinline__ void act_backward(float (&d)[N], const float (&x)[N], int act) {
  if (act == DG_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = x[i] <= 0.f ? 0.f : d[i];
  } else if (act == DG_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float s = act_sigmoid(x[i]);
      d[i] *= s * __builtin_fmaf(x[i], 1.f - s, 1.f);
    }
  } else if (act == DG_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      // x < 0: Phi(-z) - z phi(z); x > 0: 1 minus that
      const float z = fabsf(x[i]);
      const float s = act_tail(z, -0.3989422804014327f * z) * act_bell(z);
      d[i] *= x[i] > 0.f ? 1.f - s : s;
    }
  } else if (act == DG_ACT_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float s = act_sigmoid(act_gelu_tanh_u(x[i]));
      // t = x s (1 - s) before x^2: where x^2 overflows t is 0, and 0 times infinity is NaN
      const float t = x[i] * s * (1.f - s);
      const float du = __builtin_fmaf(0.134145f * x[i], t * x[i], t);
      d[i] *= __builtin_fmaf(1.5957691216057308f, du, s);
    }
  }
}

}  // namespace dg
