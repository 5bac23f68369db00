// act.h -- the activations of the stored-weight product, in fp32, and its
// epilogue on VEC consecutive columns of one row.
#pragma once

#include "plan_block.h"
#include "rowvec.h"

namespace e4b {

// 1 / (1 + e^-z) with the hardware's exp2 and reciprocal (about a step each).
// e^-z is off by |z| 2^-24 more, which z s (1 - s) <= 0.23 keeps below a step of s
// or, far below zero, below a step of anything added to it.
__device__ __forceinline__ float sigmoid_f32(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

// GELU's two forms: z Phi(z), and the tanh form with u = sqrt(2/pi) (z + 0.044715 z^3),
// 0.5 (1 + tanh u) = sigmoid(2 u).
__device__ __forceinline__ float gelu_tanh_arg(float z) {
  return 1.5957691216057308f * (z + 0.044715f * z * z * z);  // 2 u
}

// Phi(z) = 0.5 erfc(-z / sqrt 2). With x = |z| / sqrt 2, erfc(x) = e^-x^2 t P(t),
// t = 1 / (1 + 0.33 x): the form of Abramowitz and Stegun 7.1.26 with P of degree 7, fitted
// here to the least relative error of erfc(x) e^x^2 on 0 <= x <= 9.3 (8.2e-8; 4e-7 in
// fp32), beyond which e^-x^2 is below the smallest normal fp32. So the tail is
// right relative to itself (their degree 4 is right to 7.5e-8 of 1: 3 % off at z = -12.5).
// e^-x^2 gives the density too. The library's erff took 25 us of a 256 x 256 tile's
// epilogue; P's degree 7 takes no longer than degree 4 (2048 rows of nf4 2048 -> 4096 with
// GELU and a residual: 52.3 us, 52.9 with degree 4).
__device__ __forceinline__ float normal_cdf(float z, float &density) {
  const float x = fabsf(z) * 0.7071067811865476f;
  const float e = __expf(-x * x);
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.33f * x);
  float p = -0.135928765f;
  p = 0.462688088f + t * p;
  p = -0.355438709f + t * p;
  p = 0.41254139f + t * p;
  p = 0.0450107642f + t * p;
  p = 0.201923788f + t * p;
  p = 0.182837248f + t * p;
  p = 0.186366111f + t * p;
  const float tail = 0.5f * (t * p) * e;  // Phi(-|z|)
  density = e * 0.3989422804014327f;
  return z < 0.0f ? tail : 1.0f - tail;
}

// v = act(v), the branch outside the elements; a NaN stays one
template <int VEC>
__device__ __forceinline__ void act_values(int act, float (&v)[VEC]) {
  if (act == E4B_ACT_RELU) {
#pragma unroll
    for (int q = 0; q < VEC; ++q) v[q] = v[q] <= 0.0f ? 0.0f : v[q];
  } else if (act == E4B_ACT_SILU) {
#pragma unroll
    for (int q = 0; q < VEC; ++q) v[q] *= sigmoid_f32(v[q]);
  } else if (act == E4B_ACT_GELU) {
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
      float density;
      v[q] *= normal_cdf(v[q], density);
    }
  } else if (act == E4B_ACT_GELU_TANH) {
#pragma unroll
    for (int q = 0; q < VEC; ++q) v[q] *= sigmoid_f32(gelu_tanh_arg(v[q]));
  }
}

// v *= act'(z); a NaN of either stays one
template <int VEC>
__device__ __forceinline__ void act_grads(int act, const float (&z)[VEC], float (&v)[VEC]) {
  if (act == E4B_ACT_RELU) {
#pragma unroll
    for (int q = 0; q < VEC; ++q) v[q] *= z[q] > 0.0f ? 1.0f : z[q] <= 0.0f ? 0.0f : z[q];
  } else if (act == E4B_ACT_SILU) {
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
      const float s = sigmoid_f32(z[q]);
      v[q] *= s * (1.0f + z[q] * (1.0f - s));
    }
  } else if (act == E4B_ACT_GELU) {
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
      float density;
      const float cdf = normal_cdf(z[q], density);
      v[q] *= cdf + z[q] * density;
    }
  } else if (act == E4B_ACT_GELU_TANH) {
    // d/dz z S(w) = S + z S (1 - S) w', w' = 2 sqrt(2/pi) (1 + 3 0.044715 z^2), z^2 taken
    // into t = z S (1 - S), which is 0 before z^2 overflows (0 times infinity has no value)
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
      const float s = sigmoid_f32(gelu_tanh_arg(z[q]));
      const float t = z[q] * s * (1.0f - s);
      v[q] *= s + 1.5957691216057308f * (t + 0.134145f * (t * z[q] * z[q]));
    }
  }
}

// v: the product of VEC columns from element `at` of the [rows, out] outputs;
// b their bias. Writes the pre-activation (when kept) and y.
template <int VEC>
__device__ __forceinline__ void linear_epilogue(const LinearArgs &g, int64_t at, const float (&b)[VEC],
                                                float (&v)[VEC]) {
#pragma unroll
  for (int q = 0; q < VEC; ++q) v[q] += b[q];
  if (g.pre) store_row<VEC>(g.pre + at, v);
  if (!g.y) return;
  act_values<VEC>(g.act, v);
  if (g.residual) {
    float r[VEC];
    load_row<VEC>(reinterpret_cast<const bf16_t *>(g.residual) + at, r);
#pragma unroll
    for (int q = 0; q < VEC; ++q) v[q] += r[q];
  }
  if (g.y_f32)
    store_row<VEC>(static_cast<float *>(g.y) + at, v);
  else
    store_row<VEC>(static_cast<bf16_t *>(g.y) + at, v);
}

}  // namespace e4b
