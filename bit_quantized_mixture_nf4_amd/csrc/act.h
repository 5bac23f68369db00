// act.h -- the activations of the stored-weight product, in fp32, and its
// epilogue on VEC consecutive columns of one row.
#pragma once

#include "plan_block.h"
#include "rowvec.h"

namespace e4b {

// exp and the quotient keep fp32's accuracy: outputs may be fp32
__device__ __forceinline__ float sigmoid_f32(float z) { return 1.0f / (1.0f + expf(-z)); }

// GELU's two forms: z Phi(z), and the tanh form with u = sqrt(2/pi) (z + 0.044715 z^3),
// 0.5 (1 + tanh u) = sigmoid(2 u).
__device__ __forceinline__ float gelu_tanh_arg(float z) {
  return 1.5957691216057308f * (z + 0.044715f * z * z * z);  // 2 u
}

__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case E4B_ACT_RELU: return z > 0.0f ? z : 0.0f;
    case E4B_ACT_SILU: return z * sigmoid_f32(z);
    case E4B_ACT_GELU: return z * (0.5f * (1.0f + erff(z * 0.7071067811865476f)));
    case E4B_ACT_GELU_TANH: return z * sigmoid_f32(gelu_tanh_arg(z));
    default: return z;
  }
}

__device__ __forceinline__ float act_grad(int act, float z) {
  switch (act) {
    case E4B_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
    case E4B_ACT_SILU: {
      const float s = sigmoid_f32(z);
      return s * (1.0f + z * (1.0f - s));
    }
    case E4B_ACT_GELU:
      return 0.5f * (1.0f + erff(z * 0.7071067811865476f)) + z * expf(-0.5f * z * z) * 0.3989422804014327f;
    case E4B_ACT_GELU_TANH: {
      // d/dz z S(v) = S + z S (1 - S) v', v' = 2 sqrt(2/pi) (1 + 3 0.044715 z^2)
      const float s = sigmoid_f32(gelu_tanh_arg(z));
      return s + z * s * (1.0f - s) * 1.5957691216057308f * (1.0f + 0.134145f * z * z);
    }
    default: return 1.0f;
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
  if (g.act != E4B_ACT_NONE) {
#pragma unroll
    for (int q = 0; q < VEC; ++q) v[q] = act_value(g.act, v[q]);
  }
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
