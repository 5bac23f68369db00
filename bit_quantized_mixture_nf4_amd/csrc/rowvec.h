// rowvec.h -- row pieces of bf16 / fp32 tensors as fp32 registers: VEC
// consecutive elements per thread, one or two 16-byte accesses for VEC = 8
// (rows whose length is a multiple of 8 elements keep every piece 16-byte
// aligned), half of that for VEC = 4, single elements for VEC = 1 (any length).
#pragma once

#include "device.h"

namespace e4b {

struct bf16_t {
  uint16_t v;
};

// Streaming tensors are read once and written once; the plain accesses below
// let the second reader of a row (the gather's k copies, the norm weights)
// find it in L2.
template <int VEC>
__device__ __forceinline__ void load_row(const bf16_t *p, float (&f)[VEC]) {
  if constexpr (VEC == 8) {
    const u32x4 v = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f[2 * q] = bf16_lo(v[q]);
      f[2 * q + 1] = bf16_hi(v[q]);
    }
  } else if constexpr (VEC == 4) {
    const u32x2 v = *reinterpret_cast<const u32x2 *>(p);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      f[2 * q] = bf16_lo(v[q]);
      f[2 * q + 1] = bf16_hi(v[q]);
    }
  } else {
    static_assert(VEC == 1, "16- or 8-byte pieces or single elements");
    f[0] = bf16_to_f32(p->v);
  }
}

template <int VEC>
__device__ __forceinline__ void load_row(const float *p, float (&f)[VEC]) {
  if constexpr (VEC == 8) {
    const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 4);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f[q] = a[q];
      f[4 + q] = b[q];
    }
  } else if constexpr (VEC == 4) {
    const f32x4 v = *reinterpret_cast<const f32x4 *>(p);
#pragma unroll
    for (int q = 0; q < 4; ++q) f[q] = v[q];
  } else {
    static_assert(VEC == 1, "16-byte pieces or single elements");
    f[0] = *p;
  }
}

template <int VEC>
__device__ __forceinline__ void store_row(bf16_t *p, const float (&f)[VEC]) {
  if constexpr (VEC == 8) {
    *reinterpret_cast<u32x4 *>(p) = u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                          pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
  } else if constexpr (VEC == 4) {
    *reinterpret_cast<u32x2 *>(p) = u32x2{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])};
  } else {
    p->v = f32_to_bf16(f[0]);
  }
}

template <int VEC>
__device__ __forceinline__ void store_row(float *p, const float (&f)[VEC]) {
  if constexpr (VEC == 8) {
    *reinterpret_cast<f32x4 *>(p) = f32x4{f[0], f[1], f[2], f[3]};
    *reinterpret_cast<f32x4 *>(p + 4) = f32x4{f[4], f[5], f[6], f[7]};
  } else if constexpr (VEC == 4) {
    *reinterpret_cast<f32x4 *>(p) = f32x4{f[0], f[1], f[2], f[3]};
  } else {
    *p = f[0];
  }
}

// A piece as it is stored, for rows fetched ahead of their use; zeros when `in`
// is false. hide() makes it another value to the compiler, which then computes what
// is made from it again instead of holding that.
template <typename T, int VEC>
struct Raw;
template <>
struct Raw<bf16_t, 8> {
  u32x4 v;
  __device__ __forceinline__ void fetch(const bf16_t *p, bool in) {
    v = u32x4{0u, 0u, 0u, 0u};
    if (in) v = *reinterpret_cast<const u32x4 *>(p);
  }
  __device__ __forceinline__ void hide() { asm volatile("" : "+v"(v)); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f[2 * q] = bf16_lo(v[q]);
      f[2 * q + 1] = bf16_hi(v[q]);
    }
  }
};
template <>
struct Raw<bf16_t, 1> {
  uint32_t v;
  __device__ __forceinline__ void fetch(const bf16_t *p, bool in) {
    v = 0;
    if (in) v = p->v;
  }
  __device__ __forceinline__ void hide() { asm volatile("" : "+v"(v)); }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = bf16_to_f32(uint16_t(v)); }
};
template <int VEC>
struct Raw<float, VEC> {
  float v[VEC];
  __device__ __forceinline__ void fetch(const float *p, bool in) {
#pragma unroll
    for (int q = 0; q < VEC; ++q) v[q] = 0.0f;
    if (in) load_row<VEC>(p, v);
  }
  __device__ __forceinline__ void hide() {
#pragma unroll
    for (int q = 0; q < VEC; ++q) asm volatile("" : "+v"(v[q]));
  }
  __device__ __forceinline__ void get(float (&f)[VEC]) const {
#pragma unroll
    for (int q = 0; q < VEC; ++q) f[q] = v[q];
  }
};

// the sum over each run of L lanes, on all of them
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = L / 2; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ float wave_sum(float v) { return lanes_sum<64>(v); }

}  // namespace e4b
