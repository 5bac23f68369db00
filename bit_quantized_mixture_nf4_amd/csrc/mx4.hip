// mx4.hip -- rows of activations in microscaled 4-bit floats: E2M1 codes with an
// E8M0 scale for every 32 consecutive elements, in the layout of a stored MXFP4
// stack (the even element of a byte in its high half). The conversion is the OCP
// Microscaling Formats (MX) v1.0 one, as for the stacks: shared exponent
// floor(log2(max |v|)) - 2 clamped to [-127, 127], elements to the nearest value,
// ties to even, beyond 6 saturated.
//
// The exponent is read from the largest magnitude's bits and the elements are
// rounded by v_cvt_scalef32_pk_fp4, which takes two of them, bf16 as they are stored,
// and divides by the scale: its results equal the definition's for all 255 scales,
// every tie and border, subnormal inputs among them (checked against the oracle). Infinity and
// NaN have no E2M1 code, and the instruction would make 6 of them: a block that holds one gets
// the scale NaN (255) and codes of 0, and so reads as NaN throughout.
//
// Gated rows are v = silu(g) u of rows [g | u]. In fp32 v is off by a few steps, enough to
// take the other of two codes, or exponents, that it lies between; where a step of 2^-20
// relative to it either way would, the block's lanes compute it in 64 bits. So the codes are those
// of the exact v.
#include <type_traits>

#include "kernels.h"
#include "rowvec.h"

namespace e4b {

namespace {

// i / d by one wide product: floor(i m / 2^64) with m = floor(2^64 / d) + 1 is it while
// i (m d - 2^64) <= i d < 2^64 (i below 2^32 pieces, d a row's, at most 2^17).
struct Divisor {
  uint64_t m;
  uint32_t d;
};
inline Divisor divisor_of(uint32_t d) { return {~uint64_t(0) / d + 1, d}; }  // (d at least 8)
__device__ __forceinline__ uint64_t quotient(uint64_t i, Divisor d) { return __umul64hi(i, d.m); }

// Four lanes hold a block, 8 elements each: their integers' maximum, on all four.
__device__ __forceinline__ uint32_t block_max(uint32_t v) {
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0xB1, 0xF, 0xF, false)));  // quad_perm 1 0 3 2
  return max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x4E, 0xF, 0xF, false)));  // 2 3 0 1
}

// The scale byte of a block from the bits of its largest magnitude: the biased exponent less 2.
// (Exponent fields 0 to 2, fp32's subnormals among them, are clamped to 2^-127.)
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return e == 255 ? 255u : max(e, 2u) - 2u;
}

__device__ __forceinline__ uint32_t codes_of(const float (&v)[8], uint32_t byte) {
  const float s = __uint_as_float(byte << 23);
  uint32_t w = 0;
  // the first of a pair goes to the low half, so that the even element comes second
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[1], v[0], s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[3], v[2], s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[5], v[4], s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[7], v[6], s, 3);
  return byte == 255 ? 0u : w;
}

__device__ __forceinline__ uint32_t magnitude(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) m = max(m, __float_as_uint(v[q]) & 0x7FFFFFFFu);
  return m;
}

// e^a of full relative precision, |a| up to kFar: the product a log2 e is off by half a step of its own, which
// the second term adds back. (Down to -128 the power leaves fp32's range; far beyond, the product does.)
constexpr float kFar = 64.0f;
__device__ __forceinline__ float exponential(float a) {
  const float t = a * 1.4426950408889634f;
  const float r = fmaf(a, 1.9259629911266175e-8f, fmaf(a, 1.4426950408889634f, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return fmaf(e, r * 0.6931471805599453f, e);
}
// silu(g) for g above -kFar, off by 2^-21 of itself at most (steps of 2^-24: two of the power, one each of its
// correction, the sum and the product, two of the quotient).
constexpr float kOff = 0x1p-20f;
__device__ __forceinline__ float silu(float g) {
  return g * __builtin_amdgcn_rcpf(1.0f + exponential(fmaxf(-g, -kFar)));
}
__device__ __forceinline__ double silu64(double g) {
  const double e = exp(-fabs(g));
  const double s = (g < 0.0 ? e : 1.0) / (1.0 + e);
  return s == 0.0 ? -0.0 : g * s;  // (silu(-inf) = -0)
}
// The fp32 value that lies where d does among the values and borders of a block: towards
// zero, with the last bit standing for what was cut off. Beyond fp32's range: infinite.
__device__ __forceinline__ float in_place(double d) {
  const float f = __double2float_rz(d);
  if (fabs(d) > 0x1.fffffep127) return d > 0.0 ? INFINITY : -INFINITY;
  return double(f) != d ? __uint_as_float(__float_as_uint(f) | 1u) : f;
}

// Bound by memory: 8191 x 4096 in fp32 take 25 us, 6.0 TB/s.
template <typename T>
__global__ __launch_bounds__(256) void mx4_rows_kernel(const T *__restrict__ x, int64_t pieces,
                                                       uint32_t *__restrict__ codes, uint8_t *__restrict__ scales) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  float v[8];
  load_row<8>(x + min(i, pieces - 1) * 8, v);
  const uint32_t byte = scale_byte(block_max(magnitude(v)));
  if (i >= pieces) return;
  codes[i] = codes_of(v, byte);
  if ((threadIdx.x & 3) == 0) scales[i >> 2] = uint8_t(byte);
}

// The same of silu(g) u. `per` = pieces of 8 to a row of K. 32768 rows of 2 x 1024 in bf16: 34 us, 4.4 TB/s
// (with the checks below made for each value and not for the block, 40: 45 instructions a value, now 24).
template <typename T>
__global__ __launch_bounds__(256) void mx4_gated_kernel(const T *__restrict__ x, int64_t pieces, Divisor per,
                                                        uint32_t *__restrict__ codes, uint8_t *__restrict__ scales) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t j = min(i, pieces - 1);
  const T *p = x + (j + int64_t(quotient(j, per)) * per.d) * 8;  // row * 2 K + column
  float g[8], u[8], v[8];
  load_row<8>(p, g);
  load_row<8>(p + int64_t(per.d) * 8, u);
  float low = 0.0f, least = INFINITY, top = 0.0f;
  bool nan = false;
#pragma unroll
  for (int q = 0; q < 8; q += 2) {
    v[q] = silu(g[q]) * u[q];
    v[q + 1] = silu(g[q + 1]) * u[q + 1];
    low = fminf(fminf(low, g[q]), g[q + 1]);
    least = fminf(fminf(least, fabsf(g[q])), fabsf(g[q + 1]));
    top = fmaxf(fmaxf(top, fabsf(v[q])), fabsf(v[q + 1]));
    nan |= __builtin_isunordered(v[q], v[q + 1]);
  }
  // Not to be had in fp32: far below zero; a block near either end of fp32's range (in one that is not, a value
  // that lost bits as a subnormal has the code 0), and a g that lost some.
  const uint32_t amax = block_max(nan ? 0x7FC00000u : __float_as_uint(top));
  uint32_t unsure = low < -kFar || amax >= 0x7F000000u /* 2^127 */ || (amax < 0x0D800000u /* 2^-100 */ && amax != 0);
  if (least < 0x1p-100f)
#pragma unroll
    for (int q = 0; q < 8; ++q) unsure |= fabsf(g[q]) < 0x1p-100f && g[q] != 0.0f && u[q] != 0.0f;
  const float most = __uint_as_float(amax);
  uint32_t byte = scale_byte(__float_as_uint(fmaf(most, -kOff, most)));
  unsure |= byte ^ scale_byte(__float_as_uint(fmaf(most, kOff, most)));
  float lo[8], hi[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    lo[q] = fmaf(v[q], -kOff, v[q]);
    hi[q] = fmaf(v[q], kOff, v[q]);
  }
  uint32_t w = codes_of(lo, byte);
  unsure |= w ^ codes_of(hi, byte);
  if (block_max(unsure)) {  // all four lanes of a block
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = in_place(silu64(double(g[q])) * double(u[q]));
    byte = scale_byte(block_max(magnitude(v)));
    w = codes_of(v, byte);
  }
  if (i >= pieces) return;
  codes[i] = w;
  if ((threadIdx.x & 3) == 0) scales[i >> 2] = uint8_t(byte);
}

// The gradient of [g | u] from that of silu(g) u: du = ga g s, dg = ga u s (1 + g (1 - s)), s = sigmoid(g).
// Bound by memory: 32768 rows of 2 x 1024 in bf16 take 58 us, 5.8 TB/s.
template <typename T, typename G>
__global__ __launch_bounds__(256) void mx4_gated_bwd_kernel(const T *__restrict__ x, const G *__restrict__ grad,
                                                            int64_t pieces, Divisor per, T *__restrict__ out) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= pieces) return;
  const int64_t at = (i + int64_t(quotient(i, per)) * per.d) * 8, half = int64_t(per.d) * 8;
  float g[8], u[8], ga[8];
  load_row<8>(x + at, g);
  load_row<8>(x + at + half, u);
  load_row<8>(grad + i * 8, ga);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const bool neg = g[q] < 0.0f;
    float gs, slope;
    if (g[q] < -kFar) {
      // the sigmoid leaves fp32's range before its products with a gradient do
      const double gd = g[q], e = exp(gd), s = e / (1.0 + e);
      g[q] = float(double(ga[q]) * double(u[q]) * (s == 0.0 ? 0.0 : s * (1.0 + gd / (1.0 + e))));
      u[q] = float(double(ga[q]) * silu64(gd));
      continue;
    }
    // (an argument beyond what `exponential` takes: at -128 the power is 0 already. A NaN stays one.)
    const float a = -fabsf(g[q]), e = exponential(a < -128.0f ? -128.0f : a), r = __builtin_amdgcn_rcpf(1.0f + e);
    const float s = neg ? e * r : r, rest = neg ? r : e * r;  // 1 - s, without a difference
    gs = g[q] * s;
    slope = e == 0.0f ? s : s * fmaf(g[q], rest, 1.0f);  // (an infinite g times 0)
    // The factors in an order that stays in range where the result does: ga u is infinite with a slope down to 2^-92
    // to follow (|ga| and |u| are above 1 then, and the slope below 1.1), and half of a subnormal g loses its last bit.
    const float p = ga[q] * u[q];
    const float dg = fabsf(p) == INFINITY ? ga[q] * slope * u[q] : p * slope;
    u[q] = fabsf(g[q]) < 0x1p-100f ? ga[q] * g[q] * s : ga[q] * gs;
    g[q] = dg;
  }
  store_row<8>(out + at, g);
  store_row<8>(out + at + half, u);
}

}  // namespace
}  // namespace e4b

using namespace e4b;

extern "C" e4b_status e4b_mx4_rows(const void *x, int32_t dtype, int64_t rows, int64_t K, int32_t gated, uint8_t *codes,
                                   uint8_t *scales, hipStream_t stream) {
  const e4b_status s = check_mx_rows(rows, K);
  if (s != E4B_OK) return s;
  if (dtype != E4B_F32 && dtype != E4B_BF16) return E4B_ERR_DTYPE;
  if (rows == 0) return E4B_OK;
  if (!x || !codes || !scales) return E4B_ERR_NULL;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return E4B_ERR_ALIGN;
  const int64_t pieces = rows * (K / 8);
  const dim3 grid(uint32_t((pieces + 255) / 256));
  const Divisor per = divisor_of(uint32_t(K / 8));
  uint32_t *c = reinterpret_cast<uint32_t *>(codes);
  auto go = [&](auto *p) {
    using T = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    if (gated)
      hipLaunchKernelGGL(mx4_gated_kernel<T>, grid, dim3(256), 0, stream, p, pieces, per, c, scales);
    else
      hipLaunchKernelGGL(mx4_rows_kernel<T>, grid, dim3(256), 0, stream, p, pieces, c, scales);
  };
  if (dtype == E4B_F32)
    go(static_cast<const float *>(x));
  else
    go(static_cast<const bf16_t *>(x));
  return hipGetLastError() == hipSuccess ? E4B_OK : E4B_ERR_HIP;
}

extern "C" e4b_status e4b_mx4_rows_backward(const void *x, int32_t dtype, const void *grad, int32_t grad_dtype,
                                            int64_t rows, int64_t K, void *grad_x, hipStream_t stream) {
  const e4b_status s = check_mx_rows(rows, K);
  if (s != E4B_OK) return s;
  if ((dtype != E4B_F32 && dtype != E4B_BF16) || (grad_dtype != E4B_F32 && grad_dtype != E4B_BF16)) return E4B_ERR_DTYPE;
  if (rows == 0) return E4B_OK;
  if (!x || !grad || !grad_x) return E4B_ERR_NULL;
  if (!aligned16(x) || !aligned16(grad) || !aligned16(grad_x)) return E4B_ERR_ALIGN;
  const int64_t pieces = rows * (K / 8);
  const dim3 grid(uint32_t((pieces + 255) / 256));
  const Divisor per = divisor_of(uint32_t(K / 8));
  auto go = [&](auto *p, auto *g, auto *o) {
    using T = std::remove_pointer_t<decltype(o)>;
    using G = std::remove_const_t<std::remove_pointer_t<decltype(g)>>;
    hipLaunchKernelGGL((mx4_gated_bwd_kernel<T, G>), grid, dim3(256), 0, stream, p, g, pieces, per, o);
  };
  const bool gf = grad_dtype == E4B_F32;
  if (dtype == E4B_F32) {
    const float *p = static_cast<const float *>(x);
    float *o = static_cast<float *>(grad_x);
    gf ? go(p, static_cast<const float *>(grad), o) : go(p, static_cast<const bf16_t *>(grad), o);
  } else {
    const bf16_t *p = static_cast<const bf16_t *>(x);
    bf16_t *o = static_cast<bf16_t *>(grad_x);
    gf ? go(p, static_cast<const float *>(grad), o) : go(p, static_cast<const bf16_t *>(grad), o);
  }
  return hipGetLastError() == hipSuccess ? E4B_OK : E4B_ERR_HIP;
}
