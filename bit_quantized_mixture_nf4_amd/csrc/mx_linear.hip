// mx_linear.hip -- the product of rows in microscaled 4-bit floats with a stored
// MXFP4 stack, with bias, activation and residual in its epilogue:
//   z[r, n] = sum_k xq[row(r), k] W[e(r)][n, k],  y = act(z + b[e]) + residual
// Both operands are E2M1 codes with an E8M0 scale for every 32 along k, which is
// what gfx950's block-scaled MFMA multiplies: the codes go from memory to the matrix
// cores as they are stored, and the accumulators are fp32. The even element of a byte
// lies in its high half, where the instruction looks for the odd one; both operands
// are stored so, and a sum over k does not mind.
//
// v_mfma_scale_f32_16x16x128_f8f6f4, both operands E2M1: lane (row r = l % 16, quarter
// q = l / 16) gives 16 bytes = the 32 k of block q of its row, and that block's scale
// byte; D: lane l, register t: row 4 (l / 16) + t of A, row l % 16 of B. Weights are A,
// so that a lane's results are 4 consecutive columns of one row.
//
// Row r of the product is row r of x, or, with the pairs of an expert order, the
// token of its pair: k pairs of a token read its one row, and no copy in expert
// order is made.
#include <type_traits>

#include "act.h"
#include "kernels.h"
#include "tiles_dev.h"

namespace e4b {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
__device__ __forceinline__ i32x8 operand(const u32x4 &q) {
  return i32x8{int(q[0]), int(q[1]), int(q[2]), int(q[3]), 0, 0, 0, 0};
}
enum { MX_E2M1 = 4 };  // cbsz / blgp: the operand's format

// The row of x that row r of the product takes (an order that names none reads the last one).
__device__ __forceinline__ int64_t source_row(const MxLinearArgs &g, int64_t r) {
  if (!g.sorted) return r;
  const uint32_t t = uint32_t(g.sorted[r]) / uint32_t(g.top_k);
  return min(t, uint32_t(g.tokens - 1));
}

// One workgroup per block of 16 MT rows of an expert (found from the offsets) and 8 / wk
// groups of 16 columns; wk waves share a column group's k and join their sums in order.
constexpr int kRowThreads = 512;
template <int MT>
__global__ __launch_bounds__(kRowThreads) void mx_rows_kernel(MxLinearArgs m, const int32_t *__restrict__ offsets,
                                                              int32_t rows, int wk, int32_t blocks, int32_t zeros) {
  constexpr int kRows = 16 * MT;
  __shared__ __attribute__((aligned(16))) float part[8][MT][64 * 4];
  const LinearArgs &g = m.lin;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = 8 / wk, slice = wave % wk;
  const int32_t block = int32_t(blockIdx.z * gridDim.y + blockIdx.y);
  if (block >= blocks) {  // the rows of no expert
    const int32_t z = block - blocks;
    if (z >= zeros) return;
    const int64_t from = clamped_offset(offsets, g.E, g.E, rows) * int64_t(g.out), to = rows * int64_t(g.out);
    const int64_t i = (int64_t(z) * gridDim.x + blockIdx.x) * kRowThreads + tid;
    const int64_t n = int64_t(zeros) * gridDim.x * kRowThreads;
    if (g.pre) clear_bytes(reinterpret_cast<char *>(g.pre), from * 4, to * 4, i, n);
    const int y_bytes = g.y_f32 ? 4 : 2;
    clear_bytes(static_cast<char *>(g.y), from * y_bytes, to * y_bytes, i, n);
    return;
  }
  int e;
  int32_t r0, hi;
  if (!block_of(offsets, g.E, rows, kRows, block, lane, e, r0, hi)) return;

  const int col0 = (blockIdx.x * wn + wave / wk) * 16;  // the wave's columns
  const int r = lane & 15, q = lane >> 4;
  const int64_t w_row = int64_t(e) * g.out + min(col0 + r, g.out - 1);
  const uint8_t *wp = g.packed + w_row * (g.in / 2), *ws = g.scales + w_row * (g.in / 32);
  const uint8_t *xp[MT], *xs[MT];
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t x_row = source_row(m, min(r0 + 16 * i + r, hi - 1));
    xp[i] = m.x + x_row * (g.in / 2);
    xs[i] = m.xs + x_row * (g.in / 32);
    acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  const int blocks_k = g.in / 32;
#pragma unroll 2
  for (int b0 = slice * 4; b0 < blocks_k; b0 += wk * 4) {
    const int b = b0 + q;
    // past the row's end (half a step): codes of 0 and scales of 1
    const bool in = b < blocks_k;
    u32x4 w = u32x4{0u, 0u, 0u, 0u};
    uint32_t sw = 127;
    if (in) {
      w = *reinterpret_cast<const u32x4 *>(wp + b * 16);
      sw = ws[b];
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      u32x4 x = u32x4{0u, 0u, 0u, 0u};
      uint32_t sx = 127;
      if (in) {
        x = *reinterpret_cast<const u32x4 *>(xp[i] + b * 16);
        sx = xs[i][b];
      }
      acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(w), operand(x), acc[i], MX_E2M1, MX_E2M1, 0,
                                                                int(sw), 0, int(sx));
    }
  }
  if (wk > 1) {
#pragma unroll
    for (int i = 0; i < MT; ++i) *reinterpret_cast<f32x4 *>(&part[wave][i][lane * 4]) = acc[i];
    __syncthreads();
    if (slice) return;
    for (int s = 1; s < wk; ++s)
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[i] += *reinterpret_cast<const f32x4 *>(&part[wave + s][i][lane * 4]);
  }
  const int c = col0 + 4 * q;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int32_t row = r0 + i * 16 + r;
    if (row >= hi) continue;
    if (g.out % 4 == 0) {
      if (c < g.out) {
        float b[4] = {}, v[4] = {acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
        if (g.bias) load_row<4>(g.bias + int64_t(e) * g.out + c, b);
        linear_epilogue<4>(g, int64_t(row) * g.out + c, b, v);
      }
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (c + t < g.out) {
          float b[1] = {g.bias ? g.bias[int64_t(e) * g.out + c + t] : 0.0f}, v[1] = {acc[i][t]};
          linear_epilogue<1>(g, int64_t(row) * g.out + c + t, b, v);
        }
    }
  }
}

template <int MT>
hipError_t launch_rows_mt(const MxLinearPlan &p, const MxLinearArgs &m, const int32_t *offsets, hipStream_t s) {
  const LinearArgs &a = m.lin;
  const int64_t busy = a.E < p.rows ? a.E : p.rows, groups = (a.out + 15) / 16, steps = (a.in + 127) / 128;
  int wk = 1;
  while (wk < 8 && 2 * wk <= steps && busy * groups * wk < 4096) wk *= 2;
  const int64_t slabs = (groups + 8 / wk - 1) / (8 / wk);
  const int64_t blocks = tiles_at_most(a.E, p.rows, 16 * MT);
  const int64_t bytes = p.rows * a.out * ((a.y_f32 ? 4 : 2) + (a.pre ? 4 : 0));
  const int64_t zeros = offsets ? (clear_groups(bytes, 1024) + slabs - 1) / slabs : 0;
  const int64_t y = blocks + zeros < 32768 ? blocks + zeros : 32768;
  const dim3 grid(uint32_t(slabs), uint32_t(y), uint32_t((blocks + zeros + y - 1) / y));
  hipLaunchKernelGGL(mx_rows_kernel<MT>, grid, dim3(kRowThreads), 0, s, m, offsets, int32_t(p.rows), wk,
                     int32_t(blocks), int32_t(zeros));
  return hipGetLastError();
}

}  // namespace
}  // namespace e4b

using namespace e4b;

extern "C" size_t e4b_mx_linear_workspace_bytes(const e4b_stack *st, int64_t rows) {
  MxLinearPlan p;
  return plan_mx_linear(st, rows, 1, false, E4B_ACT_NONE, E4B_BF16, &p) == E4B_OK ? 0 : 0;
}

extern "C" e4b_status e4b_mx_linear(const e4b_stack *st, int64_t rows, const int32_t *offsets,
                                    const int32_t *sorted_pair, int32_t top_k, const uint8_t *x_codes,
                                    const uint8_t *x_scales, const float *bias, int32_t act, const void *residual_bf16,
                                    int32_t y_dtype, void *y, float *pre, void *ws, size_t ws_bytes,
                                    hipStream_t stream) {
  MxLinearPlan p;
  const e4b_status s = plan_mx_linear(st, rows, top_k, sorted_pair != nullptr, act, y_dtype, &p);
  if (s != E4B_OK) return s;
  if (!offsets && st->E != 1) return E4B_ERR_NULL;
  if (rows == 0) return E4B_OK;
  if (!x_codes || !x_scales || !y) return E4B_ERR_NULL;
  if (!aligned16(offsets) || !aligned16(sorted_pair) || !aligned16(x_codes) || !aligned16(x_scales) ||
      !aligned16(bias) || !aligned16(residual_bf16) || !aligned16(y) || !aligned16(pre) || !aligned16(ws))
    return E4B_ERR_ALIGN;
  (void)ws_bytes;
  MxLinearArgs m{};
  m.x = x_codes;
  m.xs = x_scales;
  m.sorted = sorted_pair;
  m.top_k = sorted_pair ? top_k : 1;
  m.tokens = int32_t(rows / m.top_k);
  LinearArgs &a = m.lin;
  a.packed = st->packed;
  a.scales = st->scales;
  a.E = int32_t(st->E);
  a.out = int32_t(st->out);
  a.in = int32_t(st->in);
  a.rows = rows;
  a.bias = bias;
  a.act = act;
  a.residual = static_cast<const uint16_t *>(residual_bf16);
  a.y = y;
  a.y_f32 = y_dtype == E4B_F32;
  a.pre = pre;
  const int64_t mean = (rows + st->E - 1) / st->E;
  const hipError_t err = mean <= 16   ? launch_rows_mt<1>(p, m, offsets, stream)
                         : mean <= 32 ? launch_rows_mt<2>(p, m, offsets, stream)
                                      : launch_rows_mt<4>(p, m, offsets, stream);
  return err == hipSuccess ? E4B_OK : E4B_ERR_HIP;
}
