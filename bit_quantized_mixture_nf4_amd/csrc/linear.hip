// linear.hip -- the product of expert-sorted rows with a stored weight stack,
// with bias, activation and residual in its epilogue, and its gradient for a
// frozen stack:
//   z = W[e] x + b[e],  y = act(z) + residual
//   dz = grad_y act'(z),  grad_x = W[e]^T dz,  grad_b[e] = sum over e's rows of dz
// W is the bf16 view of the stored weights (bf16(fl32(code * scale))), the
// products are bf16 MFMAs accumulated in fp32 and the epilogue is fp32 from
// the accumulators on: bias, activation and residual cost no pass of their
// own. dz is rounded to bf16 once, as the MFMA's operand; the bias gradient
// sums the unrounded dz. The pre-activation is kept (or recomputed) in fp32, so
// that nothing but dz's own rounding separates grad_x from the formula.
//
// Rows of expert e are offsets[e] .. offsets[e + 1] - 1 (no offsets: every row
// is expert 0's). A tile map made on the device lists the row tiles, so the
// host never waits for the counts; rows behind the last expert's are zeros in
// every output.
#include <type_traits>

#include "act.h"
#include "codebook8.h"
#include "gemm_dev.h"
#include "plan_block.h"
#include "rowvec.h"

namespace e4b {

namespace {

// ---- the tile map ----

// Workgroup 0 lists the row tiles of every expert: tile_offsets[e] = first
// tile of e, map[t] = (e, first row of e, first row within e, rows). The
// others write zeros to the rows of up to two outputs that no expert has.
// Offsets are clamped to [0, rows] and to ascending order, so that no list of
// offsets leads out of a buffer.
constexpr int kMapThreads = 1024;
constexpr int kZeroBlocks = 64;

__device__ __forceinline__ int32_t clamped_offset(const int32_t *offsets, int i, int E, int32_t rows) {
  if (!offsets) return i < E ? 0 : rows;
  return min(max(offsets[i], 0), rows);
}

__global__ __launch_bounds__(kMapThreads) void tile_map_kernel(const int32_t *__restrict__ offsets, int E,
                                                               int32_t rows, int bm, int32_t *__restrict__ tile_offsets,
                                                               int4 *__restrict__ map, int64_t bound, char *zero_a,
                                                               int64_t row_bytes_a, char *zero_b, int64_t row_bytes_b) {
  if (blockIdx.x > 0) {
    const int64_t live = clamped_offset(offsets, E, E, rows);
    const int64_t i0 = int64_t(blockIdx.x - 1) * kMapThreads + threadIdx.x;
    const int64_t step = int64_t(gridDim.x - 1) * kMapThreads;
    // row lengths are multiples of 2 bytes; the rows' start may be unaligned
    if (zero_a)
      for (int64_t i = live * row_bytes_a / 2 + i0; i < rows * row_bytes_a / 2; i += step)
        reinterpret_cast<uint16_t *>(zero_a)[i] = 0;
    if (zero_b)
      for (int64_t i = live * row_bytes_b / 2 + i0; i < rows * row_bytes_b / 2; i += step)
        reinterpret_cast<uint16_t *>(zero_b)[i] = 0;
    return;
  }
  __shared__ int32_t first[kMaxE + 1];  // first tile of each expert
  __shared__ int32_t wsum[kMapThreads / 64];
  const int e = threadIdx.x, lane = e & 63, wave = e >> 6;
  int32_t lo = 0, n = 0;
  if (e < E) {
    lo = clamped_offset(offsets, e, E, rows);
    n = max(clamped_offset(offsets, e + 1, E, rows) - lo, 0);
  }
  const int32_t tiles = (n + bm - 1) / bm;
  int32_t incl = tiles;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int32_t u = __shfl_up(incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 63) wsum[wave] = incl;
  __syncthreads();
  int64_t before = 0;
  for (int w = 0; w < wave; ++w) before += wsum[w];
  // descending offsets may list more tiles than the map holds: what does not fit is left out
  const int64_t mine = before + incl - tiles;
  if (e < E) first[e] = int32_t(mine < bound ? mine : bound);
  if (e == E - 1) first[E] = int32_t(before + incl < bound ? before + incl : bound);
  __syncthreads();
  for (int q = e; q < E + 1; q += kMapThreads) tile_offsets[q] = first[q];
  const int32_t total = first[E];
  for (int32_t t = threadIdx.x; t < total; t += kMapThreads) {
    // the last expert whose first tile is <= t
    int a = 0, b = E;
    while (b - a > 1) {
      const int m = (a + b) >> 1;
      if (first[m] <= t)
        a = m;
      else
        b = m;
    }
    const int32_t s = clamped_offset(offsets, a, E, rows);
    const int32_t cnt = clamped_offset(offsets, a + 1, E, rows) - s, r0 = (t - first[a]) * bm;
    map[t] = int4{a, s, r0, min(bm, cnt - r0)};
  }
}

// ---- the tiled product ----

// 128 rows x 128 columns x 64: 4 waves of 64 x 64 (2 x 2 MFMA 32x32x16 bf16),
// the weight as the MFMA's A operand, so that a lane's accumulators are runs of
// 4 columns of one row. While K-step ks runs from one LDS stage, the registers
// hold K-step ks + 1, which goes to the other stage (weights decoded on the
// way). 78 KB of LDS: two workgroups per CU cover each other's waits.
constexpr int kTM = 128, kTN = 128;
constexpr int kTThreads = 256;
constexpr int kTBn = kTN + 32;  // row stride of the [k][n] weight tile (dgrad)
constexpr int kTOut = kTN + 4;  // row stride of the epilogue's fp32 tile
constexpr int kStageA = kTM * kLds, kStageB = kBK * kTBn;  // elements of a stage

// How a weight reaches bf16: the 32 codes of one thread's piece.
enum { LK_ABSMAX = 0, LK_MX = 1, LK_BF16 = 2, LK_CODE8 = 3 };

template <int SK>
struct Piece {
  u32x4 v[SK == LK_BF16 ? 4 : SK == LK_CODE8 ? 2 : 1];
  float s;
};

template <int SK>
__device__ __forceinline__ void decode_piece(const Piece<SK> &p, const float *code, u32x4 (&o)[4]) {
  if constexpr (SK == LK_BF16) {
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = p.v[q];
  } else if constexpr (SK == LK_CODE8) {
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const uint32_t w = p.v[q >> 3][(q >> 1) & 3] >> (16 * (q & 1));
      o[q >> 2][q & 3] = pack_bf16x2(__fmul_rn(code[w & 255], p.s), __fmul_rn(code[(w >> 8) & 255], p.s));
    }
  } else {
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const uint32_t b = p.v[0][q >> 2] >> (8 * (q & 3));
      o[q >> 2][q & 3] = pack_bf16x2(__fmul_rn(code[(b >> 4) & 15], p.s), __fmul_rn(code[b & 15], p.s));
    }
  }
}

template <int SK>
__device__ __forceinline__ void fill_codes(float *code, int cb) {
  if constexpr (SK == LK_CODE8) {
    for (int i = threadIdx.x; i < 256; i += blockDim.x) {
      const float m = kMag8[cb - E4B_CB_INT8].v[i & 127];
      code[i] = i < 128 ? m : -m;
    }
  } else if constexpr (SK != LK_BF16) {
    if (threadIdx.x < 16) code[threadIdx.x] = codebook_value(cb, threadIdx.x);
  }
}

// bytes of n stored weights
template <int SK>
__device__ __forceinline__ int64_t code_bytes(int64_t n) {
  return SK == LK_BF16 ? n * 2 : SK == LK_CODE8 ? n : n / 2;
}

// the 32 consecutive weights from column c of stored row `row`
template <int SK>
__device__ __forceinline__ void load_piece(const LinearArgs &g, int64_t e, int64_t row, int c, Piece<SK> &p) {
  const int64_t at = (e * g.out + row) * g.in + c;
  const u32x4 *src = reinterpret_cast<const u32x4 *>(g.packed + code_bytes<SK>(at));
#pragma unroll
  for (int q = 0; q < int(sizeof(p.v) / sizeof(p.v[0])); ++q) p.v[q] = src[q];
  p.s = SK == LK_MX ? e8m0_value(g.scales[at >> 5]) : SK == LK_BF16 ? 1.0f : g.absmax[at >> 6];
}

// NN = false: C[row, n] = sum_k A[row, k] W[n, k] with the epilogue;
// NN = true:  C[row, n] = sum_k A[row, k] W[k, n], stored as bf16.
template <int SK, bool NN>
__global__ __launch_bounds__(kTThreads, 2) void linear_tile_kernel(LinearArgs g) {
  __shared__ __attribute__((aligned(64))) float code[SK == LK_CODE8 ? 256 : 16];
  __shared__ __attribute__((aligned(16))) uint16_t lds[2 * (kStageA + kStageB)];
  static_assert(kTN * kLds <= kStageB, "either form of the weight tile fits its stage");
  static_assert(kTM * kTOut * 4 <= (kStageA + kStageB) * 4, "the epilogue's tile fits the stages");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;

  // real tiles split evenly over the 8 XCDs (block b runs on XCD b % 8), in
  // groups of 8 row tiles so that an XCD's L2 sees both operands again
  const int n_mt = g.tile_offsets[g.E];
  const int N = NN ? g.in : g.out;
  const uint32_t n_nt = uint32_t((N + kTN - 1) / kTN), W = uint32_t(n_mt) * n_nt;
  const uint32_t per = (W + 7) / 8, xi = blockIdx.x / 8;
  const uint32_t L = (blockIdx.x % 8) * per + xi;
  if (xi >= per || L >= W) return;
  constexpr uint32_t kGroup = 8;
  const uint32_t grp = L / (kGroup * n_nt), rem = L % (kGroup * n_nt), m0 = grp * kGroup;
  const uint32_t gm = min(kGroup, uint32_t(n_mt) - m0);
  const int nt = int(rem / gm);
  const int4 tm = g.tile_map[m0 + rem % gm];
  const int64_t e = tm.x, row0 = int64_t(tm.y) + tm.z;
  const int valid = tm.w;

  fill_codes<SK>(code, g.cb);

  // A: 16-byte chunk tid & 7 of rows (tid >> 3) + 32 i; rows past the tile's
  // last repeat it (their results are not stored)
  const uint16_t *a_src[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    a_src[i] = g.A + (row0 + min((tid >> 3) + 32 * i, valid - 1)) * g.lda + (tid & 7) * 8;
  // B: 32 weights. !NN: half tid & 1 of weight row (tile column) tid >> 1;
  // NN: columns 32 (tid & 3) .. of weight row (K-step's) tid >> 2
  const int b_n = nt * kTN + (tid >> 1);
  const int64_t b_row = b_n < N ? b_n : 0;
  const int b_c = nt * kTN + (tid & 3) * 32 < N ? nt * kTN + (tid & 3) * 32 : 0;
  const int K = NN ? (g.out + kBK - 1) / kBK * kBK : g.in;
  const int nK = K / kBK;

  u32x4 ra[4];
  Piece<SK> rb;
  auto load = [&](int ks) {
#pragma unroll
    for (int i = 0; i < 4; ++i) ra[i] = *reinterpret_cast<const u32x4 *>(a_src[i] + ks * kBK);
    if (!NN)
      load_piece<SK>(g, e, b_row, ks * kBK + (tid & 1) * 32, rb);
    else  // weight rows past the last meet zeros of A
      load_piece<SK>(g, e, min(ks * kBK + (tid >> 2), g.out - 1), b_c, rb);
  };
  auto store = [&](int st) {
    uint16_t *sA = lds + st * kStageA, *sB = lds + 2 * kStageA + st * kStageB;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<u32x4 *>(sA + ((tid >> 3) + 32 * i) * kLds + (tid & 7) * 8) = ra[i];
    u32x4 o[4];
    decode_piece<SK>(rb, code, o);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (!NN)
        *reinterpret_cast<u32x4 *>(sB + (tid >> 1) * kLds + (tid & 1) * 32 + q * 8) = o[q];
      else
        *reinterpret_cast<u32x4 *>(sB + (tid >> 2) * kTBn + nn_unit(4 * (tid & 3) + q) * 8) = o[q];
    }
  };
  // transpose-read addresses of the [k][n] tile (see gemm_wide.hip)
  int q_off[2];
  {
    const int qg = lane >> 4, qs = lane & 15, rrow = 8 * (qg >> 1) + (qs >> 2);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col = wn * 64 + 32 * j + 16 * (qg & 1) + 4 * (qs & 3);
      q_off[j] = rrow * kTBn + nn_unit(col >> 3) * 8 + (col & 7);
    }
  }

  f32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  load(0);
  __syncthreads();  // the code table
  store(0);
  if (nK > 1) load(1);
  __syncthreads();
  for (int ks = 0; ks < nK; ++ks) {
    const uint16_t *sA = lds + (ks & 1) * kStageA, *sB = lds + 2 * kStageA + (ks & 1) * kStageB;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      bf16x8 af[2], bf[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        af[i] = *reinterpret_cast<const bf16x8 *>(sA + (wm * 64 + i * 32 + (lane & 31)) * kLds + (lane >> 5) * 8 + kk * 16);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (!NN) {
          bf[j] = *reinterpret_cast<const bf16x8 *>(sB + (wn * 64 + j * 32 + (lane & 31)) * kLds + (lane >> 5) * 8 + kk * 16);
        } else {
          const uint16_t *p = sB + q_off[j] + kk * 16 * kTBn;
          const s16x4 lo = lds_read_tr16(p), hi = lds_read_tr16(p + 4 * kTBn);
          bf[j] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf[j], af[i], acc[i][j], 0, 0, 0);
    }
    if (ks + 1 < nK) {
      store((ks + 1) & 1);
      if (ks + 2 < nK) load(ks + 2);
    }
    __syncthreads();
  }

  // ---- epilogue: the fp32 tile goes through LDS, so that every global access
  // is a run of a row; acc[i][j][4 q + t] is row wm 64 + 32 i + lane % 32,
  // column wn 64 + 32 j + 8 q + 4 (lane / 32) + t ----
  float *tile = reinterpret_cast<float *>(lds);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x16 &c = acc[i][j];
        *reinterpret_cast<f32x4 *>(tile + (wm * 64 + i * 32 + (lane & 31)) * kTOut + wn * 64 + j * 32 + 8 * q +
                                   4 * (lane >> 5)) = f32x4{c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
      }
  __syncthreads();
  if (NN) {
    const int cc = (tid & 15) * 8, col = nt * kTN + cc;
    if (col < N)  // N is a multiple of 64
      for (int r = tid >> 4; r < valid; r += 16) {
        float v[8];
        load_row<8>(tile + r * kTOut + cc, v);
        store_row<8>(reinterpret_cast<bf16_t *>(g.y) + (row0 + r) * N + col, v);
      }
    return;
  }
  auto rows_of = [&](auto vec_c) {
    constexpr int VEC = decltype(vec_c)::value;
    constexpr int kCols = kTN / VEC;
    const int cc = (tid % kCols) * VEC, col = nt * kTN + cc;
    if (col >= N) return;
    float b[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) b[q] = 0.0f;
    if (g.bias) load_row<VEC>(g.bias + e * g.out + col, b);
    for (int r = tid / kCols; r < valid; r += kTThreads / kCols) {
      float v[VEC];
      load_row<VEC>(tile + r * kTOut + cc, v);
      linear_epilogue<VEC>(g, (row0 + r) * g.out + col, b, v);
    }
  };
  if (g.out % 8 == 0)
    rows_of(std::integral_constant<int, 8>{});
  else
    rows_of(std::integral_constant<int, 1>{});
}

// ---- dz and the bias gradient ----

// dz[row, c] = bf16(grad_y act'(pre)), zeros for the columns that pad a row to
// whole K-steps, and per row tile the fp32 column sums. One workgroup per row
// tile (128 rows of one expert) and 32 VEC columns.
template <typename G, int VEC>
__global__ __launch_bounds__(256) void linear_dz_kernel(LinearArgs g, const G *__restrict__ gy,
                                                        const float *__restrict__ pre, uint16_t *__restrict__ dz,
                                                        int ldz, float *__restrict__ part) {
  __shared__ float red[8][32 * VEC];
  if (int(blockIdx.x) >= g.tile_offsets[g.E]) return;
  const int4 tm = g.tile_map[blockIdx.x];
  const int64_t row0 = int64_t(tm.y) + tm.z;
  const int cl = (threadIdx.x & 31) * VEC, col = blockIdx.y * 32 * VEC + cl, rl = threadIdx.x >> 5;
  float sum[VEC];
#pragma unroll
  for (int q = 0; q < VEC; ++q) sum[q] = 0.0f;
  if (col < g.out) {
#pragma unroll 4
    for (int r = rl; r < tm.w; r += 8) {
      float v[VEC], z[VEC];
      load_row<VEC>(gy + (row0 + r) * g.out + col, v);
      if (g.act != E4B_ACT_NONE) {
        load_row<VEC>(pre + (row0 + r) * g.out + col, z);
#pragma unroll
        for (int q = 0; q < VEC; ++q) v[q] *= act_grad(g.act, z[q]);
      }
#pragma unroll
      for (int q = 0; q < VEC; ++q) sum[q] += v[q];
      if (dz) store_row<VEC>(reinterpret_cast<bf16_t *>(dz) + (row0 + r) * ldz + col, v);
    }
  } else if (col < ldz && dz) {
    const float zero[VEC] = {};
    for (int r = rl; r < tm.w; r += 8) store_row<VEC>(reinterpret_cast<bf16_t *>(dz) + (row0 + r) * ldz + col, zero);
  }
  if (!part) return;
#pragma unroll
  for (int q = 0; q < VEC; ++q) red[rl][cl + q] = sum[q];
  __syncthreads();
  for (int c = threadIdx.x; c < 32 * VEC; c += 256) {
    const int gc = blockIdx.y * 32 * VEC + c;
    if (gc >= g.out) continue;
    float v = 0.0f;
#pragma unroll
    for (int q = 0; q < 8; ++q) v += red[q][c];
    part[int64_t(blockIdx.x) * g.out + gc] = v;
  }
}

// grad_b[e] = the sums of e's row tiles, in order (0 for an expert without rows).
__global__ __launch_bounds__(256) void linear_bias_kernel(LinearArgs g, const float *__restrict__ part,
                                                          float *__restrict__ gb) {
  const int e = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
  if (c >= g.out) return;
  const int t0 = g.tile_offsets[e], t1 = g.tile_offsets[e + 1];
  float v = 0.0f;
#pragma unroll 8
  for (int t = t0; t < t1; ++t) v += part[int64_t(t) * g.out + c];
  gb[int64_t(e) * g.out + c] = v;
}

__global__ __launch_bounds__(256) void fill_zero_kernel(float *p, int64_t n) {
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) p[i] = 0.0f;
}

template <bool NN>
hipError_t launch_tiles(const LinearArgs &a, int64_t m_bound, hipStream_t s) {
  const int64_t N = NN ? a.in : a.out, tiles = m_bound * ((N + kTN - 1) / kTN);
  const dim3 grid(uint32_t((tiles + 7) / 8 * 8)), block(kTThreads);
  switch (a.cb) {
    case E4B_CB_BF16: hipLaunchKernelGGL((linear_tile_kernel<LK_BF16, NN>), grid, block, 0, s, a); break;
    case E4B_CB_MXFP4: hipLaunchKernelGGL((linear_tile_kernel<LK_MX, NN>), grid, block, 0, s, a); break;
    case E4B_CB_INT8:
    case E4B_CB_FP8: hipLaunchKernelGGL((linear_tile_kernel<LK_CODE8, NN>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((linear_tile_kernel<LK_ABSMAX, NN>), grid, block, 0, s, a); break;
  }
  return hipGetLastError();
}

hipError_t launch_map(const LinearPlan &p, const LinearArgs &a, const int32_t *offsets, int bm, int64_t bound,
                      void *zero_a, int64_t bytes_a, void *zero_b, int64_t bytes_b, hipStream_t s) {
  // without offsets every row belongs to an expert: nothing to clear
  const uint32_t grid = offsets && (zero_a || zero_b) ? 1 + kZeroBlocks : 1;
  hipLaunchKernelGGL(tile_map_kernel, dim3(grid), dim3(kMapThreads), 0, s, offsets, int(a.E), int32_t(p.rows), bm,
                     const_cast<int32_t *>(a.tile_offsets), const_cast<int4 *>(a.tile_map), bound,
                     static_cast<char *>(zero_a), bytes_a, static_cast<char *>(zero_b), bytes_b);
  return hipGetLastError();
}

template <typename G, int VEC>
hipError_t launch_dz(const LinearPlan &p, const LinearArgs &a, const void *gy, const float *pre, uint16_t *dz,
                     float *part, hipStream_t s) {
  const int64_t width = dz ? p.ldz : a.out;
  const dim3 grid(uint32_t(p.m_bound), uint32_t((width + 32 * VEC - 1) / (32 * VEC)));
  hipLaunchKernelGGL((linear_dz_kernel<G, VEC>), grid, dim3(256), 0, s, a, static_cast<const G *>(gy), pre, dz,
                     int(p.ldz), part);
  return hipGetLastError();
}

LinearArgs args_of(const LinearPlan &p, const e4b_stack *st, char *ws) {
  LinearArgs a{};
  a.packed = st->packed;
  a.absmax = st->absmax;
  a.scales = st->scales;
  a.E = int32_t(st->E);
  a.out = int32_t(st->out);
  a.in = int32_t(st->in);
  a.cb = st->codebook;
  a.tile_offsets = reinterpret_cast<const int32_t *>(ws + p.off_tile_offsets);
  a.tile_map = reinterpret_cast<const int4 *>(ws + p.off_tile_map);
  return a;
}

}  // namespace
}  // namespace e4b

using namespace e4b;

#define E4B_TRY(expr)                             \
  do {                                            \
    if ((expr) != hipSuccess) return E4B_ERR_HIP; \
  } while (0)

extern "C" size_t e4b_expert_linear_workspace_bytes(const e4b_stack *st, int64_t rows) {
  LinearPlan p;
  return plan_linear(st, rows, E4B_ACT_NONE, E4B_BF16, &p) == E4B_OK ? p.fwd_bytes : 0;
}

extern "C" size_t e4b_expert_linear_dgrad_workspace_bytes(const e4b_stack *st, int64_t rows, int32_t recompute) {
  LinearPlan p;
  if (plan_linear(st, rows, E4B_ACT_NONE, E4B_BF16, &p) != E4B_OK) return 0;
  return recompute ? p.bwd_recompute_bytes : p.bwd_bytes;
}

extern "C" e4b_status e4b_expert_linear(const e4b_stack *st, int64_t rows, const int32_t *offsets, const void *x_bf16,
                                        const float *bias, int32_t act, const void *residual_bf16, int32_t y_dtype,
                                        void *y, float *pre, void *ws, size_t ws_bytes, hipStream_t stream) {
  LinearPlan p;
  const e4b_status s = plan_linear(st, rows, act, y_dtype, &p);
  if (s != E4B_OK) return s;
  if (!offsets && st->E != 1) return E4B_ERR_NULL;
  if (rows == 0) return E4B_OK;
  if (!x_bf16 || !y || !ws) return E4B_ERR_NULL;
  if (ws_bytes < p.fwd_bytes) return E4B_ERR_WORKSPACE;
  if (!aligned16(offsets) || !aligned16(x_bf16) || !aligned16(bias) || !aligned16(residual_bf16) || !aligned16(y) ||
      !aligned16(pre) || !aligned16(ws))
    return E4B_ERR_ALIGN;
  LinearArgs a = args_of(p, st, static_cast<char *>(ws));
  a.A = static_cast<const uint16_t *>(x_bf16);
  a.lda = st->in;
  a.bias = bias;
  a.act = act;
  a.residual = static_cast<const uint16_t *>(residual_bf16);
  a.y = y;
  a.y_f32 = y_dtype == E4B_F32;
  a.pre = pre;
  E4B_TRY(launch_map(p, a, offsets, kTM, p.m_bound, y, st->out * (a.y_f32 ? 4 : 2), pre, st->out * 4, stream));
  E4B_TRY(launch_tiles<false>(a, p.m_bound, stream));
  return E4B_OK;
}

extern "C" e4b_status e4b_expert_linear_dgrad(const e4b_stack *st, int64_t rows, const int32_t *offsets,
                                              const void *grad_y, int32_t gy_dtype, const float *pre,
                                              const void *x_bf16, const float *bias, int32_t act, void *grad_x_bf16,
                                              float *grad_bias, void *ws, size_t ws_bytes, hipStream_t stream) {
  LinearPlan p;
  const e4b_status s = plan_linear(st, rows, act, gy_dtype, &p);
  if (s != E4B_OK) return s;
  if (!offsets && st->E != 1) return E4B_ERR_NULL;
  if (!aligned16(offsets) || !aligned16(grad_y) || !aligned16(pre) || !aligned16(x_bf16) || !aligned16(bias) ||
      !aligned16(grad_x_bf16) || !aligned16(grad_bias) || !aligned16(ws))
    return E4B_ERR_ALIGN;
  if (rows == 0) {
    // no row adds to a bias gradient
    if (!grad_bias) return E4B_OK;
    const int64_t n = st->E * st->out;
    hipLaunchKernelGGL(fill_zero_kernel, dim3(uint32_t(n < 65536 ? (n + 255) / 256 : 256)), dim3(256), 0, stream,
                       grad_bias, n);
    return hipGetLastError() == hipSuccess ? E4B_OK : E4B_ERR_HIP;
  }
  const bool recompute = act != E4B_ACT_NONE && !pre;
  if (!grad_y || !grad_x_bf16 || !ws || (recompute && !x_bf16)) return E4B_ERR_NULL;
  if (ws_bytes < (recompute ? p.bwd_recompute_bytes : p.bwd_bytes)) return E4B_ERR_WORKSPACE;
  char *w = static_cast<char *>(ws);
  LinearArgs a = args_of(p, st, w);
  a.act = act;
  E4B_TRY(launch_map(p, a, offsets, kTM, p.m_bound, grad_x_bf16, st->in * 2, nullptr, 0, stream));
  if (recompute) {
    // exactly the forward's pre-activation
    LinearArgs f = a;
    f.A = static_cast<const uint16_t *>(x_bf16);
    f.lda = st->in;
    f.bias = bias;
    f.pre = reinterpret_cast<float *>(w + p.off_pre);
    E4B_TRY(launch_tiles<false>(f, p.m_bound, stream));
    pre = f.pre;
  }
  const bool f32 = gy_dtype == E4B_F32;
  // grad_y itself is the operand when it is dz already, in whole K-steps
  const bool direct = act == E4B_ACT_NONE && !f32 && st->out == p.ldz;
  uint16_t *dz = direct ? nullptr : reinterpret_cast<uint16_t *>(w + p.off_dz);
  float *part = grad_bias ? reinterpret_cast<float *>(w + p.off_part) : nullptr;
  if (dz || part) {
    if (st->out % 8 == 0)
      E4B_TRY(f32 ? (launch_dz<float, 8>(p, a, grad_y, pre, dz, part, stream))
                  : (launch_dz<bf16_t, 8>(p, a, grad_y, pre, dz, part, stream)));
    else
      E4B_TRY(f32 ? (launch_dz<float, 1>(p, a, grad_y, pre, dz, part, stream))
                  : (launch_dz<bf16_t, 1>(p, a, grad_y, pre, dz, part, stream)));
  }
  if (part) {
    hipLaunchKernelGGL(linear_bias_kernel, dim3(uint32_t((st->out + 255) / 256), uint32_t(st->E)), dim3(256), 0, stream,
                       a, static_cast<const float *>(part), grad_bias);
    E4B_TRY(hipGetLastError());
  }
  a.A = direct ? static_cast<const uint16_t *>(grad_y) : dz;
  a.lda = direct ? st->out : p.ldz;
  a.y = grad_x_bf16;
  E4B_TRY(launch_tiles<true>(a, p.m_bound, stream));
  return E4B_OK;
}
