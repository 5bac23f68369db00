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

// zeros for the rows of no expert, by thread i of n
__device__ __forceinline__ void clear_tail(const LinearArgs &g, const int32_t *__restrict__ offsets, int64_t i, int64_t n) {
  const int64_t from = clamped_offset(offsets, g.E, g.E, int32_t(g.rows)) * int64_t(g.out), to = g.rows * int64_t(g.out);
  if (g.pre) clear_bytes(reinterpret_cast<char *>(g.pre), from * 4, to * 4, i, n);
  const int y_bytes = g.y_f32 ? 4 : 2;
  clear_bytes(static_cast<char *>(g.y), from * y_bytes, to * y_bytes, i, n);
}

// ---- few rows ----

// One workgroup per block of 16 MT rows of an expert (found from the offsets) and 8 / wk
// groups of 16 columns; wk waves share a column group's k, step by step in turn, and join their sums in
// order. Operands go from memory to registers: the weights' latency decides, and how many waves wait
// for it at a time (one row of 2048 -> 4096: 3.8 us, 3.6 of them a launch's). Four steps asked for ahead, of
// two column groups a wave, were slower (8 experts of 4096 -> 4096, one row each, 27 us against 21): the L1 takes
// one request for each row's 64 bytes of codes, and as many for its scales.
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
  if (block >= blocks) {
    const int32_t z = block - blocks;
    if (z >= zeros) return;
    clear_tail(g, offsets, (int64_t(z) * gridDim.x + blockIdx.x) * kRowThreads + tid, int64_t(zeros) * gridDim.x * kRowThreads);
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

// ---- the tiled product ----

// Tiles of 64 TM rows x 64 TN columns x 128: 4 waves (2 x 2), each of 32 TM x 32 TN as TM x TN
// v_mfma_scale_f32_32x32x64_f8f6f4 for each half of a K-step. Weights are the A operand: lane (row
// r = l % 32, half h = l / 32) gives the 32 k of block h of its row and that block's scale, and
// its results are runs of 4 columns of one row (register 4 q + t: column 8 q + 4 h + t). A row of
// a K-step is 64 bytes of codes and 4 scales, one word, staged as it is and shifted by 8: bytes 0
// and 2 of word h are the scales of the two halves (op_sel).
//
// While K-step ks runs from one LDS stage, ks + 1 goes from registers to the other and ks + 3 is
// asked for (ks + 2 is on its way). The wave's instructions are cut into 2 TM TN slots of one MFMA (32 cycles) and a
// share of that work, each closed by a scheduling barrier. The 16-byte pieces of a row lie at
// piece ^ (row / 4 % 4), so that sixteen rows of one piece fill all banks.
// HALF: the last K-step is half (in % 128 = 64).
//
// 64 x 64 is for experts of few rows and reads their weights at 5.5 to 6 TB/s (128 experts of 2048 -> 1536, one
// row each: 213 MB in 37.5 us). 128 x 128 takes 620 cycles a K-step with two workgroups on a CU (2.5 PFLOP/s at
// 8 x 4096 rows of 4096 -> 4096), twice the time of its MFMA alone: half lines of operands, and twice the requests a
// product that the 256 x 256 tile has. Four waves alone on a CU take 1100 cycles, most of it latency.
template <int I, typename F>
__device__ __forceinline__ void each_slot(F &&f) {
  if constexpr (I > 0) {
    each_slot<I - 1>(f);
    f(std::integral_constant<int, I - 1>{});
  }
}

// memory from p on as a buffer of 2^32 - 1 bytes
typedef __amdgpu_buffer_rsrc_t buffer_t;
__device__ __forceinline__ buffer_t whole_buffer(const uint8_t *p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p), 0, -1, 0x00027000);
}
// of `bytes` bytes, or as far as a lane's offset goes: loads from behind them give zeros
__device__ __forceinline__ buffer_t sized_buffer(const uint8_t *p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p), 0, int(min(bytes, int64_t(0xFFFFFFFFll))), 0x00027000);
}

template <int TM, int TN>
struct MxTile {
  static constexpr int kM = 64 * TM, kN = 64 * TN, kStage = (kM + kN) * 64, kScales = 2 * (kM + kN);  // (words of a K-step)
  static constexpr int kOutLd = 32 * TN + 4;                 // a wave's 32 rows on their way out, fp32
  static constexpr int kOut = 4 * 32 * kOutLd * 4, kIn = 2 * (kStage + 4 * kScales * 4);
  static constexpr int kBytes = kOut > kIn ? kOut : kIn;
};

template <int TM, int TN, bool HALF>
__global__ __launch_bounds__(256, 2) void mx_tile_kernel(MxLinearArgs m, const int32_t *__restrict__ offsets,
                                                         int32_t tiles) {
  using T = MxTile<TM, TN>;
  constexpr int kM = T::kM, kN = T::kN, R = TM + TN, MN = TM * TN, D = 2;
  __shared__ __attribute__((aligned(16))) uint8_t lds[T::kBytes];
  const LinearArgs &g = m.lin;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1, r32 = lane & 31, h = lane >> 5;
  int mt, nt, share;
  int64_t e = 0, row0;
  int valid;
  if (offsets) {
    // found from the offsets: a map of the tiles would cost a launch. How many there are is not known then: the
    // workgroups without one come last, and an XCD takes every eighth column tile.
    if (int32_t(blockIdx.x) >= tiles) {
      clear_tail(g, offsets, int64_t(blockIdx.x - tiles) * 256 + tid, int64_t(gridDim.x - tiles) * 256);
      return;
    }
    const uint32_t n_nt = (g.out + kN - 1) / kN;
    nt = int(blockIdx.x % n_nt);
    int32_t at, r0, hi;
    if (!block_of(offsets, g.E, int32_t(g.rows), kM, int32_t(blockIdx.x / n_nt), lane, at, r0, hi)) return;
    e = at;
    row0 = r0;
    valid = min(kM, hi - r0);
  } else {
    if (!place_of(tile_count(g, kM), (g.out + kN - 1) / kN, 1, 1024 / kM, mt, nt, share)) return;
    const int4 tm = tile_of(g, mt, kM);
    e = tm.x;
    row0 = int64_t(tm.y) + tm.z;
    valid = tm.w;
  }

  // 16-byte piece tid % 4 of rows tid / 4 + 64 i; rows past the last repeat it (their results are not
  // stored). Operands are read as buffers, by 32-bit offsets and a uniform one for the K-step: rows by
  // place and weight rows from the tile's first one (gathered ones from x's, which is checked to fit).
  const int piece = tid & 3, prow = tid >> 2;
  const uint32_t kb = g.in / 2, sb = g.in / 32;
  const int64_t skip = m.sorted ? 0 : row0;
  const buffer_t xb = whole_buffer(m.x + skip * kb), xsb = whole_buffer(m.xs + skip * sb);
  const int64_t w_first = e * g.out + nt * kN;
  const buffer_t wb = whole_buffer(g.packed + w_first * kb), wsb = whole_buffer(g.scales + w_first * sb);
  const auto x_row = [&](int r) -> uint32_t {
    r = min(r, valid - 1);
    return m.sorted ? uint32_t(source_row(m, row0 + r)) : uint32_t(r);
  };
  const auto w_row = [&](int r) -> uint32_t { return min(r, g.out - 1 - nt * kN); };
  uint32_t src[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    src[i] = (i < TM ? x_row(prow + 64 * i) : w_row(prow + 64 * (i - TM))) * kb + piece * 16;
  // the scale words of row tid % kM of x and row tid % kN of the weights (some threads repeat others'),
  // or, where a thread has one row, of either
  constexpr bool kOneRow = kM + kN <= 256;
  constexpr int kWords = kOneRow ? 1 : 2;
  uint32_t ssrc[kWords];
  int sdst[kWords];
  const bool mine_x = tid % (kM + kN) < kM;
  if constexpr (kOneRow) {
    sdst[0] = tid % (kM + kN);
    ssrc[0] = (mine_x ? x_row(sdst[0]) : w_row(sdst[0] - kM)) * sb;
  } else {
    sdst[0] = tid % kM;
    sdst[1] = kM + tid % kN;
    ssrc[0] = x_row(sdst[0]) * sb;
    ssrc[1] = w_row(sdst[1] - kM) * sb;
  }
  const int nK = (g.in + 127) / 128, last = nK - 1;

  u32x4 in[D][R];  // of the next D K-steps
  u32x4 in_s[kWords];  // of the next four, one load a row: a line of scales is read for 4 K-steps
  auto load = [&](int set, int ks, int i) {
    // (HALF: pieces 2 and 3 of the last K-step lie behind the row, and are not multiplied)
    const uint32_t at = HALF && ks == last && piece >= 2 ? src[i] - 32 : src[i];
    in[set % D][i] = __builtin_amdgcn_raw_buffer_load_b128(i < TM ? xb : wb, at, ks * 64, 0);
  };
  auto load_scales = [&](int panel) {
    const int first = 4 * panel;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      // (one row a thread: whole waves have x's or the weights')
      const buffer_t of = i == 0 && (!kOneRow || __builtin_amdgcn_readfirstlane(mine_x)) ? xsb : wsb;
      if (!HALF && first + 4 <= nK) {
        in_s[i] = __builtin_amdgcn_raw_buffer_load_b128(of, ssrc[i], first * 4, 0);
      } else {
        // words past the row's end repeat the last one
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int ks = min(first + w, last);
          if (HALF) {
            const uint32_t lo = __builtin_amdgcn_raw_buffer_load_b16(of, ssrc[i], ks * 4, 0);
            const uint32_t hi = __builtin_amdgcn_raw_buffer_load_b16(of, ssrc[i], ks * 4 + (ks == last ? 0 : 2), 0);
            in_s[i][w] = lo | hi << 16;
          } else {
            in_s[i][w] = __builtin_amdgcn_raw_buffer_load_b32(of, ssrc[i], ks * 4, 0);
          }
        }
      }
    }
  };
  auto stage = [&](int st) { return lds + st * T::kStage; };
  // the scales of K-step ks: two panels of four
  auto scales = [&](int ks) { return reinterpret_cast<uint32_t *>(lds + 2 * T::kStage) + (ks & 7) * T::kScales; };
  auto store = [&](int st, int i) {
    const int row = prow + 64 * i;
    *reinterpret_cast<u32x4 *>(stage(st) + row * 64 + (piece ^ (row >> 2 & 3)) * 16) = in[st % D][i];
  };
  auto store_scales = [&](int panel) {
#pragma unroll
    for (int i = 0; i < kWords; ++i)
#pragma unroll
      for (int w = 0; w < 4; ++w)
        *reinterpret_cast<u32x2 *>(scales(4 * panel + w) + 2 * sdst[i]) = u32x2{in_s[i][w], in_s[i][w] >> 8};
  };

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;
  u32x4 f[2][R];
  int sc[2][R];  // by the K-step's parity
  // fragment i of half kh: 0 .. TM - 1 the wave's rows of x, then its weight rows
  auto row_of = [&](int i) { return i < TM ? wm * 32 * TM + i * 32 + r32 : kM + wn * 32 * TN + (i - TM) * 32 + r32; };
  auto frag = [&](int st, int kh, int i) {
    const int row = row_of(i);
    f[kh][i] = *reinterpret_cast<const u32x4 *>(stage(st) + row * 64 + ((2 * kh + h) ^ (row >> 2 & 3)) * 16);
  };
  auto frag_scale = [&](int st, int ks, int i) { sc[st][i] = int(scales(ks)[2 * row_of(i) + h]); };

  // the first stage; loads past the last K-step repeat it
  auto load_step = [&](int set, int ks) {
#pragma unroll
    for (int i = 0; i < R; ++i) load(set, ks, i);
  };
  load_scales(0);
  load_step(0, 0);
  load_step(1, min(1, last));
#pragma unroll
  for (int i = 0; i < R; ++i) store(0, i);
  store_scales(0);
  load_scales(1);
  load_step(0, min(D, last));
  __syncthreads();
#pragma unroll
  for (int i = 0; i < R; ++i) {
    frag_scale(0, 0, i);
    frag(0, 0, i);
  }

  // fragments in the order in which the MFMAs (rows outside, columns inside) need them: the first
  // rows', all columns', the other rows'
  constexpr auto nth = [](int q) { return q == 0 ? 0 : q <= TN ? TM + q - 1 : q - TN; };
  auto kstep = [&](auto cur_c, int ks) {
    constexpr int CUR = decltype(cur_c)::value, NXT = CUR ^ 1;
    const int ahead = min(ks + 1 + D, last);
    if ((ks & 3) == 3) {  // the next four K-steps' scales, and those behind them
      store_scales((ks >> 2) + 1);
      load_scales((ks >> 2) + 2);
    }
    each_slot<2 * MN>([&](auto slot) {
      constexpr int s = decltype(slot)::value, kh = s / MN, i = s % MN / TN, j = s % TN;
      if constexpr (kh == 0)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(f[0][TM + j]), operand(f[0][i]), acc[i][j],
                                                                    MX_E2M1, MX_E2M1, 0, sc[CUR][TM + j], 0, sc[CUR][i]);
      else if (!HALF || ks < last)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(f[1][TM + j]), operand(f[1][i]), acc[i][j],
                                                                    MX_E2M1, MX_E2M1, 2, sc[CUR][TM + j], 2, sc[CUR][i]);
#pragma unroll
      for (int q = 0; q < R; ++q) {
        if (s == q * MN / R) {
          frag(CUR, 1, nth(q));
          store(NXT, q);
          load(NXT, ahead, q);
        }
        if (s == MN + q * MN / R) {
          frag_scale(NXT, ks + 1, nth(q));
          frag(NXT, 0, nth(q));
        }
      }
      // every wave has filled its share of the next stage, and read its last fragment of this one
      if constexpr (s == MN - 1) {
        __builtin_amdgcn_sched_barrier(0);
        __syncthreads();
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  int ks = 0;
  for (; ks + 1 < nK; ks += 2) {
    kstep(std::integral_constant<int, 0>{}, ks);
    kstep(std::integral_constant<int, 1>{}, ks + 1);
  }
  if (ks < nK) kstep(std::integral_constant<int, 0>{}, ks);
  __syncthreads();  // the last stage's fragments are read

  // ---- epilogue: 32 rows of the wave at a time through its own part of LDS, so that every global
  // access is a run of a row; all rows of a lane side by side, so that their accesses overlap ----
  float *tile = reinterpret_cast<float *>(lds) + wave * 32 * T::kOutLd;
  const int col0 = nt * kN + wn * 32 * TN;
  auto turn = [&](auto ic) {
    constexpr int i = decltype(ic)::value;
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x16 &c = acc[i][j];
        *reinterpret_cast<f32x4 *>(tile + r32 * T::kOutLd + j * 32 + 8 * q + 4 * h) =
            f32x4{c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
      }
    const int first = wm * 32 * TM + i * 32;
    if (g.out % 8 == 0) {
      constexpr int kL = 4 * TN, kRows = 64 / kL, kN8 = 32 / kRows;  // lanes a row, rows at once, turns
      const int cl = lane % kL * 8, col = col0 + cl, r0 = first + lane / kL;
      if (col >= g.out) return;
      const int64_t at = (row0 + r0) * g.out + col;
      float v[8 * kN8], b[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) b[q] = 0.0f;
      if (g.bias) load_row<8>(g.bias + e * g.out + col, b);
      Raw<bf16_t, 8> res[kN8];
      if (g.residual) {
#pragma unroll
        for (int n = 0; n < kN8; ++n)
          res[n].fetch(reinterpret_cast<const bf16_t *>(g.residual) + at + int64_t(n * kRows) * g.out, r0 + n * kRows < valid);
      }
#pragma unroll
      for (int n = 0; n < kN8; ++n)
        load_row<8>(tile + (lane / kL + n * kRows) * T::kOutLd + cl, reinterpret_cast<float(&)[8]>(v[8 * n]));
#pragma unroll
      for (int q = 0; q < 8 * kN8; ++q) v[q] += b[q % 8];
      if (g.pre) {
#pragma unroll
        for (int n = 0; n < kN8; ++n)
          if (r0 + n * kRows < valid)
            store_row<8>(g.pre + at + int64_t(n * kRows) * g.out, reinterpret_cast<float(&)[8]>(v[8 * n]));
      }
      act_values<8 * kN8>(g.act, v);
      if (g.residual) {
#pragma unroll
        for (int n = 0; n < kN8; ++n) {
          float r[8];
          res[n].get(r);
#pragma unroll
          for (int q = 0; q < 8; ++q) v[8 * n + q] += r[q];
        }
      }
#pragma unroll
      for (int n = 0; n < kN8; ++n) {
        if (r0 + n * kRows >= valid) continue;
        const int64_t to = at + int64_t(n * kRows) * g.out;
        if (g.y_f32)
          store_row<8>(static_cast<float *>(g.y) + to, reinterpret_cast<float(&)[8]>(v[8 * n]));
        else
          store_row<8>(static_cast<bf16_t *>(g.y) + to, reinterpret_cast<float(&)[8]>(v[8 * n]));
      }
    } else {
      for (int c = lane % (32 * TN); c < 32 * TN && col0 + c < g.out; c += 64) {
        const float b[1] = {g.bias ? g.bias[e * g.out + col0 + c] : 0.0f};
        for (int r = lane / (32 * TN); r < 32 && first + r < valid; r += TN == 1 ? 2 : 1) {
          float v[1] = {tile[r * T::kOutLd + c]};
          linear_epilogue<1>(g, (row0 + first + r) * g.out + col0 + c, b, v);
        }
      }
    }
  };
  each_slot<TM>(turn);
}

// ---- large products ----

// waits until at most N vector memory operations of the wave are under way
template <int N>
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
}

// 16 bytes a lane from a buffer straight into LDS, 1 KB from `lds` on in the order of the lanes. The
// compiler does not see that LDS is written: every reader is behind a wait for the vector memory counter and
// a barrier written out here. (No register is written, so none can be taken for free while the load flies.)
__device__ __forceinline__ void load_to_lds(buffer_t b, uint32_t offset, uint32_t step, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               :
               : "v"(offset), "s"(b), "s"(step), "s"(lds)
               : "memory", "m0");
}
// The same if `go`, without a branch that the compiler sees: the step around it stays one basic block (behind
// a branch the compiler gathered the matrix instructions, and copied the fragments).
__device__ __forceinline__ void load_to_lds_if(int go, buffer_t b, uint32_t offset, uint32_t lds) {
  asm volatile(
      "s_cmp_eq_u32 %3, 0\n\ts_cbranch_scc1 .Lmx_no_load%=\n\t"
      "s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds\n"
      ".Lmx_no_load%=:"
      :
      : "v"(offset), "s"(b), "s"(lds), "s"(go)
      : "memory", "m0", "scc");
}

// the lane's number, counted where it is needed: no register holds it meanwhile
__device__ __forceinline__ int lane_again() {
  int l;
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
  return l;
}

// Tiles of 256 rows x 256 columns x 256: 8 waves (4 x 2) of 64 x 128, one workgroup per CU that stays for all
// its tiles, whose steps are one stream: while one of two LDS stages is multiplied, the other takes the next
// step's operands, of the next tile too. Operands go to LDS without registers, in whole 128-byte lines: in
// half lines (steps of 128) a step needed twice the requests, and the L1 held all eight waves up. The
// scales of four steps come together, 32 bytes a row, into two panels in turn.
//
// A step's 64 MFMAs a SIMD take 2410 cycles when nothing else is done (37.7 each; 1.7 to 1.8 GHz under this load).
// It takes 3320 to 3430 (16384 rows of 4096 -> 28672: 3.15 PFLOP/s; MFMAs alone reach 5.5 to 6.2): 360 are
// the scales' requests, 450 operands that are not in the XCD's L2, the rest the stores of other CUs' tiles. A tile's
// epilogue takes 10000 besides.
constexpr int kStreamM = 256, kStreamN = 256, kStreamK = 256;
constexpr int kStreamRows = kStreamM + kStreamN, kStreamStage = kStreamRows * 128, kStreamPanel = kStreamRows * 32;

__global__ __launch_bounds__(512, 2) void mx_stream_kernel(MxLinearArgs m) {
  constexpr int TM = 2, TN = 4, R = TM + TN, MN = TM * TN, kPanels = 2 * kStreamStage;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kPanels + 2 * kStreamPanel];
  const LinearArgs &g = m.lin;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1, r32 = lane & 31, h = lane >> 5;
  const uint32_t lds0 = uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t *)lds));
  const uint32_t kb = g.in / 2, sb = g.in / 32;
  const int steps = g.in / kStreamK;

  // this workgroup's tiles: every so-many-th of its XCD's share
  const int n_mt = __builtin_amdgcn_readfirstlane(tile_count(g, kStreamM)), n_nt = (g.out + kStreamN - 1) / kStreamN;
  const uint32_t W = uint32_t(n_mt) * uint32_t(n_nt), per = (W + 7) / 8, each = gridDim.x / 8;
  const uint32_t begin = (blockIdx.x % 8) * per, end = min(begin + per, W);
  uint32_t L = begin + blockIdx.x / 8;
  if (L >= end) return;
  struct Tile {
    int e, valid, nt;
    int64_t row0;
  };
  auto tile_of_L = [&](uint32_t l) {
    int mt, nt;
    tile_at(l, n_mt, n_nt, 1024 / kStreamM, mt, nt);
    if (!g.tile_map) return Tile{0, int(min(int64_t(kStreamM), g.rows - int64_t(mt) * kStreamM)), nt, int64_t(mt) * kStreamM};
    // (by the scalar cache: the entry is the same for all lanes, and an earlier launch wrote it)
    const auto *t = reinterpret_cast<const __attribute__((address_space(4))) int32_t *>(reinterpret_cast<uintptr_t>(g.tile_map)) +
                    mt * 4;
    return Tile{t[0], t[3], nt, int64_t(t[1]) + t[2]};
  };

  // What a lane fetches of a step: 16 bytes of four rows of x and of four weight rows, eight lanes a row; and of
  // four steps' scales 16 bytes of two rows, x's by waves 0 .. 3 and the weights' by the others. Piece p of a
  // row lies at p ^ row / 2 % 8 (scales: at p ^ row / 8 % 2), so that the sixteen lanes of a cycle meet all
  // banks; a lane's place is fixed, so that says which piece it asks for. Rows past the tile's last
  // repeat it (their results are not stored).
  const bool s_of_x = wave < 4;
  const int d_row = wave * 32 + (lane >> 3), s_row = (wave & 3) * 64 + (lane >> 1);
  struct Rows {  // of x, by tile
    uint32_t x[4], s[2];
  };
  auto rows_of = [&](const Tile &t) {
    Rows q;
    const auto x_row = [&](int r) -> uint32_t {
      r = min(r, t.valid - 1);
      return m.sorted ? uint32_t(source_row(m, t.row0 + r)) : uint32_t(r);
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) q.x[i] = x_row(d_row + 8 * i);
#pragma unroll
    for (int i = 0; i < 2; ++i) q.s[i] = s_of_x ? x_row(s_row + 32 * i) : 0;
    return q;
  };
  const auto word = [](uint32_t v) {  // as it stands here: products taken before the steps cost registers in all of them
    asm volatile("" : "+v"(v));
    return v;
  };
  buffer_t xb, wb, ssb;
  uint32_t xo[4], so[2];
  // (pieces 0 and 1 of `i`; the rows of i + 2 lie 16 further down)
  const auto piece_of = [&](int l, int i) { return uint32_t((l & 7) ^ ((l >> 4) + 4 * (i & 1))) * 16; };
  const uint32_t wo[2] = {d_row * kb + piece_of(lane, 0), (d_row + 8) * kb + piece_of(lane, 1)};
  // The weights' rows behind the expert's last one are the next expert's, and behind the stack's end zeros by the
  // buffer's size: no store takes their results.
  auto source_w = [&](const Tile &t) {
    const int64_t first = int64_t(t.e) * g.out + t.nt * kStreamN, left = (int64_t(g.E) * g.out - first) * kb;
    wb = sized_buffer(g.packed + first * kb, left);
  };
  auto source_x = [&](const Tile &t, const Rows &q) {  // and of the scales
    const int64_t skip = m.sorted ? 0 : t.row0, first = int64_t(t.e) * g.out + t.nt * kStreamN;
    xb = whole_buffer(m.x + skip * kb);
    ssb = s_of_x ? whole_buffer(m.xs + skip * sb) : sized_buffer(g.scales + first * sb, (int64_t(g.E) * g.out - first) * sb);
    const int l = lane_again();
#pragma unroll
    for (int i = 0; i < 4; ++i) xo[i] = word(__umul24(word(q.x[i]), kb) + piece_of(l, i));
#pragma unroll
    for (int i = 0; i < 2; ++i) so[i] = word(__umul24(word(s_of_x ? q.s[i] : (wave & 3) * 64 + (l >> 1) + 32 * i), sb));
  };

  Tile cur = tile_of_L(L), next = L + each < end ? tile_of_L(L + each) : cur;
  bool more = L + each < end;
  Rows ahead = rows_of(next);
  source_x(cur, rows_of(cur));
  source_w(cur);

  // load n of ten that ask for step ks of the tile that `source_x` and `source_w` were told: the scales of its four
  // steps (the last 16 bytes of a row where fewer are left) with the first of them, then x, then the weights
  int f_panel = 1;
  struct Fetch {
    int panel;
    uint32_t s_lds, step, lds;
  };
  auto fetch_of = [&](int ks, int stage) {
    const int panel = ((ks & 3) - 1) >> 31 & 1;  // (integers: a comparison would go by way of the lanes)
    f_panel ^= panel;
    return Fetch{panel,
                 lds0 + kPanels + f_panel * kStreamPanel + wave * 2048, uint32_t(ks) * 128,
                 lds0 + stage * kStreamStage + wave * 4096};
  };
  auto load_nth = [&](const Fetch &q, int n) {
    if (n < 2) {
      const int l = lane_again();
      load_to_lds_if(q.panel, ssb, so[n] + min(int(q.step / 16) + ((l ^ l >> 4) & 1) * 16, int(sb) - 16), q.s_lds + n * 1024);
    } else if (n < 6)
      load_to_lds(xb, xo[n - 2], q.step, q.lds + (n - 2) * 1024);
    else
      // (the whole offset in the lane's part, which is what the buffer's size is held against)
      load_to_lds(wb, wo[n & 1] + (q.step + (n - 6) / 2 * 16 * kb), 0, q.lds + kStreamM * 128 + (n - 6) * 1024);
  };

  // Fragment i of quarter t of the step: 0 .. TM - 1 the wave's rows of x, then its weight rows. Lane half h has
  // the 32 k of block 4 h + t, so that one word holds its four scales, byte t for quarter t (op_sel).
  // A lane's own part of the addresses (rows 32 further on lie alike):
  f32x16 acc[TM][TN];
  u32x4 f[2][R];
  uint32_t sc[R], sc_next[R];
  const int f_lane = r32 * 128 + (4 * h ^ (r32 >> 1 & 7)) * 16;
  const int x_first = wm * TM * 32, w_first = kStreamM + wn * TN * 32;
  auto frag = [&](int stage, int t, int i) {
    const int wave_at = stage * kStreamStage + (i < TM ? x_first : w_first) * 128;
    f[t & 1][i] = *reinterpret_cast<const u32x4 *>(lds + (wave_at + (f_lane ^ t * 16)) + (i < TM ? i : i - TM) * 4096);
  };
  int c_panel = 0;  // of the step whose scales were read last
  auto scales_at = [&](int ks) {
    const int q = ks >> 1 & 1;  // the 16 bytes of a row's 32 that hold the step's
    return (kPanels + c_panel * kStreamPanel + ks * 8 - min((ks & ~1) * 8, int(sb) - 16)) | q << 24;
  };
  int s_lane = 0;
  auto frag_scale = [&](int at, int i) {
    if (i == 0) {
      const int l = lane_again();
      s_lane = ((l & 31) * 32 + (l >> 3 & 1) * 16 + (l >> 5) * 4) ^ at >> 24 << 4;
    }
    const int wave_at = (at & 0xFFFFFF) + (i < TM ? x_first : w_first) * 32;
    sc_next[i] = *reinterpret_cast<const uint32_t *>(lds + (wave_at + s_lane) + (i < TM ? i : i - TM) * 1024);
  };
  constexpr auto nth = [](int q) { return q == 0 ? 0 : q <= TN ? TM + q - 1 : q - TN; };  // in the order of their use

  Fetch ask_w;  // the step whose weights are asked for next
  {
    const Fetch q = fetch_of(0, 0);
#pragma unroll
    for (int n = 0; n < 10; ++n) load_nth(q, n);
    wait_loads<0>();
    ask_w = fetch_of(1, 1);
#pragma unroll
    for (int n = 0; n < 6; ++n) load_nth(ask_w, n);
  }
  __syncthreads();
  int stage = 0;
  const bool simple = !g.act && !g.residual && !g.pre && !g.y_f32;  // (an epilogue without the branches: 9K cycles a tile, not 16K)

  for (;;) {
    // (read here and not by the tile before, whose epilogue needs the registers)
    {
      const int at = scales_at(0);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        frag_scale(at, i);
        frag(stage, 0, i);
      }
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;
    // the slots of a step: one MFMA each (two waves of a SIMD in turn, 64 cycles) and a fragment of the next
    // quarter. Behind slot 23 the one barrier: every wave has read its last fragment of this stage, and its loads
    // of the next step have landed. From there on the stage takes the step after the next one: scales and x in
    // slots 24 .. 31, the weights in the first slots of the next step.
#pragma unroll 1
    for (int ks = 0; ks < steps; ++ks) {
      const int n_ks = ks + 1 < steps ? ks + 1 : 0, n2_ks = n_ks + 1 < steps ? n_ks + 1 : 0;
      // (behind the last tile it is asked for again, and nobody reads it)
      if (more) {
        if (n2_ks == 0) source_x(next, ahead);
        if (n_ks == 0) source_w(next);
      }
      const Fetch ask_x = fetch_of(n2_ks, stage);
      c_panel ^= ((n_ks & 3) - 1) >> 31 & 1;
      const int s_at = scales_at(n_ks);
#pragma unroll
      for (int i = 0; i < R; ++i) sc[i] = sc_next[i];
      each_slot<4 * MN>([&](auto slot) {
        constexpr int s = decltype(slot)::value, t = s / MN, i = s % MN / TN, j = s % TN;
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(f[t & 1][TM + j]), operand(f[t & 1][i]), acc[i][j],
                                                                    MX_E2M1, MX_E2M1, t, sc[TM + j], t, sc[i]);
#pragma unroll
        for (int q = 0; q < R; ++q)
          if (s % MN == q) {
            if constexpr (t < 3) {
              frag(stage, t + 1, nth(q));
            } else {
              frag_scale(s_at, nth(q));
              frag(stage ^ 1, 0, nth(q));
            }
          }
#pragma unroll
        for (int n = 0; n < 10; ++n)
          if (s == (n < 2 ? 24 : n < 6 ? 21 + 2 * n : 2 * (n - 6))) load_nth(n < 6 ? ask_x : ask_w, n);
        if constexpr (s == 3 * MN - 1) {
          __builtin_amdgcn_sched_barrier(0);
          __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0), lgkmcnt(0)
          asm volatile("" ::: "memory");
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
        }
        __builtin_amdgcn_sched_barrier(0);
      });
      stage ^= 1;
      ask_w = ask_x;
    }

    // ---- epilogue, without LDS: 32 x 32 results at a time, lane (row r32, half h) with columns 8 q + 4 h .. of
    // group q; lanes swap until 16 rows have their 32 columns in one register's four lane groups ----
    const bool last = !more;
    const Tile was = cur;
    L += each;
    cur = next;
    more = L + each < end;
    if (more) next = tile_of_L(L + each);
    const int l = lane_again(), e_row = l & 15, e_col = (l & 16) + (l >> 5) * 8;
    const int64_t down = int64_t(16) * g.out;
    const auto col_of = [&](int part) { return was.nt * kStreamN + (wn * TN + part % TN) * 32 + e_col; };
    const auto row_of = [&](int part) { return (wm * TM + part / TN) * 32 + e_row; };
    // w[8 n ..]: columns e_col .. of row e_row + 16 n
    const auto arrange = [&](float(&w)[16]) {
      uint32_t v[16];
#pragma unroll
      for (int q = 0; q < 16; ++q) v[q] = __float_as_uint(w[q]);
      const auto swap32 = [&](int a, int b) {
        const auto t = __builtin_amdgcn_permlane32_swap(v[a], v[b], false, false);
        v[a] = t[0], v[b] = t[1];
      };
      const auto swap16 = [&](int a, int b) {
        const auto t = __builtin_amdgcn_permlane16_swap(v[a], v[b], false, false);
        v[a] = t[0], v[b] = t[1];
      };
#pragma unroll
      for (int q = 0; q < 4; ++q) swap32(q, 4 + q), swap32(8 + q, 12 + q);
#pragma unroll
      for (int q = 0; q < 8; ++q) swap16(q, 8 + q);
#pragma unroll
      for (int q = 0; q < 16; ++q) w[q] = __uint_as_float(v[q]);
    };
    if (simple) {
      float b[TN][8];
#pragma unroll
      for (int j = 0; j < TN; ++j) {
#pragma unroll
        for (int q = 0; q < 8; ++q) b[j][q] = 0.0f;
        if (g.bias && col_of(j) < g.out) load_row<8>(g.bias + int64_t(was.e) * g.out + col_of(j), b[j]);
      }
      bf16_t *y = static_cast<bf16_t *>(g.y) + (was.row0 + row_of(0)) * g.out + col_of(0);
      each_slot<MN / 2>([&](auto pair) {  // (two parts at a time: their 64 bytes of a row are one line)
        constexpr int i = decltype(pair)::value * 2 / TN, j0 = decltype(pair)::value * 2 % TN;
        float w[2][16];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
#pragma unroll
          for (int q = 0; q < 16; ++q) w[m][q] = acc[i][j0 + m][q];
          arrange(w[m]);
#pragma unroll
          for (int q = 0; q < 16; ++q) w[m][q] += b[j0 + m][q % 8];
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int m = 0; m < 2; ++m)
            if (col_of(j0 + m) < g.out && row_of(i * TN) + 16 * n < was.valid)
              store_row<8>(y + (2 * i + n) * down + (j0 + m) * 32, reinterpret_cast<float(&)[8]>(w[m][8 * n]));
        __builtin_amdgcn_sched_barrier(0);
      });
    } else {
      struct Extra {  // what a part reads
        float b[8];
        Raw<bf16_t, 8> res[2];
      } extra;
      auto fetch_extra = [&](int part) {
        const int col = col_of(part), r = row_of(part);
#pragma unroll
        for (int q = 0; q < 8; ++q) extra.b[q] = 0.0f;
        if (g.bias && col < g.out) load_row<8>(g.bias + int64_t(was.e) * g.out + col, extra.b);
        if (g.residual) {
          const bf16_t *from = reinterpret_cast<const bf16_t *>(g.residual) + (was.row0 + r) * g.out + col;
#pragma unroll
          for (int n = 0; n < 2; ++n) extra.res[n].fetch(from + n * down, col < g.out && r + 16 * n < was.valid);
        }
      };
      fetch_extra(0);
      // (one body for all parts: unrolled, the activations' code did not fit the instruction cache)
#pragma unroll 1
      for (int part = 0; part < MN; ++part) {
        float w[16];
        each_slot<MN>([&](auto n) {
          constexpr int i = decltype(n)::value / TN, j = decltype(n)::value % TN;
          if (part == decltype(n)::value) {
#pragma unroll
            for (int q = 0; q < 16; ++q) w[q] = acc[i][j][q];
          }
        });
        arrange(w);
#pragma unroll
        for (int q = 0; q < 16; ++q) w[q] += extra.b[q % 8];
        Raw<bf16_t, 8> res[2] = {extra.res[0], extra.res[1]};
        if (part + 1 < MN) fetch_extra(part + 1);
        const int col = col_of(part), r = row_of(part);
        const int64_t at = (was.row0 + r) * g.out + col;
        const bool in[2] = {col < g.out && r < was.valid, col < g.out && r + 16 < was.valid};
        if (g.pre) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
            if (in[n]) store_row<8>(g.pre + at + n * down, reinterpret_cast<float(&)[8]>(w[8 * n]));
        }
        act_values<16>(g.act, w);
        if (g.residual) {
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            float f[8];
            res[n].get(f);
#pragma unroll
            for (int q = 0; q < 8; ++q) w[8 * n + q] += f[q];
          }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          if (!in[n]) continue;
          if (g.y_f32)
            store_row<8>(static_cast<float *>(g.y) + at + n * down, reinterpret_cast<float(&)[8]>(w[8 * n]));
          else
            store_row<8>(static_cast<bf16_t *>(g.y) + at + n * down, reinterpret_cast<float(&)[8]>(w[8 * n]));
        }
      }
    }
    if (last) break;
    if (more) ahead = rows_of(next);  // (the rows of the tile behind the one whose steps come now)
  }
  wait_loads<0>();
}

hipError_t launch_stream(const MxLinearPlan &p, const MxLinearArgs &m, hipStream_t s) {
  const int64_t tiles = tiles_at_most(m.lin.E, p.rows, kStreamM) * ((m.lin.out + kStreamN - 1) / kStreamN);
  const int64_t grid = tiles < 256 ? (tiles + 7) / 8 * 8 : 256;
  hipLaunchKernelGGL(mx_stream_kernel, dim3(uint32_t(grid)), dim3(512), 0, s, m);
  return hipGetLastError();
}

template <int TM, int TN>
hipError_t launch_tiles(const MxLinearPlan &p, const MxLinearArgs &m, const int32_t *offsets, hipStream_t s) {
  using T = MxTile<TM, TN>;
  const LinearArgs &a = m.lin;
  int64_t tiles = tiles_at_most(a.E, p.rows, T::kM) * ((a.out + T::kN - 1) / T::kN);
  if (!offsets) tiles = (tiles + 7) / 8 * 8;
  const int64_t bytes = p.rows * a.out * ((a.y_f32 ? 4 : 2) + (a.pre ? 4 : 0));
  const dim3 grid(uint32_t(tiles + (offsets ? clear_groups(bytes, 1024) : 0))), block(256);
  if (a.in % 128)
    hipLaunchKernelGGL((mx_tile_kernel<TM, TN, true>), grid, block, 0, s, m, offsets, int32_t(tiles));
  else
    hipLaunchKernelGGL((mx_tile_kernel<TM, TN, false>), grid, block, 0, s, m, offsets, int32_t(tiles));
  return hipGetLastError();
}

}  // namespace
}  // namespace e4b

using namespace e4b;

extern "C" size_t e4b_mx_linear_workspace_bytes(const e4b_stack *st, int64_t rows) {
  MxLinearPlan p;
  return plan_mx_linear(st, rows, 1, false, E4B_ACT_NONE, E4B_BF16, &p) == E4B_OK ? p.ws_bytes : 0;
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
  if (!x_codes || !x_scales || !y || (p.ws_bytes && !ws)) return E4B_ERR_NULL;
  if (ws_bytes < p.ws_bytes) return E4B_ERR_WORKSPACE;
  if (!aligned16(offsets) || !aligned16(sorted_pair) || !aligned16(x_codes) || !aligned16(x_scales) ||
      !aligned16(bias) || !aligned16(residual_bf16) || !aligned16(y) || !aligned16(pre) || !aligned16(ws))
    return E4B_ERR_ALIGN;
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
  hipError_t err;
  if (p.tiles == MX_ROWS) {
    // (more than 16 rows an expert: only where x is too long for the tiles)
    err = rows <= 16 * st->E ? launch_rows_mt<1>(p, m, offsets, stream) : launch_rows_mt<4>(p, m, offsets, stream);
    return err == hipSuccess ? E4B_OK : E4B_ERR_HIP;
  }
  if (offsets && !p.by_offsets) {
    a.tile_offsets = reinterpret_cast<const int32_t *>(ws);
    a.tile_map = reinterpret_cast<const int4 *>(static_cast<char *>(ws) + p.off_tile_map);
    err = launch_tile_map(offsets, a.E, rows, mx_tile_rows(p.tiles), a, y, st->out * (a.y_f32 ? 4 : 2), pre, st->out * 4,
                          stream);
    if (err != hipSuccess) return E4B_ERR_HIP;
  }
  if (!p.by_offsets) offsets = nullptr;
  err = p.tiles == MX_256   ? launch_stream(p, m, stream)
        : p.tiles == MX_128 ? launch_tiles<2, 2>(p, m, offsets, stream)
                             : launch_tiles<1, 1>(p, m, offsets, stream);
  return err == hipSuccess ? E4B_OK : E4B_ERR_HIP;
}
