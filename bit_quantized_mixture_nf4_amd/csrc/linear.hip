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
#include <utility>

#include "act.h"
#include "codebook8.h"
#include "gemm_dev.h"
#include "plan_block.h"
#include "rowvec.h"
#include "tiles_dev.h"

namespace e4b {

namespace {

// ---- the tile map ----

// Workgroup 0 lists the row tiles of every expert: tile_offsets[e] = first
// tile of e, map[t] = (e, first row of e, first row within e, rows). The
// others write zeros to the rows of up to two outputs that no expert has.
// Offsets are clamped to [0, rows] and to ascending order, so that no list of
// offsets leads out of a buffer.
constexpr int kMapThreads = 1024;

__global__ __launch_bounds__(kMapThreads) void tile_map_kernel(const int32_t *__restrict__ offsets, int E,
                                                               int32_t rows, int bm, int32_t *__restrict__ tile_offsets,
                                                               int4 *__restrict__ map, int64_t bound, char *zero_a,
                                                               int64_t row_bytes_a, char *zero_b, int64_t row_bytes_b) {
  if (blockIdx.x > 0) {
    const int64_t live = clamped_offset(offsets, E, E, rows);
    const int64_t i = int64_t(blockIdx.x - 1) * kMapThreads + threadIdx.x, n = int64_t(gridDim.x - 1) * kMapThreads;
    if (zero_a) clear_bytes(zero_a, live * row_bytes_a, rows * row_bytes_a, i, n);
    if (zero_b) clear_bytes(zero_b, live * row_bytes_b, rows * row_bytes_b, i, n);
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
// 4 columns of one row. 78 KB of LDS: two workgroups per CU.
// While K-step ks runs from one LDS stage, the other is filled for ks + 1. The
// wave's instruction stream is cut into 16 slots of one MFMA (32 cycles) and the
// share of that work that fits under it, each closed by a scheduling barrier:
//   slots 0..7   two pairs of codes (WM = 4: one) looked up (their LDS latency passes
//                under the next MFMA), slots 2..9 the pairs scaled and rounded, eight
//                weights stored one slot after their last (10 at the latest);
//   slots 7..10  the A rows stored, slots 8..11 those of ks + 2 asked for; slot 11
//                the weights of ks + 3 (two register sets by parity);
//   slots 0..11  the next k-slice's fragments, one per slot;
//   after 11     every wave has filled its share and read its last fragment: the
//                one barrier, and slots 12..15 read the next stage's first ones.
// In phases instead (fragments, MFMAs, decode, store; MFMA, VALU and LDS each busy
// 26 to 40 % of the time, in turn) nf4 2048 -> 4096 took 41 us for 1024 rows (one
// workgroup per CU) and 58 for 2048 (two); in slots 33 and 53. With two workgroups
// LDS bounds it: a K-step of one moves 64 KB of fragments, 32 KB of stores and 8192
// table entries, 2050 or more of its 128-byte cycles per pair against 1024 of MFMA.
// WM = 4 is the same wave tile in 256 rows x 128 columns, 8 waves, one workgroup per
// CU: a weight is decoded, stored and looked up once for 256 rows instead of 128
// (2048 rows of 2048 -> 4096 with GELU: 50 us, two 128 x 128 workgroups a CU 60). MFMA,
// VALU and LDS are busy 35, 36 and 42 % of the time then; a raised wave priority, the
// compiler's own order, rounding a slot later and fragments after the lookups all
// measured within 3 % of these slots.
constexpr int kTN = 128;
constexpr int kTBn = kTN + 32;  // row stride of the [k][n] weight tile (dgrad)
constexpr int kTOut = kTN + 4;  // row stride of the epilogue's fp32 tile
constexpr int kStageB = kBK * kTBn;  // elements of a stage
template <int WM>
struct Tile {
  static constexpr int kM = 64 * WM, kThreads = 128 * WM, kW = 64 / WM;  // rows, threads, weights a thread
  static constexpr int kStageA = kM * kLds;
  static constexpr int kStages = 2 * (kStageA + kStageB), kOut = kM * kTOut * 2;  // elements of 2 bytes
  static constexpr int kElems = kStages > kOut ? kStages : kOut;
  static_assert(kTN * kLds <= kStageB, "either form of the weight tile fits its stage");
};

// How a weight reaches bf16: the W codes of one thread's piece, and their scale.
enum { LK_ABSMAX = 0, LK_MX = 1, LK_BF16 = 2, LK_CODE8 = 3 };

template <int SK, int W = 32>
struct Piece {
  static constexpr int kWords = SK == LK_BF16 ? W / 2 : SK == LK_CODE8 ? W / 4 : W / 8;
  uint32_t w[kWords];
  float s;
};

// table entries of pair c of a piece (not for bf16)
template <int SK, int W>
__device__ __forceinline__ void lookup_pair(const Piece<SK, W> &p, const float *code, int c, float &a, float &b) {
  if constexpr (SK == LK_CODE8) {
    const uint32_t w = p.w[c >> 1] >> (16 * (c & 1));
    a = code[w & 255];
    b = code[(w >> 8) & 255];
  } else {
    // the byte offsets 4 code of a word's high (even) and low (odd) nibbles, a byte each;
    // one byte permute then makes an address
    const char *tbl = reinterpret_cast<const char *>(code);
    const uint32_t w = p.w[c >> 2], hi = (w >> 2) & 0x3C3C3C3Cu, lo = (w << 2) & 0x3C3C3C3Cu;
    const uint32_t sel = 0x0C0C0C00u | uint32_t(c & 3);
    a = *reinterpret_cast<const float *>(tbl + __builtin_amdgcn_perm(0u, hi, sel));
    b = *reinterpret_cast<const float *>(tbl + __builtin_amdgcn_perm(0u, lo, sel));
  }
}

// a piece as packed bf16, 8 weights to a vector
template <int SK, int W>
__device__ __forceinline__ void decode_piece(const Piece<SK, W> &p, const float *code, u32x4 (&o)[W / 8]) {
#pragma unroll
  for (int q = 0; q < W / 8; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (SK == LK_BF16) {
        o[q][i] = p.w[4 * q + i];
      } else {
        float a, b;
        lookup_pair<SK, W>(p, code, 4 * q + i, a, b);
        o[q][i] = pack_bf16x2(__fmul_rn(a, p.s), __fmul_rn(b, p.s));
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

// f(std::integral_constant<int, s>) for the 16 slots of a K-step
template <typename F, int... I>
__device__ __forceinline__ void slots_of(F &&f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <typename F>
__device__ __forceinline__ void slots(F &&f) {
  slots_of(f, std::make_integer_sequence<int, 16>{});
}

// bytes of n stored weights
template <int SK>
__device__ __forceinline__ int64_t code_bytes(int64_t n) {
  return SK == LK_BF16 ? n * 2 : SK == LK_CODE8 ? n : n / 2;
}

// the W consecutive weights from column c of stored row `row`
template <int SK, int W>
__device__ __forceinline__ void load_piece(const LinearArgs &g, int64_t e, int64_t row, int c, Piece<SK, W> &p) {
  const int64_t at = (e * g.out + row) * g.in + c;
  const uint8_t *src = g.packed + code_bytes<SK>(at);
  constexpr int kN = Piece<SK, W>::kWords;
  if constexpr (kN >= 4) {
#pragma unroll
    for (int q = 0; q < kN / 4; ++q) {
      const u32x4 v = reinterpret_cast<const u32x4 *>(src)[q];
#pragma unroll
      for (int i = 0; i < 4; ++i) p.w[4 * q + i] = v[i];
    }
  } else {
    const u32x2 v = *reinterpret_cast<const u32x2 *>(src);
    p.w[0] = v[0];
    p.w[1] = v[1];
  }
  p.s = SK == LK_MX ? e8m0_value(g.scales[at >> 5]) : SK == LK_BF16 ? 1.0f : g.absmax[at >> 6];
}

// NN = false: C[row, n] = sum_k A[row, k] W[n, k] with the epilogue;
// NN = true:  C[row, n] = sum_k A[row, k] W[k, n], stored as bf16.
// A product of few tiles is cut along k as well: with g.part, workgroup (tile, s)
// adds up its share of the K-steps and leaves fp32 sums in part[s], which
// linear_join_kernel adds in order.
template <int SK, bool NN, int WM>
__global__ __launch_bounds__(Tile<WM>::kThreads, WM == 2 ? 2 : 1) void linear_tile_kernel(LinearArgs g) {
  constexpr int kM = Tile<WM>::kM, kThreads = Tile<WM>::kThreads, kStageA = Tile<WM>::kStageA, kW = Tile<WM>::kW;
  __shared__ __attribute__((aligned(64))) float code[SK == LK_CODE8 ? 256 : 16];
  __shared__ __attribute__((aligned(16))) uint16_t lds[Tile<WM>::kElems];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;

  const int N = NN ? g.in : g.out;
  int mt, nt, share;
  if (!place_of(tile_count(g, kM), (N + kTN - 1) / kTN, g.splits, 16 / WM, mt, nt, share)) return;
  const int4 tm = tile_of(g, mt, kM);
  const int64_t e = tm.x, row0 = int64_t(tm.y) + tm.z;
  const int valid = tm.w;

  fill_codes<SK>(code, g.cb);

  // A: 16-byte chunk tid & 7 of rows (tid >> 3) + kM / 4 i; rows past the tile's
  // last repeat it (their results are not stored)
  const uint16_t *a_src[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    a_src[i] = g.A + (row0 + min((tid >> 3) + kM / 4 * i, valid - 1)) * g.lda + (tid & 7) * 8;
  // B: kW weights. !NN: part b_p of weight row (tile column) b_r; NN: columns kW b_p ..
  // of weight row (K-step's) b_r
  const int b_r = NN ? tid / (kTN / kW) : tid / (kBK / kW), b_p = NN ? tid % (kTN / kW) : tid % (kBK / kW);
  const int b_n = nt * kTN + b_r;
  const int64_t b_row = b_n < N ? b_n : 0;
  const int b_c = nt * kTN + b_p * kW < N ? nt * kTN + b_p * kW : 0;
  const int all = NN ? (g.out + kBK - 1) / kBK : g.in / kBK;  // K-steps, and this workgroup's
  const int first = all * share / g.splits, nK = all * (share + 1) / g.splits;

  u32x4 ra[4];      // A rows of the next K-step
  Piece<SK, kW> rb[2];  // weights of the next two, by the K-step's parity
  auto load_a = [&](int ks, int i) { ra[i] = *reinterpret_cast<const u32x4 *>(a_src[i] + ks * kBK); };
  auto load_b = [&](int ks, Piece<SK, kW> &p) {
    if (!NN)
      load_piece<SK, kW>(g, e, b_row, ks * kBK + b_p * kW, p);
    else  // weight rows past the last meet zeros of A
      load_piece<SK, kW>(g, e, min(ks * kBK + b_r, g.out - 1), b_c, p);
  };
  auto store_a = [&](int st, int i) {
    *reinterpret_cast<u32x4 *>(lds + st * kStageA + ((tid >> 3) + kM / 4 * i) * kLds + (tid & 7) * 8) = ra[i];
  };
  auto store_b = [&](int st, int q, const u32x4 &o) {
    uint16_t *sB = lds + 2 * kStageA + st * kStageB;
    if (!NN)
      *reinterpret_cast<u32x4 *>(sB + b_r * kLds + b_p * kW + q * 8) = o;
    else
      *reinterpret_cast<u32x4 *>(sB + b_r * kTBn + nn_unit(kW / 8 * b_p + q) * 8) = o;
  };
  // pair c of the piece: two table entries, then their packed bf16
  float cv[kW];
  uint32_t bq[kW / 2];
  auto lookup = [&](const Piece<SK, kW> &p, int c) {
    if constexpr (SK != LK_BF16) lookup_pair<SK, kW>(p, code, c, cv[2 * c], cv[2 * c + 1]);
  };
  auto scale = [&](const Piece<SK, kW> &p, int c) {
    bq[c] = SK == LK_BF16 ? p.w[SK == LK_BF16 ? c : 0]
                          : pack_bf16x2(__fmul_rn(cv[2 * c], p.s), __fmul_rn(cv[2 * c + 1], p.s));
  };
  auto quarter = [&](int q) { return u32x4{bq[4 * q], bq[4 * q + 1], bq[4 * q + 2], bq[4 * q + 3]}; };
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
  // fragment f of k-slice kk of stage st: 0, 1 the columns', 2, 3 the rows'
  bf16x8 af[2][2], bf[2][2];
  auto frag = [&](int st, int kk, int f) {
    const uint16_t *sA = lds + st * kStageA, *sB = lds + 2 * kStageA + st * kStageB;
    if (f >= 2) {
      af[kk & 1][f - 2] = *reinterpret_cast<const bf16x8 *>(sA + (wm * 64 + (f - 2) * 32 + (lane & 31)) * kLds +
                                                            (lane >> 5) * 8 + kk * 16);
    } else if (!NN) {
      bf[kk & 1][f] = *reinterpret_cast<const bf16x8 *>(sB + (wn * 64 + f * 32 + (lane & 31)) * kLds + (lane >> 5) * 8 +
                                                        kk * 16);
    } else {
      const uint16_t *p = sB + q_off[f] + kk * 16 * kTBn;
      const s16x4 lo = lds_read_tr16(p), hi = lds_read_tr16(p + 4 * kTBn);
      bf[kk & 1][f] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  };

  // the first stage; loads past the last K-step repeat it
  const int last = nK - 1;
  load_b(first, rb[0]);
#pragma unroll
  for (int i = 0; i < 4; ++i) load_a(first, i);
  load_b(min(first + 1, last), rb[1]);
  __syncthreads();  // the code table
#pragma unroll
  for (int c = 0; c < kW / 2; ++c) {
    lookup(rb[0], c);
    scale(rb[0], c);
  }
#pragma unroll
  for (int q = 0; q < kW / 8; ++q) store_b(0, q, quarter(q));
#pragma unroll
  for (int i = 0; i < 4; ++i) store_a(0, i);
#pragma unroll
  for (int i = 0; i < 4; ++i) load_a(min(first + 1, last), i);
  load_b(min(first + 2, last), rb[0]);
  __syncthreads();
#pragma unroll
  for (int f = 0; f < 4; ++f) frag(0, 0, f);

  auto kstep = [&](auto cur_c, int ks) {
    constexpr int CUR = decltype(cur_c)::value, NXT = CUR ^ 1;
    const int ka = min(ks + 2, last), kb = min(ks + 3, last);
    Piece<SK, kW> &b = rb[NXT];      // the weights of ks + 1
    constexpr int kL = kW / 16;      // pairs per slot
    slots([&](auto sc) {
      constexpr int s = decltype(sc)::value, kk = s >> 2, w = s & 3;
      acc[w >> 1][w & 1] =
          __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf[kk & 1][w & 1], af[kk & 1][w >> 1], acc[w >> 1][w & 1], 0, 0, 0);
      // in the order in which the next k-slice uses them
      if constexpr (kk < 3) frag(CUR, kk + 1, w == 0 ? 0 : w == 1 ? 2 : w == 2 ? 1 : 3);
#pragma unroll
      for (int c = 0; c < kL; ++c) {
        if constexpr (s < 8) lookup(b, kL * s + c);
        if constexpr (s >= 2 && s < 10) scale(b, kL * (s - 2) + c);
      }
      // 8 weights once their last pair is scaled
#pragma unroll
      for (int q = 0; q < kW / 8; ++q)
        if (s == (4 * q + 3) / kL + 3) store_b(NXT, q, quarter(q));
      if constexpr (s >= 7 && s < 11) store_a(NXT, s - 7);
      if constexpr (s >= 8 && s < 12) load_a(ka, s - 8);
      if constexpr (s == 11) {
        load_b(kb, b);
        __builtin_amdgcn_sched_barrier(0);
        __syncthreads();
      }
      if constexpr (s >= 12) frag(NXT, 0, w == 0 ? 0 : w == 1 ? 2 : w == 2 ? 1 : 3);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  int ks = first;
  for (; ks + 1 < nK; ks += 2) {
    kstep(std::integral_constant<int, 0>{}, ks);
    kstep(std::integral_constant<int, 1>{}, ks + 1);
  }
  if (ks < nK) kstep(std::integral_constant<int, 0>{}, ks);
  __syncthreads();  // the last stage's fragments are read

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
  if (g.part) {
    float *out = g.part + int64_t(share) * g.rows * N;
    const int cc = (tid & 31) * 4, col = nt * kTN + cc;
    for (int r = tid >> 5; r < valid; r += kThreads / 32) {
      const f32x4 v = *reinterpret_cast<const f32x4 *>(tile + r * kTOut + cc);
      float *o = out + (row0 + r) * N + col;
      if (N % 4 == 0) {
        if (col < N) *reinterpret_cast<f32x4 *>(o) = v;
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (col + q < N) o[q] = v[q];
      }
    }
    return;
  }
  if (NN) {
    const int cc = (tid & 15) * 8, col = nt * kTN + cc;
    if (col < N)  // N is a multiple of 64
      for (int r = tid >> 4; r < valid; r += kThreads / 16) {
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
    for (int r = tid / kCols; r < valid; r += kThreads / kCols) {
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

// The sums of a product's splits, in order, and its epilogue. One workgroup per
// 8 rows of a row tile and 32 VEC columns.
template <bool NN, int VEC>
__global__ __launch_bounds__(256) void linear_join_kernel(LinearArgs g) {
  constexpr int kGroups = kLinearM / 8;
  if (int(blockIdx.x / kGroups) >= tile_count(g, kLinearM)) return;
  const int4 tm = tile_of(g, blockIdx.x / kGroups, kLinearM);
  const int64_t row0 = int64_t(tm.y) + tm.z, N = NN ? g.in : g.out;
  const int r = blockIdx.x % kGroups * 8 + (threadIdx.x >> 5);
  const int64_t col = int64_t(blockIdx.y) * 32 * VEC + (threadIdx.x & 31) * VEC;
  if (col >= N || r >= tm.w) return;
  const int64_t at = (row0 + r) * N + col;
  float b[VEC], v[VEC];
#pragma unroll
  for (int q = 0; q < VEC; ++q) b[q] = v[q] = 0.0f;
  if (!NN && g.bias) load_row<VEC>(g.bias + int64_t(tm.x) * N + col, b);
#pragma unroll 8
  for (int s = 0; s < g.splits; ++s) {
    float u[VEC];
    load_row<VEC>(g.part + int64_t(s) * g.rows * N + at, u);
#pragma unroll
    for (int q = 0; q < VEC; ++q) v[q] += u[q];
  }
  if constexpr (NN)
    store_row<VEC>(static_cast<bf16_t *>(g.y) + at, v);
  else
    linear_epilogue<VEC>(g, at, b, v);
}

// ---- few rows to an expert ----

// A decode step's experts have a row or two each, so the touched weights are the
// whole cost and each is read once: no row tile is worth filling, and there is
// no time for a tile map. Workgroup (column group, n-th block of 16 MT rows) finds
// its expert and rows straight from the offsets. Blocks are counted over every
// expert, so that a routing that sends most rows to one spreads over the chip as well:
// 100000 rows of 64 -> 64 on one of 4 experts take 22 us a call, 19 with that expert
// alone (a fixed 4 row slices to an expert took 1200). One MFMA 16x16x32
// takes 16 weight rows (the A operand: a lane's D registers are 4 consecutive
// columns of one row) and 16 of the expert's rows. A lane reads 16 bytes of
// codes = 32 consecutive k of its weight row, the operands of four MFMAs; the
// order of k inside the 128 of a step is the same for x, so the weights go from
// HBM to the MFMA through registers alone, kRowDepth steps in flight per wave.
// x waits in LDS (kRowK / MT columns of it at a time); rows past the expert's
// last are not filled, since each only reaches its own results. The 8 waves lie
// along the columns (8 / wk) and along k (wk slices, joined through LDS in
// order).
constexpr int kRowThreads = 512;
constexpr int kRowStep = 128;  // k per step
constexpr int kRowK = 2048;    // k of x in LDS for 16 rows
constexpr int kRowDepth = 4;
// 16 waves per CU: each workgroup's start (offsets, x, the first weights) costs
// about 4 us, so more slices than the chip needs are slower (64 rows on 40 of
// 128 experts, nf4 2048 -> 1536: 28 us with 1 slice, 33 with 2, 43 with 4; 8 rows
// of bf16 2048 -> 128: 20.4 us with 1 slice, 6.5 with 8)
constexpr int64_t kRowWaves = 4096;

template <int SK, int MT>
__global__ __launch_bounds__(kRowThreads) void linear_rows_kernel(LinearArgs g, const int32_t *__restrict__ offsets,
                                                                  int32_t rows, int wk, int32_t blocks,
                                                                  int32_t zeros) {
  constexpr int kRows = 16 * MT, kK = kRowK / MT, kLd = kK + 8;
  __shared__ __attribute__((aligned(64))) float code[SK == LK_CODE8 ? 256 : 16];
  __shared__ __attribute__((aligned(16))) uint16_t sx[16 * MT * kLd];
  static_assert(8 * MT * 64 * 16 <= sizeof(sx), "the slices' sums fit x's place");
  const int tid = threadIdx.x, lane = tid & 63;
  // uniform over the wave, so that the loops below branch on scalars
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
    if (g.y) clear_bytes(static_cast<char *>(g.y), from * y_bytes, to * y_bytes, i, n);
    return;
  }
  int e;
  int32_t r0, hi;
  if (!block_of(offsets, g.E, rows, kRows, block, lane, e, r0, hi)) return;

  const int col0 = (blockIdx.x * wn + wave / wk) * 16;  // the wave's columns
  const int m = lane & 15, grp = lane >> 4;
  const int64_t w_row = min(col0 + m, g.out - 1);
  Piece<SK> f[kRowDepth];
  // the wave's steps of the chunk at k0: k0 + (slice + i wk) 128; in is a
  // multiple of 64, so the last step may be half
  auto load = [&](int k0, int i, Piece<SK> &p) {
    const int k = k0 + (slice + i * wk) * kRowStep + grp * 32;
    load_piece<SK>(g, e, w_row, k < g.in ? k : 0, p);
  };
  fill_codes<SK>(code, g.cb);
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int n_rows = min(kRows, hi - r0);
  for (int k0 = 0; k0 < g.in; k0 += kK) {
    const int len = min(kK, g.in - k0);
    const int all = (len + kRowStep - 1) / kRowStep;       // steps of the chunk
    const int mine = (all - slice + wk - 1) / wk;          // this slice's
#pragma unroll
    for (int d = 0; d < kRowDepth; ++d)
      if (d < mine) load(k0, d, f[d]);
    __syncthreads();  // the last chunk's x has been read
    // a half step's second half meets zeros
    const int per_row = all * (kRowStep / 8);
    for (int i = tid; i < n_rows * per_row; i += kRowThreads) {
      const int r = i / per_row, c = (i - r * per_row) * 8;
      u32x4 v = u32x4{0u, 0u, 0u, 0u};
      if (c < len) v = *reinterpret_cast<const u32x4 *>(g.A + int64_t(r0 + r) * g.in + k0 + c);
      *reinterpret_cast<u32x4 *>(sx + r * kLd + c) = v;
    }
    // the pieces came in before x: nothing is in flight, which the compiler
    // cannot know, and without it the loop would wait for its youngest load
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    __syncthreads();
    auto step = [&](int i, const u32x4 (&w)[4]) {
      const uint16_t *xs = sx + m * kLd + (slice + i * wk) * kRowStep + grp * 32;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int q = 0; q < MT; ++q)
          acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, w[j]), *reinterpret_cast<const bf16x8 *>(xs + q * 16 * kLd + 8 * j), acc[q],
              0, 0, 0);
    };
    // whole runs of kRowDepth steps without a branch (past the end the loads
    // repeat the last step), then what is left, which is in the registers
    int i = 0;
    for (; i + kRowDepth <= mine; i += kRowDepth)
#pragma unroll
      for (int d = 0; d < kRowDepth; ++d) {
        u32x4 w[4];
        decode_piece<SK>(f[d], code, w);
        load(k0, min(i + d + kRowDepth, mine - 1), f[d]);
        step(i + d, w);
      }
#pragma unroll
    for (int d = 0; d < kRowDepth - 1; ++d)
      if (i + d < mine) {
        u32x4 w[4];
        decode_piece<SK>(f[d], code, w);
        step(i + d, w);
      }
  }
  if (wk > 1) {
    float(*part)[MT][64 * 4] = reinterpret_cast<float(*)[MT][64 * 4]>(sx);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MT; ++i) *reinterpret_cast<f32x4 *>(&part[wave][i][lane * 4]) = acc[i];
    __syncthreads();
    if (slice == 0)
      for (int q = 1; q < wk; ++q)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[i] += *reinterpret_cast<const f32x4 *>(&part[wave + q][i][lane * 4]);
  }
  if (slice == 0) {
    const int c = col0 + 4 * grp;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int32_t r = r0 + i * 16 + m;
      if (r >= hi) continue;
      if (g.out % 4 == 0) {
        if (c < g.out) {
          float b[4] = {}, v[4] = {acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
          if (g.bias) load_row<4>(g.bias + int64_t(e) * g.out + c, b);
          linear_epilogue<4>(g, int64_t(r) * g.out + c, b, v);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (c + q < g.out) {
            float b[1] = {g.bias ? g.bias[int64_t(e) * g.out + c + q] : 0.0f}, v[1] = {acc[i][q]};
            linear_epilogue<1>(g, int64_t(r) * g.out + c + q, b, v);
          }
      }
    }
  }
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
  if (int(blockIdx.x) >= tile_count(g, g.bm)) return;
  const int4 tm = tile_of(g, blockIdx.x, g.bm);
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
        act_grads<VEC>(g.act, z, v);
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
  const int t0 = g.tile_map ? g.tile_offsets[e] : 0, t1 = g.tile_map ? g.tile_offsets[e + 1] : tile_count(g, g.bm);
  float v = 0.0f;
#pragma unroll 8
  for (int t = t0; t < t1; ++t) v += part[int64_t(t) * g.out + c];
  gb[int64_t(e) * g.out + c] = v;
}

__global__ __launch_bounds__(256) void fill_zero_kernel(float *p, int64_t n) {
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) p[i] = 0.0f;
}

template <bool NN, int WM>
hipError_t launch_tiles(LinearArgs a, const LinearPlan &p, int splits, char *ws, hipStream_t s) {
  const int64_t N = NN ? a.in : a.out, tiles = tiles_at_most(a.E, p.rows, Tile<WM>::kM) * ((N + kTN - 1) / kTN);
  const dim3 grid(uint32_t((tiles * splits + 7) / 8 * 8)), block(Tile<WM>::kThreads);
  a.splits = splits;
  a.part = splits > 1 ? reinterpret_cast<float *>(ws + p.off_split) : nullptr;
  switch (a.cb) {
    case E4B_CB_BF16: hipLaunchKernelGGL((linear_tile_kernel<LK_BF16, NN, WM>), grid, block, 0, s, a); break;
    case E4B_CB_MXFP4: hipLaunchKernelGGL((linear_tile_kernel<LK_MX, NN, WM>), grid, block, 0, s, a); break;
    case E4B_CB_INT8:
    case E4B_CB_FP8: hipLaunchKernelGGL((linear_tile_kernel<LK_CODE8, NN, WM>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((linear_tile_kernel<LK_ABSMAX, NN, WM>), grid, block, 0, s, a); break;
  }
  if (splits > 1) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const bool vec = N % 8 == 0;
    const int cols = vec ? 256 : 32;
    hipLaunchKernelGGL((vec ? linear_join_kernel<NN, 8> : linear_join_kernel<NN, 1>),
                       dim3(uint32_t(p.m_bound * (kLinearM / 8)), uint32_t((N + cols - 1) / cols)), dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

template <int MT>
hipError_t launch_rows_mt(const LinearPlan &p, const LinearArgs &a, const int32_t *offsets, hipStream_t s) {
  // enough waves to fill the chip from the experts that can have rows, and a step of k for each slice
  const int64_t busy = a.E < p.rows ? a.E : p.rows, groups = (a.out + 15) / 16;
  const int64_t steps = (a.in < kRowK / MT ? a.in : kRowK / MT) / kRowStep;
  int wk = 1;
  while (wk < 8 && 2 * wk <= steps && busy * groups * wk < kRowWaves) wk *= 2;
  const int64_t slabs = (groups + 8 / wk - 1) / (8 / wk);
  // blocks of 16 MT rows, at most, and slab rows of workgroups that clear the rows of no expert
  const int64_t blocks = tiles_at_most(a.E, p.rows, 16 * MT);
  const int64_t bytes = p.rows * a.out * ((a.y ? (a.y_f32 ? 4 : 2) : 0) + (a.pre ? 4 : 0));
  const int64_t zeros = offsets ? (clear_groups(bytes, 1024) + slabs - 1) / slabs : 0;
  const int64_t y = blocks + zeros < 32768 ? blocks + zeros : 32768;
  const dim3 grid(uint32_t(slabs), uint32_t(y), uint32_t((blocks + zeros + y - 1) / y));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(kRowThreads), 0, s, a, offsets, int32_t(p.rows), wk, int32_t(blocks),
                       int32_t(zeros));
  };
  switch (a.cb) {
    case E4B_CB_BF16: go(linear_rows_kernel<LK_BF16, MT>); break;
    case E4B_CB_MXFP4: go(linear_rows_kernel<LK_MX, MT>); break;
    case E4B_CB_INT8:
    case E4B_CB_FP8: go(linear_rows_kernel<LK_CODE8, MT>); break;
    default: go(linear_rows_kernel<LK_ABSMAX, MT>); break;
  }
  return hipGetLastError();
}

hipError_t launch_rows(const LinearPlan &p, const LinearArgs &a, const int32_t *offsets, hipStream_t s) {
  const int64_t mean = (p.rows + a.E - 1) / a.E;
  return mean <= 16 ? launch_rows_mt<1>(p, a, offsets, s)
                    : mean <= 32 ? launch_rows_mt<2>(p, a, offsets, s) : launch_rows_mt<4>(p, a, offsets, s);
}

// The 256 x 256 tiles of the routed MLP's GEMM (gemm_wide.hip) for this product.
GemmArgs wide_args(const LinearPlan &p, const LinearArgs &a, bool nn) {
  GemmArgs w{};
  w.A = a.A;
  w.lda = int32_t(a.lda);
  w.topk = 1;
  w.Wp = a.packed;
  w.mx = a.cb == E4B_CB_MXFP4;
  w.Wa = w.mx ? nullptr : a.absmax;
  w.Ws = w.mx ? a.scales : nullptr;
  const int64_t n = int64_t(a.out) * a.in;
  w.w_e_bytes = a.cb == E4B_CB_BF16 ? n * 2 : a.cb == E4B_CB_INT8 || a.cb == E4B_CB_FP8 ? n : n / 2;
  w.w_e_blocks = a.cb == E4B_CB_BF16 ? 0 : n / (w.mx ? kMxBlock : kBlock);
  w.w_in = a.in;
  w.N = nn ? a.in : a.out;
  w.K = nn ? a.out : a.in;
  w.I = w.N;
  w.tile_offsets = a.tile_offsets;
  w.tile_map = a.tile_map;
  w.E = a.E;
  w.cb = a.cb;
  w.n_tiles = (w.N + kBNWide - 1) / kBNWide;
  w.grid = uint32_t(tiles_at_most(a.E, p.rows, kBM) * w.n_tiles);
  w.lin = a;
  if (nn) {
    w.C = static_cast<uint16_t *>(a.y);
    w.ldc = a.in;
  }
  return w;
}

hipError_t launch_forward(const LinearPlan &p, const LinearArgs &a, const int32_t *offsets, char *ws, hipStream_t s) {
  if (p.fwd_tiles == TILE_ROWS) return launch_rows(p, a, offsets, s);
  if (p.fwd_tiles == TILE_128) return launch_tiles<false, 2>(a, p, p.fwd_splits, ws, s);
  if (p.fwd_tiles == TILE_TALL) return launch_tiles<false, 4>(a, p, 1, ws, s);
  return launch_grouped_gemm(GEMM_LINEAR, wide_args(p, a, false), s);
}

}  // namespace

hipError_t launch_tile_map(const int32_t *offsets, int E, int64_t rows, int bm, const LinearArgs &a, void *zero_a,
                           int64_t bytes_a, void *zero_b, int64_t bytes_b, hipStream_t s) {
  // without offsets every row belongs to an expert: nothing to clear
  const int64_t bytes = rows * ((zero_a ? bytes_a : 0) + (zero_b ? bytes_b : 0));
  const uint32_t grid = 1 + uint32_t(offsets ? clear_groups(bytes, 256) : 0);
  hipLaunchKernelGGL(tile_map_kernel, dim3(grid), dim3(kMapThreads), 0, s, offsets, E, int32_t(rows), bm,
                     const_cast<int32_t *>(a.tile_offsets), const_cast<int4 *>(a.tile_map), tiles_at_most(E, rows, bm),
                     static_cast<char *>(zero_a), bytes_a, static_cast<char *>(zero_b), bytes_b);
  return hipGetLastError();
}

namespace {

// Makes the map for a kind of tiles where they need one, in `a`'s place for it.
hipError_t launch_map(const LinearPlan &p, LinearArgs &a, const int4 *place, const int32_t *offsets, int tiles,
                      void *zero_a, int64_t bytes_a, void *zero_b, int64_t bytes_b, hipStream_t s) {
  const int bm = a.bm = tiles == TILE_128 ? kLinearM : kBM;
  a.tile_map = offsets || tiles == TILE_256 ? place : nullptr;
  if (!a.tile_map) return hipSuccess;
  return launch_tile_map(offsets, a.E, p.rows, bm, a, zero_a, bytes_a, zero_b, bytes_b, s);
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
  a.rows = p.rows;
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
  if (!x_bf16 || !y || (p.fwd_bytes && !ws)) return E4B_ERR_NULL;
  if (ws_bytes < p.fwd_bytes) return E4B_ERR_WORKSPACE;
  if (!aligned16(offsets) || !aligned16(x_bf16) || !aligned16(bias) || !aligned16(residual_bf16) || !aligned16(y) ||
      !aligned16(pre) || !aligned16(ws))
    return E4B_ERR_ALIGN;
  char *w = static_cast<char *>(ws);
  LinearArgs a = args_of(p, st, w);
  a.A = static_cast<const uint16_t *>(x_bf16);
  a.lda = st->in;
  a.bias = bias;
  a.act = act;
  a.residual = static_cast<const uint16_t *>(residual_bf16);
  a.y = y;
  a.y_f32 = y_dtype == E4B_F32;
  a.pre = pre;
  if (p.fwd_tiles != TILE_ROWS)
    E4B_TRY(launch_map(p, a, reinterpret_cast<const int4 *>(w + p.off_tile_map), offsets, p.fwd_tiles, y,
                       st->out * (a.y_f32 ? 4 : 2), pre, st->out * 4, stream));
  E4B_TRY(launch_forward(p, a, offsets, w, stream));
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
  const int tiles = p.bwd_tiles;
  const int4 *place = reinterpret_cast<const int4 *>(w + p.off_tile_map);
  if (recompute) {
    // exactly the forward's pre-activation, in the forward's tiles
    LinearArgs f = a;
    f.A = static_cast<const uint16_t *>(x_bf16);
    f.lda = st->in;
    f.bias = bias;
    f.pre = reinterpret_cast<float *>(w + p.off_pre);
    if (p.fwd_tiles != TILE_ROWS) E4B_TRY(launch_map(p, f, place, offsets, p.fwd_tiles, nullptr, 0, nullptr, 0, stream));
    E4B_TRY(launch_forward(p, f, offsets, w, stream));
    pre = f.pre;
  }
  E4B_TRY(launch_map(p, a, place, offsets, tiles, grad_x_bf16, st->in * 2, nullptr, 0, stream));
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
  if (tiles == TILE_256)
    E4B_TRY(launch_grouped_gemm(GEMM_GATE_UP_DGRAD, wide_args(p, a, true), stream));
  else if (tiles == TILE_TALL)
    E4B_TRY((launch_tiles<true, 4>(a, p, 1, w, stream)));
  else
    E4B_TRY((launch_tiles<true, 2>(a, p, p.bwd_splits, w, stream)));
  return E4B_OK;
}
