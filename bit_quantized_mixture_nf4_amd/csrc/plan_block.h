// plan_block.h -- host-side checks and plans of the operators around the
// experts (routing, expert order, block norms, stored-weight products). Like
// plan.h, this makes no HIP call.
#pragma once

#include "plan.h"

namespace e4b {

// ---- expert order (order.hip) ----
struct OrderArgs {
  int64_t T;
  int32_t k, E, H, f32;
  const void *x;  // gather: tokens; the way back: expert rows
  const void *gy;
  void *rows;  // gather: expert rows; the way back: tokens (its gradient: expert rows)
  const int32_t *offsets, *pos;
  const float *w;
  float *gw;
  const int32_t *ids;  // the order's input and outputs
  int32_t *out_offsets, *out_sorted, *out_pos;
};
// 0 <= T < 2^24, 1 <= top_k <= 32, 1 <= E <= 1024, 1 <= H < 2^24.
e4b_status plan_order(int64_t T, int32_t top_k, int64_t E, int64_t H, int32_t dtype, OrderArgs *a);

// ---- block norms (norm.hip) ----
constexpr int kNormMaxH = 16384;  // a row is held by one workgroup's registers
// Threads of the backward's workgroups: 512 leave each thread the registers to hold
// its columns' weights and sums; beyond 4096 columns a row takes 1024.
inline int norm_bwd_threads(int64_t H) { return H <= 4096 ? 512 : 1024; }
struct NormArgs {
  int64_t T;
  int32_t H, f32;
  int32_t tpr, groups;  // the backward's threads per row, and its workgroups
  float eps, scale;
  const float *w_post, *w_pre, *gate_token, *gate_channel;
  const void *x, *y;
  void *r, *h;
  float *rstd_y, *rstd_r;
  const void *grad_r, *grad_h;
  void *grad_x, *grad_y;
  float *grad_gate, *grad_w_post, *grad_w_pre;
  float *part_pre, *part_post, *part_gate;  // [groups, H] each
};
// The descriptor's checks; groups = the backward's workgroups (one row of
// column sums each).
// (An empty batch has no y to show for its gate.)
e4b_status plan_norm(const e4b_norm *n, bool has_y, NormArgs *a);
inline size_t norm_ws_bytes(const NormArgs &a) {
  return a.groups > 1 ? size_t(a.groups) * size_t(a.H) * 3 * sizeof(float) : 0;  // one group writes its sums in place
}

// ---- stored-weight products (linear.hip) ----
constexpr int kLinearM = 128;  // rows per tile
// how a product is tiled: few rows, 128 x 128, 256 x 128, 256 x 256
enum { TILE_ROWS = 0, TILE_128, TILE_TALL, TILE_256 };
// row tiles of bm rows, at most: the last one of every expert with rows may be partial
inline int64_t tiles_at_most(int64_t E, int64_t rows, int64_t bm) {
  return (rows + (bm - 1) * (E < rows ? E : rows)) / bm;
}
struct LinearPlan {
  int fwd_tiles, bwd_tiles;    // of the product, and of its gradient
  int fwd_splits, bwd_splits;  // 128-row tiles: workgroups along k
  size_t off_split;            // their fp32 sums
  int64_t rows, m_bound;  // m_bound: row tiles of kLinearM rows, at most
  int64_t ldz;            // row length of dz: out in whole K-steps
  size_t off_tile_offsets, off_tile_map, off_dz, off_part, off_pre;
  size_t fwd_bytes, bwd_bytes, bwd_recompute_bytes;
};
struct LinearArgs {
  const uint16_t *A;  // bf16 rows
  int64_t lda;
  const uint8_t *packed, *scales;
  const float *absmax;
  int32_t E, out, in, cb;
  const int32_t *tile_offsets;
  const int4 *tile_map;
  const float *bias;         // [E, out] or null
  const uint16_t *residual;  // [rows, out] bf16 or null
  void *y;                   // [rows, out] bf16 / fp32; dgrad: grad_x [rows, in] bf16
  float *pre;                // [rows, out] or null
  int32_t act, y_f32;
  int32_t bm;  // rows per tile
  int64_t rows;
  int32_t splits;  // workgroups along k of one tile
  float *part;     // [splits, rows, out] (dgrad: in) or null
};
e4b_status plan_linear(const e4b_stack *st, int64_t rows, int32_t act, int32_t dtype, LinearPlan *p);

// ---- routing (route.hip) ----
e4b_status check_route(int64_t T, int64_t E, int32_t top_k);

}  // namespace e4b
