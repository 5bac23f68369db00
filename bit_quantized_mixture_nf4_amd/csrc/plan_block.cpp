// plan_block.cpp -- host-side checks of the operators around the experts (no HIP calls).
#include "plan_block.h"

namespace e4b {

e4b_status plan_order(int64_t T, int32_t top_k, int64_t E, int64_t H, int32_t dtype, OrderArgs *a) {
  if (T < 0 || top_k < 1 || top_k > kMaxTopK || E < 1 || E > kMaxE || H < 1 || H >= (int64_t(1) << 24))
    return E4B_ERR_SHAPE;
  if (T >= (int64_t(1) << 29) || T * top_k >= (int64_t(1) << 29)) return E4B_ERR_SHAPE;
  if (dtype != E4B_F32 && dtype != E4B_BF16) return E4B_ERR_DTYPE;
  a->T = T;
  a->k = top_k;
  a->E = int32_t(E);
  a->H = int32_t(H);
  a->f32 = dtype == E4B_F32;
  return E4B_OK;
}

e4b_status plan_norm(const e4b_norm *n, bool has_y, NormArgs *a) {
  if (!n) return E4B_ERR_NULL;
  if (n->T < 0 || n->H < 1 || n->H > kNormMaxH || n->T >= (int64_t(1) << 31)) return E4B_ERR_SHAPE;
  if (n->dtype != E4B_F32 && n->dtype != E4B_BF16) return E4B_ERR_DTYPE;
  // a mean square of zero has to have an inverse; the comparison also refuses NaN
  if (!(n->eps > 0.0f)) return E4B_ERR_SHAPE;
  if (n->gate_kind != E4B_GATE_NONE && n->gate_kind != E4B_GATE_TOKEN && n->gate_kind != E4B_GATE_CHANNEL)
    return E4B_ERR_SHAPE;
  if ((n->gate_kind != E4B_GATE_NONE) != (n->gate != nullptr)) return E4B_ERR_NULL;
  if (!has_y && (n->w_post || n->gate)) return E4B_ERR_NULL;  // they act on y
  if (!has_y && !n->w_pre) return E4B_ERR_NULL;               // nothing to compute
  if (!aligned16(n->w_post) || !aligned16(n->w_pre) || !aligned16(n->gate)) return E4B_ERR_ALIGN;
  a->T = n->T;
  a->H = int32_t(n->H);
  a->f32 = n->dtype == E4B_F32;
  a->eps = n->eps;
  a->scale = n->scale;
  a->w_post = n->w_post;
  a->w_pre = n->w_pre;
  a->gate_token = n->gate_kind == E4B_GATE_TOKEN ? n->gate : nullptr;
  a->gate_channel = n->gate_kind == E4B_GATE_CHANNEL ? n->gate : nullptr;
  // whole waves to a row, 8 elements to a thread where the workgroup can hold it so
  const int threads = norm_bwd_threads(n->H);
  a->tpr = 64;
  while (a->tpr < threads && a->tpr * 8 < n->H) a->tpr *= 2;
  const int64_t rows = threads / a->tpr, need = (n->T + rows - 1) / rows;
  // One workgroup per CU; two where their registers fit side by side and the column sums
  // stay small (bf16 without a channel gate). 4096 x 2048 bf16: 25.1 us with 256, 22.5 with
  // 512; 8191 x 4096 fp32 with a channel gate: 122.8 with 256, 128.5 with 512 (and 1.8 more
  // to add the partial rows).
  const int64_t most = !a->f32 && !a->gate_channel && n->H <= 4096 ? 512 : 256;
  a->groups = int32_t(need < most ? (need ? need : 1) : most);
  return E4B_OK;
}

e4b_status plan_linear(const e4b_stack *st, int64_t rows, int32_t act, int32_t dtype, LinearPlan *p) {
  *p = LinearPlan{};
  const e4b_status s = check_stack(st);
  if (s != E4B_OK) return s;
  if (st->E > kMaxE || rows < 0 || rows > (int64_t(1) << 30)) return E4B_ERR_SHAPE;
  if (act < E4B_ACT_NONE || act > E4B_ACT_GELU_TANH) return E4B_ERR_ACT;
  if (dtype != E4B_F32 && dtype != E4B_BF16) return E4B_ERR_DTYPE;
  p->rows = rows;
  // every expert may end in a partial tile
  p->m_bound = rows / kLinearM + (st->E < rows ? st->E : rows);
  p->ldz = (st->out + kBK - 1) / kBK * kBK;
  // the launch grids: one workgroup per tile, and column slabs in grid.y
  const int64_t wide = st->out > st->in ? st->out : st->in;
  if (p->m_bound * (wide / 128 + 1) >= (int64_t(1) << 30) || st->out > (int64_t(1) << 20)) return E4B_ERR_SHAPE;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = (off + bytes + 255) / 256 * 256;
    return o;
  };
  p->off_tile_offsets = take(size_t(st->E + 1) * 4);
  p->off_tile_map = take(size_t(p->m_bound) * 16);
  p->fwd_bytes = off;
  p->off_part = take(size_t(p->m_bound) * size_t(st->out) * 4);
  p->off_dz = take(size_t(rows) * size_t(p->ldz) * 2);
  p->bwd_bytes = off;
  p->off_pre = take(size_t(rows) * size_t(st->out) * 4);
  p->bwd_recompute_bytes = off;
  return E4B_OK;
}

e4b_status check_route(int64_t T, int64_t E, int32_t top_k) {
  if (T < 0 || E < 1 || E > kMaxE || top_k < 1 || top_k > kMaxTopK || top_k > E) return E4B_ERR_SHAPE;
  if (T >= (int64_t(1) << 29) || T * top_k >= (int64_t(1) << 29)) return E4B_ERR_SHAPE;
  return E4B_OK;
}

}  // namespace e4b
