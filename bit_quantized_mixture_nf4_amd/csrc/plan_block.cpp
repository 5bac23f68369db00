// plan_block.cpp -- host-side checks of the operators around the experts (no HIP calls).
#include "plan_block.h"

namespace e4b {

// Tokens of one call: a launch dimension has less than 2^32 threads, and the kernels
// that give a token a workgroup give it 256 (the norms up to 512).
constexpr int64_t kMaxTokens = (int64_t(1) << 24) - 1, kMaxNormRows = (int64_t(1) << 23) - 1;

e4b_status plan_order(int64_t T, int32_t top_k, int64_t E, int64_t H, int32_t dtype, OrderArgs *a) {
  if (T < 0 || top_k < 1 || top_k > kMaxTopK || E < 1 || E > kMaxE || H < 1 || H >= (int64_t(1) << 24))
    return E4B_ERR_SHAPE;
  if (T > kMaxTokens) return E4B_ERR_SHAPE;
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
  if (n->T < 0 || n->H < 1 || n->H > kNormMaxH || n->T > kMaxNormRows) return E4B_ERR_SHAPE;
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
  // A few rows are one workgroup's, which then writes the column gradients itself: a
  // second launch costs more than its turns.
  if (need <= 4) a->groups = 1;
  return E4B_OK;
}

// Row tiles to expect of an even routing: one at least for every expert with rows, and
// for a quarter of them one more than their rows fill.
static int64_t row_tiles(const e4b_stack *st, int64_t rows, int64_t bm) {
  const int64_t busy = st->E < rows ? st->E : rows;
  if (busy <= 1) return (rows + bm - 1) / bm;
  const int64_t n = (rows + bm / 4 * busy + bm - 1) / bm;
  return n > busy ? n : busy;
}

// How a product is tiled: by the kernel for few rows, or in tiles of 128 x 128
// (cut along k where they are few), 256 x 128 or 256 x 256. In us on one MI355X, nf4
// unless said; few rows / 128 x 128 / 256 x 256:
//   few rows to an expert, up to 8 on average: 64 experts of 2048 -> 2048, 4 rows each
//     47 / 93 / 117, 8 each 48 / 93 / 117, 24 each 78 / 95 / 119; beyond 8 a skewed
//     routing gives one expert too many rows for a kernel that reads its weights again
//     for every 16
//   up to 2^29 products: 4096 -> 4096, 32 rows 14 / 19 / 92, 64 rows 27 / 21 / 94;
//     2048 -> 2048, 64 rows 15 / 14 / 53; 30000 rows of 128 -> 128 9 / 11 / 17 (a call takes
//     16 us with one expert and with two); 4096 rows
//     of 512 -> 512 18 / 13 / 24; 8- and 16-bit weights, which are two and four times the
//     bytes to read again, up to 2^28: bf16 4096 -> 4096, 16 rows 12.5 / 13 / 76, 32 rows
//     20 / 14 / 77
//   else the tiles that take the least time by the rounds that the chip needs for them:
//     a K-step of a round takes 0.82 us with one 128 x 128 tile on every CU, 1.5 with
//     two, 1.15 with a 256 x 128 tile and 1.9 with a 256 x 256 one, beside the 10 us or
//     so of a launch and its epilogue (2048 -> 4096 with GELU, 128 x 128 / 256 x 128 /
//     256 x 256: 1024 rows 37 / 46 / 65, 2048 rows 60 / 50 / 71, 4096 rows 112 / 95 / 86;
//     64 experts of 2048 -> 2048, 64 rows each 102 / 155 / 132, 128 each 153 / 159 / 140;
//     8 experts of 4096 -> 4096, 128 rows each 91 / 78 / 104, 256 each 140 / 137 / 116)
static int best_tiles(const e4b_stack *st, int64_t rows, int64_t cols, bool wide) {
  const int64_t low = row_tiles(st, rows, 128), tall = row_tiles(st, rows, 256);
  const int64_t narrow = (cols + 127) / 128, broad = (cols + 255) / 256;
  const int64_t n = low * narrow;
  const int64_t t128 = n <= 256 ? 82 : (n + 511) / 512 * 150, ttall = (tall * narrow + 255) / 256 * 115;
  const int64_t t256 = (tall * broad + 255) / 256 * 190;
  // 512 threads a workgroup: a launch dimension has fewer than 2^32 (many experts' partial
  // 256-row tiles can pass that where 128-row tiles of 256 threads still fit)
  const auto fits = [&](int64_t slabs) { return tiles_at_most(st->E, rows, 256) * slabs <= (int64_t(1) << 23) - 8; };
  // (the 256 x 256 tiles address their rows in 32 bits)
  const int64_t longest = (st->out > st->in ? st->out : st->in) + kBK;
  if (wide && rows * longest < (int64_t(1) << 32) && fits(broad) && t256 < t128 && t256 < ttall) return TILE_256;
  return ttall < t128 && fits(narrow) ? TILE_TALL : TILE_128;
}

static int forward_tiles(const e4b_stack *st, int64_t rows) {
  const bool four = st->codebook == E4B_CB_NF4 || st->codebook == E4B_CB_FP4 || st->codebook == E4B_CB_MXFP4;
  const int64_t most = int64_t(1) << (four ? 29 : 28);
  if ((st->E > 1 && rows <= 8 * st->E) || rows * st->out * st->in <= most) return TILE_ROWS;
  return best_tiles(st, rows, st->out, st->out % 8 == 0);
}

static int dgrad_tiles(const e4b_stack *st, int64_t rows) { return best_tiles(st, rows, st->in, st->out % kBK == 0); }

// Workgroups along k, where 128 x 128 tiles leave most of the chip idle: of the shares
// that still leave one workgroup per CU (512 in all took 40 us for 512 rows of nf4
// 4096 -> 4096, 256 take 38) the one with the least time, in us 0.68 a K-step, and for
// the sums that are written and joined 3 and one for every 2 MB of them. nf4
// 4096 -> 4096, 64 rows: 20 us with 8 shares, 31 with 2, 51 uncut; 512 rows of
// 2048 -> 2048: 22.7 with 4, 29 uncut; 4096 rows of 512 -> 512: 12.7 uncut, 21 with 2.
static int k_splits(const e4b_stack *st, int64_t rows, int64_t cols, int64_t k) {
  const int64_t tiles = row_tiles(st, rows, kLinearM) * ((cols + 127) / 128);
  const int64_t steps = (k + kBK - 1) / kBK;
  int best = 1;
  if (tiles == 0 || tiles > 128) return best;
  int64_t least = steps * 680;  // ns
  for (int s = 2; s <= 16 && s <= steps && s * tiles <= 256; ++s) {
    const int64_t t = (steps + s - 1) / s * 680 + 3000 + s * rows * cols * 2 / 1000;
    if (t < least) least = t, best = s;
  }
  return best;
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
  p->m_bound = tiles_at_most(st->E, rows, kLinearM);
  p->ldz = (st->out + kBK - 1) / kBK * kBK;
  // the launch grids: 256 threads per tile, and column slabs in grid.y
  const int64_t wide = st->out > st->in ? st->out : st->in;
  if (wide > (int64_t(1) << 20) || p->m_bound * (wide / 128 + 1) >= (int64_t(1) << 24) - 8) return E4B_ERR_SHAPE;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = (off + bytes + 255) / 256 * 256;
    return o;
  };
  p->fwd_tiles = forward_tiles(st, rows);
  p->bwd_tiles = dgrad_tiles(st, rows);
  p->fwd_splits = p->fwd_tiles == TILE_128 ? k_splits(st, rows, st->out, st->in) : 1;
  p->bwd_splits = p->bwd_tiles == TILE_128 ? k_splits(st, rows, st->in, st->out) : 1;
  p->off_tile_offsets = take(size_t(st->E + 1) * 4);
  p->off_tile_map = take(size_t(p->m_bound) * 16);
  p->off_split = off;
  const size_t fwd_split = p->fwd_splits > 1 ? size_t(p->fwd_splits) * size_t(rows) * size_t(st->out) * 4 : 0;
  const size_t bwd_split = p->bwd_splits > 1 ? size_t(p->bwd_splits) * size_t(rows) * size_t(st->in) * 4 : 0;
  // (the kernel for few rows reads the offsets itself)
  p->fwd_bytes = p->fwd_tiles == TILE_ROWS || rows == 0 ? 0 : (off + fwd_split + 255) / 256 * 256;
  // a recomputed forward is done with its sums before the gradient's begin
  take(bwd_split > fwd_split ? bwd_split : fwd_split);
  p->off_part = take(size_t(p->m_bound) * size_t(st->out) * 4);
  p->off_dz = take(size_t(rows) * size_t(p->ldz) * 2);
  p->bwd_bytes = off;
  p->off_pre = take(size_t(rows) * size_t(st->out) * 4);
  p->bwd_recompute_bytes = off;
  return E4B_OK;
}

e4b_status check_route(int64_t T, int64_t E, int32_t top_k) {
  if (T < 0 || E < 1 || E > kMaxE || top_k < 1 || top_k > kMaxTopK || top_k > E) return E4B_ERR_SHAPE;
  if (T > kMaxTokens) return E4B_ERR_SHAPE;
  return E4B_OK;
}

e4b_status plan_balance(const e4b_balance *b, BalanceArgs *a) {
  *a = BalanceArgs{};
  if (!b) return E4B_ERR_NULL;
  const e4b_status s = check_route(b->T, b->E, b->top_k);
  if (s != E4B_OK) return s;
  if (b->sequences < 1 || b->sequences > 65536) return E4B_ERR_SHAPE;
  if (!b->cu_tokens && b->sequences != 1) return E4B_ERR_NULL;
  if (!aligned16(b->cu_tokens) || !aligned16(b->token_mask)) return E4B_ERR_ALIGN;
  a->T = b->T;
  a->E = int32_t(b->E);
  a->k = b->top_k;
  a->S = int32_t(b->sequences);
  a->cu = b->cu_tokens;
  a->mask = b->token_mask;
  // a workgroup of 512 threads to a CU where there are tokens for them
  a->chunk = int32_t((b->T + 255) / 256 + 31) / 32 * 32;
  if (a->chunk < 32) a->chunk = 32;
  if (!a->cu && b->T <= kBalanceOne) a->chunk = int32_t(kBalanceOne);
  a->slots = b->T / a->chunk + a->S;
  return E4B_OK;
}

size_t balance_ws_bytes(const BalanceArgs &a) {
  if (a.T == 0 || (!a.cu && a.T <= kBalanceOne)) return 0;
  return ((size_t(a.slots) * size_t(a.E) * 8 + 255) / 256 + (size_t(a.slots) * 8 + 255) / 256) * 256;
}

e4b_status check_mx_rows(int64_t rows, int64_t K) {
  if (rows < 0 || rows > (int64_t(1) << 30) || K <= 0 || K % kBlock != 0 || K > (int64_t(1) << 20)) return E4B_ERR_SHAPE;
  // a launch dimension has fewer than 2^32 threads, one for 8 elements
  if (rows * K >= (int64_t(1) << 35) - 2048) return E4B_ERR_SHAPE;
  return E4B_OK;
}

// How a microscaled product is tiled: by the kernel for few rows, or in tiles of 64 x 64, 128 x 128 or
// 256 x 256. In us on one MI355X:
//   few rows / 64 / 128, one expert of 2048 -> 4096: 1 row 3.8 / 6.3 / 8.9, 16 rows 4.7 / 6.6 / 9.2, 48 rows
//     7.6 / 6.9 / 9.5; 8 experts of 768 -> 2048, 16 rows each 4.9 / 4.7 / 6.4; 8 of 4096 -> 4096, one row each
//     20.6 / 15.8 / 17.8: it wins where the larger tiles leave most CUs idle
//   64 / 128, 8 experts of 4096 -> 4096, rows each: 32 16.9 / 17.4, 64 18.7 / 18.4, 96 30.0 / 19.5; 64 experts of
//     1024 -> 2816: 32 27.9 / 28.5, 64 34.2 / 32.1; 256 rows of 2048 -> 4096: 7.6 / 10.0
//   128 / 256, 8 experts of 4096 -> 4096, rows each: 256 33.3 / 38.3, 512 59.9 / 44.4, 2048 225 / 146; 64
//     experts of 1024 -> 2816: 128 38.7 / 44.9, 192 54.7 / 49.0: a tile of 256 costs what three of 128 do
//     (2.8 to 3.2), and less than one a CU costs the same
static int mx_tiles(const e4b_stack *st, int64_t rows, int64_t tokens) {
  // (the tiles address gathered rows of x in 32 bits)
  if (tokens * (st->in / 2) >= (int64_t(1) << 32)) return MX_ROWS;
  const auto tiles = [&](int64_t bm) { return row_tiles(st, rows, bm) * ((st->out + bm - 1) / bm); };
  if (rows <= 16 * st->E && tiles(64) <= 128) return MX_ROWS;
  // (a launch dimension has fewer than 2^32 threads)
  const bool fits = tiles_at_most(st->E, rows, 64) * ((st->out + 63) / 64) < (int64_t(1) << 24) - 8;
  if (fits && (rows <= 48 * st->E || tiles(64) <= 512)) return MX_64;
  if (st->in % 256 != 0 || st->in < 512 || st->out % 8 != 0) return MX_128;
  const int64_t wide = tiles(256);
  return 3 * (wide > 224 ? wide : 224) < tiles(128) ? MX_256 : MX_128;
}

e4b_status plan_mx_linear(const e4b_stack *st, int64_t rows, int32_t top_k, bool gathered, int32_t act, int32_t dtype,
                          MxLinearPlan *p) {
  *p = MxLinearPlan{};
  // the refusals of the product with bf16 rows, for stacks of this format
  LinearPlan linear;
  const e4b_status s = plan_linear(st, rows, act, dtype, &linear);
  if (s != E4B_OK) return s;
  if (st->codebook != E4B_CB_MXFP4) return E4B_ERR_CODEBOOK;
  if (gathered && (top_k < 1 || top_k > kMaxTopK || rows % top_k != 0)) return E4B_ERR_SHAPE;
  p->rows = rows;
  p->tiles = mx_tiles(st, rows, gathered ? rows / top_k : 0);
  // Each workgroup finds its tile by itself where that is cheaper than a launch that maps them (3.4 us; 8 experts of
  // 4096 -> 4096, one row each: 15.8 us, with a map 19.2; 64 of 1024 -> 2816, 48 rows each 30.8 / 33.0, 96 each 35.3 / 36.5,
  // 192 each 59.5 / 54.7: the map knows how many there are).
  p->by_offsets = p->tiles != MX_256 && rows <= 4096 && st->E <= 512;
  // (rows in place and gathered ones agree about the map, but that the longest gathered ones have none)
  if (rows == 0 || p->tiles == MX_ROWS || p->by_offsets) return E4B_OK;
  p->off_tile_map = (size_t(st->E + 1) * 4 + 255) / 256 * 256;
  p->ws_bytes = p->off_tile_map + size_t(tiles_at_most(st->E, rows, mx_tile_rows(p->tiles))) * 16;
  return E4B_OK;
}

}  // namespace e4b
