// order.hip -- tokens into expert order and back, for callers that run the
// experts' products themselves: rows[pos(t, j)] = x[t], and
// y[t] = sum_j w[t, j] rows[pos(t, j)], with both gradients.
//
// The order is the stable counting sort of the routed pairs p = t k + j by
// expert id: pos(p) = #{q : key_q < key_p} + #{q < p : key_q = key_p}, where
// key is the id, or E for an id outside [0, E) (a pair that goes to no expert
// here). Everything below is a copy or a k-term sum, so memory bounds it: the
// floor is (T + P) rows moved. Sums run in slot order in fp32; no atomics
// touch a result.
#include "plan_block.h"
#include "kernels.h"
#include "rowvec.h"

namespace e4b {

namespace {

constexpr int kOrderThreads = 1024;
constexpr int kOrderIt = 32;                          // ids per lane and pass
constexpr int kOrderPass = kOrderThreads * kOrderIt;  // 32768 pairs per pass
constexpr int kOrderSmall = 4096;                     // pairs that one launch orders and copies
constexpr int kGatherThreads = 256;
constexpr int kNarrow = 16;  // threads to a token whose row has no more pieces
template <int KU>
constexpr int kUnpermutePieces = KU == 2 ? 2 : 1;

// The bucket of an id: itself, or E for one outside [0, E).
__device__ __forceinline__ uint32_t bucket(int32_t id, int E) { return min(uint32_t(id), uint32_t(E)); }

// One workgroup per bucket e (the experts, then the bucket of dropped pairs).
// It reads every id: lower buckets give this one's first position, equal ones
// the ranks. A wave takes runs of 64 consecutive pairs, so the compare's lane
// mask is the rank information: position = base + masks' population before it.
// E + 1 readings of 4 P bytes come from L2 and stay far below the rows' own
// traffic (P = 32768, E = 64: 8.5 MB against 151 MB).
__global__ __launch_bounds__(kOrderThreads) void order_kernel(const int32_t *__restrict__ ids, int32_t P, int E,
                                                              int32_t *__restrict__ offsets,
                                                              int32_t *__restrict__ sorted,
                                                              int32_t *__restrict__ pos) {
  __shared__ int32_t s_less[kOrderThreads / 64], s_eq[kOrderThreads / 64];
  const uint32_t e = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint64_t below = (1ull << lane) - 1;
  uint32_t b[kOrderIt];  // the lane's buckets of one pass; past the end, one that nothing matches
  auto fetch = [&](int32_t p0) {
    const int32_t w0 = p0 + wave * (64 * kOrderIt) + lane;
    // (clamped rather than guarded: the loads stay together, ahead of their first use)
#pragma unroll
    for (int i = 0; i < kOrderIt; ++i) b[i] = uint32_t(ids[min(w0 + i * 64, P - 1)]);
#pragma unroll
    for (int i = 0; i < kOrderIt; ++i) b[i] = w0 + i * 64 < P ? bucket(int32_t(b[i]), E) : 0xFFFFFFFFu;
  };
  int32_t less = 0, eq = 0;
  for (int32_t p0 = 0; p0 < P; p0 += kOrderPass) {
    fetch(p0);
#pragma unroll
    for (int i = 0; i < kOrderIt; ++i) less += b[i] < e ? 1 : 0;
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) less += __shfl_xor(less, o);
  if (lane == 0) s_less[wave] = less;
  int32_t before = 0;  // pairs of the bucket in earlier passes
  for (int32_t p0 = 0; p0 < P; p0 += kOrderPass) {
    if (P > kOrderPass) fetch(p0);
    eq = 0;
#pragma unroll
    for (int i = 0; i < kOrderIt; ++i) eq += __popcll(__ballot(b[i] == e));
    __syncthreads();
    if (lane == 0) s_eq[wave] = eq;
    __syncthreads();
    int32_t at = before;
    for (int w = 0; w < kOrderThreads / 64; ++w) {
      at += s_less[w] + (w < wave ? s_eq[w] : 0);
      before += s_eq[w];
    }
    const int32_t w0 = p0 + wave * (64 * kOrderIt) + lane;
#pragma unroll
    for (int i = 0; i < kOrderIt; ++i) {
      const uint64_t m = __ballot(b[i] == e);
      if (b[i] == e) {
        const int32_t s = at + __popcll(m & below);
        sorted[s] = w0 + i * 64;
        pos[w0 + i * 64] = s;
      }
      at += __popcll(m);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int32_t first = 0;
    for (int w = 0; w < kOrderThreads / 64; ++w) first += s_less[w];
    offsets[e] = first;
  }
}

// The piece of token t's row that this thread copies goes to each of the
// token's k places; dropped pairs (places from offsets[E] on) get zeros.
template <typename T, int VEC>
__device__ __forceinline__ void copy_row(const T *__restrict__ x, int64_t t, int k, int H, const int32_t *s_pos,
                                         int32_t live, T *__restrict__ rows) {
  for (int h = threadIdx.x * VEC; h < H; h += kGatherThreads * VEC) {
    float f[VEC], zero[VEC];
    load_row<VEC>(x + t * H + h, f);
#pragma unroll
    for (int q = 0; q < VEC; ++q) zero[q] = 0.0f;
    for (int j = 0; j < k; ++j) {
      const int32_t s = s_pos[j];
      if (s < live)
        store_row<VEC>(rows + int64_t(s) * H + h, f);
      else
        store_row<VEC>(rows + int64_t(s) * H + h, zero);
    }
  }
}

// One workgroup per token: its row is read once and written k times.
template <typename T, int VEC>
__global__ __launch_bounds__(kGatherThreads) void gather_kernel(const T *__restrict__ x, int k, int H, int E,
                                                                const int32_t *__restrict__ offsets,
                                                                const int32_t *__restrict__ pos,
                                                                T *__restrict__ rows) {
  __shared__ int32_t s_pos[kMaxTopK];
  const int64_t t = blockIdx.x;
  if (threadIdx.x < k) s_pos[threadIdx.x] = pos[t * k + threadIdx.x];
  __syncthreads();
  copy_row<T, VEC>(x, t, k, H, s_pos, offsets[E], rows);
}

// Few pairs: one launch instead of two. The workgroup of token t counts its
// pairs' places from all the ids, which it holds in LDS (a wave per slot: 64
// compares and one population count per 64 ids), then copies its row; the
// workgroup behind the tokens' writes the offsets. 8 tokens of 128 experts:
// 4.6 us against 9.3 + 2.9 in two launches.
template <typename T, int VEC>
__global__ __launch_bounds__(kGatherThreads) void order_gather_kernel(const int32_t *__restrict__ ids, int32_t n_tok,
                                                                      const T *__restrict__ x, int k, int H, int E,
                                                                      int32_t *__restrict__ offsets,
                                                                      int32_t *__restrict__ sorted,
                                                                      int32_t *__restrict__ pos, T *__restrict__ rows) {
  __shared__ uint16_t s_b[kOrderSmall];
  __shared__ int32_t s_pos[kMaxTopK];
  __shared__ int32_t s_n[kMaxE + 1];
  const int P = n_tok * k, t = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < P; i += kGatherThreads) s_b[i] = uint16_t(bucket(ids[i], E));
  if (t == n_tok) {
    for (int e = threadIdx.x; e <= E; e += kGatherThreads) s_n[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < P; i += kGatherThreads) atomicAdd(&s_n[s_b[i]], 1);
    __syncthreads();
    if (wave == 0) {
      // pairs of lower buckets, 64 buckets at a time
      int32_t carry = 0;
      for (int e0 = 0; e0 <= E; e0 += 64) {
        const int e = e0 + lane;
        const int32_t v = e <= E ? s_n[e] : 0;
        int32_t incl = v;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
          const int32_t u = __shfl_up(incl, o);
          if (lane >= o) incl += u;
        }
        if (e <= E) offsets[e] = carry + incl - v;
        carry += __shfl(incl, 63);
      }
    }
    return;
  }
  __syncthreads();
  for (int j = wave; j < k; j += kGatherThreads / 64) {
    const int p = t * k + j;
    const uint32_t b = s_b[p];
    int32_t s = 0;
    for (int q0 = 0; q0 < P; q0 += 64) {
      const int q = q0 + lane;
      const uint32_t c = q < P ? s_b[q] : 0xFFFFFFFFu;
      s += __popcll(__ballot(c < b || (c == b && q < p)));
    }
    if (lane == 0) {
      s_pos[j] = b == uint32_t(E) ? ~s : s;  // (complement: a dropped pair)
      sorted[s] = p;
      pos[p] = s;
    }
  }
  if (!rows) return;
  __syncthreads();
  for (int h = threadIdx.x * VEC; h < H; h += kGatherThreads * VEC) {
    float f[VEC], zero[VEC];
    load_row<VEC>(x + int64_t(t) * H + h, f);
#pragma unroll
    for (int q = 0; q < VEC; ++q) zero[q] = 0.0f;
    for (int j = 0; j < k; ++j) {
      const int32_t s = s_pos[j];
      if (s >= 0)
        store_row<VEC>(rows + int64_t(s) * H + h, f);
      else
        store_row<VEC>(rows + int64_t(~s) * H + h, zero);
    }
  }
}

// y[t] = sum_j w[t, j] rows[pos(t, j)], in slot order (no weights: the plain
// sum, which is the gradient of the copies). One workgroup per token and
// slab of columns, so that its places and weights are scalars and a row's
// neighbouring pieces are read together: a wave per token, or per token and 1
// KB of its row, was slower (8192 x 2 x 4096 bf16: 57 us). KU slots and CU
// pieces are in flight at a time. Rows of 16 pieces or fewer leave a workgroup almost
// empty: TPT = 16 threads take a token then (48482 tokens of 27 x 3 fp32: 26 us, 211
// with a workgroup each).
template <typename T, int VEC, int KU, int TPT>
__global__ __launch_bounds__(kGatherThreads) void unpermute_kernel(const T *__restrict__ rows, int64_t n_tok, int k,
                                                                   int H, int E, const int32_t *__restrict__ offsets,
                                                                   const int32_t *__restrict__ pos,
                                                                   const float *__restrict__ w, T *__restrict__ y) {
  constexpr int CU = TPT == kGatherThreads ? kUnpermutePieces<KU> : 1;
  constexpr int kPiece = TPT * VEC;
  const int64_t t = TPT == kGatherThreads ? int64_t(blockIdx.x)
                                          : int64_t(blockIdx.x) * (kGatherThreads / TPT) + threadIdx.x / TPT;
  if (TPT < kGatherThreads && t >= n_tok) return;
  const int32_t live = int32_t(min(int64_t(offsets[E]), n_tok * k));  // no place leads out of the rows
  const int h0 = blockIdx.y * CU * kPiece + threadIdx.x % TPT * VEC;
  float acc[CU][VEC];
#pragma unroll
  for (int c = 0; c < CU; ++c)
#pragma unroll
    for (int q = 0; q < VEC; ++q) acc[c][q] = 0.0f;
  for (int j0 = 0; j0 < k; j0 += KU) {
    Raw<T, VEC> v[KU][CU];
    float wj[KU];
#pragma unroll
    for (int j = 0; j < KU; ++j) {
      const int32_t s = j0 + j < k ? pos[t * k + j0 + j] : -1;
      const bool in = s >= 0 && s < live;
      wj[j] = w && j0 + j < k ? w[t * k + j0 + j] : 1.0f;
      if (!in) wj[j] = 0.0f;  // (its piece is zeros, whatever the row holds)
#pragma unroll
      for (int c = 0; c < CU; ++c) v[j][c].fetch(rows + int64_t(s) * H + h0 + c * kPiece, in && h0 + c * kPiece < H);
    }
#pragma unroll
    for (int j = 0; j < KU; ++j)
#pragma unroll
      for (int c = 0; c < CU; ++c) {
        float f[VEC];
        v[j][c].get(f);
#pragma unroll
        for (int q = 0; q < VEC; ++q) acc[c][q] += wj[j] * f[q];
      }
  }
#pragma unroll
  for (int c = 0; c < CU; ++c)
    if (h0 + c * kPiece < H) store_row<VEC>(y + t * H + h0 + c * kPiece, acc[c]);
}

// The gradients: a wave per token, so that nothing waits at a barrier for the dots
// (8192 x 2 x 4096 bf16: 65 us; 78 with a workgroup per token).
// grad_rows[pos(t, j)] = w[t, j] grad_y[t] and grad_w[t, j] = rows[pos(t, j)] . grad_y[t];
// grad_y's row is read once per KU slots, each pair's row once. Fewer than 4096 tokens:
// a wave to each KU of a token's slots (its `groups`), fewer still: to every slot with 8
// pieces in flight, since a wave's own turns bound it then (17 tokens of 17 x 2337 fp32
// 107 us with a wave per token, 11 so; 1 of 32 x 16383 1200 and 25; 4096 tokens of
// 16 x 2048 read grad_y twice so, 60 against 50). Lanes sum their columns in
// ascending order, the sums meet in a fixed tree; LPT = 16 lanes take a token where its
// row has no more pieces (the tree's first two levels would add zeros).
template <typename T, int VEC, int KU, int CU, int LPT>
__global__ __launch_bounds__(kGatherThreads) void unpermute_bwd_kernel(
    const T *__restrict__ rows, const T *__restrict__ gy, int64_t n_tok, int k, int H, int E,
    const int32_t *__restrict__ offsets, const int32_t *__restrict__ pos, const float *__restrict__ w,
    T *__restrict__ grows, float *__restrict__ gw, uint32_t groups) {
  const int lane = threadIdx.x % LPT;
  const uint32_t item = LPT == 64 ? blockIdx.x * (kGatherThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)
                                  : blockIdx.x * (kGatherThreads / LPT) + threadIdx.x / LPT;
  const int64_t t = item / groups;
  if (t >= n_tok) return;
  const int32_t live = offsets[E];
  const int64_t P = n_tok * k;
  for (int j0 = int(item % groups) * KU; j0 < k; j0 += int(groups) * KU) {
    int32_t s[KU];
    float wj[KU], dot[KU];
#pragma unroll
    for (int j = 0; j < KU; ++j) {
      s[j] = j0 + j < k ? pos[t * k + j0 + j] : -1;
      if (s[j] >= P) s[j] = -1;
      // a pair without an expert: zeros in its row, no weight gradient
      wj[j] = s[j] >= live ? 0.0f : w && j0 + j < k ? w[t * k + j0 + j] : 1.0f;
      dot[j] = 0.0f;
    }
    for (int h0 = lane * VEC; h0 < H; h0 += CU * LPT * VEC) {
      float g[CU][VEC], v[KU][CU][VEC];
#pragma unroll
      for (int c = 0; c < CU; ++c) {
        const int h = h0 + c * LPT * VEC;
        if (h < H) load_row<VEC>(gy + t * H + h, g[c]);
      }
      if (gw)
#pragma unroll
        for (int j = 0; j < KU; ++j)
          if (s[j] >= 0 && s[j] < live)
#pragma unroll
            for (int c = 0; c < CU; ++c) {
              const int h = h0 + c * LPT * VEC;
              if (h < H) load_row<VEC>(rows + int64_t(s[j]) * H + h, v[j][c]);
            }
#pragma unroll
      for (int j = 0; j < KU; ++j) {
        if (s[j] < 0) continue;
#pragma unroll
        for (int c = 0; c < CU; ++c) {
          const int h = h0 + c * LPT * VEC;
          if (h >= H) continue;
          float o[VEC];
#pragma unroll
          for (int q = 0; q < VEC; ++q) o[q] = s[j] < live ? wj[j] * g[c][q] : 0.0f;
          store_row<VEC>(grows + int64_t(s[j]) * H + h, o);
          if (gw && s[j] < live)
#pragma unroll
            for (int q = 0; q < VEC; ++q) dot[j] += v[j][c][q] * g[c][q];
        }
      }
    }
    if (gw)
#pragma unroll
      for (int j = 0; j < KU; ++j) {
        const float d = lanes_sum<LPT>(dot[j]);
        if (lane == 0 && j0 + j < k) gw[t * k + j0 + j] = d;
      }
  }
}

template <typename T, int VEC>
hipError_t gather(const OrderArgs &a, hipStream_t s) {
  hipLaunchKernelGGL((gather_kernel<T, VEC>), dim3(uint32_t(a.T)), dim3(kGatherThreads), 0, s,
                     static_cast<const T *>(a.x), a.k, a.H, a.E, a.offsets, a.pos, static_cast<T *>(a.rows));
  return hipGetLastError();
}
template <typename T, int VEC>
hipError_t order_gather(const OrderArgs &a, hipStream_t s) {
  hipLaunchKernelGGL((order_gather_kernel<T, VEC>), dim3(uint32_t(a.T + 1)), dim3(kGatherThreads), 0, s, a.ids,
                     int32_t(a.T), static_cast<const T *>(a.x), a.k, a.H, a.E, a.out_offsets, a.out_sorted, a.out_pos,
                     static_cast<T *>(a.rows));
  return hipGetLastError();
}
template <typename T, int VEC>
hipError_t unpermute(const OrderArgs &a, hipStream_t s) {
  const bool narrow = a.H <= kNarrow * VEC;  // a token's row in kNarrow threads
  const int piece = kGatherThreads * VEC * (a.k <= 2 ? kUnpermutePieces<2> : 1), per = kGatherThreads / kNarrow;
  const dim3 grid = narrow ? dim3(uint32_t((a.T + per - 1) / per)) : dim3(uint32_t(a.T), uint32_t((a.H + piece - 1) / piece));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(kGatherThreads), 0, s, static_cast<const T *>(a.x), a.T, a.k, a.H, a.E,
                       a.offsets, a.pos, a.w, static_cast<T *>(a.rows));
  };
  if (narrow)
    go(unpermute_kernel<T, VEC, 8, kNarrow>);
  else if (a.k <= 2)
    go(unpermute_kernel<T, VEC, 2, kGatherThreads>);
  else if (a.k <= 4)
    go(unpermute_kernel<T, VEC, 4, kGatherThreads>);
  else
    go(unpermute_kernel<T, VEC, 8, kGatherThreads>);
  return hipGetLastError();
}
template <typename T, int VEC>
hipError_t unpermute_bwd(const OrderArgs &a, hipStream_t s) {
  auto go = [&](auto kernel, int ku, int lanes) {
    const int64_t groups = a.T < 4096 ? (a.k + ku - 1) / ku : 1, items = a.T * groups, per = kGatherThreads / lanes;
    hipLaunchKernelGGL(kernel, dim3(uint32_t((items + per - 1) / per)), dim3(kGatherThreads), 0, s,
                       static_cast<const T *>(a.x), static_cast<const T *>(a.gy), a.T, a.k, a.H, a.E, a.offsets, a.pos,
                       a.w, static_cast<T *>(a.rows), a.gw, uint32_t(groups));
  };
  if (a.H <= kNarrow * VEC)
    go(unpermute_bwd_kernel<T, VEC, 8, 1, kNarrow>, 8, kNarrow);
  else if (a.T * ((a.k + 7) / 8) < 1024)  // fewer waves than SIMDs
    go(unpermute_bwd_kernel<T, VEC, 1, 8, 64>, 1, 64);
  else if (a.k <= 2)
    go(unpermute_bwd_kernel<T, VEC, 2, 2, 64>, 2, 64);
  else if (a.k <= 4)
    go(unpermute_bwd_kernel<T, VEC, 4, 2, 64>, 4, 64);
  else
    go(unpermute_bwd_kernel<T, VEC, 8, 1, 64>, 8, 64);
  return hipGetLastError();
}

#define E4B_ROWS(F, a, s)                                                                 \
  (a.f32 ? (a.H % 8 ? F<float, 1>(a, s) : F<float, 8>(a, s))                              \
         : (a.H % 8 ? F<bf16_t, 1>(a, s) : F<bf16_t, 8>(a, s)))

}  // namespace

hipError_t launch_order(const OrderArgs &a, hipStream_t s) {
  hipLaunchKernelGGL(order_kernel, dim3(uint32_t(a.E + 1)), dim3(kOrderThreads), 0, s, a.ids, int32_t(a.T * a.k), a.E,
                     a.out_offsets, a.out_sorted, a.out_pos);
  return hipGetLastError();
}
hipError_t launch_order_gather(const OrderArgs &a, hipStream_t s) { return E4B_ROWS(order_gather, a, s); }
hipError_t launch_gather(const OrderArgs &a, hipStream_t s) { return E4B_ROWS(gather, a, s); }
hipError_t launch_unpermute(const OrderArgs &a, hipStream_t s) { return E4B_ROWS(unpermute, a, s); }
hipError_t launch_unpermute_bwd(const OrderArgs &a, hipStream_t s) { return E4B_ROWS(unpermute_bwd, a, s); }

}  // namespace e4b

using namespace e4b;

#define E4B_TRY(expr)                             \
  do {                                            \
    if ((expr) != hipSuccess) return E4B_ERR_HIP; \
  } while (0)

extern "C" e4b_status e4b_permute(int64_t T, int32_t top_k, int64_t E, int64_t H, int32_t dtype,
                                  const int32_t *topk_idx, const void *x, void *rows, int32_t *offsets,
                                  int32_t *sorted_pair, int32_t *pos_of_pair, hipStream_t stream) {
  OrderArgs a{};
  e4b_status st = plan_order(T, top_k, E, H, dtype, &a);
  if (st != E4B_OK) return st;
  // T = 0 still writes the (all zero) offsets
  if (!offsets || (T && (!topk_idx || !sorted_pair || !pos_of_pair))) return E4B_ERR_NULL;
  if (T && (!x) != (!rows)) return E4B_ERR_NULL;
  if (!aligned16(offsets) || !aligned16(topk_idx) || !aligned16(sorted_pair) || !aligned16(pos_of_pair) ||
      !aligned16(x) || !aligned16(rows))
    return E4B_ERR_ALIGN;
  a.ids = topk_idx;
  a.x = x;
  a.rows = rows;
  a.offsets = a.out_offsets = offsets;
  a.out_sorted = sorted_pair;
  a.pos = a.out_pos = pos_of_pair;
  if (T * top_k <= kOrderSmall) {
    E4B_TRY(launch_order_gather(a, stream));
    return E4B_OK;
  }
  E4B_TRY(launch_order(a, stream));
  if (!rows) return E4B_OK;
  E4B_TRY(launch_gather(a, stream));
  return E4B_OK;
}

extern "C" e4b_status e4b_unpermute(int64_t T, int32_t top_k, int64_t E, int64_t H, int32_t dtype,
                                    const int32_t *offsets, const int32_t *pos_of_pair, const float *topk_w,
                                    const void *rows, void *y, hipStream_t stream) {
  OrderArgs a{};
  e4b_status st = plan_order(T, top_k, E, H, dtype, &a);
  if (st != E4B_OK || T == 0) return st;
  if (!offsets || !pos_of_pair || !rows || !y) return E4B_ERR_NULL;
  if (!aligned16(offsets) || !aligned16(pos_of_pair) || !aligned16(topk_w) || !aligned16(rows) || !aligned16(y))
    return E4B_ERR_ALIGN;
  a.x = rows;
  a.rows = y;
  a.offsets = offsets;
  a.pos = pos_of_pair;
  a.w = topk_w;
  E4B_TRY(launch_unpermute(a, stream));
  return E4B_OK;
}

extern "C" e4b_status e4b_unpermute_backward(int64_t T, int32_t top_k, int64_t E, int64_t H, int32_t dtype,
                                             const int32_t *offsets, const int32_t *pos_of_pair,
                                             const float *topk_w, const void *rows, const void *grad_y,
                                             void *grad_rows, float *grad_topk_w, hipStream_t stream) {
  OrderArgs a{};
  e4b_status st = plan_order(T, top_k, E, H, dtype, &a);
  if (st != E4B_OK || T == 0) return st;
  if (!offsets || !pos_of_pair || !grad_y || !grad_rows || (grad_topk_w && !rows)) return E4B_ERR_NULL;
  if (!aligned16(offsets) || !aligned16(pos_of_pair) || !aligned16(topk_w) || !aligned16(rows) ||
      !aligned16(grad_y) || !aligned16(grad_rows) || !aligned16(grad_topk_w))
    return E4B_ERR_ALIGN;
  a.x = rows;
  a.gy = grad_y;
  a.rows = grad_rows;
  a.offsets = offsets;
  a.pos = pos_of_pair;
  a.w = topk_w;
  a.gw = grad_topk_w;
  E4B_TRY(launch_unpermute_bwd(a, stream));
  return E4B_OK;
}
