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
constexpr int kOrderIt = 32;                                   // ids per lane and pass
constexpr int kOrderPass = kOrderThreads * kOrderIt;           // 32768 pairs per pass
constexpr int kGatherThreads = 256;

// One workgroup per bucket e (the experts, then the bucket of dropped pairs).
// It reads every id: lower keys give the bucket's first position, equal ones
// the ranks. A wave takes runs of 64 consecutive pairs, so the compare's lane
// mask is the rank information: position = base + masks' population before it.
// E + 1 readings of 4 P bytes come from L2 and stay far below the rows' own
// traffic (P = 32768, E = 64: 8.5 MB against 151 MB).
__global__ __launch_bounds__(kOrderThreads) void order_kernel(const int32_t *__restrict__ ids, int64_t P, int E,
                                                              int32_t *__restrict__ offsets,
                                                              int32_t *__restrict__ sorted,
                                                              int32_t *__restrict__ pos) {
  __shared__ int32_t s_less[kOrderThreads / 64], s_eq[kOrderThreads / 64];
  const uint32_t e = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint64_t below = (1ull << lane) - 1;
  const bool drop = e == uint32_t(E);
  auto equal = [&](int32_t id) { return drop ? uint32_t(id) >= uint32_t(E) : uint32_t(id) == e; };
  uint64_t mask[kOrderIt];
  int32_t less = 0, eq = 0;
  // the masks of the wave's ids in the pass at p0
  auto scan = [&](int64_t p0, bool count_less) {
    const int64_t w0 = p0 + int64_t(wave) * (64 * kOrderIt);
    int32_t id[kOrderIt];
#pragma unroll
    for (int i = 0; i < kOrderIt; ++i) {
      const int64_t p = w0 + i * 64 + lane;
      id[i] = p < P ? ids[p] : 0;
    }
    eq = 0;
#pragma unroll
    for (int i = 0; i < kOrderIt; ++i) {
      const bool in = w0 + i * 64 + lane < P;
      mask[i] = __ballot(in && equal(id[i]));
      eq += __popcll(mask[i]);
      if (count_less) less += __popcll(__ballot(in && uint32_t(id[i]) < e));
    }
  };
  // first: how many pairs come before the bucket. One pass keeps its masks.
  int64_t total_eq = 0;
  for (int64_t p0 = 0; p0 < P; p0 += kOrderPass) scan(p0, true);
  if (lane == 0) s_less[wave] = less;
  __syncthreads();
  int32_t first = 0;
  for (int w = 0; w < kOrderThreads / 64; ++w) first += s_less[w];
  if (threadIdx.x == 0 && e < uint32_t(E) + 1) offsets[e] = first;
  // then the ranks, pass by pass
  for (int64_t p0 = 0; p0 < P; p0 += kOrderPass) {
    if (P > kOrderPass) scan(p0, false);
    __syncthreads();
    if (lane == 0) s_eq[wave] = eq;
    __syncthreads();
    int64_t at = first + total_eq;
    int32_t all = 0;
    for (int w = 0; w < kOrderThreads / 64; ++w) {
      if (w < wave) at += s_eq[w];
      all += s_eq[w];
    }
    total_eq += all;
    const int64_t w0 = p0 + int64_t(wave) * (64 * kOrderIt);
#pragma unroll
    for (int i = 0; i < kOrderIt; ++i) {
      if ((mask[i] >> lane) & 1) {
        const int32_t p = int32_t(w0) + i * 64 + lane, s = int32_t(at) + __popcll(mask[i] & below);
        sorted[s] = p;
        pos[p] = s;
      }
      at += __popcll(mask[i]);
    }
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

// y[t] = sum_j w[t, j] rows[pos(t, j)] (no weights: the plain sum, which is
// the gradient of the copies). One workgroup per token and kGatherThreads *
// VEC columns, up to 8 rows in flight.
template <typename T, int VEC>
__global__ __launch_bounds__(kGatherThreads) void unpermute_kernel(const T *__restrict__ rows, int k, int H, int E,
                                                                   const int32_t *__restrict__ offsets,
                                                                   const int32_t *__restrict__ pos,
                                                                   const float *__restrict__ w, T *__restrict__ y) {
  __shared__ int32_t s_pos[kMaxTopK];
  __shared__ float s_w[kMaxTopK];
  const int64_t t = blockIdx.x;
  if (threadIdx.x < k) {
    const int32_t s = pos[t * k + threadIdx.x], live = offsets[E];
    s_pos[threadIdx.x] = s >= 0 && s < live ? s : -1;
    s_w[threadIdx.x] = w ? w[t * k + threadIdx.x] : 1.0f;
  }
  __syncthreads();
  const int h = (blockIdx.y * kGatherThreads + threadIdx.x) * VEC;
  if (h >= H) return;
  float acc[VEC];
#pragma unroll
  for (int q = 0; q < VEC; ++q) acc[q] = 0.0f;
  for (int j0 = 0; j0 < k; j0 += 8) {
    float v[8][VEC];
#pragma unroll
    for (int jj = 0; jj < 8; ++jj)
      if (j0 + jj < k && s_pos[j0 + jj] >= 0) load_row<VEC>(rows + int64_t(s_pos[j0 + jj]) * H + h, v[jj]);
#pragma unroll
    for (int jj = 0; jj < 8; ++jj)
      if (j0 + jj < k && s_pos[j0 + jj] >= 0) {
        const float wj = s_w[j0 + jj];
#pragma unroll
        for (int q = 0; q < VEC; ++q) acc[q] += wj * v[jj][q];
      }
  }
  store_row<VEC>(y + t * H + h, acc);
}

// grad_rows[pos(t, j)] = w[t, j] grad_y[t] and grad_w[t, j] = rows[pos(t, j)] . grad_y[t].
// One workgroup per token: grad_y's row is read once per 8 slots, each pair's
// row once; the dots end in a fixed tree over the workgroup.
template <typename T, int VEC>
__global__ __launch_bounds__(kGatherThreads) void unpermute_bwd_kernel(
    const T *__restrict__ rows, const T *__restrict__ gy, int64_t P, int k, int H, int E,
    const int32_t *__restrict__ offsets, const int32_t *__restrict__ pos, const float *__restrict__ w,
    T *__restrict__ grows, float *__restrict__ gw) {
  __shared__ int32_t s_pos[kMaxTopK];
  __shared__ float s_w[kMaxTopK];
  __shared__ float s_dot[kGatherThreads / 64][8];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t live = offsets[E];
  if (threadIdx.x < k) {
    const int32_t s = pos[t * k + threadIdx.x];
    s_pos[threadIdx.x] = s >= 0 && s < P ? s : -1;
    s_w[threadIdx.x] = w ? w[t * k + threadIdx.x] : 1.0f;
  }
  __syncthreads();
  for (int j0 = 0; j0 < k; j0 += 8) {
    float dot[8];
#pragma unroll
    for (int jj = 0; jj < 8; ++jj) dot[jj] = 0.0f;
    for (int h = threadIdx.x * VEC; h < H; h += kGatherThreads * VEC) {
      float g[VEC];
      load_row<VEC>(gy + t * H + h, g);
      float v[8][VEC];
      if (gw) {
#pragma unroll
        for (int jj = 0; jj < 8; ++jj)
          if (j0 + jj < k && s_pos[j0 + jj] >= 0 && s_pos[j0 + jj] < live)
            load_row<VEC>(rows + int64_t(s_pos[j0 + jj]) * H + h, v[jj]);
      }
#pragma unroll
      for (int jj = 0; jj < 8; ++jj) {
        if (j0 + jj >= k || s_pos[j0 + jj] < 0) continue;
        const int32_t s = s_pos[j0 + jj];
        const bool in = s < live;
        float o[VEC];
#pragma unroll
        for (int q = 0; q < VEC; ++q) o[q] = in ? s_w[j0 + jj] * g[q] : 0.0f;
        store_row<VEC>(grows + int64_t(s) * H + h, o);
        if (gw && in) {
#pragma unroll
          for (int q = 0; q < VEC; ++q) dot[jj] += v[jj][q] * g[q];
        }
      }
    }
    if (gw) {
#pragma unroll
      for (int jj = 0; jj < 8; ++jj) {
        const float d = wave_sum(dot[jj]);
        if (lane == 0) s_dot[wave][jj] = d;
      }
      __syncthreads();
      const int jj = threadIdx.x;
      if (jj < 8 && j0 + jj < k) {
        float d = 0.0f;
        for (int q = 0; q < kGatherThreads / 64; ++q) d += s_dot[q][jj];
        gw[t * k + j0 + jj] = d;
      }
      __syncthreads();
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
hipError_t unpermute(const OrderArgs &a, hipStream_t s) {
  const uint32_t slabs = uint32_t((a.H + kGatherThreads * VEC - 1) / (kGatherThreads * VEC));
  hipLaunchKernelGGL((unpermute_kernel<T, VEC>), dim3(uint32_t(a.T), slabs), dim3(kGatherThreads), 0, s,
                     static_cast<const T *>(a.x), a.k, a.H, a.E, a.offsets, a.pos, a.w, static_cast<T *>(a.rows));
  return hipGetLastError();
}
template <typename T, int VEC>
hipError_t unpermute_bwd(const OrderArgs &a, hipStream_t s) {
  hipLaunchKernelGGL((unpermute_bwd_kernel<T, VEC>), dim3(uint32_t(a.T)), dim3(kGatherThreads), 0, s,
                     static_cast<const T *>(a.x), static_cast<const T *>(a.gy), a.T * a.k, a.k, a.H, a.E, a.offsets,
                     a.pos, a.w, static_cast<T *>(a.rows), a.gw);
  return hipGetLastError();
}

#define E4B_ROWS(F, a, s)                                                                 \
  (a.f32 ? (a.H % 8 ? F<float, 1>(a, s) : F<float, 8>(a, s))                              \
         : (a.H % 8 ? F<bf16_t, 1>(a, s) : F<bf16_t, 8>(a, s)))

}  // namespace

hipError_t launch_order(const int32_t *ids, const OrderArgs &a, int32_t *offsets, int32_t *sorted, int32_t *pos,
                        hipStream_t s) {
  hipLaunchKernelGGL(order_kernel, dim3(uint32_t(a.E + 1)), dim3(kOrderThreads), 0, s, ids, a.T * a.k, a.E, offsets,
                     sorted, pos);
  return hipGetLastError();
}
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
  E4B_TRY(launch_order(topk_idx, a, offsets, sorted_pair, pos_of_pair, stream));
  if (!T || !rows) return E4B_OK;
  a.x = x;
  a.rows = rows;
  a.offsets = offsets;
  a.pos = pos_of_pair;
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
