// route.hip -- top-k routing and the token-by-expert permutation.
//
// experts4bit-qlora 0.1.0 sdist, _vendor/experts.py, Experts4bit.forward takes
// (top_k_index, top_k_weights) from a router outside the module and groups the
// routed (token, slot) pairs per expert with a one-hot mask and torch.where,
// paying a device-to-host sync for every expert. Here the grouping is a stable
// counting sort done entirely on the device:
//   1. histogram of expert ids per chunk of kPermChunk pairs,
//   2. per expert, exclusive scan of its chunk counts,
//   3. per chunk, one wavefront assigns each pair its sorted position
//      (expert offset + chunk base + rank among equal ids, lanes in pair order).
#include "device.h"
#include "kernels.h"
#include "plan_block.h"
#include "route_dev.h"
#include "rowvec.h"

namespace e4b {

// One wavefront per token (route_dev.h).
__global__ __launch_bounds__(256) void route_kernel(const float *__restrict__ logits, int64_t T,
                                                    int E, int k, int32_t *__restrict__ idx,
                                                    float *__restrict__ wts) {
  __shared__ RouteLds s_route[4];
  const int lane = threadIdx.x & 63;
  const int64_t t = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  route_token(logits, t, E, k, lane, idx, wts, nullptr, s_route[threadIdx.x >> 6]);
}

// The router as an operator of its own: the selection and weights of
// route_kernel, for logits that may also be -inf (an expert out of service
// for this token). Such an expert gets weight 0 when it has to fill a slot; a
// row that is -inf throughout selects experts 0 .. k - 1 with weights 0.
//
// L lanes hold a token's logits, PER each (expert i L + lane), as integers of
// the same order (so that a taken one can be less than any logit): k rounds of
// a maximum and the lowest id that has it. With 16 lanes to a token the
// reductions are four DPP moves within a row and serve four tokens at once; a
// wave per token took 15.1 us at 16384 x 128, top 8, this one 7.6 us (8 MB
// read). More than 128 experts of few tokens keep the wave (see e4b_route).
__device__ __forceinline__ int32_t order_key(float v) {
  const int32_t b = __builtin_bit_cast(int32_t, v + 0.0f);  // -0 is +0
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float key_value(int32_t key) {
  return __builtin_bit_cast(float, key ^ ((key >> 31) & 0x7FFFFFFF));
}
template <int CTRL>
__device__ __forceinline__ int32_t dpp(int32_t v) {
  return __builtin_amdgcn_update_dpp(v, v, CTRL, 0xF, 0xF, false);
}
// the largest / smallest value of a token's L lanes, on all of them
template <int L>
__device__ __forceinline__ int32_t lanes_max(int32_t v) {
  v = max(v, dpp<0x128>(v));  // row_ror 8, 4, 2, 1
  v = max(v, dpp<0x124>(v));
  v = max(v, dpp<0x122>(v));
  v = max(v, dpp<0x121>(v));
  if (L == 64)
    v = max(max(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16)),
            max(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48)));
  return v;
}
template <int L>
__device__ __forceinline__ int32_t lanes_min(int32_t v) {
  return ~lanes_max<L>(~v);
}

template <int L, int PER>
__global__ __launch_bounds__(256) void route_masked_kernel(const float *__restrict__ logits, int64_t T, int E, int k,
                                                           int32_t *__restrict__ idx, float *__restrict__ wts) {
  const int l = threadIdx.x % L;
  const int64_t t = int64_t(blockIdx.x) * (256 / L) + threadIdx.x / L;
  const int64_t row = min(t, T - 1) * E;  // (all lanes stay for the reductions)
  int32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) key[i] = order_key(logits[row + min(i * L + l, E - 1)]);
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (i * L + l >= E) key[i] = INT32_MIN;
  constexpr int kSlots = (kMaxTopK + L - 1) / L;  // slots j = s L + lane that a lane keeps
  int32_t id[kSlots];
  float z[kSlots], top = 0.0f, sum = 0.0f;
  for (int j = 0; j < k; ++j) {
    int32_t best = key[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) best = max(best, key[i]);
    best = lanes_max<L>(best);
    int32_t at = INT32_MAX;
#pragma unroll
    for (int i = PER - 1; i >= 0; --i) at = key[i] == best ? i * L + l : at;
    at = lanes_min<L>(at);
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = i * L + l == at ? INT32_MIN : key[i];
    const float v = key_value(best);
    if (j == 0) top = v;
    const float zj = expf(v - top);
    sum += zj;
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
      if (j == s * L + l) {
        id[s] = at;
        z[s] = zj;
      }
  }
  if (t >= T) return;
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    const int j = s * L + l;
    if (j < k) {
      idx[t * k + j] = id[s];
      wts[t * k + j] = top == -INFINITY ? 0.0f : z[s] / sum;
    }
  }
}

// Gradient of the logits through w = softmax(selected logits), the selection
// held fixed: dl[idx_j] = w_j (g_j - sum_i w_i g_i), 0 for every other expert.
// tpt threads to a token, each with 4 (VEC) consecutive experts at a time: the
// token's k (id, value) pairs come from LDS, the row leaves in one write of 4
// E bytes per token, which is the floor.
template <int VEC>
__global__ __launch_bounds__(256) void route_bwd_kernel(const int32_t *__restrict__ idx, const float *__restrict__ wts,
                                                        const float *__restrict__ gw, int64_t T, int E, int k, int tpt,
                                                        float *__restrict__ gl) {
  constexpr int kMost = 16;  // tokens per workgroup
  __shared__ int32_t s_id[kMost * kMaxTopK];
  __shared__ float s_w[kMost * kMaxTopK], s_g[kMost * kMaxTopK], s_d[kMost * kMaxTopK];
  const int tokens = 256 / tpt;
  const int64_t t0 = int64_t(blockIdx.x) * tokens;
  const int pairs = int(min(int64_t(tokens), T - t0)) * k;
  for (int i = threadIdx.x; i < pairs; i += 256) {
    s_id[i] = idx[t0 * k + i];
    s_w[i] = wts[t0 * k + i];
    s_g[i] = gw[t0 * k + i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += 256) {
    const int first = i / k * k;
    float dot = 0.0f;
    for (int j = 0; j < k; ++j) dot += s_w[first + j] * s_g[first + j];
    s_d[i] = s_w[i] * (s_g[i] - dot);
  }
  __syncthreads();
  const int tok = threadIdx.x / tpt;
  const int64_t t = t0 + tok;
  if (t >= T) return;
  for (int e0 = (threadIdx.x % tpt) * VEC; e0 < E; e0 += tpt * VEC) {
    float v[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) v[q] = 0.0f;
    for (int j = 0; j < k; ++j) {
      const int32_t id = s_id[tok * k + j] - e0;
      const float d = s_d[tok * k + j];
#pragma unroll
      for (int q = 0; q < VEC; ++q) v[q] += id == q ? d : 0.0f;
    }
    store_row<VEC>(gl + t * E + e0, v);
  }
}

// hist[e * nchunks + c] = number of pairs of chunk c routed to expert e.
__global__ __launch_bounds__(256) void perm_hist_kernel(const int32_t *__restrict__ flat_idx,
                                                        int64_t P, int E, int64_t nchunks,
                                                        int32_t *__restrict__ hist) {
  __shared__ int32_t h[kMaxE];
  for (int e = threadIdx.x; e < E; e += 256) h[e] = 0;
  __syncthreads();
  const int64_t c = blockIdx.x;
  const int64_t p0 = c * kPermChunk;
  for (int i = threadIdx.x; i < kPermChunk; i += 256) {
    const int64_t p = p0 + i;
    if (p < P) atomicAdd(&h[safe_expert(flat_idx[p], E)], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 256) hist[int64_t(e) * nchunks + c] = h[e];
}

// One workgroup per expert: chunk_base[e][c] = sum_{c' < c} hist[e][c'],
// counts[e] = total.
__global__ __launch_bounds__(256) void perm_scan_kernel(const int32_t *__restrict__ hist,
                                                        int64_t nchunks,
                                                        int32_t *__restrict__ chunk_base,
                                                        int32_t *__restrict__ counts) {
  __shared__ int32_t wsum[4];
  const int e = blockIdx.x;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int32_t *hrow = hist + int64_t(e) * nchunks;
  int32_t *brow = chunk_base + int64_t(e) * nchunks;
  int32_t carry = 0;
  for (int64_t c0 = 0; c0 < nchunks; c0 += 256) {
    const int64_t c = c0 + threadIdx.x;
    const int32_t v = c < nchunks ? hrow[c] : 0;
    int32_t incl = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int32_t n = __shfl_up(incl, o);
      if (lane >= o) incl += n;
    }
    if (lane == 63) wsum[wv] = incl;
    __syncthreads();
    int32_t before = carry;
    for (int i = 0; i < wv; ++i) before += wsum[i];
    if (c < nchunks) brow[c] = before + incl - v;
    const int32_t total = wsum[0] + wsum[1] + wsum[2] + wsum[3];
    __syncthreads();
    carry += total;
  }
  if (threadIdx.x == 0) counts[e] = carry;
}

// One wavefront per chunk. Writes sorted_pair / pos_of_pair; workgroup 0 also
// writes offsets[E+1], tile_offsets[E+1] (m-tiles of kBM rows per expert) and
// the tile map (expert, segment start, first row, rows) of every m-tile, so a
// GEMM workgroup finds its tile with one load.
__global__ __launch_bounds__(64) void perm_scatter_kernel(
    const int32_t *__restrict__ flat_idx, int64_t P, int E, int nbits, int64_t nchunks,
    const int32_t *__restrict__ counts, const int32_t *__restrict__ chunk_base,
    int32_t *__restrict__ sorted_pair, int32_t *__restrict__ pos_of_pair,
    int32_t *__restrict__ offsets, int32_t *__restrict__ tile_offsets,
    int4 *__restrict__ tile_map, int64_t m_tiles_bound) {
  __shared__ int32_t base[kMaxE];
  const int lane = threadIdx.x;
  const int64_t c = blockIdx.x;
  const int64_t p0 = c * kPermChunk;
  // the chunk's expert ids, all loads issued before the scan below
  constexpr int kIt = kPermChunk / 64;
  int ids[kIt];
#pragma unroll
  for (int it = 0; it < kIt; ++it) {
    const int64_t p = p0 + it * 64 + lane;
    ids[it] = p < P ? safe_expert(flat_idx[p], E) : 0;
  }
  // exclusive scan of counts (and of m-tiles) over experts, 64 at a time
  int32_t carry = 0, tcarry = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    const int32_t v = e < E ? counts[e] : 0;
    const int32_t tv = (v + kBM - 1) / kBM;
    int32_t incl = v, tincl = tv;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int32_t n = __shfl_up(incl, o), tn = __shfl_up(tincl, o);
      if (lane >= o) {
        incl += n;
        tincl += tn;
      }
    }
    if (e < E) {
      const int32_t off = carry + incl - v;
      base[e] = off + chunk_base[int64_t(e) * nchunks + c];
      if (c == 0) {
        offsets[e] = off;
        const int32_t t0 = tcarry + tincl - tv;
        tile_offsets[e] = t0;
        for (int t = 0; t < tv; ++t)
          tile_map[t0 + t] = int4{e, off, t * kBM, min(kBM, v - t * kBM)};
      }
    }
    carry += __shfl(incl, 63);
    tcarry += __shfl(tincl, 63);
  }
  if (c == 0 && lane == 0) {
    offsets[E] = carry;
    tile_offsets[E] = tcarry;
  }
  // unused tile map entries are zeroed (no stale bytes in a saved buffer)
  if (c == 0)
    for (int64_t t = tcarry + lane; t < m_tiles_bound; t += 64) tile_map[t] = int4{0, 0, 0, 0};
  __syncthreads();
  const uint64_t lt = (lane == 0) ? 0ull : (~0ull >> (64 - lane));
#pragma unroll
  for (int it = 0; it < kIt; ++it) {
    const int64_t p = p0 + it * 64 + lane;
    const bool valid = p < P;
    const int e = ids[it];
    uint64_t match = __ballot(valid);
    for (int b = 0; b < nbits; ++b) {
      const bool bit = (e >> b) & 1;
      const uint64_t bal = __ballot(bit);
      match &= bit ? bal : ~bal;
    }
    const int rank = __popcll(match & lt);
    const int32_t my_base = valid ? base[e] : 0;
    __syncthreads();
    if (valid) {
      const int32_t pos = my_base + rank;
      sorted_pair[pos] = int32_t(p);
      pos_of_pair[p] = pos;
      // the highest lane of each equal-id group advances that expert's base
      if ((match >> lane) == 1ull) base[e] = my_base + __popcll(match);
    }
    __syncthreads();
  }
}

hipError_t launch_route(const float *logits, int64_t T, int E, int k, int32_t *idx, float *w,
                        hipStream_t s, const e4b_kernel_events *ev) {
  if (T == 0) return hipSuccess;
  return launch_k(ev, E4B_K_ROUTE, route_kernel, dim3(uint32_t((T + 3) / 4)), dim3(256), s, logits,
                  T, E, k, idx, w);
}

PermView perm_in_workspace(const MoePlan &p, char *ws) {
  PermView v;
  v.offsets = reinterpret_cast<int32_t *>(ws + p.off_offsets);
  v.tile_offsets = reinterpret_cast<int32_t *>(ws + p.off_tile_offsets);
  v.tile_map = reinterpret_cast<int4 *>(ws + p.off_tile_map);
  v.sorted = reinterpret_cast<int32_t *>(ws + p.off_sorted);
  v.pos = reinterpret_cast<int32_t *>(ws + p.off_pos);
  return v;
}

PermView perm_in_saved(const MoePlan &p, char *saved) {
  PermView v;
  v.offsets = reinterpret_cast<int32_t *>(saved + p.sv_offsets);
  v.tile_offsets = reinterpret_cast<int32_t *>(saved + p.sv_tile_offsets);
  v.tile_map = reinterpret_cast<int4 *>(saved + p.sv_tile_map);
  v.sorted = reinterpret_cast<int32_t *>(saved + p.sv_sorted);
  v.pos = reinterpret_cast<int32_t *>(saved + p.sv_pos);
  return v;
}

hipError_t launch_permute(const MoePlan &p, const int32_t *idx, char *ws, const PermView &v,
                          hipStream_t s, const e4b_kernel_events *ev) {
  if (p.P == 0) return hipSuccess;
  int32_t *hist = reinterpret_cast<int32_t *>(ws + p.off_hist);
  int32_t *cbase = reinterpret_cast<int32_t *>(ws + p.off_chunk_base);
  int32_t *counts = reinterpret_cast<int32_t *>(ws + p.off_counts);
  const int E = int(p.E);
  // E4B_K_PERMUTE spans the three launches: start event on the first, stop on the last
  hipEvent_t e0 = ev ? ev->start[E4B_K_PERMUTE] : nullptr, e1 = ev ? ev->stop[E4B_K_PERMUTE] : nullptr;
  const bool timed = e0 && e1;
  if (timed)
    hipExtLaunchKernelGGL(perm_hist_kernel, dim3(uint32_t(p.nchunks)), dim3(256), 0, s, e0,
                          static_cast<hipEvent_t>(nullptr), 0, idx, p.P, E, p.nchunks, hist);
  else
    hipLaunchKernelGGL(perm_hist_kernel, dim3(uint32_t(p.nchunks)), dim3(256), 0, s, idx, p.P, E,
                       p.nchunks, hist);
  hipLaunchKernelGGL(perm_scan_kernel, dim3(uint32_t(E)), dim3(256), 0, s, hist, p.nchunks, cbase,
                     counts);
  if (timed)
    hipExtLaunchKernelGGL(perm_scatter_kernel, dim3(uint32_t(p.nchunks)), dim3(64), 0, s,
                          static_cast<hipEvent_t>(nullptr), e1, 0, idx, p.P, E, p.nbits_e,
                          p.nchunks, static_cast<const int32_t *>(counts),
                          static_cast<const int32_t *>(cbase), v.sorted, v.pos, v.offsets,
                          v.tile_offsets, v.tile_map, p.m_tiles_bound);
  else
    hipLaunchKernelGGL(perm_scatter_kernel, dim3(uint32_t(p.nchunks)), dim3(64), 0, s, idx, p.P, E,
                       p.nbits_e, p.nchunks, counts, cbase, v.sorted, v.pos, v.offsets,
                       v.tile_offsets, v.tile_map, p.m_tiles_bound);
  return hipGetLastError();
}

}  // namespace e4b

using namespace e4b;

extern "C" e4b_status e4b_route(const float *logits, int64_t T, int64_t E, int32_t top_k, int32_t *topk_idx,
                                float *topk_w, hipStream_t stream) {
  const e4b_status st = check_route(T, E, top_k);
  if (st != E4B_OK || T == 0) return st;
  if (!logits || !topk_idx || !topk_w) return E4B_ERR_NULL;
  if (!aligned16(logits) || !aligned16(topk_idx) || !aligned16(topk_w)) return E4B_ERR_ALIGN;
  auto go = [&](auto kernel, int lanes) {
    const int64_t tokens = 256 / lanes;
    hipLaunchKernelGGL(kernel, dim3(uint32_t((T + tokens - 1) / tokens)), dim3(256), 0, stream, logits, T, int(E),
                       int(top_k), topk_idx, topk_w);
  };
  // 16 lanes a token do least in all, 64 get a token's maxima soonest (in us for top 16,
  // 16 / 64 lanes: 256 experts, 2048 tokens 7.9 / 7.0, 16384 tokens 15.4 / 31.5; 512
  // experts, 2048 tokens 12.4 / 8.0, 16384 tokens 24.8 / 37.6; 1000 experts 21 / 10, 48 / 51)
  const bool many = T > 4096;
  if (E <= 16)
    go(route_masked_kernel<16, 1>, 16);
  else if (E <= 32)
    go(route_masked_kernel<16, 2>, 16);
  else if (E <= 64)
    go(route_masked_kernel<16, 4>, 16);
  else if (E <= 128)
    go(route_masked_kernel<16, 8>, 16);
  else if (E <= 256 && !many)
    go(route_masked_kernel<64, 4>, 64);
  else if (E <= 256)
    go(route_masked_kernel<16, 16>, 16);
  else if (E <= 512 && many)
    go(route_masked_kernel<16, 32>, 16);
  else if (E <= 512)
    go(route_masked_kernel<64, 8>, 64);
  else
    go(route_masked_kernel<64, 16>, 64);
  return hipGetLastError() == hipSuccess ? E4B_OK : E4B_ERR_HIP;
}

extern "C" e4b_status e4b_route_backward(const int32_t *topk_idx, const float *topk_w, const float *grad_topk_w,
                                         int64_t T, int64_t E, int32_t top_k, float *grad_logits,
                                         hipStream_t stream) {
  const e4b_status st = check_route(T, E, top_k);
  if (st != E4B_OK || T == 0) return st;
  if (!topk_idx || !topk_w || !grad_topk_w || !grad_logits) return E4B_ERR_NULL;
  if (!aligned16(topk_idx) || !aligned16(topk_w) || !aligned16(grad_topk_w) || !aligned16(grad_logits))
    return E4B_ERR_ALIGN;
  const bool vec = E % 4 == 0;
  int tpt = 16;  // at most 16 tokens to a workgroup
  while (tpt < 256 && tpt * (vec ? 4 : 1) < E) tpt *= 2;
  const int64_t tokens = 256 / tpt;
  hipLaunchKernelGGL(vec ? route_bwd_kernel<4> : route_bwd_kernel<1>, dim3(uint32_t((T + tokens - 1) / tokens)), dim3(256),
                     0, stream, topk_idx, topk_w, grad_topk_w, T, int(E), int(top_k), tpt, grad_logits);
  return hipGetLastError() == hipSuccess ? E4B_OK : E4B_ERR_HIP;
}
