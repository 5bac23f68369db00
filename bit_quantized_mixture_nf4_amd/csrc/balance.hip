// balance.hip -- how evenly a router uses its experts, and the gradient that keeps it even:
//   lse_t = log sum_e exp l_te,  p_te = exp(l_te - lse_t)
//   N_s = counted tokens of sequence s,  c_se = their pairs (t, j) with idx = e,  prob_se = sum_t p_te
//   loss_s = E / (k N_s^2) sum_e c_se prob_se,  z_s = 1 / N_s sum_t lse_t^2
//   dl_te = gl_s E / (k N_s^2) p_te (c_se - sum_j c_sj p_tj) + gz_s 2 / N_s lse_t p_te
// A token is counted if the mask has it, it lies in a sequence and its row is not
// -inf throughout; lse is -inf for every other one, which is how the gradient
// knows them. The logits are read once in each direction and held in registers; both
// kernels have nothing else of their size to move. Sums over tokens run in a fixed
// order (a lane's tokens, the lanes, the waves, the chunks), the counts are whole
// numbers: results are the same on every run.
#include "kernels.h"
#include "rowvec.h"

namespace e4b {

namespace {

__device__ __forceinline__ int32_t first_token(const BalanceArgs &g, int s) {
  if (!g.cu) return s ? int32_t(g.T) : 0;
  return min(max(g.cu[s], 0), int32_t(g.T));
}

// the last s of [0, S) with key(s) <= w, 0 if there is none: 64 keys at a time. Uniform over a wave.
template <typename F>
__device__ __forceinline__ int last_not_above(int S, int64_t w, int lane, F key) {
  int lo = 0, n = S;
  while (n > 1) {
    const int step = (n + 63) / 64, s = lo + lane * step;
    const int below = __popcll(__ballot(lane * step < n && key(s) <= w));
    if (below == 0) return lo;
    const int at = (below - 1) * step;
    lo += at;
    n = min(step, n - at);
  }
  return lo;
}

// the sum / largest of a token's L lanes, on all of them: four moves within a row of 16
template <int CTRL>
__device__ __forceinline__ float dppf(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int32_t, v), CTRL, 0xF, 0xF, false));
}
template <int L>
__device__ __forceinline__ float token_sum(float v) {
  v += dppf<0x128>(v);  // row_ror 8, 4, 2, 1
  v += dppf<0x124>(v);
  v += dppf<0x122>(v);
  v += dppf<0x121>(v);
  if (L == 64) {
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
  }
  return v;
}
template <int L>
__device__ __forceinline__ float token_max(float v) {
  v = fmaxf(v, dppf<0x128>(v));
  v = fmaxf(v, dppf<0x124>(v));
  v = fmaxf(v, dppf<0x122>(v));
  v = fmaxf(v, dppf<0x121>(v));
  if (L == 64) {
    v = fmaxf(v, __shfl_xor(v, 16));
    v = fmaxf(v, __shfl_xor(v, 32));
  }
  return v;
}

// A token's row in L lanes: VEC consecutive experts at (i L + lane) VEC, i < PER.
template <int L, int PER, int VEC>
struct Row {
  float v[PER][VEC];
  __device__ __forceinline__ static int column(int i) { return (i * L + threadIdx.x % L) * VEC; }
  __device__ __forceinline__ void load(const float *p, int E, float fill) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
#pragma unroll
      for (int q = 0; q < VEC; ++q) v[i][q] = fill;
      if (column(i) < E) load_row<VEC>(p + column(i), v[i]);
    }
  }
  // v becomes exp(v - max); returns the sum, and the maximum that was taken off (0 for a row of -inf)
  __device__ __forceinline__ float exponentials(float &top) {
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
      for (int q = 0; q < VEC; ++q) top = fmaxf(top, v[i][q]);
    top = token_max<L>(top);
    if (top == -INFINITY) top = 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        v[i][q] = expf(v[i][q] - top);
        sum += v[i][q];
      }
    return token_sum<L>(sum);
  }
};

struct Total {
  int32_t n;
  float z;
  double dot;
};

__device__ __forceinline__ void write_losses(const BalanceArgs &g, int s, const Total &t) {
  const double inv = t.n ? 1.0 / double(t.n) : 0.0;
  g.tokens[s] = t.n;
  g.loss[s] = float(t.dot * inv * inv * (double(g.E) / double(g.k)));
  g.z[s] = float(double(t.z) * inv);
}

// One workgroup per slot (and, behind the slots, per so many threads' tokens that may lie outside every
// sequence): a chunk of at most g.chunk tokens of one sequence, kThreads / L of them at a time. (Half as many chunks of
// twice the threads take the same time here, and the join half.)
constexpr int balance_threads(bool one) { return one ? 256 : 512; }
template <int L, int PER, int VEC, bool ONE>
__global__ __launch_bounds__(balance_threads(ONE)) void balance_kernel(BalanceArgs g) {
  constexpr int kThreads = balance_threads(ONE), kGroups = kThreads / L, kWaves = kThreads / 64;
  __shared__ float s_prob[kWaves][kMaxE];
  __shared__ int32_t s_counts[kMaxE];
  __shared__ float s_z[kWaves];
  __shared__ int32_t s_n[kWaves];
  __shared__ double s_dot[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int s = 0;
  int32_t lo = 0, hi = int32_t(g.T);
  if (!ONE) {
    if (int64_t(blockIdx.x) >= g.slots) {
      const int64_t t = (int64_t(blockIdx.x) - g.slots) * kThreads + tid;
      if (t < g.T && (t < first_token(g, 0) || t >= first_token(g, g.S))) g.lse[t] = -INFINITY;
      return;
    }
    const int64_t w = blockIdx.x;
    s = last_not_above(g.S, w, lane, [&](int i) { return int64_t(first_token(g, i) / g.chunk) + i; });
    const int32_t a = first_token(g, s);
    const int64_t from = a + (w - (a / g.chunk + s)) * g.chunk;
    hi = first_token(g, s + 1);
    if (w < a / g.chunk + s || from >= hi) return;  // a slot without a chunk
    lo = int32_t(from);
    hi = int32_t(min(int64_t(hi), from + g.chunk));
  }
  for (int e = tid; e < g.E; e += kThreads) s_counts[e] = 0;
  __syncthreads();
  float prob[PER][VEC], z = 0.0f;
  int32_t n = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int q = 0; q < VEC; ++q) prob[i][q] = 0.0f;
  // (all lanes stay for the reductions: the bound is the workgroup's)
  for (int32_t t0 = lo; t0 < hi; t0 += kGroups) {
    const int32_t t = t0 + tid / L;
    const bool in = t < hi;
    Row<L, PER, VEC> row;
    row.load(g.logits + int64_t(min(t, hi - 1)) * g.E, g.E, -INFINITY);
    float top;
    const float sum = row.exponentials(top);
    // (a NaN counts: it is to be seen in the losses)
    const bool counted = in && !(sum == 0.0f) && (!g.mask || g.mask[t]);
    const float lse = counted ? top + logf(sum) : -INFINITY;
    if (in && tid % L == 0) g.lse[t] = lse;
    if (counted) {
      const float inv = 1.0f / sum;
#pragma unroll
      for (int i = 0; i < PER; ++i)
#pragma unroll
        for (int q = 0; q < VEC; ++q) prob[i][q] += row.v[i][q] * inv;
      for (int j = tid % L; j < g.k; j += L) {
        const int32_t e = g.idx[int64_t(t) * g.k + j];
        if (uint32_t(e) < uint32_t(g.E)) atomicAdd(&s_counts[e], 1);
      }
      if (tid % L == 0) {
        z += lse * lse;
        n += 1;
      }
    }
  }
  // the wave's tokens, then the waves
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
      float p = prob[i][q];
      if (L == 16) {
        p += __shfl_xor(p, 16);
        p += __shfl_xor(p, 32);
      }
      const int e = Row<L, PER, VEC>::column(i) + q;
      if (lane < L && e < g.E) s_prob[wave][e] = p;
    }
  z = wave_sum(z);
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) n += __shfl_xor(n, o);
  if (lane == 0) {
    s_z[wave] = z;
    s_n[wave] = n;
  }
  __syncthreads();
  double dot = 0.0;
  for (int e = tid; e < g.E; e += kThreads) {
    float p = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) p += s_prob[w][e];
    if (ONE) {
      g.prob[e] = p;
      g.counts[e] = s_counts[e];
      dot += double(p) * double(s_counts[e]);
    } else {
      const int64_t at = int64_t(blockIdx.x) * g.E + e;
      g.part_prob[at] = p;
      g.part_counts[at] = s_counts[e];
    }
  }
  z = 0.0f;
  n = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    z += s_z[w];
    n += s_n[w];
  }
  if (ONE) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) dot += __shfl_xor(dot, o);
    if (lane == 0) s_dot[wave] = dot;
    __syncthreads();
    if (tid == 0) {
      dot = 0.0;
      for (int w = 0; w < kWaves; ++w) dot += s_dot[w];
      write_losses(g, 0, Total{n, z, dot});
    }
  } else if (tid == 0) {
    g.part_z[blockIdx.x] = z;
    g.part_tokens[blockIdx.x] = n;
  }
}

// One workgroup per sequence: its chunks' sums, in order. A thread takes VEC experts of every so-many-th chunk,
// kJoinAhead chunks at a time: waiting for one row after the other took 28 us for 512 chunks of 128
// experts, so they take 9, and the 256 chunks of 16384 tokens (whose own sums take 7) 6.
constexpr int kJoinThreads = 1024, kJoinAhead = 8;
template <int VEC>
__global__ __launch_bounds__(kJoinThreads) void balance_join_kernel(BalanceArgs g, int cols) {
  __shared__ __attribute__((aligned(16))) float s_prob[kJoinThreads * VEC];
  __shared__ __attribute__((aligned(16))) int32_t s_counts[kJoinThreads * VEC];
  __shared__ double s_dot[kJoinThreads / 64];
  __shared__ float s_z[kJoinThreads / 64];
  __shared__ int32_t s_n[kJoinThreads / 64];
  typedef float values __attribute__((ext_vector_type(VEC)));
  typedef int32_t numbers __attribute__((ext_vector_type(VEC)));
  const int s = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int32_t a = first_token(g, s), b = first_token(g, s + 1);
  const int64_t w0 = a / g.chunk + s;
  const int32_t chunks = b > a ? (b - a + g.chunk - 1) / g.chunk : 0;
  // cols threads to a row of E sums (cols a power of two, cols VEC at least E)
  const int e = (tid & (cols - 1)) * VEC, rows = kJoinThreads / cols;
  values p = 0.0f;
  numbers c = 0;
  if (e < g.E) {
    for (int32_t i0 = tid / cols; i0 < chunks; i0 += kJoinAhead * rows) {
      values dp[kJoinAhead];
      numbers dc[kJoinAhead];
#pragma unroll
      for (int u = 0; u < kJoinAhead; ++u) {
        const int64_t at = (w0 + min(i0 + u * rows, chunks - 1)) * g.E + e;
        dp[u] = *reinterpret_cast<const values *>(g.part_prob + at);
        dc[u] = *reinterpret_cast<const numbers *>(g.part_counts + at);
      }
#pragma unroll
      for (int u = 0; u < kJoinAhead; ++u)
        if (i0 + u * rows < chunks) {
          p += dp[u];
          c += dc[u];
        }
    }
  }
  float z = 0.0f;
  int32_t n = 0;
  for (int32_t i = tid; i < chunks; i += kJoinThreads) {
    z += g.part_z[w0 + i];
    n += g.part_tokens[w0 + i];
  }
  *reinterpret_cast<values *>(&s_prob[tid * VEC]) = p;
  *reinterpret_cast<numbers *>(&s_counts[tid * VEC]) = c;
  __syncthreads();
  double dot = 0.0;
  if (tid < g.E) {
    float sum = 0.0f;
    int32_t count = 0;
    for (int r = 0; r < rows; ++r) {
      sum += s_prob[r * cols * VEC + tid];
      count += s_counts[r * cols * VEC + tid];
    }
    g.prob[int64_t(s) * g.E + tid] = sum;
    g.counts[int64_t(s) * g.E + tid] = count;
    dot = double(sum) * double(count);
  }
  z = wave_sum(z);
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    n += __shfl_xor(n, o);
    dot += __shfl_xor(dot, o);
  }
  if (lane == 0) {
    s_z[wave] = z;
    s_n[wave] = n;
    s_dot[wave] = dot;
  }
  __syncthreads();
  if (tid) return;
  Total t{0, 0.0f, 0.0};
  for (int i = 0; i < kJoinThreads / 64; ++i) {
    t.n += s_n[i];
    t.z += s_z[i];
    t.dot += s_dot[i];
  }
  write_losses(g, s, t);
}

// The gradient: 256 / L tokens a workgroup.
template <int L, int PER, int VEC>
__global__ __launch_bounds__(256) void balance_bwd_kernel(BalanceArgs g) {
  using R = Row<L, PER, VEC>;
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t t0 = int64_t(blockIdx.x) * (256 / L), t = t0 + tid / L;
  const int64_t at = min(t, g.T - 1) * g.E;
  R row, out;
  row.load(g.logits + at, g.E, -INFINITY);
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int q = 0; q < VEC; ++q) out.v[i][q] = 0.0f;
  if (g.add) out.load(g.add + at, g.E, 0.0f);
  const float lse = g.lse[min(t, g.T - 1)];
  int s = 0;
  if (g.cu) {
    s = last_not_above(g.S, t0, lane, [&](int i) { return int64_t(first_token(g, i)); });
    while (s + 1 < g.S && first_token(g, s + 1) <= t) ++s;
  }
  float top;
  const float sum = row.exponentials(top);
  const float inv = 1.0f / sum;
  R c;
  float dot = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = R::column(i);
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
      row.v[i][q] *= inv;
      c.v[i][q] = 0.0f;
      if (e < g.E) c.v[i][q] = float(g.counts[int64_t(s) * g.E + e + q]);
      dot += c.v[i][q] * row.v[i][q];
    }
  }
  dot = token_sum<L>(dot);
  if (t >= g.T) return;
  if (!(lse == -INFINITY)) {
    const double n = double(g.tokens[s]);
    const double per = n > 0.0 ? 1.0 / n : 0.0;
    const float gl = g.grad_loss ? float(double(g.grad_loss[s]) * per * per * (double(g.E) / double(g.k))) : 0.0f;
    const float gz = g.grad_z ? float(2.0 * per * double(g.grad_z[s])) * lse : 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
      for (int q = 0; q < VEC; ++q) out.v[i][q] += row.v[i][q] * (gl * (c.v[i][q] - dot) + gz);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (R::column(i) < g.E) store_row<VEC>(g.grad + at + R::column(i), out.v[i]);
}

// An empty batch: nothing was counted.
__global__ __launch_bounds__(256) void balance_empty_kernel(BalanceArgs g) {
  const int64_t n = int64_t(g.S) * g.E;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
    g.prob[i] = 0.0f;
    g.counts[i] = 0;
    if (i < g.S) {
      g.tokens[i] = 0;
      g.loss[i] = 0.0f;
      g.z[i] = 0.0f;
    }
  }
}

// 16 lanes a token up to 256 experts, 64 beyond: a lane holds 16 experts at most.
template <typename F>
hipError_t by_experts(int E, F go) {
  if (E % 4 == 0) {
    if (E <= 64)
      go(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{}, std::integral_constant<int, 4>{});
    else if (E <= 128)
      go(std::integral_constant<int, 16>{}, std::integral_constant<int, 2>{}, std::integral_constant<int, 4>{});
    else if (E <= 256)
      go(std::integral_constant<int, 16>{}, std::integral_constant<int, 4>{}, std::integral_constant<int, 4>{});
    else if (E <= 512)
      go(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{}, std::integral_constant<int, 4>{});
    else
      go(std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{}, std::integral_constant<int, 4>{});
  } else if (E <= 64) {
    go(std::integral_constant<int, 16>{}, std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
  } else if (E <= 256) {
    go(std::integral_constant<int, 16>{}, std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
  } else {
    go(std::integral_constant<int, 64>{}, std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace e4b

using namespace e4b;

#define E4B_TRY(expr)                             \
  do {                                            \
    if ((expr) != hipSuccess) return E4B_ERR_HIP; \
  } while (0)

extern "C" size_t e4b_moe_balance_workspace_bytes(const e4b_balance *b) {
  BalanceArgs a;
  return plan_balance(b, &a) == E4B_OK ? balance_ws_bytes(a) : 0;
}

extern "C" e4b_status e4b_moe_balance(const e4b_balance *b, const float *logits, const int32_t *topk_idx,
                                      int32_t *counts, int32_t *tokens, float *prob, float *loss, float *z_loss,
                                      float *lse, void *ws, size_t ws_bytes, hipStream_t stream) {
  BalanceArgs a;
  const e4b_status s = plan_balance(b, &a);
  if (s != E4B_OK) return s;
  if (!counts || !tokens || !prob || !loss || !z_loss) return E4B_ERR_NULL;
  if (a.T && (!logits || !topk_idx || !lse)) return E4B_ERR_NULL;
  const size_t need = balance_ws_bytes(a);
  if (need && !ws) return E4B_ERR_NULL;
  if (ws_bytes < need) return E4B_ERR_WORKSPACE;
  if (!aligned16(logits) || !aligned16(topk_idx) || !aligned16(counts) || !aligned16(tokens) || !aligned16(prob) ||
      !aligned16(loss) || !aligned16(z_loss) || !aligned16(lse) || !aligned16(ws))
    return E4B_ERR_ALIGN;
  a.logits = logits;
  a.idx = topk_idx;
  a.counts = counts;
  a.tokens = tokens;
  a.prob = prob;
  a.loss = loss;
  a.z = z_loss;
  a.lse = lse;
  if (a.T == 0) {
    const int64_t n = (int64_t(a.S) * a.E + 255) / 256;
    hipLaunchKernelGGL(balance_empty_kernel, dim3(uint32_t(n < 1024 ? n : 1024)), dim3(256), 0, stream, a);
    E4B_TRY(hipGetLastError());
    return E4B_OK;
  }
  if (!need) {
    E4B_TRY(by_experts(a.E, [&](auto l, auto per, auto vec) {
      hipLaunchKernelGGL((balance_kernel<l(), per(), vec(), true>), dim3(1), dim3(balance_threads(true)), 0, stream, a);
    }));
    return E4B_OK;
  }
  char *w = static_cast<char *>(ws);
  a.part_prob = reinterpret_cast<float *>(w);
  a.part_counts = reinterpret_cast<int32_t *>(w) + a.slots * a.E;
  w += (size_t(a.slots) * size_t(a.E) * 8 + 255) / 256 * 256;
  a.part_z = reinterpret_cast<float *>(w);
  a.part_tokens = reinterpret_cast<int32_t *>(w) + a.slots;
  const int64_t grid = a.slots + (a.cu ? (a.T + balance_threads(false) - 1) / balance_threads(false) : 0);
  E4B_TRY(by_experts(a.E, [&](auto l, auto per, auto vec) {
    hipLaunchKernelGGL((balance_kernel<l(), per(), vec(), false>), dim3(uint32_t(grid)),
                       dim3(balance_threads(false)), 0, stream, a);
  }));
  const int vec = a.E % 4 == 0 ? 4 : 1;
  int cols = 1;
  while (cols * vec < a.E) cols *= 2;
  if (vec == 4)
    hipLaunchKernelGGL(balance_join_kernel<4>, dim3(uint32_t(a.S)), dim3(kJoinThreads), 0, stream, a, cols);
  else
    hipLaunchKernelGGL(balance_join_kernel<1>, dim3(uint32_t(a.S)), dim3(kJoinThreads), 0, stream, a, cols);
  E4B_TRY(hipGetLastError());
  return E4B_OK;
}

extern "C" e4b_status e4b_moe_balance_backward(const e4b_balance *b, const float *logits, const int32_t *counts,
                                               const int32_t *tokens, const float *lse, const float *grad_loss,
                                               const float *grad_z, const float *add, float *grad_logits,
                                               hipStream_t stream) {
  BalanceArgs a;
  const e4b_status s = plan_balance(b, &a);
  if (s != E4B_OK || a.T == 0) return s;
  if (!logits || !counts || !tokens || !lse || !grad_logits) return E4B_ERR_NULL;
  if (!aligned16(logits) || !aligned16(counts) || !aligned16(tokens) || !aligned16(lse) || !aligned16(grad_loss) ||
      !aligned16(grad_z) || !aligned16(add) || !aligned16(grad_logits))
    return E4B_ERR_ALIGN;
  a.logits = logits;
  a.counts = const_cast<int32_t *>(counts);
  a.tokens = const_cast<int32_t *>(tokens);
  a.lse = const_cast<float *>(lse);
  a.grad_loss = grad_loss;
  a.grad_z = grad_z;
  a.add = add;
  a.grad = grad_logits;
  E4B_TRY(by_experts(a.E, [&](auto l, auto per, auto vec) {
    constexpr int64_t tokens_each = 256 / l();
    hipLaunchKernelGGL((balance_bwd_kernel<l(), per(), vec()>), dim3(uint32_t((a.T + tokens_each - 1) / tokens_each)),
                       dim3(256), 0, stream, a);
  }));
  return E4B_OK;
}
