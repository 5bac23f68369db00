// norm.hip -- the norm after a block, its gate and residual scale, and the
// norm before the next block, in one pass over the rows, and their gradients
// in another.
//
// Row by row, with N(v) = v / sqrt(mean(v^2) + eps), s the residual scale and
// g a gate per token or per channel (1 without one):
//   u = N(y) w_post (or y)     r = x + s g u     h = N(r) w_pre
// Gradients, with a = s g du/dN-side factors and n = N(r), m = N(y):
//   c = grad_h w_pre                      grad_w_pre  = sum_t grad_h n
//   dr = grad_r + rstd_r (c - n mean(c n))          = grad_x
//   du = s g dr                           grad_w_post = sum_t du m
//   grad_y = rstd_y (b - m mean(b m)), b = du w_post   (or du)
//   grad_g = s sum(dr u) over the row (token gate) or over t (channel gate)
// A row is held in registers by TPR threads, VEC C elements each, so every
// tensor is read once and written once: HBM bounds both kernels. Statistics,
// sums and h's and the gradients' arithmetic are fp32; h comes from the
// unrounded r. r is not stored for the backward: it is rebuilt from x, y and
// rstd_y, which are read anyway.
#include "kernels.h"
#include "plan_block.h"
#include "rowvec.h"

namespace e4b {

namespace {

constexpr int kNormThreads = 512;
constexpr int kLongThreads = 1024;  // norm_bwd_threads of a row beyond 4096 columns
static_assert(kNormMaxH == 16 * kLongThreads, "16 elements a thread hold the longest row");

// Sum of N values over each group of TPR threads (whole waves), the same on
// every thread. `red` holds N floats per wave and is free again on return.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (TPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[wave][i] = v[i];
    __syncthreads();
    constexpr int kW = TPR / 64;
    const int w0 = wave / kW * kW;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.0f;
#pragma unroll
      for (int q = 0; q < kW; ++q) v[i] += red[w0 + q][i];
    }
    __syncthreads();
  }
}

// Rows addressed as buffers of their own length, which return zeros and drop stores past it.
typedef __amdgpu_buffer_rsrc_t buffer_t;

// `n` elements from p as a buffer; without p an empty one
template <typename T>
__device__ __forceinline__ buffer_t buffer_of(const T *p, int n) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<T *>(p), 0, p ? n * int(sizeof(T)) : 0, 0x00027000);
}
// the VEC elements from h
template <int VEC>
__device__ __forceinline__ void buffer_row(buffer_t b, int h, float (&f)[VEC]) {
  if constexpr (VEC == 8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x4 v = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(b, h * 4 + 16 * i, 0, 0));
#pragma unroll
      for (int q = 0; q < 4; ++q) f[4 * i + q] = v[q];
    }
  } else {
    f[0] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(b, h * 4, 0, 0));
  }
}
template <int VEC>
__device__ __forceinline__ void buffer_fetch(buffer_t b, int h, Raw<float, VEC> &r) {
  buffer_row<VEC>(b, h, r.v);
}
__device__ __forceinline__ void buffer_fetch(buffer_t b, int h, Raw<bf16_t, 8> &r) {
  r.v = __builtin_amdgcn_raw_buffer_load_b128(b, h * 2, 0, 0);
}
__device__ __forceinline__ void buffer_fetch(buffer_t b, int h, Raw<bf16_t, 1> &r) {
  r.v = __builtin_amdgcn_raw_buffer_load_b16(b, h * 2, 0, 0);
}
template <typename T, int VEC>
__device__ __forceinline__ void buffer_store(buffer_t b, int h, const float (&f)[VEC]) {
  if constexpr (sizeof(T) == 2 && VEC == 8) {
    __builtin_amdgcn_raw_buffer_store_b128(u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                                 pack_bf16x2(f[6], f[7])},
                                           b, h * 2, 0, 0);
  } else if constexpr (sizeof(T) == 2) {
    __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16(f[0]), b, h * 2, 0, 0);
  } else if constexpr (VEC == 8) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      __builtin_amdgcn_raw_buffer_store_b128(
          __builtin_bit_cast(u32x4, f32x4{f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]}), b, h * 4 + 16 * i, 0, 0);
  } else {
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, f[0]), b, h * 4, 0, 0);
  }
}

// the same value, from which the compiler makes its offsets here and does not hold them
// from elsewhere
__device__ __forceinline__ int here(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// One group of TPR threads per row; piece c of a thread is the VEC elements
// from (c TPR + thread) VEC on, so a wave's accesses are consecutive.
// Single elements (lengths that no 16-byte access divides), 32 to a thread, come from the
// rows as buffers, piece by piece as far as the row goes: a guard and an address for
// each took 141 registers, so one workgroup a CU (10860 x 12358 fp32 without weights
// 852 us, 492 so; 4096 x 8191 bf16 206 and 98).
template <typename X, int TPR, int VEC, int C>
__global__ __launch_bounds__(kNormThreads) void norm_fwd_kernel(NormArgs a) {
  __shared__ float red[kNormThreads / 64][1];
  constexpr int R = kNormThreads / TPR;
  constexpr bool kBuffer = VEC == 1 && C > 8;
  const int th = threadIdx.x % TPR;
  const int64_t t = int64_t(blockIdx.x) * R + __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
  const bool on = t < a.T;
  const int64_t row = on ? t * a.H : 0;
  // a row of a tensor, or nothing; the VEC elements from h of it
  auto row_of = [&](auto *p) { return buffer_of(on && p ? p + row : p, on ? a.H : 0); };
  auto load = [&](auto *p, buffer_t b, int h, float(&f)[VEC]) {
    if constexpr (!kBuffer)
      load_row<VEC>(p + h, f);
    else if constexpr (sizeof(*p) == 4)
      buffer_row<VEC>(b, h, f);
    else
      f[0] = bf16_to_f32(__builtin_amdgcn_raw_buffer_load_b16(b, h * 2, 0, 0));
  };
  const X *px = static_cast<const X *>(a.x);
  const bf16_t *py = static_cast<const bf16_t *>(a.y);
  X *pr = static_cast<X *>(a.r);
  bf16_t *ph = static_cast<bf16_t *>(a.h);
  const buffer_t bx = row_of(px), by = row_of(py), br = row_of(pr), bh = row_of(ph);
  const buffer_t b_post = buffer_of(a.w_post, a.H), b_pre = buffer_of(a.w_pre, a.H);
  const buffer_t b_gate = buffer_of(a.gate_channel, a.H);
  float x[C][VEC], y[C][VEC];
  int tv = kBuffer ? here(th) : th;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int h = (c * TPR + tv) * VEC;
#pragma unroll
    for (int q = 0; q < VEC; ++q) x[c][q] = y[c][q] = 0.0f;
    if (kBuffer ? c * TPR < a.H : on && h < a.H) {
      load(px + row, bx, h, x[c]);
      if (a.y) load(py + row, by, h, y[c]);
    }
  }
  const float inv = 1.0f / float(a.H);
  if (a.y) {
    float f = a.scale;
    if (a.w_post) {
      float ss[1] = {0.0f};
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int q = 0; q < VEC; ++q) ss[0] += y[c][q] * y[c][q];
      row_sums<TPR, 1>(ss, red);
      const float rs = 1.0f / sqrtf(ss[0] * inv + a.eps);
      if (on && th == 0) a.rstd_y[t] = rs;
      f *= rs;
    }
    if (a.gate_token && on) f *= a.gate_token[t];
    if (kBuffer) tv = here(th);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int h = (c * TPR + tv) * VEC;
      if (kBuffer ? c * TPR >= a.H : !on || h >= a.H) continue;
      float w[VEC], g[VEC];
      if (a.w_post) load(a.w_post, b_post, h, w);
      if (a.gate_channel) load(a.gate_channel, b_gate, h, g);
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        float u = f * y[c][q];
        if (a.w_post) u *= w[q];
        if (a.gate_channel) u *= g[q];
        x[c][q] += u;
      }
      if constexpr (kBuffer)
        buffer_store<X, VEC>(br, h, x[c]);
      else
        store_row<VEC>(pr + row + h, x[c]);
    }
  }
  if (a.w_pre) {
    float ss[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int q = 0; q < VEC; ++q) ss[0] += x[c][q] * x[c][q];
    row_sums<TPR, 1>(ss, red);
    const float rs = 1.0f / sqrtf(ss[0] * inv + a.eps);
    if (on && th == 0) a.rstd_r[t] = rs;
    if (kBuffer) tv = here(th);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int h = (c * TPR + tv) * VEC;
      if (kBuffer ? c * TPR >= a.H : !on || h >= a.H) continue;
      float w[VEC];
      load(a.w_pre, b_pre, h, w);
#pragma unroll
      for (int q = 0; q < VEC; ++q) w[q] = x[c][q] * rs * w[q];
      if constexpr (kBuffer)
        buffer_store<bf16_t, VEC>(bh, h, w);
      else
        store_row<VEC>(ph + row + h, w);
    }
  }
}

// The backward. The three row sums it needs are taken at once: with
// v = the factor of dr in the gate / post-norm products (u for a token gate,
// else s g u), dr = grad_r + rstd_r (c - n m1) gives
//   sum dr v = sum (grad_r + rstd_r c) v - rstd_r m1 sum n v,   m1 = mean(c n).
// Rows of up to 4096 columns: a workgroup walks rows blockIdx.x R, + gridDim.x R, ...
// with tpr threads to a row (R = NT / tpr rows at a time) and 8 elements to a thread:
// each thread keeps its columns' weights and its share of the column gradients
// in registers, and the next rows' pieces, as stored, while it works on these. 32
// elements to a thread spilled 150 registers and took 59.6 us at 4096 x 2048
// bf16 and 326 us at 8191 x 4096 fp32. At the end the workgroup adds its rows' shares
// through LDS and writes one partial row; norm_cols_kernel adds those in order. The
// grid depends on the descriptor alone, so results are the same on every run.
template <typename X, int NT, int VEC, int C, bool CHANNEL>
__global__ __launch_bounds__(NT) void norm_bwd_kernel(NormArgs a) {
  constexpr int kE = VEC * C;
  __shared__ float red[2][NT / 64][3];
  __shared__ float cols[NT * kE];
  const int tpr = a.tpr, R = NT / tpr;
  const int th = threadIdx.x & (tpr - 1), grp = threadIdx.x / tpr;
  const int wave = threadIdx.x >> 6, waves = tpr >> 6, w0 = wave & ~(waves - 1);
  const float inv = 1.0f / float(a.H);
  const X *px = static_cast<const X *>(a.x), *pgr = static_cast<const X *>(a.grad_r);
  const bf16_t *py = static_cast<const bf16_t *>(a.y), *pgh = static_cast<const bf16_t *>(a.grad_h);
  const bool pre = a.w_pre != nullptr, post = a.w_post != nullptr;
  float s_pre[C][VEC], s_post[C][VEC], s_gate[C][VEC], wp[C][VEC], wq[C][VEC], gc[C][VEC];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int h = (c * tpr + th) * VEC;
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
      s_pre[c][q] = s_post[c][q] = s_gate[c][q] = wq[c][q] = 0.0f;
      wp[c][q] = gc[c][q] = 1.0f;
    }
    if (h < a.H) {
      if (post) load_row<VEC>(a.w_post + h, wp[c]);
      if (pre) load_row<VEC>(a.w_pre + h, wq[c]);
      if (CHANNEL) load_row<VEC>(a.gate_channel + h, gc[c]);
    }
  }
  struct Row {
    Raw<X, VEC> x[C], gr[C];
    Raw<bf16_t, VEC> y[C], gh[C];
    float rs_y, rs_r, gt;
  };
  auto fetch = [&](int64_t t, Row &f) {
    const bool on = t < a.T;
    const int64_t row = on ? t * a.H : 0;
    f.rs_y = post && on ? a.rstd_y[t] : 1.0f;
    f.rs_r = pre && on ? a.rstd_r[t] : 0.0f;
    f.gt = !CHANNEL && a.gate_token && on ? a.gate_token[t] : 1.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int h = (c * tpr + th) * VEC;
      const bool in = on && h < a.H;
      f.x[c].fetch(px + row + h, in && pre);
      f.y[c].fetch(py + row + h, in && py);
      f.gr[c].fetch(pgr + row + h, in && pgr);
      f.gh[c].fetch(pgh + row + h, in && pre);
    }
  };
  const int64_t step = int64_t(gridDim.x) * R;
  Row cur;
  fetch(int64_t(blockIdx.x) * R + grp, cur);
  int turn = 0;
  for (int64_t t0 = int64_t(blockIdx.x) * R; t0 < a.T; t0 += step, turn ^= 1) {
    const int64_t t = t0 + grp;
    const bool on = t < a.T;
    const int64_t row = on ? t * a.H : 0;
    const float rs_y = cur.rs_y, rs_r = cur.rs_r, sg = a.scale * cur.gt;
    // m = N(y) (or y), n = N(r), d = grad_r + rstd_r c; absent pieces are zeros
    float m[C][VEC], n[C][VEC], d[C][VEC];
    float sums[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float gh[VEC];
      cur.x[c].get(n[c]);
      cur.y[c].get(m[c]);
      cur.gr[c].get(d[c]);
      cur.gh[c].get(gh);
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        m[c][q] *= rs_y;
        const float v = m[c][q] * wp[c][q] * (CHANNEL ? gc[c][q] : 1.0f);  // u, or g u
        // (without a pre-norm nothing of r reaches a gradient, not even as 0 times an infinity)
        n[c][q] = pre ? (n[c][q] + sg * v) * rs_r : 0.0f;
        const float cc = gh[q] * wq[c][q];
        sums[0] += cc * n[c][q];
        sums[2] += pre ? n[c][q] * v : 0.0f;
        d[c][q] += rs_r * cc;
        s_pre[c][q] += gh[q] * n[c][q];
        sums[1] += d[c][q] * v;
      }
    }
    // the next rows are on their way while this one's sums meet
    fetch(t + step, cur);
#pragma unroll
    for (int i = 0; i < 3; ++i) sums[i] = wave_sum(sums[i]);
    if (waves > 1) {
      // two buffers in turn: one barrier orders both the writes and the next turn's
      if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < 3; ++i) red[turn][wave][i] = sums[i];
      __syncthreads();
      sums[0] = sums[1] = sums[2] = 0.0f;
      for (int q = 0; q < waves; ++q)
#pragma unroll
        for (int i = 0; i < 3; ++i) sums[i] += red[turn][w0 + q][i];
    }
    const float m1 = rs_r * sums[0] * inv;    // times n: what dr loses
    const float dv = sums[1] - m1 * sums[2];  // sum over the row of dr v
    if (!CHANNEL && a.gate_token && a.grad_gate && on && th == 0) a.grad_gate[t] = a.scale * dv;
    // mean of b m: b m = s g_t g_h w_post dr m = s g_t (dr v)
    const float m2 = post ? sg * dv * inv : 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int h = (c * tpr + th) * VEC;
      float o[VEC];
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        const float dr = d[c][q] - m1 * n[c][q];
        const float du = sg * dr * (CHANNEL ? gc[c][q] : 1.0f);
        if (CHANNEL) s_gate[c][q] += a.scale * dr * (m[c][q] * wp[c][q]);
        s_post[c][q] += du * m[c][q];
        d[c][q] = dr;
        o[q] = post ? rs_y * (du * wp[c][q] - m[c][q] * m2) : du;
      }
      if (on && h < a.H) {
        store_row<VEC>(static_cast<X *>(a.grad_x) + row + h, d[c]);
        if (py) store_row<VEC>(static_cast<bf16_t *>(a.grad_y) + row + h, o);
      }
    }
  }
  // this workgroup's share of the column sums
  auto put = [&](const float(&s)[C][VEC], float *out) {
    if (!out) return;
    __syncthreads();
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int q = 0; q < VEC; ++q) cols[grp * (tpr * kE) + (c * tpr + th) * VEC + q] = s[c][q];
    __syncthreads();
    for (int h = threadIdx.x; h < a.H; h += NT) {
      float v = 0.0f;
      for (int r = 0; r < R; ++r) v += cols[r * (tpr * kE) + h];
      out[int64_t(blockIdx.x) * a.H + h] = v;
    }
  };
  put(s_pre, a.part_pre);
  put(s_post, a.part_post);
  if (CHANNEL) put(s_gate, a.part_gate);
}

// The same for rows beyond 4096 columns: the whole workgroup takes one row, 8 elements to
// a thread, 16 beyond 8192. A lane of 1024 threads has 128 registers, too few for what
// the kernel above holds (it spilled up to 473 here, and some calls were slower than
// elementary operations), so
//   * the row is kept as stored, and m, n, d are computed from it twice, before and
//     after the row sums (hide() keeps the compiler from holding them instead);
//   * column sums that registers have no room for lie in LDS, each column its own
//     thread's: 8 elements with a channel gate all three, 16 elements two;
//   * rows are addressed as buffers of their own length, which return zeros and drop
//     stores past it: no guards, and an offset in place of an address a tensor;
//   * at 16 elements the weights are read again from L2 for each row and half, and the
//     next row is not fetched ahead.
// Forward and backward in us, in parentheses with the kernel above: 1024 x 16384 bf16
// token gate 102 (202), fp32 channel gate 175 (423), 4096 x 8192 fp32 channel gate 229
// (331), bf16 token gate 156 (161), 1024 x 16383 fp32 channel gate 168 (675).
// VEC elements of x, y, grad_r and grad_h as stored; single bf16 elements two to a register
template <typename X, int VEC>
struct Stored {
  Raw<X, VEC> x, gr;
  Raw<bf16_t, VEC> y, gh;
  __device__ __forceinline__ void fetch(buffer_t bx, buffer_t by, buffer_t br, buffer_t bh, int h) {
    buffer_fetch(bx, h, x);
    buffer_fetch(by, h, y);
    buffer_fetch(br, h, gr);
    buffer_fetch(bh, h, gh);
    if constexpr (VEC == 1) {
      y.v |= gh.v << 16;
      if constexpr (sizeof(X) == 2) x.v |= gr.v << 16;
    }
  }
  __device__ __forceinline__ void hide() {
    x.hide();
    y.hide();
    if (VEC > 1 || sizeof(X) > 2) gr.hide();
    if (VEC > 1) gh.hide();
  }
  __device__ __forceinline__ void get(float (&fx)[VEC], float (&fy)[VEC], float (&fr)[VEC], float (&fh)[VEC]) const {
    if constexpr (VEC == 1) {
      fy[0] = bf16_lo(y.v);
      fh[0] = bf16_hi(y.v);
      if constexpr (sizeof(X) == 2) {
        fx[0] = bf16_lo(x.v);
        fr[0] = bf16_hi(x.v);
        return;
      }
    } else {
      y.get(fy);
      gh.get(fh);
    }
    if constexpr (VEC > 1 || sizeof(X) > 2) {
      x.get(fx);
      gr.get(fr);
    }
  }
};

template <typename X, int VEC, int C, bool CHANNEL>
__global__ __launch_bounds__(kLongThreads) void norm_bwd_long_kernel(NormArgs a) {
  constexpr int NT = kLongThreads, kE = VEC * C;
  constexpr bool kAhead = kE <= 8;  // weights held, the next row fetched ahead
  // where the column sums are: in LDS where that is not one of the two
  constexpr bool kPreLds = CHANNEL ? kE <= 8 : kE > 8, kPostLds = CHANNEL || kE > 8;
  __shared__ float red[2][NT / 64][3];
  __shared__ __attribute__((aligned(16))) float s_gate[CHANNEL ? NT * kE : 1], s_post[kPostLds ? NT * kE : 1],
      s_pre[kPreLds ? NT * kE : 1];
  const int th = threadIdx.x, wave = threadIdx.x >> 6, H = a.H;
  const float inv = 1.0f / float(H);
  const bool pre = a.w_pre != nullptr, post = a.w_post != nullptr;
  const buffer_t b_post = buffer_of(a.w_post, H), b_pre = buffer_of(a.w_pre, H);
  const buffer_t b_gate = buffer_of(a.gate_channel, H);
  struct Weights {
    float p[VEC], q[VEC], g[VEC];  // post, pre, gate
  };
  auto weights = [&](int h, Weights &w) {
    buffer_row<VEC>(b_post, h, w.p);
    buffer_row<VEC>(b_pre, h, w.q);
    if (CHANNEL) buffer_row<VEC>(b_gate, h, w.g);
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
      w.p[q] = post ? w.p[q] : 1.0f;
      if (!CHANNEL) w.g[q] = 1.0f;
    }
  };
  Weights held[kAhead ? C : 1];
  float r_pre[kPreLds ? 1 : C][VEC], r_post[kPostLds ? 1 : C][VEC];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int h = (c * NT + th) * VEC;
    if constexpr (kAhead) weights(h, held[c]);
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
      if constexpr (CHANNEL) s_gate[h + q] = 0.0f;
      if constexpr (kPostLds)
        s_post[h + q] = 0.0f;
      else
        r_post[c][q] = 0.0f;
      if constexpr (kPreLds)
        s_pre[h + q] = 0.0f;
      else
        r_pre[c][q] = 0.0f;
    }
  }
  struct Row {
    Stored<X, VEC> e[C];
    float rs_y, rs_r, gt;
  };
  // element t H of a tensor, or nothing
  auto row_of = [&](const void *p, auto type, int64_t t, bool in) {
    typedef decltype(type) T;
    return buffer_of(in && p ? static_cast<const T *>(p) + t * H : static_cast<const T *>(nullptr), H);
  };
  auto fetch = [&](int64_t t, Row &f) {
    const bool on = t < a.T;
    f.rs_y = post && on ? a.rstd_y[t] : 1.0f;
    f.rs_r = pre && on ? a.rstd_r[t] : 0.0f;
    f.gt = !CHANNEL && a.gate_token && on ? a.gate_token[t] : 1.0f;
    const buffer_t bx = row_of(a.x, X{}, t, on && pre), by = row_of(a.y, bf16_t{}, t, on);
    const buffer_t br = row_of(a.grad_r, X{}, t, on), bh = row_of(a.grad_h, bf16_t{}, t, on && pre);
    const int tv = here(th);
#pragma unroll
    for (int c = 0; c < C; ++c) f.e[c].fetch(bx, by, br, bh, (c * NT + tv) * VEC);
  };
  // (the weights of 4 single elements at a time are on their way, not those of 16)
  auto apart = [](int c) {
    if (kE > 8 && VEC == 1 && c % 4 == 3) {
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  Row cur, nxt;
  if constexpr (kAhead) fetch(blockIdx.x, nxt);
  const bool reduce = pre || post || (!CHANNEL && a.grad_gate);  // what needs the row sums
  int turn = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
    if constexpr (kAhead)
      cur = nxt;
    else
      fetch(t, cur);
    const float rs_y = cur.rs_y, rs_r = cur.rs_r, sg = a.scale * cur.gt;
    // element q of piece c: m = N(y) (or y), n = N(r), d = grad_r + rstd_r c, v = u or g u, cc = c
    struct Piece {
      float m[VEC], n[VEC], d[VEC], v[VEC], cc[VEC], gh[VEC];
    };
    auto piece = [&](int c, const Weights &w, Piece &e) {
      cur.e[c].get(e.n, e.m, e.d, e.gh);
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        e.m[q] *= rs_y;
        e.v[q] = e.m[q] * w.p[q] * (CHANNEL ? w.g[q] : 1.0f);
        // (without a pre-norm nothing of r reaches a gradient, not even as 0 times an infinity)
        e.n[q] = pre ? (e.n[q] + sg * e.v[q]) * rs_r : 0.0f;
        e.cc[q] = e.gh[q] * w.q[q];
        e.d[q] += rs_r * e.cc[q];
      }
    };
    float sums[3] = {0.0f, 0.0f, 0.0f};
    int tv = here(th);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int h = (c * NT + tv) * VEC;
      Piece e;
      Weights w;
      if constexpr (kAhead)
        w = held[c];
      else
        weights(h, w);
      piece(c, w, e);
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        sums[0] += e.cc[q] * e.n[q];
        sums[2] += pre ? e.n[q] * e.v[q] : 0.0f;
        if constexpr (!kPreLds)
          r_pre[c][q] += e.gh[q] * e.n[q];
        else
          s_pre[h + q] += e.gh[q] * e.n[q];
        sums[1] += e.d[q] * e.v[q];
      }
      apart(c);
    }
    if constexpr (kAhead) fetch(t + gridDim.x, nxt);
    if (reduce) {
#pragma unroll
      for (int i = 0; i < 3; ++i) sums[i] = wave_sum(sums[i]);
      // two buffers in turn: one barrier orders both the writes and the next turn's
      if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < 3; ++i) red[turn][wave][i] = sums[i];
      __syncthreads();
      sums[0] = sums[1] = sums[2] = 0.0f;
      for (int q = 0; q < NT / 64; ++q)
#pragma unroll
        for (int i = 0; i < 3; ++i) sums[i] += red[turn][q][i];
    }
    const float m1 = rs_r * sums[0] * inv;    // times n: what dr loses
    const float dv = sums[1] - m1 * sums[2];  // sum over the row of dr v
    if (!CHANNEL && a.gate_token && a.grad_gate && th == 0) a.grad_gate[t] = a.scale * dv;
    const float m2 = post ? sg * dv * inv : 0.0f;  // mean of b m: b m = s g_t (dr v)
    const buffer_t bx = row_of(a.grad_x, X{}, t, true), by = row_of(a.grad_y, bf16_t{}, t, a.y != nullptr);
    tv = here(th);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int h = (c * NT + tv) * VEC;
      cur.e[c].hide();
      Piece e;
      Weights w;
      if constexpr (kAhead)
        w = held[c];
      else
        weights(h, w);
      piece(c, w, e);
      float o[VEC];
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        const float dr = e.d[q] - m1 * e.n[q];
        const float du = sg * dr * (CHANNEL ? w.g[q] : 1.0f);
        if constexpr (CHANNEL)
          s_gate[h + q] += a.scale * dr * (e.m[q] * w.p[q]);
        if constexpr (!kPostLds)
          r_post[c][q] += du * e.m[q];
        else
          s_post[h + q] += du * e.m[q];
        e.d[q] = dr;
        o[q] = post ? rs_y * (du * w.p[q] - e.m[q] * m2) : du;
      }
      buffer_store<X, VEC>(bx, h, e.d);
      buffer_store<bf16_t, VEC>(by, h, o);
      apart(c);
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
      const int h = (c * NT + th) * VEC + q;
      if (h >= H) continue;
      const int64_t at = int64_t(blockIdx.x) * H + h;
      if (a.part_pre) a.part_pre[at] = kPreLds ? s_pre[kPreLds ? h : 0] : r_pre[kPreLds ? 0 : c][q];
      if (a.part_post) a.part_post[at] = kPostLds ? s_post[kPostLds ? h : 0] : r_post[kPostLds ? 0 : c][q];
      if constexpr (CHANNEL)
        if (a.part_gate) a.part_gate[at] = s_gate[h];
    }
}

// out[h] = sum over the n partial rows, 16 interleaved runs added in a fixed order.
__global__ __launch_bounds__(1024) void norm_cols_kernel(const float *__restrict__ p0, const float *__restrict__ p1,
                                                         const float *__restrict__ p2, float *__restrict__ o0,
                                                         float *__restrict__ o1, float *__restrict__ o2, int n, int H) {
  __shared__ float s[16][64];
  const float *p = blockIdx.y == 0 ? p0 : blockIdx.y == 1 ? p1 : p2;
  float *o = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
  if (!o) return;
  const int lane = threadIdx.x & 63, run = threadIdx.x >> 6;
  const int h = blockIdx.x * 64 + lane;
  float v = 0.0f;
  if (h < H)
#pragma unroll 16
    for (int i = run; i < n; i += 16) v += p[int64_t(i) * H + h];
  s[run][lane] = v;
  __syncthreads();
  if (run == 0 && h < H) {
    for (int r = 1; r < 16; ++r) v += s[r][lane];
    o[h] = v;
  }
}

template <typename X, int TPR, int VEC, int C>
hipError_t forward(const NormArgs &a, hipStream_t s) {
  constexpr int R = kNormThreads / TPR;
  hipLaunchKernelGGL((norm_fwd_kernel<X, TPR, VEC, C>), dim3(uint32_t((a.T + R - 1) / R)), dim3(kNormThreads), 0, s, a);
  return hipGetLastError();
}

template <typename X>
hipError_t forward_by_length(const NormArgs &a, hipStream_t s) {
  const int H = a.H;
  if (H % 8 == 0) {
    if (H <= 512) return forward<X, 64, 8, 1>(a, s);
    if (H <= 1024) return forward<X, 64, 8, 2>(a, s);
    if (H <= 2048) return forward<X, 64, 8, 4>(a, s);
    if (H <= 4096) return forward<X, 128, 8, 4>(a, s);
    if (H <= 8192) return forward<X, 256, 8, 4>(a, s);
    return forward<X, 512, 8, 4>(a, s);
  }
  if (H <= 512) return forward<X, 64, 1, 8>(a, s);
  if (H <= 2048) return forward<X, 64, 1, 32>(a, s);
  if (H <= 4096) return forward<X, 128, 1, 32>(a, s);
  if (H <= 8192) return forward<X, 256, 1, 32>(a, s);
  return forward<X, 512, 1, 32>(a, s);
}

template <typename X, int NT, int VEC, int C>
hipError_t backward(const NormArgs &a, hipStream_t s) {
  if (a.gate_channel)
    hipLaunchKernelGGL((norm_bwd_kernel<X, NT, VEC, C, true>), dim3(uint32_t(a.groups)), dim3(NT), 0, s, a);
  else
    hipLaunchKernelGGL((norm_bwd_kernel<X, NT, VEC, C, false>), dim3(uint32_t(a.groups)), dim3(NT), 0, s, a);
  return hipGetLastError();
}

template <typename X, int VEC, int C>
hipError_t backward_long(const NormArgs &a, hipStream_t s) {
  if (a.gate_channel)
    hipLaunchKernelGGL((norm_bwd_long_kernel<X, VEC, C, true>), dim3(uint32_t(a.groups)), dim3(kLongThreads), 0, s, a);
  else
    hipLaunchKernelGGL((norm_bwd_long_kernel<X, VEC, C, false>), dim3(uint32_t(a.groups)), dim3(kLongThreads), 0, s, a);
  return hipGetLastError();
}

template <typename X>
hipError_t backward_by_length(const NormArgs &a, hipStream_t s) {
  if (a.H % 8 == 0)
    return a.H <= 4096 ? backward<X, 512, 8, 1>(a, s) : a.H <= 8192 ? backward_long<X, 8, 1>(a, s) : backward_long<X, 8, 2>(a, s);
  return a.H <= 4096 ? backward<X, 512, 1, 8>(a, s) : a.H <= 8192 ? backward_long<X, 1, 8>(a, s) : backward_long<X, 1, 16>(a, s);
}

}  // namespace

hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t s) {
  return a.f32 ? forward_by_length<float>(a, s) : forward_by_length<bf16_t>(a, s);
}

hipError_t launch_norm_bwd(const NormArgs &a, hipStream_t s) {
  if (a.T) {
    const hipError_t e = a.f32 ? backward_by_length<float>(a, s) : backward_by_length<bf16_t>(a, s);
    if (e != hipSuccess) return e;
  }
  float *gate = a.gate_channel ? a.grad_gate : nullptr;
  if ((!a.grad_w_pre && !a.grad_w_post && !gate) || (a.T && a.groups == 1)) return hipSuccess;
  hipLaunchKernelGGL(norm_cols_kernel, dim3(uint32_t((a.H + 63) / 64), 3), dim3(1024), 0, s, a.part_pre, a.part_post,
                     a.part_gate, a.grad_w_pre, a.grad_w_post, gate, a.T ? a.groups : 0, a.H);
  return hipGetLastError();
}

}  // namespace e4b

using namespace e4b;

extern "C" e4b_status e4b_block_norm(const e4b_norm *n, const void *x, const void *y, void *r, void *h, float *rstd_y,
                                     float *rstd_r, hipStream_t stream) {
  NormArgs a{};
  const e4b_status st = plan_norm(n, y != nullptr || (n && n->T == 0), &a);
  if (st != E4B_OK || a.T == 0) return st;
  if (!x || (y && !r) || (a.w_post && !rstd_y) || (a.w_pre && (!h || !rstd_r))) return E4B_ERR_NULL;
  for (const void *p : {x, y, static_cast<const void *>(r), static_cast<const void *>(h),
                        static_cast<const void *>(rstd_y), static_cast<const void *>(rstd_r)})
    if (!aligned16(p)) return E4B_ERR_ALIGN;
  a.x = x;
  a.y = y;
  a.r = r;
  a.h = h;
  a.rstd_y = rstd_y;
  a.rstd_r = rstd_r;
  return launch_norm_fwd(a, stream) == hipSuccess ? E4B_OK : E4B_ERR_HIP;
}

extern "C" e4b_status e4b_block_norm_backward(const e4b_norm *n, const void *x, const void *y, const float *rstd_y,
                                              const float *rstd_r, const void *grad_r, const void *grad_h,
                                              void *grad_x, void *grad_y, float *grad_gate, float *grad_w_post,
                                              float *grad_w_pre, void *ws, size_t ws_bytes, hipStream_t stream) {
  NormArgs a{};
  const e4b_status st = plan_norm(n, y != nullptr || (n && n->T == 0), &a);
  if (st != E4B_OK) return st;
  // T = 0 still writes the (zero) column gradients
  if (a.T && (!x || !grad_x || (y && !grad_y) || (a.w_post && !rstd_y) || (a.w_pre && (!rstd_r || !grad_h)) ||
              (!a.w_pre && !grad_r)))
    return E4B_ERR_NULL;
  const bool g = a.gate_token || a.gate_channel;
  if ((grad_gate && !g) || (grad_w_post && !a.w_post) || (grad_w_pre && !a.w_pre)) return E4B_ERR_NULL;
  // what takes the workspace
  const bool columns = (grad_w_post || grad_w_pre || (grad_gate && a.gate_channel)) && norm_ws_bytes(a);
  if (a.T && columns && !ws) return E4B_ERR_NULL;
  if (a.T && columns && ws_bytes < norm_ws_bytes(a)) return E4B_ERR_WORKSPACE;
  for (const void *p :
       {x, y, static_cast<const void *>(rstd_y), static_cast<const void *>(rstd_r), grad_r, grad_h,
        static_cast<const void *>(grad_x), static_cast<const void *>(grad_y), static_cast<const void *>(grad_gate),
        static_cast<const void *>(grad_w_post), static_cast<const void *>(grad_w_pre), static_cast<const void *>(ws)})
    if (!aligned16(p)) return E4B_ERR_ALIGN;
  a.x = x;
  a.y = y;
  a.rstd_y = const_cast<float *>(rstd_y);
  a.rstd_r = const_cast<float *>(rstd_r);
  a.grad_r = grad_r;
  a.grad_h = grad_h;
  a.grad_x = grad_x;
  a.grad_y = grad_y;
  a.grad_gate = grad_gate;
  a.grad_w_post = grad_w_post;
  a.grad_w_pre = grad_w_pre;
  // the partial rows in the workspace's (at most) three arrays, 16-byte aligned or not: they
  // are read and written by single columns; one group's only row is the gradient itself
  float *w = static_cast<float *>(ws);
  const int64_t each = int64_t(a.groups) * a.H;
  const bool one = a.groups == 1;
  a.part_pre = grad_w_pre ? (one ? grad_w_pre : w) : nullptr;
  a.part_post = grad_w_post ? (one ? grad_w_post : w + each) : nullptr;
  a.part_gate = grad_gate && a.gate_channel ? (one ? grad_gate : w + 2 * each) : nullptr;
  return launch_norm_bwd(a, stream) == hipSuccess ? E4B_OK : E4B_ERR_HIP;
}

extern "C" size_t e4b_block_norm_workspace_bytes(const e4b_norm *n) {
  NormArgs a{};
  return plan_norm(n, true, &a) == E4B_OK ? norm_ws_bytes(a) : 0;
}
