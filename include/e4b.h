/*
 * e4b.h -- C ABI of the MI355X (gfx950) fused blockwise-4-bit Mixture-of-Experts
 * expert MLP: quantize / dequantize a fused expert stack, the routed SwiGLU
 * forward, and the frozen-base input gradient (dgrad).
 *
 * Sources (page titles; sections named per entry point below):
 *   [sdist]  experts4bit-qlora 0.1.0 source distribution, module
 *            experts4bit_qlora/_vendor/experts.py, class Experts4bit.
 *   [PR]     bitsandbytes pull request #1965, "Add Experts4bit for 4-bit
 *            quantization of fused MoE experts".
 *   [README] experts4bit-qlora 0.4.0 README (PyPI wheel metadata).
 *
 * Conventions shared by every call
 * --------------------------------
 * - Stacks are row-major [E, out, in] per expert ([sdist] class docstring):
 *   gate_up is [E, 2I, H] with rows 0..I-1 the gate and rows I..2I-1 the up
 *   projection; down is [E, H, I].
 * - Packed codes: uint8 [E, out*in/2], two 4-bit codes per byte, the even
 *   element of the flattened row-major [out, in] in the high nibble.
 * - absmax: fp32 [E, out*in/64], one scale per 64 consecutive elements of a
 *   row; in % 64 == 0 so a block never straddles a row or an expert
 *   ([sdist] Experts4bit.__init__ block-alignment check). absmax is always
 *   fp32 and the codebook is a library constant chosen by enum, never a
 *   caller buffer ([PR] "Dtype-cast safety" bullet).
 * - bf16 tensors are raw IEEE bfloat16 bit patterns (uint16).
 * - Every pointer argument except the `const e4b_stack*`/`const
 *   e4b_moe_layer*` descriptors (host memory, read during the call only) is
 *   a DEVICE pointer owned by the caller; the library never allocates or
 *   frees memory and keeps no state between calls beyond its code objects.
 * - Device buffers must be 16-byte aligned (E4B_ERR_ALIGN otherwise).
 * - Asynchrony: every call validates its arguments on the host, enqueues
 *   kernels on `stream` and returns; no call synchronizes. A non-OK status is
 *   returned synchronously and nothing is enqueued for validation errors.
 * - Errors follow the pages' fail-loudly rule ([README] support matrix
 *   "Unsupported" definition): a bad argument is reported, never ignored.
 *   T == 0 is a valid no-op.
 * - Device preconditions that are NOT checked: finite weights and logits;
 *   0 <= topk_idx < E when it is an input. An id outside [0, E) never leads
 *   to an out-of-bounds access: every kernel that reads ids treats it as
 *   expert 0, so the pair's result is meaningless but the call stays in
 *   bounds (the Python binding can check the ids first). Given ids may
 *   repeat an expert within a token: each slot is a pair of its own.
 */
#ifndef E4B_H
#define E4B_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  E4B_OK = 0,
  E4B_ERR_NULL = 1,      /* a required pointer is NULL */
  E4B_ERR_SHAPE = 2,     /* a dimension <= 0, in % 64 != 0, top_k not in [1, min(E, 32)],
                            E > 1024, inconsistent gate_up/down shapes, or a size too large */
  E4B_ERR_BLOCKSIZE = 3, /* blocksize != 64 (MXFP4: != 32) */
  E4B_ERR_CODEBOOK = 4,  /* unknown codebook, or gate_up/down codebooks differ */
  E4B_ERR_DTYPE = 5,     /* unknown output dtype */
  E4B_ERR_WORKSPACE = 6, /* workspace NULL or smaller than e4b_moe_workspace_bytes() */
  E4B_ERR_ALIGN = 7,     /* a device buffer is not 16-byte aligned */
  E4B_ERR_PATH = 8,      /* unknown path, or the decode path was asked for but does not apply (a BF16, INT8 or FP8 layer, T > 8, saved != NULL, or max(H, I) above 16384) */
  E4B_ERR_HIP = 9,       /* a kernel launch failed (hipGetLastError after the launch) */
  E4B_ERR_ACT = 10       /* unknown activation (e4b_act) */
} e4b_status;

/* MXFP4 = the MX storage the [0.31.1] project page names for gpt-oss experts
 * ("dequantised bit-identically") and for its native MXFP4 row, read as the
 * OCP Microscaling Formats (MX) v1.0 FP4 format: E2M1 codes (same code layout
 * and nibble order as FP4, unscaled magnitudes {0,.5,1,1.5,2,3,4,6}) with one
 * E8M0 scale 2^(s-127) per 32 consecutive elements of a row in `scales`
 * (uint8 [E, out*in/32]); blocksize 32, `absmax` unused. The dequantized
 * weight code * 2^(s-127) is exact in fp32 and bf16, so every path (grouped
 * forward, dgrad, decode GEMV, LoRA) runs on exactly the stored values.
 *
 * Storage modes. The 16-entry codebooks ([sdist] Experts4bit.__init__
 * quant_type "nf4"/"fp4"): NF4 = the NormalFloat-4 table of the QLoRA paper
 * (arXiv:2305.14314); FP4 = e2m1 (sign bit 3, magnitudes {0,.5,1,1.5,2,3,4,6}/6).
 * BF16 = the 16-bit passthrough lane of the [README] support matrix (the
 * reference baseline, no absmax buffer): `packed` holds the bf16 weight
 * [E, out*in] (two bytes per element, round-to-nearest-even of the fp32
 * weight), `absmax` is unused and may be NULL. A BF16 layer runs the grouped
 * path only (the decode GEMV reads 4-bit codes). */
/* Storage modes ([README] "Storage modes: the support matrix"): the 4-bit
 * codebooks NF4 and FP4 (two codes per byte), the bf16 passthrough lane, MXFP4
 * (E2M1 codes + E8M0 scales), and the 8-bit blockwise lanes INT8 (the
 * dynamic tree map) and FP8 (an E4M3 codebook), one code byte per element:
 * sign bit 7 | index into 128 ascending magnitudes from 0 to 1 (the tables
 * are defined in csrc/codebook8.h). The grouped GEMMs decode the code bytes
 * in their weight staging through a 256-entry table, as they decode the 4-bit
 * codes (bf16(fl32(value * absmax))); as on the pages, the 8-bit lanes have
 * no decode GEMV. */
typedef enum {
  E4B_CB_NF4 = 0,
  E4B_CB_FP4 = 1,
  E4B_CB_BF16 = 2,
  E4B_CB_MXFP4 = 3,
  E4B_CB_INT8 = 4,
  E4B_CB_FP8 = 5
} e4b_codebook;

typedef enum { E4B_F32 = 0, E4B_BF16 = 1 } e4b_dtype;

/* Forward path selection. AUTO = the decode dequant-GEMV path when T <= 8,
 * saved == NULL and the layer is a gated 4-bit one (NF4, FP4, MXFP4), else
 * the grouped MFMA path. MX8 = the MX forward of an
 * MXFP4 gated layer on gfx950's block-scaled MFMA ([0.31.1] native MXFP4
 * row): x and a = bf16(silu(g) * u) are converted per row to MXFP8 (E4M3, an
 * E8M0 scale per 32; the OCP MX v1.0 rule with emax 8: saturating,
 * round-to-nearest-even), so the result approximates the exact-weights
 * forward to about the E4M3 rounding (2^-4 relative per activation); it
 * needs H % 128 == 0, I % 128 == 0 and saved == NULL (E4B_ERR_PATH
 * otherwise). */
typedef enum {
  E4B_PATH_AUTO = 0,
  E4B_PATH_GROUPED = 1,
  E4B_PATH_DECODE = 2,
  E4B_PATH_MX8 = 3
} e4b_path;

/* One quantized stack (device pointers; the struct itself is host memory). */
typedef struct {
  const uint8_t *packed; /* [E, out*in/2]; BF16: [E, out*in] bf16; INT8, FP8: [E, out*in] codes */
  const float *absmax;   /* [E, out*in/64]; BF16, MXFP4: unused */
  int64_t E, out, in;
  int32_t blocksize; /* 64; MXFP4: 32 */
  int32_t codebook;  /* e4b_codebook */
  const uint8_t *scales; /* MXFP4: E8M0 [E, out*in/32]; other modes: unused */
} e4b_stack;

/* A MoE layer: gate_up (out = 2I, in = H) and down (out = H, in = I), same E,
 * same codebook ([README] "one module, one scheme"). A first stack of out = I
 * rows selects the ungated variant ([sdist] Experts4bit has_gate=False: a
 * plain up projection h, a = silu(h)); it runs the grouped path and takes no
 * LoRA adapters. */
typedef struct {
  e4b_stack gate_up;
  e4b_stack down;
} e4b_moe_layer;

/* Blockwise absmax quantization of an fp32 [E, out, in] stack.
 * [sdist] Experts4bit.from_float / _quantize_stack (per expert, blocksize 64,
 * no double quantization; [PR] "Non-goals" keeps absmax a plain fp32 buffer).
 * absmax = max |w| over each 64-block; code = nearest codebook entry to
 * w/absmax decided exactly (ties: NF4 lower code, FP4 smaller magnitude; FP4
 * sign bit = sign bit of w); an NF4 block of zeros stores code 7. INT8 and
 * FP8: the magnitude nearest |w|/absmax (ties: the smaller one), sign bit 7 =
 * sign bit of w, one code byte per element.
 *   w      : device fp32 [E, out, in], finite (unchecked)
 *   packed : device uint8 [E, out*in/2]; INT8, FP8: [E, out*in]   (written)
 *   absmax : device fp32  [E, out*in/64]  (written)
 * codebook E4B_CB_BF16 writes the bf16 rounding (nearest even) of w to
 * `packed` ([E, out*in] bf16) and leaves `absmax` (may be NULL) untouched.
 * Errors: NULL, SHAPE (E/out/in <= 0, in % 64 != 0), BLOCKSIZE, CODEBOOK,
 * ALIGN, HIP. */
e4b_status e4b_quantize_nf4(const float *w, int64_t E, int64_t out, int64_t in,
                            int32_t blocksize, int32_t codebook, uint8_t *packed,
                            float *absmax, hipStream_t stream);

/* MXFP4 conversion of an fp32 [E, out, in] stack (OCP MX v1.0, read for the
 * [0.31.1] project page's MXFP4 experts): per block of 32 consecutive
 * elements, shared exponent = floor(log2(max |w|)) - 2 clamped to
 * [-127, 127] (a block of zeros: -127), scale byte = shared + 127; each
 * element is w / 2^shared rounded to the nearest E2M1 value (ties to the even
 * mantissa, beyond 6 saturated), sign bit = sign bit of w.
 *   w      : device fp32 [E, out, in], finite (unchecked); in % 32 == 0
 *   packed : device uint8 [E, out*in/2]   (written)
 *   scales : device uint8 [E, out*in/32]  (written)
 * Errors: NULL, SHAPE, ALIGN, HIP. */
e4b_status e4b_quantize_mxfp4(const float *w, int64_t E, int64_t out, int64_t in, uint8_t *packed,
                              uint8_t *scales, hipStream_t stream);

/* MXFP8 conversion of bf16 activation rows, as the MX forward (E4B_PATH_MX8)
 * feeds them to the block-scaled MFMA: per block of 32 consecutive elements
 * of a row, shared exponent = floor(log2(max |x|)) - 8 clamped to
 * [-127, 127] (a block of zeros: -127), scale byte = shared + 127, element =
 * x / 2^shared rounded to E4M3 (nearest even, saturating at 448; sign bit 7).
 * Layout: codes [rows, K] with the two bytes of every element pair swapped
 * (byte 2p holds element 2p + 1), scales [rows, K/32].
 *   x_bf16 : device bf16 [rows, K]; K % 32 == 0
 * Errors: NULL, SHAPE, ALIGN, HIP. */
e4b_status e4b_mx8_rows(const void *x_bf16, int64_t rows, int64_t K, uint8_t *codes,
                        uint8_t *scales, hipStream_t stream);

/* Dequantize a whole stack: w_out[e, r, c] = fl32(code * absmax) (one fp32
 * rounding of the exact product), or its round-to-nearest-even bf16 when
 * dtype == E4B_BF16. [sdist] Experts4bit._dequantize_expert. A BF16 stack
 * gives its stored values (exact in fp32); an MXFP4 stack gives code *
 * 2^(s-127) (exact in both dtypes), and NaN for a scale of 255.
 *   st    : host descriptor of device buffers
 *   w_out : device [E, out, in] fp32 or bf16 (written)
 * Errors: NULL, SHAPE, BLOCKSIZE, CODEBOOK, DTYPE, ALIGN, HIP. */
e4b_status e4b_dequantize_nf4(const e4b_stack *st, int32_t dtype, void *w_out,
                              hipStream_t stream);

/* Asynchronous copy of one stored stack (packed codes or bf16 weights, and
 * the absmax when the mode has one) from `src` to `dst`, on `stream`
 * (hipMemcpyAsync: host-to-device from pinned host memory, or device-to-
 * device). It is the transfer of the layer-granular prefetch of the
 * [README] "Prefetched expert offload" bullet (decode with experts that
 * exceed device memory): the caller copies layer L+1 into a second set of
 * device buffers on a side stream while layer L computes, and orders the
 * two streams with events, so at most two layers are resident.
 *   dst, src : host descriptors; dst's buffers on the device, src's on the
 *              device or in pinned host memory; same E, out, in, blocksize
 *              and codebook
 * Errors: NULL, SHAPE (descriptors differ), BLOCKSIZE, CODEBOOK, ALIGN, HIP. */
e4b_status e4b_stack_copy_async(const e4b_stack *dst, const e4b_stack *src, hipStream_t stream);

/* Routed SwiGLU expert forward. [sdist] Experts4bit.forward: for each
 * (token t, slot j) with expert e = topk_idx[t, j],
 *   h = W_gu[e] x_t ; g = h[:I] ; u = h[I:] ; a = silu(g) * u ;
 *   y_t = sum_j topk_w[t, j] * (W_dn[e] a), accumulated in fp32,
 * with W the dequantized stacks (bf16 operands, fp32 accumulation); an
 * ungated layer has a = silu(W_up[e] x_t).
 *   x_bf16        : device bf16 [T, H]
 *   router_logits : device fp32 [T, E] or NULL. Given: topk_idx/topk_w are
 *                   OUTPUTS = the top_k largest logits (descending, ties to the
 *                   lower expert id) and the softmax over them. NULL: topk_idx
 *                   and topk_w are INPUTS.
 *   topk_idx      : device int32 [T, top_k]
 *   topk_w        : device fp32  [T, top_k]
 *   y_bf16        : device bf16 [T, H] (written)
 *   saved         : device buffer of e4b_moe_saved_bytes() or NULL; when given,
 *                   the bf16 gate and up projections (ungated: h) of every pair and the
 *                   routing permutation are stored for e4b_moe_dgrad
 *                   (grouped path only)
 *   ws, ws_bytes  : device workspace, >= e4b_moe_workspace_bytes()
 *   path          : e4b_path
 * Errors: NULL, SHAPE, BLOCKSIZE, CODEBOOK, WORKSPACE, ALIGN, PATH, HIP. */
e4b_status e4b_moe_forward(const e4b_moe_layer *L, int64_t T, int32_t top_k,
                           const void *x_bf16, const float *router_logits,
                           int32_t *topk_idx, float *topk_w, void *y_bf16,
                           void *saved, void *ws, size_t ws_bytes, int32_t path,
                           hipStream_t stream);

/* Frozen-base input gradient of e4b_moe_forward with routing held fixed.
 * [PR] "What this adds", recompute-in-backward bullet: each projection's
 * backward forms grad_output @ W from a re-dequantized W (never a saved W);
 * frozen-base bullet: no weight gradient. Per pair (t, j), expert e:
 *   G2 = W_dn[e]^T grad_y_t ; grad_topk_w[t, j] = G2 . a ;
 *   grad_a = topk_w[t, j] G2 ; s = sigmoid(g) ;
 *   dg = grad_a u s (1 + g (1 - s)) ; du = grad_a g s ;
 *   grad_x_t = sum_j W_gu[e]^T [dg ; du]   (ungated: dh = grad_a s (1 + h (1 - s)),
 *   grad_x_t = sum_j W_up[e]^T dh).
 *   topk_idx, topk_w : device [T, top_k] (inputs, as used by the forward)
 *   x_bf16           : device bf16 [T, H]; required when saved == NULL
 *                      (the gate/up projections are recomputed), ignored otherwise
 *   saved            : the buffer filled by e4b_moe_forward, or NULL. Its
 *                      permutation replaces topk_idx (which must be the
 *                      forward's). Recompute and saved give bitwise-identical
 *                      results.
 *   grad_y_bf16      : device bf16 [T, H]
 *   grad_x_bf16      : device bf16 [T, H] (written)
 *   grad_topk_w      : device fp32 [T, top_k] (written) or NULL
 * Errors: NULL, SHAPE, BLOCKSIZE, CODEBOOK, WORKSPACE, ALIGN, HIP. */
e4b_status e4b_moe_dgrad(const e4b_moe_layer *L, int64_t T, int32_t top_k,
                         const int32_t *topk_idx, const float *topk_w,
                         const void *x_bf16, const void *saved,
                         const void *grad_y_bf16, void *grad_x_bf16,
                         float *grad_topk_w, void *ws, size_t ws_bytes,
                         hipStream_t stream);

/* Workspace bytes that e4b_moe_forward and e4b_moe_dgrad need for (L, T,
 * top_k) (one size serves both); 0 when the arguments are invalid. */
size_t e4b_moe_workspace_bytes(const e4b_moe_layer *L, int64_t T, int32_t top_k);

/* Bytes of the `saved` buffer (its contents are internal to the library): the
 * bf16 gate and up projections of every routed pair (gated: in blocks of 256
 * sorted pairs x 128 intermediate columns, g and u side by side, one block per
 * m-tile and column block; ungated: h as [T*top_k, I]) followed by the routing
 * permutation (int32 arrays over experts, m-tiles and pairs) and room for the
 * LoRA forward's two per-pair rank projections (fp32 [T*top_k, 16] each; the
 * base forward leaves it unwritten); 0 when invalid. The forward never writes
 * the padding of the blocks (rows past an expert's pairs, blocks of m-tiles
 * the routing does not produce) and nothing reads it. */
size_t e4b_moe_saved_bytes(const e4b_moe_layer *L, int64_t T, int32_t top_k);

/* Allocation-free forward, for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): e4b_moe_forward with its workspace in a fixed per-GPU device
 * array of the library (E4B_NOALLOC_SCRATCH_BYTES) instead of a caller
 * buffer; the other arguments are those of e4b_moe_forward. Each GPU holds
 * its own copy of the array until the process ends; every call on that GPU
 * shares it and it keeps the last call's contents (no kernel of the forward
 * reads a workspace byte that the same call did not write, so nothing is
 * cleared). Calls that overlap on one GPU (two streams or two threads) race
 * on the array: the caller serializes them. No call allocates; the first
 * call on a device looks up the array's device address once.
 * Errors: as e4b_moe_forward; WORKSPACE when e4b_moe_workspace_bytes(L, T,
 * top_k) exceeds E4B_NOALLOC_SCRATCH_BYTES; HIP when the address lookup fails. */
#define E4B_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
e4b_status e4b_moe_forward_noalloc(const e4b_moe_layer *L, int64_t T, int32_t top_k,
                                   const void *x_bf16, const float *router_logits,
                                   int32_t *topk_idx, float *topk_w, void *y_bf16, void *saved,
                                   int32_t path, hipStream_t stream);

/* Per-expert LoRA adapters over the frozen base (fp32 device buffers).
 * [README] Quickstart: ExpertsLoRA(base, r=8, alpha=16) attaches trainable
 * per-expert LoRA to a frozen 4-bit stack; only the adapters train. The
 * adapter module is not printed on the pages; the usual LoRA form is used on
 * both projections of every expert e, with scale s = alpha / r:
 *   h = W_gu[e] x + s B_gu[e] (A_gu[e] x),  o = W_dn[e] a + s B_dn[e] (A_dn[e] a).
 *   A_gu : [E, r, H]    B_gu : [E, 2I, r]  (rows follow the gate | up rows)
 *   A_dn : [E, r, I]    B_dn : [E, H, r]
 * 1 <= r <= 16. The low-rank term enters each grouped GEMM as one extra
 * 16-deep MFMA slice (bf16 operands, fp32 accumulation). */
typedef struct {
  const float *A_gu, *B_gu, *A_dn, *B_dn;
  int32_t r;
  float alpha;
} e4b_lora;

/* Forward of e4b_moe_forward with LoRA adapters; always the grouped path
 * (saved, when given, is filled as by e4b_moe_forward, with the adapted g|u,
 * plus the rank projections x A_gu^T and a A_dn^T that the backward reuses).
 * ws must hold e4b_moe_lora_workspace_bytes(). Errors as e4b_moe_forward,
 * plus NULL / SHAPE for the adapter descriptor (r outside [1, 16]). */
e4b_status e4b_moe_lora_forward(const e4b_moe_layer *L, const e4b_lora *lora, int64_t T,
                                int32_t top_k, const void *x_bf16, const float *router_logits,
                                int32_t *topk_idx, float *topk_w, void *y_bf16, void *saved,
                                void *ws, size_t ws_bytes, hipStream_t stream);

/* Backward of e4b_moe_lora_forward with routing held fixed: the input
 * gradient and grad_topk_w as e4b_moe_dgrad (the base stays frozen) plus the
 * adapter gradients of sum(grad_y * y), per pair (t, j), G_o = topk_w grad_y_t:
 *   grad_a = W_dn^T G_o + s A_dn^T (B_dn^T G_o)
 *   dB_dn += s G_o (A_dn a)^T         dA_dn += s (B_dn^T G_o) a^T
 *   grad_h = [dg ; du] from grad_a     grad_x_t += W_gu^T grad_h + s A_gu^T (B_gu^T grad_h)
 *   dB_gu += s grad_h (A_gu x_t)^T     dA_gu += s (B_gu^T grad_h) x_t^T
 *   x_bf16   : device bf16 [T, H], required (the adapter gradients use it)
 *   saved    : the buffer filled by e4b_moe_lora_forward with the same
 *              adapters, or NULL (recomputes the forward's projections,
 *              bitwise equal to the saved ones)
 *   dA_gu, dB_gu, dA_dn, dB_dn : device fp32, adapter shapes (written, not
 *              accumulated); each sum runs over an expert's pairs in sorted
 *              order, so results are deterministic
 * Errors as e4b_moe_dgrad, plus NULL / SHAPE for the adapters. */
e4b_status e4b_moe_lora_backward(const e4b_moe_layer *L, const e4b_lora *lora, int64_t T,
                                 int32_t top_k, const int32_t *topk_idx, const float *topk_w,
                                 const void *x_bf16, const void *saved, const void *grad_y_bf16,
                                 void *grad_x_bf16, float *grad_topk_w, float *dA_gu,
                                 float *dB_gu, float *dA_dn, float *dB_dn, void *ws,
                                 size_t ws_bytes, hipStream_t stream);

/* Workspace bytes of the two LoRA calls (the base workspace plus the
 * adapters' per-pair projections, their bf16 operand packs and, for a
 * backward without saved state, the recomputed bf16 a [T*top_k, I]); 0 when
 * invalid. */
size_t e4b_moe_lora_workspace_bytes(const e4b_moe_layer *L, int64_t T, int32_t top_k);

/* Kernels of the forward and dgrad calls that the *_timed entry points can
 * bracket with events (benchmark instrumentation). */
typedef enum {
  E4B_K_GATE_UP_FWD = 0,   /* grouped gate_up GEMM + SiLU*up epilogue (MX path: its MX GEMM) */
  E4B_K_DOWN_FWD = 1,      /* grouped down GEMM (MX path: its MX GEMM) */
  E4B_K_DOWN_DGRAD = 2,    /* grouped GEMM on W_dn^T + SiLU-backward epilogue */
  E4B_K_GATE_UP_DGRAD = 3, /* grouped GEMM on W_gu^T */
  E4B_K_DECODE_GATE_UP = 4,/* decode dequant-GEMV, gate_up + SiLU*up (routes and groups the pairs too) */
  E4B_K_DECODE_DOWN = 5,   /* decode dequant-GEMV, down (+ the weighted combine) */
  E4B_K_ROUTE = 6,         /* top-k routing from logits */
  E4B_K_PERMUTE = 7,       /* the permutation (the first of its kernels to the last) */
  E4B_K_COMBINE = 8,       /* forward gather-combine */
  E4B_K_COMBINE_DGRAD = 9, /* dgrad gather-combine + routing-weight gradient */
  E4B_K_COUNT = 10
} e4b_kernel;

/* Per-call kernel timing. For every kernel id whose start and stop events
 * are both non-NULL, the call launches that kernel with
 * hipExtLaunchKernelGGL(start, stop), so the two events carry the start and
 * end time of that dispatch on the launch stream (hipEventElapsedTime gives
 * the kernel's duration). A kernel launched twice in one call (the gate_up
 * GEMM recomputed by a dgrad without saved state) records the last launch;
 * E4B_K_PERMUTE spans its three launches. Events are caller-owned and
 * created beforehand. The library keeps no reference after the call. */
typedef struct {
  hipEvent_t start[E4B_K_COUNT];
  hipEvent_t stop[E4B_K_COUNT];
} e4b_kernel_events;

/* e4b_moe_forward / e4b_moe_dgrad with per-call kernel timing (`events` may
 * be NULL: then identical to the untimed calls). Same arguments, results
 * and errors. */
e4b_status e4b_moe_forward_timed(const e4b_moe_layer *L, int64_t T, int32_t top_k,
                                 const void *x_bf16, const float *router_logits,
                                 int32_t *topk_idx, float *topk_w, void *y_bf16, void *saved,
                                 void *ws, size_t ws_bytes, int32_t path, hipStream_t stream,
                                 const e4b_kernel_events *events);
e4b_status e4b_moe_dgrad_timed(const e4b_moe_layer *L, int64_t T, int32_t top_k,
                               const int32_t *topk_idx, const float *topk_w, const void *x_bf16,
                               const void *saved, const void *grad_y_bf16, void *grad_x_bf16,
                               float *grad_topk_w, void *ws, size_t ws_bytes, hipStream_t stream,
                               const e4b_kernel_events *events);

/* Where the grouped forward (saved == NULL) leaves its routing permutation
 * in the workspace, for inspection (int32 arrays; byte offsets from ws):
 * counts [E], offsets [E + 1] (first sorted position of each expert),
 * tile_offsets [E + 1] (first m-tile of each expert, m-tiles of 256 sorted
 * pairs), sorted_pair [P] (flat pair id t * top_k + j at each sorted
 * position, stable: ascending within an expert), pos_of_pair [P] (its
 * inverse), tile_map [m_tiles_bound] (int32 x4 per m-tile: expert, segment
 * start, first row, rows). Errors as e4b_moe_workspace_bytes' arguments
 * (NULL for a NULL `out`). */
typedef struct {
  size_t counts, offsets, tile_offsets, sorted_pair, pos_of_pair, tile_map;
  int64_t m_tiles_bound;
} e4b_perm_layout;
e4b_status e4b_moe_perm_layout(const e4b_moe_layer *L, int64_t T, int32_t top_k,
                               e4b_perm_layout *out);

/* ---- The block around the experts ----
 *
 * What a MoE block needs next to its expert MLP: the router with the gradient
 * of its logits, tokens into expert order and back, the product of expert rows
 * with a stored stack and an epilogue, and the norms before and after a block.
 * [sdist] Experts4bit.forward takes its routing from outside the module and
 * scales and adds the experts' rows inside it; these calls are for callers who
 * need the pieces (gradients through a router, experts with biases or another
 * activation, experts on another rank, dense projections over the same storage
 * modes). They follow the conventions above. All sums, statistics and
 * epilogues are fp32; results are the same on every run. */

/* The router: topk_idx / topk_w exactly as e4b_moe_forward makes them from
 * logits (the top_k largest, descending, ties to the lower id, and the softmax
 * over them). A logit may be -inf (an expert out of service for that token):
 * it gets weight 0 when it has to fill a slot, and a row that is -inf
 * throughout selects experts 0 .. top_k - 1 with weights 0. NaN and +inf are
 * not checked: such a row's weights are meaningless, its ids are valid.
 *   logits   : device fp32 [T, E]
 *   topk_idx : device int32 [T, top_k]  (written)
 *   topk_w   : device fp32  [T, top_k]  (written)
 * Errors: NULL, SHAPE (E outside [1, 1024], top_k outside [1, min(E, 32)], T outside
 * [0, 2^24)), ALIGN, HIP. */
e4b_status e4b_route(const float *logits, int64_t T, int64_t E, int32_t top_k, int32_t *topk_idx,
                     float *topk_w, hipStream_t stream);

/* Gradient of the logits, the selection held fixed (it takes grad_topk_w where
 * e4b_moe_dgrad leaves it): grad_logits[t, idx_j] = w_j (g_j - sum_i w_i g_i),
 * 0 for every other expert. An id given twice adds up; an id outside [0, E)
 * gets no gradient.
 *   topk_idx, topk_w : device [T, top_k], as e4b_route wrote them
 *   grad_topk_w      : device fp32 [T, top_k]
 *   grad_logits      : device fp32 [T, E] (written whole)
 * Errors: as e4b_route. */
e4b_status e4b_route_backward(const int32_t *topk_idx, const float *topk_w, const float *grad_topk_w,
                              int64_t T, int64_t E, int32_t top_k, float *grad_logits,
                              hipStream_t stream);

/* Tokens into expert order: the routed pairs p = t top_k + j by expert id,
 * stable, and each pair's row. A pair whose id lies outside [0, E) goes to no
 * expert (one of another rank, a padding token): such pairs come last, from
 * offsets[E] on, and their rows are zeros.
 *   topk_idx    : device int32 [T, top_k]; top_k in [1, 32], also above E
 *   x, rows     : device [T, H], [T top_k, H] (written), bf16 or fp32 (dtype);
 *                 both NULL: only the order is made
 *   offsets     : device int32 [E + 1]      (written; offsets[E] = pairs with an expert)
 *   sorted_pair : device int32 [T top_k]    (written: pair at each place)
 *   pos_of_pair : device int32 [T, top_k]   (written: place of each pair)
 * T = 0 writes offsets only. Errors: NULL, SHAPE (E outside [1, 1024], H outside
 * [1, 2^24), T outside [0, 2^24)), DTYPE, ALIGN, HIP. */
e4b_status e4b_permute(int64_t T, int32_t top_k, int64_t E, int64_t H, int32_t dtype,
                       const int32_t *topk_idx, const void *x, void *rows, int32_t *offsets,
                       int32_t *sorted_pair, int32_t *pos_of_pair, hipStream_t stream);

/* And back: y[t] = sum_j topk_w[t, j] rows[pos_of_pair[t, j]], in slot order;
 * pairs without an expert add nothing, whatever their rows hold. topk_w NULL:
 * the plain sum, which is the gradient of x in e4b_permute (rows = grad_rows).
 * A place outside [0, offsets[E]) is read as a pair without an expert.
 *   rows : device [T top_k, H];  y : device [T, H] (written)
 * Errors: as e4b_permute. */
e4b_status e4b_unpermute(int64_t T, int32_t top_k, int64_t E, int64_t H, int32_t dtype,
                         const int32_t *offsets, const int32_t *pos_of_pair, const float *topk_w,
                         const void *rows, void *y, hipStream_t stream);

/* Gradients of e4b_unpermute: grad_rows[pos(t, j)] = topk_w[t, j] grad_y[t] (zeros
 * for a pair without an expert) and grad_topk_w[t, j] = rows[pos(t, j)] . grad_y[t]
 * (0 for one). grad_topk_w may be NULL; rows is read only for it.
 * Errors: as e4b_permute. */
e4b_status e4b_unpermute_backward(int64_t T, int32_t top_k, int64_t E, int64_t H, int32_t dtype,
                                  const int32_t *offsets, const int32_t *pos_of_pair,
                                  const float *topk_w, const void *rows, const void *grad_y,
                                  void *grad_rows, float *grad_topk_w, hipStream_t stream);

/* Activations of e4b_expert_linear: none, max(z, 0), z sigmoid(z), z Phi(z), and
 * GELU's tanh form. A NaN passes every one of them, and its gradient. */
typedef enum {
  E4B_ACT_NONE = 0,
  E4B_ACT_RELU = 1,
  E4B_ACT_SILU = 2,
  E4B_ACT_GELU = 3,
  E4B_ACT_GELU_TANH = 4
} e4b_act;

/* Product of expert-sorted rows with a stored stack: for a row r of expert e
 * (offsets[e] <= r < offsets[e + 1]),
 *   z = W[e] x_r + bias[e],   y_r = act(z) + residual_r
 * with W the bf16 view of the stack (any storage mode) and fp32 accumulation.
 * E = 1 with offsets NULL is a dense projection of every row. Rows from
 * offsets[E] on belong to no expert: y and pre are zeros there.
 *   st       : any out >= 1; in % 64 == 0; both at most 2^20; E <= 1024
 *   rows     : 0 to 2^30, and fewer than 2^24 tiles of 128 x 128 (rows, columns)
 *   offsets  : device int32 [E + 1], ascending from 0 (as e4b_permute writes them), or
 *              NULL for E = 1. Values are not checked on the host; the kernels
 *              clamp them, so that no list leads out of a buffer.
 *   x_bf16   : device bf16 [rows, in]
 *   bias     : device fp32 [E, out] or NULL
 *   residual : device bf16 [rows, out] or NULL
 *   y        : device [rows, out], bf16 or fp32 (y_dtype)  (written); a bf16 y may be
 *              the residual, in place, and must not overlap x
 *   pre      : device fp32 [rows, out] or NULL: z, for the gradient  (written)
 *   ws       : device workspace of e4b_expert_linear_workspace_bytes() (0 for few
 *              rows, or for invalid arguments: then ws may be NULL)
 * Errors: NULL, SHAPE, BLOCKSIZE, CODEBOOK, ACT, DTYPE, WORKSPACE, ALIGN, HIP. */
e4b_status e4b_expert_linear(const e4b_stack *st, int64_t rows, const int32_t *offsets,
                             const void *x_bf16, const float *bias, int32_t act,
                             const void *residual_bf16, int32_t y_dtype, void *y, float *pre,
                             void *ws, size_t ws_bytes, hipStream_t stream);
size_t e4b_expert_linear_workspace_bytes(const e4b_stack *st, int64_t rows);

/* Its gradient, the stack frozen: dz = grad_y act'(z), rounded to bf16 as the
 * product's operand;
 *   grad_x = W[e]^T dz,   grad_bias[e] = sum over e's rows of dz (unrounded)
 * (the residual's gradient is grad_y; the stack itself gets none). act needs z:
 * pre as the forward kept it, or x_bf16 and bias, from which it is computed
 * again, bit for bit.
 * Rows from offsets[E] on get zeros in grad_x; an expert without rows gets a
 * zero bias gradient.
 *   grad_y    : device [rows, out], bf16 or fp32 (gy_dtype)
 *   grad_x    : device bf16 [rows, in]  (written)
 *   grad_bias : device fp32 [E, out] (written) or NULL
 *   ws        : e4b_expert_linear_dgrad_workspace_bytes(); recompute != 0 when act
 *               is not NONE and pre is NULL
 * Errors: as e4b_expert_linear. */
e4b_status e4b_expert_linear_dgrad(const e4b_stack *st, int64_t rows, const int32_t *offsets,
                                   const void *grad_y, int32_t gy_dtype, const float *pre,
                                   const void *x_bf16, const float *bias, int32_t act,
                                   void *grad_x_bf16, float *grad_bias, void *ws, size_t ws_bytes,
                                   hipStream_t stream);
size_t e4b_expert_linear_dgrad_workspace_bytes(const e4b_stack *st, int64_t rows, int32_t recompute);

/* Norms before and after a block, with the block's gate and residual scale.
 * With N(v) = v / sqrt(mean(v^2) + eps) over a row:
 *   u = N(y) w_post (w_post NULL: u = y);  r = x + scale g u;  h = N(r) w_pre
 * y is the block's output, x the residual stream before it, r after it, h the
 * next block's input. y NULL: r = x, only h is made. w_pre NULL: no h. The
 * gate g is one value per token, per channel, or 1. */
typedef enum { E4B_GATE_NONE = 0, E4B_GATE_TOKEN = 1, E4B_GATE_CHANNEL = 2 } e4b_gate;
typedef struct {
  int64_t T, H;       /* rows (fewer than 2^23), and their length in [1, 16384] */
  int32_t dtype;      /* of x, r and their gradients: E4B_BF16 or E4B_F32 */
  int32_t gate_kind;  /* e4b_gate */
  float eps, scale;   /* eps > 0 */
  const float *w_post, *w_pre; /* device fp32 [H] or NULL */
  const float *gate;           /* device fp32 [T] or [H]; NULL exactly for E4B_GATE_NONE */
} e4b_norm;

/*   x      : device [T, H] (dtype);  y : device bf16 [T, H] or NULL
 *   r      : device [T, H] (dtype), written when y is given
 *   h      : device bf16 [T, H], written when w_pre is given
 *   rstd_y : device fp32 [T], written when w_post is given
 *   rstd_r : device fp32 [T], written when w_pre is given
 * h is made from the unrounded r. Errors: NULL (a needed pointer is missing; a
 * gate or w_post without y; neither y nor w_pre), SHAPE (also eps not above 0 or
 * an unknown gate), DTYPE, ALIGN, HIP. */
e4b_status e4b_block_norm(const e4b_norm *n, const void *x, const void *y, void *r, void *h,
                          float *rstd_y, float *rstd_r, hipStream_t stream);

/* Gradients of sum(grad_r r) + sum(grad_h h). r is rebuilt from x and y; without
 * w_pre grad_x is grad_r, whatever y holds.
 *   x, y, rstd_y, rstd_r : as in the forward
 *   grad_r      : device [T, H] (dtype), or NULL for zeros (with w_pre only)
 *   grad_h      : device bf16 [T, H], with w_pre
 *   grad_x      : device [T, H] (dtype)   (written)
 *   grad_y      : device bf16 [T, H]      (written, with y)
 *   grad_gate   : device fp32, as gate    (written) or NULL
 *   grad_w_post, grad_w_pre : device fp32 [H] (written) or NULL
 *   ws          : e4b_block_norm_workspace_bytes() (0 for a few rows, or for invalid
 *                 arguments); NULL is enough for 0, and without the gradients of
 *                 w_post, w_pre and a channel gate
 * T = 0 writes the column gradients (zeros). Errors: as e4b_block_norm, plus
 * WORKSPACE, and NULL for a gradient of something not given. */
e4b_status e4b_block_norm_backward(const e4b_norm *n, const void *x, const void *y,
                                   const float *rstd_y, const float *rstd_r, const void *grad_r,
                                   const void *grad_h, void *grad_x, void *grad_y,
                                   float *grad_gate, float *grad_w_post, float *grad_w_pre,
                                   void *ws, size_t ws_bytes, hipStream_t stream);
size_t e4b_block_norm_workspace_bytes(const e4b_norm *n);

/* ---- Balance of a router ----
 *
 * How evenly a router uses its experts, sequence by sequence, and the losses that
 * keep it even. With lse_t = log sum_e exp l_te and p_te = exp(l_te - lse_t), over
 * the N_s counted tokens t of sequence s,
 *   counts_se = pairs (t, j) with topk_idx = e,     prob_se = sum_t p_te,
 *   loss_s = E / (top_k N_s^2) sum_e counts_se prob_se   (1 for an even use),
 *   z_loss_s = 1 / N_s sum_t lse_t^2.
 * A token is counted if token_mask has it, a sequence does, and its logits are not
 * -inf throughout. A sequence without one has losses of 0. Ids outside [0, E) are
 * pairs of no expert. */
typedef struct {
  int64_t T, E;              /* tokens (fewer than 2^24), experts in [1, 1024] */
  int64_t sequences;         /* in [1, 65536] */
  int32_t top_k;             /* in [1, min(E, 32)] */
  const int32_t *cu_tokens;  /* device int32 [sequences + 1], ascending: sequence s has tokens
                                cu_tokens[s] .. cu_tokens[s + 1] - 1; those of no sequence are
                                not counted. NULL for one sequence of all T. Values are not
                                checked on the host; the kernels clamp them to [0, T]. */
  const uint8_t *token_mask; /* device [T], 0: a token that is not counted (whatever its logits
                                hold), or NULL */
} e4b_balance;

/*   logits   : device fp32 [T, E]; entries may be -inf (probability 0)
 *   topk_idx : device int32 [T, top_k]
 *   counts   : device int32 [sequences, E] (written)
 *   tokens   : device int32 [sequences], N_s (written)
 *   prob     : device fp32 [sequences, E] (written)
 *   loss, z_loss : device fp32 [sequences] (written)
 *   lse      : device fp32 [T] (written; -inf for a token that is not counted)
 *   ws       : e4b_moe_balance_workspace_bytes() (0 for a few tokens of one sequence, or
 *              for invalid arguments: then ws may be NULL)
 * T = 0 writes zeros. Errors: NULL, SHAPE, WORKSPACE, ALIGN, HIP. */
e4b_status e4b_moe_balance(const e4b_balance *b, const float *logits, const int32_t *topk_idx,
                           int32_t *counts, int32_t *tokens, float *prob, float *loss,
                           float *z_loss, float *lse, void *ws, size_t ws_bytes,
                           hipStream_t stream);
size_t e4b_moe_balance_workspace_bytes(const e4b_balance *b);

/* Gradient of sum_s (grad_loss_s loss_s + grad_z_s z_loss_s), the selection (the counts)
 * held fixed:
 *   grad_logits_te = add_te + grad_loss_s E / (top_k N_s^2) p_te (counts_se - sum_j counts_sj p_tj)
 *                    + grad_z_s 2 / N_s lse_t p_te
 * and add_te alone for a token that is not counted.
 *   b         : as in the forward; token_mask is not read (lse tells)
 *   counts, tokens, lse : as the forward wrote them; summed over ranks before the
 *               call, counts and tokens give the gradient of the loss over the tokens of all
 *   grad_loss, grad_z : device fp32 [sequences], or NULL for zeros
 *   add       : device fp32 [T, E] (the gradient through the routing weights), or NULL
 *   grad_logits : device fp32 [T, E] (written whole); may be add itself, in place, and must not
 *               overlap anything else that is read
 * Errors: as e4b_moe_balance. */
e4b_status e4b_moe_balance_backward(const e4b_balance *b, const float *logits, const int32_t *counts,
                                    const int32_t *tokens, const float *lse, const float *grad_loss,
                                    const float *grad_z, const float *add, float *grad_logits,
                                    hipStream_t stream);

/* ---- Rows in microscaled 4-bit floats, and their product with an MXFP4 stack ---- */

/* Rows of activations converted to E2M1 codes with an E8M0 scale for every 32 consecutive
 * elements, by the rule of e4b_quantize_mxfp4 and in its layout (n rows are a stack of
 * E = 1, out = n). A block that holds an infinity or a NaN gets the scale 255 (NaN) and
 * codes of 0: all of it reads as NaN.
 *   x      : device [rows, K] (dtype), or with `gated` [rows, 2 K] = [g | u], whose
 *            silu(g) u is converted (as computed without rounding; beyond fp32's range it
 *            counts as infinite)
 *   rows   : 0 to 2^30;  K % 64 == 0, at most 2^20;  rows K below 2^35
 *   codes  : device uint8 [rows, K/2]   (written)
 *   scales : device uint8 [rows, K/32]  (written)
 * Errors: NULL, SHAPE, DTYPE, ALIGN, HIP. */
e4b_status e4b_mx4_rows(const void *x, int32_t dtype, int64_t rows, int64_t K, int32_t gated,
                        uint8_t *codes, uint8_t *scales, hipStream_t stream);

/* Gradient of the gated rows, straight through their rounding: of [g | u] from that of
 * silu(g) u. (Rows that are not gated pass their gradient on.) At an infinite g the
 * derivative of silu is its limit, 1 or 0.
 *   x      : device [rows, 2 K] (dtype)
 *   grad   : device [rows, K], bf16 or fp32 (grad_dtype)
 *   grad_x : device [rows, 2 K] (dtype)  (written; must not overlap x or grad)
 * Errors: as e4b_mx4_rows. */
e4b_status e4b_mx4_rows_backward(const void *x, int32_t dtype, const void *grad, int32_t grad_dtype,
                                 int64_t rows, int64_t K, void *grad_x, hipStream_t stream);

/* Product of microscaled rows with a stored MXFP4 stack: for a row r of expert e
 * (offsets[e] <= r < offsets[e + 1]),
 *   z = W[e] x_row(r) + bias[e],   y_r = act(z) + residual_r
 * on gfx950's block-scaled MFMA, both operands as they are stored, with fp32 accumulation. row(r) is r,
 * or with an expert order (sorted_pair, as e4b_permute writes it) the token
 * sorted_pair[r] / top_k, so that tokens are not copied into expert order first. Rows
 * from offsets[E] on belong to no expert: y and pre are zeros there.
 * The gradient of x, its rounding passed straight through, and that of bias are
 * e4b_expert_linear_dgrad's, with pre as kept here (in expert order:
 * e4b_unpermute without weights adds up a token's).
 *   st          : codebook E4B_CB_MXFP4 (CODEBOOK otherwise); sizes, rows, offsets, bias, act,
 *                 residual, y and pre as in e4b_expert_linear
 *   sorted_pair : device int32 [rows] or NULL; top_k in [1, 32] is read only with it, and then
 *                 divides rows. Values are clamped to the rows of x.
 *   x_codes     : device uint8 [rows, in/2] (with sorted_pair [rows / top_k, in/2])
 *   x_scales    : device uint8 [rows, in/32] (or [rows / top_k, in/32])
 *   ws          : e4b_mx_linear_workspace_bytes() (NULL is enough for 0)
 * Errors: NULL, SHAPE, BLOCKSIZE, CODEBOOK, ACT, DTYPE, WORKSPACE, ALIGN, HIP. */
e4b_status e4b_mx_linear(const e4b_stack *st, int64_t rows, const int32_t *offsets,
                         const int32_t *sorted_pair, int32_t top_k, const uint8_t *x_codes,
                         const uint8_t *x_scales, const float *bias, int32_t act,
                         const void *residual_bf16, int32_t y_dtype, void *y, float *pre, void *ws,
                         size_t ws_bytes, hipStream_t stream);
size_t e4b_mx_linear_workspace_bytes(const e4b_stack *st, int64_t rows);

/* Static, human-readable text for a status code. */
const char *e4b_status_string(e4b_status status);

#ifdef __cplusplus
}
#endif

#endif /* E4B_H */
