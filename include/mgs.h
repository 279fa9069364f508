/*
 * mgs.h -- C ABI of the MI355X (gfx950) library for the fused MoE expert-MLP hot path:
 * per-row scaled activation + grouped block quantization (MXFP8 / NVFP4 / MXFP4) + grouped MX GEMM.
 *
 * Sources (web pages the method is described on):
 *   [P1] "[PyTorch] Enable fused activation recompute for ScaledTanhSReLU" (TransformerEngine PR 3473)
 *   [P2] "Activation + GroupedLinear Fusion for MOE" (TransformerEngine PR 3238)
 *   [P3] "[PyTorch] Preserve FP8 recompute state for inner autocast" (TransformerEngine PR 3284)
 *
 * General conventions (all entry points):
 *   - Every pointer argument named *_bf16, probs, dprobs, group_amax, data, scales, group_scale, c and
 *     bias is a DEVICE pointer; mgs_groups.split_sizes and the mgs_* structs themselves are HOST memory.
 *   - The caller owns every buffer, workspaces included.  The library allocates no memory and keeps no
 *     state between calls, apart from the static device scratch of mgs_grouped_scaled_act_bwd_noalloc
 *     (and the per-device address of that scratch).
 *   - Every call validates its arguments on the host, then enqueues its kernels on `stream` (a
 *     hipStream_t; NULL = the null stream) and returns without synchronizing.
 *   - A NULL output pointer (or an mgs_qbuf with data == NULL) means "not requested": it is not computed.
 *   - Return value: MGS_OK (0) or a negative MGS_ERR_* code; nothing is enqueued when validation
 *     fails.  mgs_last_error() returns a thread-local message describing the last failure.
 *   - Row groups: `groups->split_sizes[g]` rows belong to group (expert) g, stored contiguously in
 *     group order ([P2] sequence diagram: split_sizes).  M = sum of split sizes.
 *   - Quantized widths (the quantized, contiguous dimension) must be multiples of 32, at most 2^24.
 *   - Size limits of the quantizing entry points (MGS_ERR_SHAPE beyond them): one group's columnwise
 *     matrix, roundup(m_g, 128) x W elements, stays below 2^31, and so does the byte size of the
 *     rowwise MXFP8 / MXFP4 scale array, 4 * M * ceil(W / 128).  The MXFP4 grouped GEMM refuses operands
 *     past them too.
 *   - Arithmetic follows IEEE FP32 with round-to-nearest-even; results are deterministic (no float
 *     atomics, fixed reduction orders).
 *
 * Quantized tensor layouts (mgs_qbuf), for a logical [M x W] tensor quantized along W:
 *   MXFP8 (E4M3 elements, E8M0 scale per 32):
 *     rowwise : data u8 [M, W]                      scales: K-step grouped over [M, W]
 *     colwise : group g at data + W*coff[g]:        data [W, mp_g]   (tokens contiguous)
 *               group g at scales + W*coff[g]/32:   scales: K-step grouped over [W, mp_g]
 *   NVFP4 (E2M1 elements two per byte, element 2i in the low nibble; E4M3 scale per 16; FP32 per group):
 *     rowwise : data u8 [M, W/2]                    scales u8 [M, W/16]   group_scale f32 [E]
 *     colwise : group g at data + W*coff[g]/2:      data [W, mp_g/2]
 *               group g at scales + W*coff[g]/16:   scales [W, mp_g/16]   group_scale f32 [E]
 *   where mp_g = roundup(m_g, 128) and coff[g] = sum_{h<g} mp_h; padding tokens are written as zeros.
 *   MXFP4 (E2M1 elements two per byte as NVFP4's, E8M0 scale per 32, no group scale):
 *     rowwise : data u8 [M, W/2]                    scales: K-step grouped over [M, W]
 *     colwise : group g at data + W*coff[g]/2:      data [W, mp_g/2]
 *               group g at scales + W*coff[g]/32:   scales: K-step grouped over [W, mp_g]
 *   "K-step grouped" MXFP8 and MXFP4 scales of an [R x K] matrix keep the four 32-block scales of each
 *   128-wide K step together per row, steps outermost: the scale of (row r, block kb) is the byte
 *   ((kb / 4) * R + r) * 4 + kb % 4; 4 * R * ceil(K / 128) bytes, unused bytes of a partial last
 *   step zero.  (One aligned dword per row and K step: what the grouped GEMM stages per step.)
 *   MXFP8 scale of a block with maximum magnitude amax: E8M0 code clamp(floor(log2 amax) - 8 + 127, 0, 254)
 *   (0 for an all-zero block), element = E4M3(y / 2^(code-127)) rounded to nearest-even, saturated at 448.
 *   MXFP4 scale of a block: E8M0 code clamp(floor(log2 amax) - 2 + 127, 0, 254) (0 for an all-zero
 *     block), element = E2M1(y / 2^(code-127)) rounded to nearest-even, saturated at 6 (the OCP
 *     microscaling rule: the largest E2M1 exponent is 2).  Finite inputs.
 *   NVFP4 (per group g, FP32): S_enc = 2688 / amax_g (1 if amax_g == 0, FLT_MAX on overflow);
 *   block scale s_b = E4M3((amax_b / 6) * S_enc); element = E2M1(y * (S_enc / s_b)) (0 if s_b == 0);
 *   group_scale[g] = S_dec = 1 / S_enc; dequantized value = e2m1 * s_b * S_dec.
 */
#ifndef MGS_H
#define MGS_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MGS_ABI_VERSION 8
#define MGS_MAX_GROUPS 256
#define MGS_MAX_TOPK 16
/* Size of the static per-device scratch of mgs_grouped_scaled_act_bwd_noalloc (16 MiB). */
#define MGS_NOALLOC_SCRATCH_BYTES ((int64_t)16 << 20)

enum mgs_status {
  MGS_OK = 0,
  MGS_ERR_INVALID_ARG = -1, /* NULL required pointer, unknown enum value, bad group count      */
  MGS_ERR_SHAPE = -2,       /* width not a multiple of 32, negative split, split sum mismatch,
                               size limits (see the conventions above)                          */
  MGS_ERR_UNSUPPORTED = -3, /* a valid but unsupported combination (e.g. NVFP4 recompute
                               without the forward's group amax)                                 */
  MGS_ERR_HIP = -4          /* a HIP launch error                                                */
};

/* Activation kinds.  [P2] Greptile summary (first bullet) and Important Files Changed
 * (csrc/extensions/activation.cpp): scaled SwiGLU, clamped SwiGLU and SReLU; [P1] title:
 * ScaledTanhSReLU.  With x the BF16 FC1 output row and p the row's routing probability:
 *   IDENTITY        a = x                                       (plain grouped quantize)
 *   SRELU           a = relu(x)^2
 *   TANH_SRELU      a = (s * tanh(relu(x) / s))^2               (bounded at s^2, [P1] reviewer comment)
 *   SWIGLU          x = [gate | up], a = silu(gate) * up        (output width = width_in / 2)
 *   CLAMPED_SWIGLU  g = min(gate, limit), u = clamp(up, -limit, limit), a = g * sigmoid(alpha g) * (u + beta)
 * and, through the same fused kernels and recompute path ([P1] review discussion: nothing in the
 * fused recompute is specific to SReLU; GeLU, sigmoid and the GLU family fit the same scheme):
 *   GELU            a = x * Phi(x) = x/2 * (1 + erf(x / sqrt(2)))   (the exact form, not tanh-approximated)
 *   SIGMOID         a = 1 / (1 + exp(-x))
 *   GLU             x = [gate | up], a = sigmoid(gate) * up          (output width = width_in / 2)
 * The forward output is y = a * p, kept in FP32 until it is quantized. */
typedef enum {
  MGS_ACT_IDENTITY = 0,
  MGS_ACT_SRELU = 1,
  MGS_ACT_TANH_SRELU = 2,
  MGS_ACT_SWIGLU = 3,
  MGS_ACT_CLAMPED_SWIGLU = 4,
  MGS_ACT_GELU = 5,
  MGS_ACT_SIGMOID = 6,
  MGS_ACT_GLU = 7
} mgs_act_kind;

typedef enum { MGS_FMT_MXFP8 = 0, MGS_FMT_NVFP4 = 1, MGS_FMT_MXFP4 = 2 } mgs_fmt;

typedef enum { MGS_DTYPE_BF16 = 0, MGS_DTYPE_F32 = 1 } mgs_dtype;

typedef enum {
  MGS_GEMM_FPROP = 0, /* grouped over M: C[M x N] = A[M x K] . B_g^T, B = [E x N x K]          */
  MGS_GEMM_DGRAD = 1, /* same contraction as FPROP; B is the columnwise copy of the weight     */
  MGS_GEMM_WGRAD = 2  /* grouped over K: C_g[Mc x N] = A_g[Mc x mp_g] . B_g[N x mp_g]^T          */
} mgs_gemm_mode;

typedef enum { MGS_NBYTES_DATA = 0, MGS_NBYTES_SCALES = 1, MGS_NBYTES_GROUP_SCALE = 2 } mgs_nbytes_which;

typedef struct {
  int32_t kind;  /* mgs_act_kind */
  float s;       /* TANH_SRELU bound parameter (> 0) */
  float limit;   /* CLAMPED_SWIGLU clamp (> 0) */
  float alpha;   /* CLAMPED_SWIGLU sigmoid slope (default 1) */
  float beta;    /* CLAMPED_SWIGLU up-projection offset (default 0) */
} mgs_act_params;

/* Row groups.  Host split sizes: split_sizes points to them; max_rows and dev_table are ignored.
 *
 * Device-resident split sizes (split_sizes == NULL): the graph-safe form.  [P2] Greptile summary,
 * third bullet (GroupedLinear's graph-safe forward, _fuser_forward_graph_safe): the split sizes stay in
 * device memory, so a captured HIP graph can be replayed for a different routing without a host sync.
 *   max_rows   row capacity (> 0): every layout is strided for it, so buffer sizes do not depend on the
 *              split sizes -- rowwise tensors have max_rows rows (rows past the sum are neither read nor
 *              written), columnwise tensors a padded token count of 128 * (ceil(max_rows / 128) +
 *              num_groups), rowwise MXFP8 scales are K-step grouped over max_rows rows, and an
 *              M-grouped GEMM's m (a WGRAD's k) is max_rows.  mgs_qtensor_nbytes and the workspace-size
 *              calls return the capacity sizes.
 *   dev_table  DEVICE buffer of mgs_groups_table_bytes() bytes holding the offsets, written on the
 *              stream by mgs_groups_update (call it after every change of the split sizes; kernels of
 *              the calls enqueued after it read them).  Calls sharing a dev_table must not overlap.
 * Every call takes device-resident split sizes, for both formats; NVFP4's per-group amax and S_dec
 * are taken over the rows of each group as the device table holds them at the time of the call. */
typedef struct {
  int32_t num_groups;         /* 1 .. MGS_MAX_GROUPS */
  const int64_t* split_sizes; /* host array [num_groups], each >= 0; NULL: device-resident (above) */
  int64_t max_rows;
  void* dev_table;
} mgs_groups;

/* One orientation (rowwise or columnwise) of a grouped quantized tensor; see the layouts above. */
typedef struct {
  void* data;
  void* scales;
  float* group_scale; /* NVFP4 only: S_dec per group [E]; ignored for MXFP8 */
  /* NVFP4 columnwise copies only (0 elsewhere): random Hadamard transform of every 16-token block
   * of a column before quantization, v -> H16 diag(s) v / 4 (H16[k][n] = (-1)^popcount(k & n)).
   * 0 = off; otherwise bit 16 must be set and bits 0..15 give the signs (bit n set: s_n = -1).
   * [P1] names this recipe NVFP4_RHT for its NVFP4 measurements without defining it; it is for the
   * two operands of a weight-gradient GEMM, made with the same signs, whose product the orthogonal
   * transform leaves unchanged.  The transformed copy's per-group encode scale comes from its own
   * amax (see group_amax below); the GEMM reads such a copy like any other. */
  uint32_t rht;
} mgs_qbuf;

/* Bytes of the device table of device-resident split sizes (mgs_groups.dev_table). */
int64_t mgs_groups_table_bytes(void);

/* Device-resident split sizes: enqueues on `stream` the computation of groups->dev_table from
 * split_sizes_dev (DEVICE int64 [num_groups]).  status_dev (DEVICE int32, nullable) receives 0, or 1
 * when a split size is negative or their sum exceeds max_rows; the table then holds empty groups, so
 * the calls that follow write no output rows (a WGRAD writes zero weight gradients).  The host cannot
 * see this without a synchronization: read status_dev after the step. */
int mgs_groups_update(const mgs_groups* groups, const int64_t* split_sizes_dev, int32_t* status_dev,
                      void* stream);

/* Library ABI version (MGS_ABI_VERSION). */
int mgs_abi_version(void);

/* Thread-local description of the last error returned on this thread ("" if none). */
const char* mgs_last_error(void);

/* Byte size of one buffer of a grouped quantized tensor of width `width`:
 * which = DATA, SCALES or GROUP_SCALE (4 * E for NVFP4, 0 for MXFP8).  Negative MGS_ERR_* on error. */
int64_t mgs_qtensor_nbytes(int32_t fmt, int32_t colwise, const mgs_groups* groups, int64_t width,
                           int32_t which);

/* Fused forward: y = act(x) * p, quantized rowwise and/or columnwise in one pass over x.
 * [P2] Greptile summary, first bullet (the per-row scale, the activation and the grouped quantization
 * share one pass) and sequence diagram (the forward activation call takes x, the scales, the
 * quantizer and split_sizes and returns the grouped quantized tensor).
 *   x_bf16     [M x width_in] BF16, row-major (required unless M == 0)
 *   probs      [M] FP32 per-row scale; NULL means 1 for every row
 *   out_row    rowwise qtensor of y [M x W_a] (W_a = width_in, or width_in/2 for gated kinds); nullable
 *   out_col    columnwise qtensor of y; nullable (NULL in the recompute forward, [P1] Description)
 *   group_amax [E] FP32: NVFP4 only, required there; receives max|y| per group (the per-tensor
 *              amax of each expert slice) and must be kept for a later recompute.  Ignored for MXFP8.
 *              [2E] when out_col has the Hadamard transform (mgs_qbuf.rht): entries E..2E-1 receive
 *              the transformed values' amax, which scales the columnwise copy.
 * NVFP4 runs two passes over x (group amax, then quantize). */
int mgs_grouped_scaled_act_fwd(const mgs_act_params* act, int32_t fmt, const mgs_groups* groups,
                               int64_t width_in, const void* x_bf16, const float* probs,
                               const mgs_qbuf* out_row, const mgs_qbuf* out_col, float* group_amax,
                               void* stream);

/* Fused forward from the FP32 FC1 output.  [P1] Description and review discussion: in the fused
 * forward the activation is applied to the FP32 accumulator of the FC1 GEMM, while the backward and
 * the recompute read the saved BF16 FC1 output; the regenerated FC2 input therefore differs slightly
 * from the forward's (the deviation that page tabulates for the FC2 weight gradient).  Same outputs
 * and rules as mgs_grouped_scaled_act_fwd, except:
 *   x_f32      [M x width_in] FP32, row-major (required unless M == 0); width_in * 128 < 2^31
 *   x_bf16_out [M x width_in] BF16 nullable: receives x rounded to nearest-even, the tensor the
 *              backward and the recompute take as x_bf16 (written in the same pass)
 * At least one of out_row, out_col, x_bf16_out must be requested. */
int mgs_grouped_scaled_act_fwd_f32(const mgs_act_params* act, int32_t fmt, const mgs_groups* groups,
                                   int64_t width_in, const float* x_f32, const float* probs,
                                   const mgs_qbuf* out_row, const mgs_qbuf* out_col, float* group_amax,
                                   void* x_bf16_out, void* stream);

/* Fused backward.  [P2] sequence diagram, backward half: grouped_scaled_d{swiglu,srelu}(grad, input_,
 * scales, quantizer) -> (grouped_dy, dense_dy, grad_scales), where grad = dL/d(act_out * scales);
 * [P1] Description: activation recompute regenerates FC2's input from the saved BF16 FC1 output.
 *   x_bf16        [M x width_in] BF16 saved FC1 output (required unless M == 0)
 *   dy_bf16       [M x W_a] BF16 dL/d(a * p) (required unless M == 0)
 *   probs         [M] FP32; NULL means 1
 *   dx_bf16       [M x width_in] BF16 dense dL/dx = dy * p * a'(x); nullable
 *   dx_row/dx_col quantized dL/dx (rowwise / columnwise); nullable
 *   dx_group_amax [E] FP32: required when dx is quantized to NVFP4 (receives max|dL/dx| per group);
 *                 [2E] when dx_col has the Hadamard transform (transformed amax at E..2E-1)
 *   dprobs        [M] FP32 dL/dp = sum_j dy * a(x); nullable
 *   dx_col_sum    [E x width_in] FP32 per-group column sums of the dense BF16 dL/dx (the values dx_bf16
 *                 holds, whether or not it is requested): the FC1 bias gradient.  [P1] Description,
 *                 second paragraph (bias in the fused step).  Nullable; empty groups give zeros.
 *   act_col       columnwise qtensor of y = a(x) * p regenerated from x (recompute); nullable.  Its bytes
 *                 equal those the forward's out_col would have held.
 *   saved_group_amax [E] FP32 group amax written by the forward; required for an NVFP4 act_col
 *                 without the Hadamard transform.  With it (act_col.rht) the transformed values'
 *                 amax is taken again from x in this call (the same bits the forward's copy used)
 *                 and the workspace is required.
 *   workspace     DEVICE scratch of at least mgs_act_bwd_workspace_bytes() bytes, required when dprobs
 *                 or dx_col_sum is requested, or act_col has the Hadamard transform (else ignored;
 *                 may be NULL); owned by the caller,
 *                 contents undefined before and after the call.  The kernel writes partial sums there
 *                 (dprobs: one per row and 128-column tile; column sums: one per 128-token block and
 *                 column) and second kernels add them in a fixed order, so both are deterministic.
 *                 Calls that share a workspace must not overlap.
 *   workspace_bytes its size; MGS_ERR_INVALID_ARG when it is needed and too small. */
int mgs_grouped_scaled_act_bwd(const mgs_act_params* act, int32_t fmt, const mgs_groups* groups,
                               int64_t width_in, const void* x_bf16, const void* dy_bf16,
                               const float* probs, void* dx_bf16, const mgs_qbuf* dx_row,
                               const mgs_qbuf* dx_col, float* dx_group_amax, float* dprobs,
                               float* dx_col_sum, const mgs_qbuf* act_col,
                               const float* saved_group_amax, void* workspace,
                               int64_t workspace_bytes, void* stream);

/* The fused backward above without a workspace argument, for callers that cannot allocate device
 * memory: code under HIP graph capture, tight serving loops, harnesses that forbid hipMalloc.  Same
 * arguments, outputs and results (bit for bit, the same kernels) as mgs_grouped_scaled_act_bwd;
 * the partial sums go to a static scratch array of MGS_NOALLOC_SCRATCH_BYTES (16 MiB) in device
 * memory that each device holds from the first call on it until the process ends.  The call
 * allocates nothing (no hipMalloc / hipFree, no allocating library routine).
 *   - MGS_ERR_SHAPE when the workspace the request needs (mgs_act_bwd_workspace_bytes, counted only
 *     when dprobs, dx_col_sum or a transformed act_col is requested) exceeds the scratch; nothing is
 *     enqueued then.
 *   - Every call on one device shares that device's scratch, and the scratch keeps the last call's
 *     contents (each call writes every partial it reads and zeroes its group maxima itself): calls
 *     that overlap on one device (other streams, other threads) race and must be serialized by the
 *     caller. */
int mgs_grouped_scaled_act_bwd_noalloc(const mgs_act_params* act, int32_t fmt, const mgs_groups* groups,
                                       int64_t width_in, const void* x_bf16, const void* dy_bf16,
                                       const float* probs, void* dx_bf16, const mgs_qbuf* dx_row,
                                       const mgs_qbuf* dx_col, float* dx_group_amax, float* dprobs,
                                       float* dx_col_sum, const mgs_qbuf* act_col,
                                       const float* saved_group_amax, void* stream);

/* Workspace bytes mgs_grouped_scaled_act_bwd needs for dprobs, dx_col_sum and a transformed act_col:
 * roundup(roundup(4 * M * ceil(W_a / 128), 256) + 4 * (P / 128) * width_in, 256) + 8 * E,
 * P = sum_g roundup(m_g, 128).
 * Negative MGS_ERR_* on invalid arguments. */
int64_t mgs_act_bwd_workspace_bytes(const mgs_act_params* act, const mgs_groups* groups,
                                    int64_t width_in);

/* Plain grouped quantization of a BF16 tensor (weights, upstream gradients, FC1 input): the forward
 * above with act = IDENTITY and p = 1.  [P2] Greptile summary, second bullet (GroupedLinear consumes a
 * pre-quantized grouped tensor); [P3] "A behaviour change worth calling out" (columnwise usage).
 *   out_row, out_col, group_amax as in mgs_grouped_scaled_act_fwd (group_amax required for NVFP4 when
 *              a quantized output is requested)
 *   col_sum    [E x width] FP32 per-group column sums of x in the same pass (the FC2 bias gradient when
 *              x is dL/dY2); nullable; empty groups give zeros.  At least one of out_row, out_col,
 *              col_sum must be requested.
 *   workspace  DEVICE scratch of at least mgs_grouped_mx_quantize_workspace_bytes() bytes, required
 *              when col_sum is requested (per-block partial sums, added in block order by a second
 *              kernel); caller-owned, contents undefined before and after; calls sharing it must not
 *              overlap.  workspace_bytes: its size (MGS_ERR_INVALID_ARG when needed and too small). */
int mgs_grouped_mx_quantize(int32_t fmt, const mgs_groups* groups, int64_t width, const void* x_bf16,
                            const mgs_qbuf* out_row, const mgs_qbuf* out_col, float* group_amax,
                            float* col_sum, void* workspace, int64_t workspace_bytes, void* stream);

/* Workspace bytes of mgs_grouped_mx_quantize's col_sum: 4 * (P / 128) * width,
 * P = sum_g roundup(m_g, 128).  Negative MGS_ERR_* on invalid arguments. */
int64_t mgs_grouped_mx_quantize_workspace_bytes(const mgs_groups* groups, int64_t width);

/* Grouped GEMM on quantized operands with FP32 accumulation.  [P2] Greptile summary, second bullet and
 * sequence diagram (GroupedLinear forward / backward on a pre-built grouped tensor).
 *   FPROP, DGRAD (grouped over M; m = M = sum of splits, n, k = reduction width, k % 32 == 0):
 *     A = rowwise qtensor [M x k];
 *     B (FPROP) = rowwise qtensor of the weight [E * n x k] (expert g owns rows g*n .. g*n + n - 1);
 *     B (DGRAD) = columnwise qtensor of the weight [E * k x n] with split_sizes [k] * E (per expert
 *                 [n x roundup(k, 128)], zero padded);
 *     C [M x n] row-major; bias_bf16 [E x n] optional.
 *   WGRAD (grouped over K; k = M = sum of splits; m, n = widths of A and B):
 *     A = columnwise qtensor of width m, B = columnwise qtensor of width n, both over the same groups;
 *     C [E x m x n] row-major (an empty group writes zeros, or leaves C unchanged if accumulating).
 *   c_dtype BF16 or F32; accumulate != 0 adds into C (F32 only).
 *   NVFP4 operands also scale each group's result by A.group_scale[g] * B.group_scale[g]. */
int mgs_grouped_gemm_mx(int32_t mode, int32_t fmt, const mgs_groups* groups, int64_t m, int64_t n,
                        int64_t k, const mgs_qbuf* a, const mgs_qbuf* b, void* c, int32_t c_dtype,
                        const void* bias_bf16, int32_t accumulate, void* stream);

/* FC1's forward GEMM with the scaled activation and MXFP8 rowwise quantization in its epilogue.
 * [P1] Description and review discussion: the fused forward applies the activation to FC1's output
 * inside the GEMM and hands FC2 its quantized input; [P2] Greptile summary (per-row scale, activation
 * and grouped quantization in one pass).  An FPROP of mgs_grouped_gemm_mx (same A, B, groups, m, n, k,
 * bias; MXFP8 only) that also writes
 *   out_row    rowwise MXFP8 qtensor [M x n] of y = act(c) * probs[row], required: the bytes
 *              mgs_grouped_scaled_act_fwd (act_input BF16) or mgs_grouped_scaled_act_fwd_f32
 *              (act_input F32) writes for out_row from this C, bit for bit
 *   c_bf16     [M x n] BF16 FC1 output, required (the tensor the backward and the recompute read)
 *   act        unary kinds only (IDENTITY, SRELU, TANH_SRELU, GELU, SIGMOID); gated kinds return
 *              MGS_ERR_UNSUPPORTED (their two halves lie in different output tiles)
 *   probs      [M] FP32 per-row scale; NULL means 1
 *   act_input  MGS_DTYPE_F32: activate the FP32 value c = A.B^T + bias; MGS_DTYPE_BF16: its BF16 rounding
 * No columnwise copy: the recompute forward needs none; callers wanting one use the separate forward. */
int mgs_grouped_gemm_mx_fprop_act(const mgs_groups* groups, int64_t m, int64_t n, int64_t k,
                                  const mgs_qbuf* a, const mgs_qbuf* b, void* c_bf16,
                                  const void* bias_bf16, const mgs_act_params* act, const float* probs,
                                  int32_t act_input, const mgs_qbuf* out_row, void* stream);

/* Per-group column sums (bias gradient): out[g, j] = sum over group g's rows of x[r, j], FP32,
 * fixed summation order.  [P1] Description, second paragraph: bias changes what wgrad consumes.
 *   x_bf16 [M x width] BF16; out [E x width] FP32 (empty groups give zeros). */
int mgs_grouped_col_sum(const mgs_groups* groups, int64_t width, const void* x_bf16, float* out,
                        void* stream);

/* ---- Routing around the expert MLP ---------------------------------------------------------------
 * [P2] sequence diagram: the grouped calls above take rows sorted by expert with split_sizes.  These
 * calls make both from a router's logits, and bring the expert outputs back into token order; nothing
 * leaves the device, so a captured graph follows each replay's routing (mgs_groups_update takes
 * split_sizes as it is written here).  A slot is one (token, choice) pair, numbered token * topk + choice.
 * Experts 1 .. MGS_MAX_GROUPS, topk 1 .. MGS_MAX_TOPK, tokens * topk below 2^31 and tokens such that a
 * launch has fewer than 2^32 threads (up to 2^24 - 1 tokens always); tokens == 0 is allowed, and tensors without
 * elements may be NULL.  An output (and the workspace) must not be or overlap another tensor of the call; this is
 * refused as far as contiguous tensors and the first rows of strided ones show it.
 * Every pointer is a DEVICE pointer but the params.  Results are deterministic. */

typedef enum { MGS_SCORE_SOFTMAX = 0, MGS_SCORE_SIGMOID = 1 } mgs_score;

typedef struct {
  int32_t score;       /* mgs_score */
  int32_t renormalize; /* nonzero: the picked scores are divided by their sum */
  float scale;         /* finite factor on the weights */
} mgs_route_params;

/* Router: the topk largest logits of every token, in descending order (equal logits: the lower expert
 * first; NaN ranks above everything), and their weights
 *   p = softmax(logits) over all experts, or 1 / (1 + exp(-logit)) each,
 *   w = scale * p, or with renormalize scale * p / (sum of the token's picked p).
 * An expert whose logit is -inf is not available: it is never picked, and a choice that finds no
 * available expert gets expert -1 and weight 0 (a token whose logits are all -inf gets none at all).
 * NaN or +inf logits give NaN weights as the formulas say; sigmoid scores that all underflow to 0 keep
 * weights of 0 when renormalized.
 *   logits      [tokens x experts] BF16 or F32 (logits_dtype), row stride ld >= experts elements
 *   expert_idx  [tokens x topk] int32; weights [tokens x topk] FP32 */
int mgs_moe_route(const mgs_route_params* params, int64_t tokens, int32_t experts, int32_t topk,
                  const void* logits, int32_t logits_dtype, int64_t ld, int32_t* expert_idx, float* weights,
                  void* stream);

/* The logits' gradient of the router's weights: dlogits [tokens x experts], of the logits' type, row
 * stride ld_dlogits, every element written (zeros where the formulas give none).  expert_idx is the
 * forward's (a token's experts are distinct); dweights [tokens x topk] FP32 (ignored where expert_idx is -1). */
int mgs_moe_route_bwd(const mgs_route_params* params, int64_t tokens, int32_t experts, int32_t topk,
                      const void* logits, int32_t logits_dtype, int64_t ld, const int32_t* expert_idx,
                      const float* dweights, void* dlogits, int64_t ld_dlogits, void* stream);

/* Workspace bytes of mgs_moe_dispatch (0 for few slots).  Negative MGS_ERR_* on invalid arguments. */
int64_t mgs_moe_dispatch_workspace_bytes(int64_t tokens, int32_t topk, int32_t experts);

/* Tokens into expert order: a stable sort of the slots by expert, and the token rows copied to it.
 *   expert_idx   [tokens x topk] int32; an entry outside [0, experts) is a slot without an expert
 *   row_of_slot  [tokens x topk] int32, required: the slot's row in expert order, -1 without an expert
 *   split_sizes  [experts] int64, required: rows of each expert
 *   x            [tokens x hidden] BF16 or F32 (dtype), row stride ldx; NULL (with rows NULL): only the sort
 *   rows         [num_rows x hidden] contiguous, num_rows >= tokens * topk: rows[row_of_slot[s]] = x[token];
 *                rows past the last used one are left as they were
 *   weights, row_weights  both or neither: row_weights[row_of_slot[s]] = weights[s] ([tokens x topk], the
 *                per-row scale `probs` of the activation calls)
 *   workspace    mgs_moe_dispatch_workspace_bytes() bytes of scratch (ignored, may be NULL, when that
 *                is 0), caller-owned, contents undefined before and after; calls sharing it must not
 *                overlap */
int mgs_moe_dispatch(int64_t tokens, int32_t topk, int32_t experts, const int32_t* expert_idx, int64_t hidden,
                     int32_t dtype, const void* x, int64_t ldx, const float* weights, void* rows,
                     int64_t num_rows, float* row_weights, int32_t* row_of_slot, int64_t* split_sizes,
                     void* workspace, int64_t workspace_bytes, void* stream);

/* Gradient of the dispatch: dx[token] = the sum of its slots' drows (in slot order, FP32, one rounding),
 * and with drow_weights [num_rows] and dweights [tokens x topk] (both or neither) dweights[s] =
 * drow_weights[row_of_slot[s]] (the activation backward's dprobs), 0 for a slot without a row.
 * Rows outside [0, num_rows) in row_of_slot count as no row, here and below. */
int mgs_moe_dispatch_bwd(int64_t tokens, int32_t topk, int64_t hidden, int32_t dtype,
                         const int32_t* row_of_slot, int64_t num_rows, const void* drows,
                         const float* drow_weights, void* dx, int64_t lddx, float* dweights, void* stream);

/* Expert outputs back into token order: y[token] = sum over its slots of w * rows[row_of_slot[s]], in slot
 * order in FP32, one rounding; weights [tokens x topk] NULL means 1 (where the experts applied them).  A
 * token without any row gets zeros.  rows [num_rows x hidden] contiguous, y row stride ldy. */
int mgs_moe_combine(int64_t tokens, int32_t topk, int64_t hidden, int32_t dtype, const int32_t* row_of_slot,
                    int64_t num_rows, const void* rows, const float* weights, void* y, int64_t ldy,
                    void* stream);

/* Gradient of the combine: drows[row_of_slot[s]] = w * dy[token] (nullable; rows that no slot has are
 * left as they were) and dweights[s] = <dy[token], rows[row_of_slot[s]]> (nullable; needs rows; 0 for a slot
 * without a row).  At least one of them is requested. */
int mgs_moe_combine_bwd(int64_t tokens, int32_t topk, int64_t hidden, int32_t dtype,
                        const int32_t* row_of_slot, int64_t num_rows, const void* dy, int64_t lddy,
                        const void* rows, const float* weights, void* drows, float* dweights, void* stream);

/* ---- The expert block without quantization --------------------------------------------------------
 * [P2] sequence diagram: the same grouped calls (FC1, gated activation with the row's scale, FC2, and back) on
 * BF16 operands as they lie in memory, for a layer that is trained in BF16.  Group conventions as above (host or
 * device-resident split sizes; rows past the last used one are neither read nor written).  Widths are multiples
 * of 8 up to 2^20; BF16 and FP32 tensors start on 16-byte boundaries (probs, dprobs and the workspace: 4).  No
 * output may be or overlap another tensor of its call.  Products accumulate in FP32; results are deterministic. */

/* Grouped product of BF16 tensors:
 *   FPROP   C [M x n] = A_g B_g^T    a [M x k], b [E x n x k]; bias_bf16 [E x n] nullable
 *   DGRAD   C [M x n] = A_g B_g      a [M x k], b [E x k x n] (the forward's weight as it is stored); bias as above
 *   WGRAD   C_g [m x n] = A_g^T B_g  a [M x m], b [M x n], k = M, c [E x m x n] (an empty group writes zeros, or leaves
 *                                    C unchanged if accumulating)
 *   c_dtype BF16 (one rounding) or F32; accumulate != 0 adds into C (F32 only). */
int mgs_grouped_gemm_bf16(int32_t mode, const mgs_groups* groups, int64_t m, int64_t n, int64_t k, const void* a_bf16,
                          const void* b_bf16, void* c, int32_t c_dtype, const void* bias_bf16, int32_t accumulate,
                          void* stream);

/* Forward of the gated block in one kernel: with [gate | up] = x_g W_g^T + bias in FP32,
 *   h = act(gate, up) * probs[row], rounded to BF16 once.  The clamps keep a NaN: h is NaN where
 *   gate or up is, and so are, in the backward, the row's dprobs and what the derivatives make of it in dpre.
 *   act      a gated kind (SWIGLU, CLAMPED_SWIGLU, GLU)
 *   x_bf16   [M x k]; w_bf16 [E x 2f x k]; bias_bf16 [E x 2f] nullable; probs [M] FP32, NULL means 1
 *   h_bf16   [M x f]
 *   pre      [M x 2f] nullable: [gate | up], which the backward takes, of pre_dtype F32 or BF16 (half the bytes, and the
 *            gradients are of the rounded values; CLAMPED_SWIGLU: of the nearest ones on the same side of the clamps,
 *            where the derivative jumps) */
int mgs_grouped_gated_fwd(const mgs_act_params* act, const mgs_groups* groups, int64_t f, int64_t k, const void* x_bf16,
                          const void* w_bf16, const void* bias_bf16, const float* probs, void* h_bf16, void* pre,
                          int32_t pre_dtype, void* stream);

/* Backward of the second linear and the activation in one kernel: with da = dy_g W2_g in FP32,
 *   dpre = da * probs[row] * (d act / d gate, d act / d up) at pre, dprobs[row] = sum_j da * act(pre).
 *   dy_bf16 [M x n]; w2_bf16 [E x n x f]; pre [M x 2f] of the forward, of pre_dtype; probs as in the forward
 *   dpre_bf16 [M x 2f]; the weights' and inputs' gradients are products of it (DGRAD and WGRAD above)
 *   h_bf16   [M x f] nullable: act(pre) * probs again, the second linear's input (recompute)
 *   dprobs   [M] FP32 nullable; needs the workspace, mgs_grouped_gated_bwd_workspace_bytes() bytes of
 *            scratch, caller-owned, contents undefined before and after; calls sharing it must not overlap */
int mgs_grouped_gated_bwd(const mgs_act_params* act, const mgs_groups* groups, int64_t f, int64_t n, const void* dy_bf16,
                          const void* w2_bf16, const void* pre, int32_t pre_dtype, const float* probs, void* dpre_bf16,
                          void* h_bf16, float* dprobs, void* workspace, int64_t workspace_bytes, void* stream);

/* Workspace bytes of mgs_grouped_gated_bwd's dprobs (negative MGS_ERR_* on invalid arguments). */
int64_t mgs_grouped_gated_bwd_workspace_bytes(const mgs_groups* groups, int64_t f);

/* ---- Weights in 4 bits with BF16 rows --------------------------------------------------------------
 * The serving form of the block above: each weight is (q - z) s with a code q in 0 .. 15 and, per group of 32, 64 or
 * 128 elements along k, a BF16 scale s and a zero point z in 0 .. 15 (8 where there are none).  Rows stay in BF16, sums
 * are FP32, no weight is rounded.  Made for few rows per expert (decoding); any number is right.  x is finite, and so is 31
 * times the sum of a group's |x| in FP32 (codes are multiplied as 16 + q): a row with an infinity, a NaN or such a sum gives
 * NaN, in that row only.  n up to 2^20 of any size, k a multiple of the group up to 2^20. */

/* Bytes of packed weights [experts x n x k] (negative MGS_ERR_* on invalid arguments). */
int64_t mgs_w4_nbytes(int32_t experts, int64_t n, int64_t k, int32_t group, int32_t zeros);

/* Lays weights out for the products below, once.
 *   codes [experts x n x k / 2], two codes a byte, the even element in the low half; scales_bf16 [experts x n x k / group];
 *   zeros [experts x n x k / group] (0 .. 15) or NULL; out mgs_w4_nbytes() bytes, 16-byte aligned */
int mgs_w4_pack(int32_t experts, int64_t n, int64_t k, int32_t group, const uint8_t* codes, const void* scales_bf16,
                const uint8_t* zeros, void* out, void* stream);

/* Codes, scales and zero points (NULL: symmetric) of finite BF16 weights [experts x n x k], round to nearest.  With zero
 * points the steps cover [min(w, 0), max(w, 0)] of a group in 15, without them [-amax, amax] in 14; the scale is
 * rounded to BF16 before the codes are taken. */
int mgs_w4_quantize(int32_t experts, int64_t n, int64_t k, int32_t group, const void* w_bf16, uint8_t* codes, void* scales_bf16,
                    uint8_t* zeros, void* stream);

/* c [M x n] = x_g w_g^T + bias: x_bf16 [M x k] and w (packed [E x n x k], `zeros` as it was packed) 16-byte aligned,
 * bias_bf16 [E x n] nullable, c BF16 or F32.  No output may be or overlap another tensor of the call, here and below. */
int mgs_grouped_gemm_w4(const mgs_groups* groups, int64_t n, int64_t k, int32_t group, int32_t zeros, const void* x_bf16,
                        const void* w, const void* bias_bf16, void* c, int32_t c_dtype, void* stream);

/* h [M x f] BF16 = act(gate, up) * probs[row] in one kernel, [gate | up] = x_g w_g^T + bias; w packed [E x 2f x k], f a
 * multiple of 16 up to 2^19; act, bias_bf16 [E x 2f] and probs as in mgs_grouped_gated_fwd. */
int mgs_grouped_gated_w4(const mgs_act_params* act, const mgs_groups* groups, int64_t f, int64_t k, int32_t group, int32_t zeros,
                         const void* x_bf16, const void* w, const void* bias_bf16, const float* probs, void* h_bf16, void* stream);

/* ---- Norm of the gradients ------------------------------------------------------------------------- */

/* One gradient: `numel` contiguous elements, and where its scaled values go (the same address and type: in place). */
typedef struct {
  const void* grad;
  void* out;
  int64_t numel;
  int32_t grad_dtype, out_dtype; /* mgs_dtype */
} mgs_grad;

/* norm[0] = the square root of the sum of the squares of all elements of all gradients, summed in FP64 in a fixed order;
 * with clip != 0 also out = grad * min(1, max_norm / (norm + eps)): the factor is taken from the FP64 norm and rounded to
 * FP32, the product is FP32, and a BF16 output rounds that product again.  A NaN norm makes every output NaN, an infinite
 * gradient zeros (NaN in its own place); a finite norm past FP32's range is returned as infinity and clips like any other.
 * `grads` is a HOST array of `count`; empty gradients may be NULL.  No output may be or overlap another tensor of the
 * call, but for a gradient scaled in place.
 *   workspace  mgs_grad_norm_workspace_bytes() bytes, 8-byte aligned, caller-owned, contents undefined before and
 *              after; calls sharing it must not overlap */
int mgs_grad_norm(int32_t count, const mgs_grad* grads, float* norm, void* workspace, int64_t workspace_bytes, int32_t clip,
                  float max_norm, float eps, void* stream);

int64_t mgs_grad_norm_workspace_bytes(int32_t count, const mgs_grad* grads);

#ifdef __cplusplus
}
#endif

#endif /* MGS_H */
