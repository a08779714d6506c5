/*
 * emu_block -- the operators of a transformer block around the GEMMs of
 * emu_sgemm.h, on AMD MI355X (gfx950): layer norm, the linear layer with its
 * activation and residual sum in the GEMM's epilogue, the gated feed-forward
 * projection, the weight-gradient product, and their backward passes.
 *
 * An interatomic potential derives forces from the input gradient, and
 * training on forces differentiates that gradient once more ("Unlocking
 * Tensor Core Performance for Machine Learning Interatomic Potentials",
 * section "TF32x3 on Ampere GPUs").  Every operator therefore has a backward
 * pass, and each backward pass that is not itself a matrix product has one
 * of its own (the *_backward2 functions).
 *
 * Conventions
 *   - All of emu_sgemm.h's: row-major FP32 device arrays owned by the caller,
 *     leading dimensions in elements, emu_status_t results, argument checks
 *     before any HIP call, asynchronous work on `stream`, re-entrant.
 *   - Nothing is allocated, on the host or the device.  A function that needs
 *     a workspace takes one from the caller: `workspace` of at least the
 *     bytes its *_workspace function reports, 256-byte aligned, not in use by
 *     work that may overlap the call.  EMU_STATUS_INVALID_VALUE if it is too
 *     small, NULL while bytes are needed, or misaligned.  Every call can
 *     therefore be captured in a HIP graph, which then owns its workspace
 *     through its caller.
 *   - Any pointer alignment (4 bytes) and any leading dimension meeting the
 *     bounds is accepted.  Arrays of an element count past 2^31 are.
 *   - Results are deterministic: no atomics, sums in a fixed order.
 *   - Outputs may not overlap inputs unless said otherwise.
 *   - Non-finite values follow the formulas in FP32.
 */
#ifndef EMU_BLOCK_H
#define EMU_BLOCK_H

#include "emu_sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Version of this header (major * 100 + minor). */
int emu_block_version(void);

/* ---- layer norm ------------------------------------------------------------
 *
 * Per row of x (rows x cols, ldx >= cols), with n = cols:
 *   mu = mean(x), r = (mean((x - mu)^2) + eps)^(-1/2), xhat = (x - mu) r,
 *   y = xhat * weight + bias.
 * weight, bias: cols floats, or NULL (1 and 0).  mean, rstd: rows floats that
 * receive mu and r, or NULL.  The row is held in registers: mean and squared
 * deviations are two sums over exact inputs, not a difference of moments, and
 * the mean, corrected by that of the centred row, is good to its own rounding
 * (in a row of one value it is that value).
 * y may be x.
 * Errors: EMU_STATUS_INVALID_VALUE for rows < 0, cols < 1, a leading
 * dimension < cols, eps < 0 or NaN, or (rows > 0) a NULL x or y;
 * EMU_STATUS_NOT_SUPPORTED for cols > EMU_LAYER_NORM_MAX_COLS or a device
 * that is not gfx950.
 */
#define EMU_LAYER_NORM_MAX_COLS 16384

emu_status_t emu_layer_norm(int64_t rows, int64_t cols, const float* x, int64_t ldx,
                            const float* weight, const float* bias, float eps, float* y, int64_t ldy,
                            float* mean, float* rstd, void* stream);

/*
 * Gradients of layer norm from dy (rows x cols), with a = weight * dy:
 *   dx = r (a - mean(a) - xhat mean(a xhat)),
 *   dweight = sum over rows of dy xhat,  dbias = sum over rows of dy.
 * x, weight as in the forward call, mean and rstd as it wrote them.  dx,
 * dweight, dbias: each may be NULL.  rows == 0 zeroes dweight and dbias.
 * dx may be dy.  A workspace is needed for dweight and dbias only.
 */
emu_status_t emu_layer_norm_backward_workspace(int64_t rows, int64_t cols, size_t* bytes);
emu_status_t emu_layer_norm_backward(int64_t rows, int64_t cols, const float* dy, int64_t lddy,
                                     const float* x, int64_t ldx, const float* weight,
                                     const float* mean, const float* rstd, float* dx, int64_t lddx,
                                     float* dweight, float* dbias, void* workspace,
                                     size_t workspace_bytes, void* stream);

/*
 * Gradients of the backward pass: for a scalar L with v = dL/d(dx) (rows x
 * cols), p = dL/d(dweight), q = dL/d(dbias) (cols; each of the three may be
 * NULL = zero), and a = weight * dy:
 *   s    = r (v - mean(v) - xhat mean(v xhat)),
 *   gdy  = weight * s + p * xhat + q             (dL/d(dy), rows x cols)
 *   gw   = sum over rows of dy * s               (dL/d(weight), cols)
 *   h    = p * dy - r (a mean(v xhat) + v mean(a xhat)),
 *   gx   = r (h - mean(h) - xhat mean(h xhat)) - xhat r^2 mean(v P a),
 *          P a = a - mean(a) - xhat mean(a xhat)  (dL/dx, rows x cols).
 * gdy, gx, gw: each may be NULL.  A workspace (that of the backward pass)
 * is needed for gw only.
 */
emu_status_t emu_layer_norm_backward2(int64_t rows, int64_t cols, const float* v, int64_t ldv,
                                      const float* p, const float* q, const float* dy, int64_t lddy,
                                      const float* x, int64_t ldx, const float* weight,
                                      const float* mean, const float* rstd, float* gdy, int64_t ldgdy,
                                      float* gx, int64_t ldgx, float* gw, void* workspace,
                                      size_t workspace_bytes, void* stream);

/* ---- activations -------------------------------------------------------------
 * GELU is z Phi(z); GELU_TANH its form z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715
 * z^3))); SILU z / (1 + e^-z); RELU's slope at 0 is 0. */
typedef enum {
    EMU_ACT_IDENTITY = 0,
    EMU_ACT_RELU = 1,
    EMU_ACT_SILU = 2,
    EMU_ACT_GELU = 3,
    EMU_ACT_GELU_TANH = 4,
    EMU_ACT_TANH = 5
} emu_act_t;

/* dz = dy * act'(z), all rows x cols.  dz may be dy or z. */
emu_status_t emu_act_backward(int64_t rows, int64_t cols, const float* dy, int64_t lddy,
                              const float* z, int64_t ldz, emu_act_t act, float* dz, int64_t lddz,
                              void* stream);
/* From v = dL/d(dz): gdy = v act'(z), gz = v dy act''(z) (each may be NULL). */
emu_status_t emu_act_backward2(int64_t rows, int64_t cols, const float* v, int64_t ldv,
                               const float* dy, int64_t lddy, const float* z, int64_t ldz,
                               emu_act_t act, float* gdy, int64_t ldgdy, float* gz, int64_t ldgz,
                               void* stream);

/* ---- linear layer with activation and residual ---------------------------------
 *
 *   z = A . op(B) + bias,   C = act(z) + R
 * A: M x K, op(B): K x N (transB as in emu_sgemm), bias: N floats or NULL, R:
 * M x N (ldr >= N) or NULL, C: M x N.  C may be R.
 * Z: M x N (ldz >= N) receives z, for the backward pass, or NULL.
 * One rounding per operation, in the order written; act in FP32.
 *
 * mode: as emu_sgemm's, and the product is emu_sgemm's in the explicit modes,
 * bit for bit (a row of C never depends on the other rows).  EMU_MODE_AUTO: for few
 * rows (where a cost model predicts it faster: emu_sgemm_act_route) one launch
 * that reads the operands as they are, on FP32 matrix instructions or as
 * BF16X9, otherwise what emu_sgemm's AUTO runs, its K split plan included.
 * The explicit emulated modes take such a launch for few rows too, with the
 * same bits.
 * planes: op(B) split by emu_presplit_b in `mode` (an emulated one), or in
 * BF16X9 for EMU_MODE_AUTO, which then runs BF16X9 whatever the shape; B and
 * ldb are not read.  NULL: the call splits op(B) into the workspace.
 * K == 0: z = bias.  M == 0 or N == 0: nothing is done.
 * Errors: EMU_STATUS_INVALID_VALUE as emu_sgemm_ex and for a bad act, NULL
 * required pointers or leading dimensions below their bounds;
 * EMU_STATUS_NOT_SUPPORTED for K above 8,388,604 or N above 2^30.
 */
emu_status_t emu_sgemm_act_workspace(emu_op_t transB, int64_t M, int64_t N, int64_t K, const float* A,
                                     int64_t lda, int has_planes, emu_mode_t mode, size_t* bytes);
emu_status_t emu_sgemm_act(emu_op_t transB, int64_t M, int64_t N, int64_t K, const float* A,
                           int64_t lda, const float* B, int64_t ldb, const void* planes,
                           const float* bias, emu_act_t act, float* Z, int64_t ldz, const float* R,
                           int64_t ldr, float* C, int64_t ldc,
                           emu_mode_t mode, void* workspace, size_t workspace_bytes, void* stream);
/* *few_rows = 1 where AUTO takes the one-launch FP32 kernel for this shape, 2
 * where it takes the one-launch BF16X9 kernel, else 0 (then AUTO is
 * emu_sgemm_select's mode).  A host function. */
emu_status_t emu_sgemm_act_route(emu_op_t transB, int64_t M, int64_t N, int64_t K, int* few_rows);

/* ---- gated feed-forward projection ---------------------------------------------
 *
 * W: 2F x K (rows 0..F-1 the gate's, F..2F-1 the up projection's; ldw >= K),
 * bias: 2F floats in the same order, or NULL:
 *   [g | u] = A . W^T + bias  (M x 2F),   C = act(g) * u  (M x F).
 * Z: M x 2F (ldz >= 2F) receives [g | u] for the backward pass, or NULL.
 * mode, errors: as emu_sgemm_act.  planes: W split by emu_presplit_gated.
 */
emu_status_t emu_sgemm_gated_workspace(int64_t M, int64_t F, int64_t K, const float* A, int64_t lda,
                                       int has_planes, emu_mode_t mode, size_t* bytes);
emu_status_t emu_sgemm_gated(int64_t M, int64_t F, int64_t K, const float* A, int64_t lda,
                             const float* W, int64_t ldw, const void* planes, const float* bias,
                             emu_act_t act, float* Z, int64_t ldz, float* C, int64_t ldc,
                             emu_mode_t mode, void* workspace, size_t workspace_bytes, void* stream);
emu_status_t emu_presplit_gated_bytes(int64_t F, int64_t K, emu_mode_t mode, size_t* bytes);
emu_status_t emu_presplit_gated(int64_t F, int64_t K, const float* W, int64_t ldw, emu_mode_t mode,
                                void* planes, void* stream);

/* From dh (M x F) and Z = [g | u]: dZ = [dh u act'(g) | dh act(g)] (M x 2F).
 * dZ may be Z. */
emu_status_t emu_gated_backward(int64_t M, int64_t F, const float* dh, int64_t lddh, const float* Z,
                                int64_t ldz, emu_act_t act, float* dZ, int64_t lddz, void* stream);
/* From V = [vg | vu] = dL/d(dZ): gdh = vg u act'(g) + vu act(g) (M x F), and
 * gZ = [vg dh u act''(g) + vu dh act'(g) | vg dh act'(g)] (M x 2F); each may
 * be NULL. */
emu_status_t emu_gated_backward2(int64_t M, int64_t F, const float* V, int64_t ldv, const float* dh,
                                 int64_t lddh, const float* Z, int64_t ldz, emu_act_t act, float* gdh,
                                 int64_t ldgdh, float* gZ, int64_t ldgz, void* stream);

/* ---- weight gradient --------------------------------------------------------------
 *
 *   dW = dZ^T X  (M x N),   db = sum over rows of dZ  (M; or NULL)
 * dZ: rows x M (lddz >= M), X: rows x N (ldx >= N).  In FP32 on the FP32
 * matrix instruction ("ordinary precision", as the pages keep the weight
 * gradient); rows are summed in segments that are joined in order.  rows ==
 * 0: zeros.  M == 0 or N == 0: dW is empty, db is still formed.
 * EMU_STATUS_NOT_SUPPORTED for lddz or ldx above 16,777,088.
 */
emu_status_t emu_wgrad_workspace(int64_t rows, int64_t M, int64_t N, size_t* bytes);
emu_status_t emu_wgrad(int64_t rows, int64_t M, int64_t N, const float* dZ, int64_t lddz,
                       const float* X, int64_t ldx, float* dW, int64_t lddw, float* db,
                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * The same with the activation's backward pass on the way: dZ, which the
 * input-gradient product needs too, is made from dY and Z as by
 * emu_act_backward (emu_gated_backward: dH, Z = [g | u], dZ = [dg | du], dW
 * 2F x N, db 2F), written once and multiplied in the same pass.  dZ may not
 * overlap dY or Z.  Workspaces: emu_wgrad_workspace(rows, M, N),
 * emu_wgrad_gated_workspace(rows, F, N).
 */
emu_status_t emu_wgrad_act(int64_t rows, int64_t M, int64_t N, const float* dY, int64_t lddy,
                           const float* Z, int64_t ldz, emu_act_t act, float* dZ, int64_t lddz,
                           const float* X, int64_t ldx, float* dW, int64_t lddw, float* db,
                           void* workspace, size_t workspace_bytes, void* stream);
emu_status_t emu_wgrad_gated_workspace(int64_t rows, int64_t F, int64_t N, size_t* bytes);
emu_status_t emu_wgrad_gated(int64_t rows, int64_t F, int64_t N, const float* dH, int64_t lddh,
                             const float* Z, int64_t ldz, emu_act_t act, float* dZ, int64_t lddz,
                             const float* X, int64_t ldx, float* dW, int64_t lddw, float* db,
                             void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* EMU_BLOCK_H */
