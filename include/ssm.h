/*
 * ssm.h -- C ABI of the MI355X (gfx950) operators that follow the short causal convolution of
 * conv1d.h in a mixer block: the selective state space scan with head-wise decay (forward over
 * packed prompts, training backward, one-token step against a slot pool), the gated RMS norm of the
 * scan's output, and the residual addition with the RMS norm before the next block.
 *
 * The scan, for every packed sequence, head h of group g = h / (H / G) and row t:
 *     dt'_t = softplus(dt_t + dt_bias[h])   (or dt_t + dt_bias[h] without softplus)
 *     S_t   = exp(dt'_t A[h]) S_{t-1} + dt'_t x_t B_t^T        S is [P, N], FP32
 *     y_t   = S_t C_t + D[h] x_t                                rounded to bf16 once
 * x, y: [rows, H, P], B, C: [rows, G, N], dt: [rows, H].
 *
 * Conventions, as in conv1d.h: device pointers, caller-owned buffers, no allocation, no host read of
 * device memory, no synchronization, every call only enqueues on `stream` (graph capturable);
 * host-checkable preconditions return CONV1D_EINVAL / CONV1D_EWORKSPACE with nothing launched; offsets
 * and slots are the caller's constraint (for memory safety offsets are clamped to [0, rows] and a slot
 * outside [0, slots) acts as -1).  Status codes are conv1d_status.
 *   - x, y, dy, dx, B, C, dB, dC: bf16; a row's heads (groups) and columns are contiguous, the row
 *     stride `*_ld` (elements) is free, so they may be column ranges of one wider array (the
 *     convolution's output holds x, B and C side by side).  dt, ddt: FP32 or bf16 (`dt_dtype`).
 *     A, D, dt_bias, states and all parameter gradients: FP32.
 *   - 1 <= N <= SSM_MAX_STATE, G divides H, any P >= 1.
 *   - seq: the cu_seqlens or the batch-row form of conv1d_seq (seq_idx must be NULL).
 *   - States, their sums over rows, decays, norms and every reduction are FP32 or better.  Matrix
 *     instructions take bf16 operands: x, B, C and dy as they are; what is FP32 is rounded or cut into
 *     parts.  Scan: the decayed scores and the state in S_t C_t are rounded to bf16, 2^-8 of a term of y at
 *     most each; a state's new terms enter as two parts, 2^-16 of a term.  Its backward: the decayed scores in
 *     dx, dB and dC and the state's adjoint in dx are rounded to bf16; all else (states and adjoints, ddt, dA,
 *     dinitial_state) enters as three parts, FP32's 24 bits.  The step and the norms are FP32 throughout.
 *   - Results do not depend on the workspace's contents or address, and there are no atomics: equal calls
 *     give equal bits.
 */
#ifndef SSM_H
#define SSM_H

#include "conv1d.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SSM_MAX_STATE 256
#define SSM_MAX_NORM_GROUP 32768
#define SSM_MAX_ROW_STRIDE (1 << 24) /* elements; the scan's row strides are at most this */

typedef struct {
  int64_t H, P, G, N;
  int dt_dtype;    /* conv1d_dtype of dt and ddt */
  int dt_softplus; /* 1: softplus(dt + dt_bias), 0: dt + dt_bias */
} ssm_shape;

/* FP32 states [slots, H, P, N], [H, P, N] contiguous, slots s_slot elements apart (s_slot >= H*P*N).
   Sequence i uses slot cache_indices[i] (int32, -1: +0 output rows and no state access), or slot i
   when cache_indices is NULL (then slots >= nseq).  initial: read where has_initial_state (uint8
   [nseq]) is true, zeros elsewhere; NULL = zeros everywhere.  has_initial_state NULL: all false with
   cache_indices, as in conv1d_pool, and all true without.  final: written with the state after the
   sequence's last row; NULL = not wanted.  initial == final updates a pool in place: slots of empty
   sequences then stay as they are; a separate final array gets their start. */
typedef struct {
  const float* initial;
  float* final;
  int64_t slots, s_slot;
  const int32_t* cache_indices;
  const uint8_t* has_initial_state;
} ssm_states;

/* Forward.  states: NULL for zero start and no final states.  D, dt_bias: FP32 [H] or NULL.  y must
   not overlap any input; rows outside every sequence are not written.  An infinity or NaN makes
   not finite what the recurrence takes it to and changes nothing else: of x, its column from its row on; of dt
   and B, their head and group from the row on; of C, its group in the row.  ws: at least
   ssm_scan_fwd_workspace_bytes(...) bytes, 16-byte aligned (NULL when that is 0). */
int ssm_scan_fwd(const ssm_shape* shape, int64_t rows, const void* x, int64_t x_ld, const void* dt, int64_t dt_ld,
                 const float* A, const void* B, int64_t B_ld, const void* C, int64_t C_ld, const float* D,
                 const float* dt_bias, const conv1d_seq* seq, const ssm_states* states, void* y, int64_t y_ld,
                 void* ws, size_t ws_bytes, hipStream_t stream);
size_t ssm_scan_fwd_workspace_bytes(const ssm_shape* shape, int64_t rows, int64_t nseq);

/* Backward of ssm_scan_fwd with start states initial_state [nseq, H, P, N] (NULL: zeros), given
   dy = dL/dy and dfinal_state = dL/d(final states) [nseq, H, P, N] (NULL: zero).  Writes dx, ddt
   (gradient of the raw dt, dt's type), dB, dC (summed over the group's heads in FP32, rounded once),
   dA [H], and, unless NULL, dD [H], ddt_bias [H], dinitial_state [nseq, H, P, N] (an empty sequence's
   is its dfinal_state).  Outputs must not overlap inputs or one another.  Rows outside every sequence
   are not written.  An infinity or NaN stays in its sequence and its head (that of B and C, and all in dB
   and dC, in the group); there it may reach rows on either side.  It recomputes everything from the
   inputs; ws: at least ssm_scan_bwd_workspace_bytes(...) bytes, 16-byte aligned. */
int ssm_scan_bwd(const ssm_shape* shape, int64_t rows, const void* dy, int64_t dy_ld, const void* x, int64_t x_ld,
                 const void* dt, int64_t dt_ld, const float* A, const void* B, int64_t B_ld, const void* C,
                 int64_t C_ld, const float* D, const float* dt_bias, const conv1d_seq* seq,
                 const float* initial_state, const float* dfinal_state, void* dx, int64_t dx_ld, void* ddt,
                 int64_t ddt_ld, float* dA, void* dB, int64_t dB_ld, void* dC, int64_t dC_ld, float* dD,
                 float* ddt_bias, float* dinitial_state, void* ws, size_t ws_bytes, hipStream_t stream);
size_t ssm_scan_bwd_workspace_bytes(const ssm_shape* shape, int64_t rows, int64_t nseq);

/* One token a sequence: x, y [nseq, H, P], dt [nseq, H], B, C [nseq, G, N].  pool: initial == final,
   cache_indices required (has_initial_state is ignored: the state is always read).  The scan's
   recurrence for one row; slot -1 gives +0 and no state access. */
int ssm_state_update(const ssm_shape* shape, int64_t nseq, const void* x, int64_t x_ld, const void* dt, int64_t dt_ld,
                     const float* A, const void* B, int64_t B_ld, const void* C, int64_t C_ld, const float* D,
                     const float* dt_bias, const ssm_states* pool, void* y, int64_t y_ld, hipStream_t stream);

/* Gated RMS norm over groups of `group` channels (group divides d, at most SSM_MAX_NORM_GROUP):
     norm_before_gate = 0:  u = x silu(z),  y = w u / rms(u)
     norm_before_gate = 1:  u = x,          y = w u / rms(u) silu(z)
   with rms(u)^2 = mean(u^2) + eps.  x, z, y: bf16 [rows, d], row strides free; w: [d], FP32 or bf16.
   The backward recomputes the norm and writes dx, dz (bf16) and dw (FP32 [d]); ws: at least
   norm_bwd_workspace_bytes(rows, d, group) bytes, 16-byte aligned. */
int gated_norm_fwd(int64_t rows, int64_t d, int64_t group, const void* x, int64_t x_ld, const void* z, int64_t z_ld,
                   const void* w, int w_dtype, int norm_before_gate, float eps, void* y, int64_t y_ld,
                   hipStream_t stream);
int gated_norm_bwd(int64_t rows, int64_t d, int64_t group, const void* dy, int64_t dy_ld, const void* x, int64_t x_ld,
                   const void* z, int64_t z_ld, const void* w, int w_dtype, int norm_before_gate, float eps, void* dx,
                   int64_t dx_ld, void* dz, int64_t dz_ld, float* dw, void* ws, size_t ws_bytes, hipStream_t stream);

/* Residual addition and RMS norm: r' = residual + scale x, stored in the residual's type (FP32 or
   bf16), y = w r' / rms(r') from the stored r'.  r' may be the residual's own buffer.  The backward
   takes dy, the stored r' and dr_out = dL/dr' from its other reader (NULL: none), and writes
   dresidual = dr_out + (gradient through the norm) in r's type, dx = scale dresidual (bf16), dw.
   dresidual may be dr_out's own buffer. */
int residual_norm_fwd(int64_t rows, int64_t d, const void* x, int64_t x_ld, const void* residual, int64_t residual_ld,
                      int residual_dtype, float scale, const void* w, int w_dtype, float eps, void* y, int64_t y_ld,
                      void* residual_out, int64_t residual_out_ld, hipStream_t stream);
int residual_norm_bwd(int64_t rows, int64_t d, const void* dy, int64_t dy_ld, const void* dr_out, int64_t dr_out_ld,
                      const void* residual_out, int64_t residual_out_ld, int residual_dtype, float scale,
                      const void* w, int w_dtype, float eps, void* dx, int64_t dx_ld, void* dresidual,
                      int64_t dresidual_ld, float* dw, void* ws, size_t ws_bytes, hipStream_t stream);
size_t norm_bwd_workspace_bytes(int64_t rows, int64_t d, int64_t group);

#ifdef __cplusplus
}
#endif

#endif /* SSM_H */
