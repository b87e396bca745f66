/*
 * delta.h -- C ABI of the MI355X (gfx950) operators of a mixer block with the gated delta rule, beside those of conv1d.h
 * and ssm.h: the rule over packed prompts, its training backward, its one-token step against a slot pool; the layer
 * norm before a block, alone or of the residual's sum; and copies between the slots of any of the pools.
 *
 * The rule, for every packed sequence, value head h of key head g = h / (H / G) and row t:
 *     a_t = exp(A[h] softplus(dt_t + dt_bias[h]))          (or A[h] (dt_t + dt_bias[h]) without softplus)
 *     r_t = beta_max / (1 + exp(-b_t))
 *     u_t = r_t (v_t - a_t S_{t-1} k_t)
 *     S_t = a_t S_{t-1} + u_t k_t^T                         S is [P, N], FP32, as in ssm.h
 *     y_t = scale S_t q_t                                   rounded to bf16 once
 * v, y: [rows, H, P], q, k: [rows, G, N], dt, b: [rows, H].  With qk_norm, q and k stand for q / sqrt(|q|^2 + norm_eps)
 * and k / sqrt(|k|^2 + norm_eps); without, the rule grows without bound where r_t |k_t|^2 > 2.
 *
 * Conventions, status codes, sequences, row strides, slots and states are those of ssm.h: device pointers,
 * caller-owned buffers, no allocation, no host read of device memory, no synchronization, every call only enqueues on
 * `stream`.  q, k, v, y and their gradients: bf16; dt, b, ddt, db: FP32 or bf16 (`gate_dtype`); A, dt_bias, states and
 * the parameters' gradients: FP32.  1 <= N <= SSM_MAX_STATE, G divides H, any P >= 1.
 *   - States, decays, norms, the chunks' triangular systems and every reduction are FP32 or better.  Matrix instructions
 *     take FP32 operands as two fp16 parts, which hold 22 bits of the largest value of a state's column, of a row of new
 *     values or of a tile and an absolute 2^-25 of it below; the walked state therefore keeps 22 bits of its column's
 *     largest.  Norms and rates are FP32 factors beside the products.  What enters y, dq and dk alone is rounded further: in
 *     y the state that comes into a chunk to its first part (2^-12 of a term), new values and decayed scores to two bf16
 *     parts (2^-17); in dq and dk the decayed scores to two.
 *   - scale is finite, beta_max finite and positive, norm_eps finite and not negative.  The squares of a row of q or k are
 *     summed in FP32 in the step and the backward: a row whose sum overflows counts as not finite there.  norm_eps = 0 gives
 *     a row of zeros no direction, NaN.
 *   - Equal calls give equal bits, whatever the workspace holds.
 */
#ifndef DELTA_H
#define DELTA_H

#include "ssm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int64_t H, P, G, N;
  int gate_dtype;  /* conv1d_dtype of dt, b, ddt and db */
  int dt_softplus; /* 1: A softplus(dt + dt_bias), 0: A (dt + dt_bias) */
  int qk_norm;     /* 1: unit q and k */
  float scale, beta_max, norm_eps;
} delta_shape;

/* Forward.  states: as for ssm_scan_fwd, NULL for zero start and no final states.  dt_bias: [H] or NULL.  y must not
   overlap any input; rows outside every sequence are not written.  An infinity or NaN of v makes its column of its head
   not finite from its row on; one of k, dt or b the whole head; of q, its row.  ws: at least
   delta_scan_fwd_workspace_bytes(...) bytes, 16-byte aligned. */
int delta_scan_fwd(const delta_shape* shape, int64_t rows, const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                   const void* v, int64_t v_ld, const void* dt, int64_t dt_ld, const void* b, int64_t b_ld,
                   const float* A, const float* dt_bias, const conv1d_seq* seq, const ssm_states* states, void* y,
                   int64_t y_ld, void* ws, size_t ws_bytes, hipStream_t stream);
size_t delta_scan_fwd_workspace_bytes(const delta_shape* shape, int64_t rows, int64_t nseq);

/* Backward with start states initial_state [nseq, H, P, N] (NULL: zeros), given dy = dL/dy and dfinal_state =
   dL/d(final states) (NULL: zero).  Writes dq, dk (summed over a key head's value heads in FP32, rounded once), dv, ddt and
   db (gradients of the raw dt and b), dA [H], and, unless NULL, ddt_bias [H] and dinitial_state [nseq, H, P, N] (an empty
   sequence's is its dfinal_state).  Outputs must not overlap inputs or one another.  Rows outside every sequence are not
   written.  An infinity or NaN stays in its sequence and its key head's heads; there it may reach rows on either side.
   ws: at least delta_scan_bwd_workspace_bytes(...) bytes, 16-byte aligned. */
int delta_scan_bwd(const delta_shape* shape, int64_t rows, const void* dy, int64_t dy_ld, const void* q, int64_t q_ld,
                   const void* k, int64_t k_ld, const void* v, int64_t v_ld, const void* dt, int64_t dt_ld,
                   const void* b, int64_t b_ld, const float* A, const float* dt_bias, const conv1d_seq* seq,
                   const float* initial_state, const float* dfinal_state, void* dq, int64_t dq_ld, void* dk,
                   int64_t dk_ld, void* dv, int64_t dv_ld, void* ddt, int64_t ddt_ld, void* db, int64_t db_ld,
                   float* dA, float* ddt_bias, float* dinitial_state, void* ws, size_t ws_bytes, hipStream_t stream);
size_t delta_scan_bwd_workspace_bytes(const delta_shape* shape, int64_t rows, int64_t nseq);

/* One token a sequence: q, k [nseq, G, N], v, y [nseq, H, P], dt, b [nseq, H].  pool as for ssm_state_update: the state is
   always read; slot -1 gives +0 and no state access.  FP32 throughout. */
int delta_state_update(const delta_shape* shape, int64_t nseq, const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                       const void* v, int64_t v_ld, const void* dt, int64_t dt_ld, const void* b, int64_t b_ld,
                       const float* A, const float* dt_bias, const ssm_states* pool, void* y, int64_t y_ld,
                       hipStream_t stream);

/* Layer norm over the d channels of a row (d at most SSM_MAX_NORM_GROUP): y = w (h - mean(h)) / sqrt(var(h) + eps) + bias.
   residual NULL: h = x (residual_out is not written).  Otherwise h = residual + scale x, stored to residual_out in the
   residual's type (FP32 or bf16) and read as stored; it may be the residual's own buffer.  x, y: bf16 [rows, d]; w and
   bias (NULL: zero): [d], FP32 or bf16 (`w_dtype`).
   The backward takes dy, the normed h as it is stored (x itself, or residual_out), and dr_out = dL/dh from its other reader
   (NULL: none), and writes, with g = dr_out + (gradient through the norm): dx = scale g (bf16), dresidual = g in h's type
   (NULL: not wanted; it may be dr_out's own buffer), dw, dbias (NULL: not wanted), FP32 [d].  ws: at least
   layer_norm_bwd_workspace_bytes(rows, d) bytes, 16-byte aligned. */
int layer_norm_fwd(int64_t rows, int64_t d, const void* x, int64_t x_ld, const void* residual, int64_t residual_ld,
                   int residual_dtype, float scale, const void* w, const void* bias, int w_dtype, float eps, void* y,
                   int64_t y_ld, void* residual_out, int64_t residual_out_ld, hipStream_t stream);
int layer_norm_bwd(int64_t rows, int64_t d, const void* dy, int64_t dy_ld, const void* dr_out, int64_t dr_out_ld,
                   const void* h, int64_t h_ld, int h_dtype, float scale, const void* w, int w_dtype, float eps,
                   void* dx, int64_t dx_ld, void* dresidual, int64_t dresidual_ld, float* dw, float* dbias, void* ws,
                   size_t ws_bytes, hipStream_t stream);
size_t layer_norm_bwd_workspace_bytes(int64_t rows, int64_t d);

/* Copies between slots, of up to SLOT_MAX_POOLS pools in one call: for every pair i < n, slot target[i] of each pool
   becomes what slot source[i] held before the call (all reads come before all writes, so slots may be swapped or taken
   several times), or zero bytes where source[i] is negative.  A pair with a target outside [0, slots) or a source >= slots
   of a pool leaves that pool as it is.  A pool's slots are slot_bytes long and s_slot >= slot_bytes bytes apart, of any
   alignment.  Targets must be distinct; pools must not share a byte.  n is at most SLOT_MAX_PAIRS. */
#define SLOT_MAX_POOLS 8
#define SLOT_MAX_PAIRS 8192
typedef struct {
  void* ptr;
  int64_t slots, slot_bytes, s_slot;
} slot_pool;
int state_copy(const slot_pool* pools, int npools, int64_t n, const int32_t* source, const int32_t* target,
               hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DELTA_H */
