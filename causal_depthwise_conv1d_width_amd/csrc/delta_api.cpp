// delta_api.cpp -- the C ABI of include/delta.h: host-side validation, workspace layout and launches.
// Every precondition the host can see is checked before anything is enqueued; nothing here reads
// device memory, allocates or synchronizes.
#include "delta.h"

#include <stdint.h>

#include "api_checks.h"
#include "delta_launch.h"

using namespace cssm;

namespace {

constexpr float kMaxFloat = 3.40282347e38f;

bool shape_ok(const delta_shape* s) {
  return s && s->H >= 1 && s->P >= 1 && s->G >= 1 && s->N >= 1 && s->N <= kMaxState && s->H % s->G == 0 &&
         s->H <= (1 << 20) && s->P <= (1 << 20) && dtype_ok(s->gate_dtype) && (s->dt_softplus == 0 || s->dt_softplus == 1) &&
         (s->qk_norm == 0 || s->qk_norm == 1) && s->norm_eps >= 0.f && s->norm_eps <= kMaxFloat && s->beta_max > 0.f &&
         s->beta_max <= kMaxFloat && s->scale >= -kMaxFloat && s->scale <= kMaxFloat;
}

// every extent of the workspace and every launch, bounded by one chunk a row and sequence
bool sizes_ok(const delta_shape* s, int64_t rows, int64_t nseq) {
  const int64_t hp = s->H * ceil_div(s->P, kPTile);
  return rows >= 0 && nseq >= 0 && mul_ok(rows, s->H * s->P) && mul_ok(rows, 64 * s->G * s->N) &&
         mul_ok(ceil_div(rows, kChunk) + nseq + 1, hp * 64 * kMaxState);
}
int64_t chunk_ids(int64_t rows, int64_t nseq) { return ceil_div(rows, kChunk) + nseq; }
// the key heads' records, first in either workspace, and then the sequences' order
int64_t keys_bytes(const delta_shape* s, int64_t rows, int64_t nseq) {
  return align_up(chunk_ids(rows, nseq) * s->G * 2 * key_tile(state_tile(s->N)));
}
int64_t order_bytes(int64_t nseq) { return align_up(nseq * 4); }
bool launches_ok(const delta_shape* s, int64_t rows, int64_t nseq) {
  return unit_blocks(nseq, s->H, s->G, ceil_div(s->P, kPTile), 1) <= kMaxBlocks / 2 &&
         mul_ok(chunk_ids(rows, nseq), s->H) && chunk_ids(rows, nseq) * s->H < kMaxBlocks;
}
// sequences of unknown lengths, the chunk kernel being run
void set_order(DeltaArgs* d, const delta_shape* s, int64_t rows, int64_t nseq) {
  if (d->s.q.cu && nseq > 1 && rows > 0) d->order = reinterpret_cast<int32_t*>(d->keys + keys_bytes(s, rows, nseq));
}
bool vec_ok(const delta_shape* s) { return s->P % 8 == 0 && s->N % 8 == 0; }

void fill(DeltaArgs* d, const delta_shape* s, int64_t rows, const void* q, int64_t q_ld, const void* k, int64_t k_ld,
          const void* v, int64_t v_ld, const void* dt, int64_t dt_ld, const void* b, int64_t b_ld, const float* A,
          const float* dt_bias, const conv1d_seq* seq, int64_t nseq) {
  ScanArgs* a = &d->s;
  a->x = static_cast<const uint16_t*>(v);
  a->B = static_cast<const uint16_t*>(k);
  a->C = static_cast<const uint16_t*>(q);
  a->dt = dt, d->b = b;
  a->x_ld = v_ld, a->B_ld = k_ld, a->C_ld = q_ld, a->dt_ld = dt_ld, d->b_ld = b_ld;
  a->A = A, a->bias = dt_bias;
  a->dt_f32 = s->gate_dtype == CONV1D_F32;
  a->softplus = s->dt_softplus;
  a->H = (int)s->H, a->P = (int)s->P, a->G = (int)s->G, a->N = (int)s->N;
  a->ptiles = (int)ceil_div(s->P, kPTile);
  a->q = Seqs{seq->cu_seqlens, nseq, seq->cu_seqlens ? 1 : seq->seqlen, rows};
  d->scale = s->scale, d->beta_max = s->beta_max, d->norm_eps = s->norm_eps, d->qk_norm = s->qk_norm;
  d->n_chunk_slots = ceil_div(rows, kChunk);
}

int layer_check(int64_t rows, int64_t d, const void* w, const void* bias, int w_dtype, float eps) {
  if (rows < 0 || d < 1 || d > kMaxGroup || !w || !dtype_ok(w_dtype) || !(eps >= 0.f) || !mul_ok(rows, d)) return CONV1D_EINVAL;
  return aligned(w, dsize(w_dtype)) && aligned(bias, dsize(w_dtype)) ? CONV1D_OK : CONV1D_EINVAL;
}

// Byte offsets into the backward's workspace.
struct BwdPlan {
  int64_t rec, rec_rev, tiles, head, bytes;
};
BwdPlan plan_bwd(const delta_shape* s, int64_t rows, int64_t nseq) {
  BwdPlan p{};
  const int64_t ids = chunk_ids(rows, nseq);
  int64_t at = keys_bytes(s, rows, nseq);
  at += order_bytes(nseq);
  p.rec = at, at += align_up(ids * s->H * kRecFwd);
  p.rec_rev = at, at += align_up(ids * s->H * kRecRev);
  p.tiles = at, at += align_up(ids * s->H * ceil_div(s->P, kPTile) * tile_floats(state_tile(s->N)) * 4);
  p.head = at, at += align_up(ids * s->H * 2 * 4);
  p.bytes = at;
  return p;
}

}  // namespace

extern "C" {

size_t delta_scan_fwd_workspace_bytes(const delta_shape* shape, int64_t rows, int64_t nseq) {
  if (!shape_ok(shape) || rows <= 0 || nseq <= 0 || !sizes_ok(shape, rows, nseq)) return 0;
  return (size_t)(keys_bytes(shape, rows, nseq) + order_bytes(nseq) + align_up(chunk_ids(rows, nseq) * shape->H * kRecFwd));
}

int delta_scan_fwd(const delta_shape* shape, int64_t rows, const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                   const void* v, int64_t v_ld, const void* dt, int64_t dt_ld, const void* b, int64_t b_ld,
                   const float* A, const float* dt_bias, const conv1d_seq* seq, const ssm_states* states, void* y,
                   int64_t y_ld, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!shape_ok(shape) || rows < 0 || !A) return CONV1D_EINVAL;
  int64_t nseq = 0;
  if (check_seq(seq, rows, &nseq) != CONV1D_OK || !sizes_ok(shape, rows, nseq)) return CONV1D_EINVAL;
  const int64_t H = shape->H, hp = H * shape->P, gn = shape->G * shape->N, e = dsize(shape->gate_dtype);
  const Operand ops[6] = {{q, q_ld, gn}, {k, k_ld, gn}, {v, v_ld, hp}, {y, y_ld, hp}, {dt, dt_ld, H}, {b, b_ld, H}};
  for (int i = 0; i < 6; ++i)
    if (!scan_operand_ok(ops[i], rows) || !aligned(ops[i].p, i < 4 ? 2 : e)) return CONV1D_EINVAL;
  DeltaArgs d{};
  Span si, sf, sci, shi;
  if (check_states(hp * shape->N, states, nseq, &d.s, &si, &sf, &sci, &shi) != CONV1D_OK) return CONV1D_EINVAL;
  const size_t need = delta_scan_fwd_workspace_bytes(shape, rows, nseq);
  if (need > ws_bytes || (need && !ws)) return CONV1D_EWORKSPACE;
  if (need && !aligned(ws, 16)) return CONV1D_EINVAL;
  const Span reads[10] = {span(q, rows, gn, q_ld, 2), span(k, rows, gn, k_ld, 2), span(v, rows, hp, v_ld, 2),
                          span(dt, rows, H, dt_ld, e), span(b, rows, H, b_ld, e), span(A, H * 4), span(dt_bias, H * 4),
                          sci, shi, span(seq->cu_seqlens, (nseq + 1) * 4)};
  const Span outs[3] = {span(y, rows, hp, y_ld, 2), sf, span(ws, (int64_t)need)};
  if (clash(outs, reads) || overlap(outs[0], si) || overlap(outs[2], si)) return CONV1D_EINVAL;
  // no rows: an in-place pool stays as it is, so only separate final states are left to write
  if (nseq == 0 || (rows == 0 && (!d.s.fin || d.s.fin == d.s.init))) return CONV1D_OK;
  if (!launches_ok(shape, rows, nseq)) return CONV1D_EINVAL;
  fill(&d, shape, rows, q, q_ld, k, k_ld, v, v_ld, dt, dt_ld, b, b_ld, A, dt_bias, seq, nseq);
  d.s.y = static_cast<uint16_t*>(y);
  d.s.y_ld = y_ld;
  d.keys = static_cast<char*>(ws);
  d.rec = d.keys + keys_bytes(shape, rows, nseq) + order_bytes(nseq);
  set_order(&d, shape, rows, nseq);
  return launch_delta_fwd(d, vec_ok(shape), stream) == hipSuccess ? CONV1D_OK : CONV1D_EHIP;
}

size_t delta_scan_bwd_workspace_bytes(const delta_shape* shape, int64_t rows, int64_t nseq) {
  if (!shape_ok(shape) || rows < 0 || nseq <= 0 || !sizes_ok(shape, rows, nseq)) return 0;
  return (size_t)plan_bwd(shape, rows, nseq).bytes;
}

int delta_scan_bwd(const delta_shape* shape, int64_t rows, const void* dy, int64_t dy_ld, const void* q, int64_t q_ld,
                   const void* k, int64_t k_ld, const void* v, int64_t v_ld, const void* dt, int64_t dt_ld,
                   const void* b, int64_t b_ld, const float* A, const float* dt_bias, const conv1d_seq* seq,
                   const float* initial_state, const float* dfinal_state, void* dq, int64_t dq_ld, void* dk,
                   int64_t dk_ld, void* dv, int64_t dv_ld, void* ddt, int64_t ddt_ld, void* db, int64_t db_ld,
                   float* dA, float* ddt_bias, float* dinitial_state, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!shape_ok(shape) || rows < 0 || !A || !dA) return CONV1D_EINVAL;
  int64_t nseq = 0;
  if (check_seq(seq, rows, &nseq) != CONV1D_OK || !sizes_ok(shape, rows, nseq)) return CONV1D_EINVAL;
  const int64_t H = shape->H, hp = H * shape->P, gn = shape->G * shape->N, e = dsize(shape->gate_dtype);
  if (!mul_ok(nseq, hp * shape->N)) return CONV1D_EINVAL;
  const int64_t states = nseq * hp * shape->N * 4;
  const Operand ops[11] = {{dy, dy_ld, hp}, {q, q_ld, gn}, {k, k_ld, gn}, {v, v_ld, hp}, {dq, dq_ld, gn}, {dk, dk_ld, gn},
                           {dv, dv_ld, hp}, {dt, dt_ld, H}, {b, b_ld, H}, {ddt, ddt_ld, H}, {db, db_ld, H}};
  for (int i = 0; i < 11; ++i)
    if (!scan_operand_ok(ops[i], rows) || !aligned(ops[i].p, i < 7 ? 2 : e)) return CONV1D_EINVAL;
  const size_t need = delta_scan_bwd_workspace_bytes(shape, rows, nseq);
  if (need > ws_bytes || (need && !ws)) return CONV1D_EWORKSPACE;
  if (need && !aligned(ws, 16)) return CONV1D_EINVAL;
  const Span reads[11] = {span(dy, rows, hp, dy_ld, 2), span(q, rows, gn, q_ld, 2), span(k, rows, gn, k_ld, 2),
                          span(v, rows, hp, v_ld, 2), span(dt, rows, H, dt_ld, e), span(b, rows, H, b_ld, e),
                          span(A, H * 4), span(dt_bias, H * 4), span(initial_state, states), span(dfinal_state, states),
                          span(seq->cu_seqlens, (nseq + 1) * 4)};
  const Span outs[9] = {span(dq, rows, gn, dq_ld, 2), span(dk, rows, gn, dk_ld, 2), span(dv, rows, hp, dv_ld, 2),
                        span(ddt, rows, H, ddt_ld, e), span(db, rows, H, db_ld, e), span(dA, H * 4), span(ddt_bias, H * 4),
                        span(dinitial_state, states), span(ws, (int64_t)need)};
  if (clash(outs, reads)) return CONV1D_EINVAL;
  DeltaBwdArgs g{};
  g.dA = dA, g.dbias = ddt_bias;
  g.d.s.H = (int)H;
  if (nseq > 0) {
    if (!launches_ok(shape, rows, nseq)) return CONV1D_EINVAL;
    const BwdPlan p = plan_bwd(shape, rows, nseq);
    char* w = static_cast<char*>(ws);
    fill(&g.d, shape, rows, q, q_ld, k, k_ld, v, v_ld, dt, dt_ld, b, b_ld, A, dt_bias, seq, nseq);
    g.d.s.init = initial_state;
    g.d.s.slots = nseq;
    g.d.s.s_slot = hp * shape->N;
    g.d.keys = w;
    g.d.rec = w + p.rec;
    set_order(&g.d, shape, rows, nseq);
    g.dy = static_cast<const uint16_t*>(dy), g.dy_ld = dy_ld;
    g.dfin = dfinal_state, g.dinit = dinitial_state;
    g.dq = static_cast<uint16_t*>(dq), g.dq_ld = dq_ld;
    g.dk = static_cast<uint16_t*>(dk), g.dk_ld = dk_ld;
    g.dv = static_cast<uint16_t*>(dv), g.dv_ld = dv_ld;
    g.ddt = ddt, g.ddt_ld = ddt_ld, g.db = db, g.db_ld = db_ld;
    g.rec_rev = w + p.rec_rev;
    g.tiles = reinterpret_cast<float*>(w + p.tiles);
    g.head_part = reinterpret_cast<float*>(w + p.head);
  }
  return launch_delta_bwd(g, vec_ok(shape), stream) == hipSuccess ? CONV1D_OK : CONV1D_EHIP;
}

int delta_state_update(const delta_shape* shape, int64_t nseq, const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                       const void* v, int64_t v_ld, const void* dt, int64_t dt_ld, const void* b, int64_t b_ld,
                       const float* A, const float* dt_bias, const ssm_states* pool, void* y, int64_t y_ld,
                       hipStream_t stream) {
  if (!shape_ok(shape) || nseq < 0 || !A || !pool || !pool->initial || pool->initial != pool->final) return CONV1D_EINVAL;
  if (!pool->cache_indices || !sizes_ok(shape, nseq, nseq)) return CONV1D_EINVAL;
  const int64_t H = shape->H, hp = H * shape->P, gn = shape->G * shape->N, e = dsize(shape->gate_dtype);
  const Operand ops[6] = {{q, q_ld, gn}, {k, k_ld, gn}, {v, v_ld, hp}, {y, y_ld, hp}, {dt, dt_ld, H}, {b, b_ld, H}};
  for (int i = 0; i < 6; ++i)
    if (!operand_ok(ops[i], nseq) || !aligned(ops[i].p, i < 4 ? 2 : e)) return CONV1D_EINVAL;
  ScanArgs s{};
  Span si, sf, sci, shi;
  if (check_states(hp * shape->N, pool, nseq, &s, &si, &sf, &sci, &shi) != CONV1D_OK) return CONV1D_EINVAL;
  const Span reads[8] = {span(q, nseq, gn, q_ld, 2), span(k, nseq, gn, k_ld, 2), span(v, nseq, hp, v_ld, 2),
                         span(dt, nseq, H, dt_ld, e), span(b, nseq, H, b_ld, e), span(A, H * 4), span(dt_bias, H * 4), sci};
  const Span outs[2] = {span(y, nseq, hp, y_ld, 2), sf};
  if (clash(outs, reads)) return CONV1D_EINVAL;
  if (nseq == 0) return CONV1D_OK;
  if (!mul_ok(nseq, hp) || nseq * H * ceil_div(shape->P, 4) > kMaxBlocks) return CONV1D_EINVAL;
  DeltaStepArgs a{};
  a.q = static_cast<const uint16_t*>(q), a.k = static_cast<const uint16_t*>(k), a.v = static_cast<const uint16_t*>(v);
  a.dt = dt, a.b = b;
  a.q_ld = q_ld, a.k_ld = k_ld, a.v_ld = v_ld, a.dt_ld = dt_ld, a.b_ld = b_ld, a.y_ld = y_ld, a.nseq = nseq;
  a.A = A, a.bias = dt_bias;
  a.f32 = shape->gate_dtype == CONV1D_F32, a.softplus = shape->dt_softplus, a.qk_norm = shape->qk_norm;
  a.H = (int)H, a.P = (int)shape->P, a.G = (int)shape->G, a.N = (int)shape->N;
  a.scale = shape->scale, a.beta_max = shape->beta_max, a.norm_eps = shape->norm_eps;
  a.pool = pool->final;
  a.slots = pool->slots, a.s_slot = pool->s_slot, a.ci = pool->cache_indices;
  a.y = static_cast<uint16_t*>(y);
  return launch_delta_step(a, stream) == hipSuccess ? CONV1D_OK : CONV1D_EHIP;
}

size_t layer_norm_bwd_workspace_bytes(int64_t rows, int64_t d) {
  if (rows < 0 || d < 1 || d > kMaxGroup) return 0;
  return (size_t)align_up(norm_parts(rows, 1, d) * 2 * d * 4);
}

int layer_norm_fwd(int64_t rows, int64_t d, const void* x, int64_t x_ld, const void* residual, int64_t residual_ld,
                   int residual_dtype, float scale, const void* w, const void* bias, int w_dtype, float eps, void* y,
                   int64_t y_ld, void* residual_out, int64_t residual_out_ld, hipStream_t stream) {
  if (layer_check(rows, d, w, bias, w_dtype, eps) != CONV1D_OK) return CONV1D_EINVAL;
  const Operand xy[2] = {{x, x_ld, d}, {y, y_ld, d}};
  for (const Operand& o : xy)
    if (!operand_ok(o, rows) || !aligned(o.p, 2)) return CONV1D_EINVAL;
  Span sr, so;
  if (residual) {
    if (!dtype_ok(residual_dtype)) return CONV1D_EINVAL;
    const int64_t re = dsize(residual_dtype);
    const Operand rr[2] = {{residual, residual_ld, d}, {residual_out, residual_out_ld, d}};
    for (const Operand& o : rr)
      if (!operand_ok(o, rows) || !aligned(o.p, re)) return CONV1D_EINVAL;
    sr = span(residual, rows, d, residual_ld, re);
    so = span(residual_out, rows, d, residual_out_ld, re);
  }
  const int64_t we = dsize(w_dtype);
  const Span reads[3] = {span(x, rows, d, x_ld, 2), span(w, d * we), span(bias, d * we)};
  const Span outs[2] = {span(y, rows, d, y_ld, 2), so};
  const bool same = residual == residual_out && residual_ld == residual_out_ld;
  if (clash(outs, reads) || overlap(outs[0], sr) || (!same && overlap(outs[1], sr))) return CONV1D_EINVAL;
  if (rows == 0) return CONV1D_OK;
  LayerArgs l{};
  NormArgs& a = l.n;
  a.x = static_cast<const uint16_t*>(x), a.r = residual, a.y = static_cast<uint16_t*>(y), a.r_out = residual_out;
  a.x_ld = x_ld, a.r_ld = residual_ld, a.y_ld = y_ld, a.ro_ld = residual_out_ld;
  a.w = w, a.w_f32 = w_dtype == CONV1D_F32, a.r_f32 = residual_dtype == CONV1D_F32;
  a.rows = rows, a.groups = 1, a.group = d, a.eps = eps, a.scale = scale;
  a.parts = norm_fwd_parts(rows, 1, d, kResidualFwdWaves);
  l.bias = bias;
  return launch_layer_fwd(l, stream) == hipSuccess ? CONV1D_OK : CONV1D_EHIP;
}

int layer_norm_bwd(int64_t rows, int64_t d, const void* dy, int64_t dy_ld, const void* dr_out, int64_t dr_out_ld,
                   const void* h, int64_t h_ld, int h_dtype, float scale, const void* w, int w_dtype, float eps,
                   void* dx, int64_t dx_ld, void* dresidual, int64_t dresidual_ld, float* dw, float* dbias, void* ws,
                   size_t ws_bytes, hipStream_t stream) {
  if (layer_check(rows, d, w, nullptr, w_dtype, eps) != CONV1D_OK || !dtype_ok(h_dtype) || !dw) return CONV1D_EINVAL;
  const int64_t he = dsize(h_dtype);
  const Operand ops[3] = {{dy, dy_ld, d}, {dx, dx_ld, d}, {h, h_ld, d}};
  for (int i = 0; i < 3; ++i)
    if (!operand_ok(ops[i], rows) || !aligned(ops[i].p, i == 2 ? he : 2)) return CONV1D_EINVAL;
  const Operand optional[2] = {{dr_out, dr_out_ld, d}, {dresidual, dresidual_ld, d}};
  for (const Operand& o : optional)
    if (o.p && (!operand_ok(o, rows) || !aligned(o.p, he))) return CONV1D_EINVAL;
  if (!aligned(dw, 4) || !aligned(dbias, 4)) return CONV1D_EINVAL;
  const size_t need = layer_norm_bwd_workspace_bytes(rows, d);
  if (need > ws_bytes || (need && !ws)) return CONV1D_EWORKSPACE;
  if (need && !aligned(ws, 16)) return CONV1D_EINVAL;
  const Span sdr = span(dr_out, rows, d, dr_out_ld, he);
  const Span reads[3] = {span(dy, rows, d, dy_ld, 2), span(h, rows, d, h_ld, he), span(w, d * dsize(w_dtype))};
  const Span outs[5] = {span(dresidual, rows, d, dresidual_ld, he), span(dx, rows, d, dx_ld, 2), span(dw, d * 4),
                        span(dbias, d * 4), span(ws, (int64_t)need)};
  const bool same = dr_out == dresidual && dr_out_ld == dresidual_ld;
  if (clash(outs, reads) || (!same && overlap(outs[0], sdr))) return CONV1D_EINVAL;
  for (int i = 1; i < 5; ++i)
    if (overlap(outs[i], sdr)) return CONV1D_EINVAL;
  LayerArgs l{};
  NormArgs& a = l.n;
  a.dy = static_cast<const uint16_t*>(dy), a.r = h, a.dr_in = dr_out, a.dx = static_cast<uint16_t*>(dx), a.r_out = dresidual;
  a.dy_ld = dy_ld, a.r_ld = h_ld, a.dri_ld = dr_out_ld, a.dx_ld = dx_ld, a.ro_ld = dresidual_ld;
  a.w = w, a.w_f32 = w_dtype == CONV1D_F32, a.r_f32 = h_dtype == CONV1D_F32;
  a.rows = rows, a.groups = 1, a.group = d, a.eps = eps, a.scale = scale;
  a.parts = norm_parts(rows, 1, d);
  a.part = static_cast<float*>(ws), a.dw = dw;
  l.db = dbias;
  return launch_layer_bwd(l, stream) == hipSuccess ? CONV1D_OK : CONV1D_EHIP;
}

// A block holds one strip of all pairs in registers: 1024 pieces of 16 bytes, or 8192 from 129 pairs on, where 1024 would
// leave strips below 128 bytes.
int state_copy(const slot_pool* pools, int npools, int64_t n, const int32_t* source, const int32_t* target,
               hipStream_t stream) {
  if (npools < 0 || npools > SLOT_MAX_POOLS || (npools > 0 && !pools) || n < 0 || n > SLOT_MAX_PAIRS) return CONV1D_EINVAL;
  if (n > 0 && (!source || !target || !aligned(source, 4) || !aligned(target, 4))) return CONV1D_EINVAL;
  Span all[SLOT_MAX_POOLS];
  const Span index[2] = {span(source, n * 4), span(target, n * 4)};
  for (int i = 0; i < npools; ++i) {
    const slot_pool& p = pools[i];
    if (p.slots < 0 || p.slot_bytes < 0 || p.s_slot < p.slot_bytes || !mul_ok(p.slots, p.s_slot) ||
        (!p.ptr && p.slots > 0 && p.slot_bytes > 0))
      return CONV1D_EINVAL;
    all[i] = span(p.ptr, p.slots, p.slot_bytes, p.s_slot, 1);
    for (int j = 0; j < i; ++j)
      if (overlap(all[i], all[j])) return CONV1D_EINVAL;
    if (overlap(all[i], index[0]) || overlap(all[i], index[1])) return CONV1D_EINVAL;
  }
  const int threads = n <= 128 ? 256 : 1024, pieces = n <= 128 ? 4 : 8;
  SlotArgs a{};
  a.n = (int)n, a.source = source, a.target = target;
  while (((int64_t)2 << a.strip) * n <= threads * pieces && a.strip < 6) ++a.strip;
  int64_t blocks = 0;
  for (int i = 0; i < npools; ++i) {
    const slot_pool& p = pools[i];
    if (p.slots == 0 || p.slot_bytes == 0) continue;
    const int at = a.pools++;
    a.ptr[at] = static_cast<char*>(p.ptr);
    a.slots[at] = p.slots, a.s_slot[at] = p.s_slot, a.bytes[at] = p.slot_bytes;
    a.first[at] = (uint32_t)blocks;
    blocks += ceil_div(p.slot_bytes, (int64_t)16 << a.strip);
    if (blocks > kMaxBlocks) return CONV1D_EINVAL;
  }
  if (n == 0 || blocks == 0) return CONV1D_OK;
  return launch_slots(a, threads, pieces, (uint32_t)blocks, stream) == hipSuccess ? CONV1D_OK : CONV1D_EHIP;
}

}  // extern "C"
