// ssm_api.cpp -- the C ABI of include/ssm.h: host-side validation, workspace layout and launches.
// Every precondition the host can see is checked before anything is enqueued; nothing here reads
// device memory, allocates or synchronizes.
#include "ssm.h"

#include <stdint.h>

#include "api_checks.h"

using namespace cssm;

namespace {

// log2 of a piece's rows, 0 for whole sequences.  A block walks a piece chunk by chunk for kUnits units.
// Sequences are cut into pieces where whole ones give too few blocks, or, with offsets (the host does not
// know the lengths), where one could be long against the rest; the cost is a first walk for the pieces' states
// and a join.
//
// Forward (64 heads of 64 columns, N = 128), `want` blocks: 4 sequences of 4096 rows 194 us with 256, 324 with
// 128, 212 with 512, 437 whole; 2048 rows of one sequence 60 us with 256, 69 with 128, 60 with 512, 218 whole; 64 mixed
// prompts 458 us with pieces for 512 blocks, 493 for 256, 451 whole (but only because none is long).
//
// Backward: the walk is bound by its stores, both directions are one launch, and few blocks reach that bound.
// 4 sequences of 4096 rows (64 walks a direction) 870 us whole, 967 for 128, 981 for 256; 2 sequences of 8192 1088
// whole, 971 for 128; one of 16384 1500 whole, 1056 for 64, 978 for 128, 995 for 256.  Mixed sequences, means over
// six draws: nine in 2777 rows (24 heads) 140 us with pieces of at least 256 rows, 154 with 512, 160 with 1024; six in
// 8192 rows 292, 292 and 324 us.
struct Cut {
  int64_t whole, want;  // blocks that make equal sequences stay whole; blocks wanted of pieces
  int least;            // log2 of the fewest rows of a piece
};
constexpr Cut kCutFwd{256, 256, 7}, kCutBwd{64, 128, 8};
int piece_log2(const ssm_shape* s, int64_t rows, int64_t nseq, bool batch_rows, const Cut& cut) {
  const int64_t sets = s->G * ceil_div(s->H / s->G * ceil_div(s->P, kPTile), kUnits);
  if (nseq <= 0 || (batch_rows && nseq * sets >= cut.whole)) return 0;
  const int64_t want = nseq * sets >= cut.want ? 2 * cut.want : cut.want;
  int seg = cut.least;
  while (((int64_t)1 << seg) * want < rows * sets) ++seg;
  return ((int64_t)1 << seg) < (batch_rows ? rows / nseq : rows - nseq + 1) ? seg : 0;
}

struct FwdPlan {
  int seg;
  int64_t n_slots, piece, decay, bytes;  // byte offsets into the workspace
};
FwdPlan plan_fwd(const ssm_shape* s, int64_t rows, int64_t nseq, bool batch_rows, const Cut& cut = kCutFwd) {
  FwdPlan p{};
  p.seg = piece_log2(s, rows, nseq, batch_rows, cut);
  if (!p.seg) return p;
  p.n_slots = batch_rows ? nseq * (ceil_div(rows / nseq, (int64_t)1 << p.seg) - 1) : ceil_div(rows, (int64_t)1 << p.seg);
  const int64_t items = p.n_slots + nseq, hp = s->H * ceil_div(s->P, kPTile);
  p.decay = align_up(items * hp * 64 * state_tile(s->N) * 4);
  p.bytes = p.decay + align_up(items * s->H * 4);
  return p;
}

struct BwdPlan {
  FwdPlan f;
  int64_t ids, n_chunk_slots, piece_t, piece_t_decay, cs, ct, head, bc, bytes;
  int hsplit;
};
// Blocks of the chunk kernel: one a chunk and group; heads of a group go to several blocks (FP32
// parts of dB and dC, added by another kernel) only where that many blocks would leave CUs idle: up to one a CU, as more
// parts cost more than they hide.  The backward with 256, 512 and 1024 blocks: 2777 rows, 24 heads in 2 groups, 133, 140
// and 151 us; 1024 rows, 64 heads in 4 groups, 124, 133 and 149; 4096 rows, 64 heads in one group, 343, 339 and 333.
constexpr int64_t kWantChunkBlocks = 256;
BwdPlan plan_bwd(const ssm_shape* s, int64_t rows, int64_t nseq, bool batch_rows) {
  BwdPlan p{};
  p.f = plan_fwd(s, rows, nseq, batch_rows, kCutBwd);
  p.n_chunk_slots = ceil_div(rows, kChunk);
  p.ids = p.n_chunk_slots + nseq;
  const int64_t hp = s->H * ceil_div(s->P, kPTile), tile = 64 * state_tile(s->N), chunks = ceil_div(rows, kChunk);
  int64_t split = ceil_div(kWantChunkBlocks, chunks * s->G > 0 ? chunks * s->G : 1);
  const int64_t hg = s->H / s->G;
  if (split > hg) split = hg;
  split = ceil_div(hg, ceil_div(hg, split));  // no empty parts
  p.hsplit = (int)split;
  int64_t at = align_up(p.f.bytes);
  p.piece_t = at;
  if (p.f.seg) at += align_up((p.f.n_slots + nseq) * hp * tile * 4);
  p.piece_t_decay = at;
  if (p.f.seg) at += align_up((p.f.n_slots + nseq) * s->H * 4);
  p.cs = at;
  at += align_up(p.ids * hp * tile * 4);
  p.ct = at;
  at += align_up(p.ids * hp * tile * 4);
  p.head = at;
  at += align_up(p.ids * s->H * 3 * 4);
  p.bc = at;
  if (split > 1) at += align_up(2 * split * rows * s->G * s->N * 4);
  p.bytes = at;
  return p;
}

bool shape_ok(const ssm_shape* s) {
  return s && s->H >= 1 && s->P >= 1 && s->G >= 1 && s->N >= 1 && s->N <= kMaxState && s->H % s->G == 0 &&
         s->H <= (1 << 20) && s->P <= (1 << 20) && dtype_ok(s->dt_dtype) && (s->dt_softplus == 0 || s->dt_softplus == 1);
}

void fill(ScanArgs* a, const ssm_shape* s, int64_t rows, const void* x, int64_t x_ld, const void* dt, int64_t dt_ld,
          const float* A, const void* B, int64_t B_ld, const void* C, int64_t C_ld, const float* D,
          const float* dt_bias, const conv1d_seq* seq, int64_t nseq, const FwdPlan& p, char* ws) {
  a->x = static_cast<const uint16_t*>(x);
  a->B = static_cast<const uint16_t*>(B);
  a->C = static_cast<const uint16_t*>(C);
  a->dt = dt;
  a->x_ld = x_ld, a->B_ld = B_ld, a->C_ld = C_ld, a->dt_ld = dt_ld;
  a->A = A, a->D = D, a->bias = dt_bias;
  a->dt_f32 = s->dt_dtype == CONV1D_F32;
  a->softplus = s->dt_softplus;
  a->H = (int)s->H, a->P = (int)s->P, a->G = (int)s->G, a->N = (int)s->N;
  a->ptiles = (int)ceil_div(s->P, kPTile);
  a->q = Seqs{seq->cu_seqlens, nseq, seq->cu_seqlens ? 1 : seq->seqlen, rows};
  a->seg = p.seg;
  a->n_slots = p.n_slots;
  if (p.seg) {
    a->piece = reinterpret_cast<float*>(ws + p.piece);
    a->piece_decay = reinterpret_cast<float*>(ws + p.decay);
  }
}

bool scan_sizes_ok(const ssm_shape* s, int64_t rows, int64_t nseq) {
  const int64_t hp = s->H * ceil_div(s->P, kPTile);
  // workspace extents and launches of every kernel, bounded by one block a row and sequence
  return rows >= 0 && nseq >= 0 && mul_ok(rows, s->H * s->P) && mul_ok(rows, s->G * s->N) &&
         mul_ok(ceil_div(rows, kChunk) + nseq + 1, hp * 64 * kMaxState) && mul_ok(rows, 64 * s->G * s->N);
}

bool vec_ok(const ssm_shape* s) { return s->P % 8 == 0 && s->N % 8 == 0; }

int norm_check(int64_t rows, int64_t d, int64_t group, const void* w, int w_dtype, float eps) {
  if (rows < 0 || d < 1 || group < 1 || group > kMaxGroup || d % group != 0 || !w || !dtype_ok(w_dtype)) return CONV1D_EINVAL;
  if (!(eps >= 0.f) || !mul_ok(rows, d) || !aligned(w, dsize(w_dtype))) return CONV1D_EINVAL;
  if (rows > 0 && (d / group) > kMaxBlocks / 4096) return CONV1D_EINVAL;
  return CONV1D_OK;
}

}  // namespace

extern "C" {

size_t ssm_scan_fwd_workspace_bytes(const ssm_shape* shape, int64_t rows, int64_t nseq) {
  if (!shape_ok(shape) || rows <= 0 || nseq <= 0 || !scan_sizes_ok(shape, rows, nseq)) return 0;
  const int64_t a = plan_fwd(shape, rows, nseq, false).bytes;
  const int64_t b = rows % nseq == 0 ? plan_fwd(shape, rows, nseq, true).bytes : 0;
  return (size_t)(a > b ? a : b);  // offsets or batch rows
}

size_t ssm_scan_bwd_workspace_bytes(const ssm_shape* shape, int64_t rows, int64_t nseq) {
  if (!shape_ok(shape) || rows < 0 || nseq <= 0 || !scan_sizes_ok(shape, rows, nseq)) return 0;
  const int64_t a = plan_bwd(shape, rows, nseq, false).bytes;
  const int64_t b = rows % nseq == 0 ? plan_bwd(shape, rows, nseq, true).bytes : 0;
  return (size_t)(a > b ? a : b);  // offsets or batch rows
}

size_t norm_bwd_workspace_bytes(int64_t rows, int64_t d, int64_t group) {
  if (rows < 0 || d < 1 || group < 1 || group > kMaxGroup || d % group != 0 || !mul_ok(4096, d)) return 0;
  return (size_t)align_up(norm_parts(rows, d / group, group) * d * 4);
}

int ssm_scan_fwd(const ssm_shape* shape, int64_t rows, const void* x, int64_t x_ld, const void* dt, int64_t dt_ld,
                 const float* A, const void* B, int64_t B_ld, const void* C, int64_t C_ld, const float* D,
                 const float* dt_bias, const conv1d_seq* seq, const ssm_states* states, void* y, int64_t y_ld,
                 void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!shape_ok(shape) || rows < 0 || !A) return CONV1D_EINVAL;
  int64_t nseq = 0;
  if (check_seq(seq, rows, &nseq) != CONV1D_OK || !scan_sizes_ok(shape, rows, nseq)) return CONV1D_EINVAL;
  const int64_t H = shape->H, hp = H * shape->P, gn = shape->G * shape->N, dte = dsize(shape->dt_dtype);
  const Operand ops[5] = {{x, x_ld, hp}, {dt, dt_ld, H}, {B, B_ld, gn}, {C, C_ld, gn}, {y, y_ld, hp}};
  for (const Operand& o : ops)
    if (!scan_operand_ok(o, rows)) return CONV1D_EINVAL;
  if (!aligned(x, 2) || !aligned(B, 2) || !aligned(C, 2) || !aligned(y, 2) || !aligned(dt, dte)) return CONV1D_EINVAL;
  ScanArgs a{};
  Span si, sf, sci, shi;
  if (check_states(shape->H * shape->P * shape->N, states, nseq, &a, &si, &sf, &sci, &shi) != CONV1D_OK) return CONV1D_EINVAL;
  const FwdPlan p = plan_fwd(shape, rows, nseq, !seq->cu_seqlens);
  if ((size_t)p.bytes > ws_bytes || (p.bytes && !ws)) return CONV1D_EWORKSPACE;
  if (p.bytes && !aligned(ws, 16)) return CONV1D_EINVAL;
  const Span reads[10] = {span(x, rows, hp, x_ld, 2), span(dt, rows, H, dt_ld, dte), span(B, rows, gn, B_ld, 2),
                          span(C, rows, gn, C_ld, 2), span(A, H * 4), span(D, H * 4), span(dt_bias, H * 4), sci, shi,
                          span(seq->cu_seqlens, (nseq + 1) * 4)};
  const Span outs[3] = {span(y, rows, hp, y_ld, 2), sf, span(ws, p.bytes)};
  if (clash(outs, reads) || overlap(outs[0], si) || overlap(outs[2], si)) return CONV1D_EINVAL;
  // no rows: an in-place pool stays as it is, so only separate final states are left to write
  if (nseq == 0 || (rows == 0 && (!a.fin || a.fin == a.init))) return CONV1D_OK;
  if ((p.n_slots + nseq) * H * ceil_div(shape->P, kPTile) > kMaxBlocks / 16) return CONV1D_EINVAL;
  fill(&a, shape, rows, x, x_ld, dt, dt_ld, A, B, B_ld, C, C_ld, D, dt_bias, seq, nseq, p, static_cast<char*>(ws));
  a.y = static_cast<uint16_t*>(y);
  a.y_ld = y_ld;
  return launch_scan_fwd(a, vec_ok(shape), stream) == hipSuccess ? CONV1D_OK : CONV1D_EHIP;
}

int ssm_scan_bwd(const ssm_shape* shape, int64_t rows, const void* dy, int64_t dy_ld, const void* x, int64_t x_ld,
                 const void* dt, int64_t dt_ld, const float* A, const void* B, int64_t B_ld, const void* C,
                 int64_t C_ld, const float* D, const float* dt_bias, const conv1d_seq* seq,
                 const float* initial_state, const float* dfinal_state, void* dx, int64_t dx_ld, void* ddt,
                 int64_t ddt_ld, float* dA, void* dB, int64_t dB_ld, void* dC, int64_t dC_ld, float* dD,
                 float* ddt_bias, float* dinitial_state, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!shape_ok(shape) || rows < 0 || !A || !dA) return CONV1D_EINVAL;
  int64_t nseq = 0;
  if (check_seq(seq, rows, &nseq) != CONV1D_OK || !scan_sizes_ok(shape, rows, nseq)) return CONV1D_EINVAL;
  const int64_t H = shape->H, hp = H * shape->P, gn = shape->G * shape->N, dte = dsize(shape->dt_dtype);
  const int64_t states = nseq * hp * shape->N * 4;
  if (!mul_ok(nseq, hp * shape->N)) return CONV1D_EINVAL;
  const Operand ops[9] = {{dy, dy_ld, hp}, {x, x_ld, hp}, {dt, dt_ld, H}, {B, B_ld, gn}, {C, C_ld, gn},
                          {dx, dx_ld, hp}, {ddt, ddt_ld, H}, {dB, dB_ld, gn}, {dC, dC_ld, gn}};
  for (const Operand& o : ops)
    if (!scan_operand_ok(o, rows) || !aligned(o.p, o.p == dt || o.p == ddt ? dte : 2)) return CONV1D_EINVAL;
  const BwdPlan p = nseq > 0 ? plan_bwd(shape, rows, nseq, !seq->cu_seqlens) : BwdPlan{};
  if ((size_t)p.bytes > ws_bytes || (p.bytes && !ws)) return CONV1D_EWORKSPACE;
  if (p.bytes && !aligned(ws, 16)) return CONV1D_EINVAL;
  const Span reads[11] = {span(dy, rows, hp, dy_ld, 2), span(x, rows, hp, x_ld, 2), span(dt, rows, H, dt_ld, dte),
                          span(B, rows, gn, B_ld, 2), span(C, rows, gn, C_ld, 2), span(A, H * 4), span(D, H * 4),
                          span(dt_bias, H * 4), span(initial_state, states), span(dfinal_state, states),
                          span(seq->cu_seqlens, (nseq + 1) * 4)};
  const Span outs[9] = {span(dx, rows, hp, dx_ld, 2), span(ddt, rows, H, ddt_ld, dte), span(dB, rows, gn, dB_ld, 2),
                        span(dC, rows, gn, dC_ld, 2), span(dA, H * 4), span(dD, H * 4), span(ddt_bias, H * 4),
                        span(dinitial_state, states), span(ws, p.bytes)};
  if (clash(outs, reads)) return CONV1D_EINVAL;
  ScanBwdArgs b{};
  b.dA = dA, b.dD = dD, b.dbias = ddt_bias;
  b.s.H = (int)H;
  if (nseq > 0) {
    if ((p.f.n_slots + nseq) * H * ceil_div(shape->P, kPTile) > kMaxBlocks / 16 ||
        p.ids * shape->G * p.hsplit > kMaxBlocks || ceil_div(rows * gn, 256) > kMaxBlocks)
      return CONV1D_EINVAL;
    char* w = static_cast<char*>(ws);
    fill(&b.s, shape, rows, x, x_ld, dt, dt_ld, A, B, B_ld, C, C_ld, D, dt_bias, seq, nseq, p.f, w);
    b.s.init = initial_state;
    b.s.slots = nseq;
    b.s.s_slot = hp * shape->N;
    b.dy = static_cast<const uint16_t*>(dy), b.dy_ld = dy_ld;
    b.dfin = dfinal_state, b.dinit = dinitial_state;
    b.dx = static_cast<uint16_t*>(dx), b.dx_ld = dx_ld;
    b.ddt = ddt, b.ddt_ld = ddt_ld;
    b.dB = static_cast<uint16_t*>(dB), b.dB_ld = dB_ld;
    b.dC = static_cast<uint16_t*>(dC), b.dC_ld = dC_ld;
    b.piece_t = reinterpret_cast<float*>(w + p.piece_t);
    b.piece_t_decay = reinterpret_cast<float*>(w + p.piece_t_decay);
    b.cs = reinterpret_cast<float*>(w + p.cs);
    b.ct = reinterpret_cast<float*>(w + p.ct);
    b.n_chunk_slots = p.n_chunk_slots;
    b.head_part = reinterpret_cast<float*>(w + p.head);
    b.bc_part = reinterpret_cast<float*>(w + p.bc);
    b.hsplit = p.hsplit;
  }
  return launch_scan_bwd(b, vec_ok(shape), stream) == hipSuccess ? CONV1D_OK : CONV1D_EHIP;
}

int ssm_state_update(const ssm_shape* shape, int64_t nseq, const void* x, int64_t x_ld, const void* dt, int64_t dt_ld,
                     const float* A, const void* B, int64_t B_ld, const void* C, int64_t C_ld, const float* D,
                     const float* dt_bias, const ssm_states* pool, void* y, int64_t y_ld, hipStream_t stream) {
  if (!shape_ok(shape) || nseq < 0 || !A || !pool || !pool->initial || pool->initial != pool->final) return CONV1D_EINVAL;
  if (!pool->cache_indices || !scan_sizes_ok(shape, nseq, nseq)) return CONV1D_EINVAL;
  const int64_t H = shape->H, hp = H * shape->P, gn = shape->G * shape->N, dte = dsize(shape->dt_dtype);
  const Operand ops[5] = {{x, x_ld, hp}, {dt, dt_ld, H}, {B, B_ld, gn}, {C, C_ld, gn}, {y, y_ld, hp}};
  for (const Operand& o : ops)
    if (!operand_ok(o, nseq) || !aligned(o.p, o.p == dt ? dte : 2)) return CONV1D_EINVAL;
  ScanArgs s{};
  Span si, sf, sci, shi;
  if (check_states(hp * shape->N, pool, nseq, &s, &si, &sf, &sci, &shi) != CONV1D_OK) return CONV1D_EINVAL;
  const Span reads[8] = {span(x, nseq, hp, x_ld, 2), span(dt, nseq, H, dt_ld, dte), span(B, nseq, gn, B_ld, 2),
                         span(C, nseq, gn, C_ld, 2), span(A, H * 4), span(D, H * 4), span(dt_bias, H * 4), sci};
  const Span outs[2] = {span(y, nseq, hp, y_ld, 2), sf};
  if (clash(outs, reads)) return CONV1D_EINVAL;
  if (nseq == 0) return CONV1D_OK;
  if (!mul_ok(nseq, H * shape->P) || nseq * H * ceil_div(shape->P, 8) > kMaxBlocks) return CONV1D_EINVAL;
  StepArgs a{};
  a.x = static_cast<const uint16_t*>(x), a.B = static_cast<const uint16_t*>(B), a.C = static_cast<const uint16_t*>(C);
  a.dt = dt;
  a.x_ld = x_ld, a.B_ld = B_ld, a.C_ld = C_ld, a.dt_ld = dt_ld, a.y_ld = y_ld, a.nseq = nseq;
  a.A = A, a.D = D, a.bias = dt_bias;
  a.dt_f32 = shape->dt_dtype == CONV1D_F32, a.softplus = shape->dt_softplus;
  a.H = (int)H, a.P = (int)shape->P, a.G = (int)shape->G, a.N = (int)shape->N;
  a.pool = pool->final;
  a.slots = pool->slots, a.s_slot = pool->s_slot, a.ci = pool->cache_indices;
  a.y = static_cast<uint16_t*>(y);
  return launch_step(a, stream) == hipSuccess ? CONV1D_OK : CONV1D_EHIP;
}

int gated_norm_fwd(int64_t rows, int64_t d, int64_t group, const void* x, int64_t x_ld, const void* z, int64_t z_ld,
                   const void* w, int w_dtype, int norm_before_gate, float eps, void* y, int64_t y_ld,
                   hipStream_t stream) {
  if (norm_check(rows, d, group, w, w_dtype, eps) != CONV1D_OK) return CONV1D_EINVAL;
  const Operand ops[3] = {{x, x_ld, d}, {z, z_ld, d}, {y, y_ld, d}};
  for (const Operand& o : ops)
    if (!operand_ok(o, rows) || !aligned(o.p, 2)) return CONV1D_EINVAL;
  const Span reads[3] = {span(x, rows, d, x_ld, 2), span(z, rows, d, z_ld, 2), span(w, d * dsize(w_dtype))};
  const Span outs[1] = {span(y, rows, d, y_ld, 2)};
  if (clash(outs, reads)) return CONV1D_EINVAL;
  if (rows == 0) return CONV1D_OK;
  NormArgs a{};
  a.x = static_cast<const uint16_t*>(x), a.z = static_cast<const uint16_t*>(z), a.y = static_cast<uint16_t*>(y);
  a.x_ld = x_ld, a.z_ld = z_ld, a.y_ld = y_ld;
  a.w = w, a.w_f32 = w_dtype == CONV1D_F32, a.norm_first = norm_before_gate != 0;
  a.rows = rows, a.groups = d / group, a.group = group, a.eps = eps;
  a.parts = norm_fwd_parts(rows, a.groups, group, kGatedFwdWaves);
  return launch_gated_fwd(a, stream) == hipSuccess ? CONV1D_OK : CONV1D_EHIP;
}

int gated_norm_bwd(int64_t rows, int64_t d, int64_t group, const void* dy, int64_t dy_ld, const void* x, int64_t x_ld,
                   const void* z, int64_t z_ld, const void* w, int w_dtype, int norm_before_gate, float eps, void* dx,
                   int64_t dx_ld, void* dz, int64_t dz_ld, float* dw, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (norm_check(rows, d, group, w, w_dtype, eps) != CONV1D_OK || !dw) return CONV1D_EINVAL;
  const Operand ops[5] = {{dy, dy_ld, d}, {x, x_ld, d}, {z, z_ld, d}, {dx, dx_ld, d}, {dz, dz_ld, d}};
  for (const Operand& o : ops)
    if (!operand_ok(o, rows) || !aligned(o.p, 2)) return CONV1D_EINVAL;
  const size_t need = norm_bwd_workspace_bytes(rows, d, group);
  if (need > ws_bytes || (need && !ws)) return CONV1D_EWORKSPACE;
  if (need && !aligned(ws, 16)) return CONV1D_EINVAL;
  const Span reads[4] = {span(dy, rows, d, dy_ld, 2), span(x, rows, d, x_ld, 2), span(z, rows, d, z_ld, 2),
                         span(w, d * dsize(w_dtype))};
  const Span outs[4] = {span(dx, rows, d, dx_ld, 2), span(dz, rows, d, dz_ld, 2), span(dw, d * 4), span(ws, (int64_t)need)};
  if (clash(outs, reads)) return CONV1D_EINVAL;
  NormArgs a{};
  a.x = static_cast<const uint16_t*>(x), a.z = static_cast<const uint16_t*>(z), a.dy = static_cast<const uint16_t*>(dy);
  a.dx = static_cast<uint16_t*>(dx), a.dz = static_cast<uint16_t*>(dz);
  a.x_ld = x_ld, a.z_ld = z_ld, a.dy_ld = dy_ld, a.dx_ld = dx_ld, a.dz_ld = dz_ld;
  a.w = w, a.w_f32 = w_dtype == CONV1D_F32, a.norm_first = norm_before_gate != 0;
  a.rows = rows, a.groups = d / group, a.group = group, a.eps = eps;
  a.parts = norm_parts(rows, a.groups, group);
  a.part = static_cast<float*>(ws), a.dw = dw;
  return launch_gated_bwd(a, stream) == hipSuccess ? CONV1D_OK : CONV1D_EHIP;
}

int residual_norm_fwd(int64_t rows, int64_t d, const void* x, int64_t x_ld, const void* residual, int64_t residual_ld,
                      int residual_dtype, float scale, const void* w, int w_dtype, float eps, void* y, int64_t y_ld,
                      void* residual_out, int64_t residual_out_ld, hipStream_t stream) {
  if (norm_check(rows, d, d, w, w_dtype, eps) != CONV1D_OK || !dtype_ok(residual_dtype)) return CONV1D_EINVAL;
  const int64_t re = dsize(residual_dtype);
  const Operand ops[4] = {{x, x_ld, d}, {residual, residual_ld, d}, {y, y_ld, d}, {residual_out, residual_out_ld, d}};
  for (int i = 0; i < 4; ++i)
    if (!operand_ok(ops[i], rows) || !aligned(ops[i].p, i % 2 ? re : 2)) return CONV1D_EINVAL;
  const Span sr = span(residual, rows, d, residual_ld, re);
  const Span reads[2] = {span(x, rows, d, x_ld, 2), span(w, d * dsize(w_dtype))};
  const Span outs[2] = {span(y, rows, d, y_ld, 2), span(residual_out, rows, d, residual_out_ld, re)};
  const bool same = residual == residual_out && residual_ld == residual_out_ld;
  if (clash(outs, reads) || overlap(outs[0], sr) || (!same && overlap(outs[1], sr))) return CONV1D_EINVAL;
  if (rows == 0) return CONV1D_OK;
  NormArgs a{};
  a.x = static_cast<const uint16_t*>(x), a.r = residual, a.y = static_cast<uint16_t*>(y), a.r_out = residual_out;
  a.x_ld = x_ld, a.r_ld = residual_ld, a.y_ld = y_ld, a.ro_ld = residual_out_ld;
  a.w = w, a.w_f32 = w_dtype == CONV1D_F32, a.r_f32 = residual_dtype == CONV1D_F32;
  a.rows = rows, a.groups = 1, a.group = d, a.eps = eps, a.scale = scale;
  a.parts = norm_fwd_parts(rows, 1, d, kResidualFwdWaves);
  return launch_residual_fwd(a, stream) == hipSuccess ? CONV1D_OK : CONV1D_EHIP;
}

int residual_norm_bwd(int64_t rows, int64_t d, const void* dy, int64_t dy_ld, const void* dr_out, int64_t dr_out_ld,
                      const void* residual_out, int64_t residual_out_ld, int residual_dtype, float scale,
                      const void* w, int w_dtype, float eps, void* dx, int64_t dx_ld, void* dresidual,
                      int64_t dresidual_ld, float* dw, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (norm_check(rows, d, d, w, w_dtype, eps) != CONV1D_OK || !dtype_ok(residual_dtype) || !dw) return CONV1D_EINVAL;
  const int64_t re = dsize(residual_dtype);
  const Operand ops[4] = {{dy, dy_ld, d}, {residual_out, residual_out_ld, d}, {dx, dx_ld, d}, {dresidual, dresidual_ld, d}};
  for (int i = 0; i < 4; ++i)
    if (!operand_ok(ops[i], rows) || !aligned(ops[i].p, i % 2 ? re : 2)) return CONV1D_EINVAL;
  if (dr_out && (dr_out_ld < d || !mul_ok(rows, dr_out_ld) || !aligned(dr_out, re))) return CONV1D_EINVAL;
  const size_t need = norm_bwd_workspace_bytes(rows, d, d);
  if (need > ws_bytes || (need && !ws)) return CONV1D_EWORKSPACE;
  if (need && !aligned(ws, 16)) return CONV1D_EINVAL;
  const Span sdr = span(dr_out, rows, d, dr_out_ld, re);
  const Span reads[3] = {span(dy, rows, d, dy_ld, 2), span(residual_out, rows, d, residual_out_ld, re),
                         span(w, d * dsize(w_dtype))};
  const Span outs[4] = {span(dresidual, rows, d, dresidual_ld, re), span(dx, rows, d, dx_ld, 2), span(dw, d * 4),
                        span(ws, (int64_t)need)};
  const bool same = dr_out == dresidual && dr_out_ld == dresidual_ld;
  if (clash(outs, reads) || (!same && overlap(outs[0], sdr))) return CONV1D_EINVAL;
  for (int i = 1; i < 4; ++i)
    if (overlap(outs[i], sdr)) return CONV1D_EINVAL;
  NormArgs a{};
  a.dy = static_cast<const uint16_t*>(dy), a.r = residual_out, a.dr_in = dr_out, a.dx = static_cast<uint16_t*>(dx);
  a.r_out = dresidual;
  a.dy_ld = dy_ld, a.r_ld = residual_out_ld, a.dri_ld = dr_out_ld, a.dx_ld = dx_ld, a.ro_ld = dresidual_ld;
  a.w = w, a.w_f32 = w_dtype == CONV1D_F32, a.r_f32 = residual_dtype == CONV1D_F32;
  a.rows = rows, a.groups = 1, a.group = d, a.eps = eps, a.scale = scale;
  a.parts = norm_parts(rows, 1, d);
  a.part = static_cast<float*>(ws), a.dw = dw;
  return launch_residual_bwd(a, stream) == hipSuccess ? CONV1D_OK : CONV1D_EHIP;
}

}  // extern "C"
