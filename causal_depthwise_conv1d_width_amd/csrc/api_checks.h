// api_checks.h -- what the entry points of ssm.h and delta.h check on the host before anything is
// enqueued: sizes, alignment and shared bytes of arrays, sequence descriptions.  No device memory is read.
#pragma once

#include <stdint.h>

#include "ssm.h"
#include "ssm_launch.h"

namespace cssm {

constexpr int64_t kMaxElems = (int64_t)1 << 48;  // no extent below overflows 64-bit bytes
constexpr int64_t kMaxBlocks = 0x7fffffff;

inline bool mul_ok(int64_t a, int64_t b) {
  return a >= 0 && b >= 0 && a <= kMaxElems && b <= kMaxElems && (b == 0 || a <= kMaxElems / b);
}
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
inline bool dtype_ok(int d) { return d == CONV1D_BF16 || d == CONV1D_F32; }
inline int64_t dsize(int d) { return d == CONV1D_F32 ? 4 : 2; }

// Byte range of a strided array: rows of `len` bytes, `ld` bytes apart.
struct Span {
  uintptr_t lo = 0, ld = 0, rows = 0, len = 0;
  uintptr_t hi() const { return rows ? lo + (rows - 1) * ld + len : lo; }
};
inline Span span(const void* p, int64_t rows, int64_t len, int64_t ld, int64_t esz) {
  Span s;
  if (!p || rows <= 0 || len <= 0) return s;
  s.lo = reinterpret_cast<uintptr_t>(p);
  s.ld = (uintptr_t)(ld * esz);
  s.rows = (uintptr_t)rows;
  s.len = (uintptr_t)(len * esz);
  return s;
}
inline Span span(const void* p, int64_t bytes) { return span(p, 1, bytes, bytes, 1); }
// Whether two arrays share a byte.  Column ranges of the same wider rows (equal row strides) do not,
// though their address ranges interleave.
inline bool overlap(const Span& a, const Span& b) {
  if (!a.rows || !b.rows || a.lo >= b.hi() || b.lo >= a.hi()) return false;
  if (a.rows > 1 && b.rows > 1 && a.ld == b.ld) {
    const uintptr_t ld = a.ld;
    const uintptr_t off = a.lo >= b.lo ? (a.lo - b.lo) % ld : (ld - (b.lo - a.lo) % ld) % ld;  // a's start in b's rows
    return !(off >= b.len && off + a.len <= ld);
  }
  return true;
}
template <int NO, int NI>
inline bool clash(const Span (&outs)[NO], const Span (&ins)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (const Span& in : ins)
      if (overlap(outs[i], in)) return true;
    for (int j = i + 1; j < NO; ++j)
      if (overlap(outs[i], outs[j])) return true;
  }
  return false;
}

inline int64_t align_up(int64_t v) { return (v + 255) / 256 * 256; }

inline int check_seq(const conv1d_seq* q, int64_t rows, int64_t* nseq) {
  if (!q || q->seq_idx) return CONV1D_EINVAL;
  if (q->cu_seqlens) {
    if (q->nseq < 0) return CONV1D_EINVAL;
    *nseq = q->nseq;
    return CONV1D_OK;
  }
  if (q->seqlen < 1 || rows % q->seqlen != 0) return CONV1D_EINVAL;
  *nseq = rows / q->seqlen;
  return CONV1D_OK;
}

// States argument (hpn values a state) against nseq; fills the kernel's fields and the byte ranges.
inline int check_states(int64_t hpn, const ssm_states* st, int64_t nseq, ScanArgs* a, Span* init, Span* fin, Span* ci,
                 Span* hi) {
  if (!st || (!st->initial && !st->final)) {
    if (st && st->cache_indices) return CONV1D_EINVAL;
    return CONV1D_OK;
  }
  if (st->slots < 1 || st->s_slot < hpn || !mul_ok(st->slots, st->s_slot)) return CONV1D_EINVAL;
  if (!st->cache_indices && st->slots < nseq) return CONV1D_EINVAL;
  *init = span(st->initial, st->slots, hpn, st->s_slot, 4);
  *fin = span(st->final, st->slots, hpn, st->s_slot, 4);
  if (st->initial != st->final && overlap(*init, *fin)) return CONV1D_EINVAL;
  *ci = span(st->cache_indices, nseq * 4);
  *hi = span(st->has_initial_state, nseq);
  a->init = st->initial;
  a->fin = st->final;
  a->slots = st->slots;
  a->s_slot = st->s_slot;
  a->ci = st->cache_indices;
  a->has_init = st->has_initial_state;
  return CONV1D_OK;
}

struct Operand {
  const void* p;
  int64_t ld, len;
};
inline bool operand_ok(const Operand& o, int64_t rows) {
  return (rows == 0 || o.p) && o.ld >= o.len && mul_ok(rows, o.ld);
}
// The scan addresses the 64 rows of a chunk by 32-bit byte offsets from the first.
inline bool scan_operand_ok(const Operand& o, int64_t rows) { return operand_ok(o, rows) && o.ld <= SSM_MAX_ROW_STRIDE; }

}  // namespace cssm
