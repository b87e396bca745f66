// delta_scan.hip -- forward gated delta rule over packed rows: the walk of the states.
//
// A block walks one sequence for 64 (or 32) columns of one head, a chunk of 64 rows at a time (delta_chunk.hip: L, r, T, P):
//   R = r (V - e^L K S^T),   U = T R,   Y = scale e^L Q S^T + P U,   S' = e^{L_Q} S + U^T (e^{L_Q - L} K)
// Each of its waves owns 16 columns p of V, U, Y and S, which depend on no other column: nothing passes between waves.
// The state's accumulators (registers n, lanes p) are, unmoved, the operand that K S^T and Q S^T contract over n, and R's
// and U's the ones that T, P and K contract over rows.  Shared memory holds K, Q, V and the chunk's record for all waves;
// the next chunk's are loaded over the current one's products.
// FP32 operands enter as two fp16 parts (delta_device.h), T R with three products, so that states keep 22 bits of their
// column's largest value; y takes the first part of S alone (2^-12 of a term).  P U is of bf16 parts, two of each: the
// scores and new values of a chunk's rows may lie far apart, and each row of y is to keep its own precision.
#include "delta_device.h"

namespace cssm {

// What shared memory holds of a chunk for the waves that walk the state, 16 W columns: the chunk's and the next one's
template <int NT, int W>
struct ChainShared {
  __align__(16) uint16_t k[key_tile(NT) / 2];
  __align__(16) char t[kRecT];
  Factors fac;
  __align__(16) uint16_t v[64 * kLd<16 * W, 16>];
};
// and for the waves that make y, with what the others hand them: S's first parts, U, the columns' scales and first rows that
// are not finite
template <int NT, int W>
struct OutputShared {
  __align__(16) uint16_t q[key_tile(NT) / 2];
  __align__(16) char p[kTriBlocks * 2 * kTriPart];
  f16x8 s[W][NT / 32][64];
  f32x4 u[W][4][64];
  __align__(16) float down[W][16];
  __align__(16) int bad[W][16];
};

// Waves 0 to W - 1 walk the state and make U, a chain of products that each wait for the last; the other W make y of what the
// first ones leave in shared memory, a half chunk behind, and bring the next chunks' tiles there.  Two barriers a chunk:
// after S's parts (1) and after U (2) are there.  Before (1) of a chunk its K, T, V and factors and Q are in place; the
// next chunk's K, T, V and factors come between (1) and (2), with this chunk's P, the next Q after (2).
// What bounds it: R needs S, U needs R and the next S needs U, and y's products share the SIMDs: a chunk takes 3.1 us at 128 x 128
// columns (2.7 with 32 columns a block), in which a SIMD's matrix instructions are busy for 0.8.  Without y's products or without
// the walk's it would be a seventh less, without either (copies, barriers, scalings) a third; two chunks' tiles on their way instead
// of one change nothing.  4 x 4096 rows of 32 heads of 128 x 128: 322 us with the chunk kernel's 125; with all of it in
// four waves, which waited for y's products and for the tiles between the chain's, 454.
template <int NT, int W, bool VEC>
__global__ __launch_bounds__(128 * W) void delta_scan_fwd_kernel(DeltaArgs d) {
  constexpr int NB = NT / 16, TH = 64 * W, COLS = 16 * W;
  __shared__ ChainShared<NT, W> chain[2];
  __shared__ OutputShared<NT, W> outp;
  const ScanArgs& a = d.s;  // its ptiles are of COLS columns
  const Units<1> us(a, blockIdx.x);
  if (!us.ok) return;
  const int tile = us.group * us.units + us.first, h = (uint32_t)tile / (uint32_t)a.ptiles, p_first = (tile - h * a.ptiles) * COLS;
  const int pn = a.P - p_first < COLS ? a.P - p_first : COLS;
  const uint32_t col = (uint32_t)h * a.P + p_first;
  const int w = wave_id() & (W - 1);
  const bool walks = wave_id() < W;
  Piece pc;
  pc.seq = walk_sequence(d, us.item);
  seq_bounds(a.q, pc.seq, pc.s, pc.e);
  int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15;
  const int64_t state_at = ((int64_t)h * a.P + p_first) * a.N;
  int64_t slot = 0;
  const bool has_slot = state_slot(a, pc.seq, slot), from = has_slot && starts_from_state(a, pc.seq);
  if (pc.e <= pc.s) {  // an empty sequence: a separate final state array still gets the start state
    if (a.fin && a.fin != a.init && has_slot)
      for (int e = threadIdx.x; e < pn * a.N; e += 2 * TH)
        a.fin[slot * a.s_slot + state_at + e] = from ? a.init[slot * a.s_slot + state_at + e] : 0.f;
    return;
  }
  uint16_t* yb = a.y + col;
  if (!has_slot) {  // zero rows, no state access
    for (int64_t r = pc.s + wave_id(); r < pc.e; r += 2 * W)
      for (int c = lane; c < pn; c += 64) yb[r * a.y_ld + c] = 0;
    return;
  }
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  Chunks<false> c(pc.s, pc.e);
  int rows = c.rows();

  if (!walks) {
    const int tid = threadIdx.x - TH;
    CopyRegs<(int)key_tile(NT), TH> tK, tQ;
    CopyRegs<kRecT, TH> tT, tP;
    CopyRegs<kRecVec, TH> tF;
    u32x4 tV[2];
    auto id_of = [&](const Chunks<false>& n) { return chunk_id(pc, n.c0, d.n_chunk_slots); };
    auto load_chain = [&](const Chunks<false>& n, int left) {
      const int64_t id = id_of(n);
      const char* rec = d.rec + (id * a.H + h) * kRecFwd;
      load_bytes(tK, d.keys + (id * a.G + us.group) * 2 * key_tile(NT), left > 0, tid);
      load_bytes(tT, rec, left > 0, tid);
      load_bytes(tF, rec + kRecFwd - kRecVec, left > 0, tid);
      load_rows<COLS, VEC>(tV, Rows(a.x + n.c0 * a.x_ld + col, a.x_ld, left, pn, 2), (uint32_t)a.x_ld, pn, tid);
    };
    auto store_chain = [&](ChainShared<NT, W>& to) {
      store_bytes(to.k, tK, tid);
      store_bytes(to.t, tT, tid);
      store_bytes(&to.fac, tF, tid);
      store_rows<COLS>(to.v, tV, tid);
    };
    auto load_q = [&](const Chunks<false>& n, int left) {
      load_bytes(tQ, d.keys + ((id_of(n) * a.G + us.group) * 2 + 1) * key_tile(NT), left > 0, tid);
    };
    auto load_p = [&](const Chunks<false>& n, int left) {
      load_bytes(tP, d.rec + (id_of(n) * a.H + h) * kRecFwd + kRecT, left > 0, tid);
    };
    load_chain(c, rows);
    load_q(c, rows);
    load_p(c, rows);
    Chunks<false> next = c, after = c;
    int next_rows = rows, after_rows = rows;
    next = step_chunk(next, next_rows);
    store_chain(chain[0]);
    store_bytes(outp.q, tQ, tid);
    load_chain(next, next_rows);
    load_q(next, next_rows);
    __syncthreads();
    for (int buf = 0;; buf ^= 1) {
      lane = fresh(lane);
      g = lane >> 4, i = lane & 15;
      after = next, after_rows = next_rows;
      after = step_chunk(after, after_rows);
      __syncthreads();  // (1)
      store_bytes(outp.p, tP, tid);
      store_chain(chain[buf ^ 1]);
      load_p(next, next_rows);
      load_chain(after, after_rows);
      phase();
      f32x4 y[4];  // columns p in the registers, rows in the lanes
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) y[ib] = zero;
#pragma unroll
      for (int ks = 0; ks < NT / 32; ++ks) {
        const f16x8 s = outp.s[w][ks][lane];
#pragma unroll
        for (int ib = 0; ib < 4; ++ib) y[ib] = mmah(s, key_rows<NT>(outp.q, 16 * ib, 32 * ks, lane), y[ib]);
      }
      const f32x4 down = *reinterpret_cast<const f32x4*>(&outp.down[w][4 * g]);
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) y[ib] *= down * chain[buf].fac.read[16 * ib + i];
      phase();
      __syncthreads();  // (2)
      store_bytes(outp.q, tQ, tid);
      load_q(after, after_rows);
      phase();
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const Parts up = split(outp.u[w][2 * ks][lane], outp.u[w][2 * ks + 1][lane]);
#pragma unroll
        for (int ib = 2 * ks; ib < 4; ++ib) {
          const bf16x8 p = __builtin_bit_cast(bf16x8, tri_rows<2>(outp.p, ib, ks, 0, lane));
          y[ib] = mma(up.p[0], __builtin_bit_cast(bf16x8, tri_rows<2>(outp.p, ib, ks, 1, lane)), y[ib]);
          y[ib] = mma(up.p[1], p, y[ib]);
          y[ib] = mma(up.p[0], p, y[ib]);
        }
      }
      typedef int i32x4 __attribute__((ext_vector_type(4)));
      const i32x4 bad = *reinterpret_cast<const i32x4*>(&outp.bad[w][4 * g]);
      if (__builtin_expect(__ballot(min(min(bad[0], bad[1]), min(bad[2], bad[3])) < 64) != 0, 0)) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int ib = 0; ib < 4; ++ib)
            if (16 * ib + i >= bad[e]) y[ib][e] = __builtin_nanf("");
      }
      const Rows out(yb + c.c0 * a.y_ld, a.y_ld, rows, pn, 2);
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) {
        const f32x4 v = y[ib];
        store4<VEC>(out, (uint32_t)a.y_ld, 16 * ib + i, 16 * w + 4 * g, pn, u32x2{pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])});
      }
      if (next_rows == 0) return;
      c = next, rows = next_rows;
      next = after, next_rows = after_rows;
    }
  }

  const int p_in = 16 * w + i;  // this lane's state row
  f32x4 S[NB];
  load_state(S, from && p_in < pn ? a.init + slot * a.s_slot + state_at + (int64_t)p_in * a.N : nullptr, a.N, g);
  float s_down = 1.f;  // the state is s_down S
  {
    const Pow2 scale = state_scale<1>(state_max(S));
    s_down = scale.down;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) S[nb] *= scale.up;
  }
  __syncthreads();
  for (int buf = 0;; buf ^= 1) {
    lane = fresh(lane);
    g = lane >> 4, i = lane & 15;
    const ChainShared<NT, W>& sh = chain[buf];
    const Factors& fac = sh.fac;
    f32x4 r[4];  // rows in the registers, columns p in the lanes
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) r[ib] = zero;
    if (g == 0) outp.down[w][i] = s_down;
    Halves s[NT / 32];
#pragma unroll
    for (int ks = 0; ks < NT / 32; ++ks) {
      s[ks] = halves(S[2 * ks], S[2 * ks + 1]);
      outp.s[w][ks][lane] = s[ks].hi;
    }
    __syncthreads();  // (1)
#pragma unroll
    for (int ks = 0; ks < NT / 32; ++ks)
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) r[ib] = mma2(key_rows<NT>(sh.k, 16 * ib, 32 * ks, lane), s[ks], r[ib]);
    const float s_max = state_max(S);
    float r_max = 0.f;
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) {
      const f32x4 f = *reinterpret_cast<const f32x4*>(fac.in + 16 * ib + 4 * g) * s_down;
      r[ib] = fma4(-f, r[ib], column4<COLS>(sh.v, 16 * ib, 16 * w, g, i)) * *reinterpret_cast<const f32x4*>(fac.rate + 16 * ib + 4 * g);
      r_max = max4_nan(r_max, r[ib]);
    }
    // The first row of this lane's column that is not finite: it and the later ones are left out of the products, whose
    // zeros would spread them, and put in at the end
    int bad = __builtin_amdgcn_readfirstlane(fac.bad);
    const bool any_bad = bad < 64 || __ballot(!__builtin_isfinite(r_max)) != 0;
    if (__builtin_expect(any_bad, 0)) {
#pragma unroll
      for (int ib = 3; ib >= 0; --ib)
#pragma unroll
        for (int e = 3; e >= 0; --e) {
          const int row = 16 * ib + 4 * g + e;
          if (!__builtin_isfinite(r[ib][e]) && row < bad) bad = row;
        }
      bad = min(bad, __shfl_xor(bad, 16));
      bad = min(bad, __shfl_xor(bad, 32));
      r_max = 0.f;
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (16 * ib + 4 * g + e >= bad) r[ib][e] = 0.f;
        r_max = max4(r_max, r[ib]);
      }
    }
    const Pow2 rs = bring_to<10>(max_across16(r_max));
    f32x4 u[4];
    {
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) r[ib] *= rs.up;
      const Halves rp[2] = {halves(r[0], r[1]), halves(r[2], r[3])};
      const float u_down = rs.down * fac.t_scale;
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) {
        u[ib] = zero;
#pragma unroll
        for (int ks = 0; ks <= ib / 2; ++ks) u[ib] = mma3(t_rows(sh.t, ib, ks, lane), rp[ks], u[ib]);
      }
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) {
        u[ib] *= u_down;
        outp.u[w][ib][lane] = u[ib];
      }
      if (g == 0) outp.bad[w][i] = bad;
    }
    __syncthreads();  // (2)
    // what goes into the state and its scale
    float o_max = 0.f;
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) {
      u[ib] *= *reinterpret_cast<const f32x4*>(fac.out + 16 * ib + 4 * g);
      o_max = max4(o_max, u[ib]);
    }
    const float grown = fac.decay * s_down;
    const Pow2 ss = state_scale<1>(__builtin_fmaxf(max_across16(o_max), s_max * grown));
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) S[nb] *= grown * ss.up;
    s_down = ss.down;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const Halves o = halves(u[2 * ks] * ss.up, u[2 * ks + 1] * ss.up);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) S[nb] = mma2(key_cols<NT>(sh.k, 32 * ks, 16 * nb, lane), o, S[nb]);
    }
    if (__builtin_expect(any_bad, 0)) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        if (bad < 64) S[nb] = f32x4{1.f, 1.f, 1.f, 1.f} * __builtin_nanf("");
    }
    c = step_chunk(c, rows);
    if (rows == 0) break;
  }
  if (a.fin && p_in < pn) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) S[nb] *= s_down;
    store_state(S, a.fin + slot * a.s_slot + state_at + (int64_t)p_in * a.N, a.N, lane >> 4);
  }
}

// The same for states of more than 128 columns, whose tiles shared memory does not hold twice: four waves that walk and make y,
// a wave's 16 x 256 values of the state in 64 registers a lane.  Shared memory is filled between the chunks.
template <int NT, bool VEC>
__global__ __launch_bounds__(256, NT <= 128 ? 2 : 1) void delta_scan_fwd_wide_kernel(DeltaArgs d) {
  constexpr int T = 256, NB = NT / 16, kKeys = 2 * (int)key_tile(NT);
  __shared__ __align__(16) uint16_t sKQ[kKeys / 2];
  __shared__ __align__(16) uint16_t sV[64 * kLd<64, 16>];
  __shared__ __align__(16) char sR[kRecFwd];
  const uint16_t *sK = sKQ, *sQ = sKQ + kKeys / 4;
  const ScanArgs& a = d.s;
  const Units<1> us(a, blockIdx.x);
  if (!us.ok) return;
  const Unit me(a, us, 0);
  const int w = wave_id(), pn = me.pn;
  Piece pc;
  pc.seq = walk_sequence(d, us.item);
  seq_bounds(a.q, pc.seq, pc.s, pc.e);
  int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15;
  const int p_in = 16 * w + i;  // this lane's state row
  const int64_t state_at = ((int64_t)me.h * a.P + me.p_first) * a.N;
  int64_t slot = 0;
  const bool has_slot = state_slot(a, pc.seq, slot), from = has_slot && starts_from_state(a, pc.seq);
  if (pc.e <= pc.s) {  // an empty sequence: a separate final state array still gets the start state
    if (a.fin && a.fin != a.init && has_slot)
      for (int e = threadIdx.x; e < pn * a.N; e += T)
        a.fin[slot * a.s_slot + state_at + e] = from ? a.init[slot * a.s_slot + state_at + e] : 0.f;
    return;
  }
  uint16_t* yb = a.y + me.col;
  if (!has_slot) {  // zero rows, no state access
    for (int64_t r = pc.s + w; r < pc.e; r += 4)
      if (lane < pn) yb[r * a.y_ld + lane] = 0;
    return;
  }
  f32x4 S[NB];
  load_state(S, from && p_in < pn ? a.init + slot * a.s_slot + state_at + (int64_t)p_in * a.N : nullptr, a.N, g);
  float s_down = 1.f;  // the state is s_down S
  {
    const Pow2 scale = state_scale<1>(state_max(S));
    s_down = scale.down;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) S[nb] *= scale.up;
  }

  CopyRegs<kKeys, T> tK;
  TileRegs<64, T> tV;
  CopyRegs<kRecFwd, T> tR;
  auto load = [&](const Chunks<false>& c, int rows) {
    const int64_t id = chunk_id(pc, c.c0, d.n_chunk_slots);
    load_bytes(tK, d.keys + (id * a.G + us.group) * kKeys, rows > 0, threadIdx.x);
    load_bytes(tR, d.rec + (id * a.H + me.h) * kRecFwd, rows > 0, threadIdx.x);
    load_tile<VEC>(tV, Rows(a.x + c.c0 * a.x_ld + me.col, a.x_ld, rows, pn, 2), (uint32_t)a.x_ld, pn);
  };
  Chunks<false> c(pc.s, pc.e);
  int rows = c.rows();
  load(c, rows);
  const char* sT = sR;
  const char* sP = sR + kRecT;
  const Factors& fac = *reinterpret_cast<const Factors*>(sR + kRecFwd - kRecVec);
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  for (;;) {
    lane = fresh(lane);
    g = lane >> 4, i = lane & 15;
    store_bytes(sKQ, tK, threadIdx.x);
    store_bytes(sR, tR, threadIdx.x);
    store_tile<16>(sV, tV);
    __syncthreads();
    const Rows out(yb + c.c0 * a.y_ld, a.y_ld, rows, pn, 2);
    c = step_chunk(c, rows);  // rows == 0: that was the last one
    load(c, rows);
    phase();
    f32x4 r[4], y[4];  // rows in the registers, columns p in the lanes; y the other way round
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) r[ib] = y[ib] = zero;
#pragma unroll
    for (int ks = 0; ks < NT / 32; ++ks) {
      const Halves s = halves(S[2 * ks], S[2 * ks + 1]);
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) {
        r[ib] = mma2(key_rows<NT>(sK, 16 * ib, 32 * ks, lane), s, r[ib]);
        y[ib] = mmah(s.hi, key_rows<NT>(sQ, 16 * ib, 32 * ks, lane), y[ib]);
      }
    }
    const float s_max = state_max(S);
    {
      f32x4 sd;  // the columns' scales, where columns are in the registers
#pragma unroll
      for (int e = 0; e < 4; ++e) sd[e] = __shfl(s_down, 4 * g + e);
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) y[ib] *= sd * fac.read[16 * ib + i];
    }
    float r_max = 0.f;
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) {
      const f32x4 f = *reinterpret_cast<const f32x4*>(fac.in + 16 * ib + 4 * g) * s_down;
      r[ib] = fma4(-f, r[ib], column4(sV, 16 * ib, 16 * w, g, i)) * *reinterpret_cast<const f32x4*>(fac.rate + 16 * ib + 4 * g);
      r_max = max4_nan(r_max, r[ib]);
    }
    // The first row of this lane's column that is not finite: it and the later ones are left out of the products, whose
    // zeros would spread them, and put in at the end
    int bad = __builtin_amdgcn_readfirstlane(fac.bad);
    const bool any_bad = bad < 64 || __ballot(!__builtin_isfinite(r_max)) != 0;
    if (__builtin_expect(any_bad, 0)) {
#pragma unroll
      for (int ib = 3; ib >= 0; --ib)
#pragma unroll
        for (int e = 3; e >= 0; --e) {
          const int row = 16 * ib + 4 * g + e;
          if (!__builtin_isfinite(r[ib][e]) && row < bad) bad = row;
        }
      bad = min(bad, __shfl_xor(bad, 16));
      bad = min(bad, __shfl_xor(bad, 32));
      r_max = 0.f;
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (16 * ib + 4 * g + e >= bad) r[ib][e] = 0.f;
        r_max = max4(r_max, r[ib]);
      }
    }
    const Pow2 rs = bring_to<10>(max_across16(r_max));
    f32x4 u[4];
    {
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) r[ib] *= rs.up;
      const Halves rp[2] = {halves(r[0], r[1]), halves(r[2], r[3])};
      const float u_down = rs.down * fac.t_scale;
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) {
        u[ib] = zero;
#pragma unroll
        for (int ks = 0; ks <= ib / 2; ++ks)
          u[ib] = mma3(t_rows(sT, ib, ks, lane), rp[ks], u[ib]);
      }
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) u[ib] *= u_down;
    }
    // what goes into the state and its scale
    f32x4 o[4];
    float o_max = 0.f;
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) {
      o[ib] = u[ib] * *reinterpret_cast<const f32x4*>(fac.out + 16 * ib + 4 * g);
      o_max = max4(o_max, o[ib]);
    }
    const float grown = fac.decay * s_down;
    const Pow2 ss = state_scale<1>(__builtin_fmaxf(max_across16(o_max), s_max * grown));
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) S[nb] *= grown * ss.up;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const Halves op = halves(o[2 * ks] * ss.up, o[2 * ks + 1] * ss.up);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) S[nb] = mma2(key_cols<NT>(sK, 32 * ks, 16 * nb, lane), op, S[nb]);
      const Parts up = split(u[2 * ks], u[2 * ks + 1]);
#pragma unroll
      for (int ib = 2 * ks; ib < 4; ++ib) {
        const bf16x8 p = __builtin_bit_cast(bf16x8, tri_rows<2>(sP, ib, ks, 0, lane));
        y[ib] = mma(up.p[0], __builtin_bit_cast(bf16x8, tri_rows<2>(sP, ib, ks, 1, lane)), y[ib]);
        y[ib] = mma(up.p[1], p, y[ib]);
        y[ib] = mma(up.p[0], p, y[ib]);
      }
    }
    s_down = ss.down;
    if (__builtin_expect(any_bad, 0)) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        if (bad < 64) S[nb] = f32x4{1.f, 1.f, 1.f, 1.f} * __builtin_nanf("");
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int first = __shfl(bad, 4 * g + e);
#pragma unroll
        for (int ib = 0; ib < 4; ++ib)
          if (16 * ib + i >= first) y[ib][e] = __builtin_nanf("");
      }
    }
    const int p_out = 16 * w + 4 * g;
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) {
      const f32x4 v = y[ib];
      store4<VEC>(out, (uint32_t)a.y_ld, 16 * ib + i, p_out, pn, u32x2{pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])});
    }
    if (rows == 0) break;
    __syncthreads();
  }
  if (a.fin && p_in < pn) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) S[nb] *= s_down;
    store_state(S, a.fin + slot * a.s_slot + state_at + (int64_t)p_in * a.N, a.N, lane >> 4);
  }
}

// 64 columns a block, or 32 if there is a CU for every such block: a wave that walks then has its SIMD for itself.  One prompt of
// 2048 rows, 32 heads of 128: 122 us with 32, 129 with 64 (110 since the instructions of a chunk became fewer); 4 x 4096 rows, which
// fill the card with 64: 495 and 328.  (128 columns,
// 16 waves of 128 registers: 490, and 64 mixed prompts 990 for 800.)
template <int NT, int W>
static void walk(DeltaArgs a, bool vec, hipStream_t s) {
  a.s.ptiles = (a.s.P + 16 * W - 1) / (16 * W);
  const dim3 grid((uint32_t)unit_blocks(a.s.q.nseq, a.s.H, a.s.G, a.s.ptiles, 1));
  if (vec) delta_scan_fwd_kernel<NT, W, true><<<grid, 128 * W, 0, s>>>(a);
  else delta_scan_fwd_kernel<NT, W, false><<<grid, 128 * W, 0, s>>>(a);
}

template <int NT>
static void launch(const DeltaArgs& a, bool vec, hipStream_t s) {
  if constexpr (NT > 128) {
    const dim3 grid((uint32_t)unit_blocks(a.s.q.nseq, a.s.H, a.s.G, a.s.ptiles, 1));
    if (vec) delta_scan_fwd_wide_kernel<NT, true><<<grid, 256, 0, s>>>(a);
    else delta_scan_fwd_wide_kernel<NT, false><<<grid, 256, 0, s>>>(a);
  } else {
    if (a.s.q.nseq * a.s.H * ((a.s.P + 31) / 32) <= 256) walk<NT, 2>(a, vec, s);
    else walk<NT, 4>(a, vec, s);
  }
}

hipError_t launch_delta_fwd(const DeltaArgs& a, bool vec, hipStream_t s) {
  if (a.s.q.rows > 0) {
    const hipError_t e = launch_delta_chunks(a, nullptr, vec, s);
    if (e != hipSuccess) return e;
  }
  switch (state_tile(a.s.N)) {
    case 64: launch<64>(a, vec, s); break;
    case 128: launch<128>(a, vec, s); break;
    default: launch<256>(a, vec, s); break;
  }
  return hipGetLastError();
}

}  // namespace cssm
