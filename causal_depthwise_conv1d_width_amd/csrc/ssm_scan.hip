// ssm_scan.hip -- forward selective state space scan over packed rows.
//
// A block walks one piece of one sequence for U units (64 columns of a head) of one group, a chunk of
// 64 rows at a time, with the FP32 states in registers from chunk to chunk (no state travels through memory):
//   Y = e^{L} (C S) + (M * dt * (C B^T)) X + D X,    S' = e^{L_Q} S + X^T (e^{L_Q - L} dt B)
// The units share the chunk's B and C rows and its 64 x 64 scores C B^T, whose ten 16 x 16 blocks up to the
// diagonal go to the waves; each wave decays its blocks for every unit.  Then a wave owns 16 * PB columns p of Y
// and of its unit's state, which it holds transposed ([n, p]: registers n), as the operand that C S needs.
// Shared memory feeds the matrix instructions: with four units and PB = 2 a wave uses every B, C and score operand
// twice.  The 256-column state tile leaves no registers for that: two units, PB = 1.
// Exponents of decays between two rows are differences of 64-bit sums (Rate::exponent).  The decayed scores and the
// state's operand in C S are rounded to bf16 once each: y is bf16.  The new state's
// terms enter as two bf16 parts, 2^-16 of a term: a pool came out 0.6e-7 to 3.5e-7 off; a third part costs 6%.
// Bound by what two waves a SIMD leave of the waves' own latency, shared memory reads first.  64 heads of 64
// columns, N = 128:
// 16384 rows of 4 sequences 140 us (280 TFLOP/s of the formula's products) and 64 us for the walk before
// and the join; 32512 rows of 64 prompts 385 us.
#include "ssm_state.h"

namespace cssm {

// Non-finite x.  The decayed scores hold zeros past the diagonal, and zero times a non-finite x of a later row is a
// NaN.  A product of x with zeros finds them: any in a wave's columns of the chunk makes it NaN.  64 mixed prompts (head of
// the file) 456 us, 445 without; a look per 32 rows at their use 461, at the bits on their way to shared memory 469.
template <int PB>
__device__ __forceinline__ bool any_non_finite(const bf16x8 (&x)[2][PB]) {
  f32x4 t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int ks = 0; ks < 2; ++ks)
#pragma unroll
    for (int pb = 0; pb < PB; ++pb) t = mma(x[ks][pb], bf16x8{}, t);
  const float v = (t[0] + t[1]) + (t[2] + t[3]);
  return __ballot(v != v) != 0;
}
// Makes Y NaN in the column of a non-finite x from its row on (the rows i with a one at j <= i in the product of the
// places of such x with the lower triangle), and that x zero in the operand.  ks: the operand's half of the chunk.
__device__ __forceinline__ void contain_non_finite(bf16x8& x, f32x4 (&y)[4], int ks, int g, int i) {
  u32x4 u = __builtin_bit_cast(u32x4, x), at;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const bool lo = (u[e] & 0x7f80u) == 0x7f80u, hi = (u[e] & 0x7f800000u) == 0x7f800000u;
    at[e] = (lo ? 0x3f80u : 0u) | (hi ? 0x3f800000u : 0u);
    u[e] &= (lo ? 0u : 0xffffu) | (hi ? 0u : 0xffff0000u);
  }
  x = __builtin_bit_cast(bf16x8, u);
#pragma unroll
  for (int ib = 0; ib < 4; ++ib) {
    u32x4 lower;
#pragma unroll
    for (int e = 0; e < 4; ++e) {  // positions 2 e, 2 e + 1 of the split order
      const int j = 32 * ks + 16 * (e >> 1) + 4 * g + 2 * (e & 1), row = 16 * ib + i;
      lower[e] = (j <= row ? 0x3f80u : 0u) | (j < row ? 0x3f800000u : 0u);
    }
    const f32x4 n = mma(__builtin_bit_cast(bf16x8, at), __builtin_bit_cast(bf16x8, lower), f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
    for (int r = 0; r < 4; ++r) y[ib][r] = n[r] > 0.f ? __builtin_nanf("") : y[ib][r];
  }
}

template <int NT, int U, int PB, bool VEC>
__global__ __launch_bounds__(256 / PB * U, 2) void ssm_scan_fwd_kernel(ScanArgs a) {
  constexpr int T = 256 / PB * U, NB = NT / 16, WU = 4 / PB;  // threads, state blocks, waves a unit
  __shared__ __align__(16) uint16_t sx_[U][64 * kLd<64, 16>];
  __shared__ __align__(16) uint16_t sB[64 * kLd<NT, 16>];
  __shared__ __align__(16) uint16_t sC[64 * kLd<NT>];
  __shared__ __align__(16) uint16_t sP_[U][64 * kLd<64>];
  // this chunk's and the next one's, by unit: prefix sums L; steps, 2^L, weights of the state update
  __shared__ __align__(16) double ssum[2][U][64];
  __shared__ __align__(16) float sdecay[2][U][3][64];
  const int hp = a.H * a.ptiles;
  const Units<U> us(a, blockIdx.x);
  if (!us.ok) return;
  const int wave = wave_id(), un = wave / WU, w = wave % WU;
  const Unit me(a, us, un);
  const int pn = me.pn;
  const Piece pc = find_piece(a.q, us.item, a.seg, a.n_slots);
  int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15;
  const int p_in = 16 * PB * w + i;       // this lane's first state column
  const int64_t state_at = ((int64_t)me.h * a.P + me.p_first) * a.N;
  int64_t slot = 0;
  if (!pc.ok) {
    // an empty sequence: a separate final state array still gets the start state
    if (us.item >= a.n_slots && a.fin && a.fin != a.init && state_slot(a, pc.seq, slot)) {
      const bool from = starts_from_state(a, pc.seq);
      for (int e = threadIdx.x % (64 * WU); e < pn * a.N; e += 64 * WU)
        a.fin[slot * a.s_slot + state_at + e] = from ? a.init[slot * a.s_slot + state_at + e] : 0.f;
    }
    return;
  }
  uint16_t* yb = a.y + (int64_t)me.h * a.P + me.p_first;
  if (!state_slot(a, pc.seq, slot)) {  // no slot: zero rows, no state access
    for (int64_t r = pc.r0 + w; r < pc.r1; r += WU)
      if (lane < pn) yb[r * a.y_ld + lane] = 0;
    return;
  }

  f32x4 S[PB][NB];
#pragma unroll
  for (int pb = 0; pb < PB; ++pb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) S[pb][nb] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (a.seg > 0 && piece_count(pc.e - pc.s, a.seg) > 1) {
    const float* src = a.piece + (us.item * hp + me.tile) * (64 * NT) + p_in * NT + 4 * g;
#pragma unroll
    for (int pb = 0; pb < PB; ++pb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) S[pb][nb] = *reinterpret_cast<const f32x4*>(src + pb * 16 * NT + 16 * nb);
  } else if (starts_from_state(a, pc.seq)) {
#pragma unroll
    for (int pb = 0; pb < PB; ++pb) {
      if (p_in + 16 * pb >= pn) continue;
      const float* src = a.init + slot * a.s_slot + state_at + (int64_t)(p_in + 16 * pb) * a.N + 4 * g;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        if (16 * nb + 4 * g + 3 < a.N) {
          S[pb][nb] = *reinterpret_cast<const f32x4_a4*>(src + 16 * nb);
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (16 * nb + 4 * g + r < a.N) S[pb][nb][r] = src[16 * nb + r];
        }
      }
    }
  }

  const Rate rate(a, me.h);
  const float Dh = a.D ? uniform(a.D[me.h]) : 0.f;
  const int64_t gn = (int64_t)us.group * a.N;
  const uint16_t *Bb = a.B + gn, *Cb = a.C + gn;
  TileRegs<64, T> tx[U];
  TileRegs<NT, T> tB, tC;
  auto load = [&](const Chunks<false>& c, int rows) {
    const Rows xr(a.x + c.c0 * a.x_ld, a.x_ld, rows, a.H * a.P, 2);
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const Unit o(a, us, q);
      load_tile<VEC>(tx[q], xr, (uint32_t)a.x_ld, o.pn, o.col);
    }
    load_tile<VEC>(tB, Rows(Bb + c.c0 * a.B_ld, a.B_ld, rows, a.N, 2), (uint32_t)a.B_ld, a.N);
    load_tile<VEC>(tC, Rows(Cb + c.c0 * a.C_ld, a.C_ld, rows, a.N, 2), (uint32_t)a.C_ld, a.N);
  };
  // a chunk's decays into buffer `at`: a unit's first wave the prefix sums, steps and their powers, its
  // second, whose lanes count from the chunk's end, the weights of the state update
  RawStep raw{};
  const int my = w == 0 ? (int)(threadIdx.x & 63) : 63 - (int)(threadIdx.x & 63);
  auto decays = [&](int rows, int at) {
    const float d = rate.step(raw, my < rows);
    if (w == 0) {
      const double L = wave_prefix(rate.exponent(d));
      ssum[at][un][lane] = L;
      sdecay[at][un][0][lane] = d;
      sdecay[at][un][1][lane] = ex2((float)L);
    } else {
      sdecay[at][un][2][my] = ex2(dpp0<0x138, 0xf>(wave_prefix(d * rate.A2))) * d;
    }
  };
  Chunks<false> c(pc.r0, pc.r1);
  int rows = c.rows();
  load(c, rows);
  raw = raw_step(a, c.c0, rows, my, me.h);
  if (w < 2) decays(rows, 0);
  Chunks<false> after = c;
  int after_rows = rows;  // the chunk whose raw steps come next
  after = step_chunk(after, after_rows);
  raw = raw_step(a, after.c0, after_rows, my, me.h);
  // products over 32 columns read two blocks past the diagonal, which no wave writes
  for (int e = threadIdx.x; e < U * 64 * kLd<64> / 2; e += T) reinterpret_cast<uint32_t*>(sP_)[e] = 0u;
  const uint16_t *sx = sx_[un], *sP = sP_[un];
  for (int buf = 0;; buf ^= 1) {
    lane = fresh(lane);
    g = lane >> 4, i = lane & 15;
    const int p_out = 16 * PB * w + 4 * g;  // this lane's first of four output columns
#pragma unroll
    for (int q = 0; q < U; ++q) store_tile<16>(sx_[q], tx[q]);
    store_tile<16>(sB, tB);
    store_tile(sC, tC);
    __syncthreads();
    const Rows out(yb + c.c0 * a.y_ld, a.y_ld, rows, pn, 2);
    c = step_chunk(c, rows);  // rows == 0: that was the last one
    load(c, rows);
    if (w < 2) decays(rows, buf ^ 1);
    after = step_chunk(after, after_rows);
    raw = raw_step(a, after.c0, after_rows, my, me.h);
    // score block (ib, jb): rows i in the lanes, columns j in the registers, decayed, times dt_j
    auto scores = [&](int ib, int jb) {
      f32x4 t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < NT / 32; ++ks)
        t = mma(op_straight<NT, 16>(sB, 16 * jb, 32 * ks, lane), op_straight<NT>(sC, 16 * ib, 32 * ks, lane), t);
#pragma unroll
      for (int q = 0; q < U; ++q) {
        const double *sL = ssum[buf][q], Li = sL[16 * ib + i];
        const f32x4 dj = *reinterpret_cast<const f32x4*>(sdecay[buf][q][0] + 16 * jb + 4 * g);
        f32x4 v;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          v[r] = t[r] * (ex2((float)(Li - sL[16 * jb + 4 * g + r])) * dj[r]);
          v[r] = 16 * jb + 4 * g + r <= 16 * ib + i ? v[r] : 0.f;
        }
        *reinterpret_cast<u32x2*>(sP_[q] + at<64>(16 * ib + i, 16 * jb + 4 * g)) =
            u32x2{pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])};
      }
    };
#pragma unroll
    for (int k = 0; k < 10; k += T / 64) {
      int ib, jb;
      lower_block(wave + k, ib, jb);
      if (wave + k < 10) scores(ib, jb);
    }
    phase();
    // Y^T (registers p, lanes i) from the state before the chunk
    f32x4 y[PB][4];
#pragma unroll
    for (int pb = 0; pb < PB; ++pb)
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) y[pb][ib] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < NT / 32; ++ks) {
      bf16x8 s[PB];
#pragma unroll
      for (int pb = 0; pb < PB; ++pb) s[pb] = op_result(S[pb][2 * ks], S[pb][2 * ks + 1]);
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) {
        const bf16x8 cv = op_split<NT>(sC, 16 * ib, 32 * ks, lane);
#pragma unroll
        for (int pb = 0; pb < PB; ++pb) y[pb][ib] = mma(s[pb], cv, y[pb][ib]);
      }
    }
    const float *se = sdecay[buf][un][1], *sw = sdecay[buf][un][2];
#pragma unroll
    for (int ib = 0; ib < 4; ++ib)
#pragma unroll
      for (int pb = 0; pb < PB; ++pb) y[pb][ib] *= se[16 * ib + i];
    phase();
    bf16x8 x[2][PB];  // x as an operand: columns p, contracted rows
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int pb = 0; pb < PB; ++pb) x[ks][pb] = op_cols<64, 16>(sx, 32 * ks, 16 * (PB * w + pb), lane);
    const bool bad = any_non_finite(x);
    if (__builtin_expect(bad, 0)) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int pb = 0; pb < PB; ++pb) contain_non_finite(x[ks][pb], y[pb], ks, g, i);
    }
    __syncthreads();
    const float et = se[63];
#pragma unroll
    for (int pb = 0; pb < PB; ++pb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) S[pb][nb] *= et;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      Parts xw[PB];
      {
#pragma unroll
        for (int ib = 2 * ks; ib < 4; ++ib) {
          const bf16x8 pv = op_split<64>(sP, 16 * ib, 32 * ks, lane);
#pragma unroll
          for (int pb = 0; pb < PB; ++pb) y[pb][ib] = mma(x[ks][pb], pv, y[pb][ib]);
        }
        if (__builtin_expect(bad, 0)) {  // the state takes them as they are
#pragma unroll
          for (int pb = 0; pb < PB; ++pb) x[ks][pb] = op_cols<64, 16>(sx, 32 * ks, 16 * (PB * w + pb), lane);
        }
        const f32x4 wa = *reinterpret_cast<const f32x4*>(sw + 32 * ks + 4 * g);
        const f32x4 wb = *reinterpret_cast<const f32x4*>(sw + 32 * ks + 16 + 4 * g);
#pragma unroll
        for (int pb = 0; pb < PB; ++pb) xw[pb] = split_scaled(x[ks][pb], wa, wb);
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const bf16x8 b = op_cols<NT, 16>(sB, 32 * ks, 16 * nb, lane);
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int pb = 0; pb < PB; ++pb) S[pb][nb] = mma(b, xw[pb].p[q], S[pb][nb]);
      }
      phase();
    }
#pragma unroll
    for (int ib = 0; ib < 4; ++ib)
#pragma unroll
      for (int pb = 0; pb < PB; ++pb) {
        const int row = 16 * ib + i, p = p_out + 16 * pb;
        const u32x2 xv = *reinterpret_cast<const u32x2*>(sx + at<64, 16>(row, p));
        const f32x4 v = y[pb][ib];
        const u32x2 o = {pk_bf16(v[0] + Dh * bf_lo(xv.x), v[1] + Dh * bf_hi(xv.x)),
                         pk_bf16(v[2] + Dh * bf_lo(xv.y), v[3] + Dh * bf_hi(xv.y))};
        store4<VEC>(out, (uint32_t)a.y_ld, row, p, pn, o);
      }
    if (rows == 0) break;
    __syncthreads();
  }

  if (a.fin && pc.r1 == pc.e) {
#pragma unroll
    for (int pb = 0; pb < PB; ++pb) {
      if (p_in + 16 * pb >= pn) continue;
      float* dst = a.fin + slot * a.s_slot + state_at + (int64_t)(p_in + 16 * pb) * a.N + 4 * g;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        if (16 * nb + 4 * g + 3 < a.N) {
          *reinterpret_cast<f32x4_a4*>(dst + 16 * nb) = S[pb][nb];
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (16 * nb + 4 * g + r < a.N) dst[16 * nb + r] = S[pb][nb][r];
        }
      }
    }
  }
}

template <int NT, bool VEC>
static hipError_t launch(const ScanArgs& a, hipStream_t s) {
  const int64_t items = a.n_slots + a.q.nseq;
  if (a.seg > 0) {
    StateArgs k{};
    k.s = a;
    k.u = a.x;
    k.v = a.B;
    k.u_ld = a.x_ld;
    k.v_ld = a.B_ld;
    k.start = a.init;
    k.piece = a.piece;
    k.decay = a.piece_decay;
    const dim3 walk((uint32_t)unit_blocks(items, a.H, a.G, a.ptiles, kUnits));
    ssm_state_local_kernel<NT, kUnits, VEC><<<walk, 128 * kUnits, 0, s>>>(k);
    ssm_join_kernel<NT, false><<<join_grid(a, NT), 1024, 0, s>>>(k);
  }
  constexpr int U = NT > 128 ? 2 : kUnits, PB = NT > 128 ? 1 : 2;
  ssm_scan_fwd_kernel<NT, U, PB, VEC>
      <<<dim3((uint32_t)unit_blocks(items, a.H, a.G, a.ptiles, U)), 256 / PB * U, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_scan_fwd(const ScanArgs& a, bool vec, hipStream_t s) {
  switch (state_tile(a.N)) {
    case 64: return vec ? launch<64, true>(a, s) : launch<64, false>(a, s);
    case 128: return vec ? launch<128, true>(a, s) : launch<128, false>(a, s);
    default: return vec ? launch<256, true>(a, s) : launch<256, false>(a, s);
  }
}

}  // namespace cssm
