// ssm_scan.hip -- forward selective state space scan over packed rows.
//
// A block walks one piece of one sequence for one head (64 of its columns), a chunk of 64 rows at a
// time, with the FP32 state in registers from chunk to chunk (no state travels through memory):
//   Y = e^{L} (C S) + (M * dt * (C B^T)) X + D X,    S' = e^{L_Q} S + X^T (e^{L_Q - L} dt B)
// Four waves: each computes 16 rows of the 64 x 64 score tile, then owns 16 columns p of Y and of the
// state, which it holds transposed ([n, p]: registers n), as the operand that C S needs.
#include "ssm_state.h"

namespace cssm {

template <int NT, bool VEC>
__global__ __launch_bounds__(256, NT > 128 ? 1 : 2) void ssm_scan_fwd_kernel(ScanArgs a) {
  constexpr int NB = NT / 16;
  __shared__ __align__(16) uint16_t sx[64 * kLd<64>];
  __shared__ __align__(16) uint16_t sB[64 * kLd<NT>];
  __shared__ __align__(16) uint16_t sC[64 * kLd<NT>];
  __shared__ __align__(16) uint16_t sP[64 * kLd<64>];
  __shared__ __align__(16) float sdecay[2][4][64];  // this chunk's and the next one's
  const int hp = a.H * a.ptiles;
  const uint32_t blk = xcd_block(blockIdx.x, gridDim.x);
  const int64_t item = blk / hp;
  const int head_tile = blk % hp, h = head_tile / a.ptiles, p_first = head_tile % a.ptiles * kPTile;
  const Piece pc = find_piece(a.q, item, a.seg, a.n_slots);
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = lane >> 4, i = lane & 15;
  const int pn = a.P - p_first < kPTile ? a.P - p_first : kPTile;
  const int p_in = 16 * w + i;         // this lane's state column
  const int p_out = 16 * w + 4 * g;    // this lane's first of four output columns
  const int64_t state_at = ((int64_t)h * a.P + p_first) * a.N;
  int64_t slot = 0;
  if (!pc.ok) {
    // an empty sequence: a separate final state array still gets the start state
    if (item >= a.n_slots && a.fin && a.fin != a.init && state_slot(a, pc.seq, slot)) {
      const bool from = starts_from_state(a, pc.seq);
      for (int e = threadIdx.x; e < pn * a.N; e += 256)
        a.fin[slot * a.s_slot + state_at + e] = from ? a.init[slot * a.s_slot + state_at + e] : 0.f;
    }
    return;
  }
  uint16_t* yb = a.y + (int64_t)h * a.P + p_first;
  if (!state_slot(a, pc.seq, slot)) {  // no slot: zero rows, no state access
    for (int64_t r = pc.r0 + w; r < pc.r1; r += 4)
      if (lane < pn) yb[r * a.y_ld + lane] = 0;
    return;
  }

  f32x4 S[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) S[nb] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (a.seg > 0) {
    const float* src = a.piece + (item * hp + head_tile) * (64 * NT) + p_in * NT + 4 * g;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) S[nb] = *reinterpret_cast<const f32x4*>(src + 16 * nb);
  } else if (starts_from_state(a, pc.seq) && p_in < pn) {
    const float* src = a.init + slot * a.s_slot + state_at + (int64_t)p_in * a.N + 4 * g;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      if (16 * nb + 4 * g + 3 < a.N) {
        S[nb] = *reinterpret_cast<const f32x4_a4*>(src + 16 * nb);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (16 * nb + 4 * g + r < a.N) S[nb][r] = src[16 * nb + r];
      }
    }
  }

  const Rate rate(a, h);
  const float Dh = a.D ? a.D[h] : 0.f;
  const uint16_t* xb = a.x + (int64_t)h * a.P + p_first;
  const int64_t gn = (int64_t)(h / (a.H / a.G)) * a.N;
  const uint16_t *Bb = a.B + gn, *Cb = a.C + gn;
  TileRegs<64> tx;
  TileRegs<NT> tB, tC;
  // a chunk's decays into buffer `at`: wave 0 the prefix sums, steps and their powers, wave 1, whose lanes
  // count from the chunk's end, the weights of the state update
  float raw = 0.f;
  const int my = w == 0 ? lane : 63 - lane;
  auto decays = [&](const Chunks<false>& c, int at) {
    const float d = rate.step(raw, my < c.rows());
    const float L = wave_prefix(d * rate.A2);
    if (w == 0) {
      sdecay[at][0][lane] = L;
      sdecay[at][1][lane] = d;
      sdecay[at][2][lane] = ex2(L);
    } else {
      sdecay[at][3][my] = ex2(dpp0<0x138, 0xf>(L)) * d;
    }
  };
  Chunks<false> c(pc.r0, pc.r1);
  load_tile<64, VEC>(tx, xb + c.c0 * a.x_ld, a.x_ld, c.rows(), pn);
  load_tile<NT, VEC>(tB, Bb + c.c0 * a.B_ld, a.B_ld, c.rows(), a.N);
  load_tile<NT, VEC>(tC, Cb + c.c0 * a.C_ld, a.C_ld, c.rows(), a.N);
  if (w < 2) {
    raw = raw_step(a, c.c0 + my, c.c0, c.c1, h);
    decays(c, 0);
    if (!c.last()) raw = raw_step(a, c.next().c0 + my, c.next().c0, c.next().c1, h);
  }
  for (int buf = 0;; buf ^= 1) {
    store_tile<64>(sx, tx);
    store_tile<NT>(sB, tB);
    store_tile<NT>(sC, tC);
    __syncthreads();
    const int64_t r0 = c.c0;
    const int rows = c.rows();
    const bool more = !c.last();
    const float *sL = sdecay[buf][0], *sd = sdecay[buf][1], *se = sdecay[buf][2], *sw = sdecay[buf][3];
    if (more) {
      c = c.next();
      load_tile<64, VEC>(tx, xb + c.c0 * a.x_ld, a.x_ld, c.rows(), pn);
      load_tile<NT, VEC>(tB, Bb + c.c0 * a.B_ld, a.B_ld, c.rows(), a.N);
      load_tile<NT, VEC>(tC, Cb + c.c0 * a.C_ld, a.C_ld, c.rows(), a.N);
      if (w < 2) {  // these waves have the fewer score blocks
        decays(c, buf ^ 1);
        if (!c.last()) raw = raw_step(a, c.next().c0 + my, c.next().c0, c.next().c1, h);
      }
    }
    // scores of rows 16 w .. 16 w + 15 (lanes) against columns j (registers), decayed, times dt_j
    {
      bf16x8 c[NT / 32];
#pragma unroll
      for (int ks = 0; ks < NT / 32; ++ks) c[ks] = op_straight<NT>(sC, 16 * w, 32 * ks);
      const float Li = sL[16 * w + i];
#pragma unroll
      for (int jb = 0; jb < 4; ++jb) {
        if (jb > (w | 1)) continue;  // pairs of blocks past the diagonal are never read
        f32x4 t = {0.f, 0.f, 0.f, 0.f};
        if (jb <= w) {
#pragma unroll
          for (int ks = 0; ks < NT / 32; ++ks) t = mma(op_straight<NT>(sB, 16 * jb, 32 * ks), c[ks], t);
          const f32x4 Lj = *reinterpret_cast<const f32x4*>(sL + 16 * jb + 4 * g);
          const f32x4 dj = *reinterpret_cast<const f32x4*>(sd + 16 * jb + 4 * g);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float v = t[r] * (ex2(Li - Lj[r]) * dj[r]);
            t[r] = 16 * jb + 4 * g + r <= 16 * w + i ? v : 0.f;
          }
        }
        const u32x2 o = {pk_bf16(t[0], t[1]), pk_bf16(t[2], t[3])};
        *reinterpret_cast<u32x2*>(sP + at<64>(16 * w + i, 16 * jb + 4 * g)) = o;
      }
    }
    // Y^T (registers p, lanes i) from the state before the chunk
    f32x4 y[4];
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) y[ib] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < NT / 32; ++ks) {
      const bf16x8 s = op_result(S[2 * ks], S[2 * ks + 1]);
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) y[ib] = mma(s, op_split<NT>(sC, 16 * ib, 32 * ks), y[ib]);
    }
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) y[ib] *= se[16 * ib + i];
    __syncthreads();
    const float et = se[63];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) S[nb] *= et;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const bf16x8 x = op_cols<64>(sx, 32 * ks, 16 * w);
#pragma unroll
      for (int ib = 2 * ks; ib < 4; ++ib) y[ib] = mma(x, op_split<64>(sP, 16 * ib, 32 * ks), y[ib]);
      const f32x4 wa = *reinterpret_cast<const f32x4*>(sw + 32 * ks + 4 * g);
      const f32x4 wb = *reinterpret_cast<const f32x4*>(sw + 32 * ks + 16 + 4 * g);
      bf16x8 hi, lo;
      split_scaled(x, wa, wb, hi, lo);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const bf16x8 b = op_cols<NT>(sB, 32 * ks, 16 * nb);
        S[nb] = mma(b, hi, S[nb]);
        S[nb] = mma(b, lo, S[nb]);
      }
    }
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) {
      const int row = 16 * ib + i;
      const u32x2 xv = *reinterpret_cast<const u32x2*>(sx + at<64>(row, p_out));
      const u32x2 o = {pk_bf16(y[ib][0] + Dh * bf_lo(xv.x), y[ib][1] + Dh * bf_hi(xv.x)),
                       pk_bf16(y[ib][2] + Dh * bf_lo(xv.y), y[ib][3] + Dh * bf_hi(xv.y))};
      if (row < rows) {
        uint16_t* dst = yb + (r0 + row) * a.y_ld + p_out;
        if (VEC || p_out + 3 < pn) {
          if (p_out < pn) *reinterpret_cast<u32x2_a2*>(dst) = o;
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (p_out + r < pn) dst[r] = (uint16_t)(o[r >> 1] >> (16 * (r & 1)));
        }
      }
    }
    if (!more) break;
    __syncthreads();
  }

  if (a.fin && pc.r1 == pc.e && p_in < pn) {
    float* dst = a.fin + slot * a.s_slot + state_at + (int64_t)p_in * a.N + 4 * g;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      if (16 * nb + 4 * g + 3 < a.N) {
        *reinterpret_cast<f32x4_a4*>(dst + 16 * nb) = S[nb];
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (16 * nb + 4 * g + r < a.N) dst[16 * nb + r] = S[nb][r];
      }
    }
  }
}

template <int NT, bool VEC>
static hipError_t launch(const ScanArgs& a, hipStream_t s) {
  const int64_t items = a.n_slots + a.q.nseq, hp = (int64_t)a.H * a.ptiles;
  if (a.seg > 0) {
    StateArgs k{};
    k.s = a;
    k.u = a.x;
    k.v = a.B;
    k.u_ld = a.x_ld;
    k.v_ld = a.B_ld;
    k.start = a.init;
    k.piece = a.piece;
    ssm_state_local_kernel<NT, VEC><<<dim3((uint32_t)(items * hp)), 256, 0, s>>>(k);
    ssm_join_kernel<NT, false><<<dim3((uint32_t)(a.q.nseq * hp * (64 * NT / 1024))), 256, 0, s>>>(k);
  }
  ssm_scan_fwd_kernel<NT, VEC><<<dim3((uint32_t)(items * hp)), 256, 0, s>>>(a);
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
