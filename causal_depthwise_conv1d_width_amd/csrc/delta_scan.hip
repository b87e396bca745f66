// delta_scan.hip -- forward gated delta rule over packed rows: the walk of the states.
//
// A block walks one sequence for 64 columns of one head, a chunk of 64 rows at a time (delta_chunk.hip: L, r, T, P):
//   R = V - e^L K S^T,   U = T r R,   Y = scale e^L Q S^T + P U,   S' = e^{L_Q} S + U^T (e^{L_Q - L} K)
// Each of its 4 waves owns 16 columns p of V, U, Y and S, which depend on no other column: nothing passes between waves.
// The state's accumulators (registers n, lanes p) are, unmoved, the operand that K S^T and Q S^T contract over n, and R's
// and U's the ones that T, P and K contract over rows.  Shared memory holds K, Q, V and the chunk's record for all waves;
// the next chunk's are loaded over the current one's products.
// FP32 operands enter as three bf16 parts (K S^T, S') or, both being FP32, six products (T R), so that states keep
// FP32's precision; y takes the state, the scores and U in two: with one of the state and the scores it was up to
// 2.7e-3 off where its terms cancel (its own rounding: 1.66e-3), PCT faster.
#include "delta_device.h"

namespace cssm {

template <int NT, bool VEC>
__global__ __launch_bounds__(256, NT <= 128 ? 2 : 1) void delta_scan_fwd_kernel(DeltaArgs d) {
  constexpr int T = 256, NB = NT / 16;
  __shared__ __align__(16) uint16_t sK[64 * kLd<NT, 16>];
  __shared__ __align__(16) uint16_t sQ[64 * kLd<NT>];
  __shared__ __align__(16) uint16_t sV[64 * kLd<64, 16>];
  __shared__ __align__(16) char sR[kRecFwd];
  const ScanArgs& a = d.s;
  const Units<1> us(a, blockIdx.x);
  if (!us.ok) return;
  const Unit me(a, us, 0);
  const int w = wave_id(), pn = me.pn;
  Piece pc;
  pc.seq = us.item;
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

  const int64_t gn = (int64_t)us.group * a.N;
  TileRegs<NT, T> tK, tQ;
  TileRegs<64, T> tV;
  RecordRegs<kRecFwd, T> tR;
  auto load = [&](const Chunks<false>& c, int rows) {
    load_tile<VEC>(tK, Rows(a.B + c.c0 * a.B_ld + gn, a.B_ld, rows, a.N, 2), (uint32_t)a.B_ld, a.N);
    load_tile<VEC>(tQ, Rows(a.C + c.c0 * a.C_ld + gn, a.C_ld, rows, a.N, 2), (uint32_t)a.C_ld, a.N);
    load_tile<VEC>(tV, Rows(a.x + c.c0 * a.x_ld + me.col, a.x_ld, rows, pn, 2), (uint32_t)a.x_ld, pn);
    load_record(tR, d.rec + (chunk_id(pc, c.c0, d.n_chunk_slots) * a.H + me.h) * kRecFwd, rows > 0);
  };
  Chunks<false> c(pc.s, pc.e);
  int rows = c.rows();
  load(c, rows);
  const char* sT = sR;
  const char* sP = sR + kRecT;
  const Factors& fac = *reinterpret_cast<const Factors*>(sR + kRecFwd - kRecVec);
  for (;;) {
    lane = fresh(lane);
    g = lane >> 4, i = lane & 15;
    store_tile<16>(sK, tK);
    store_tile(sQ, tQ);
    store_tile<16>(sV, tV);
    store_record(sR, tR);
    __syncthreads();
    const Rows out(yb + c.c0 * a.y_ld, a.y_ld, rows, pn, 2);
    c = step_chunk(c, rows);  // rows == 0: that was the last one
    load(c, rows);
    phase();
    f32x4 r[4], y[4];  // rows in the registers, columns p in the lanes; y the other way round
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) r[ib] = y[ib] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < NT / 32; ++ks) {
      const Parts s = split(S[2 * ks], S[2 * ks + 1]);
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) {
        r[ib] = mma3(op_split<NT, 16>(sK, 16 * ib, 32 * ks, lane), s, r[ib]);
        const bf16x8 q = op_split<NT>(sQ, 16 * ib, 32 * ks, lane);
        y[ib] = mma(s.p[1], q, y[ib]);
        y[ib] = mma(s.p[0], q, y[ib]);
      }
      phase();
    }
    bool fine = true;
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) {
      const f32x4 f = *reinterpret_cast<const f32x4*>(fac.f[0] + 16 * ib + 4 * g);
      const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s16x4*)(sV + at<64, 16>(16 * ib + 4 * g + (i >> 2), 16 * w + 4 * (i & 3))));
      const u32x2 v = __builtin_bit_cast(u32x2, t);
      r[ib] = f32x4{bf_lo(v.x), bf_hi(v.x), bf_lo(v.y), bf_hi(v.y)} - f * r[ib];
#pragma unroll
      for (int e = 0; e < 4; ++e) fine = fine && __builtin_isfinite(r[ib][e]);
      y[ib] *= fac.f[1][16 * ib + i];
    }
    // The first row of this lane's column that is not finite: it and the later ones are left out of the products, whose
    // zeros would spread them, and put in at the end
    int bad = __builtin_amdgcn_readfirstlane(fac.bad);
    const bool any_bad = bad < 64 || __ballot(!fine) != 0;
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
#pragma unroll
      for (int ib = 0; ib < 4; ++ib)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (16 * ib + 4 * g + e >= bad) r[ib][e] = 0.f;
    }
    phase();
    f32x4 u[4];
    {
      const Parts rp[2] = {split(r[0], r[1]), split(r[2], r[3])};
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) {
        u[ib] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks <= ib / 2; ++ks) {
          const Parts t = {{tri_rows<3>(sT, ib, ks, 0, lane), tri_rows<3>(sT, ib, ks, 1, lane), tri_rows<3>(sT, ib, ks, 2, lane)}};
          u[ib] = mma6(t, rp[ks], u[ib]);
        }
        phase();
      }
    }
    const float decay = fac.decay;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) S[nb] *= decay;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      {
        const Parts up = split(u[2 * ks], u[2 * ks + 1]);
#pragma unroll
        for (int ib = 2 * ks; ib < 4; ++ib) {
          const bf16x8 p = tri_rows<2>(sP, ib, ks, 0, lane);
          y[ib] = mma(up.p[0], tri_rows<2>(sP, ib, ks, 1, lane), y[ib]);
          y[ib] = mma(up.p[1], p, y[ib]);
          y[ib] = mma(up.p[0], p, y[ib]);
        }
      }
      const f32x4 wa = *reinterpret_cast<const f32x4*>(fac.f[2] + 32 * ks + 4 * g);
      const f32x4 wb = *reinterpret_cast<const f32x4*>(fac.f[2] + 32 * ks + 16 + 4 * g);
      const Parts us_ = split(u[2 * ks] * wa, u[2 * ks + 1] * wb);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) S[nb] = mma3(op_cols<NT, 16>(sK, 32 * ks, 16 * nb, lane), us_, S[nb]);
      phase();
    }
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
  if (a.fin && p_in < pn) store_state(S, a.fin + slot * a.s_slot + state_at + (int64_t)p_in * a.N, a.N, lane >> 4);
}

template <int NT>
static void launch(const DeltaArgs& a, bool vec, hipStream_t s) {
  const dim3 grid((uint32_t)unit_blocks(a.s.q.nseq, a.s.H, a.s.G, a.s.ptiles, 1));
  if (vec) delta_scan_fwd_kernel<NT, true><<<grid, 256, 0, s>>>(a);
  else delta_scan_fwd_kernel<NT, false><<<grid, 256, 0, s>>>(a);
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
