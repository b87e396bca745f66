// delta_chunk.hip -- what a chunk of 64 rows gives the delta rule's walks before any state is known.
//
// With L the prefix sums of the log decays, r the rates, k and q unit or as they are, inside one chunk and head
//   X_ij = r_i e^{L_i - L_j} k_i . k_j  (i > j),   T = (I + X)^-1,   P_ij = scale e^{L_i - L_j} q_i . k_j  (i >= j)
// the walk needs U = T (r (V - e^L K S)) and P U.  A block takes one chunk and key head: the products K K^T and Q K^T of
// the raw bf16 rows are made once, and each of its value heads decays them; row norms, steps and rates are FP32 factors
// beside the products, so nothing is rounded before T is complete.
// T: the four 16 x 16 blocks on the diagonal by substitution, a column a lane; then pairs of them, then pairs of pairs,
// [T1 0; -T2 X21 T1, T2], by FP32 matrix instructions.  The rates of the columns are taken into T, whose FP32 values are
// stored as three bf16 parts, P's as two (forward).
// A row of k, dt or b that is not finite makes the head's state and all later rows so; zeros times it would reach earlier
// rows of the chunk.  Such rows are left out here, and the record names the first.
#include "delta_device.h"

namespace cssm {

template <int NT, bool VEC, bool BWD>
__global__ __launch_bounds__(256) void delta_chunk_kernel(DeltaArgs d, char* rec_rev) {
  constexpr int LD = 68;  // rows of 64 FP32 values, 16 bytes further apart
  __shared__ __align__(16) uint16_t sK[64 * kLd<NT>];
  __shared__ __align__(16) uint16_t sQ[64 * kLd<NT>];
  __shared__ __align__(16) float sX[64 * LD];
  __shared__ __align__(16) float sT[64 * LD];
  __shared__ __align__(16) double sL[64];
  __shared__ __align__(16) float s_rate[64], s_kn[64], s_qn[64];
  __shared__ int s_bad;
  const ScanArgs& a = d.s;
  const int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15, w = wave_id();
  const uint32_t blk = xcd_block(blockIdx.x, gridDim.x);
  const int grp = blk % (uint32_t)a.G;
  const int64_t id = blk / (uint32_t)a.G;
  const Piece pc = find_chunk(a.q, id, d.n_chunk_slots);
  if (!pc.ok) return;
  const int rows = (int)(pc.r1 - pc.r0), hg = a.H / a.G;
  const int64_t gn = (int64_t)grp * a.N;
  {
    TileRegs<NT, 256> tk, tq;
    load_tile<VEC>(tk, Rows(a.B + pc.r0 * a.B_ld + gn, a.B_ld, rows, a.N, 2), (uint32_t)a.B_ld, a.N);
    load_tile<VEC>(tq, Rows(a.C + pc.r0 * a.C_ld + gn, a.C_ld, rows, a.N, 2), (uint32_t)a.C_ld, a.N);
    store_tile(sK, tk);
    store_tile(sQ, tq);
    auto norms = [&](const TileRegs<NT, 256>& t, float* to, float factor) {
#pragma unroll
      for (int k = 0; k < NT / 32; ++k) {
        const int row = (threadIdx.x + 256 * k) / (NT / 8);
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float lo = bf_lo(t.v[k][e]), hi = bf_hi(t.v[k][e]);
          s = __builtin_fmaf(lo, lo, s);
          s = __builtin_fmaf(hi, hi, s);
        }
#pragma unroll
        for (int m = NT / 16; m > 0; m >>= 1) s += __shfl_xor(s, m);
        // s - s: a NaN where the row is not finite
        const float f = (d.qk_norm ? rsqrtf(s + d.norm_eps) : 1.f) + (s - s);
        if (threadIdx.x % (NT / 8) == 0) to[row] = row < rows ? f * factor : 0.f;
      }
    };
    norms(tk, s_kn, 1.f);
    norms(tq, s_qn, d.scale);
  }
  __syncthreads();
  // score blocks (ib, jb) of this wave: rows i in the lanes, columns j in the registers
  f32x4 kk[3], qk[3];
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    int ib, jb;
    lower_block(w + 4 * t, ib, jb);
    kk[t] = qk[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (w + 4 * t < 10) {
#pragma unroll
      for (int ks = 0; ks < NT / 32; ++ks) {
        const bf16x8 kj = op_straight<NT>(sK, 16 * jb, 32 * ks, lane);
        kk[t] = mma(kj, op_straight<NT>(sK, 16 * ib, 32 * ks, lane), kk[t]);
        qk[t] = mma(kj, op_straight<NT>(sQ, 16 * ib, 32 * ks, lane), qk[t]);
      }
    }
  }
  f32x4 qkt[3];  // rows in the registers
  if constexpr (BWD) {
#pragma unroll
    for (int t = 0; t < 3; ++t) {
      int ib, jb;
      lower_block(w + 4 * t, ib, jb);
      qkt[t] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (w + 4 * t < 10) {
#pragma unroll
        for (int ks = 0; ks < NT / 32; ++ks)
          qkt[t] = mma(op_straight<NT>(sQ, 16 * ib, 32 * ks, lane), op_straight<NT>(sK, 16 * jb, 32 * ks, lane), qkt[t]);
      }
    }
  }

  for (int hh = 0; hh < hg; ++hh) {
    const int h = grp * hg + hh;
    char* rec = d.rec + (id * a.H + h) * kRecFwd;
    char* rev = BWD ? rec_rev + (id * a.H + h) * kRecRev : nullptr;
    if (w == 0) {  // lane = row
      const Rate rate(a, h);
      const float step = rate.step(raw_step(a, pc.r0, rows, lane, h), lane < rows);
      const int64_t at = (pc.r0 + lane) * d.b_ld + h;
      const float b = lane < rows ? load_num(d.b, at, a.dt_f32) : 0.f;
      float r = lane < rows ? d.beta_max / (1.f + ex2(-kLog2e * b)) : 0.f;
      float kn = s_kn[lane], qn = s_qn[lane];
      double l = rate.exponent(step);
      const bool fine = __builtin_isfinite((float)l) && __builtin_isfinite(r) && __builtin_isfinite(kn);
      const uint64_t not_fine = __ballot(!fine);
      const int bad = not_fine && !BWD ? __builtin_ctzll(not_fine) : 64;  // backward, they may reach every row
      if (lane >= bad) l = 0.0, r = kn = qn = 0.f;
      const double L = wave_prefix(l);
      const double end = __shfl(L, 63);
      sL[lane] = L;
      s_rate[lane] = r;
      if (lane == 0) s_bad = bad;
      const float grown = ex2((float)L), left = ex2((float)(end - L));
      auto factors = [&](char* to) {
        Factors* f = reinterpret_cast<Factors*>(to);
        f->f[0][lane] = grown * kn;
        f->f[1][lane] = grown * qn;
        f->f[2][lane] = left * kn;
        f->f[3][lane] = r;
        if (lane == 0) {
          f->decay = ex2((float)end);
          f->bad = bad;
        }
      };
      factors(rec + kRecFwd - kRecVec);
      if constexpr (BWD) factors(rev + kRecRev - kRecVec);
    }
    __syncthreads();
    const int bad = s_bad;
#pragma unroll
    for (int t = 0; t < 3; ++t) {
      int ib, jb;
      lower_block(w + 4 * t, ib, jb);
      if (w + 4 * t < 10) {
        const int row = 16 * ib + i, col = 16 * jb + 4 * g;
        const double Li = sL[row];
        const f32x4 knj = *reinterpret_cast<const f32x4*>(s_kn + col);
        const float kni = s_kn[row] * s_rate[row], qni = s_qn[row];
        f32x4 x, p;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float m = ex2((float)(Li - sL[col + r])) * knj[r];
          const bool in = row < bad;  // and so is every column up to the diagonal
          x[r] = in && col + r < row ? kk[t][r] * (m * kni) : 0.f;
          p[r] = in && col + r <= row ? qk[t][r] * (m * qni) : 0.f;
        }
        *reinterpret_cast<f32x4*>(sX + row * LD + col) = x;
        if constexpr (!BWD) {
          store_tri<2>(rec + kRecT, tri_block(ib, jb), p, lane);
        } else {  // column 16 jb + i in the lanes, rows in the registers
          const int c = 16 * jb + i, r0 = 16 * ib + 4 * g;
          const float knc = s_kn[c];
          f32x4 pt;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float m = ex2((float)(sL[r0 + r] - sL[c])) * knc * s_qn[r0 + r];
            pt[r] = r0 + r < bad && c <= r0 + r ? qkt[t][r] * m : 0.f;
          }
          store_tri<3>(rev + kRecT, tri_block(ib, jb), pt, lane);
        }
      }
    }
    __syncthreads();
    {  // diagonal block w: column i of its inverse; the four groups of lanes do the same
      const float* X = sX + 16 * w * LD + 16 * w;
      float t[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float v = r == i ? 1.f : 0.f;
#pragma unroll
        for (int m4 = 0; m4 < r; m4 += 4) {
          const f32x4 x = *reinterpret_cast<const f32x4*>(X + r * LD + m4);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (m4 + e < r) v = __builtin_fmaf(-x[e], t[m4 + e], v);
        }
        t[r] = v;
      }
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if ((r >> 2) == g) sT[(16 * w + r) * LD + 16 * w + i] = t[r];
    }
    __syncthreads();
    auto x_rows = [&](int ib, int jb) { return *reinterpret_cast<const f32x4*>(sX + (16 * ib + i) * LD + 16 * jb + 4 * g); };
    auto t_rows = [&](int ib, int jb) { return *reinterpret_cast<const f32x4*>(sT + (16 * ib + i) * LD + 16 * jb + 4 * g); };
    auto t_cols = [&](int ib, int jb) {  // column i in the lanes, rows in the registers
      const float* p = sT + (16 * ib + 4 * g) * LD + 16 * jb + i;
      return f32x4{p[0], p[LD], p[2 * LD], p[3 * LD]};
    };
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    if (w < 2) {
      const int lo = 2 * w, hi = lo + 1;
      const f32x4 y = mma_f32(x_rows(hi, lo), t_cols(lo, lo), zero);  // X T: rows in the registers, columns in the lanes
      *reinterpret_cast<f32x4*>(sT + (16 * hi + i) * LD + 16 * lo + 4 * g) = -mma_f32(y, t_rows(hi, hi), zero);
    }
    __syncthreads();
    {
      const int ib = 2 + (w >> 1), jb = w & 1;
      f32x4 sum = zero;
      for (int m = 2; m <= ib; ++m) {
        f32x4 y = zero;
        for (int c = jb; c < 2; ++c) y = mma_f32(x_rows(m, c), t_cols(c, jb), y);
        sum = mma_f32(y, t_rows(ib, m), sum);
      }
      *reinterpret_cast<f32x4*>(sT + (16 * ib + i) * LD + 16 * jb + 4 * g) = -sum;
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 3; ++t) {
      int ib, jb;
      lower_block(w + 4 * t, ib, jb);
      if (w + 4 * t < 10) {
        const f32x4 rate = *reinterpret_cast<const f32x4*>(s_rate + 16 * jb + 4 * g);
        store_tri<3>(rec, tri_block(ib, jb), t_rows(ib, jb) * rate, lane);
        if constexpr (BWD) store_tri<3>(rev, tri_block(ib, jb), t_cols(ib, jb), lane);
      }
    }
    __syncthreads();
  }
}

template <int NT>
static void launch(const DeltaArgs& a, char* rec_rev, bool vec, hipStream_t s) {
  const dim3 grid((uint32_t)((a.n_chunk_slots + a.s.q.nseq) * a.s.G));
  if (rec_rev) {
    if (vec) delta_chunk_kernel<NT, true, true><<<grid, 256, 0, s>>>(a, rec_rev);
    else delta_chunk_kernel<NT, false, true><<<grid, 256, 0, s>>>(a, rec_rev);
  } else {
    if (vec) delta_chunk_kernel<NT, true, false><<<grid, 256, 0, s>>>(a, nullptr);
    else delta_chunk_kernel<NT, false, false><<<grid, 256, 0, s>>>(a, nullptr);
  }
}

hipError_t launch_delta_chunks(const DeltaArgs& a, char* rec_rev, bool vec, hipStream_t s) {
  switch (state_tile(a.s.N)) {
    case 64: launch<64>(a, rec_rev, vec, s); break;
    case 128: launch<128>(a, rec_rev, vec, s); break;
    default: launch<256>(a, rec_rev, vec, s); break;
  }
  return hipGetLastError();
}

}  // namespace cssm
