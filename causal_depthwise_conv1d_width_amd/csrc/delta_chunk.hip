// delta_chunk.hip -- what a chunk of 64 rows gives the delta rule's walks before any state is known.
//
// With L the prefix sums of the log decays, r the rates, k and q unit or as they are, inside one chunk and head
//   X_ij = r_i e^{L_i - L_j} k_i . k_j  (i > j),   T = (I + X)^-1,   P_ij = scale e^{L_i - L_j} q_i . k_j  (i >= j)
// the walk needs U = T (r (V - e^L K S)) and P U.  A block takes one chunk and key head.  Rows of k and q go into fp16 tiles,
// times a power of two that is exact; the products K K^T and Q K^T are made once, and each of the value heads decays
// them.  Norms, steps and rates are FP32 factors beside the products, so nothing is rounded before T is complete.
// T: the four 16 x 16 blocks on the diagonal by substitution, a column a lane; then pairs of them, then pairs of pairs,
// [T1 0; -T2 X21 T1, T2], by FP32 matrix instructions.
// A row of k, dt or b that is not finite makes the head's state and all later rows so; zeros times it would reach earlier
// rows of the chunk.  Forward, such rows are left out here, and the record names the first.
#include "delta_device.h"

namespace cssm {

// the largest of 8 bf16 magnitudes, as bf16 bits (an infinity or NaN is larger than all numbers)
__device__ __forceinline__ uint32_t max_bits(u32x4 v) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t lo = v[e] & 0x7fffu, hi = v[e] >> 16 & 0x7fffu;
    m = m > lo ? m : lo;
    m = m > hi ? m : hi;
  }
  return m;
}

// The sequences from long to short (by chunks, 255 and more alike; which of equal ones comes first makes no difference to
// any result): a walk lasts as long as its sequence, and one that began last would keep the others waiting.  64 mixed
// prompts (longest 4000 of 32512 rows) take 800 us forward, 865 to 925 in the order of their rows.
__device__ __forceinline__ void order_sequences(const Seqs& q, int32_t* order) {
  __shared__ uint32_t s_at[256];
  s_at[threadIdx.x] = 0;
  __syncthreads();
  auto key = [&](int64_t i) {
    int64_t s = q.cu[i], e = q.cu[i + 1];
    s = s < 0 ? 0 : s, e = e > q.rows ? q.rows : e;
    const int64_t chunks = e > s ? (e - s + kChunk - 1) / kChunk : 0;
    return 255 - (int)(chunks < 255 ? chunks : 255);
  };
  for (int64_t i = threadIdx.x; i < q.nseq; i += 256) atomicAdd(&s_at[key(i)], 1u);
  __syncthreads();
  uint32_t before = 0;
  for (int k = 0; k < (int)threadIdx.x; ++k) before += s_at[k];
  __syncthreads();
  s_at[threadIdx.x] = before;
  __syncthreads();
  for (int64_t i = threadIdx.x; i < q.nseq; i += 256) order[atomicAdd(&s_at[key(i)], 1u)] = (int32_t)i;
}

template <int NT, bool VEC, bool BWD>
__global__ __launch_bounds__(256, NT <= 128 ? 3 : 2) void delta_chunk_kernel(DeltaArgs d, char* rec_rev) {
  constexpr int LD = 68;  // rows of 64 FP32 values, 16 bytes further apart
  // the tiles of k and q until their products are made, then X and T
  constexpr int kTiles = 2 * (int)key_tile(NT), kSystems = 2 * 64 * LD * 4;
  __shared__ __align__(16) char sAll[kTiles > kSystems ? kTiles : kSystems];
  uint16_t *sK = reinterpret_cast<uint16_t*>(sAll), *sQ = sK + key_tile(NT) / 2;
  float *sX = reinterpret_cast<float*>(sAll), *sT = sX + 64 * LD;
  __shared__ __align__(16) double sL_[4][64];  // of four heads
  __shared__ __align__(16) float s_rate_[4][64], s_kn[64], s_qn[64], s_max[4];
  __shared__ int s_bad_[4];
  const ScanArgs& a = d.s;
  int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15;
  const int w = wave_id();
  if (blockIdx.x + 1 == gridDim.x) {
    if (d.order) order_sequences(a.q, d.order);
    return;
  }
  const uint32_t blk = xcd_block(blockIdx.x, gridDim.x - 1);
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
    char* keys = d.keys + (id * a.G + grp) * 2 * key_tile(NT);
    auto convert = [&](const TileRegs<NT, 256>& t, uint16_t* lds, char* to, float* norm, float factor) {
#pragma unroll
      for (int k = 0; k < NT / 32; ++k) {
        const int q = fresh((int)threadIdx.x) + 256 * k, row = q / (NT / 8), c = q % (NT / 8) * 8;
        uint32_t m = max_bits(t.v[k]);
        m = row_lanes<NT / 8>(m, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
        uint32_t e = m >> 7;  // the largest one's exponent
        e = e < 1 ? 1 : (e > 253 ? 253 : e);
        const float up = __uint_as_float((254 - e) << 23), down = __uint_as_float(e << 23);
        float s = 0.f;
        u32x4 h;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float lo = bf_lo(t.v[k][x]) * up, hi = bf_hi(t.v[k][x]) * up;
          s = __builtin_fmaf(lo, lo, s);
          s = __builtin_fmaf(hi, hi, s);
          h[x] = pk_f16(lo, hi);
        }
        s = __uint_as_float(row_lanes<NT / 8>(__float_as_uint(s), [](uint32_t a, uint32_t b) {
          return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
        }));
        *reinterpret_cast<u32x4*>(lds + key_at<NT>(row, c)) = h;
        *reinterpret_cast<u32x4*>(to + key_at<NT>(row, c) * 2) = h;
        // s - s: a NaN where the row is not finite
        const float f = (d.qk_norm ? rsqrtf(s + (d.norm_eps > 0.f ? d.norm_eps * up * up : 0.f)) : down) + (s - s);
        if (c == 0) norm[row] = row < rows ? f * factor : 0.f;
        phase();
      }
    };
    convert(tk, sK, keys, s_kn, 1.f);
    convert(tq, sQ, keys + key_tile(NT), s_qn, d.scale);
  }
  __syncthreads();
  // score blocks (ib, jb) of this wave: rows i in the lanes, columns j in the registers (qkt: the other way round)
  f32x4 kk[3], qk[3];
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    int ib, jb;
    lower_block(w + 4 * t, ib, jb);
    kk[t] = qk[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (w + 4 * t < 10) {
#pragma unroll
      for (int ks = 0; ks < NT / 32; ++ks) {
        const f16x8 kj = key_rows<NT>(sK, 16 * jb, 32 * ks, lane);
        const f16x8 qi = key_rows<NT>(sQ, 16 * ib, 32 * ks, lane);
        kk[t] = mmah(kj, key_rows<NT>(sK, 16 * ib, 32 * ks, lane), kk[t]);
        qk[t] = BWD ? mmah(qi, kj, qk[t]) : mmah(kj, qi, qk[t]);
        phase();
      }
    }
  }

  for (int hh = 0; hh < hg; ++hh) {
    lane = fresh(lane);
    g = lane >> 4, i = lane & 15;
    const int h = grp * hg + hh, at4 = hh & 3;
    char* rec = d.rec + (id * a.H + h) * kRecFwd;
    char* rev = BWD ? rec_rev + (id * a.H + h) * kRecRev : nullptr;
    if (at4 == 0) {  // the gates of the next four heads, one a wave; lane = row
      if (hh > 0) __syncthreads();  // the last four are read
      if (hh + w < hg) {
        const int hw = h + w;
        const Rate rate(a, hw);
        const float step = rate.step(raw_step(a, pc.r0, rows, lane, hw), lane < rows);
        const float b = lane < rows ? load_num(d.b, (pc.r0 + lane) * d.b_ld + hw, a.dt_f32) : 0.f;
        float r = lane < rows ? d.beta_max / (1.f + ex2(-kLog2e * b)) : 0.f;
        float kn = s_kn[lane], qn = s_qn[lane];
        double l = rate.exponent(step);
        const bool fine = __builtin_isfinite((float)l) && __builtin_isfinite(r) && __builtin_isfinite(kn);
        const uint64_t not_fine = __ballot(!fine);
        const int bad = not_fine && !BWD ? __builtin_ctzll(not_fine) : 64;  // backward, they may reach every row
        if (lane >= bad) l = 0.0, r = kn = qn = 0.f;
        const double L = wave_prefix(l);
        const double end = __shfl(L, 63);
        sL_[w][lane] = L;
        s_rate_[w][lane] = r;
        if (lane == 0) s_bad_[w] = bad;
        const float up = ex2((float)L), left = ex2((float)(end - L));
        auto factors = [&](char* to) {
          Factors* f = reinterpret_cast<Factors*>(to);
          f->in[lane] = up * kn;
          f->read[lane] = up * qn;
          f->out[lane] = left * kn;
          f->rate[lane] = r;
          if (lane == 0) {
            f->decay = ex2((float)end);
            f->bad = bad;
          }
        };
        factors(rec + w * kRecFwd + kRecFwd - kRecVec);
        if constexpr (BWD) factors(rev + w * kRecRev + kRecRev - kRecVec);
      }
      __syncthreads();
    }
    const double* sL = sL_[at4];
    const float* s_rate = s_rate_[at4];
    const int bad = s_bad_[at4];
#pragma unroll
    for (int t = 0; t < 3; ++t) {
        lane = fresh(lane);
      g = lane >> 4, i = lane & 15;
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
          x[r] = row < bad && col + r < row ? kk[t][r] * (m * kni) : 0.f;
          p[r] = row < bad && col + r <= row ? qk[t][r] * (m * qni) : 0.f;
        }
        *reinterpret_cast<f32x4*>(sX + row * LD + col) = x;
        if constexpr (!BWD) {
          store_tri<2>(rec + kRecT, tri_block(ib, jb), p, lane);
        } else {  // column 16 jb + i in the lanes, rows in the registers
          const int c = 16 * jb + i, r0 = 16 * ib + 4 * g;
          const double Lc = sL[c];
          const float knc = s_kn[c];
#pragma unroll
          for (int r = 0; r < 4; ++r)
            p[r] = c <= r0 + r ? qk[t][r] * (ex2((float)(sL[r0 + r] - Lc)) * knc * s_qn[r0 + r]) : 0.f;
          store_tri<3>(rev + kRecT, tri_block(ib, jb), p, lane);
        }
      }
    }
    __syncthreads();
    lane = fresh(lane);
    g = lane >> 4, i = lane & 15;
    {  // diagonal block w: column i of its inverse; the four groups of lanes do the same
      const float* X = sX + 16 * w * LD + 16 * w;
      float t[16];
      f32x4 x[2][4];  // a row of X, and the next one on its way
      x[1][0] = *reinterpret_cast<const f32x4*>(X + LD);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
#pragma unroll
        for (int m4 = 0; m4 <= r; m4 += 4)
          if (r < 15) x[(r + 1) & 1][m4 / 4] = *reinterpret_cast<const f32x4*>(X + (r + 1) * LD + m4);
        float v = r == i ? 1.f : 0.f;
#pragma unroll
        for (int m = 0; m < r; ++m) v = __builtin_fmaf(-x[r & 1][m / 4][m % 4], t[m], v);
        t[r] = v;
        phase();
      }
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if ((r >> 2) == g) sT[(16 * w + r) * LD + 16 * w + i] = t[r];
    }
    __syncthreads();
    lane = fresh(lane);
    g = lane >> 4, i = lane & 15;
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
      // the largest of T: its blocks of level two are here, the others in shared memory
      float m = max4(max4(0.f, sum), t_rows(w, w));
      if (w < 2) m = max4(m, t_rows(2 * w + 1, 2 * w));
      m = max_across16(m);
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) m = __builtin_fmaxf(m, __shfl_xor(m, x));
      if (lane == 0) s_max[w] = m;
    }
    __syncthreads();
    const Pow2 scale = bring_to<10>(__builtin_fmaxf(__builtin_fmaxf(s_max[0], s_max[1]), __builtin_fmaxf(s_max[2], s_max[3])));
    if (threadIdx.x == 0) {
      reinterpret_cast<Factors*>(rec + kRecFwd - kRecVec)->t_scale = scale.down;
      if constexpr (BWD) reinterpret_cast<Factors*>(rev + kRecRev - kRecVec)->t_scale = scale.down;
    }
    lane = fresh(lane);
    g = lane >> 4, i = lane & 15;
#pragma unroll
    for (int t = 0; t < 3; ++t) {
      int ib, jb;
      lower_block(w + 4 * t, ib, jb);
      if (w + 4 * t < 10) {
        store_halves(rec, tri_block(ib, jb), t_rows(ib, jb) * scale.up, lane);
        if constexpr (BWD) store_halves(rev, tri_block(ib, jb), t_cols(ib, jb) * scale.up, lane);
      }
    }
  }
}

template <int NT>
static void launch(const DeltaArgs& a, char* rec_rev, bool vec, hipStream_t s) {
  const dim3 grid((uint32_t)((a.n_chunk_slots + a.s.q.nseq) * a.s.G + 1));  // the last block orders the sequences
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
