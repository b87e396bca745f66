// ssm_scan_bwd.hip -- backward of the selective state space scan.
//
// For a chunk of 64 rows of one sequence and one head, with S the state before the chunk, T the adjoint
// of the state after it, L the prefix sums of l_t = dt_t A, M_ij = e^{L_i - L_j} (i >= j), and
//   G = C B^T,  W = dY X^T,  Z_ij = M_ij dt_j W_ij,  K_ij = G_ij M_ij W_ij:
//   dC_i = sum over heads of  e^{L_i} S^T dy_i + sum_j Z_ij B_j
//   dB_j = sum over heads of  dt_j e^{L_Q - L_j} T^T x_j + sum_i Z_ij C_i
//   dx_j = dt_j (e^{L_Q - L_j} T B_j + sum_i G_ij M_ij dy_i) + D dy_j
//   dl_t = e^{L_Q} <T, S> + sum_{i >= t} e^{L_i} dy_i . S C_i + sum_{j < t} dt_j e^{L_Q - L_j} x_j . T B_j
//          + sum_{i >= t > j} dt_j K_ij
//   d(dt_t) = A dl_t + e^{L_Q - L_t} x_t . T B_t + sum_i K_it
// The first kernel walks the states forward and the adjoints in reverse and stores both at every chunk;
// then every chunk is independent: a block takes one chunk and the heads of one group (or a part of
// them), keeps dB and dC in registers over its heads, and sums nothing through memory.  S and T are stored as
// FP32, already in matrix-operand order, and enter their products as three bf16 parts: the row sums that feed
// d(dt) and dA share the products of dC and dB and keep FP32's precision (packed sequences: d(dt) 1.7e-7 off and
// dA 2e-7; with two parts 1e-6 and 1.4e-6 in 2% less time; with states kept in 16 bits of two bf16 planes 1.4e-6 and
// 3.4e-6 in 9% less).  dx, rounded to bf16 in the end, takes the first part of T alone; Z and G M are rounded
// to bf16 once, as operands.
// The stored states and adjoints have a sign that turns from chunk to chunk (ssm_state.h).
#include <type_traits>

#include "ssm_state.h"

namespace cssm {

template <int NT, int U, bool VEC, bool STORE>
__global__ __launch_bounds__(128 * U, U > 2 || NT <= 128 ? 2 : 1) void ssm_states_kernel(StateArgs f, StateArgs r) {
  __shared__ StateShared<NT, U> sh;
  if (blockIdx.y == 0) state_walk<NT, U, 3, VEC, false, STORE, true>(f, sh);
  else state_walk<NT, U, 3, VEC, true, STORE, true>(r, sh);
}

// sum over the four rows of 16 lanes, in every lane: swapping the odd rows of a copy with the even rows of
// another puts the rows' neighbours side by side, and the same for halves
__device__ __forceinline__ float across16(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t x = __float_as_uint(__uint_as_float(p[0]) + __uint_as_float(p[1]));
  const auto q = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

constexpr int kThreads = 256;

// A block of 4 waves takes a chunk and walks the 64-column units of its heads.  A wave owns a quarter of the
// columns n of dB and dC, and 16 columns of dX.  Two blocks share a CU (with the 256-column state tile, one), so that
// one's loads from shared memory run beside the other's products: 8 waves in one block go through the phases
// together, and took a tenth longer.  16384 rows, 64 heads of 64 columns, N = 128: 590 us, in which it reads 1.5 GB
// (2.5 TB/s, the states two thirds of them) and 9 products a head are made; the states' walks take 290 us, a
// store of 1.07 GB at 3.7 TB/s.  C B^T is made anew for every head: kept, its 12 registers spill, and the kernel
// takes a fifth longer.
template <int NT, bool VEC>
__global__ __launch_bounds__(kThreads, NT > 128 ? 1 : 2) void ssm_scan_bwd_kernel(ScanBwdArgs b) {
  constexpr int NBW = NT / 64;  // 16-column blocks n of a wave
  constexpr int KB = 4;         // 16-row blocks
  constexpr int R = (NT > 128 ? NT : 128) * kLd<64>;
  __shared__ __align__(16) uint16_t sx[64 * kLd<64>];
  __shared__ __align__(16) uint16_t sy[64 * kLd<64>];
  __shared__ __align__(16) uint16_t sB[64 * kLd<NT>];
  __shared__ __align__(16) uint16_t sC[64 * kLd<NT>];
  __shared__ __align__(16) uint16_t sR[R];  // T^T [n][p], then Z and G M [i][j]
  // three heads': the last one's gradients are put together while the next one's decays are made
  __shared__ __align__(16) double sdecay[2][64];
  __shared__ __align__(16) float ssteps[3][3][64];
  __shared__ __align__(16) float s_col[2][4][64];
  __shared__ float s_row[2][4][64], s_diag[2][64], s_trace[2][4], s_rint[4][64], s_u[4][64], s_dot[4];
  uint16_t *sZ = sR, *sG = sR + 64 * kLd<64>;
  const ScanArgs& a = b.s;
  int lane = threadIdx.x & 63;
  const int w = wave_id();
  const uint32_t blk = xcd_block(blockIdx.x, gridDim.x);
  const int part = blk % b.hsplit, grp = blk / b.hsplit % a.G;
  const int64_t id = blk / b.hsplit / a.G;
  const int hg = a.H / a.G, per = (hg + b.hsplit - 1) / b.hsplit;
  const int h_lo = grp * hg + part * per, h_hi = h_lo + per < (grp + 1) * hg ? h_lo + per : (grp + 1) * hg;
  const Piece pc = find_chunk(a.q, id, b.n_chunk_slots);
  if (!pc.ok) {
    for (int e = threadIdx.x; e < (h_hi - h_lo) * 3; e += kThreads) b.head_part[(id * a.H + h_lo) * 3 + e] = 0.f;
    return;
  }
  const int rows = (int)(pc.r1 - pc.r0);
  // the signs of the stored states and adjoints, taken into the decays beside them
  int64_t w0, w1;
  piece_around(pc.s, pc.e, pc.r0, a.seg, w0, w1);
  const float turn_s = turn_of((pc.r0 >> 6) - (w0 >> 6)), turn_t = turn_of(((w1 - 1) >> 6) - (pc.r0 >> 6));
  const int hp = a.H * a.ptiles;
  const int tiles = (h_hi - h_lo) * a.ptiles;
  const int64_t gn = (int64_t)grp * a.N;
  const int nw = 16 * NBW * w;  // this wave's first column n
  const int pw = 16 * w;        // and of dX

  f32x4 dC[NBW][KB], dB[NBW][KB];
#pragma unroll
  for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
    for (int k = 0; k < KB; ++k) dC[nb][k] = dB[nb][k] = f32x4{0.f, 0.f, 0.f, 0.f};

  TileRegs<64, kThreads> tx, ty;
  f32x4 S[NBW][2][2], T[NBW][2][2];  // [n block][p step of 32][half of it]
  auto load_rows = [&](int t) {
    const int h = h_lo + t / a.ptiles, p_first = t % a.ptiles * kPTile;
    const int pn = a.P - p_first < kPTile ? a.P - p_first : kPTile;
    const int64_t o = (int64_t)h * a.P + p_first;
    const int n = t < tiles ? rows : 0;  // past the last one nothing is read
    load_tile<VEC>(tx, Rows(a.x + pc.r0 * a.x_ld + o, a.x_ld, n, pn, 2), (uint32_t)a.x_ld, pn);
    load_tile<VEC>(ty, Rows(b.dy + pc.r0 * b.dy_ld + o, b.dy_ld, n, pn, 2), (uint32_t)b.dy_ld, pn);
  };
  // a head's decays into its buffer, by wave 3 (waves 0 and 1 have three score blocks, these two): prefix sums,
  // steps and powers, and the decays to the chunk's end, summed from there
  RawStep raw{};
  auto load_raw = [&](int t) { raw = raw_step(a, pc.r0, t < tiles ? rows : 0, lane, h_lo + (uint32_t)t / (uint32_t)a.ptiles); };
  auto decays = [&](int t) {
    const Rate rate(a, h_lo + (uint32_t)t / (uint32_t)a.ptiles);
    const float d = rate.step(raw, lane < rows);
    const double l = rate.exponent(d), L = wave_prefix(l);
    const double back = wave_prefix(__shfl(l, 63 - lane));
    sdecay[t & 1][lane] = L;
    ssteps[t % 3][0][lane] = d;
    ssteps[t % 3][1][lane] = turn_s * ex2((float)L);
    ssteps[t % 3][2][63 - lane] = turn_t * ex2((float)dpp0<0x138, 0xf>(back));  // the rows after this one
  };
  // one of the chunk's states of head t
  auto load_states = [&](int t, const float* from, f32x4(&v)[NBW][2][2]) {
    const int n = t < tiles ? 64 * NT : 0;
    const Rows r(from + (id * hp + h_lo * a.ptiles + t) * (64 * NT), n, 1, n, 4);
#pragma unroll
    for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          v[nb][ks][q] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
              r.r, ((q * (NT / 16) + nw / 16 + nb) * 2 + ks) * 1024 + lane * 16, 0, 0));
  };
  load_rows(0);
  load_states(0, b.ct, T);
  load_states(0, b.cs, S);
  load_raw(0);
  if (w == 3) decays(0);
  load_raw(1);
  {
    TileRegs<NT, kThreads> t;
    load_tile<VEC>(t, Rows(a.B + pc.r0 * a.B_ld + gn, a.B_ld, rows, a.N, 2), (uint32_t)a.B_ld, a.N);
    store_tile(sB, t);
    load_tile<VEC>(t, Rows(a.C + pc.r0 * a.C_ld + gn, a.C_ld, rows, a.N, 2), (uint32_t)a.C_ld, a.N);
    store_tile(sC, t);
  }
  __syncthreads();
  float dl_sum = 0.f, q_sum = 0.f, trace_sum = 0.f;  // wave 2: over a head's column tiles
  // lane = row: the gradients of head t's decays and steps, by wave 2
  auto finish = [&](const int t) {
    const int h = h_lo + t / a.ptiles, ptile = t % a.ptiles;
    const float *sd = ssteps[t % 3][0], *se = ssteps[t % 3][1];
    const float d = sd[lane];
    float rint = 0.f, u = 0.f, col = 0.f, dots = 0.f, trace = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      dots += s_dot[k];
      rint += s_rint[k][lane];
      u += s_u[k][lane];
      trace += s_trace[t & 1][k];
    }
    // dl of row r takes K_ij d_j of all i >= r > j.  Differences of rows' and columns' sums would lose it in
    // what cancels; by blocks of 16, with r in block m: rows i >= r of the blocks left of the diagonal's, columns j < r
    // of those below it, all of the blocks below and left of it, and the diagonal's own sum as the scores left it
    const int m = lane >> 4;
    float left = 0.f, below = 0.f, on = 0.f, corner[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float r = s_row[t & 1][k][lane], c = s_col[t & 1][k][lane];
      left += k < m ? r : 0.f;
      below += k > m ? d * c : 0.f;
      on += k == m ? r : 0.f;
      col += k >= m ? c : 0.f;
      if (k == 0) corner[0] = m >= 2 ? r : 0.f;
      if (k <= 1) corner[1] += m == 3 ? r : 0.f;
    }
    const float corner1 = wave_sum(corner[0]), corner2 = wave_sum(corner[1]);
    const float rows_on = row16_suffix(left);  // rows >= this one
    const float columns = dpp0<0x111, 0xf>(row16_sum(below));
    const float inside = rows_on + on + columns + (m == 1 ? corner1 : m == 2 ? corner2 : 0.f);
    const float suffix = __shfl(wave_prefix(__shfl(rint, 63 - lane)), 63 - lane) + inside;  // rows >= this one
    const float before = dpp0<0x138, 0xf>(wave_prefix(d * u));                              // rows < this one
    dl_sum += turn_t * se[63] * dots + suffix + before;  // both signs: one is se's
    q_sum += col + s_diag[t & 1][lane] + u;
    trace_sum += trace;
    if (ptile + 1 == a.ptiles) {
      const float step = a.A[h] * dl_sum + q_sum;
      const float grad = a.softplus ? step * -expm1f(-d) : step;  // softplus' = 1 - e^{-softplus}
      const int size = a.dt_f32 ? 4 : 2;
      const Rows to(static_cast<char*>(b.ddt) + (pc.r0 * b.ddt_ld + h) * size, b.ddt_ld, rows, 1, size);
      const int off = (int)((uint32_t)lane * (uint32_t)b.ddt_ld * size);
      if (a.dt_f32) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(grad), to.r, off, 0, 0);
      else __builtin_amdgcn_raw_buffer_store_b16(to_bf16(grad), to.r, off, 0, 0);
      const float sum_A = wave_sum(lane < rows ? d * dl_sum : 0.f), sum_b = wave_sum(lane < rows ? grad : 0.f);
      if (lane == 0) {
        float* dst = b.head_part + (id * a.H + h) * 3;
        dst[0] = sum_A;
        dst[1] = sum_b;
        dst[2] = trace_sum;
      }
      dl_sum = q_sum = trace_sum = 0.f;
    }
  };
  for (int t = 0; t < tiles; ++t) {
    lane = fresh(lane);
    const int g = lane >> 4, i = lane & 15;
    const int h = h_lo + t / a.ptiles, ptile = t % a.ptiles, p_first = ptile * kPTile;
    const int pn = a.P - p_first < kPTile ? a.P - p_first : kPTile;
    const double* sL = sdecay[t & 1];
    const float *sd = ssteps[t % 3][0], *se = ssteps[t % 3][1], *sr = ssteps[t % 3][2];
    store_tile(sx, tx);
    store_tile(sy, ty);
#pragma unroll
    for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const int n = nw + 16 * nb + i;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const f32x4 v = T[nb][ks][q];
          *reinterpret_cast<u32x2*>(sR + at<64>(n, 32 * ks + 16 * q + 4 * g)) = u32x2{pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])};
        }
      }
    phase();
    __syncthreads();
    load_rows(t + 1);
    phase();

    f32x4 dX[4];  // registers p = pw + 4 g + r, lanes j
#pragma unroll
    for (int k = 0; k < 4; ++k) dX[k] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < NT / 32; ++ks) {
      const bf16x8 tt = op_cols<64>(sR, 32 * ks, pw, lane);
#pragma unroll
      for (int k = 0; k < 4; ++k) dX[k] = mma(tt, op_split<NT>(sB, 16 * k, 32 * ks, lane), dX[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) dX[k] *= sr[16 * k + i];
    phase();
    __syncthreads();

    // score block (ib, jb), G its C B^T.  s_row: a row's sum of K_ij d_j, on the diagonal row r's of all i >= r > j of
    // the block.  The diagonal's own K is kept out of both sums.
    auto scores = [&](const int ib, const int jb) {
      f32x4 G = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < NT / 32; ++ks) G = mma(op_straight<NT>(sB, 16 * jb, 32 * ks, lane), op_straight<NT>(sC, 16 * ib, 32 * ks, lane), G);
      f32x4 W = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) W = mma(op_straight<64>(sx, 16 * jb, 32 * ks, lane), op_straight<64>(sy, 16 * ib, 32 * ks, lane), W);
      const double Li = sL[16 * ib + i];
      const f32x4 dj = *reinterpret_cast<const f32x4*>(sd + 16 * jb + 4 * g);
      f32x4 z, gm;
      float row = 0.f, on_diagonal = 0.f, trace = 0.f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float m = 16 * jb + 4 * g + r <= 16 * ib + i ? ex2((float)(Li - sL[16 * jb + 4 * g + r])) : 0.f;
        gm[r] = G[r] * m;
        z[r] = W[r] * (m * dj[r]);
        float K = gm[r] * W[r];
        const bool here = 16 * jb + 4 * g + r == 16 * ib + i;
        on_diagonal = here ? K : on_diagonal;
        trace += here ? W[r] : 0.f;
        K = here ? 0.f : K;
        const float from = row16_suffix(K);  // rows >= i of column j
        if (i == 0) s_col[t & 1][ib][16 * jb + 4 * g + r] = from;
        row = __builtin_fmaf(dj[r], ib != jb ? K : (4 * g + r < i ? from : 0.f), row);
      }
      *reinterpret_cast<u32x2*>(sZ + at<64>(16 * ib + i, 16 * jb + 4 * g)) = u32x2{pk_bf16(z[0], z[1]), pk_bf16(z[2], z[3])};
      *reinterpret_cast<u32x2*>(sG + at<64>(16 * ib + i, 16 * jb + 4 * g)) = u32x2{pk_bf16(gm[0], gm[1]), pk_bf16(gm[2], gm[3])};
      row = across16(row);
      if (g == 0) s_row[t & 1][jb][16 * ib + i] = row;
      if (ib == jb) {
        if ((i >> 2) == g) s_diag[t & 1][16 * ib + i] = on_diagonal;
        trace = wave_sum(trace);
        if (lane == 0) s_trace[t & 1][ib] = trace;
      }
      phase();
    };
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      int ib, jb;
      lower_block(w + 4 * k, ib, jb);
      if (w + 4 * k < 10) scores(ib, jb);
    }
    if (w < 2) {  // blocks (0, 1), (2, 3): products over 32 columns read them
      *reinterpret_cast<u32x2*>(sZ + at<64>(32 * w + i, 32 * w + 16 + 4 * g)) = u32x2{0u, 0u};
      *reinterpret_cast<u32x2*>(sG + at<64>(32 * w + i, 32 * w + 16 + 4 * g)) = u32x2{0u, 0u};
    } else if (w == 2) {
      if (t > 0) finish(t - 1);
    } else if (t + 1 < tiles) {
      decays(t + 1);
    }
    load_raw(t + 2);
    phase();
    __syncthreads();

    float dot = 0.f;
#pragma unroll
    for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) dot = __builtin_fmaf(S[nb][ks][q][e], T[nb][ks][q][e], dot);
    dot = wave_sum(dot);
    if (lane == 0) s_dot[w] = dot;
    phase();
    // dC and the rows' sums with S
    float rint[KB] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int nb = 0; nb < NBW; ++nb) {
      f32x4 p[KB];
#pragma unroll
      for (int ib = 0; ib < KB; ++ib) p[ib] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const Parts sp = split(S[nb][ks][0], S[nb][ks][1]);
#pragma unroll
        for (int ib = 0; ib < KB; ++ib) {
          const bf16x8 y = op_split<64>(sy, 16 * ib, 32 * ks, lane);
#pragma unroll
          for (int q = 0; q < 3; ++q) p[ib] = mma(sp.p[q], y, p[ib]);
        }
        phase();
      }
#pragma unroll
      for (int ib = 0; ib < KB; ++ib) {
        f32x4 v = p[ib];
        v *= se[16 * ib + i];
        const u32x2 c = *reinterpret_cast<const u32x2*>(sC + at<NT>(16 * ib + i, nw + 16 * nb + 4 * g));
        rint[ib] += v[0] * bf_lo(c.x) + v[1] * bf_hi(c.x) + v[2] * bf_lo(c.y) + v[3] * bf_hi(c.y);
        f32x4 acc = dC[nb][ib] + v;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          if (ks <= ib / 2) acc = mma(op_cols<NT>(sB, 32 * ks, nw + 16 * nb, lane), op_split<64>(sZ, 16 * ib, 32 * ks, lane), acc);
        dC[nb][ib] = acc;
        phase();
      }
    }
#pragma unroll
    for (int ib = 0; ib < KB; ++ib) {
      const float v = across16(rint[ib]);
      if (g == 0) s_rint[w][16 * ib + i] = v;
    }
    phase();
    load_states(t + 1, b.cs, S);
    phase();
    // dB and the rows' sums with T
    float u[KB] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int nb = 0; nb < NBW; ++nb) {
      f32x4 p[KB];
#pragma unroll
      for (int jb = 0; jb < KB; ++jb) p[jb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const Parts tp = split(T[nb][ks][0], T[nb][ks][1]);
#pragma unroll
        for (int jb = 0; jb < KB; ++jb) {
          const bf16x8 x = op_split<64>(sx, 16 * jb, 32 * ks, lane);
#pragma unroll
          for (int q = 0; q < 3; ++q) p[jb] = mma(tp.p[q], x, p[jb]);
        }
        phase();
      }
#pragma unroll
      for (int jb = 0; jb < KB; ++jb) {
        f32x4 v = p[jb];
        v *= sr[16 * jb + i];
        const u32x2 c = *reinterpret_cast<const u32x2*>(sB + at<NT>(16 * jb + i, nw + 16 * nb + 4 * g));
        u[jb] += v[0] * bf_lo(c.x) + v[1] * bf_hi(c.x) + v[2] * bf_lo(c.y) + v[3] * bf_hi(c.y);
        f32x4 acc = dB[nb][jb] + v * sd[16 * jb + i];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          if (ks >= jb / 2) acc = mma(op_cols<NT>(sC, 32 * ks, nw + 16 * nb, lane), op_cols<64>(sZ, 32 * ks, 16 * jb, lane), acc);
        dB[nb][jb] = acc;
        phase();
      }
    }
#pragma unroll
    for (int jb = 0; jb < KB; ++jb) {
      const float v = across16(u[jb]);
      if (g == 0) s_u[w][16 * jb + i] = v;
    }
    load_states(t + 1, b.ct, T);
    phase();

#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const bf16x8 y = op_cols<64>(sy, 32 * ks, pw, lane);
#pragma unroll
      for (int k = 0; k < 2 * ks + 2; ++k) dX[k] = mma(y, op_cols<64>(sG, 32 * ks, 16 * k, lane), dX[k]);
    }
    const int p_out = pw + 4 * g;
    const Rows out(b.dx + pc.r0 * b.dx_ld + (int64_t)h * a.P + p_first, b.dx_ld, rows, pn, 2);
    const float Dh = a.D ? uniform(a.D[h]) : 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = 16 * k + i;
      const float d = sd[row];
      const u32x2 yv = *reinterpret_cast<const u32x2*>(sy + at<64>(row, p_out));
      const u32x2 o = {pk_bf16(d * dX[k][0] + Dh * bf_lo(yv.x), d * dX[k][1] + Dh * bf_hi(yv.x)),
                       pk_bf16(d * dX[k][2] + Dh * bf_lo(yv.y), d * dX[k][3] + Dh * bf_hi(yv.y))};
      store4<VEC>(out, (uint32_t)b.dx_ld, row, p_out, pn, o);
    }
    phase();
    __syncthreads();

  }
  __syncthreads();
  if (w == 2) finish(tiles - 1);

#pragma unroll
  for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
    for (int k = 0; k < KB; ++k) {
      const int row = 16 * k + (lane & 15), n = nw + 16 * nb + 4 * (lane >> 4);
      if (row >= rows || n >= a.N) continue;
      const int64_t r = pc.r0 + row;
      if (b.hsplit > 1) {
        const int64_t width = (int64_t)a.G * a.N;
        float* dst = b.bc_part + ((int64_t)part * a.q.rows + r) * width + gn + n;
        const int64_t other = (int64_t)b.hsplit * a.q.rows * width;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < a.N) {
            dst[e] = dB[nb][k][e];
            dst[other + e] = dC[nb][k][e];
          }
      } else {
        uint16_t *pB = b.dB + r * b.dB_ld + gn + n, *pC = b.dC + r * b.dC_ld + gn + n;
        const u32x2 vB = {pk_bf16(dB[nb][k][0], dB[nb][k][1]), pk_bf16(dB[nb][k][2], dB[nb][k][3])};
        const u32x2 vC = {pk_bf16(dC[nb][k][0], dC[nb][k][1]), pk_bf16(dC[nb][k][2], dC[nb][k][3])};
        if (VEC || n + 3 < a.N) {
          *reinterpret_cast<u32x2_a2*>(pB) = vB;
          *reinterpret_cast<u32x2_a2*>(pC) = vC;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n + e < a.N) {
              pB[e] = (uint16_t)(vB[e >> 1] >> (16 * (e & 1)));
              pC[e] = (uint16_t)(vC[e >> 1] >> (16 * (e & 1)));
            }
        }
      }
    }
}

// dB, dC from the head parts, in ascending order of the parts
__global__ __launch_bounds__(256) void ssm_bc_reduce_kernel(ScanBwdArgs b) {
  const int64_t width = (int64_t)b.s.G * b.s.N, rows = b.s.q.rows;
  // the rows of sequences: the chunks wrote no parts of others
  const int64_t begin = b.s.q.cu ? cu_at(b.s.q, 0) : 0, end = b.s.q.cu ? cu_at(b.s.q, b.s.q.nseq) : rows;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e < begin * width || e >= end * width) return;
  const float* src = b.bc_part + (blockIdx.y ? (int64_t)b.hsplit * rows * width : 0) + e;
  float s = src[0];
  for (int k = 1; k < b.hsplit; ++k) s += src[(int64_t)k * rows * width];
  const int64_t row = e / width, c = e % width;
  if (blockIdx.y) b.dC[row * b.dC_ld + c] = to_bf16(s);
  else b.dB[row * b.dB_ld + c] = to_bf16(s);
}

// dA, d(dt_bias), dD of one head: the chunks' sums, 256 strided subsets and then a fixed tree
__global__ __launch_bounds__(256) void ssm_head_reduce_kernel(ScanBwdArgs b, int64_t ids) {
  __shared__ float lds[4][3];
  const int h = blockIdx.x, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  float s[3] = {0.f, 0.f, 0.f};
  for (int64_t id = threadIdx.x; id < ids; id += 256) {
    const float* src = b.head_part + (id * b.s.H + h) * 3;
#pragma unroll
    for (int e = 0; e < 3; ++e) s[e] += src[e];
  }
#pragma unroll
  for (int e = 0; e < 3; ++e) {
    const float v = wave_sum(s[e]);
    if (lane == 0) lds[w][e] = v;
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    const int e = threadIdx.x;
    const float v = lds[0][e] + lds[1][e] + lds[2][e] + lds[3][e];
    float* dst = e == 0 ? b.dA : (e == 1 ? b.dbias : b.dD);
    if (dst) dst[h] = v;
  }
}

template <int NT, int U, bool VEC>
static hipError_t launch(const ScanBwdArgs& b, hipStream_t s) {
  const ScanArgs& a = b.s;
  const int64_t items = a.n_slots + a.q.nseq, ids = b.n_chunk_slots + a.q.nseq;
  StateArgs f{}, r{};
  f.s = r.s = a;
  f.u = a.x, f.u_ld = a.x_ld, f.v = a.B, f.v_ld = a.B_ld;
  r.u = b.dy, r.u_ld = b.dy_ld, r.v = a.C, r.v_ld = a.C_ld;
  f.start = a.init, f.piece = a.piece, f.store = b.cs;
  r.start = b.dfin, r.piece = b.piece_t, r.store = b.ct, r.end = b.dinit;
  f.decay = a.piece_decay, r.decay = b.piece_t_decay;
  f.n_chunk_slots = r.n_chunk_slots = b.n_chunk_slots;
  const dim3 walk((uint32_t)unit_blocks(items, a.H, a.G, a.ptiles, U), 2);
  if (a.seg > 0) {
    const dim3 join = join_grid(a, NT);
    ssm_states_kernel<NT, U, VEC, false><<<walk, 128 * U, 0, s>>>(f, r);
    ssm_join_kernel<NT, false><<<join, 1024, 0, s>>>(f);
    ssm_join_kernel<NT, true><<<join, 1024, 0, s>>>(r);
  }
  ssm_states_kernel<NT, U, VEC, true><<<walk, 128 * U, 0, s>>>(f, r);
  ssm_scan_bwd_kernel<NT, VEC><<<dim3((uint32_t)(ids * a.G * b.hsplit)), kThreads, 0, s>>>(b);
  if (b.hsplit > 1 && a.q.rows > 0) {
    const int64_t n = a.q.rows * a.G * a.N;
    ssm_bc_reduce_kernel<<<dim3((uint32_t)((n + 255) / 256), 2), 256, 0, s>>>(b);
  }
  ssm_head_reduce_kernel<<<dim3((uint32_t)a.H), 256, 0, s>>>(b, ids);
  return hipGetLastError();
}

// The walks take two units a block where four would leave many CUs without one (4 sequences of 4096 rows, 64 heads,
// 128 blocks of four: 870 us against 912; 1024 rows of 2 sequences, 8 heads: 73 against 80); with more blocks four are
// faster, whose rows of B and C serve more units (nine mixed sequences in 2777 rows, 24 heads, 240 blocks: 140 us
// against 142; 32 sequences in 16384 rows, 64 heads: 829 against 840).
template <int NT, bool VEC>
static hipError_t launch(const ScanBwdArgs& b, hipStream_t s) {
  const ScanArgs& a = b.s;
  if (a.q.nseq == 0) {  // no sequences: the parameters' gradients are zero
    ssm_head_reduce_kernel<<<dim3((uint32_t)a.H), 256, 0, s>>>(b, 0);
    return hipGetLastError();
  }
  if constexpr (NT <= 128)
    if (2 * unit_blocks(a.n_slots + a.q.nseq, a.H, a.G, a.ptiles, kUnits) <= 192) return launch<NT, 2, VEC>(b, s);
  return launch<NT, kUnits, VEC>(b, s);
}

hipError_t launch_scan_bwd(const ScanBwdArgs& b, bool vec, hipStream_t s) {
  switch (state_tile(b.s.N)) {
    case 64: return vec ? launch<64, true>(b, s) : launch<64, false>(b, s);
    case 128: return vec ? launch<128, true>(b, s) : launch<128, false>(b, s);
    default: return vec ? launch<256, true>(b, s) : launch<256, false>(b, s);
  }
}

}  // namespace cssm
