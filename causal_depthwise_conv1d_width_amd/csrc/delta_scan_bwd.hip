// delta_scan_bwd.hip -- backward of the gated delta rule.
//
// For a chunk of 64 rows of one sequence and one head, with S the state before the chunk, D the adjoint of the state
// after it, L, r, T = (I + X)^-1 and P as in delta_chunk.hip, k and q unit or as they are:
//   U = T r (V - e^L K S^T)                                     forward walk
//   F = T^T (P^T dY + e^{L_Q - L} K D^T)                        reverse walk: what reaches r (V - e^L K S^T)
//   D' = e^{L_Q} D + dY^T (scale e^L Q) - F^T (r e^L K)
// Neither walk needs the other's: both run in one launch and store S, U, D and F, FP32, at every chunk.  Then every chunk is
// independent.  With W_ij = dY_i . U_j, Y_ij = F_i . U_j and m_ij = e^{L_i - L_j}:
//   dv_i = r_i F_i
//   dq_i = scale (e^{L_i} S^T dY_i + sum_{j <= i} m_ij W_ij k_j)                       summed over the key head's heads
//   dk_i = e^{L_Q - L_i} D^T U_i - r_i e^{L_i} S^T F_i + sum_{j >= i} scale m_ji W_ji q_j
//          - sum_{j < i} r_i m_ij Y_ij k_j - sum_{j > i} r_j m_ji Y_ji k_j
//   db_i = F_i . U_i (1 - r_i / beta_max)
//   dl_t = e^{L_Q} <D, S> + sum_{i >= t} (q_i . scale e^{L_i} S^T dY_i - k_i . r_i e^{L_i} S^T F_i)
//          + sum_{j < t} k_j . e^{L_Q - L_j} D^T U_j + sum_{i >= t > j} (P_ij W_ij - X_ij Y_ij)
//   d(dt_t) = A dl_t softplus',  and through the norms of q and k at the end.
// All of dl's terms are sums of what decays over row t, by blocks of 16 rows: no differences of longer sums.
// dl, db, dA and the initial states' gradient are FP32 results: S, D, U and F enter their products as two fp16 parts
// (delta_device.h), dY as it is.
// The decayed scores that go into dq and dk alone enter as two: with one these were up to 2.7e-3 off where terms cancel (their own
// rounding: 1.66e-3).
#include "delta_device.h"

namespace cssm {

constexpr int kWalkThreads = 256;

// The walks hold their state, and with it U or F, with a sign that changes from chunk to chunk.  What matrix instructions add up
// comes out a little low, whatever its sign; dl's terms are sums of both signs, and over all the rows of dA and d(dt_bias)
// such offsets add up: 2.8e-6 of dA over 16384 rows, 8e-6 with rates up to two.  With the signs they cancel:
// 2.3e-7.  The forward walk's change at every chunk, the reverse walk's at every second, so that their products'
// change as well.
__device__ __forceinline__ float sign_at(int64_t chunk, bool rev) { return (rev ? chunk >> 1 : chunk) & 1 ? -1.f : 1.f; }

// a tile's element (at, where a place in the workspace has that name)
template <int W, int PAD = 8>
__device__ __forceinline__ int at_(int row, int col) {
  return at<W, PAD>(row, col);
}

// A tile's record as a buffer (past the last one, with nothing in it)
template <int NT>
__device__ __forceinline__ Rows tile_record(const DeltaBwdArgs& b, int64_t tile, bool in) {
  return Rows(b.tiles + tile * tile_floats(NT), tile_floats(NT), 1, in ? tile_floats(NT) : 0, 4);
}
// 16 x 16 blocks of a state (registers n, lanes p)
template <int NB>
__device__ __forceinline__ void store_blocks(const Rows& to, int at, const f32x4 (&S)[NB], float scale, int w, int lane) {
  const int o = (at + w * NB * 256 + (lane & 15) * 16 + (lane >> 4) * 4) * 4;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, S[nb] * scale), to.r, o + nb * 1024, 0, 0);
}
// 64 rows of 64 columns (registers rows, lanes columns), this wave's 16 columns
__device__ __forceinline__ void store_rows(const Rows& to, int at, const f32x4 (&v)[4], int w, int lane) {
  const int o = (at + 4 * (lane >> 4) * 64 + 16 * w + (lane & 15)) * 4;
#pragma unroll
  for (int ib = 0; ib < 4; ++ib)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[ib][e]), to.r, o + (16 * ib + e) * 256, 0, 0);
}

// the largest of 8 and of 64 neighbouring lanes, in every one of them (v >= 0)
__device__ __forceinline__ float max8_lanes(float v) {
  v = __builtin_fmaxf(v, dpp0<0xb1, 0xf>(v));
  v = __builtin_fmaxf(v, dpp0<0x4e, 0xf>(v));
  return __builtin_fmaxf(v, dpp0<0x141, 0xf>(v));
}
__device__ __forceinline__ float wave_max(float v) {
  v = max8_lanes(v);
  return max_across16(__builtin_fmaxf(v, dpp0<0x140, 0xf>(v)));
}

__device__ __forceinline__ float max16_lanes(float v) {
  v = max8_lanes(v);
  return __builtin_fmaxf(v, dpp0<0x140, 0xf>(v));
}
// four values to two fp16 tiles `other` elements apart
__device__ __forceinline__ void store_half4(uint16_t* to, int other, f32x4 v) {
  const u32x2 u = {pk_f16(v[0], v[1]), pk_f16(v[2], v[3])};
  *reinterpret_cast<u32x2*>(to) = u;
  *reinterpret_cast<u32x2*>(to + other) = u32x2{rest_f16(v[0], v[1], u.x), rest_f16(v[2], v[3], u.y)};
}

template <int NT>
struct WalkShared {
  __align__(16) uint16_t kq[key_tile(NT)];  // both tiles' bytes
  __align__(16) uint16_t v[64 * kLd<64, 16>];
  __align__(16) char rec[kRecRev];
};

template <int NT, bool VEC, bool REV>
__device__ __forceinline__ void delta_walk(const DeltaBwdArgs& b, WalkShared<NT>& sh) {
  constexpr int T = kWalkThreads, NB = NT / 16, kBytes = REV ? kRecRev : kRecFwd;
  constexpr int kKeys = (REV ? 2 : 1) * (int)key_tile(NT);  // the forward walk reads k alone
  const DeltaArgs& d = b.d;
  const ScanArgs& a = d.s;
  const Units<1> us(a, blockIdx.x);
  if (!us.ok) return;
  const Unit me(a, us, 0);
  const int w = wave_id(), pn = me.pn;
  Piece pc;
  pc.seq = walk_sequence(d, us.item);
  seq_bounds(a.q, pc.seq, pc.s, pc.e);
  int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15;
  const int p_in = 16 * w + i;
  const int64_t state_at = ((pc.seq * a.H + me.h) * a.P + me.p_first) * a.N;
  const float* start = REV ? b.dfin : a.init;
  if (pc.e <= pc.s) {  // an empty sequence's adjoint passes through
    if (REV && b.dinit)
      for (int e = threadIdx.x; e < pn * a.N; e += T) b.dinit[state_at + e] = start ? start[state_at + e] : 0.f;
    return;
  }
  f32x4 S[NB];
  load_state(S, start && p_in < pn ? start + state_at + (int64_t)p_in * a.N : nullptr, a.N, g);
  int64_t walked = pc.seq;  // sequences of few chunks do not all begin with the same signs
  float turn = sign_at(walked, REV);  // the state's sign in the chunk
  float s_down;  // the state is turn s_down S
  {
    const Pow2 scale = state_scale<REV ? 2 : 1>(state_max(S));
    s_down = scale.down;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) S[nb] *= turn * scale.up;
  }

  const uint16_t* vb = REV ? b.dy : a.x;
  const int64_t v_ld = REV ? b.dy_ld : a.x_ld;
  const char* recs = REV ? b.rec_rev : d.rec;
  CopyRegs<kKeys, T> tK;
  TileRegs<64, T> tV;
  CopyRegs<kBytes, T> tR;
  auto load = [&](const Chunks<REV>& c, int rows) {
    const int64_t id = chunk_id(pc, c.c0, d.n_chunk_slots);
    load_bytes(tK, d.keys + (id * a.G + us.group) * 2 * key_tile(NT), rows > 0, threadIdx.x);
    load_bytes(tR, recs + (id * a.H + me.h) * kBytes, rows > 0, threadIdx.x);
    load_tile<VEC>(tV, Rows(vb + c.c0 * v_ld + me.col, v_ld, rows, pn, 2), (uint32_t)v_ld, pn);
  };
  Chunks<REV> c(pc.s, pc.e);
  int rows = c.rows();
  load(c, rows);
  const uint16_t *sK = sh.kq, *sQ = sh.kq + key_tile(NT) / 2;
  const char *sT = sh.rec, *sP = sh.rec + kRecT;
  const Factors& fac = *reinterpret_cast<const Factors*>(sh.rec + kBytes - kRecVec);
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  for (;;) {
    lane = fresh(lane);
    g = lane >> 4, i = lane & 15;
    store_bytes(sh.kq, tK, threadIdx.x);
    store_bytes(sh.rec, tR, threadIdx.x);
    store_tile<16>(sh.v, tV);
    __syncthreads();
    const Rows to = tile_record<NT>(b, (chunk_id(pc, c.c0, d.n_chunk_slots) * a.H + me.h) * a.ptiles + me.p_first / kPTile, true);
    c = step_chunk(c, rows);  // rows == 0: that was the last one
    load(c, rows);
    store_blocks(to, REV ? tile_d(NT) : tile_s(NT), S, s_down, w, lane);
    phase();
    f32x4 r[4];  // K S: rows in the registers, columns p in the lanes
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) r[ib] = zero;
#pragma unroll
    for (int ks = 0; ks < NT / 32; ++ks) {
      const Halves s = halves(S[2 * ks], S[2 * ks + 1]);
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) r[ib] = mma2(key_rows<NT>(sK, 16 * ib, 32 * ks, lane), s, r[ib]);
    }
    const float s_max = state_max(S);
    {
      const float top = max16_lanes(s_max * s_down);
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(top), to.r,
                                            (int)(lane == 0 ? (tile_tops(NT) + (REV ? 4 : 0) + w) * 4 : kOutside), 0, 0);
    }
    bf16x8 y[2];
    if constexpr (!REV) {
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) {
        const f32x4 f = *reinterpret_cast<const f32x4*>(fac.in + 16 * ib + 4 * g) * s_down;
        r[ib] = fma4(-f, r[ib], column4(sh.v, 16 * ib, 16 * w, g, i) * turn) *
                *reinterpret_cast<const f32x4*>(fac.rate + 16 * ib + 4 * g);
      }
    } else {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        u32x4 v = __builtin_bit_cast(u32x4, op_cols<64, 16>(sh.v, 32 * ks, 16 * w, lane));
        v ^= turn < 0.f ? 0x80008000u : 0u;
        y[ks] = __builtin_bit_cast(bf16x8, v);
      }
#pragma unroll
      for (int jb = 0; jb < 4; ++jb) {
        r[jb] *= *reinterpret_cast<const f32x4*>(fac.out + 16 * jb + 4 * g) * s_down;
#pragma unroll
        for (int ks = jb / 2; ks < 2; ++ks)
#pragma unroll
          for (int p = 2; p >= 0; --p)
            r[jb] = mma(__builtin_bit_cast(bf16x8, tri_cols<3>(sP, jb, ks, p, lane)), y[ks], r[jb]);
      }
    }
    float r_max = 0.f;
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) r_max = max4(r_max, r[ib]);
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
        for (int ks = 0; ks < 2; ++ks)
          if (REV ? ks >= ib / 2 : ks <= ib / 2)
            u[ib] = mma3(REV ? t_cols(sT, ib, ks, lane) : t_rows(sT, ib, ks, lane), rp[ks], u[ib]);
      }
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) u[ib] *= u_down;
    }
    store_rows(to, REV ? tile_f(NT) : tile_u(NT), u, w, lane);
    // what goes into the state and its scale
    f32x4 yo[4];
    float o_max = 0.f;
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) {
      const int row = 16 * ib + 4 * g;
      if constexpr (REV) {
        const u32x4 v = __builtin_bit_cast(u32x4, y[ib / 2]);
        const uint32_t v0 = v[2 * (ib & 1)], v1 = v[2 * (ib & 1) + 1];
        yo[ib] = f32x4{bf_lo(v0), bf_hi(v0), bf_lo(v1), bf_hi(v1)} * *reinterpret_cast<const f32x4*>(fac.read + row);
        o_max = max4(o_max, yo[ib]);
        u[ib] *= -*reinterpret_cast<const f32x4*>(fac.in + row) * *reinterpret_cast<const f32x4*>(fac.rate + row);
      } else {
        u[ib] *= *reinterpret_cast<const f32x4*>(fac.out + row);
      }
      o_max = max4(o_max, u[ib]);
    }
    const float next = sign_at(++walked, REV), change = turn * next, kept = fac.decay * s_down;
    const Pow2 ss = state_scale<REV ? 2 : 1>(__builtin_fmaxf(max_across16(o_max), s_max * kept));
    const float up = change * ss.up;
    s_down = ss.down;
    turn = next;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) S[nb] *= kept * up;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const Halves o = halves(u[2 * ks] * up, u[2 * ks + 1] * up);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) S[nb] = mma2(key_cols<NT>(sK, 32 * ks, 16 * nb, lane), o, S[nb]);
      if constexpr (REV) {
        const Halves q = halves(yo[2 * ks] * up, yo[2 * ks + 1] * up);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) S[nb] = mma2(key_cols<NT>(sQ, 32 * ks, 16 * nb, lane), q, S[nb]);
      }
    }
    if (rows == 0) break;
    __syncthreads();
  }
  if (REV && b.dinit && p_in < pn) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) S[nb] *= turn * s_down;
    store_state(S, b.dinit + state_at + (int64_t)p_in * a.N, a.N, lane >> 4);
  }
}

template <int NT, bool VEC>
__global__ __launch_bounds__(kWalkThreads, NT <= 128 ? 2 : 1) void delta_walks_kernel(DeltaBwdArgs b) {
  __shared__ WalkShared<NT> sh;
  if (blockIdx.y == 0) delta_walk<NT, VEC, true>(b, sh);  // the longer one first
  else delta_walk<NT, VEC, false>(b, sh);
}

// 64 x 64 values as two fp16 tiles
constexpr int kTile = 64 * kLd<64>;
__device__ __forceinline__ Halves tile_halves(const uint16_t* tiles, int row0, int k0, int l) {
  return Halves{as_f16(op_split<64>(tiles, row0, k0, l)), as_f16(op_split<64>(tiles + kTile, row0, k0, l))};
}
// The chunk kernel's tiles, of NT + 8 columns: of 16 rows, 0 to 3 and 8 to 11 in the even places, the others in the odd ones.
// Places are 4 or 36 banks apart (mod 64): the 16 bytes that 16 rows hold of 8 columns fall on different banks, and so do the
// transposing reads' 8 rows of 32 bytes, which contract rows in the same order, 8 (l / 16) on.
template <int NT>
__device__ __forceinline__ int spot_at(int row, int col) {
  return ((row & ~15) + 2 * ((row & 3) + (row >> 1 & 4)) + (row >> 2 & 1)) * (NT + 8) + col;
}
// rows row0 .. row0 + 15 (a multiple of 16), contracted columns k0 .. k0 + 31
template <int NT>
__device__ __forceinline__ bf16x8 spot_rows(const uint16_t* tile, int row0, int k0, int l) {
  return *reinterpret_cast<const bf16x8*>(tile + spot_at<NT>(l & 15, (l >> 4) * 8) + row0 * (NT + 8) + k0);
}
// columns c0 .. c0 + 15, contracted rows k0 .. k0 + 31
template <int NT>
__device__ __forceinline__ bf16x8 spot_cols(const uint16_t* tile, int k0, int c0, int l) {
  const uint16_t* p = tile + spot_at<NT>((l >> 4) * 8 + ((l & 15) >> 2), (l & 3) * 4) + k0 * (NT + 8) + c0;
  const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
  const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + NT + 8)));
  return __builtin_bit_cast(bf16x8, u32x4{a.x, a.y, b.x, b.y});
}
__device__ __forceinline__ Halves spot_halves(const uint16_t* tiles, int row0, int k0, int l) {
  return Halves{as_f16(spot_rows<64>(tiles, row0, k0, l)), as_f16(spot_rows<64>(tiles + kTile, row0, k0, l))};
}
template <int NT>
__device__ __forceinline__ bf16x8 key_bf16(const uint16_t* tile, int row0, int k0, int l) {
  return __builtin_bit_cast(bf16x8, key_rows<NT>(tile, row0, k0, l));
}

// four bf16 values of a row times four FP32 ones
__device__ __forceinline__ float row_dot(const uint16_t* at, f32x4 v) {
  const u32x2 u = *reinterpret_cast<const u32x2*>(at);
  float s = bf_lo(u.x) * v[0];
  s = __builtin_fmaf(bf_hi(u.x), v[1], s);
  s = __builtin_fmaf(bf_lo(u.y), v[2], s);
  return __builtin_fmaf(bf_hi(u.y), v[3], s);
}

// four values of a row as two parts
__device__ __forceinline__ void store_parts(uint16_t* tiles, f32x4 v) {
  const u32x2 u = {pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])};
  *reinterpret_cast<u32x2*>(tiles) = u;
  v -= f32x4{bf_lo(u.x), bf_hi(u.x), bf_lo(u.y), bf_hi(u.y)};
  *reinterpret_cast<u32x2*>(tiles + kTile) = u32x2{pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])};
}

// The sum of the chunk's dl terms and the gradients made of it, one lane a row (a wave): `in`, `out` and `dots` are the rows'
// products with the state, with the adjoint, and the product of both; s_row and s_col the sums by blocks of 16 rows and
// columns of P W - X Y below the diagonal (s_row's diagonal blocks: row r's of all i >= r > j); `diag` is F . U.
struct RowSums {
  float in, out, dots, diag, step, rate, grow_end;
};
__device__ __forceinline__ void finish_rows(const DeltaBwdArgs& b, const RowSums& x, const float (&s_row)[4][64],
                                            const float (&s_col)[4][64], int64_t id, int h, int64_t r0, int rows, int lane) {
  const ScanArgs& a = b.d.s;
  const int m = lane >> 4;
  float left = 0.f, below = 0.f, on = 0.f, corner[2] = {0.f, 0.f};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float r = k <= m ? s_row[k][lane] : 0.f, c = k >= m ? s_col[k][lane] : 0.f;
    left += k < m ? r : 0.f;
    below += k > m ? c : 0.f;
    on += k == m ? r : 0.f;
    if (k == 0) corner[0] = m >= 2 ? r : 0.f;
    if (k <= 1) corner[1] += m == 3 ? r : 0.f;
  }
  const float corner1 = wave_sum(corner[0]), corner2 = wave_sum(corner[1]);
  const float rows_on = row16_suffix(left);  // rows >= this one
  const float columns = dpp0<0x111, 0xf>(row16_sum(below));
  const float inside = rows_on + on + columns + (m == 1 ? corner1 : m == 2 ? corner2 : 0.f);
  const float suffix = __shfl(wave_prefix(__shfl(x.in, 63 - lane)), 63 - lane);  // rows >= this one
  const float before = dpp0<0x138, 0xf>(wave_prefix(x.out));                     // rows < this one
  const float dl = x.grow_end * x.dots + suffix + inside + before;
  const float dstep = a.A[h] * dl, ddt = a.softplus ? dstep * -expm1f(-x.step) : dstep;
  const float db = x.diag * (1.f - x.rate / b.d.beta_max);
  const int size = a.dt_f32 ? 4 : 2;
  const Rows to(static_cast<char*>(b.ddt) + (r0 * b.ddt_ld + h) * size, b.ddt_ld, rows, 1, size);
  const Rows tb(static_cast<char*>(b.db) + (r0 * b.db_ld + h) * size, b.db_ld, rows, 1, size);
  const int o = (int)((uint32_t)lane * (uint32_t)b.ddt_ld * size), ob = (int)((uint32_t)lane * (uint32_t)b.db_ld * size);
  if (a.dt_f32) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(ddt), to.r, o, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(db), tb.r, ob, 0, 0);
  } else {
    __builtin_amdgcn_raw_buffer_store_b16(to_bf16(ddt), to.r, o, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b16(to_bf16(db), tb.r, ob, 0, 0);
  }
  const float sum_A = wave_sum(lane < rows ? x.step * dl : 0.f), sum_b = wave_sum(lane < rows ? ddt : 0.f);
  if (lane == 0) {
    b.head_part[(id * a.H + h) * 2] = sum_A;
    b.head_part[(id * a.H + h) * 2 + 1] = sum_b;
  }
}

// A block takes a chunk and a key head and walks the 64-column tiles of its value heads: U, F, dY, S and D of a tile go
// to shared memory as fp16 parts while the next tile's are loaded.  A wave owns 16 columns n of dq and dk and 32 of the 64
// rows, and one of the ten score blocks: 16 waves (N > 64) in 128 registers, four a SIMD, to cover what each of them
// waits for.  (8 waves of 256 registers that held their parts of S and D spilled: the whole backward took
// 1794 us at 4 x 4096 rows, with these 1510.)  Reading the tiles by 16 bytes from places without bank conflicts made that 1410,
// of which this kernel takes 750: it reads 1.6 GB of tiles, and one block a CU hides little of what its passes wait for.
template <int NT, int WR, bool VEC>
__global__ __launch_bounds__(4 * NT * WR) void delta_scan_bwd_kernel(DeltaBwdArgs b) {
  constexpr int T = 4 * NT * WR, NB = NT / 16, QR = 4 / WR;  // threads, blocks of columns n, of rows a wave
  constexpr int KV = 1024 / T, KS = 64 * NT / 4 / T;  // pieces of four values of U (F, dY), of S (D) a thread
  constexpr int SB = (10 + T / 64 - 1) / (T / 64);    // score blocks a wave
  constexpr int kState = 64 * (NT + 8);               // elements of one part of S
  // all in spot_at's places: K and Q, bf16; then Y, U's and F's parts and S's and D's, or the four decayed scores' two parts
  __shared__ __align__(16) uint16_t sKQ[2 * kState];
  __shared__ __align__(16) uint16_t sAll[5 * kTile + 4 * kState > 8 * kTile ? 5 * kTile + 4 * kState : 8 * kTile];
  __shared__ __align__(16) double sL[64];
  __shared__ __align__(16) float s_rate[64], s_kn[64], s_qn[64], s_step[64], s_grow;
  __shared__ __align__(16) float s_read[64], s_in_f[64], s_out_f[64], s_dv[64];  // signed factors of S^T dY, S^T F, D^T U, F
  __shared__ __align__(16) float s_u[64], s_f[64], s_y[64];  // the tiles' rows are these times their values
  __shared__ float s_row[4][64], s_col[4][64], s_diag[64], s_in[NB][64], s_out[NB][64], s_dot[T / 64];
  uint16_t *sK = sKQ, *sQ = sKQ + kState;
  uint16_t *sY = sAll, *sU = sAll + kTile, *sF = sU + 2 * kTile, *sS = sF + 2 * kTile, *sD = sS + 2 * kState;
  uint16_t *sZk = sAll, *sZq = sAll + 2 * kTile, *sNj = sAll + 4 * kTile, *sNi = sAll + 6 * kTile;
  const DeltaArgs& d = b.d;
  const ScanArgs& a = d.s;
  int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15;
  const int w = wave_id(), nb = w % NB, rh = w / NB;  // columns n from 16 nb on, rows from 16 QR rh on
  const uint32_t blk = xcd_block(blockIdx.x, gridDim.x);
  const int grp = blk % (uint32_t)a.G;
  const int64_t id = blk / (uint32_t)a.G;
  const int hg = a.H / a.G;
  const Piece pc = find_chunk(a.q, id, d.n_chunk_slots);
  if (!pc.ok) {
    for (int e = threadIdx.x; e < hg * 2; e += T) b.head_part[(id * a.H + grp * hg) * 2 + e] = 0.f;
    return;
  }
  const int rows = (int)(pc.r1 - pc.r0), tiles = hg * a.ptiles;
  const int64_t gn = (int64_t)grp * a.N;
  // the signs of the stored states and adjoints
  const float sign_s = sign_at((pc.r0 >> 6) - (pc.s >> 6) + pc.seq, false);
  const float sign_t = sign_at(((pc.e - 1) >> 6) - (pc.r0 >> 6) + pc.seq, true);
  const float sign = sign_s * sign_t;
  // four values a thread and piece, a tile ahead; the tile's scales beside them
  f32x4 lu[KV], lf[KV], ls[KS], lt[KS];
  u32x2 ly[KV];
  float lm[2];
  auto load_all = [&](int t) {
    const int tid = fresh((int)threadIdx.x);
    const int64_t at = (id * a.H + grp * hg) * a.ptiles + t;
    const int h = grp * hg + (uint32_t)t / (uint32_t)a.ptiles, p_first = (uint32_t)t % (uint32_t)a.ptiles * kPTile;
    const int pn = a.P - p_first < kPTile ? a.P - p_first : kPTile;
    const bool in = t < tiles;
    const Rows rt = tile_record<NT>(b, at, in);
    const Rows ry(b.dy + pc.r0 * b.dy_ld + (int64_t)h * a.P + p_first, b.dy_ld, in ? rows : 0, pn, 2);
    lm[0] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rt.r, (tile_tops(NT) + (tid & 3)) * 4, 0, 0));
    lm[1] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rt.r, (tile_tops(NT) + (tid & 3)) * 4 + 16, 0, 0));
#pragma unroll
    for (int k = 0; k < KV; ++k) {
      const int o = tid + T * k, row = o / 16, c = o % 16 * 4;
      lu[k] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rt.r, o * 16 + tile_u(NT) * 4, 0, 0));
      lf[k] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rt.r, o * 16 + tile_f(NT) * 4, 0, 0));
      const uint32_t at_y = (row * (uint32_t)b.dy_ld + c) * 2;
      if constexpr (VEC) {
        ly[k] = __builtin_amdgcn_raw_buffer_load_b64(ry.r, (int)(c < pn ? at_y : kOutside), 0, 0);
      } else {
        ly[k] = u32x2{0u, 0u};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t v = __builtin_amdgcn_raw_buffer_load_b16(ry.r, (int)(c + e < pn ? at_y + 2 * e : kOutside), 0, 0);
          ly[k][e >> 1] |= v << (16 * (e & 1));
        }
      }
    }
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      ls[k] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rt.r, (tid + T * k) * 16, 0, 0));
      lt[k] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rt.r, (tid + T * k) * 16 + tile_d(NT) * 4, 0, 0));
    }
  };
  load_all(0);
  {
    TileRegs<NT, T> tk, tq;
    load_tile<VEC>(tk, Rows(a.B + pc.r0 * a.B_ld + gn, a.B_ld, rows, a.N, 2), (uint32_t)a.B_ld, a.N);
    load_tile<VEC>(tq, Rows(a.C + pc.r0 * a.C_ld + gn, a.C_ld, rows, a.N, 2), (uint32_t)a.C_ld, a.N);
    auto place = [&](const TileRegs<NT, T>& t, uint16_t* tile, float* to) {
#pragma unroll
      for (int k = 0; k < NT * 8 / T; ++k) {
        const int q = threadIdx.x + T * k, row = q / (NT / 8);
        *reinterpret_cast<u32x4*>(tile + spot_at<NT>(row, q % (NT / 8) * 8)) = t.v[k];
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float lo = bf_lo(t.v[k][e]), hi = bf_hi(t.v[k][e]);
          s = __builtin_fmaf(lo, lo, s);
          s = __builtin_fmaf(hi, hi, s);
        }
#pragma unroll
        for (int m = NT / 16; m > 0; m >>= 1) s += __shfl_xor(s, m);
        if (q % (NT / 8) == 0) to[row] = row < rows ? (d.qk_norm ? rsqrtf(s + d.norm_eps) : 1.f) + (s - s) : 0.f;
      }
    };
    place(tk, sK, s_kn);
    place(tq, sQ, s_qn);
  }
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  f32x4 dQ[QR], dK[QR];  // registers n, lanes rows; summed over the heads
#pragma unroll
  for (int q = 0; q < QR; ++q) dQ[q] = dK[q] = zero;

  for (int hh = 0; hh < hg; ++hh) {
    const int h = grp * hg + hh;
    if (w == T / 64 - 1) {  // lane = row
      const Rate rate(a, h);
      const float step = rate.step(raw_step(a, pc.r0, rows, lane, h), lane < rows);
      const float bv = lane < rows ? load_num(d.b, (pc.r0 + lane) * d.b_ld + h, a.dt_f32) : 0.f;
      const double L = wave_prefix(rate.exponent(step));
      const double end = __shfl(L, 63);
      sL[lane] = L;
      s_step[lane] = step;
      s_rate[lane] = lane < rows ? d.beta_max / (1.f + ex2(-kLog2e * bv)) : 0.f;
      const float grow = ex2((float)L);
      if (lane == 63) s_grow = sign * grow;
      s_read[lane] = sign_s * d.scale * grow;
      s_in_f[lane] = -sign * s_rate[lane] * grow;
      s_out_f[lane] = sign * ex2((float)(end - L));
      s_dv[lane] = sign_t * s_rate[lane];
    }
    f32x4 W[SB], Y[SB];  // score blocks: columns j in the registers, rows i in the lanes
#pragma unroll
    for (int t = 0; t < SB; ++t) W[t] = Y[t] = zero;
    float in[QR] = {}, out[QR] = {};  // the rows' products with the state and the adjoint
    float dot = 0.f;
    for (int pt = 0; pt < a.ptiles; ++pt) {
      lane = fresh(lane);
      g = lane >> 4, i = lane & 15;
      const int p_first = pt * kPTile, pn = a.P - p_first < kPTile ? a.P - p_first : kPTile;
      const float ms = __builtin_fmaxf(lm[0], dpp0<0xb1, 0xf>(lm[0])), mt = __builtin_fmaxf(lm[1], dpp0<0xb1, 0xf>(lm[1]));
      const Pow2 ss = bring_to<10>(uniform(__builtin_fmaxf(ms, dpp0<0x4e, 0xf>(ms))));
      const Pow2 ts = bring_to<10>(uniform(__builtin_fmaxf(mt, dpp0<0x4e, 0xf>(mt))));
      __syncthreads();  // the last tile's or head's reads are done; this head's factors are there
      const int tid = fresh((int)threadIdx.x);
      const Rows dv(b.dv + pc.r0 * b.dv_ld + (int64_t)h * a.P + p_first, b.dv_ld, rows, pn, 2);
#pragma unroll
      for (int k = 0; k < KV; ++k) {
        const int q = tid + T * k, row = q / 16, c = q % 16 * 4, o = spot_at<64>(row, c);
        const f32x4 y = {bf_lo(ly[k].x), bf_hi(ly[k].x), bf_lo(ly[k].y), bf_hi(ly[k].y)};
        const Pow2 us = bring_to<10>(max16_lanes(max4(0.f, lu[k])));
        const Pow2 fs = bring_to<10>(max16_lanes(max4(0.f, lf[k])));
        const Pow2 ys = bring_to<10>(max16_lanes(max4(0.f, y)));
        store_half4(sU + o, kTile, lu[k] * us.up);
        store_half4(sF + o, kTile, lf[k] * fs.up);
        const f32x4 yv = y * ys.up;
        *reinterpret_cast<u32x2*>(sY + o) = u32x2{pk_f16(yv[0], yv[1]), pk_f16(yv[2], yv[3])};
        if (c == 0) {
          s_u[row] = us.down;
          s_f[row] = fs.down;
          s_y[row] = ys.down;
        }
        const f32x4 v = lf[k] * s_dv[row];
        store4<VEC>(dv, (uint32_t)b.dv_ld, row, c, pn, u32x2{pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])});
      }
#pragma unroll
      for (int k = 0; k < KS; ++k) {  // 16 x 16 blocks, [p block][n block][16 p][16 n]
        const int q = tid + T * k, p = q / (4 * NT) * 16 + q / 4 % 16, n = q / 64 % NB * 16 + q % 4 * 4;
        store_half4(sS + spot_at<NT>(p, n), kState, ls[k] * ss.up);
        store_half4(sD + spot_at<NT>(p, n), kState, lt[k] * ts.up);
#pragma unroll
        for (int e = 0; e < 4; ++e) dot = __builtin_fmaf(ls[k][e], lt[k][e], dot);
      }
      here(dot);
      load_all(hh * a.ptiles + pt + 1);
      phase();
      __syncthreads();
      lane = fresh(lane);
      g = lane >> 4, i = lane & 15;
      {
        Halves sp[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          sp[ks] = Halves{as_f16(spot_cols<NT>(sS, 32 * ks, 16 * nb, lane)), as_f16(spot_cols<NT>(sS + kState, 32 * ks, 16 * nb, lane))};
#pragma unroll
        for (int q = 0; q < QR; ++q) {
          const int row0 = 16 * (QR * rh + q), row = row0 + i, n = 16 * nb + 4 * g;
          f32x4 q4 = zero, f4 = zero;
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            q4 = mma2(sp[ks], as_f16(spot_rows<64>(sY, row0, 32 * ks, lane)), q4);
            f4 = mma3(sp[ks], spot_halves(sF, row0, 32 * ks, lane), f4);
          }
          const f32x4 vq = q4 * (s_read[row] * s_y[row] * ss.down);
          const f32x4 vf = f4 * (s_in_f[row] * s_f[row] * ss.down);
          in[q] += row_dot(sQ + spot_at<NT>(row, n), vq) * s_qn[row] + row_dot(sK + spot_at<NT>(row, n), vf) * s_kn[row];
          dQ[q] += vq;
          dK[q] += vf;
          here(in[q]), here(dQ[q]), here(dK[q]);
          phase();
        }
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          sp[ks] = Halves{as_f16(spot_cols<NT>(sD, 32 * ks, 16 * nb, lane)), as_f16(spot_cols<NT>(sD + kState, 32 * ks, 16 * nb, lane))};
#pragma unroll
        for (int q = 0; q < QR; ++q) {
          const int row0 = 16 * (QR * rh + q), row = row0 + i, n = 16 * nb + 4 * g;
          f32x4 u4 = zero;
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) u4 = mma3(sp[ks], spot_halves(sU, row0, 32 * ks, lane), u4);
          const f32x4 vu = u4 * (s_out_f[row] * s_u[row] * ts.down);
          out[q] += row_dot(sK + spot_at<NT>(row, n), vu) * s_kn[row];
          dK[q] += vu;
          here(out[q]), here(dK[q]);
          phase();
        }
      }
#pragma unroll
      for (int s = 0; s < SB; ++s) {
        int ib, jb;
        lower_block(w + T / 64 * s, ib, jb);
        if (w + T / 64 * s >= 10) continue;
        f32x4 w4 = zero, y4 = zero;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const Halves u = spot_halves(sU, 16 * jb, 32 * ks, lane);
          w4 = mma2(u, as_f16(spot_rows<64>(sY, 16 * ib, 32 * ks, lane)), w4);
          y4 = mma3(u, spot_halves(sF, 16 * ib, 32 * ks, lane), y4);
        }
        const f32x4 uj = *reinterpret_cast<const f32x4*>(s_u + 16 * jb + 4 * g);
        W[s] = fma4(w4, uj * s_y[16 * ib + i], W[s]);
        Y[s] = fma4(y4, uj * s_f[16 * ib + i], Y[s]);
        here(W[s]), here(Y[s]);
      }
      phase();
    }
    dot = wave_sum(dot);
    if (lane == 0) s_dot[w] = dot;
#pragma unroll
    for (int q = 0; q < QR; ++q) {
      const float x = sum_across16(in[q]), o = sum_across16(out[q]);
      if (g == 0) {
        s_in[nb][16 * (QR * rh + q) + i] = x;
        s_out[nb][16 * (QR * rh + q) + i] = o;
      }
    }
    __syncthreads();  // the tile is read
    lane = fresh(lane);
    g = lane >> 4, i = lane & 15;
#pragma unroll
    for (int s = 0; s < SB; ++s) {
      int ib, jb;
      lower_block(w + T / 64 * s, ib, jb);
      if (w + T / 64 * s >= 10) continue;
      const int row = 16 * ib + i, col = 16 * jb + 4 * g;
      f32x4 kk = zero, qk = zero;
#pragma unroll
      for (int ks = 0; ks < NT / 32; ++ks) {
        const bf16x8 kj = spot_rows<NT>(sK, 16 * jb, 32 * ks, lane);
        kk = mma(kj, spot_rows<NT>(sK, 16 * ib, 32 * ks, lane), kk);
        qk = mma(kj, spot_rows<NT>(sQ, 16 * ib, 32 * ks, lane), qk);
      }
      const double Li = sL[row];
      const float ri = s_rate[row], kni = s_kn[row], qni = d.scale * s_qn[row];
      const f32x4 knj = *reinterpret_cast<const f32x4*>(s_kn + col);
      f32x4 zk, zq, nj, ni;
      float sum = 0.f, diag = 0.f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool under = col + r < row, here = col + r == row;
        const float m = under || here ? ex2((float)(Li - sL[col + r])) : 0.f;
        const float z = m * (sign_s * W[s][r]), y = sign * Y[s][r], n = under ? -(m * ri) * y : 0.f;
        zk[r] = z * (d.scale * knj[r]);
        zq[r] = z * qni;
        nj[r] = n * knj[r];
        ni[r] = n * kni;
        // P W - X Y below the diagonal
        const float x = under ? qk[r] * zq[r] * knj[r] + kk[r] * nj[r] * kni : 0.f;
        diag = here ? y : diag;
        const float from = row16_suffix(x);  // rows >= i of column j
        if (i == 0) s_col[ib][col + r] = from;
        sum += ib != jb ? x : (4 * g + r < i ? from : 0.f);
      }
      const int o = spot_at<64>(row, col);
      store_parts(sZk + o, zk);
      store_parts(sZq + o, zq);
      store_parts(sNj + o, nj);
      store_parts(sNi + o, ni);
      sum = sum_across16(sum);
      if (g == 0) s_row[jb][row] = sum;
      if (ib == jb && (i >> 2) == g) s_diag[row] = diag;
    }
    // blocks (0, 1), (2, 3): products over 32 rows or columns read them
    if (w < 2) {
      const int o = spot_at<64>(32 * w + i, 32 * w + 16 + 4 * g);
      store_parts(sZk + o, zero);
      store_parts(sZq + o, zero);
      store_parts(sNj + o, zero);
      store_parts(sNi + o, zero);
    }
    __syncthreads();
    if (w == T / 64 - 1) {  // lane = row
      RowSums x{0.f, 0.f, 0.f, s_diag[lane], s_step[lane], s_rate[lane], s_grow};
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        x.in += s_in[k][lane];
        x.out += s_out[k][lane];
      }
#pragma unroll
      for (int k = 0; k < T / 64; ++k) x.dots += s_dot[k];
      finish_rows(b, x, s_row, s_col, id, h, pc.r0, rows, lane);
    }
    phase();
    lane = fresh(lane);
    g = lane >> 4, i = lane & 15;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const bf16x8 k = spot_cols<NT>(sK, 32 * ks, 16 * nb, lane);
      const bf16x8 qq = spot_cols<NT>(sQ, 32 * ks, 16 * nb, lane);
#pragma unroll
      for (int q = 0; q < QR; ++q) {
        const int row0 = 16 * (QR * rh + q);
        if (ks <= (QR * rh + q) / 2) {  // contracted columns j of these rows
#pragma unroll
          for (int p = 1; p >= 0; --p) {
            dQ[q] = mma(k, spot_rows<64>(sZk + p * kTile, row0, 32 * ks, lane), dQ[q]);
            dK[q] = mma(k, spot_rows<64>(sNj + p * kTile, row0, 32 * ks, lane), dK[q]);
          }
        }
        if (ks >= (QR * rh + q) / 2) {  // contracted rows i of these columns
#pragma unroll
          for (int p = 1; p >= 0; --p) {
            dK[q] = mma(qq, spot_cols<64>(sZq + p * kTile, 32 * ks, row0, lane), dK[q]);
            dK[q] = mma(k, spot_cols<64>(sNi + p * kTile, 32 * ks, row0, lane), dK[q]);
          }
        }
      }
      phase();
    }
  }
  // through the norms: x = f y, f = (|y|^2 + eps)^(-1/2):  dy = f dx - f^3 y (y . dx)
  __syncthreads();
#pragma unroll
  for (int q = 0; q < QR; ++q) {
    const int row = 16 * (QR * rh + q) + i, n = 16 * nb + 4 * g;
    const u32x2 qv = *reinterpret_cast<const u32x2*>(sQ + spot_at<NT>(row, n));
    const u32x2 kv = *reinterpret_cast<const u32x2*>(sK + spot_at<NT>(row, n));
    const f32x4 x = dQ[q], y = dK[q];
    const float dq = sum_across16(x[0] * bf_lo(qv.x) + x[1] * bf_hi(qv.x) + x[2] * bf_lo(qv.y) + x[3] * bf_hi(qv.y));
    const float dk = sum_across16(y[0] * bf_lo(kv.x) + y[1] * bf_hi(kv.x) + y[2] * bf_lo(kv.y) + y[3] * bf_hi(kv.y));
    if (g == 0) {
      s_in[nb][row] = dq;
      s_out[nb][row] = dk;
    }
  }
  __syncthreads();
  const Rows oq(b.dq + pc.r0 * b.dq_ld + gn, b.dq_ld, rows, a.N, 2), ok(b.dk + pc.r0 * b.dk_ld + gn, b.dk_ld, rows, a.N, 2);
#pragma unroll
  for (int q = 0; q < QR; ++q) {
    const int row = 16 * (QR * rh + q) + i, n = 16 * nb + 4 * g;
    const float fq = s_qn[row], fk = s_kn[row];
    float dq = 0.f, dk = 0.f;
    if (d.qk_norm) {
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        dq += s_in[k][row];
        dk += s_out[k][row];
      }
      dq *= fq * fq * fq;
      dk *= fk * fk * fk;
    }
    const u32x2 qv = *reinterpret_cast<const u32x2*>(sQ + spot_at<NT>(row, n));
    const u32x2 kv = *reinterpret_cast<const u32x2*>(sK + spot_at<NT>(row, n));
    const f32x4 x = dQ[q] * fq - f32x4{bf_lo(qv.x), bf_hi(qv.x), bf_lo(qv.y), bf_hi(qv.y)} * dq;
    const f32x4 y = dK[q] * fk - f32x4{bf_lo(kv.x), bf_hi(kv.x), bf_lo(kv.y), bf_hi(kv.y)} * dk;
    store4<VEC>(oq, (uint32_t)b.dq_ld, row, n, a.N, u32x2{pk_bf16(x[0], x[1]), pk_bf16(x[2], x[3])});
    store4<VEC>(ok, (uint32_t)b.dk_ld, row, n, a.N, u32x2{pk_bf16(y[0], y[1]), pk_bf16(y[2], y[3])});
  }
}

// The same for states of more than 128 columns, whose tiles shared memory does not hold: a wave keeps its columns' part of S and
// D in registers.  It owns 16 NBW columns n of dq and dk and one or two of the ten score blocks.
template <int NT, int WAVES, bool VEC>
__global__ __launch_bounds__(64 * WAVES, WAVES / 4) void delta_scan_bwd_wide_kernel(DeltaBwdArgs b) {
  constexpr int T = 64 * WAVES, NBW = NT / 16 / WAVES, SB = (10 + WAVES - 1) / WAVES, KT = 512 / T;
  __shared__ __align__(16) uint16_t sK[key_tile(NT) / 2];  // bf16, in the places of the walks' tiles
  __shared__ __align__(16) uint16_t sQ[key_tile(NT) / 2];
  __shared__ __align__(16) uint16_t sY[kTile];
  __shared__ __align__(16) uint16_t sUF[8 * kTile];  // U's and F's parts, then the four decayed scores' two
  __shared__ __align__(16) double sL[64];
  __shared__ __align__(16) float s_rate[64], s_kn[64], s_qn[64], s_step[64], s_grow[64], s_left[64];
  __shared__ __align__(16) float s_u[64], s_f[64], s_y[64];  // the tiles' rows are these times their values
  __shared__ float s_row[4][64], s_col[4][64], s_diag[64], s_in[WAVES][64], s_out[WAVES][64], s_dot[WAVES];
  uint16_t *sU = sUF, *sF = sUF + 2 * kTile;
  uint16_t *sZk = sUF, *sZq = sUF + 2 * kTile, *sNj = sUF + 4 * kTile, *sNi = sUF + 6 * kTile;
  const DeltaArgs& d = b.d;
  const ScanArgs& a = d.s;
  int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15;
  const int w = wave_id();
  const uint32_t blk = xcd_block(blockIdx.x, gridDim.x);
  const int grp = blk % (uint32_t)a.G;
  const int64_t id = blk / (uint32_t)a.G;
  const int hg = a.H / a.G;
  const Piece pc = find_chunk(a.q, id, d.n_chunk_slots);
  if (!pc.ok) {
    for (int e = threadIdx.x; e < hg * 2; e += T) b.head_part[(id * a.H + grp * hg) * 2 + e] = 0.f;
    return;
  }
  const int rows = (int)(pc.r1 - pc.r0);
  const int64_t gn = (int64_t)grp * a.N;
  // the signs of the stored states and adjoints
  const float sign_s = sign_at((pc.r0 >> 6) - (pc.s >> 6) + pc.seq, false);
  const float sign_t = sign_at(((pc.e - 1) >> 6) - (pc.r0 >> 6) + pc.seq, true);
  const float sign = sign_s * sign_t;
  {
    TileRegs<NT, T> tk, tq;
    load_tile<VEC>(tk, Rows(a.B + pc.r0 * a.B_ld + gn, a.B_ld, rows, a.N, 2), (uint32_t)a.B_ld, a.N);
    load_tile<VEC>(tq, Rows(a.C + pc.r0 * a.C_ld + gn, a.C_ld, rows, a.N, 2), (uint32_t)a.C_ld, a.N);
#pragma unroll
    for (int k = 0; k < NT * 8 / T; ++k) {
      const int q = threadIdx.x + T * k, o = key_at<NT>(q / (NT / 8), q % (NT / 8) * 8);
      *reinterpret_cast<u32x4*>(sK + o) = tk.v[k];
      *reinterpret_cast<u32x4*>(sQ + o) = tq.v[k];
    }
    auto norms = [&](const TileRegs<NT, T>& t, float* to) {
#pragma unroll
      for (int k = 0; k < NT * 8 / T; ++k) {
        const int row = (threadIdx.x + T * k) / (NT / 8);
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float lo = bf_lo(t.v[k][e]), hi = bf_hi(t.v[k][e]);
          s = __builtin_fmaf(lo, lo, s);
          s = __builtin_fmaf(hi, hi, s);
        }
#pragma unroll
        for (int m = NT / 16; m > 0; m >>= 1) s += __shfl_xor(s, m);
        if (threadIdx.x % (NT / 8) == 0) to[row] = row < rows ? (d.qk_norm ? rsqrtf(s + d.norm_eps) : 1.f) + (s - s) : 0.f;
      }
    };
    norms(tk, s_kn);
    norms(tq, s_qn);
  }
  __syncthreads();
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  f32x4 dQ[NBW][4], dK[NBW][4];  // registers n, lanes rows; summed over the heads
#pragma unroll
  for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) dQ[nb][ib] = dK[nb][ib] = zero;

  // rows of U, F and dY, 8 values a thread and step, loaded a tile ahead
  f32x4 lu[KT][2], lf[KT][2];
  TileRegs<64, T> ly;
  const int tiles = hg * a.ptiles;
  auto load_values = [&](int t) {
    const int h = grp * hg + (uint32_t)t / (uint32_t)a.ptiles, pt = (uint32_t)t % (uint32_t)a.ptiles, p_first = pt * kPTile;
    const int pn = a.P - p_first < kPTile ? a.P - p_first : kPTile, n = t < tiles ? 4096 : 0;
    const int64_t at = (id * a.H + h) * a.ptiles + pt;
    const Rows rt = tile_record<NT>(b, at, n > 0);
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int o = (threadIdx.x + T * k) * 32 + 16 * e;
        lu[k][e] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rt.r, o + tile_u(NT) * 4, 0, 0));
        lf[k][e] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rt.r, o + tile_f(NT) * 4, 0, 0));
      }
    load_tile<VEC>(ly, Rows(b.dy + pc.r0 * b.dy_ld + (int64_t)h * a.P + p_first, b.dy_ld, n ? rows : 0, pn, 2),
                   (uint32_t)b.dy_ld, pn);
  };
  // the state and the adjoint: this wave's columns n in the lanes, contracted rows p in the registers
  f32x4 ls[NBW][2][2], lt[NBW][2][2];
  auto load_states = [&](int t) {
    const int64_t at = (id * a.H + grp * hg) * a.ptiles + t;
    const Rows rt = tile_record<NT>(b, at, t < tiles);
#pragma unroll
    for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int o = (((2 * ks + q) * (NT / 16) + w * NBW + nb) * 256 + (4 * g + e) * 16 + i) * 4;
            ls[nb][ks][q][e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rt.r, o, 0, 0));
            lt[nb][ks][q][e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rt.r, o + tile_d(NT) * 4, 0, 0));
          }
  };
  load_values(0);
  load_states(0);
  for (int hh = 0; hh < hg; ++hh) {
    lane = fresh(lane);
    g = lane >> 4, i = lane & 15;
    const int h = grp * hg + hh;
    if (w == 0) {  // lane = row
      const Rate rate(a, h);
      const float step = rate.step(raw_step(a, pc.r0, rows, lane, h), lane < rows);
      const float bv = lane < rows ? load_num(d.b, (pc.r0 + lane) * d.b_ld + h, a.dt_f32) : 0.f;
      const double L = wave_prefix(rate.exponent(step));
      const double end = __shfl(L, 63);
      sL[lane] = L;
      s_step[lane] = step;
      s_rate[lane] = lane < rows ? d.beta_max / (1.f + ex2(-kLog2e * bv)) : 0.f;
      s_grow[lane] = ex2((float)L);
      s_left[lane] = ex2((float)(end - L));
    }
    f32x4 W[SB], Y[SB];
    float in[4] = {0.f, 0.f, 0.f, 0.f}, out[4] = {0.f, 0.f, 0.f, 0.f};  // the rows' products with the state and the adjoint
#pragma unroll
    for (int t = 0; t < SB; ++t) W[t] = Y[t] = zero;
    float dot = 0.f;
    for (int pt = 0; pt < a.ptiles; ++pt) {
      lane = fresh(lane);
      g = lane >> 4, i = lane & 15;
      const int p_first = pt * kPTile, pn = a.P - p_first < kPTile ? a.P - p_first : kPTile;
      const int64_t col = (int64_t)h * a.P + p_first;
      __syncthreads();  // the last tile's or head's reads are done; this head's factors are there
      {
        const Rows dv(b.dv + pc.r0 * b.dv_ld + col, b.dv_ld, rows, pn, 2);
#pragma unroll
        for (int k = 0; k < KT; ++k) {
          const int row = (threadIdx.x + T * k) / 8, c = (threadIdx.x + T * k) % 8 * 8, o = at_<64>(row, c);
          const u32x4 yv = ly.v[k];
          f32x4 y0 = {bf_lo(yv.x), bf_hi(yv.x), bf_lo(yv.y), bf_hi(yv.y)}, y1 = {bf_lo(yv.z), bf_hi(yv.z), bf_lo(yv.w), bf_hi(yv.w)};
          const Pow2 us = bring_to<10>(max8_lanes(max4(max4(0.f, lu[k][0]), lu[k][1])));
          const Pow2 fs = bring_to<10>(max8_lanes(max4(max4(0.f, lf[k][0]), lf[k][1])));
          const Pow2 ys = bring_to<10>(max8_lanes(max4(max4(0.f, y0), y1)));
          const Halves hu = halves(lu[k][0] * us.up, lu[k][1] * us.up), hf = halves(lf[k][0] * fs.up, lf[k][1] * fs.up);
          *reinterpret_cast<f16x8*>(sU + o) = hu.hi;
          *reinterpret_cast<f16x8*>(sU + kTile + o) = hu.lo;
          *reinterpret_cast<f16x8*>(sF + o) = hf.hi;
          *reinterpret_cast<f16x8*>(sF + kTile + o) = hf.lo;
          *reinterpret_cast<f16x8*>(sY + o) = halves_hi(y0 * ys.up, y1 * ys.up);
          if (c == 0) {
            s_u[row] = us.down;
            s_f[row] = fs.down;
            s_y[row] = ys.down;
          }
          const float rate = sign_t * s_rate[row];
          const f32x4 v0 = lf[k][0] * rate, v1 = lf[k][1] * rate;
          store4<VEC>(dv, (uint32_t)b.dv_ld, row, c, pn, u32x2{pk_bf16(v0[0], v0[1]), pk_bf16(v0[2], v0[3])});
          store4<VEC>(dv, (uint32_t)b.dv_ld, row, c + 4, pn, u32x2{pk_bf16(v1[0], v1[1]), pk_bf16(v1[2], v1[3])});
        }
      }
      Halves sp[NBW][2], tp[NBW][2];
      float s_dn[NBW], t_dn[NBW];
#pragma unroll
      for (int nb = 0; nb < NBW; ++nb) {
        float ms = 0.f, mt = 0.f;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            ms = max4(ms, ls[nb][ks][q]);
            mt = max4(mt, lt[nb][ks][q]);
#pragma unroll
            for (int e = 0; e < 4; ++e) dot = __builtin_fmaf(ls[nb][ks][q][e], lt[nb][ks][q][e], dot);
          }
        here(dot);
        const Pow2 ss = bring_to<10>(wave_max(ms)), ts = bring_to<10>(wave_max(mt));
        s_dn[nb] = ss.down, t_dn[nb] = ts.down;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          sp[nb][ks] = halves(ls[nb][ks][0] * ss.up, ls[nb][ks][1] * ss.up);
          tp[nb][ks] = halves(lt[nb][ks][0] * ts.up, lt[nb][ks][1] * ts.up);
        }
      }
      phase();
      load_values(hh * a.ptiles + pt + 1);
      load_states(hh * a.ptiles + pt + 1);
      phase();
      __syncthreads();
      lane = fresh(lane);
      g = lane >> 4, i = lane & 15;
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) {
        const int row = 16 * ib + i;
        f32x4 q4[NBW], f4[NBW], u4[NBW];
#pragma unroll
        for (int nb = 0; nb < NBW; ++nb) q4[nb] = f4[nb] = u4[nb] = zero;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const f16x8 y = as_f16(op_split<64>(sY, 16 * ib, 32 * ks, lane));
          const Halves f = tile_halves(sF, 16 * ib, 32 * ks, lane), u = tile_halves(sU, 16 * ib, 32 * ks, lane);
#pragma unroll
          for (int nb = 0; nb < NBW; ++nb) {
            q4[nb] = mma2(sp[nb][ks], y, q4[nb]);
            f4[nb] = mma3(sp[nb][ks], f, f4[nb]);
            u4[nb] = mma3(tp[nb][ks], u, u4[nb]);
          }
        }
        const float gq = sign_s * d.scale * s_grow[row] * s_y[row], gf = -sign * s_rate[row] * s_grow[row] * s_f[row];
        const float gu = sign * s_left[row] * s_u[row];
        float in_q = 0.f, in_k = 0.f, ou = 0.f;
#pragma unroll
        for (int nb = 0; nb < NBW; ++nb) {
          const int n = 16 * (w * NBW + nb) + 4 * g;
          const u32x2 qv = *reinterpret_cast<const u32x2*>(sQ + key_at<NT>(row, n));
          const u32x2 kv = *reinterpret_cast<const u32x2*>(sK + key_at<NT>(row, n));
          const f32x4 qr = {bf_lo(qv.x), bf_hi(qv.x), bf_lo(qv.y), bf_hi(qv.y)};
          const f32x4 kr = {bf_lo(kv.x), bf_hi(kv.x), bf_lo(kv.y), bf_hi(kv.y)};
          const f32x4 vq = q4[nb] * (gq * s_dn[nb]), vf = f4[nb] * (gf * s_dn[nb]), vu = u4[nb] * (gu * t_dn[nb]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            in_q = __builtin_fmaf(qr[e], vq[e], in_q);
            in_k = __builtin_fmaf(kr[e], vf[e], in_k);
            ou = __builtin_fmaf(kr[e], vu[e], ou);
          }
          dQ[nb][ib] += vq;
          dK[nb][ib] += vf + vu;
          here(dQ[nb][ib]), here(dK[nb][ib]);
        }
        in[ib] += in_q * s_qn[row] + in_k * s_kn[row];
        out[ib] += ou * s_kn[row];
        phase();
      }
#pragma unroll
      for (int t = 0; t < SB; ++t) {
        int ib, jb;
        lower_block(w + WAVES * t, ib, jb);
        if (w + WAVES * t < 10) {
          f32x4 w4 = zero, y4 = zero;
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            const Halves u = tile_halves(sU, 16 * jb, 32 * ks, lane);
            w4 = mma2(u, as_f16(op_split<64>(sY, 16 * ib, 32 * ks, lane)), w4);
            y4 = mma3(u, tile_halves(sF, 16 * ib, 32 * ks, lane), y4);
          }
          const f32x4 uj = *reinterpret_cast<const f32x4*>(s_u + 16 * jb + 4 * g);
          W[t] += w4 * (uj * s_y[16 * ib + i]);
          Y[t] += y4 * (uj * s_f[16 * ib + i]);
        }
      }
    }
    dot = wave_sum(dot);
    if (lane == 0) s_dot[w] = dot;
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) {
      const float x = sum_across16(in[ib]), o = sum_across16(out[ib]);
      if (g == 0) {
        s_in[w][16 * ib + i] = x;
        s_out[w][16 * ib + i] = o;
      }
    }
    __syncthreads();  // U's and F's parts are read
    lane = fresh(lane);
    g = lane >> 4, i = lane & 15;
#pragma unroll
    for (int t = 0; t < SB; ++t) {
      int ib, jb;
      lower_block(w + WAVES * t, ib, jb);
      if (w + WAVES * t < 10) {
        const int row = 16 * ib + i, col = 16 * jb + 4 * g;
        // the products again for every head: kept, their registers spill
        f32x4 kk = zero, qk = zero;
#pragma unroll
        for (int ks = 0; ks < NT / 32; ++ks) {
          const bf16x8 kj = key_bf16<NT>(sK, 16 * jb, 32 * ks, lane);
          kk = mma(kj, key_bf16<NT>(sK, 16 * ib, 32 * ks, lane), kk);
          qk = mma(kj, key_bf16<NT>(sQ, 16 * ib, 32 * ks, lane), qk);
        }
        const double Li = sL[row];
        const float ri = s_rate[row], kni = s_kn[row], qni = d.scale * s_qn[row];
        const f32x4 knj = *reinterpret_cast<const f32x4*>(s_kn + col);
        f32x4 zk, zq, nj, ni;
        float sum = 0.f, diag = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool under = col + r < row, here = col + r == row;
          const float m = under || here ? ex2((float)(Li - sL[col + r])) : 0.f;
          const float z = m * (sign_s * W[t][r]), y = sign * Y[t][r], n = under ? -(m * ri) * y : 0.f;
          zk[r] = z * (d.scale * knj[r]);
          zq[r] = z * qni;
          nj[r] = n * knj[r];
          ni[r] = n * kni;
          // P W - X Y below the diagonal
          const float x = under ? qk[r] * zq[r] * knj[r] + kk[r] * nj[r] * kni : 0.f;
          diag = here ? y : diag;
          const float from = row16_suffix(x);  // rows >= i of column j
          if (i == 0) s_col[ib][col + r] = from;
          sum += ib != jb ? x : (4 * g + r < i ? from : 0.f);
        }
        const int o = at_<64>(row, col);
        store_parts(sZk + o, zk);
        store_parts(sZq + o, zq);
        store_parts(sNj + o, nj);
        store_parts(sNi + o, ni);
        sum = sum_across16(sum);
        if (g == 0) s_row[jb][row] = sum;
        if (ib == jb && (i >> 2) == g) s_diag[row] = diag;
        phase();
      }
    }
    // blocks (0, 1), (2, 3): products over 32 rows or columns read them
    if (w < 2) {
      const int o = at_<64>(32 * w + i, 32 * w + 16 + 4 * g);
      store_parts(sZk + o, zero);
      store_parts(sZq + o, zero);
      store_parts(sNj + o, zero);
      store_parts(sNi + o, zero);
    }
    __syncthreads();
    if (w == 0) {  // lane = row
      RowSums x{0.f, 0.f, 0.f, s_diag[lane], s_step[lane], s_rate[lane], sign * s_grow[63]};
#pragma unroll
      for (int k = 0; k < WAVES; ++k) {
        x.in += s_in[k][lane];
        x.out += s_out[k][lane];
        x.dots += s_dot[k];
      }
      finish_rows(b, x, s_row, s_col, id, h, pc.r0, rows, lane);
    }
    phase();
    lane = fresh(lane);
    g = lane >> 4, i = lane & 15;
#pragma unroll
    for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const int n = 16 * (w * NBW + nb);
        const bf16x8 k = __builtin_bit_cast(bf16x8, key_cols<NT>(sK, 32 * ks, n, lane));
        const bf16x8 q = __builtin_bit_cast(bf16x8, key_cols<NT>(sQ, 32 * ks, n, lane));
#pragma unroll
        for (int ib = 0; ib < 4; ++ib) {
#pragma unroll
          for (int p = 1; p >= 0; --p) {
            if (ks <= ib / 2) {  // contracted columns j of row block ib
              dQ[nb][ib] = mma(k, op_split<64>(sZk + p * kTile, 16 * ib, 32 * ks, lane), dQ[nb][ib]);
              dK[nb][ib] = mma(k, op_split<64>(sNj + p * kTile, 16 * ib, 32 * ks, lane), dK[nb][ib]);
            }
            if (ks >= ib / 2) {  // contracted rows i of column block ib
              dK[nb][ib] = mma(q, op_cols<64>(sZq + p * kTile, 32 * ks, 16 * ib, lane), dK[nb][ib]);
              dK[nb][ib] = mma(k, op_cols<64>(sNi + p * kTile, 32 * ks, 16 * ib, lane), dK[nb][ib]);
            }
          }
        }
        phase();
      }
  }
  // through the norms: x = f y, f = (|y|^2 + eps)^(-1/2):  dy = f dx - f^3 y (y . dx)
  __syncthreads();
  if (d.qk_norm) {
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) {
      const int row = 16 * ib + i;
      float dq = 0.f, dk = 0.f;
#pragma unroll
      for (int nb = 0; nb < NBW; ++nb) {
        const int n = 16 * (w * NBW + nb) + 4 * g;
        const u32x2 qv = *reinterpret_cast<const u32x2*>(sQ + key_at<NT>(row, n));
        const u32x2 kv = *reinterpret_cast<const u32x2*>(sK + key_at<NT>(row, n));
        const f32x4 x = dQ[nb][ib], y = dK[nb][ib];
        dq += x[0] * bf_lo(qv.x) + x[1] * bf_hi(qv.x) + x[2] * bf_lo(qv.y) + x[3] * bf_hi(qv.y);
        dk += y[0] * bf_lo(kv.x) + y[1] * bf_hi(kv.x) + y[2] * bf_lo(kv.y) + y[3] * bf_hi(kv.y);
      }
      dq = sum_across16(dq), dk = sum_across16(dk);
      if (g == 0) {
        s_in[w][row] = dq;
        s_out[w][row] = dk;
      }
    }
  }
  __syncthreads();
  const Rows oq(b.dq + pc.r0 * b.dq_ld + gn, b.dq_ld, rows, a.N, 2), ok(b.dk + pc.r0 * b.dk_ld + gn, b.dk_ld, rows, a.N, 2);
#pragma unroll
  for (int ib = 0; ib < 4; ++ib) {
    const int row = 16 * ib + i;
    const float fq = s_qn[row], fk = s_kn[row];
    float dq = 0.f, dk = 0.f;
    if (d.qk_norm) {
#pragma unroll
      for (int k = 0; k < WAVES; ++k) {
        dq += s_in[k][row];
        dk += s_out[k][row];
      }
      dq *= fq * fq * fq;
      dk *= fk * fk * fk;
    }
#pragma unroll
    for (int nb = 0; nb < NBW; ++nb) {
      const int n = 16 * (w * NBW + nb) + 4 * g;
      const u32x2 qv = *reinterpret_cast<const u32x2*>(sQ + key_at<NT>(row, n));
      const u32x2 kv = *reinterpret_cast<const u32x2*>(sK + key_at<NT>(row, n));
      const f32x4 x = dQ[nb][ib] * fq - f32x4{bf_lo(qv.x), bf_hi(qv.x), bf_lo(qv.y), bf_hi(qv.y)} * dq;
      const f32x4 y = dK[nb][ib] * fk - f32x4{bf_lo(kv.x), bf_hi(kv.x), bf_lo(kv.y), bf_hi(kv.y)} * dk;
      store4<VEC>(oq, (uint32_t)b.dq_ld, row, n, a.N, u32x2{pk_bf16(x[0], x[1]), pk_bf16(x[2], x[3])});
      store4<VEC>(ok, (uint32_t)b.dk_ld, row, n, a.N, u32x2{pk_bf16(y[0], y[1]), pk_bf16(y[2], y[3])});
    }
  }
}

// dA, d(dt_bias) of one head: the chunks' sums, 256 strided subsets and then a fixed tree
__global__ __launch_bounds__(256) void delta_head_reduce_kernel(DeltaBwdArgs b, int64_t ids) {
  __shared__ float lds[4][2];
  const int h = blockIdx.x, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  float s[2] = {0.f, 0.f};
  for (int64_t id = threadIdx.x; id < ids; id += 256) {
    const float* src = b.head_part + (id * b.d.s.H + h) * 2;
    s[0] += src[0];
    s[1] += src[1];
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float v = wave_sum(s[e]);
    if (lane == 0) lds[w][e] = v;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    const int e = threadIdx.x;
    float* dst = e == 0 ? b.dA : b.dbias;
    if (dst) dst[h] = lds[0][e] + lds[1][e] + lds[2][e] + lds[3][e];
  }
}

template <int NT, bool VEC>
static hipError_t launch(const DeltaBwdArgs& b, hipStream_t s) {
  const ScanArgs& a = b.d.s;
  const int64_t ids = b.d.n_chunk_slots + a.q.nseq;
  const dim3 blocks((uint32_t)(ids * a.G));
  delta_walks_kernel<NT, VEC><<<dim3((uint32_t)unit_blocks(a.q.nseq, a.H, a.G, a.ptiles, 1), 2), kWalkThreads, 0, s>>>(b);
  if (a.q.rows > 0) {
    if constexpr (NT > 128) delta_scan_bwd_wide_kernel<NT, 8, VEC><<<blocks, 512, 0, s>>>(b);
    else delta_scan_bwd_kernel<NT, 2, VEC><<<blocks, 8 * NT, 0, s>>>(b);
  }
  delta_head_reduce_kernel<<<dim3((uint32_t)a.H), 256, 0, s>>>(b, a.q.rows > 0 ? ids : 0);
  return hipGetLastError();
}

hipError_t launch_delta_bwd(const DeltaBwdArgs& b, bool vec, hipStream_t s) {
  if (b.d.s.q.nseq == 0) {  // no sequences: the parameters' gradients are zero
    delta_head_reduce_kernel<<<dim3((uint32_t)b.d.s.H), 256, 0, s>>>(b, 0);
    return hipGetLastError();
  }
  if (b.d.s.q.rows > 0) {
    const hipError_t e = launch_delta_chunks(b.d, b.rec_rev, vec, s);
    if (e != hipSuccess) return e;
  }
  switch (state_tile(b.d.s.N)) {
    case 64: return vec ? launch<64, true>(b, s) : launch<64, false>(b, s);
    case 128: return vec ? launch<128, true>(b, s) : launch<128, false>(b, s);
    default: return vec ? launch<256, true>(b, s) : launch<256, false>(b, s);
  }
}

}  // namespace cssm
