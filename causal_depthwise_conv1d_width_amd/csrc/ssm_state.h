// ssm_state.h -- the walk of the state alone, over the chunks of a piece, forward or in reverse.
//
//   forward  S' = e^{L_Q} S + sum_j e^{L_Q - L_j} dt_j x_j B_j^T        (u = x, v = B)
//   reverse  T' = e^{L_Q} T + sum_i e^{L_i} dy_i C_i^T                   (u = dy, v = C)
//
// with L the inclusive prefix sums of l_t = dt_t A over the chunk.  States are FP32 results held in
// registers over the whole walk; the weights multiply u in FP32, and the product enters the matrix
// instructions as PARTS bf16 parts.  Backward, three: a state has FP32's precision (a gradient of initial states
// was 2.5e-6 off with two, 1.4e-7 with three, for 1% of the time).  The forward scan's states take two, 2^-16 of a
// term.  Decays to the chunk's end are summed from the end, so that the last tokens of a fast-decaying chunk
// keep exact weights.
#pragma once

#include "ssm_device.h"

namespace cssm {

struct StateArgs {
  ScanArgs s;              // sequences, pieces, decays, head counts, slot mapping
  const uint16_t* u;       // [rows, H, P]
  const uint16_t* v;       // [rows, G, N]
  int64_t u_ld, v_ld;
  const float* start;      // state before the walk [slot or seq, H, P, N], nullptr: zeros
  float* end;              // reverse: state after the walk at the sequence's start, or nullptr
  float* piece;            // [item, H * ptiles, 64, NT]
  float* decay;            // [item, H]: log2 decays of pieces, this walk's own
  float* store;            // chunk states (STORE)
  int64_t n_chunk_slots;
};

// Decays and step sizes of one chunk, computed by one wave with a row a lane from the raw steps, which
// are loaded a chunk ahead (they would otherwise stand at the head of every chunk, a memory round trip
// and a scan that all waves wait for).  Rows past the chunk's end have step 0.
struct RawStep {  // loaded as two halves and put together at use, so that nothing waits for it before
  uint16_t hi, lo;
};
__device__ __forceinline__ RawStep raw_step(const ScanArgs& a, int64_t c0, int rows, int row, int h) {
  const int size = a.dt_f32 ? 4 : 2;
  const Rows r(static_cast<const char*>(a.dt) + (c0 * a.dt_ld + h) * size, a.dt_ld, rows, 1, size);
  const uint32_t off = (uint32_t)row * (uint32_t)a.dt_ld * size;
  RawStep s;
  s.lo = __builtin_amdgcn_raw_buffer_load_b16(r.r, (int)off, 0, 0);
  s.hi = __builtin_amdgcn_raw_buffer_load_b16(r.r, (int)(off + size - 2), 0, 0);
  return s;
}
struct Rate {
  float A2, bias;  // A log2 e, and what is added to the raw step
  int softplus, f32;
  __device__ __forceinline__ Rate(const ScanArgs& a, int h)
      : A2(uniform(a.A[h] * kLog2e)), bias(a.bias ? uniform(a.bias[h]) : 0.f), softplus(a.softplus), f32(a.dt_f32) {}
  __device__ __forceinline__ float step(RawStep raw, bool in) const {
    const float v = __uint_as_float(((uint32_t)raw.hi << 16) | (f32 ? raw.lo : 0u));
    return in ? step_size(v + bias, softplus) : 0.f;
  }
  // A term of the 64-bit prefix sums whose differences are the exponents of M_ij.  FP32 sums would lose the slow
  // decays that follow a sudden one; a decay below 2^-(2^20) counts as that, still a zero, so that 64 of them leave
  // 27 bits behind the binary point and no infinities to subtract.  A NaN stays one.
  __device__ __forceinline__ double exponent(float d) const {
    const float l = d * A2;
    return (double)(l < -1048576.f ? -1048576.f : l);
  }
};

// The chunks of rows [r0, r1) in the order of the walk.
template <bool REV>
struct Chunks {
  int64_t r0, r1, c0, c1;
  __device__ __forceinline__ Chunks(int64_t r0_, int64_t r1_) : r0(r0_), r1(r1_) {
    if (REV) {
      c0 = (r1 - 1) & ~(int64_t)(kChunk - 1);
      if (c0 < r0) c0 = r0;
      c1 = r1;
    } else {
      c0 = r0;
      c1 = chunk_end(r0, r1);
    }
  }
  __device__ __forceinline__ bool last() const { return REV ? c0 <= r0 : c1 >= r1; }
  __device__ __forceinline__ Chunks next() const {
    Chunks n = *this;
    if (REV) {
      n.c1 = c0;
      n.c0 = (c0 - 1) & ~(int64_t)(kChunk - 1);
      if (n.c0 < r0) n.c0 = r0;
    } else {
      n.c0 = c1;
      n.c1 = chunk_end(c1, r1);
    }
    return n;
  }
  __device__ __forceinline__ int rows() const { return (int)(c1 - c0); }
};
// The chunk after c and its number of rows, 0 (nothing is read) after the last one.
template <bool REV>
__device__ __forceinline__ Chunks<REV> step_chunk(const Chunks<REV>& c, int& rows) {
  const bool last = rows == 0 || c.last();
  const Chunks<REV> n = last ? c : c.next();
  rows = last ? 0 : n.rows();
  return n;
}

// slot of a sequence's state, and whether it has one
__device__ __forceinline__ bool state_slot(const ScanArgs& a, int64_t seq, int64_t& slot) {
  slot = a.ci ? __builtin_amdgcn_readfirstlane(a.ci[seq]) : seq;
  if (!a.ci) return true;
  return slot >= 0 && slot < a.slots;
}
// no flags: all false for slots of a pool, all true for arrays of one state a sequence
__device__ __forceinline__ bool starts_from_state(const ScanArgs& a, int64_t seq) {
  return a.init && (a.has_init ? __builtin_amdgcn_readfirstlane(a.has_init[seq]) != 0 : a.ci == nullptr);
}

// The backward's walks (TURN) hold the state with a sign that turns from chunk to chunk of a piece, as does what they
// store.  Accumulated by matrix instructions, it comes out a little low, whatever its sign (by 0.09 * 2^-24 of its rms
// after 16 chunks).  With x, B and C that have a mean, such an offset of the adjoints adds up over all rows in dA,
// whose own terms cancel with dy of both signs: 0.8e-6 to 1.9e-6 of dA over 16384 rows, 1e-7 to 3e-7 with the turns,
// which cost nothing (the signs are those of the weights and of the decay).
__device__ __forceinline__ float turn_of(int64_t chunks) { return chunks & 1 ? -1.f : 1.f; }

// A block walks U units of a group (they share v), two waves a unit, each with 32 rows p of the state: a wave reads
// a v operand for two row blocks, which halves the shared memory traffic that bounds the walk.
// LOCAL: from zeros, the end state goes to the piece's place (pieces whose end nobody needs do nothing).
// STORE: from the piece's start state (or the sequence's), every chunk's start state goes to `store`.
template <int NT, int U>
struct StateShared {
  __align__(16) uint16_t u[U][64 * kLd<64, 16>];
  __align__(16) uint16_t v[64 * kLd<NT, 16>];
  __align__(16) float w[2][U][64];  // weights of this chunk and the next one, by unit
  float total[2][U];
};
template <int NT, int U, int PARTS, bool VEC, bool REV, bool STORE, bool TURN>
__device__ __forceinline__ void state_walk(const StateArgs& k, StateShared<NT, U>& sh) {
  constexpr int T = 128 * U, WU = 2;  // threads, and waves a unit
  constexpr int NB = NT / 16;         // 16-column blocks of the state, with two 16-row blocks a wave
  const ScanArgs& a = k.s;
  const int hp = a.H * a.ptiles;
  const Units<U> us(a, blockIdx.x);
  if (!us.ok) return;
  const int wave = wave_id(), un = wave / WU, w = wave % WU;
  const Unit me(a, us, un);
  const Piece pc = find_piece(a.q, us.item, a.seg, a.n_slots);
  const bool first = pc.r0 == pc.s, last = pc.r1 == pc.e;
  const int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15;
  const int p0 = w * 32;
  const int64_t state_at = ((pc.seq * a.H + me.h) * a.P + me.p_first) * a.N;
  float* place = k.piece + (us.item * hp + me.tile) * (64 * NT);
  const uint16_t* su = sh.u[un];
  const uint16_t* sv = sh.v;
  if (!pc.ok) {
    // an empty sequence's adjoint passes through
    if (REV && STORE && k.end && us.item >= a.n_slots) {
      for (int e = threadIdx.x % (64 * WU); e < me.pn * a.N; e += 64 * WU)
        k.end[state_at + e] = k.start ? k.start[state_at + e] : 0.f;
    }
    return;
  }
  if (!STORE && (REV ? first : last)) return;

  f32x4 S[2][NB];
#pragma unroll
  for (int pb = 0; pb < 2; ++pb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) S[pb][nb] = f32x4{0.f, 0.f, 0.f, 0.f};
  if constexpr (STORE) {
    if (a.seg > 0 && piece_count(pc.e - pc.s, a.seg) > 1) {
#pragma unroll
      for (int pb = 0; pb < 2; ++pb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int r = 0; r < 4; ++r) S[pb][nb][r] = place[(p0 + 16 * pb + 4 * g + r) * NT + 16 * nb + i];
    } else if (k.start) {
      const float* src = k.start + state_at;
#pragma unroll
      for (int pb = 0; pb < 2; ++pb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int p = p0 + 16 * pb + 4 * g + r, n = 16 * nb + i;
            if (p < me.pn && n < a.N) S[pb][nb][r] = src[(int64_t)p * a.N + n];
          }
    }
  }

  const Rate rate(a, me.h);
  const uint16_t* vb = k.v + (int64_t)us.group * a.N;
  float log_total = 0.f;
  RawStep raw{};
  TileRegs<64, T> tu[U];
  TileRegs<NT, T> tv;
  auto load = [&](const Chunks<REV>& c, int rows) {
    const Rows ur(k.u + c.c0 * k.u_ld, k.u_ld, rows, a.H * a.P, 2);
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const Unit o(a, us, q);
      load_tile<VEC>(tu[q], ur, (uint32_t)k.u_ld, o.pn, o.col);
    }
    load_tile<VEC>(tv, Rows(vb + c.c0 * k.v_ld, k.v_ld, rows, a.N, 2), (uint32_t)k.v_ld, a.N);
  };
  // a chunk's weights into buffer `at` by a unit's first wave; forward, a lane's row counts from the end
  const int my = REV ? lane : 63 - lane;
  auto weights = [&](int rows, int at, float sign) {
    const float d = rate.step(raw, my < rows);
    const float L = wave_prefix(d * rate.A2);
    // the rows after this one: the previous lane's sum
    const float v = REV ? ex2(L) : ex2(dpp0<0x138, 0xf>(L)) * d;
    sh.w[at][un][my] = TURN ? sign * v : v;
    if (lane == 63) sh.total[at][un] = L;
  };
  Chunks<REV> c(pc.r0, pc.r1);
  int rows = c.rows();
  float turn = 1.f;  // the state's sign before the chunk
  load(c, rows);
  raw = raw_step(a, c.c0, rows, my, me.h);
  if (w == 0) weights(rows, 0, -turn);
  Chunks<REV> after = c;
  int after_rows = rows;  // the chunk whose raw steps come next
  after = step_chunk(after, after_rows);
  raw = raw_step(a, after.c0, after_rows, my, me.h);
  for (int buf = 0;; buf ^= 1) {
#pragma unroll
    for (int q = 0; q < U; ++q) store_tile<16>(sh.u[q], tu[q]);
    store_tile<16>(sh.v, tv);
    __syncthreads();
    const int64_t here = c.c0;
    const float* sw = sh.w[buf][un];
    c = step_chunk(c, rows);  // rows == 0: that was the last one
    load(c, rows);
    if (w == 0) weights(rows, buf ^ 1, turn);  // the chunk after turns back
    after = step_chunk(after, after_rows);
    raw = raw_step(a, after.c0, after_rows, my, me.h);
    if constexpr (STORE) {  // operand order: [row half][n block of 16][p step of 32][lane] four FP32 values
      const int64_t id = here == pc.s ? k.n_chunk_slots + pc.seq : here >> 6;
      const Rows dst(k.store + (id * hp + me.tile) * (64 * NT), 64 * NT, 1, me.pn ? 64 * NT : 0, 4);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int pb = 0; pb < 2; ++pb)
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, S[pb][nb]), dst.r,
                                                 ((pb * (NT / 16) + nb) * 2 + w) * 1024 + lane * 16, 0, 0);
    }
    const float total = sh.total[buf][un];
    log_total += total;
    const float et = TURN ? -ex2(total) : ex2(total);
    if (TURN) turn = -turn;
#pragma unroll
    for (int pb = 0; pb < 2; ++pb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) S[pb][nb] *= et;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const f32x4 wa = *reinterpret_cast<const f32x4*>(sw + 32 * ks + 4 * g);
      const f32x4 wb = *reinterpret_cast<const f32x4*>(sw + 32 * ks + 16 + 4 * g);
      Parts x[2];
#pragma unroll
      for (int pb = 0; pb < 2; ++pb) x[pb] = split_scaled(op_cols<64, 16>(su, 32 * ks, p0 + 16 * pb, lane), wa, wb);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const bf16x8 b = op_cols<NT, 16>(sv, 32 * ks, 16 * nb, lane);
#pragma unroll
        for (int q = 0; q < PARTS; ++q)
#pragma unroll
          for (int pb = 0; pb < 2; ++pb) S[pb][nb] = mma(x[pb].p[q], b, S[pb][nb]);
      }
    }
    if (rows == 0) break;
    __syncthreads();
  }

  if (me.pn == 0) return;
  if constexpr (!STORE) {
#pragma unroll
    for (int pb = 0; pb < 2; ++pb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int r = 0; r < 4; ++r) place[(p0 + 16 * pb + 4 * g + r) * NT + 16 * nb + i] = turn * S[pb][nb][r];
    if (w == 0 && lane == 0 && me.p_first == 0) k.decay[us.item * a.H + me.h] = log_total;
  } else if (REV && first && k.end) {
    float* dst = k.end + state_at;
#pragma unroll
    for (int pb = 0; pb < 2; ++pb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int p = p0 + 16 * pb + 4 * g + r, n = 16 * nb + i;
          if (p < me.pn && n < a.N) dst[(int64_t)p * a.N + n] = turn * S[pb][nb][r];
        }
  }
}

template <int NT, int U, bool VEC>
__global__ __launch_bounds__(128 * U, U > 2 || NT <= 128 ? 2 : 1) void ssm_state_local_kernel(StateArgs k) {
  __shared__ StateShared<NT, U> sh;
  state_walk<NT, U, 2, VEC, false, false, false>(k, sh);
}

// Local end states of a sequence's pieces -> start states, in place, in the order of the walk:
// start[m + 1] = decay[m] start[m] + local[m].  Sequences of one piece start from their own state.  A thread
// takes four columns of a state; gridDim.y blocks share a sequence (few, where there are many sequences: blocks
// with nothing to do cost more than the copies themselves).
template <int NT, bool REV>
__global__ __launch_bounds__(1024) void ssm_join_kernel(StateArgs k) {
  const ScanArgs& a = k.s;
  constexpr int kPer = 64 * NT / 4;  // threads' worth of a state tile
  const int hp = a.H * a.ptiles;
  const int64_t seq = blockIdx.x;
  int64_t s, e;
  seq_bounds(a.q, seq, s, e);
  const int64_t pieces = e > s ? piece_count(e - s, a.seg) : 0;
  if (pieces <= 1) return;
  int64_t slot = seq;
  const bool live = state_slot(a, seq, slot);
  const bool from = REV ? k.start != nullptr : live && starts_from_state(a, seq);
  for (int w = blockIdx.y * 1024 + threadIdx.x; w < hp * kPer; w += gridDim.y * 1024) {
    const int tile = w / kPer, at = w % kPer * 4, h = tile / a.ptiles, p = tile % a.ptiles * kPTile + at / NT, n = at % NT;
    f32x4 S = {0.f, 0.f, 0.f, 0.f};
    if (from && p < a.P) {
      const float* src = k.start + (REV ? seq * (int64_t)a.H * a.P * a.N : slot * a.s_slot) + ((int64_t)h * a.P + p) * a.N;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < a.N) S[r] = src[n + r];
    }
    for (int64_t m = 0; m < pieces; ++m) {
      const int64_t item = piece_item(a.q, seq, s, a.seg, a.n_slots, REV ? pieces - 1 - m : m);
      f32x4* place = reinterpret_cast<f32x4*>(k.piece + (item * hp + tile) * (64 * NT) + at);
      const f32x4 local = m + 1 < pieces ? *place : S;
      *place = S;
      if (m + 1 < pieces) S = S * ex2(k.decay[item * a.H + h]) + local;
    }
  }
}
inline dim3 join_grid(const ScanArgs& a, int NT) {
  const int64_t all = ((int64_t)a.H * a.ptiles * 64 * NT / 4 + 1023) / 1024;
  int64_t y = 2048 / a.q.nseq;
  y = y < 4 ? 4 : y;
  return dim3((uint32_t)a.q.nseq, (uint32_t)(y < all ? y : all));
}

}  // namespace cssm
