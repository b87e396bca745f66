// ssm_device.h -- device-side building blocks of the scan, step and norm kernels (library-internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssm_launch.h"

namespace cssm {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// 16- and 8-byte accesses at 2-byte aligned addresses: one instruction each in the unaligned access
// mode the HSA runtime sets, so odd row strides and views into wider rows need no separate path.
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ float bf_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
// two FP32 -> two bf16, round to nearest even
__device__ __forceinline__ uint32_t pk_bf16(float a, float b) {
  f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}
__device__ __forceinline__ uint16_t to_bf16(float a) { return (uint16_t)pk_bf16(a, 0.f); }

// 2^x by the hardware instruction (about 1 ulp)
__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.f + ex2(-kLog2e * z)); }

// The step size: v, or log(1 + e^v) = max(v, 0) + log1p(e^-|v|).  The exponent's argument keeps its low
// part, and log1p(u) = log(w) u / (w - 1) with w = 1 + u rounded: right to a few ulp at every v.  Both
// comparisons of the result are false for a NaN, which is kept.
__device__ __forceinline__ float step_size(float v, int softplus) {
  if (!softplus) return v;
  const float a = __builtin_fabsf(v), t = a * kLog2e;
  const float rest = __builtin_fmaf(a, kLog2e, -t) + a * 1.92596303e-8f;  // log2 e - its FP32 value
  const float u = ex2(-t) * __builtin_fmaf(rest, -0.693147181f, 1.f);
  const float w = 1.f + u, m = w - 1.f;
  const float l = m > 0.f ? __builtin_amdgcn_logf(w) * 0.693147181f * u * __builtin_amdgcn_rcpf(m) : u;
  return (v <= 0.f ? 0.f : v) + (a >= 126.f ? 0.f : l);
}

__device__ __forceinline__ float load_num(const void* p, int64_t i, int f32) {
  return f32 ? static_cast<const float*>(p)[i] : bf_f32(static_cast<const uint16_t*>(p)[i]);
}

// ------------------------------------------------------------------ wave reductions and scans
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float dpp0(float v) {  // 0 where the source lane is masked or out of its row
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, ROW_MASK, 0xf, true));
}
// inclusive prefix sum over the wave: shifts inside rows of 16 lanes, then the rows' last lanes broadcast
__device__ __forceinline__ float wave_prefix(float v) {
  v += dpp0<0x111, 0xf>(v);
  v += dpp0<0x112, 0xf>(v);
  v += dpp0<0x114, 0xf>(v);
  v += dpp0<0x118, 0xf>(v);
  v += dpp0<0x142, 0xa>(v);
  v += dpp0<0x143, 0xc>(v);
  return v;
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ double dpp0(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROW_MASK, 0xf, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROW_MASK, 0xf, true);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double wave_prefix(double v) {
  v += dpp0<0x111, 0xf>(v);
  v += dpp0<0x112, 0xf>(v);
  v += dpp0<0x114, 0xf>(v);
  v += dpp0<0x118, 0xf>(v);
  v += dpp0<0x142, 0xa>(v);
  v += dpp0<0x143, 0xc>(v);
  return v;
}
// sum over the 16 lanes of each row; valid in lane 15 of the row
__device__ __forceinline__ float row16_sum(float v) {
  v += dpp0<0x111, 0xf>(v);
  v += dpp0<0x112, 0xf>(v);
  v += dpp0<0x114, 0xf>(v);
  v += dpp0<0x118, 0xf>(v);
  return v;
}
// sums over the lanes from this one to the end of its row; the row's sum in lane 0 of the row
__device__ __forceinline__ float row16_suffix(float v) {
  v += dpp0<0x101, 0xf>(v);
  v += dpp0<0x102, 0xf>(v);
  v += dpp0<0x104, 0xf>(v);
  v += dpp0<0x108, 0xf>(v);
  return v;
}
__device__ __forceinline__ float wave_sum(float v) { return lane_value(wave_prefix(v), 63); }

// ------------------------------------------------------------------ sequences, pieces, chunks
// Everything here is the same in all lanes; values that come from memory are moved to scalar registers,
// so that row numbers and tile bases cost no vector registers or instructions.
__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ float uniform(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readfirstlane((int)__float_as_uint(v)));
}
struct Piece {
  int64_t seq, s, e;  // the sequence's rows [s, e)
  int64_t r0, r1;     // this piece's rows
  bool ok;            // the item is a piece (false: nothing to do)
};

__device__ __forceinline__ int64_t cu_at(const Seqs& q, int64_t k) {
  const int64_t v = __builtin_amdgcn_readfirstlane(q.cu[k]);
  return v < 0 ? 0 : (v > q.rows ? q.rows : v);
}
__device__ __forceinline__ void seq_bounds(const Seqs& q, int64_t i, int64_t& s, int64_t& e) {
  if (q.cu) {
    s = cu_at(q, i);
    e = cu_at(q, i + 1);
  } else {
    s = i * q.seqlen;
    e = s + q.seqlen;
  }
}

// The sequence holding `row` (-1: none): a 64-ary search over the offsets, one probe a lane.
__device__ __forceinline__ int64_t seq_of_row(const Seqs& q, int64_t row) {
  if (!q.cu) return row / q.seqlen;
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, len = q.nseq + 1;  // offsets before lo are <= row, offsets from lo + len on are > row
  while (len > 64) {
    const int64_t step = (len + 63) / 64;
    const int64_t k = (lane + 1) * step;
    const bool le = q.cu[lo + (k < len ? k : len) - 1] <= row;
    const int64_t skip = (int64_t)__popcll(__ballot(le)) * step;
    if (skip >= len) {
      lo += len;
      len = 0;
    } else {
      lo += skip;
      len = len - skip < step ? len - skip : step;
    }
  }
  const bool le = lane < len && q.cu[lo + (lane < len ? lane : 0)] <= row;
  return lo + __popcll(__ballot(le)) - 1;
}

// Chunk `id` of the packed rows: ids below n_slots are the chunks that begin at row id * kChunk inside a
// sequence, id n_slots + i is sequence i's first.
__device__ __forceinline__ Piece find_chunk(const Seqs& q, int64_t id, int64_t n_slots) {
  Piece p;
  p.ok = false;
  p.s = p.e = p.r1 = 0;
  if (id >= n_slots) {
    p.seq = id - n_slots;
    seq_bounds(q, p.seq, p.s, p.e);
    p.r0 = p.s;
    p.ok = p.e > p.s;
  } else {
    p.r0 = id * kChunk;
    p.seq = seq_of_row(q, p.r0);
    if (p.seq < 0 || p.seq >= q.nseq) return p;
    seq_bounds(q, p.seq, p.s, p.e);
    p.ok = p.r0 > p.s && p.r0 < p.e;
  }
  const int64_t cut = (p.r0 & ~(int64_t)(kChunk - 1)) + kChunk;
  p.r1 = cut < p.e ? cut : p.e;
  return p;
}

// The pieces of the scan: a sequence is cut every 2^seg rows from its start, rounded down to whole chunks.
// Piece j >= 1 of the sequence at row s is item (s >> seg) + j: cuts of one sequence are 2^seg rows apart and
// those of the next one begin 2^seg rows after its start, so no two share an item, and row item << seg lies in
// the item's sequence.  Batch rows all have the same number of pieces, numbered without gaps, so that a
// launch has no idle blocks.  seg == 0: whole sequences.
__device__ __forceinline__ int64_t piece_count(int64_t rows, int seg) { return (rows + ((int64_t)1 << seg) - 1) >> seg; }
__device__ __forceinline__ int64_t piece_item(const Seqs& q, int64_t seq, int64_t s, int seg, int64_t n_slots, int64_t j) {
  if (j == 0) return n_slots + seq;
  return q.cu ? (s >> seg) + j : seq * (piece_count(q.seqlen, seg) - 1) + j - 1;
}
__device__ __forceinline__ Piece find_piece(const Seqs& q, int64_t it, int seg, int64_t n_slots) {
  Piece p;
  p.ok = false;
  p.s = p.e = p.r0 = p.r1 = 0;
  int64_t j = 0;
  if (it >= n_slots) {
    p.seq = it - n_slots;
  } else if (q.cu) {
    p.seq = seq_of_row(q, it << seg);
    if (p.seq < 0 || p.seq >= q.nseq) return p;
  } else {  // n_slots and so `it` is below 2^31
    const uint32_t more = (uint32_t)(piece_count(q.seqlen, seg) - 1);
    p.seq = (uint32_t)it / more;
    j = (uint32_t)it % more + 1;
  }
  seq_bounds(q, p.seq, p.s, p.e);
  if (seg == 0) {
    p.r0 = p.s;
    p.r1 = p.e;
    p.ok = p.e > p.s;
    return p;
  }
  if (it < n_slots && q.cu) j = it - (p.s >> seg);
  const int64_t from = p.s + (j << seg), to = p.s + ((j + 1) << seg);
  p.r0 = j == 0 ? p.s : from & ~(int64_t)(kChunk - 1);
  p.r1 = to < p.e ? to & ~(int64_t)(kChunk - 1) : p.e;
  p.ok = from < p.e && (j > 0 || it >= n_slots);
  return p;
}

// The rows of the piece that a chunk at `row` of the sequence [s, e) belongs to.
__device__ __forceinline__ void piece_around(int64_t s, int64_t e, int64_t row, int seg, int64_t& r0, int64_t& r1) {
  r0 = s, r1 = e;
  if (seg == 0) return;
  const int64_t last = (e - 1 - s) >> seg, at = (row + kChunk - 1 - s) >> seg, j = at < last ? at : last;
  if (j > 0) r0 = (s + (j << seg)) & ~(int64_t)(kChunk - 1);
  if (j < last) r1 = (s + ((j + 1) << seg)) & ~(int64_t)(kChunk - 1);
}

__device__ __forceinline__ int64_t chunk_end(int64_t r, int64_t r1) {
  const int64_t c = (r & ~(int64_t)(kChunk - 1)) + kChunk;
  return c < r1 ? c : r1;
}

// ------------------------------------------------------------------ tiles of 64 rows in shared memory
// [64][W] bf16, row-major, rows 16 bytes further apart than their length: 16 rows' same 16-byte piece,
// and the transposing reads of 4 rows by 16 columns a quarter wave, then fall on different banks (64
// of 4 bytes), and every address is one lane's base plus a constant.  (A permutation of each row's pieces
// has no such constants: its addresses took over a hundred registers.)
// PAD: 8 elements suit reads of a 16-byte or two 8-byte pieces of 16 rows, 16 the transposing reads (two
// quarter waves at a time: 8 rows of 32 bytes).
template <int W, int PAD = 8>
constexpr int kLd = W + PAD;
template <int W, int PAD = 8>
__device__ __forceinline__ int at(int row, int col) {
  return row * kLd<W, PAD> + col;
}

// this thread's wave, as a scalar (the compiler takes threadIdx.x / 64 for a value of each lane)
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// a tile in the registers of T threads
template <int W, int T>
struct TileRegs {
  u32x4 v[W * 8 / T];
};

// The rows of one chunk of a global array, as a buffer: offsets past its end read zeros and write nothing.
// Every load and store of the chunk loops goes through one, without a test around it: with a store under
// a branch the compiler can no longer count what is in flight and waits for all of it, the next chunk's
// loads and the stores' completion, at every chunk.  Offsets are 32-bit bytes from the chunk's first row
// (the host keeps 63 row strides under 2^32 bytes) and do not change from chunk to chunk.
struct Rows {
  __amdgpu_buffer_rsrc_t r;
  // nrows rows of ncols columns of `size` bytes, ld columns apart; no rows or columns: everything is outside
  __device__ __forceinline__ Rows(const void* first, int64_t ld, int nrows, int ncols, int size) {
    const uint32_t bytes = nrows > 0 && ncols > 0 ? (uint32_t)(((nrows - 1) * ld + ncols) * size) : 0u;
    r = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(first), 0, (int)bytes, 0x00020000);
  }
};
constexpr uint32_t kOutside = 0xffffff00u;  // an offset past every buffer's end

// Columns [0, ncols) of a chunk's rows, from column `col0` of the buffer on, into registers of T
// threads, zeros outside.  VEC: ncols is a multiple of 8.
template <bool VEC, int W, int T>
__device__ __forceinline__ void load_tile(TileRegs<W, T>& t, const Rows& rows, uint32_t ld, int ncols, uint32_t col0 = 0) {
#pragma unroll
  for (int k = 0; k < W * 8 / T; ++k) {
    const int q = threadIdx.x + T * k, row = q / (W / 8), c = (q % (W / 8)) * 8;
    const uint32_t off = (row * ld + c) * 2 + col0 * 2;
    if constexpr (VEC) {
      t.v[k] = __builtin_amdgcn_raw_buffer_load_b128(rows.r, (int)(c < ncols ? off : kOutside), 0, 0);
    } else {
      u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t u = __builtin_amdgcn_raw_buffer_load_b16(rows.r, (int)(c + e < ncols ? off + 2 * e : kOutside), 0, 0);
        v[e >> 1] |= u << (16 * (e & 1));
      }
      t.v[k] = v;
    }
  }
}

// Four bf16 columns c .. c + 3 (those below ncols) of a row
template <bool VEC>
__device__ __forceinline__ void store4(const Rows& rows, uint32_t ld, int row, int c, int ncols, u32x2 v) {
  const uint32_t off = (row * ld + c) * 2;
  if constexpr (VEC) {
    __builtin_amdgcn_raw_buffer_store_b64(v, rows.r, (int)(c < ncols ? off : kOutside), 0, 0);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(v[e >> 1] >> (16 * (e & 1))), rows.r,
                                            (int)(c + e < ncols ? off + 2 * e : kOutside), 0, 0);
  }
}

template <int PAD = 8, int W, int T>
__device__ __forceinline__ void store_tile(uint16_t* lds, const TileRegs<W, T>& t) {
#pragma unroll
  for (int k = 0; k < W * 8 / T; ++k) {
    const int q = threadIdx.x + T * k;
    *reinterpret_cast<u32x4*>(lds + at<W, PAD>(q / (W / 8), q % (W / 8) * 8)) = t.v[k];
  }
}

// What a block of the scan or of the state walk works on: U units (64 columns of one head each) of one
// group, which share the group's B and C rows; a group's last block may have fewer.  Workgroups are dealt to
// the 8 XCDs in turn, each with its own L2: the blocks of one piece and group stay on one XCD, and pieces and
// groups go to the XCDs in turn, so that long and absent pieces spread over them.
template <int U>
struct Units {
  int64_t item;
  int group, units, first, count;  // units first .. first + count - 1 of the group's
  bool ok;
  __device__ __forceinline__ Units(const ScanArgs& a, uint32_t block) {
    units = (uint32_t)a.H / (uint32_t)a.G * a.ptiles;
    const uint32_t sets = (units + U - 1) / U, eighth = block / 8, k = eighth / sets;
    const uint32_t set = k * 8 + block % 8;  // (piece, group)
    const uint32_t it = set / (uint32_t)a.G;
    item = it;
    group = set - it * a.G;
    first = (eighth - k * sets) * U;
    count = units - first < U ? units - first : U;
    ok = item < a.n_slots + a.q.nseq;
  }
};
struct Unit {
  int tile, h, p_first, pn;  // head_tile over all heads, head, first column of the head, columns
  uint32_t col;              // first column of a row of x
  // unit k of the block; past the block's last one it has no columns
  template <int U>
  __device__ __forceinline__ Unit(const ScanArgs& a, const Units<U>& u, int k) {
    const bool in = k < u.count;
    tile = u.group * u.units + u.first + (in ? k : 0);
    h = a.ptiles == 1 ? tile : (uint32_t)tile / (uint32_t)a.ptiles;
    p_first = (tile - h * a.ptiles) * kPTile;
    pn = !in ? 0 : (a.P - p_first < kPTile ? a.P - p_first : kPTile);
    col = (uint32_t)h * a.P + p_first;
  }
};

// Keeps the compiler from moving one phase's loads and products into another: with them mixed, the
// kernels need more registers than 16 waves a CU leave them.
__device__ __forceinline__ void phase() { __builtin_amdgcn_sched_barrier(0); }

// The ten 16 x 16 blocks (ib, jb) of a 64 x 64 tile up to the diagonal: (3, 0..3), (2, 0..2), (1, 0), (1, 1), (0, 0)
__device__ __forceinline__ void lower_block(int k, int& ib, int& jb) {
  ib = k < 4 ? 3 : (k < 7 ? 2 : (k < 9 ? 1 : 0));
  jb = k < 4 ? k : (k < 7 ? k - 4 : (k < 9 ? k - 7 : 0));
}

// ------------------------------------------------------------------ matrix operands
// A lane number the compiler cannot follow out of a loop: addresses computed from it are made again in every
// pass (a few instructions) instead of all being kept, or spilled, over the whole loop.
__device__ __forceinline__ int fresh(int lane) {
  asm volatile("" : "+v"(lane));
  return lane;
}

// 16x16x32 bf16: lane l holds index l % 16 of its operand and 8 of the 32 contracted positions; the
// result has the first operand's index in the registers (4 * (l / 16) + r) and the second's in the
// lanes.  The contracted positions may be taken in any order that both operands share.  Two orders
// are used: "straight", positions 8 * (l / 16) + e, and "split", positions 4 * (l / 16) + e and
// 16 + 4 * (l / 16) + e, which is how results and transposing reads come.
__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
// index = rows of the tile, contracted = columns k0 .. k0 + 31, straight
template <int W, int PAD = 8>
__device__ __forceinline__ bf16x8 op_straight(const uint16_t* lds, int row0, int k0, int l) {
  return *reinterpret_cast<const bf16x8*>(lds + at<W, PAD>(row0 + (l & 15), k0 + (l >> 4) * 8));
}
// the same, split
template <int W, int PAD = 8>
__device__ __forceinline__ bf16x8 op_split(const uint16_t* lds, int row0, int k0, int l) {
  const int row = row0 + (l & 15), c = k0 + (l >> 4) * 4;
  const u32x2 a = *reinterpret_cast<const u32x2*>(lds + at<W, PAD>(row, c));
  const u32x2 b = *reinterpret_cast<const u32x2*>(lds + at<W, PAD>(row, c + 16));
  const u32x4 v = {a.x, a.y, b.x, b.y};
  return __builtin_bit_cast(bf16x8, v);
}
// index = columns c0 .. c0 + 15, contracted = rows k0 .. k0 + 31, split (the transposing read gives
// lane i of 16 column i of the 4 rows x 16 columns that the 16 lanes address)
template <int W, int PAD = 8>
__device__ __forceinline__ bf16x8 op_cols(const uint16_t* lds, int k0, int c0, int l) {
  const int row = k0 + (l >> 4) * 4 + ((l & 15) >> 2), c = c0 + (l & 3) * 4;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds + at<W, PAD>(row, c)));
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds + at<W, PAD>(row + 16, c)));
  const u32x2 ua = __builtin_bit_cast(u32x2, a), ub = __builtin_bit_cast(u32x2, b);
  const u32x4 v = {ua.x, ua.y, ub.x, ub.y};
  return __builtin_bit_cast(bf16x8, v);
}
// results of two neighbouring blocks (registers = contracted) as an operand, split
__device__ __forceinline__ bf16x8 op_result(f32x4 a, f32x4 b) {
  const u32x4 v = {pk_bf16(a[0], a[1]), pk_bf16(a[2], a[3]), pk_bf16(b[0], b[1]), pk_bf16(b[2], b[3])};
  return __builtin_bit_cast(bf16x8, v);
}
// An FP32 operand as the sum of three bf16 ones: 8 bits each, so that its products keep FP32's 24 (with
// the first two, 16)
struct Parts {
  bf16x8 p[3];
};
__device__ __forceinline__ Parts split(f32x4 a, f32x4 b) {
  u32x4 q[3];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float x = e < 2 ? a[2 * e] : b[2 * e - 4], y = e < 2 ? a[2 * e + 1] : b[2 * e - 3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      q[k][e] = pk_bf16(x, y);
      x -= bf_lo(q[k][e]);
      y -= bf_hi(q[k][e]);
    }
  }
  return Parts{{__builtin_bit_cast(bf16x8, q[0]), __builtin_bit_cast(bf16x8, q[1]), __builtin_bit_cast(bf16x8, q[2])}};
}
// w[e] * v[e] in FP32, in three parts
__device__ __forceinline__ Parts split_scaled(bf16x8 v, f32x4 wa, f32x4 wb) {
  const u32x4 u = __builtin_bit_cast(u32x4, v);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    wa[2 * e] *= bf_lo(u[e]);
    wa[2 * e + 1] *= bf_hi(u[e]);
    wb[2 * e] *= bf_lo(u[e + 2]);
    wb[2 * e + 1] *= bf_hi(u[e + 2]);
  }
  return split(wa, wb);
}

// ------------------------------------------------------------------ XCD-aware block order
// Workgroups are dealt to the 8 XCDs in turn, each with its own L2.  Every XCD takes one contiguous
// range of logical blocks, so the heads that share a group's B and C rows meet in one L2.
__device__ __forceinline__ uint32_t xcd_block(uint32_t b, uint32_t nb) {
  const uint32_t q = nb / 8, r = nb % 8, x = b % 8, i = b / 8;
  return x < r ? x * (q + 1) + i : r * (q + 1) + (x - r) * q + i;
}

}  // namespace cssm
