// delta_device.h -- what the delta rule's chunk kernel and walks share: FP32 operands as two fp16 parts, the chunks' records.
#pragma once

#include "delta_launch.h"
#include "ssm_state.h"

namespace cssm {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// FP32 operands enter the matrix instructions as two fp16 parts: 22 bits of the values near the largest one and an
// absolute 2^-25 below, after a power of two that brings the largest of a column (or row, or tile) to 2^t.  Three
// bf16 parts hold 24 bits without a scale, but take 3 products for 2 (6 for 3, both operands being FP32) and twice the
// instructions to make: 4 x 4096 rows of 32 heads of 128 x 128 took 571 us forward, with these 454 (both before the walk was split
// over more waves).  The maxima cost a few instructions a value.  bf16 inputs are exact in fp16 but for values below 2^-14 of their row's
// largest, which keep 2^-25 of it.
struct Halves {
  f16x8 hi, lo;
};
__device__ __forceinline__ uint32_t pk_f16(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}
// what the two halves of u leave of a and b
__device__ __forceinline__ uint32_t rest_f16(float a, float b, uint32_t u) {
  const f16x2 h = __builtin_bit_cast(f16x2, u);
  float minus = -1.f;
  asm("" : "+s"(minus));  // a factor the compiler does not know: an fma takes h's halves as they are, a difference converts them
  return pk_f16(__builtin_fmaf((float)h.x, minus, a), __builtin_fmaf((float)h.y, minus, b));
}
__device__ __forceinline__ f16x8 as_f16(u32x4 v) { return __builtin_bit_cast(f16x8, v); }
__device__ __forceinline__ f16x8 as_f16(bf16x8 v) { return __builtin_bit_cast(f16x8, v); }  // the bits of an operand read
__device__ __forceinline__ f16x8 halves_hi(f32x4 a, f32x4 b) {
  return as_f16(u32x4{pk_f16(a[0], a[1]), pk_f16(a[2], a[3]), pk_f16(b[0], b[1]), pk_f16(b[2], b[3])});
}
__device__ __forceinline__ Halves halves(f32x4 a, f32x4 b) {
  const u32x4 h = {pk_f16(a[0], a[1]), pk_f16(a[2], a[3]), pk_f16(b[0], b[1]), pk_f16(b[2], b[3])};
  const u32x4 l = {rest_f16(a[0], a[1], h[0]), rest_f16(a[2], a[3], h[1]), rest_f16(b[0], b[1], h[2]), rest_f16(b[2], b[3], h[3])};
  return Halves{as_f16(h), as_f16(l)};
}
__device__ __forceinline__ f32x4 mmah(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma2(f16x8 a, const Halves& b, f32x4 c) { return mmah(a, b.hi, mmah(a, b.lo, c)); }
__device__ __forceinline__ f32x4 mma2(const Halves& a, f16x8 b, f32x4 c) { return mmah(a.hi, b, mmah(a.lo, b, c)); }
__device__ __forceinline__ f32x4 mma3(const Halves& a, const Halves& b, f32x4 c) {
  return mmah(a.hi, b.hi, mmah(a.hi, b.lo, mmah(a.lo, b.hi, c)));
}

// Has a value computed here: sums that only the next pass needs otherwise move behind the following branches, and what they are
// made of stays in registers until then.
__device__ __forceinline__ void here(float& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void here(f32x4& v) { asm volatile("" : "+v"(v)); }

// The power of two that brings m > 0 to [2^TO, 2^(TO + 1)), and its inverse.  Any m: of zeros and the smallest values the
// largest possible one, of an infinity or NaN a small one.
struct Pow2 {
  float up, down;
};
template <int TO>
__device__ __forceinline__ Pow2 bring_to(float m) {
  const uint32_t e = __float_as_uint(m) >> 23 & 0xff, c = e < TO + 1 ? TO + 1 : e;
  return Pow2{__uint_as_float((254 + TO - c) << 23), __uint_as_float((c - TO) << 23)};
}
__device__ __forceinline__ float max4(float m, f32x4 v) {
  m = __builtin_fmaxf(__builtin_fmaxf(m, __builtin_fabsf(v[0])), __builtin_fabsf(v[1]));
  return __builtin_fmaxf(__builtin_fmaxf(m, __builtin_fabsf(v[2])), __builtin_fabsf(v[3]));
}
// the same, but a NaN where one of them is
__device__ __forceinline__ float max4_nan(float m, f32x4 v) {
  m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, __builtin_fabsf(v[0])), __builtin_fabsf(v[1]));
  return __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, __builtin_fabsf(v[2])), __builtin_fabsf(v[3]));
}
// a b + c
__device__ __forceinline__ f32x4 fma4(f32x4 a, f32x4 b, f32x4 c) { return __builtin_elementwise_fma(a, b, c); }
// over the four rows of 16 lanes, in every lane: swapping the odd rows of a copy with the even rows of another puts the
// rows' neighbours side by side, and the same for halves
__device__ __forceinline__ float max_across16(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t x = __float_as_uint(__builtin_fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1])));
  const auto q = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return __builtin_fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
__device__ __forceinline__ float sum_across16(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t x = __float_as_uint(__uint_as_float(p[0]) + __uint_as_float(p[1]));
  const auto q = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}
// an associative, commutative operation over LANES (8, 16 or 32) neighbouring lanes, in every one of them: neighbours, pairs of
// them, mirrored halves of rows and rows of 16 lanes, then rows of 16
template <int CTRL>
__device__ __forceinline__ uint32_t lane_bits(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
template <int LANES, typename Op>
__device__ __forceinline__ uint32_t row_lanes(uint32_t v, Op op) {
  v = op(v, lane_bits<0xb1>(v));
  v = op(v, lane_bits<0x4e>(v));
  v = op(v, lane_bits<0x141>(v));
  if constexpr (LANES > 8) v = op(v, lane_bits<0x140>(v));
  if constexpr (LANES > 16) {
    const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = op(p[0], p[1]);
  }
  return v;
}

// 16 x 16 x 16 in FP32 by the FP32 matrix instructions: each operand holds index l % 16 and the contracted positions
// 4 (l / 16) + r, which is how results come
__device__ __forceinline__ f32x4 mma_f32(f32x4 a, f32x4 b, f32x4 c) {
#pragma unroll
  for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
  return c;
}

// ------------------------------------------------------------------ a chunk's records (delta_launch.h)
// The places of k's and q's rows in their tiles: of 16 rows, the first 8 in the even places, the others in the odd ones.  Places
// are 4 banks (mod 64) apart, so that 16 rows' same 8 bytes (two columns of lanes at a time) fall on different banks, and,
// even and odd ones for themselves 8 apart, also the transposing reads of 8 rows by 32 bytes.  In order of the rows one of the
// two always met its banks twice: the walks' shared memory was busy for 5900 cycles a chunk, 3100 of them conflicts.
template <int NT>
__device__ __forceinline__ int key_at(int row, int col) {
  return ((row & ~15) + 2 * (row & 7) + (row >> 3 & 1)) * (NT + 8) + col;
}
// rows row0 .. row0 + 15 (a multiple of 16), contracted columns k0 .. k0 + 31 in the split order
template <int NT>
__device__ __forceinline__ f16x8 key_rows(const uint16_t* tile, int row0, int k0, int l) {
  const uint16_t* p = tile + key_at<NT>(l & 15, (l >> 4) * 4) + row0 * (NT + 8) + k0;
  const u32x2 a = *reinterpret_cast<const u32x2*>(p), b = *reinterpret_cast<const u32x2*>(p + 16);
  return as_f16(u32x4{a.x, a.y, b.x, b.y});
}
// columns c0 .. c0 + 15, contracted rows k0 .. k0 + 31 in the split order
template <int NT>
__device__ __forceinline__ f16x8 key_cols(const uint16_t* tile, int k0, int c0, int l) {
  const uint16_t* p = tile + key_at<NT>((l >> 4) * 4 + ((l & 15) >> 2), (l & 3) * 4) + k0 * (NT + 8) + c0;
  const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
  const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 16 * (NT + 8))));
  return as_f16(u32x4{a.x, a.y, b.x, b.y});
}
__device__ __forceinline__ int tri_block(int ib, int jb) { return ib * (ib + 1) / 2 + jb; }
// an operand's half: part `part` of block `blk` of an image of PARTS parts, in shared memory
template <int PARTS>
__device__ __forceinline__ u32x2 tri_half(const char* image, int blk, int part, int lane) {
  return *reinterpret_cast<const u32x2*>(image + (blk * PARTS + part) * kTriPart + lane * 8);
}
// an image's operands, as 16-bit patterns (fp16 of T, bf16 of P)
// Rows 16 ib .. of a lower triangle, contracted columns 32 ks .. (split order; ks <= ib / 2)
template <int PARTS>
__device__ __forceinline__ u32x4 tri_rows(const char* image, int ib, int ks, int part, int lane) {
  const u32x2 a = tri_half<PARTS>(image, tri_block(ib, 2 * ks), part, lane);
  const u32x2 b = 2 * ks + 1 <= ib ? tri_half<PARTS>(image, tri_block(ib, 2 * ks + 1), part, lane) : u32x2{0u, 0u};
  return u32x4{a.x, a.y, b.x, b.y};
}
// Columns 16 jb .. of a transposed image, contracted rows 32 ks .. (ks >= jb / 2)
template <int PARTS>
__device__ __forceinline__ u32x4 tri_cols(const char* image, int jb, int ks, int part, int lane) {
  const u32x2 a = 2 * ks >= jb ? tri_half<PARTS>(image, tri_block(2 * ks, jb), part, lane) : u32x2{0u, 0u};
  const u32x2 b = tri_half<PARTS>(image, tri_block(2 * ks + 1, jb), part, lane);
  return u32x4{a.x, a.y, b.x, b.y};
}
// T's operands
__device__ __forceinline__ Halves t_rows(const char* image, int ib, int ks, int lane) {
  return Halves{as_f16(tri_rows<2>(image, ib, ks, 0, lane)), as_f16(tri_rows<2>(image, ib, ks, 1, lane))};
}
__device__ __forceinline__ Halves t_cols(const char* image, int jb, int ks, int lane) {
  return Halves{as_f16(tri_cols<2>(image, jb, ks, 0, lane)), as_f16(tri_cols<2>(image, jb, ks, 1, lane))};
}
// four values to a block's parts: two of fp16, or PARTS of bf16
__device__ __forceinline__ void store_halves(char* image, int blk, f32x4 v, int lane) {
  const u32x2 u = {pk_f16(v[0], v[1]), pk_f16(v[2], v[3])};
  char* to = image + blk * 2 * kTriPart + lane * 8;
  *reinterpret_cast<u32x2*>(to) = u;
  *reinterpret_cast<u32x2*>(to + kTriPart) = u32x2{rest_f16(v[0], v[1], u.x), rest_f16(v[2], v[3], u.y)};
}
template <int PARTS>
__device__ __forceinline__ void store_tri(char* image, int blk, f32x4 v, int lane) {
#pragma unroll
  for (int p = 0; p < PARTS; ++p) {
    const u32x2 u = {pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])};
    *reinterpret_cast<u32x2*>(image + (blk * PARTS + p) * kTriPart + lane * 8) = u;
    v -= f32x4{bf_lo(u.x), bf_hi(u.x), bf_lo(u.y), bf_hi(u.y)};
  }
}

// A head's factors a row, fk and fq being what makes k and q of the tiles' rows (norms and powers of two):
//   in: e^L fk, read: scale e^L fq, out: e^(L_Q - L) fk, and the rate
// then the chunk's decay, T's scale (what its parts are to be multiplied by), and the first row that is not finite (64: none).
struct Factors {
  float in[64], read[64], out[64], rate[64];
  float decay, t_scale;
  int bad;
  float pad[13];
};
static_assert(sizeof(Factors) == kRecVec, "a record's factors");

__device__ __forceinline__ int64_t chunk_id(const Piece& pc, int64_t c0, int64_t n_chunk_slots) {
  return c0 == pc.s ? n_chunk_slots + pc.seq : c0 >> 6;
}

// the sequence that the item-th walk takes
__device__ __forceinline__ int64_t walk_sequence(const DeltaArgs& d, int64_t item) {
  return d.order ? __builtin_amdgcn_readfirstlane(d.order[item]) : item;
}

// Consecutive bytes that T threads (thread numbers `tid`) copy to shared memory, 16 a thread and step
template <int BYTES, int T>
struct CopyRegs {
  u32x4 v[(BYTES / 16 + T - 1) / T];
};
template <int BYTES, int T>
__device__ __forceinline__ void load_bytes(CopyRegs<BYTES, T>& t, const char* from, bool in, int tid) {
  const Rows r(from, BYTES, 1, in ? BYTES : 0, 1);
#pragma unroll
  for (int k = 0; k < (BYTES / 16 + T - 1) / T; ++k)
    t.v[k] = __builtin_amdgcn_raw_buffer_load_b128(r.r, (tid + T * k) * 16, 0, 0);
}
template <int BYTES, int T>
__device__ __forceinline__ void store_bytes(void* lds, const CopyRegs<BYTES, T>& t, int tid) {
#pragma unroll
  for (int k = 0; k < (BYTES / 16 + T - 1) / T; ++k) {
    const int at = (tid + T * k) * 16;
    if (at < BYTES) *reinterpret_cast<u32x4*>(static_cast<char*>(lds) + at) = t.v[k];
  }
}

// 64 rows of COLS columns by 4 COLS threads (thread numbers `tid`), as load_tile and store_tile by all of a block's
template <int COLS, bool VEC>
__device__ __forceinline__ void load_rows(u32x4 (&v)[2], const Rows& rows, uint32_t ld, int ncols, int tid) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int row = tid / (COLS / 8) + 32 * k, c = tid % (COLS / 8) * 8;
    const uint32_t off = (row * ld + c) * 2;
    if constexpr (VEC) {
      v[k] = __builtin_amdgcn_raw_buffer_load_b128(rows.r, (int)(c < ncols ? off : kOutside), 0, 0);
    } else {
      v[k] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t u = __builtin_amdgcn_raw_buffer_load_b16(rows.r, (int)(c + e < ncols ? off + 2 * e : kOutside), 0, 0);
        v[k][e >> 1] |= u << (16 * (e & 1));
      }
    }
  }
}
template <int COLS>
__device__ __forceinline__ void store_rows(uint16_t* lds, const u32x4 (&v)[2], int tid) {
#pragma unroll
  for (int k = 0; k < 2; ++k)
    *reinterpret_cast<u32x4*>(lds + at<COLS, 16>(tid / (COLS / 8) + 32 * k, tid % (COLS / 8) * 8)) = v[k];
}

// four rows of this lane's column of a bf16 tile of COLS columns: rows row0 + 4 g .., column c0 + i
template <int COLS = 64>
__device__ __forceinline__ f32x4 column4(const uint16_t* tile, int row0, int c0, int g, int i) {
  const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (lds_s16x4*)(tile + at<COLS, 16>(row0 + 4 * g + (i >> 2), c0 + 4 * (i & 3))));
  const u32x2 v = __builtin_bit_cast(u32x2, t);
  return f32x4{bf_lo(v.x), bf_hi(v.x), bf_lo(v.y), bf_hi(v.y)};
}

// a state's column block: rows p of [P, N], this lane's row (nullptr: none), four columns n at 16 nb + 4 g
template <int NB>
__device__ __forceinline__ void load_state(f32x4 (&S)[NB], const float* row, int N, int g) {
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int n = 16 * nb + 4 * g;
    S[nb] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (!row) continue;
    if (n + 3 < N) {
      S[nb] = *reinterpret_cast<const f32x4_a4*>(row + n);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < N) S[nb][r] = row[n + r];
    }
  }
}
template <int NB>
__device__ __forceinline__ void store_state(const f32x4 (&S)[NB], float* row, int N, int g) {
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int n = 16 * nb + 4 * g;
    if (n + 3 < N) {
      *reinterpret_cast<f32x4_a4*>(row + n) = S[nb];
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < N) row[n + r] = S[nb][r];
    }
  }
}
template <int NB>
__device__ __forceinline__ float state_max(const f32x4 (&S)[NB]) {
  float m = 0.f;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) m = max4(m, S[nb]);
  return max_across16(m);
}

// The walks' state: true values are `down` times the accumulators', which stay below 2^15.  A chunk adds COUNT products of 64 rows
// with keys below two: |sum| <= COUNT 128 max, so the larger of the state and the addends goes to 2^7 (one) or 2^6 (two).
template <int COUNT>
__device__ __forceinline__ Pow2 state_scale(float m) {
  return bring_to<COUNT == 1 ? 7 : 6>(m);
}

}  // namespace cssm
