// delta_device.h -- what the delta rule's chunk kernel and walks share: products of operands in parts, the chunks' records.
#pragma once

#include "delta_launch.h"
#include "ssm_state.h"

namespace cssm {

// The product of FP32 operands in three parts each, up to the terms of 2^-24: six products
__device__ __forceinline__ f32x4 mma6(const Parts& a, const Parts& b, f32x4 c) {
  c = mma(a.p[2], b.p[0], c);
  c = mma(a.p[0], b.p[2], c);
  c = mma(a.p[1], b.p[1], c);
  c = mma(a.p[1], b.p[0], c);
  c = mma(a.p[0], b.p[1], c);
  return mma(a.p[0], b.p[0], c);
}
// of an FP32 operand in parts and one that is bf16
__device__ __forceinline__ f32x4 mma3(const Parts& a, bf16x8 b, f32x4 c) {
  c = mma(a.p[2], b, c);
  c = mma(a.p[1], b, c);
  return mma(a.p[0], b, c);
}
__device__ __forceinline__ f32x4 mma3(bf16x8 a, const Parts& b, f32x4 c) {
  c = mma(a, b.p[2], c);
  c = mma(a, b.p[1], c);
  return mma(a, b.p[0], c);
}
// 16 x 16 x 16 in FP32 by the FP32 matrix instructions: each operand holds index l % 16 and the contracted positions
// 4 (l / 16) + r, which is how results come
__device__ __forceinline__ f32x4 mma_f32(f32x4 a, f32x4 b, f32x4 c) {
#pragma unroll
  for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
  return c;
}

// ------------------------------------------------------------------ a chunk's record (delta_launch.h)
__device__ __forceinline__ int tri_block(int ib, int jb) { return ib * (ib + 1) / 2 + jb; }
// an operand's half: part `part` of block `blk` of an image of PARTS parts, in shared memory
template <int PARTS>
__device__ __forceinline__ u32x2 tri_half(const char* image, int blk, int part, int lane) {
  return *reinterpret_cast<const u32x2*>(image + (blk * PARTS + part) * kTriPart + lane * 8);
}
// Rows 16 ib .. of a lower triangle, contracted columns 32 ks .. (split order; ks <= ib / 2)
template <int PARTS>
__device__ __forceinline__ bf16x8 tri_rows(const char* image, int ib, int ks, int part, int lane) {
  const u32x2 a = tri_half<PARTS>(image, tri_block(ib, 2 * ks), part, lane);
  const u32x2 b = 2 * ks + 1 <= ib ? tri_half<PARTS>(image, tri_block(ib, 2 * ks + 1), part, lane) : u32x2{0u, 0u};
  return __builtin_bit_cast(bf16x8, u32x4{a.x, a.y, b.x, b.y});
}
// Columns 16 jb .. of a transposed image, contracted rows 32 ks .. (ks >= jb / 2)
template <int PARTS>
__device__ __forceinline__ bf16x8 tri_cols(const char* image, int jb, int ks, int part, int lane) {
  const u32x2 a = 2 * ks >= jb ? tri_half<PARTS>(image, tri_block(2 * ks, jb), part, lane) : u32x2{0u, 0u};
  const u32x2 b = tri_half<PARTS>(image, tri_block(2 * ks + 1, jb), part, lane);
  return __builtin_bit_cast(bf16x8, u32x4{a.x, a.y, b.x, b.y});
}
// four values to a block's parts
template <int PARTS>
__device__ __forceinline__ void store_tri(char* image, int blk, f32x4 v, int lane) {
#pragma unroll
  for (int p = 0; p < PARTS; ++p) {
    const u32x2 u = {pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])};
    *reinterpret_cast<u32x2*>(image + (blk * PARTS + p) * kTriPart + lane * 8) = u;
    v -= f32x4{bf_lo(u.x), bf_hi(u.x), bf_lo(u.y), bf_hi(u.y)};
  }
}

// A record's factors a row, then the chunk's decay and its first row that is not finite (64: none)
struct Factors {
  float f[4][64];
  float decay;
  int bad;
  float pad[14];
};
static_assert(sizeof(Factors) == kRecVec, "a record's factors");

__device__ __forceinline__ int64_t chunk_id(const Piece& pc, int64_t c0, int64_t n_chunk_slots) {
  return c0 == pc.s ? n_chunk_slots + pc.seq : c0 >> 6;
}

// A record that the four waves copy to shared memory, 16 bytes a thread and step
template <int BYTES, int T>
struct RecordRegs {
  u32x4 v[(BYTES / 16 + T - 1) / T];
};
template <int BYTES, int T>
__device__ __forceinline__ void load_record(RecordRegs<BYTES, T>& t, const char* rec, bool in) {
  const Rows r(rec, BYTES, 1, in ? BYTES : 0, 1);
#pragma unroll
  for (int k = 0; k < (BYTES / 16 + T - 1) / T; ++k)
    t.v[k] = __builtin_amdgcn_raw_buffer_load_b128(r.r, (int)((threadIdx.x + T * k) * 16), 0, 0);
}
template <int BYTES, int T>
__device__ __forceinline__ void store_record(char* lds, const RecordRegs<BYTES, T>& t) {
#pragma unroll
  for (int k = 0; k < (BYTES / 16 + T - 1) / T; ++k) {
    const int at = (threadIdx.x + T * k) * 16;
    if (at < BYTES) *reinterpret_cast<u32x4*>(lds + at) = t.v[k];
  }
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

}  // namespace cssm
