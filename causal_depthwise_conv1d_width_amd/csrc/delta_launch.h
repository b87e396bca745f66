// delta_launch.h -- launch parameters shared by the host entry points of include/delta.h (delta_api.cpp) and their
// kernels.  Plain data: pointers are device pointers the host has validated but never dereferences.
#pragma once

#include "ssm_launch.h"

namespace cssm {

// What the chunk kernel leaves for the walks, which copy it to shared memory as it is.
// A key head's record of a chunk: the tiles of k and of q, [64 places][NT + 8 columns] of fp16, each row times a power of two.
constexpr int64_t key_tile(int NT) { return 64 * (NT + 8) * 2; }
// A head's record: lower triangles of 64 x 64 in 16 x 16 blocks, block (ib, jb) at ib (ib + 1) / 2 + jb: lane l holds row
// l % 16 and the four columns from 4 (l / 16) on (for the reverse walk: column l % 16, four rows), each 16-bit part 512 bytes.
// First the triangular system's inverse T in two fp16 parts, then the scores P (in two bf16 parts forward, in three in
// reverse), then factors.
constexpr int kTriBlocks = 10, kTriPart = 512;
constexpr int kRecT = kTriBlocks * 2 * kTriPart;
constexpr int kRecVec = 4 * 64 * 4 + 64;
constexpr int kRecFwd = kRecT + kTriBlocks * 2 * kTriPart + kRecVec;
constexpr int kRecRev = kRecT + kTriBlocks * 3 * kTriPart + kRecVec;

// What the backward's walks leave of a chunk and 64 columns of a head, FP32: the state before (S) and the adjoint after the
// chunk (D) as [4 blocks of 16 rows, NT / 16 blocks of 16 columns, 16 rows, 16 columns]; the new values (U) and what reaches
// them (F) as [64 rows, 64 columns]; the largest of S by blocks of 16 rows, and of D.
constexpr int tile_s(int) { return 0; }
constexpr int tile_d(int NT) { return 64 * NT; }
constexpr int tile_u(int NT) { return 2 * 64 * NT; }
constexpr int tile_f(int NT) { return tile_u(NT) + 4096; }
constexpr int tile_tops(int NT) { return tile_f(NT) + 4096; }
constexpr int tile_floats(int NT) { return tile_tops(NT) + 32; }

// s: x = v, B = k, C = q, init, fin and slots as in the scan; y
struct DeltaArgs {
  ScanArgs s;
  const void* b;  // [rows, H], dt's type
  int64_t b_ld;
  float scale, beta_max, norm_eps;
  int qk_norm;
  int64_t n_chunk_slots;  // chunk id = row / kChunk, or n_chunk_slots + seq for a sequence's first
  char* keys;             // [chunk id, G] key heads' records of 2 key_tile(NT) bytes
  char* rec;              // [chunk id, H] heads' records of kRecFwd bytes
  int32_t* order;         // with offsets: the sequences from long to short, for the walks
};

struct DeltaBwdArgs {
  DeltaArgs d;
  const uint16_t* dy;
  int64_t dy_ld;
  const float* dfin;         // [nseq, H, P, N] or nullptr
  float* dinit;              // or nullptr
  uint16_t *dq, *dk, *dv;
  void *ddt, *db;
  int64_t dq_ld, dk_ld, dv_ld, ddt_ld, db_ld;
  float *dA, *dbias;         // [H]; dbias may be nullptr
  char* rec_rev;             // [chunk id, H] records of kRecRev bytes
  float* tiles;              // [chunk id, H, ptiles] records of tile_floats(NT)
  float* head_part;          // [chunk id, H, 2]: sums for dA, d(dt_bias)
};

struct DeltaStepArgs {
  const uint16_t *q, *k, *v;
  const void *dt, *b;
  int64_t q_ld, k_ld, v_ld, dt_ld, b_ld, y_ld, nseq;
  const float *A, *bias;
  int f32, softplus, qk_norm, H, P, G, N;
  float scale, beta_max, norm_eps;
  float* pool;
  int64_t slots, s_slot;
  const int32_t* ci;
  uint16_t* y;
};

// Layer norm: NormArgs with r = the residual or the stored sum, r_out, and
struct LayerArgs {
  NormArgs n;
  const void* bias;
  float* db;
};

struct SlotArgs {
  char* ptr[8];
  int64_t slots[8], s_slot[8], bytes[8];
  uint32_t first[9];  // a pool's first block
  int pools, n, strip;  // log2 of a strip's 16-byte pieces
  const int32_t *source, *target;
};

hipError_t launch_delta_chunks(const DeltaArgs& a, char* rec_rev, bool vec, hipStream_t s);  // rec_rev: nullptr forward
hipError_t launch_delta_fwd(const DeltaArgs& a, bool vec, hipStream_t s);
hipError_t launch_delta_bwd(const DeltaBwdArgs& b, bool vec, hipStream_t s);
hipError_t launch_delta_step(const DeltaStepArgs& a, hipStream_t s);
hipError_t launch_layer_fwd(const LayerArgs& a, hipStream_t s);
hipError_t launch_layer_bwd(const LayerArgs& a, hipStream_t s);
hipError_t launch_slots(const SlotArgs& a, int threads, int pieces, uint32_t blocks, hipStream_t s);

}  // namespace cssm
