// delta_launch.h -- launch parameters shared by the host entry points of include/delta.h (delta_api.cpp) and their
// kernels.  Plain data: pointers are device pointers the host has validated but never dereferences.
#pragma once

#include "ssm_launch.h"

namespace cssm {

// A chunk's record for one head, written by the chunk kernel and copied to shared memory by the walks.  Lower triangles of
// 64 x 64 in 16 x 16 blocks, block (ib, jb) at ib (ib + 1) / 2 + jb: lane l holds row l % 16 and the four columns from
// 4 (l / 16) on (transposed for the reverse walk: column l % 16, four rows), each bf16 part 512 bytes.
constexpr int kTriBlocks = 10, kTriPart = 512;
constexpr int kRecT = kTriBlocks * 3 * kTriPart;  // the triangular system's inverse, three parts
constexpr int kRecVec = 4 * 64 * 4 + 64;          // four factors a row, then: decay of the chunk, first row not finite
constexpr int kRecFwd = kRecT + 2 * kTriBlocks * kTriPart + kRecVec;  // the scores in two parts
constexpr int kRecRev = 2 * kRecT + kRecVec;                      // the reverse walk's, in three

// s: x = v, B = k, C = q, init, fin and slots as in the scan; y
struct DeltaArgs {
  ScanArgs s;
  const void* b;  // [rows, H], dt's type
  int64_t b_ld;
  float scale, beta_max, norm_eps;
  int qk_norm;
  int64_t n_chunk_slots;  // chunk id = row / kChunk, or n_chunk_slots + seq for a sequence's first
  char* rec;              // [chunk id, H] records of kRecFwd bytes
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
  // states before and adjoints after every chunk, [chunk id, H, ptiles, 4 blocks of 16 rows, NT / 16 blocks of 16 columns,
  // 16 rows, 16 columns]
  float *cs, *ct;
  float *u, *f;              // new values and what reaches them: [chunk id, H, ptiles, 64 rows, 64 columns]
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
