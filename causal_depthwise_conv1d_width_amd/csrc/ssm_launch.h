// ssm_launch.h -- launch parameters shared by the host entry points of include/ssm.h (ssm_api.cpp)
// and their kernels.  Plain data: pointers are device pointers the host has validated but never
// dereferences.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace cssm {

constexpr int kChunk = 64;      // rows a chunk of the scan: one lane a row where a wave scans decays
constexpr int kPTile = 64;      // head-dimension columns a block works on; wider heads take several tiles
constexpr int kMaxState = 256;  // state size limit N (three compiled sizes: 64, 128, 256)
constexpr int64_t kMaxGroup = 32768;  // channels a norm group may have

// Packed sequences: offsets (cu != nullptr) or batch rows of seqlen rows.
struct Seqs {
  const int32_t* cu;
  int64_t nseq, seqlen, rows;
};

// What the scan's kernels share.  Chunks begin at sequence starts and at multiples of kChunk rows of
// the packed array, so a chunk is found from a row number alone; pieces (the unit of one block's sequential
// walk) are whole chunks.
struct ScanArgs {
  const uint16_t* x;   // [rows, H, P]
  const uint16_t* B;   // [rows, G, N]
  const uint16_t* C;   // [rows, G, N]
  const void* dt;      // [rows, H]
  int64_t x_ld, B_ld, C_ld, dt_ld;
  const float* A;      // [H]
  const float* D;      // [H] or nullptr
  const float* bias;   // [H] or nullptr
  int dt_f32, softplus;
  int H, P, G, N, ptiles;
  Seqs q;
  int seg;               // log2 of a piece's rows, 0: a piece is a sequence
  int64_t n_slots;       // pieces other than a sequence's first: with offsets, at most one every 2^seg rows
  // states [slot, H, P, N] of FP32; slot = ci ? ci[seq] : seq
  const float* init;     // nullptr: zeros
  float* fin;            // nullptr: not wanted
  int64_t slots, s_slot;
  const int32_t* ci;
  const uint8_t* has_init;
  uint16_t* y;           // [rows, H, P]
  int64_t y_ld;
  // pieces' states [n_slots + nseq, H * ptiles, 64, NT] and log2 decays [n_slots + nseq, H]
  float* piece;
  float* piece_decay;
};

// The scan's backward.  T is the adjoint of the state.
struct ScanBwdArgs {
  ScanArgs s;               // s.init: initial states [nseq, H, P, N]; s.y unused
  const uint16_t* dy;       // [rows, H, P]
  int64_t dy_ld;
  const float* dfin;        // [nseq, H, P, N] or nullptr
  float* dinit;             // [nseq, H, P, N] or nullptr
  uint16_t* dx;
  void* ddt;                // dt's type
  uint16_t *dB, *dC;
  int64_t dx_ld, ddt_ld, dB_ld, dC_ld;
  float *dA, *dD, *dbias;   // [H]; dD, dbias may be nullptr
  // pieces' adjoints and log2 decays, as s.piece and s.piece_decay: both walks run in one launch and sum a
  // piece's decays in their own order, so each has its own
  float *piece_t, *piece_t_decay;
  // FP32 states before (S) and adjoints after (T) every chunk, in matrix-operand order; chunk id =
  // row / kChunk, or n_chunk_slots + seq for a sequence's first
  float *cs, *ct;
  int64_t n_chunk_slots;
  float* head_part;         // [chunk id, H, 3]: sums for dA, d(dt_bias), dD
  float* bc_part;           // [2, hsplit, rows, G, N] when hsplit > 1
  int hsplit;
};

struct StepArgs {
  const uint16_t *x, *B, *C;
  const void* dt;
  int64_t x_ld, B_ld, C_ld, dt_ld, y_ld, nseq;
  const float *A, *D, *bias;
  int dt_f32, softplus, H, P, G, N;
  float* pool;
  int64_t slots, s_slot;
  const int32_t* ci;
  uint16_t* y;
};

// Norms: rows of `groups` groups of `group` channels.
struct NormArgs {
  const uint16_t* x;   // input (gated) or block output to add (residual)
  const uint16_t* z;   // gate (gated)
  const void* r;       // residual: forward input; backward: the stored sum
  const uint16_t* dy;
  const void* dr_in;   // residual backward: gradient of the stored sum, or nullptr
  uint16_t *y, *dx, *dz;
  void* r_out;         // residual: forward sum; backward gradient of the incoming residual
  int64_t x_ld, z_ld, r_ld, dy_ld, dri_ld, y_ld, dx_ld, dz_ld, ro_ld;
  const void* w;       // [groups * group], FP32 or bf16
  int w_f32, r_f32, norm_first;
  int64_t rows, groups, group;
  float eps, scale;
  float* part;         // backward: [parts, groups * group] sums for dw
  int64_t parts;
  float* dw;
};

hipError_t launch_scan_fwd(const ScanArgs& a, bool vec, hipStream_t s);
hipError_t launch_scan_bwd(const ScanBwdArgs& a, bool vec, hipStream_t s);
hipError_t launch_step(const StepArgs& a, hipStream_t s);
hipError_t launch_gated_fwd(const NormArgs& a, hipStream_t s);
hipError_t launch_gated_bwd(const NormArgs& a, hipStream_t s);
hipError_t launch_residual_fwd(const NormArgs& a, hipStream_t s);
hipError_t launch_residual_bwd(const NormArgs& a, hipStream_t s);

// units a block of the scan or of the state walk takes
constexpr int kUnits = 4;
// blocks of the scan and of the state walk: U 64-column units for every piece and group, these in sets of 8
// (one an XCD)
inline int64_t unit_blocks(int64_t items, int64_t H, int64_t G, int64_t ptiles, int U) {
  return (items * G + 7) / 8 * 8 * ((H / G * ptiles + U - 1) / U);
}
inline int state_tile(int64_t N) { return N <= 64 ? 64 : (N <= 128 ? 128 : 256); }

// threads that share one (row, group) of a norm: 8 channels a thread, up to 1024 threads
inline int norm_threads(int64_t group) {
  int t = 64;
  while (t < 1024 && t * 8 < group) t *= 2;
  return t;
}
// row splits of a norm's forward: about `waves` waves; each takes every parts-th row.  Forward and backward of 16384
// rows: gated, 4096 channels, 200 us with 4096 waves, 225 with 2048, 205 with 8192; residual, 2048 channels, 174 us
// with 2048, 182 with 4096, 188 with 1024.
constexpr int64_t kGatedFwdWaves = 4096, kResidualFwdWaves = 2048;
inline int64_t norm_fwd_parts(int64_t rows, int64_t groups, int64_t group, int64_t waves) {
  int64_t p = waves / (groups * (norm_threads(group) / 64));
  if (p < 1) p = 1;
  return p < rows ? p : rows;
}
// row splits, and dweight partials, of its backward: about 4096 waves, but no more than 512 partials to add
// (16384 rows of 2048 channels, 1024 partials against 512: 200 us against 175 us forward and backward)
inline int64_t norm_parts(int64_t rows, int64_t groups, int64_t group) {
  int64_t p = 4096 / (groups * (norm_threads(group) / 64));
  if (p < 1) p = 1;
  if (p > 512) p = 512;
  return p < rows ? p : rows;
}

}  // namespace cssm
