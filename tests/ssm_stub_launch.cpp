// Launch stubs that keep their arguments, for a host-only build of the scan's entry points
// (tests/test_ssm_plan.py): no kernel is started.
#include "ssm_launch.h"
namespace cssm {
static ScanBwdArgs last;
hipError_t launch_scan_fwd(const ScanArgs& a, bool, hipStream_t) { last = ScanBwdArgs{}; last.s = a; return hipSuccess; }
hipError_t launch_scan_bwd(const ScanBwdArgs& b, bool, hipStream_t) { last = b; return hipSuccess; }
hipError_t launch_step(const StepArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_gated_fwd(const NormArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_gated_bwd(const NormArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_residual_fwd(const NormArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_residual_bwd(const NormArgs&, hipStream_t) { return hipSuccess; }
}
// the last call's workspace arrays and counts
extern "C" void ssm_last_plan(int64_t* v) {
  const cssm::ScanBwdArgs& b = cssm::last;
  const void* p[8] = {b.s.piece, b.s.piece_decay, b.piece_t, b.piece_t_decay, b.cs, b.ct, b.head_part, b.bc_part};
  for (int i = 0; i < 8; ++i) v[i] = (int64_t)(intptr_t)p[i];
  v[8] = b.s.seg;
  v[9] = b.s.n_slots + b.s.q.nseq;
  v[10] = b.n_chunk_slots + b.s.q.nseq;
  v[11] = b.hsplit;
}
