// Launch stubs that keep their arguments, for a host-only build of the delta rule's entry points
// (tests/test_delta_plan.py): no kernel is started.
#include "delta_launch.h"
namespace cssm {
static DeltaBwdArgs last;
static SlotArgs slots;
static int threads, pieces;
static uint32_t blocks;
static int launches;
hipError_t launch_delta_fwd(const DeltaArgs& a, bool, hipStream_t) { last = DeltaBwdArgs{}; last.d = a; ++launches; return hipSuccess; }
hipError_t launch_delta_bwd(const DeltaBwdArgs& b, bool, hipStream_t) { last = b; ++launches; return hipSuccess; }
hipError_t launch_delta_step(const DeltaStepArgs&, hipStream_t) { ++launches; return hipSuccess; }
hipError_t launch_layer_fwd(const LayerArgs&, hipStream_t) { ++launches; return hipSuccess; }
hipError_t launch_layer_bwd(const LayerArgs&, hipStream_t) { ++launches; return hipSuccess; }
hipError_t launch_slots(const SlotArgs& a, int t, int p, uint32_t b, hipStream_t) {
  slots = a, threads = t, pieces = p, blocks = b;
  ++launches;
  return hipSuccess;
}
}
using namespace cssm;
extern "C" int delta_launches() { return launches; }
// the last call's workspace arrays and their sizes in bytes; chunk ids
extern "C" void delta_last_plan(int64_t* v) {
  const DeltaBwdArgs& b = last;
  const DeltaArgs& d = b.d;
  const int64_t ids = d.n_chunk_slots + d.s.q.nseq;
  const int nt = d.s.N <= 64 ? 64 : d.s.N <= 128 ? 128 : 256;
  const void* p[6] = {d.keys, d.rec, d.order, b.rec_rev, b.tiles, b.head_part};
  const int64_t n[6] = {ids * d.s.G * 2 * key_tile(nt), ids * d.s.H * kRecFwd, d.order ? d.s.q.nseq * 4 : 0, ids * d.s.H * kRecRev,
                        ids * d.s.H * d.s.ptiles * tile_floats(nt) * 4, ids * d.s.H * 8};
  for (int i = 0; i < 6; ++i) v[i] = (int64_t)(intptr_t)p[i], v[6 + i] = n[i];
  v[12] = ids;
}
// The last copy's blocks as the kernel walks them: 1 if every byte of every pool's slots lies in exactly one block's strip
// and no block holds more pieces than its threads have registers for
extern "C" int delta_slots_cover() {
  const SlotArgs& a = slots;
  if (((int64_t)a.n << a.strip) > (int64_t)threads * pieces) return 0;
  int64_t at[8] = {};
  for (uint32_t b = 0; b < blocks; ++b) {
    int p = 0;
    while (p + 1 < a.pools && b >= a.first[p + 1]) ++p;
    if (((int64_t)(b - a.first[p]) << (a.strip + 4)) != at[p]) return 0;
    at[p] += (int64_t)16 << a.strip;
  }
  for (int p = 0; p < a.pools; ++p)
    if (at[p] < a.bytes[p] || at[p] - ((int64_t)16 << a.strip) >= a.bytes[p]) return 0;
  return 1;
}
