// Tensor-core path of the causal linear attention with a decay per head.
#pragma once

#include "decay.cuh"

namespace favor {

// bf16, d <= 128, whole 16-byte pieces, no broadcast axis: whatever the sizes (32 heads
// of 64 tokens of 64 took 8.7 us against 13.5 on the CUDA cores, 64 of 4096 54 against
// 363, 16 of 16384 of 128 108 against 916)
bool decay_tc_takes(const View* const* views, int n, bool bf16, int d);
// segments for `passes` passes side by side
void decay_tc_plan(DecayShape* s, int passes);
// a view, encoded once per call
struct DecayMap {
  alignas(64) unsigned char bytes[128];
};
bool decay_tc_map(DecayMap* map, const View& v);

struct DecayTcPass {
  DecayPass p;               // p.last is not written
  int64_t step;              // elements between the segments' states
  bool after_scan;           // the launch before in the stream is decay_scan_states'
  const DecayMap *a, *b, *c, *o;
};
// short sequences of one segment: no states are kept, and the gains run beside the passes
bool decay_tc_ends_beside(const DecayShape& s);
// ends: such sequences; p.out [B H][d][d] becomes the state behind it, from `first`
// (NULL: zeros, may be p.out).  The launch before must then be that of the passes,
// beside which it runs.
struct DecayTcGain {
  DecayGain p;
  const float* first;
  bool ends;
  const DecayMap *b, *c;
};
// up to three side by side
cudaError_t decay_tc_passes(const DecayTcPass* passes, int n, const DecayShape& s, cudaStream_t stream);
cudaError_t decay_tc_gains(const DecayTcGain* gains, int n, const DecayShape& s, cudaStream_t stream);

}  // namespace favor
