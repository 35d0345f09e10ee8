// kda_beam_internal.h — launch descriptors of the beam search kernels
// (kda_beam.hip) for the C ABI layer (kda_beam_api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

constexpr int kBeamMax = 16;          // beams of a group
constexpr int kBeamReorderMax = 8;    // state tensors of one reorder launch
constexpr int kBeamThreads = 256;     // of a scan workgroup
constexpr int kBeamMaxParts = 2048;   // parts of a row: one thread's share of a slice

// A row of V logits is scanned in 16-byte vectors from its first aligned
// element on (up to `head` elements before it and `tail` behind the last
// whole vector belong to threads of the first slice).  A slice is 256 threads
// x nv vectors; thread t of slice s takes the vectors s * 256 nv + 256 i + t
// (i < nv): a part.
struct BeamPlan {
  int es;       // bytes of a logit
  int nv;       // vectors per part
  int slices;   // slices per row
};

// Vectors of a row of V logits, at most (the alignment of a row is not known
// on the host when rows are of odd length).
constexpr int64_t beam_vectors(int vocab, int es) { return ((int64_t)vocab * es) / 16; }

inline BeamPlan beam_plan(int vocab, bool bf16) {
  BeamPlan p;
  p.es = bf16 ? 2 : 4;
  const int64_t nvec = beam_vectors(vocab, p.es);
  p.nv = (int)((nvec + kBeamMaxParts - 1) / kBeamMaxParts);
  if (p.nv < 1) p.nv = 1;
  p.slices = (int)((nvec + (int64_t)kBeamThreads * p.nv - 1) / ((int64_t)kBeamThreads * p.nv));
  if (p.slices < 1) p.slices = 1;
  return p;
}

struct BeamSelectArgs {
  const void* logits;        // [groups, beams, vocab]
  const float* scores;       // [groups, beams]
  const uint8_t* finished;   // [groups, beams] or null
  int groups;
  int beams;
  int vocab;
  int end_token;             // with finished
  bool bf16;
  BeamPlan plan;
  float* part_max;           // [rows][slices * 256] largest logit of each part
  int32_t* part_at;          // its index
  float* slice_max;          // [rows][slices]
  float* slice_sum;          // [rows][slices] sum of exp(x - slice_max)
  float* out_scores;
  int32_t* out_tokens;
  int32_t* out_parents;
  uint8_t* out_finished;     // or null
};

// Tensors whose rows move in units of the same size (16, 4 or 1 bytes).
struct BeamReorderArgs {
  void* state[kBeamReorderMax];       // [groups * beams][row_units]
  int64_t row_units[kBeamReorderMax];
  int64_t block0[kBeamReorderMax];    // first block (of one group) of each tensor
  int count;
  int64_t blocks;                     // blocks per group
  const int32_t* parents;             // [groups, beams]
  int groups;
  int beams;
  int64_t group0;                     // first group of the launch (set by it)
};

hipError_t launch_beam_select(const BeamSelectArgs& a, hipStream_t stream);
hipError_t launch_beam_reorder(const BeamReorderArgs& a, int unit, hipStream_t stream);

}  // namespace kda
