// kda_beam_api.hip — the C ABI of beam search over recurrent states
// (include/kda_beam.h).
#include <hip/hip_runtime.h>

#include <cstring>

#include "kda_api_util.h"
#include "kda_beam.h"
#include "kda_beam_internal.h"

namespace {

using namespace kda::api;

static_assert(KDA_BEAM_MAX == kda::kBeamMax && KDA_BEAM_REORDER_MAX == kda::kBeamReorderMax, "limits of the header");

bool beam_sizes_ok(int groups, int beams, int vocab) {
  if (groups < 1 || beams < 1 || vocab < 1) return false;
  return (int64_t)groups * beams <= (int64_t)INT32_MAX;
}

struct SelectLayout {
  size_t off_at = 0, off_smax = 0, off_ssum = 0, bytes = 0;
};
SelectLayout select_layout(int groups, int beams, const kda::BeamPlan& pl) {
  const size_t rows = (size_t)groups * beams;
  const size_t parts = rows * pl.slices * kda::kBeamThreads;
  SelectLayout l;
  l.off_at = align256(parts * 4);
  l.off_smax = l.off_at + align256(parts * 4);
  l.off_ssum = l.off_smax + align256(rows * pl.slices * 4);
  l.bytes = l.off_ssum + align256(rows * pl.slices * 4);
  return l;
}

bool select_grid_ok(int groups, int beams, const kda::BeamPlan& pl) {
  return (int64_t)groups * beams * pl.slices * kda::kBeamThreads <= (int64_t)UINT32_MAX;  // threads of a launch
}

}  // namespace

extern "C" {

size_t kda_beam_select_workspace_bytes(int groups, int beams, int vocab, kda_dtype dtype) {
  if (!beam_sizes_ok(groups, beams, vocab) || beams > kda::kBeamMax || !dtype_ok(dtype)) return 0;
  const kda::BeamPlan pl = kda::beam_plan(vocab, dtype == KDA_DTYPE_BF16);
  return select_grid_ok(groups, beams, pl) ? select_layout(groups, beams, pl).bytes : 0;
}

kda_status kda_beam_select(const void* logits, const float* scores, const uint8_t* finished, int groups, int beams,
                           int vocab, int end_token, kda_dtype dtype, float* out_scores, int32_t* out_tokens,
                           int32_t* out_parents, uint8_t* out_finished, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
  if (!beam_sizes_ok(groups, beams, vocab)) return KDA_ERR_INVALID_ARG;
  if (beams > kda::kBeamMax || !dtype_ok(dtype)) return KDA_ERR_UNSUPPORTED;
  if (!logits || !scores || !out_scores || !out_tokens || !out_parents) return KDA_ERR_INVALID_ARG;
  if ((finished != nullptr) != (out_finished != nullptr)) return KDA_ERR_INVALID_ARG;
  if (finished && (end_token < 0 || end_token >= vocab)) return KDA_ERR_INVALID_ARG;
  const size_t es = elem_size(dtype);
  if (!aligned(logits, es) || !aligned(scores, 4) || !aligned(out_scores, 4) || !aligned(out_tokens, 4) ||
      !aligned(out_parents, 4) || !aligned(workspace, 16))
    return KDA_ERR_INVALID_ARG;
  const kda::BeamPlan pl = kda::beam_plan(vocab, dtype == KDA_DTYPE_BF16);
  if (!select_grid_ok(groups, beams, pl)) return KDA_ERR_INVALID_ARG;
  const SelectLayout l = select_layout(groups, beams, pl);
  if (!workspace || workspace_bytes < l.bytes) return KDA_ERR_WORKSPACE;
  const size_t rows = (size_t)groups * beams;
  const Range r_sc = range_of(scores, rows * 4), r_fi = range_of(finished, finished ? rows : 0);
  const Range r_os = range_of(out_scores, rows * 4), r_of = range_of(out_finished, out_finished ? rows : 0);
  const Range r_lo = range_of(logits, rows * (size_t)vocab * es);
  const Range outs[] = {r_os, range_of(out_tokens, rows * 4), range_of(out_parents, rows * 4), r_of,
                        range_of(workspace, l.bytes)};
  for (size_t i = 0; i < 5; ++i) {
    if (overlap(outs[i], r_lo)) return KDA_ERR_INVALID_ARG;
    // the new scores and flags may be exactly the old ones (updated in place)
    if (overlap(outs[i], r_sc) && !(i == 0 && r_os.lo == r_sc.lo)) return KDA_ERR_INVALID_ARG;
    if (overlap(outs[i], r_fi) && !(i == 3 && r_of.lo == r_fi.lo)) return KDA_ERR_INVALID_ARG;
    for (size_t j = i + 1; j < 5; ++j)
      if (overlap(outs[i], outs[j])) return KDA_ERR_INVALID_ARG;
  }
  char* ws = static_cast<char*>(workspace);
  kda::BeamSelectArgs a;
  std::memset(&a, 0, sizeof(a));
  a.logits = logits;
  a.scores = scores;
  a.finished = finished;
  a.groups = groups;
  a.beams = beams;
  a.vocab = vocab;
  a.end_token = finished ? end_token : -1;
  a.bf16 = dtype == KDA_DTYPE_BF16;
  a.plan = pl;
  a.part_max = reinterpret_cast<float*>(ws);
  a.part_at = reinterpret_cast<int32_t*>(ws + l.off_at);
  a.slice_max = reinterpret_cast<float*>(ws + l.off_smax);
  a.slice_sum = reinterpret_cast<float*>(ws + l.off_ssum);
  a.out_scores = out_scores;
  a.out_tokens = out_tokens;
  a.out_parents = out_parents;
  a.out_finished = out_finished;
  return kda::launch_beam_select(a, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

kda_status kda_beam_reorder(void* const* states, const int64_t* row_bytes, int num_states, const int32_t* parents,
                            int groups, int beams, hipStream_t stream) {
  if (groups < 1 || beams < 1 || (int64_t)groups * beams > (int64_t)INT32_MAX) return KDA_ERR_INVALID_ARG;
  if (beams > kda::kBeamMax || num_states > kda::kBeamReorderMax) return KDA_ERR_UNSUPPORTED;
  if (num_states < 1 || !states || !row_bytes || !parents || !aligned(parents, 4)) return KDA_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)groups * beams;
  int unit[kda::kBeamReorderMax];
  Range used[kda::kBeamReorderMax + 1];
  int64_t blocks = 0;
  for (int s = 0; s < num_states; ++s) {
    if (row_bytes[s] < 0 || row_bytes[s] > INT64_MAX / 64 / rows) return KDA_ERR_INVALID_ARG;
    if (row_bytes[s] > 0 && !states[s]) return KDA_ERR_INVALID_ARG;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(states[s]) | (uintptr_t)row_bytes[s];
    unit[s] = (bits & 15) == 0 ? 16 : (bits & 3) == 0 ? 4 : 1;
    blocks += (row_bytes[s] / unit[s] + 255) / 256;
    used[s] = range_of(states[s], (size_t)(row_bytes[s] * rows));
  }
  used[num_states] = range_of(parents, (size_t)rows * 4);
  for (int i = 0; i <= num_states; ++i)
    for (int j = i + 1; j <= num_states; ++j)
      if (overlap(used[i], used[j])) return KDA_ERR_INVALID_ARG;
  if (blocks * 256 > (int64_t)UINT32_MAX) return KDA_ERR_INVALID_ARG;  // threads of a launch, for one group
  for (int u : {16, 4, 1}) {
    kda::BeamReorderArgs a;
    std::memset(&a, 0, sizeof(a));
    for (int s = 0; s < num_states; ++s)
      if (unit[s] == u) {
        a.state[a.count] = states[s];
        a.row_units[a.count++] = row_bytes[s] / u;
      }
    if (a.count == 0) continue;
    a.parents = parents;
    a.groups = groups;
    a.beams = beams;
    if (kda::launch_beam_reorder(a, u, stream) != hipSuccess) return KDA_ERR_HIP;
  }
  return KDA_OK;
}

}  // extern "C"
