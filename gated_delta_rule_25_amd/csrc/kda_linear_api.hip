// kda_linear_api.hip — the C ABI of per-head-decay linear attention
// (include/kda_linear.h): argument validation before anything is enqueued,
// the launch plan, the launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>

#include "kda_api_util.h"
#include "kda_linear.h"
#include "kda_linear_internal.h"

namespace {

using namespace kda::api;

constexpr size_t kStateBytes = (size_t)kD * kD * sizeof(float);
// The walk copies rows through 64-bit addresses; the bound is the one of the
// other prefill calls.
constexpr int kMaxHeads = 65535;
// Stretch over which the decays' gradient is summed token by token before it
// is taken from the states again.  Rounding grows with the square root of it
// and, for a constant decay, whose gradient sums the tokens' once more, with
// its power 3/2 (measured at 1024: 1.9e-6 of the result against 0.6e-6 with
// decays per token), at the price of one state written and read per stretch.
constexpr int64_t kAnchorTokens = 1024;
constexpr int64_t kAnchorTokensPerHead = 256;
constexpr int64_t kMinSegment = 512;  // a multiple of kAnchorTokensPerHead

bool linear_sizes_ok(int num_seqs, int64_t total_tokens, int num_heads, int num_qk_heads) {
  return num_seqs >= 1 && num_heads >= 1 && num_heads <= kMaxHeads && num_qk_heads >= 1 &&
         num_heads % num_qk_heads == 0 && total_tokens >= 0 && total_tokens <= (int64_t)INT32_MAX &&
         (int64_t)num_seqs * num_heads <= (int64_t)INT32_MAX / 4;
}

struct LinearPlan {
  bool segmented = false;
  bool narrow = false;
  int64_t seg = kAnchorTokens;
  int64_t slots = 0;     // segments, empty ones included
  int64_t anchored = 0;  // stretches of the decays' gradient, likewise
  int64_t boundaries = 0;  // states between them
  int64_t anchor = kAnchorTokens;
  bool own_anchors = false;  // boundary states apart from the segments'
  int blocks = 1;            // column blocks of a head
  size_t off_fsnap = 0, off_rsnap = 0, off_anchor = 0, off_decay = 0, off_change = 0, off_part = 0, off_share = 0;
  size_t bytes = 0;
};

// Whether sequences are cut into segments that run side by side and how long
// those are, and whether a walk takes half a head.  One workgroup fills a
// compute unit, so a walk per (sequence, head) leaves units idle when there are
// fewer chains than units; segments cost a pass for their contributions (two in
// the backward pass) and their states' traffic; half heads cost a second copy
// of the pair matrix but make a chain shorter (3.4 us per chunk of the dq walk
// against 4.7).
//
// Forward: segments, one per unit, from three units per chain on (8 heads x
// 131072 tokens: 367 us in segments of 4096, 440 at 1024, 3250 in one walk; 96
// heads x 8192: 226 us in one walk of half heads, 293 at 1536); half heads
// when chains are fewer than units.
// Backward, three walks a chain: segments, one per unit, from five units per
// chain on (32 heads x 8192 tokens: 290 us in segments of 1024, 338 at 512, 331
// in one walk of half heads; 48 heads: 443, 510 and 468 in one walk of whole
// ones; 64 heads: 573, 654, 518).  With more chains one walk each: whole heads
// if all chains are as long (96 heads x 8192: 690 us, segments of 1024 873; half
// heads 975 when this was chosen).  The lengths of several sequences are not
// known here, and the longest one is waited for: half heads until two rounds of
// the card are full (when this was chosen, 9 sequences of up to 2900 tokens x
// 16 heads: 157 us, whole heads 206; of up to 1200: 103 against 85).
// One rule for all sequences of a batch: one that is much longer than the rest
// is walked alone unless segment_tokens cuts it (65536 tokens among 29 sequences
// of 100 to 1136, 4 heads: 1560 us, 156 in segments of 2048).
void choose_segments(LinearPlan& pl, int num_seqs, int64_t total_tokens, int num_heads, int segment_tokens, int cus,
                     bool backward) {
  const int64_t units = (int64_t)num_seqs * num_heads;
  const bool few = (backward ? 5 : 3) * units < cus;
  if (segment_tokens > 0) {
    pl.segmented = true;
    pl.seg = segment_tokens;
  } else if (segment_tokens == 0 && few) {
    int64_t seg = (total_tokens * num_heads + cus - 1) / cus;
    seg = std::max((seg + 255) / 256 * 256, kMinSegment);
    if ((int64_t)num_seqs * seg < total_tokens) {
      pl.segmented = true;
      pl.seg = seg;
    }
  }
  if (!pl.segmented) pl.narrow = backward ? few || (num_seqs > 1 && 3 * units < 2 * cus) : units < cus;
  pl.slots = kda::linear_slots(total_tokens, num_seqs, pl.seg);
}

// One sequence, one walk each: of the heads' dv walks that start last, when
// twice as many would find a free unit as well, half heads shorten the end.
// The walks start in order (dq and dk of all heads, then dv), one to a unit; a
// dv walk takes 2 where the others take 3 (2 without the decays' gradient), by
// half heads 1.5 (96 heads x 8192 tokens on 256 units: 610, 400 and 300 us).
int whole_dv_heads(int heads, bool decay_grad, int cus) {
  const int kTimes = 64;                     // units that come free by time (in a ring)
  int64_t free_at[kTimes] = {(int64_t)cus};
  auto start = [&](int64_t& now, int64_t& walks, int time) {
    while (free_at[now % kTimes] == 0) ++now;
    const int64_t n = std::min(free_at[now % kTimes], walks);
    free_at[now % kTimes] -= n;
    free_at[(now + time) % kTimes] += n;
    walks -= n;
    return n;
  };
  int64_t now = 0, walks = 2 * (int64_t)heads;
  while (walks > 0) start(now, walks, decay_grad ? 3 : 2);
  const int64_t heavy_end = now + (decay_grad ? 3 : 2);
  walks = heads;
  while (walks > 0) {
    while (free_at[now % kTimes] == 0) ++now;
    const int64_t idle = free_at[now % kTimes];
    const int64_t n = start(now, walks, 2);
    if (walks == 0 && 2 * n <= idle && now + 2 > heavy_end) return heads - (int)n;
  }
  return heads;
}

bool plan_ok(const LinearPlan& pl, int num_heads) {
  // (one workgroup of 256 threads per stretch in a launch of below 2^32 threads,
  // beside fewer than 2^21 others: kMostShareBlocks)
  return pl.slots * num_heads <= (int64_t)INT32_MAX / 4 && pl.anchored * num_heads <= (int64_t)14 << 20;
}

LinearPlan make_fwd_plan(int num_seqs, int64_t total_tokens, int num_heads, int segment_tokens, int cus) {
  LinearPlan pl;
  choose_segments(pl, num_seqs, total_tokens, num_heads, segment_tokens, cus, false);
  if (pl.segmented) {
    const size_t units = (size_t)pl.slots * num_heads;
    size_t off = 0;
    pl.off_fsnap = off;
    off += units * kStateBytes;
    pl.off_decay = off;
    off += align256(units * sizeof(float));
    pl.bytes = off;
  }
  return pl;
}

// Pieces, each 256-byte aligned: segmented, S and dS at the segment
// boundaries ([slots][H] states); both at the boundaries of the decays'
// gradient where those are others; the segments' decays [slots][H], once
// for each direction (the same but for the order of their sums); r_t and
// c_t [column blocks][H][T]; the stretches' sums of a constant decay's
// gradient; the fp32 gradients [T, H, 128] that shared heads are summed from.
LinearPlan make_bwd_plan(int num_seqs, int64_t total_tokens, int num_heads, int num_qk_heads, int segment_tokens,
                         bool decay_grad, bool decay_per_head, bool d_final, int cus) {
  LinearPlan pl;
  choose_segments(pl, num_seqs, total_tokens, num_heads, segment_tokens, cus, true);
  const size_t units = (size_t)pl.slots * num_heads;
  const size_t rows = (size_t)total_tokens * num_heads;
  pl.anchor = decay_per_head ? kAnchorTokensPerHead : kAnchorTokens;
  if (pl.segmented) {
    // a segment's end is a boundary as well: the longest stretch of whole
    // 64-token chunks that divides it
    while (pl.seg % pl.anchor != 0) pl.anchor -= 64;  // (64 divides it)
  }
  pl.own_anchors = decay_grad && !(pl.segmented && pl.anchor == pl.seg);
  pl.anchored = decay_grad ? kda::linear_slots(total_tokens, num_seqs, pl.anchor) : 0;
  const size_t anchored = (size_t)pl.anchored * num_heads;
  if (pl.own_anchors) pl.boundaries = kda::linear_boundaries(total_tokens, num_seqs, pl.anchor, d_final);
  pl.blocks = pl.narrow ? 2 : 1;
  size_t off = 0;
  pl.off_fsnap = off;
  if (pl.segmented) off += units * kStateBytes;
  pl.off_rsnap = off;
  if (pl.segmented) off += units * kStateBytes;
  pl.off_anchor = off;
  off += 2 * (size_t)pl.boundaries * num_heads * kStateBytes;
  pl.off_decay = off;
  if (pl.segmented) off += align256(2 * units * sizeof(float));
  pl.off_change = off;
  if (decay_grad) off += align256(2 * pl.blocks * rows * sizeof(float));
  pl.off_part = off;
  if (decay_grad && decay_per_head) off += align256(anchored * sizeof(double));
  pl.off_share = off;
  if (num_qk_heads != num_heads) off += 2 * rows * kD * sizeof(float);
  pl.bytes = off;
  return pl;
}

kda_status linear_checked(const float* log_decay, int64_t count, const int32_t* cu, int num_seqs,
                          int64_t total_tokens, hipStream_t stream) {
  if (!kda::debug_checks()) return KDA_OK;
  uint32_t flags = 0;
  if (kda::run_linear_checks(log_decay, count, cu, num_seqs, total_tokens, stream, &flags) != hipSuccess)
    return KDA_ERR_HIP;
  kda::set_check_flags(flags);
  return flags ? KDA_ERR_PRECONDITION : KDA_OK;
}

bool all_aligned(const void* const* p, size_t count, uintptr_t a) {
  for (size_t i = 0; i < count; ++i)
    if (!aligned(p[i], a)) return false;
  return true;
}

// Whether an output meets an input or another output.
bool any_overlap(const Range* outs, size_t no, const Range* ins, size_t ni) {
  for (size_t i = 0; i < no; ++i) {
    for (size_t j = 0; j < ni; ++j)
      if (overlap(outs[i], ins[j])) return true;
    for (size_t j = i + 1; j < no; ++j)
      if (overlap(outs[i], outs[j])) return true;
  }
  return false;
}

// Incoming states of the segments: their own contributions, then the scan;
// forwards and, if `r` is given, backwards beside it.
hipError_t segment_states(const kda::LinearWalkArgs& f, const kda::LinearWalkArgs* r, hipStream_t stream) {
  hipError_t e = kda::launch_linear_states(f, r, stream);
  if (e != hipSuccess) return e;
  auto scan_of = [](const kda::LinearWalkArgs& w) {
    kda::LinearScanArgs s;
    std::memset(&s, 0, sizeof(s));
    s.snap = w.snap;
    s.seg_decay = w.seg_decay;
    s.init = w.init;
    s.cu = w.cu;
    s.num_seqs = w.num_seqs;
    s.total_tokens = w.total_tokens;
    s.num_heads = w.num_heads;
    s.seg = w.seg;
    return s;
  };
  kda::LinearScanArgs back;
  if (r) back = scan_of(*r);
  return kda::launch_linear_scan(scan_of(f), r ? &back : nullptr, stream);
}

}  // namespace

extern "C" {

size_t kda_linear_chunk_fwd_workspace_bytes(int num_seqs, int64_t total_tokens, int num_heads, int num_qk_heads,
                                            int d_k, int d_v, kda_dtype dtype, int segment_tokens) {
  if (!linear_sizes_ok(num_seqs, total_tokens, num_heads, num_qk_heads) || d_k != kD || d_v != kD || !dtype_ok(dtype))
    return 0;
  if (segment_tokens > 0 && segment_tokens % 64 != 0) return 0;
  const LinearPlan pl = make_fwd_plan(num_seqs, total_tokens, num_heads, segment_tokens, cu_count_for_current_device());
  return plan_ok(pl, num_heads) ? pl.bytes : 0;
}

kda_status kda_linear_chunk_fwd(const void* q, const void* k, const void* v, const float* log_decay,
                                const float* initial_state, const int32_t* cu_seqlens, int num_seqs,
                                int64_t total_tokens, int num_heads, int num_qk_heads, int decay_per_head, int d_k,
                                int d_v, kda_dtype dtype, int segment_tokens, void* o, float* final_state,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (num_seqs < 1 || num_heads < 1 || num_qk_heads < 1 || total_tokens < 0) return KDA_ERR_INVALID_ARG;
  if (d_k != kD || d_v != kD || !dtype_ok(dtype)) return KDA_ERR_UNSUPPORTED;
  if (!cu_seqlens && num_seqs != 1) return KDA_ERR_INVALID_ARG;
  if (!linear_sizes_ok(num_seqs, total_tokens, num_heads, num_qk_heads)) return KDA_ERR_INVALID_ARG;
  if (segment_tokens > 0 && segment_tokens % 64 != 0) return KDA_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!q || !k || !v || !log_decay || !o)) return KDA_ERR_INVALID_ARG;
  {
    const void* vec[] = {q, k, v, initial_state, o, final_state, workspace};
    const void* sca[] = {log_decay, cu_seqlens};
    if (!all_aligned(vec, 7, 16) || !all_aligned(sca, 2, 4)) return KDA_ERR_INVALID_ARG;
  }
  const LinearPlan pl = make_fwd_plan(num_seqs, total_tokens, num_heads, segment_tokens, cu_count_for_current_device());
  if (!plan_ok(pl, num_heads)) return KDA_ERR_INVALID_ARG;
  if (pl.bytes > 0 && (!workspace || workspace_bytes < pl.bytes)) return KDA_ERR_WORKSPACE;

  const size_t es = elem_size(dtype);
  const size_t qk = (size_t)total_tokens * num_qk_heads * kD * es, vo = (size_t)total_tokens * num_heads * kD * es;
  const int64_t decays = decay_per_head ? num_heads : total_tokens * num_heads;
  const size_t state_bytes = (size_t)num_seqs * num_heads * kStateBytes;
  const Range r_s0 = range_of(initial_state, initial_state ? state_bytes : 0);
  const Range r_fs = range_of(final_state, final_state ? state_bytes : 0);
  const Range r_cu = range_of(cu_seqlens, cu_seqlens ? (size_t)(num_seqs + 1) * sizeof(int32_t) : 0);
  const Range ins[] = {range_of(q, qk), range_of(k, qk), range_of(v, vo),
                       range_of(log_decay, (size_t)decays * sizeof(float)), r_cu};
  const Range outs[] = {range_of(o, vo), r_fs, range_of(workspace, pl.bytes)};
  if (any_overlap(outs, 3, ins, 5)) return KDA_ERR_INVALID_ARG;
  if (overlap(outs[0], r_s0) || overlap(outs[2], r_s0)) return KDA_ERR_INVALID_ARG;
  // final_state may be exactly initial_state (in-place continuation)
  if (overlap(r_fs, r_s0) && !(r_fs.lo == r_s0.lo && r_fs.hi == r_s0.hi)) return KDA_ERR_INVALID_ARG;
  {
    const kda_status cs = linear_checked(log_decay, total_tokens > 0 ? decays : 0, cu_seqlens, num_seqs, total_tokens,
                                         stream);
    if (cs != KDA_OK) return cs;
  }

  char* ws = static_cast<char*>(workspace);
  kda::LinearWalkArgs w;
  std::memset(&w, 0, sizeof(w));
  w.q = q;
  w.k = k;
  w.v = v;
  w.q_heads = w.k_heads = num_qk_heads;
  w.v_heads = w.x_heads = num_heads;
  w.log_decay = log_decay;
  w.decay_per_head = decay_per_head != 0 && total_tokens > 0;  // (without tokens there may be no decays to read)
  w.cu = cu_seqlens;
  w.num_seqs = num_seqs;
  w.total_tokens = total_tokens;
  w.num_heads = num_heads;
  w.bf16 = dtype == KDA_DTYPE_BF16;
  w.seg = (int)pl.seg;
  w.anchor = (int)pl.seg;
  w.segmented = pl.segmented;
  w.units = (pl.segmented ? pl.slots : (int64_t)num_seqs) * num_heads;
  w.narrow = pl.narrow;
  w.init = initial_state;
  w.fin = final_state;
  w.o = o;
  if (pl.segmented) {
    w.snap = reinterpret_cast<float*>(ws + pl.off_fsnap);
    w.seg_decay = reinterpret_cast<float*>(ws + pl.off_decay);
    if (segment_states(w, nullptr, stream) != hipSuccess) return KDA_ERR_HIP;
  }
  return kda::launch_linear_walk(w, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

size_t kda_linear_chunk_bwd_workspace_bytes(int num_seqs, int64_t total_tokens, int num_heads, int num_qk_heads,
                                            int decay_per_head, int need_d_log_decay, int with_d_final_state, int d_k,
                                            int d_v, kda_dtype dtype, int segment_tokens) {
  if (!linear_sizes_ok(num_seqs, total_tokens, num_heads, num_qk_heads) || d_k != kD || d_v != kD || !dtype_ok(dtype))
    return 0;
  if (segment_tokens > 0 && segment_tokens % 64 != 0) return 0;
  const LinearPlan pl = make_bwd_plan(num_seqs, total_tokens, num_heads, num_qk_heads, segment_tokens,
                                      need_d_log_decay != 0, decay_per_head != 0, with_d_final_state != 0,
                                      cu_count_for_current_device());
  return plan_ok(pl, num_heads) ? pl.bytes : 0;
}

kda_status kda_linear_chunk_bwd(const void* q, const void* k, const void* v, const float* log_decay,
                                const float* initial_state, const int32_t* cu_seqlens, const void* d_o,
                                const float* d_final_state, int num_seqs, int64_t total_tokens, int num_heads,
                                int num_qk_heads, int decay_per_head, int d_k, int d_v, kda_dtype dtype,
                                int segment_tokens, void* dq, void* dk, void* dv, float* d_log_decay,
                                float* d_initial_state, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (num_seqs < 1 || num_heads < 1 || num_qk_heads < 1 || total_tokens < 0) return KDA_ERR_INVALID_ARG;
  if (d_k != kD || d_v != kD || !dtype_ok(dtype)) return KDA_ERR_UNSUPPORTED;
  if (!cu_seqlens && num_seqs != 1) return KDA_ERR_INVALID_ARG;
  if (!linear_sizes_ok(num_seqs, total_tokens, num_heads, num_qk_heads)) return KDA_ERR_INVALID_ARG;
  if (segment_tokens > 0 && segment_tokens % 64 != 0) return KDA_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!q || !k || !v || !log_decay || !d_o || !dq || !dk || !dv)) return KDA_ERR_INVALID_ARG;
  {
    const void* vec[] = {q, k, v, initial_state, d_o, d_final_state, dq, dk, dv, d_initial_state, workspace};
    const void* sca[] = {log_decay, cu_seqlens, d_log_decay};
    if (!all_aligned(vec, 11, 16) || !all_aligned(sca, 3, 4)) return KDA_ERR_INVALID_ARG;
  }
  const bool grad = d_log_decay != nullptr, per_head = decay_per_head != 0;
  const LinearPlan pl = make_bwd_plan(num_seqs, total_tokens, num_heads, num_qk_heads, segment_tokens, grad, per_head,
                                      d_final_state != nullptr, cu_count_for_current_device());
  if (!plan_ok(pl, num_heads)) return KDA_ERR_INVALID_ARG;
  if (pl.bytes > 0 && (!workspace || workspace_bytes < pl.bytes)) return KDA_ERR_WORKSPACE;

  const size_t es = elem_size(dtype);
  const size_t qk = (size_t)total_tokens * num_qk_heads * kD * es, vo = (size_t)total_tokens * num_heads * kD * es;
  const int64_t decays = per_head ? num_heads : total_tokens * num_heads;
  const size_t state_bytes = (size_t)num_seqs * num_heads * kStateBytes;
  const Range ins[] = {range_of(q, qk),
                       range_of(k, qk),
                       range_of(v, vo),
                       range_of(log_decay, (size_t)decays * sizeof(float)),
                       range_of(cu_seqlens, cu_seqlens ? (size_t)(num_seqs + 1) * sizeof(int32_t) : 0),
                       range_of(initial_state, initial_state ? state_bytes : 0),
                       range_of(d_o, vo),
                       range_of(d_final_state, d_final_state ? state_bytes : 0)};
  const Range outs[] = {range_of(dq, qk),
                        range_of(dk, qk),
                        range_of(dv, vo),
                        range_of(d_log_decay, d_log_decay ? (size_t)decays * sizeof(float) : 0),
                        range_of(d_initial_state, d_initial_state ? state_bytes : 0),
                        range_of(workspace, pl.bytes)};
  if (any_overlap(outs, 6, ins, 8)) return KDA_ERR_INVALID_ARG;
  {
    const kda_status cs = linear_checked(log_decay, total_tokens > 0 ? decays : 0, cu_seqlens, num_seqs, total_tokens,
                                         stream);
    if (cs != KDA_OK) return cs;
  }

  char* ws = static_cast<char*>(workspace);
  const bool shared = num_qk_heads != num_heads;
  const size_t rows = (size_t)total_tokens * num_heads;
  float* share = reinterpret_cast<float*>(ws + pl.off_share);  // of dq, then of dk
  float* fsnap = pl.segmented ? reinterpret_cast<float*>(ws + pl.off_fsnap) : nullptr;
  float* rsnap = pl.segmented ? reinterpret_cast<float*>(ws + pl.off_rsnap) : nullptr;
  const size_t anchored = (size_t)pl.anchored * num_heads;
  float* anchors = reinterpret_cast<float*>(ws + pl.off_anchor);
  float* s_anchors = pl.own_anchors ? anchors : fsnap;
  float* ds_anchors = pl.own_anchors ? anchors + (size_t)pl.boundaries * num_heads * kD * kD : rsnap;
  float* change = reinterpret_cast<float*>(ws + pl.off_change);

  kda::LinearWalkArgs base;
  std::memset(&base, 0, sizeof(base));
  base.log_decay = log_decay;
  base.decay_per_head = per_head && total_tokens > 0;  // (without tokens there may be no decays to read)
  base.cu = cu_seqlens;
  base.num_seqs = num_seqs;
  base.total_tokens = total_tokens;
  base.num_heads = num_heads;
  base.bf16 = dtype == KDA_DTYPE_BF16;
  base.seg = (int)pl.seg;
  base.anchor = (int)pl.anchor;
  base.end_state = d_final_state != nullptr;
  base.segmented = pl.segmented;
  base.narrow = pl.narrow;
  base.units = (pl.segmented ? pl.slots : (int64_t)num_seqs) * num_heads;
  base.seg_decay = reinterpret_cast<float*>(ws + pl.off_decay);
  const int hq = num_qk_heads, hv = num_heads;
  auto role = [](kda::LinearWalkArgs w, const void* a, int ah, const void* b, int bh, const void* c, int ch) {
    w.q = a;
    w.q_heads = ah;
    w.k = b;
    w.k_heads = bh;
    w.v = c;
    w.v_heads = ch;
    w.x_heads = ch;
    return w;
  };
  kda::LinearGradArgs g;
  g.decay_grad = grad;
  g.dv_whole = num_seqs == 1 && !pl.segmented && !pl.narrow
                   ? whole_dv_heads(num_heads, grad, cu_count_for_current_device())
                   : num_heads;
  g.dq = role(base, d_o, hv, v, hv, k, hq);
  g.dq.init = initial_state;
  g.dq.snap = fsnap;
  g.dq.x = q;
  g.dq.x_heads = hq;
  g.dq.anchors = s_anchors;
  g.dq.change = change;
  g.dq.o = shared ? static_cast<void*>(share) : dq;
  g.dq.o_f32 = shared;
  base.init = d_final_state;
  base.snap = rsnap;
  g.dk = role(base, v, hv, d_o, hv, q, hq);
  g.dk.x = k;
  g.dk.x_heads = hq;
  g.dk.anchors = ds_anchors;
  g.dk.change = change + pl.blocks * rows;
  g.dk.o = shared ? static_cast<void*>(share + rows * kD) : dk;
  g.dk.o_f32 = shared;
  g.dv = role(base, k, hq, q, hq, d_o, hv);
  g.dv.fin = d_initial_state;
  g.dv.o = dv;
  if (pl.segmented) {
    kda::LinearWalkArgs f = role(g.dq, nullptr, hq, k, hq, v, hv);
    kda::LinearWalkArgs r = g.dv;
    r.seg_decay += (size_t)pl.slots * num_heads;
    if (segment_states(f, &r, stream) != hipSuccess) return KDA_ERR_HIP;
  }
  if (kda::launch_linear_grad(g, stream) != hipSuccess) return KDA_ERR_HIP;
  kda::LinearFinishArgs f;
  std::memset(&f, 0, sizeof(f));
  f.decay.s_anchors = s_anchors;
  f.decay.ds_anchors = ds_anchors;
  f.decay.own = pl.own_anchors;
  f.decay.r = change;
  f.decay.c = change + pl.blocks * rows;
  f.decay.blocks = pl.blocks;
  f.decay.has_d_final = d_final_state != nullptr;
  f.decay.d_log_decay = per_head ? nullptr : d_log_decay;
  f.decay.part = per_head ? reinterpret_cast<double*>(ws + pl.off_part) : nullptr;
  f.decay.cu = cu_seqlens;
  f.decay.num_seqs = num_seqs;
  f.decay.total_tokens = total_tokens;
  f.decay.num_heads = num_heads;
  f.decay.anchor = (int)pl.anchor;
  f.decay_blocks = grad && total_tokens > 0;
  f.share = shared ? share : nullptr;
  f.dq = dq;
  f.dk = dk;
  f.qk_heads = num_qk_heads;
  if (kda::launch_linear_finish(f, base.bf16, stream) != hipSuccess) return KDA_ERR_HIP;
  if (grad && per_head) {
    // (no tokens: no stretch, and the sums are zero)
    const int64_t units = total_tokens > 0 ? (int64_t)anchored : 0;
    if (kda::launch_linear_decay_sum(reinterpret_cast<double*>(ws + pl.off_part), d_log_decay, units, num_heads,
                                     stream) != hipSuccess)
      return KDA_ERR_HIP;
  }
  return KDA_OK;
}

kda_status kda_linear_decode_step(float* state, const void* q, const void* k, const void* v, const float* log_decay,
                                  int num_seqs, int num_heads, int num_qk_heads, int decay_per_head, int d_k, int d_v,
                                  kda_dtype dtype, void* o, hipStream_t stream) {
  if (num_seqs < 1 || num_heads < 1 || num_qk_heads < 1) return KDA_ERR_INVALID_ARG;
  if (d_k != kD || d_v != kD || !dtype_ok(dtype)) return KDA_ERR_UNSUPPORTED;
  if (!linear_sizes_ok(num_seqs, 0, num_heads, num_qk_heads)) return KDA_ERR_INVALID_ARG;
  if (!state || !q || !k || !v || !log_decay || !o) return KDA_ERR_INVALID_ARG;
  const size_t es = elem_size(dtype);
  if (!aligned(state, 16) || !aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(o, es) ||
      !aligned(log_decay, 4))
    return KDA_ERR_INVALID_ARG;
  const size_t units = (size_t)num_seqs * num_heads;
  if (units * 256 > UINT32_MAX) return KDA_ERR_INVALID_ARG;  // a workgroup each, below 2^32 threads
  const size_t qk = (size_t)num_seqs * num_qk_heads * kD * es;
  const int64_t decays = decay_per_head ? num_heads : (int64_t)units;
  const Range ins[] = {range_of(q, qk), range_of(k, qk), range_of(v, units * kD * es),
                       range_of(log_decay, (size_t)decays * sizeof(float))};
  const Range outs[] = {range_of(state, units * kStateBytes), range_of(o, units * kD * es)};
  if (any_overlap(outs, 2, ins, 4)) return KDA_ERR_INVALID_ARG;
  {
    const kda_status cs = linear_checked(log_decay, decays, nullptr, num_seqs, 0, stream);
    if (cs != KDA_OK) return cs;
  }
  kda::LinearDecodeArgs a;
  std::memset(&a, 0, sizeof(a));
  a.state = state;
  a.q = q;
  a.k = k;
  a.v = v;
  a.log_decay = log_decay;
  a.decay_per_head = decay_per_head != 0;
  a.o = o;
  a.num_seqs = num_seqs;
  a.num_heads = num_heads;
  a.qk_heads = num_qk_heads;
  a.bf16 = dtype == KDA_DTYPE_BF16;
  return kda::launch_linear_decode(a, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // extern "C"
