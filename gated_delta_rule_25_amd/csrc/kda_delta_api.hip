// kda_delta_api.hip — the C ABI of the gated delta rule with one decay per head
// (include/kda_delta.h): argument validation before anything is enqueued, the
// launch plan, the launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "kda_api_util.h"
#include "kda_delta.h"
#include "kda_delta_internal.h"

namespace {

using namespace kda::api;

constexpr size_t kStateBytes = (size_t)kD * kD * sizeof(float);
constexpr int kMaxHeads = 65535;
constexpr int64_t kMinSegment = 256;

bool delta_sizes_ok(int num_seqs, int64_t total_tokens, int num_heads, int num_qk_heads) {
  return num_seqs >= 1 && num_heads >= 1 && num_heads <= kMaxHeads && num_qk_heads >= 1 &&
         num_heads % num_qk_heads == 0 && total_tokens >= 0 && total_tokens <= (int64_t)INT32_MAX &&
         (int64_t)num_seqs * num_heads <= (int64_t)INT32_MAX / 4;
}

struct DeltaPlan {
  bool segmented = false;
  bool both = false, led = false;  // DeltaWalkArgs
  int64_t seg = kMinSegment;
  int64_t slots = 0;  // segments, empty ones included
  size_t off_blocks = 0, off_pairs = 0;
  size_t bytes = 0;
};

// How m segments of s tokens of every sequence and head (units of them) are walked,
// and what that takes in us.  A walk of outputs is two workgroups, one per half of the
// value columns, each of which fills a compute unit and takes 43 ns a token (fp32:
// 72).  Before it, contributions and transitions are formed of all segments but the
// last.  They have a workgroup of their own each while all run at once, else one for
// both, which takes 50 ns a token (82) for 33 (62) and half the workgroups (8 heads x
// 131072 tokens, 256 units: 545 -> 400 us; one head x 8192 tokens, where all run at
// once, 116 -> 127 us for the call).  They can be led by the walk of the first
// segments' outputs, for which none is needed then (32 heads x 32768 tokens: 1002 ->
// 854 us; one head x 8192: 116 -> 123).  The scan takes 3.7 us a segment, the two more
// launches 5 us.  The backward pass (back) walks twice, and with segments forms
// contributions and transitions of all, and in one more walk the contributions to
// what reaches their ends.
struct Cut {
  bool both = false, led = false;  // DeltaWalkArgs
  double us = 0.0;
};
Cut cut_of(int64_t m, int64_t s, int64_t units, bool bf16, bool back, bool led, int cus) {
  const double token = bf16 ? 0.043 : 0.072;
  auto rounds = [&](int64_t workgroups) { return (double)((workgroups + cus - 1) / cus); };
  const int64_t formed = units * std::max(back ? m : led ? m - 2 : m - 1, (int64_t)0), lead = led ? 2 * units : 0;
  Cut c;
  c.led = led;
  c.both = 4 * formed + lead > cus;
  const double first = c.both ? rounds(2 * formed + lead) * (bf16 ? 0.05 : 0.082) : led ? token : bf16 ? 0.033 : 0.062;
  const double walks = first + (back ? 3 : 1) * rounds(2 * units * (led ? m - 1 : m)) * token;
  c.us = walks * (double)s + (back ? 7.4 : 3.7) * (double)m + (back ? 10.0 : 5.0);
  return c;
}

// Whether and how sequences of `length` tokens are cut into segments that run side by
// side: what takes least.  Measured with 256 units in bf16, whole and cut so: one head,
// 512 tokens 46 and 52 us (whole is taken), 1024 tokens 68 and 59, 8192 tokens 370 and
// 116; 32 heads of 8192 tokens 406 and 248, 48 heads of 32768 tokens 1599 and 1187.
void choose_cut(DeltaPlan& pl, int64_t length, int64_t units, bool bf16, bool back, int cus) {
  const double token = bf16 ? 0.043 : 0.072;
  double best = (back ? 2 : 1) * (double)((2 * units + cus - 1) / cus) * (double)length * token;
  // (behind the least of the scan's and one round's sum nothing shorter is better)
  const int64_t most = (int64_t)(2.0 * std::sqrt((double)length * token / (back ? 7.4 : 3.7))) + 1;
  for (int64_t n = 2; n <= most; ++n) {
    const int64_t s = ((length + n - 1) / n + 63) / 64 * 64;
    if (s < kMinSegment) break;
    for (int led = 0; led < (back ? 1 : 2); ++led) {
      const Cut c = cut_of((length + s - 1) / s, s, units, bf16, back, led, cus);
      if (c.us < best) {
        best = c.us;
        pl.segmented = true;
        pl.seg = s;
        pl.both = c.both;
        pl.led = c.led;
      }
    }
  }
}

DeltaPlan make_plan(int num_seqs, int64_t total_tokens, int num_heads, bool bf16, bool back, int segment_tokens,
                    int cus) {
  DeltaPlan pl;
  const int64_t units = (int64_t)num_seqs * num_heads;
  // (the lengths are on the device: their mean)
  const int64_t length = (total_tokens + num_seqs - 1) / num_seqs;
  if (segment_tokens > 0) {
    const int64_t m = (length + segment_tokens - 1) / segment_tokens;
    const Cut plain = cut_of(m, segment_tokens, units, bf16, back, false, cus);
    const Cut led = cut_of(m, segment_tokens, units, bf16, back, !back, cus);
    const Cut& c = led.us < plain.us ? led : plain;
    pl.segmented = true;
    pl.seg = segment_tokens;
    pl.both = c.both;
    pl.led = c.led;
  } else if (segment_tokens == 0) {
    choose_cut(pl, length, units, bf16, back, cus);
  }
  const int chunk = kda::delta_chunk(bf16);
  size_t off = 0;
  pl.off_blocks = off;
  if (total_tokens > 0)
    off += align256((size_t)kda::delta_chunk_slots(total_tokens, num_seqs, chunk) * num_heads *
                    kda::delta_block_bytes(chunk));
  pl.off_pairs = off;
  if (pl.segmented) {
    pl.slots = kda::linear_slots(total_tokens, num_seqs, pl.seg);
    off += (size_t)pl.slots * num_heads * 2 * kStateBytes;
  }
  pl.bytes = off;
  return pl;
}

// Stretch over which the decays' gradient is summed token by token before it is
// taken from the states again.
constexpr int kAnchorTokens = 512;

struct DeltaBackPlan {
  DeltaPlan fwd;
  int64_t anchored = 0;
  size_t off_e = 0, off_u = 0, off_s = 0, off_ds = 0, off_change = 0, off_beta = 0, off_anchor = 0, off_rstates = 0;
  size_t off_yh = 0, off_exps = 0, exps_bytes = 0;
  size_t anchor_bytes = 0, change_bytes = 0;
  size_t bytes = 0;
};

// Pieces, each 256-byte aligned: the forward plan's (the prep kernel's blocks,
// segments' contributions and transitions); e and the images of S and dS' of
// every chunk; u; in bf16 dv / beta in fp16 and the exponents of the columns; the sums over each column tile of o . do, v . dv and e . y; S
// and dS at the boundaries of stretches; what reaches the segments' ends.
DeltaBackPlan make_bwd_plan(int num_seqs, int64_t total_tokens, int num_heads, bool bf16, int segment_tokens, int cus) {
  DeltaBackPlan pl;
  pl.fwd = make_plan(num_seqs, total_tokens, num_heads, bf16, true, segment_tokens, cus);
  const int chunk = kda::delta_chunk(bf16);
  const size_t es = bf16 ? 2 : 4;
  const size_t rows = (size_t)total_tokens * num_heads;
  const size_t chunks = total_tokens > 0 ? (size_t)kda::delta_chunk_slots(total_tokens, num_seqs, chunk) * num_heads : 0;
  size_t off = pl.fwd.bytes;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align256(bytes);
    return at;
  };
  pl.off_e = take(chunks * chunk * kD * sizeof(float));
  pl.off_u = take(rows * kD * es);
  pl.off_s = take(chunks * kD * kD * es);
  pl.off_ds = take(chunks * kD * kD * es);
  if (bf16) {
    pl.off_yh = take(rows * kD * 2);
    pl.exps_bytes = align256(chunks * kD * sizeof(int));
    pl.off_exps = take(2 * pl.exps_bytes);
  }
  pl.change_bytes = align256(8 * rows * sizeof(float));
  pl.off_change = take(2 * pl.change_bytes);
  pl.off_beta = take(8 * rows * sizeof(float));
  pl.anchored = kda::linear_slots(total_tokens, num_seqs, kAnchorTokens);
  pl.anchor_bytes = (size_t)kda::linear_boundaries(total_tokens, num_seqs, kAnchorTokens, true) * num_heads * kStateBytes;
  pl.off_anchor = take(2 * pl.anchor_bytes);
  if (pl.fwd.segmented) pl.off_rstates = take((size_t)pl.fwd.slots * num_heads * kStateBytes);
  pl.bytes = off;
  return pl;
}

bool plan_ok(const DeltaPlan& pl, int num_heads) { return pl.slots * num_heads <= (int64_t)INT32_MAX / 4; }

bool back_plan_ok(const DeltaBackPlan& pl, int num_heads) {
  // (one workgroup of 256 threads per stretch in a launch of below 2^32 threads)
  return plan_ok(pl.fwd, num_heads) && pl.anchored * num_heads <= (int64_t)14 << 20;
}

kda_status delta_checked(const void* k, kda_dtype dtype, int64_t k_rows, const float* log_decay, const float* beta,
                         int64_t count, const int32_t* cu, int num_seqs, int64_t total_tokens, hipStream_t stream) {
  if (!kda::debug_checks()) return KDA_OK;
  uint32_t flags = 0;
  if (kda::run_delta_checks(k, dtype == KDA_DTYPE_BF16, k_rows, log_decay, beta, count, cu, num_seqs, total_tokens,
                            stream, &flags) != hipSuccess)
    return KDA_ERR_HIP;
  kda::set_check_flags(flags);
  return flags ? KDA_ERR_PRECONDITION : KDA_OK;
}

// What comes before a forward walk: the chunks' blocks and, with segments, the
// states that enter them.
hipError_t begin_walk(kda::DeltaWalkArgs& w, const DeltaPlan& pl, char* ws, hipStream_t stream) {
  w.blocks = ws + pl.off_blocks;
  w.seg = (int)pl.seg;
  w.segmented = pl.segmented;
  w.both = pl.both;
  w.led = pl.led;
  w.units = (pl.segmented ? pl.slots : (int64_t)w.num_seqs) * w.num_heads;
  if (w.total_tokens > 0) {
    kda::DeltaPrepArgs a;
    std::memset(&a, 0, sizeof(a));
    a.k = w.k;
    a.log_decay = w.log_decay;
    a.beta = w.beta;
    a.cu = w.cu;
    a.num_seqs = w.num_seqs;
    a.total_tokens = w.total_tokens;
    a.num_heads = w.num_heads;
    a.qk_heads = w.qk_heads;
    a.bf16 = w.bf16;
    a.blocks = ws + pl.off_blocks;
    const hipError_t e = kda::launch_delta_prep(a, stream);
    if (e != hipSuccess) return e;
  }
  if (!pl.segmented) return hipSuccess;
  w.pairs = reinterpret_cast<float*>(ws + pl.off_pairs);
  kda::DeltaWalkArgs pairs = w;
  if (!w.led) {
    pairs.init = nullptr;
    pairs.fin = nullptr;
  }
  hipError_t e = kda::launch_delta_pairs(pairs, stream);
  if (e != hipSuccess) return e;
  kda::DeltaScanArgs s;
  std::memset(&s, 0, sizeof(s));
  s.pairs = w.pairs;
  s.led = w.led;
  s.init = w.init;
  s.log_decay = w.log_decay;
  s.cu = w.cu;
  s.num_seqs = w.num_seqs;
  s.total_tokens = w.total_tokens;
  s.num_heads = w.num_heads;
  s.seg = w.seg;
  // (the walk takes every state from the scan: a final state in the initial one's place is written by a
  // sequence's last segment while its first one may yet have to begin)
  w.init = nullptr;
  return kda::launch_delta_scan(s, stream);
}

}  // namespace

extern "C" {

size_t kda_delta_chunk_fwd_workspace_bytes(int num_seqs, int64_t total_tokens, int num_heads, int num_qk_heads,
                                           int d_k, int d_v, kda_dtype dtype, int segment_tokens) {
  if (!delta_sizes_ok(num_seqs, total_tokens, num_heads, num_qk_heads) || d_k != kD || d_v != kD || !dtype_ok(dtype))
    return 0;
  if (segment_tokens > 0 && segment_tokens % 64 != 0) return 0;
  const DeltaPlan pl = make_plan(num_seqs, total_tokens, num_heads, dtype == KDA_DTYPE_BF16, false, segment_tokens,
                                     cu_count_for_current_device());
  return plan_ok(pl, num_heads) ? pl.bytes : 0;
}

kda_status kda_delta_chunk_fwd(const void* q, const void* k, const void* v, const float* log_decay, const float* beta,
                               const float* initial_state, const int32_t* cu_seqlens, int num_seqs,
                               int64_t total_tokens, int num_heads, int num_qk_heads, int d_k, int d_v,
                               kda_dtype dtype, int segment_tokens, void* o, float* final_state, void* workspace,
                               size_t workspace_bytes, hipStream_t stream) {
  if (num_seqs < 1 || num_heads < 1 || num_qk_heads < 1 || total_tokens < 0) return KDA_ERR_INVALID_ARG;
  if (d_k != kD || d_v != kD || !dtype_ok(dtype)) return KDA_ERR_UNSUPPORTED;
  if (!cu_seqlens && num_seqs != 1) return KDA_ERR_INVALID_ARG;
  if (!delta_sizes_ok(num_seqs, total_tokens, num_heads, num_qk_heads)) return KDA_ERR_INVALID_ARG;
  if (segment_tokens > 0 && segment_tokens % 64 != 0) return KDA_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!q || !k || !v || !log_decay || !beta || !o)) return KDA_ERR_INVALID_ARG;
  {
    const void* vec[] = {q, k, v, initial_state, o, final_state, workspace};
    const void* sca[] = {log_decay, beta, cu_seqlens};
    if (!all_aligned(vec, 7, 16) || !all_aligned(sca, 3, 4)) return KDA_ERR_INVALID_ARG;
  }
  const bool bf16 = dtype == KDA_DTYPE_BF16;
  const DeltaPlan pl =
      make_plan(num_seqs, total_tokens, num_heads, bf16, false, segment_tokens, cu_count_for_current_device());
  if (!plan_ok(pl, num_heads)) return KDA_ERR_INVALID_ARG;
  if (pl.bytes > 0 && (!workspace || workspace_bytes < pl.bytes)) return KDA_ERR_WORKSPACE;

  const size_t es = elem_size(dtype);
  const size_t qk = (size_t)total_tokens * num_qk_heads * kD * es, vo = (size_t)total_tokens * num_heads * kD * es;
  const size_t scalars = (size_t)total_tokens * num_heads * sizeof(float);
  const size_t state_bytes = (size_t)num_seqs * num_heads * kStateBytes;
  const Range r_s0 = range_of(initial_state, initial_state ? state_bytes : 0);
  const Range r_fs = range_of(final_state, final_state ? state_bytes : 0);
  const Range ins[] = {range_of(q, qk),        range_of(k, qk),         range_of(v, vo), range_of(log_decay, scalars),
                       range_of(beta, scalars), range_of(cu_seqlens, cu_seqlens ? (size_t)(num_seqs + 1) * 4 : 0)};
  const Range outs[] = {range_of(o, vo), r_fs, range_of(workspace, pl.bytes)};
  if (any_overlap(outs, 3, ins, 6)) return KDA_ERR_INVALID_ARG;
  if (overlap(outs[0], r_s0) || overlap(outs[2], r_s0)) return KDA_ERR_INVALID_ARG;
  // final_state may be exactly initial_state (in-place continuation)
  if (overlap(r_fs, r_s0) && !(r_fs.lo == r_s0.lo && r_fs.hi == r_s0.hi)) return KDA_ERR_INVALID_ARG;
  {
    const kda_status cs = delta_checked(k, dtype, total_tokens * num_qk_heads, log_decay, beta, total_tokens * num_heads,
                                        cu_seqlens, num_seqs, total_tokens, stream);
    if (cs != KDA_OK) return cs;
  }

  kda::DeltaWalkArgs w;
  std::memset(&w, 0, sizeof(w));
  w.q = q;
  w.k = k;
  w.v = v;
  w.log_decay = log_decay;
  w.beta = beta;
  w.cu = cu_seqlens;
  w.num_seqs = num_seqs;
  w.total_tokens = total_tokens;
  w.num_heads = num_heads;
  w.qk_heads = num_qk_heads;
  w.bf16 = bf16;
  w.init = initial_state;
  w.fin = final_state;
  w.o = o;
  if (begin_walk(w, pl, static_cast<char*>(workspace), stream) != hipSuccess) return KDA_ERR_HIP;
  return kda::launch_delta_walk(w, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

size_t kda_delta_chunk_bwd_workspace_bytes(int num_seqs, int64_t total_tokens, int num_heads, int num_qk_heads,
                                           int d_k, int d_v, kda_dtype dtype, int segment_tokens) {
  if (!delta_sizes_ok(num_seqs, total_tokens, num_heads, num_qk_heads) || d_k != kD || d_v != kD || !dtype_ok(dtype))
    return 0;
  if (segment_tokens > 0 && segment_tokens % 64 != 0) return 0;
  const DeltaBackPlan pl = make_bwd_plan(num_seqs, total_tokens, num_heads, dtype == KDA_DTYPE_BF16, segment_tokens,
                                         cu_count_for_current_device());
  return back_plan_ok(pl, num_heads) ? pl.bytes : 0;
}

kda_status kda_delta_chunk_bwd(const void* q, const void* k, const void* v, const float* log_decay, const float* beta,
                               const float* initial_state, const int32_t* cu_seqlens, const void* d_o,
                               const float* d_final_state, int num_seqs, int64_t total_tokens, int num_heads,
                               int num_qk_heads, int d_k, int d_v, kda_dtype dtype, int segment_tokens, void* dq,
                               void* dk, void* dv, float* d_log_decay, float* dbeta, float* d_initial_state,
                               void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (num_seqs < 1 || num_heads < 1 || num_qk_heads < 1 || total_tokens < 0) return KDA_ERR_INVALID_ARG;
  if (d_k != kD || d_v != kD || !dtype_ok(dtype)) return KDA_ERR_UNSUPPORTED;
  if (!cu_seqlens && num_seqs != 1) return KDA_ERR_INVALID_ARG;
  if (!delta_sizes_ok(num_seqs, total_tokens, num_heads, num_qk_heads)) return KDA_ERR_INVALID_ARG;
  if (segment_tokens > 0 && segment_tokens % 64 != 0) return KDA_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!q || !k || !v || !log_decay || !beta || !d_o || !dq || !dk || !dv))
    return KDA_ERR_INVALID_ARG;
  {
    const void* vec[] = {q, k, v, initial_state, d_o, d_final_state, dq, dk, dv, d_initial_state, workspace};
    const void* sca[] = {log_decay, beta, cu_seqlens, d_log_decay, dbeta};
    if (!all_aligned(vec, 11, 16) || !all_aligned(sca, 5, 4)) return KDA_ERR_INVALID_ARG;
  }
  const bool bf16 = dtype == KDA_DTYPE_BF16;
  const DeltaBackPlan pl =
      make_bwd_plan(num_seqs, total_tokens, num_heads, bf16, segment_tokens, cu_count_for_current_device());
  if (!back_plan_ok(pl, num_heads)) return KDA_ERR_INVALID_ARG;
  if (pl.bytes > 0 && (!workspace || workspace_bytes < pl.bytes)) return KDA_ERR_WORKSPACE;

  const size_t es = elem_size(dtype);
  const size_t qk = (size_t)total_tokens * num_qk_heads * kD * es, vo = (size_t)total_tokens * num_heads * kD * es;
  const size_t scalars = (size_t)total_tokens * num_heads * sizeof(float);
  const size_t state_bytes = (size_t)num_seqs * num_heads * kStateBytes;
  const Range ins[] = {range_of(q, qk), range_of(k, qk), range_of(v, vo), range_of(d_o, vo),
                       range_of(log_decay, scalars), range_of(beta, scalars), range_of(initial_state, state_bytes),
                       range_of(d_final_state, state_bytes),
                       range_of(cu_seqlens, cu_seqlens ? (size_t)(num_seqs + 1) * 4 : 0)};
  const Range outs[] = {range_of(dq, qk), range_of(dk, qk), range_of(dv, vo), range_of(d_log_decay, scalars),
                        range_of(dbeta, scalars), range_of(d_initial_state, state_bytes),
                        range_of(workspace, pl.bytes)};
  if (any_overlap(outs, 7, ins, 9)) return KDA_ERR_INVALID_ARG;
  {
    const kda_status cs = delta_checked(k, dtype, total_tokens * num_qk_heads, log_decay, beta, total_tokens * num_heads,
                                        cu_seqlens, num_seqs, total_tokens, stream);
    if (cs != KDA_OK) return cs;
  }

  char* ws = static_cast<char*>(workspace);
  float* change = reinterpret_cast<float*>(ws + pl.off_change);
  float* anchors = reinterpret_cast<float*>(ws + pl.off_anchor);
  kda::DeltaWalkArgs w;
  std::memset(&w, 0, sizeof(w));
  w.q = q;
  w.k = k;
  w.v = v;
  w.log_decay = log_decay;
  w.beta = beta;
  w.cu = cu_seqlens;
  w.num_seqs = num_seqs;
  w.total_tokens = total_tokens;
  w.num_heads = num_heads;
  w.qk_heads = num_qk_heads;
  w.bf16 = bf16;
  w.init = initial_state;
  w.all_pairs = true;
  kda::DeltaSaveArgs& sv = w.save;
  sv.d_o = d_o;
  sv.s = ws + pl.off_s;
  sv.u = ws + pl.off_u;
  sv.e = reinterpret_cast<float*>(ws + pl.off_e);
  sv.exps = bf16 ? reinterpret_cast<int*>(ws + pl.off_exps) : nullptr;
  sv.change = d_log_decay ? change : nullptr;
  sv.anchors = d_log_decay ? anchors : nullptr;
  sv.anchor = kAnchorTokens;
  sv.end_state = d_final_state != nullptr;

  kda::DeltaBackArgs b;
  std::memset(&b, 0, sizeof(b));
  b.q = q;
  b.k = k;
  b.v = v;
  b.d_o = d_o;
  b.e = sv.e;
  b.cu = cu_seqlens;
  b.num_seqs = num_seqs;
  b.total_tokens = total_tokens;
  b.num_heads = num_heads;
  b.qk_heads = num_qk_heads;
  b.bf16 = bf16;
  b.d_final = d_final_state;
  b.d_initial = d_initial_state;
  b.dv = dv;
  b.ds = ws + pl.off_ds;
  b.yh = bf16 ? ws + pl.off_yh : nullptr;
  b.exps = bf16 ? reinterpret_cast<int*>(ws + pl.off_exps + pl.exps_bytes) : nullptr;
  b.change = d_log_decay ? change + pl.change_bytes / sizeof(float) : nullptr;
  b.beta_part = dbeta ? reinterpret_cast<float*>(ws + pl.off_beta) : nullptr;
  b.anchors = d_log_decay ? anchors + pl.anchor_bytes / sizeof(float) : nullptr;
  b.anchor = kAnchorTokens;
  b.end_state = sv.end_state;

  if (total_tokens > 0) {
    if (begin_walk(w, pl.fwd, ws, stream) != hipSuccess) return KDA_ERR_HIP;
    if (kda::launch_delta_save(w, stream) != hipSuccess) return KDA_ERR_HIP;
  }
  b.blocks = w.blocks;
  b.seg = w.seg;
  b.segmented = w.segmented;
  b.units = total_tokens > 0 ? w.units : (int64_t)num_seqs * num_heads;
  if (total_tokens == 0) b.segmented = false;
  if (b.segmented) {
    b.rstates = reinterpret_cast<float*>(ws + pl.off_rstates);
    if (kda::launch_delta_back_states(b, stream) != hipSuccess) return KDA_ERR_HIP;
    kda::DeltaBackScanArgs s;
    std::memset(&s, 0, sizeof(s));
    s.rstates = b.rstates;
    s.pairs = w.pairs;
    s.d_final = d_final_state;
    s.cu = cu_seqlens;
    s.num_seqs = num_seqs;
    s.total_tokens = total_tokens;
    s.num_heads = num_heads;
    s.seg = w.seg;
    if (kda::launch_delta_back_scan(s, stream) != hipSuccess) return KDA_ERR_HIP;
  }
  if (kda::launch_delta_back(b, stream) != hipSuccess) return KDA_ERR_HIP;
  if (total_tokens == 0) return KDA_OK;

  kda::DeltaGradArgs gr;
  std::memset(&gr, 0, sizeof(gr));
  gr.q = q;
  gr.k = k;
  gr.d_o = d_o;
  gr.u = sv.u;
  gr.dv = dv;
  gr.yh = b.yh;
  gr.s = sv.s;
  gr.ds = b.ds;
  gr.s_exps = sv.exps;
  gr.ds_exps = b.exps;
  gr.blocks = w.blocks;
  gr.cu = cu_seqlens;
  gr.num_seqs = num_seqs;
  gr.total_tokens = total_tokens;
  gr.num_heads = num_heads;
  gr.qk_heads = num_qk_heads;
  gr.bf16 = bf16;
  gr.dq = dq;
  gr.dk = dk;
  if (kda::launch_delta_grad(gr, stream) != hipSuccess) return KDA_ERR_HIP;

  if (d_log_decay) {
    kda::LinearFinishArgs f;
    std::memset(&f, 0, sizeof(f));
    f.decay.s_anchors = sv.anchors;
    f.decay.ds_anchors = b.anchors;
    f.decay.own = true;
    f.decay.r = sv.change;
    f.decay.c = b.change;
    f.decay.blocks = 8;
    f.decay.has_d_final = d_final_state != nullptr;
    f.decay.d_log_decay = d_log_decay;
    f.decay.cu = cu_seqlens;
    f.decay.num_seqs = num_seqs;
    f.decay.total_tokens = total_tokens;
    f.decay.num_heads = num_heads;
    f.decay.anchor = kAnchorTokens;
    f.decay_blocks = 1;
    f.qk_heads = num_qk_heads;
    if (kda::launch_linear_finish(f, bf16, stream) != hipSuccess) return KDA_ERR_HIP;
  }
  if (dbeta && kda::launch_delta_beta(b.beta_part, dbeta, cu_seqlens, num_seqs, total_tokens, num_heads, stream) != hipSuccess)
    return KDA_ERR_HIP;
  return KDA_OK;
}

kda_status kda_delta_decode_step(float* state, const void* q, const void* k, const void* v, const float* log_decay,
                                 const float* beta, int num_seqs, int num_heads, int num_qk_heads, int d_k, int d_v,
                                 kda_dtype dtype, void* o, hipStream_t stream) {
  if (num_seqs < 1 || num_heads < 1 || num_qk_heads < 1) return KDA_ERR_INVALID_ARG;
  if (d_k != kD || d_v != kD || !dtype_ok(dtype)) return KDA_ERR_UNSUPPORTED;
  if (!delta_sizes_ok(num_seqs, 0, num_heads, num_qk_heads)) return KDA_ERR_INVALID_ARG;
  if (!state || !q || !k || !v || !log_decay || !beta || !o) return KDA_ERR_INVALID_ARG;
  const size_t es = elem_size(dtype);
  if (!aligned(state, 16) || !aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(o, es) ||
      !aligned(log_decay, 4) || !aligned(beta, 4))
    return KDA_ERR_INVALID_ARG;
  const size_t units = (size_t)num_seqs * num_heads;
  if (units * 256 > UINT32_MAX) return KDA_ERR_INVALID_ARG;  // a workgroup each, below 2^32 threads
  const size_t qk = (size_t)num_seqs * num_qk_heads * kD * es;
  const Range ins[] = {range_of(q, qk), range_of(k, qk), range_of(v, units * kD * es),
                       range_of(log_decay, units * sizeof(float)), range_of(beta, units * sizeof(float))};
  const Range outs[] = {range_of(state, units * kStateBytes), range_of(o, units * kD * es)};
  if (any_overlap(outs, 2, ins, 5)) return KDA_ERR_INVALID_ARG;
  {
    const kda_status cs = delta_checked(k, dtype, (int64_t)num_seqs * num_qk_heads, log_decay, beta, (int64_t)units,
                                        nullptr, num_seqs, 0, stream);
    if (cs != KDA_OK) return cs;
  }
  kda::DeltaDecodeArgs a;
  std::memset(&a, 0, sizeof(a));
  a.state = state;
  a.q = q;
  a.k = k;
  a.v = v;
  a.log_decay = log_decay;
  a.beta = beta;
  a.o = o;
  a.num_seqs = num_seqs;
  a.num_heads = num_heads;
  a.qk_heads = num_qk_heads;
  a.bf16 = dtype == KDA_DTYPE_BF16;
  return kda::launch_delta_decode(a, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // extern "C"
