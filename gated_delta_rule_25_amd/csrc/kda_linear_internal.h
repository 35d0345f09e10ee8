// kda_linear_internal.h — launch descriptors of the per-head-decay linear
// attention kernels (kda_linear.hip) for the C ABI layer (kda_linear_api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

// Segments.  Every sequence is cut into segments of `seg` tokens (a multiple
// of 64) counted from its own start; segment j of sequence n has the slot
//   cu[n] / seg + 2 n + j.
// ceil(L_n / seg) <= floor(cu[n+1] / seg) - floor(cu[n] / seg) + 1, so the
// slots of two sequences never meet and each sequence has one spare slot
// behind its last segment (the state it ends with); a slot's sequence is
// found by bisection, with no table and no prefix sum.
constexpr int64_t linear_slots(int64_t total_tokens, int num_seqs, int64_t seg) {
  return total_tokens / seg + 2 * (int64_t)num_seqs;
}

// Boundaries between a sequence's stretches of `anchor` tokens, and its end if
// `ends`: boundary j = 1 .. of sequence n has the index
//   cu[n] / anchor + j - 1 (+ n with the ends),
// again without two that meet, as a sequence has at most (L - 1) / anchor of
// the former: nothing for sequences of one stretch.
constexpr int64_t linear_boundaries(int64_t total_tokens, int num_seqs, int64_t anchor, bool ends) {
  return total_tokens / anchor + (ends ? num_seqs : 0);
}

// One walk of a state over the chunks of a sequence or of a segment.  The
// recurrence and its three gradients are the same walk with the tensors in
// other roles:
//   forward   queries q,  keys k,  values v,  forwards in time,  state S
//   dq        queries do, keys v,  values k,  forwards,          state S^T
//   dv        queries k,  keys q,  values do, backwards,         state dS
//   dk        queries v,  keys do, values q,  backwards,         state dS^T
struct LinearWalkArgs {
  const void* q;  // [T, q_heads, 128]: the query role; state head h reads head h / (H / q_heads)
  const void* k;
  const void* v;
  const void* x;  // the tensor whose product with the state's part of the output enters d_log_decay
  int q_heads, k_heads, v_heads, x_heads;
  const float* log_decay;  // [T, H], or [H] (decay_per_head)
  bool decay_per_head;
  const int32_t* cu;       // [N+1] or null (one sequence)
  int num_seqs;
  int64_t total_tokens;
  int num_heads;
  bool bf16;
  int seg;                 // tokens per segment
  bool segmented;          // work items are (segment, head), else (sequence, head)
  int64_t units;           // work items
  int64_t unit0;           // first item of the launch (set by it)
  bool narrow;             // 64 value columns per workgroup instead of 128
  const float* init;       // [N,H,128,128] or null (zero): enters at the sequence's first (reverse: last) token
  float* fin;              // [N,H,128,128] or null: the state behind the last (reverse: before the first) token
  float* snap;             // [slots][H][128,128] segmented: incoming states; states pass: contributions (written)
  float* seg_decay;        // [slots][H] states pass: product of the segment's decays (written)
  void* o;                 // [T, H, 128] in the I/O dtype, or fp32 (o_f32)
  bool o_f32;
  // gradient of the decays
  int anchor;              // tokens between the boundaries at which it is taken from the states (a multiple of 64)
  bool end_state;          // a sequence's end is such a boundary too (dS there is given)
  float* anchors;          // [linear_boundaries][H][128,128] S (dq walk) or dS (dk walk) at the boundaries (written); or
                           // `snap` itself when segments are of that length: the scan has left there what enters
                           // them, and the dq walk adds S behind the last token
  float* change;           // [column blocks][H][T]: r_t (dq walk) or c_t (dk walk) by the block's columns (written)
};

// The three walks of the backward pass.
struct LinearGradArgs {
  LinearWalkArgs dq, dk, dv;
  int64_t item0;           // first sequence (or segment) of the launch (set by it)
  bool decay_grad;
  int dv_whole;            // heads whose dv walk is whole; half heads for the rest (whole heads elsewhere only)
};

// Blocks of a work item in the launch of the three walks, in multiples of 8
// (XCDs): dq and dk, dv by whole heads (or the column blocks all take), dv by
// half heads.
struct GradGrid {
  int heavy, whole, blocks;
  __host__ __device__ GradGrid(int heads, int column_blocks, int dv_whole)
      : heavy(2 * column_blocks * round8(heads)), whole(column_blocks * round8(dv_whole)),
        blocks(heavy + whole + 2 * round8(heads - dv_whole)) {}
  static __host__ __device__ int round8(int x) { return (x + 7) / 8 * 8; }
};

struct LinearDecayGradArgs {
  const float* s_anchors;  // as LinearWalkArgs::anchors
  const float* ds_anchors;
  bool own;                // by boundaries (not by segments)
  const float* r;          // [blocks][H][T]
  const float* c;
  int blocks;
  bool has_d_final;        // dS behind a sequence's last token is not zero
  float* d_log_decay;      // [T, H] or null
  double* part;            // [slots by `anchor`][H] sums over the stretch (a constant decay), or null
  const int32_t* cu;
  int num_seqs;
  int64_t total_tokens;
  int num_heads;
  int anchor;
};

struct LinearFinishArgs {
  LinearDecayGradArgs decay;  // (its sizes and cu also hold for the sums over shared heads)
  int64_t decay_blocks;       // nonzero: the decays' gradient is wanted
  const float* share;         // [2][T, H, 128] fp32 gradients of the value heads' dq and dk, or null
  void* dq;                   // [T, qk_heads, 128] in the I/O dtype
  void* dk;
  int qk_heads;
  int64_t share_blocks;       // set by the launch
};

struct LinearScanArgs {
  int64_t unit0;           // first (sequence, head) of the launch (set by it)
  float* snap;             // contributions in, incoming states out
  const float* seg_decay;
  const float* init;       // as above
  const int32_t* cu;
  int num_seqs;
  int64_t total_tokens;
  int num_heads;
  int seg;
};

struct LinearDecodeArgs {
  float* state;            // [N,H,128,128], in place
  const void* q;           // [N, qk_heads, 128]
  const void* k;
  const void* v;           // [N, H, 128]
  const float* log_decay;  // [N, H] or [H]
  bool decay_per_head;
  void* o;
  int num_seqs;
  int num_heads;
  int qk_heads;
  bool bf16;
};

hipError_t launch_linear_walk(const LinearWalkArgs& a, hipStream_t stream);
// Segments: their own contributions to the state and, by the scan, the states
// that enter them; forwards and, if given, backwards.
hipError_t launch_linear_states(const LinearWalkArgs& f, const LinearWalkArgs* r, hipStream_t stream);
hipError_t launch_linear_grad(const LinearGradArgs& a, hipStream_t stream);
hipError_t launch_linear_finish(LinearFinishArgs a, bool bf16, hipStream_t stream);
hipError_t launch_linear_scan(LinearScanArgs f, const LinearScanArgs* r, hipStream_t stream);
hipError_t launch_linear_decay_sum(const double* part, float* dst, int64_t units, int num_heads, hipStream_t stream);
hipError_t launch_linear_decode(const LinearDecodeArgs& a, hipStream_t stream);
// Checks the documented input ranges (log_decay <= 0 and not NaN; cu_seqlens)
// on `stream`, waits, and returns the KDA_CHECK_* bits that failed.
hipError_t run_linear_checks(const float* log_decay, int64_t count, const int32_t* cu, int num_seqs,
                             int64_t total_tokens, hipStream_t stream, uint32_t* flags);

}  // namespace kda
