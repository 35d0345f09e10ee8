// kda_delta_internal.h — launch descriptors of the gated delta rule's kernels
// (one decay per head) for the C ABI layer (kda_delta_api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_linear_internal.h"

namespace kda {

// Chunks.  Sequence n's chunk j of C tokens (64 in bf16, 32 in fp32) has the
// slot cu[n] / C + n + j: ceil(L / C) <= floor(cu[n+1] / C) - floor(cu[n] / C) + 1,
// so no two meet.
constexpr int delta_chunk(bool bf16) { return bf16 ? 64 : 32; }
constexpr int64_t delta_chunk_slots(int64_t total_tokens, int num_seqs, int chunk) {
  return total_tokens / chunk + num_seqs;
}

// What the prep kernel leaves of a chunk of one head, a block of two parts:
//   the matrix -X of delta_prep_kernel, strictly lower triangular, as 16 x 16 tiles
//   on and below the diagonal (tile (a, b) is number a (a + 1) / 2 + b), first the
//   leading terms of fp16, then what they leave (kda_delta_util.h);
//   float [6][C] and one more: the prefix sums of the log decays (in powers of two;
//   high and low part), e^{G_i}, e^{G_C - G_j}, beta, beta e^{G_i}, and e^{G_C}.
constexpr int delta_tiles(int chunk) { return (chunk / 16) * (chunk / 16 + 1) / 2; }
constexpr int kDeltaTileBytes = 512;
constexpr int delta_matrix_bytes(int chunk) { return 2 * delta_tiles(chunk) * kDeltaTileBytes; }
constexpr int delta_factor_bytes(int chunk) { return (6 * chunk * 4 + 4 + 1023) / 1024 * 1024; }
constexpr int delta_block_bytes(int chunk) { return delta_matrix_bytes(chunk) + delta_factor_bytes(chunk); }

struct DeltaPrepArgs {
  const void* k;           // [T, qk_heads, 128]
  const float* log_decay;  // [T, H]
  const float* beta;       // [T, H]
  const int32_t* cu;       // [N+1] or null (one sequence)
  int num_seqs;
  int64_t total_tokens;
  int num_heads, qk_heads;
  bool bf16;
  char* blocks;            // [chunk slots][H] blocks (written)
  int64_t unit0;           // first (chunk slot, head) of the launch (set by it)
};

// What the forward walk leaves for the backward pass.
struct DeltaSaveArgs {
  const void* d_o;         // [T, H, 128]
  void* s;                 // [chunk slots][H] images of the states that enter the chunks: fp32, or
  void* u;                 // [T, H, 128]                            (bf16) fp16, scaled by columns:
  int* exps;               // (bf16) [chunk slots][H][128]: times 2^exps
  float* e;                // [chunk slots][H][8 column tiles][C / 16][64][4]: u / beta
  float* change;           // [8 column tiles][H][T] o . d_o
  float* anchors;          // [linear_boundaries][H][128,128] states at the boundaries of stretches, or null
  int anchor;              // tokens of a stretch (a multiple of 64)
  bool end_state;          // a sequence's end is a boundary too
};

struct DeltaWalkArgs {
  const void* q;           // [T, qk_heads, 128]
  const void* k;
  const void* v;           // [T, H, 128]
  const float* log_decay;
  const float* beta;       // (the prep kernel's)
  const char* blocks;      // the prep kernel's
  const int32_t* cu;
  int num_seqs;
  int64_t total_tokens;
  int num_heads, qk_heads;
  bool bf16;
  int seg;                 // tokens per segment
  bool segmented;          // work items are (segment, head), else (sequence, head)
  int64_t unit0, units;    // work items (set by the launch)
  const float* init;       // [N,H,128,128] or null (zero); read where a sequence is walked whole, and by the pairs
                           // pass (led)
  float* fin;              // [N,H,128,128] or null; may be init: no launch that walks a sequence's first segment apart
                           // from its last one may be given both
  float* pairs;            // [segment slots][H][2][128,128]: pairs pass (written), else the states that enter segments
  bool all_pairs;          // pairs pass: of all segments, as the backward pass reads
  bool led;                // the pairs pass walks the first segments' outputs
  bool both;               // pairs pass: a workgroup walks a segment's contribution and its transition
  void* o;                 // [T, H, 128]
  DeltaSaveArgs save;
};

struct DeltaScanArgs {
  float* pairs;            // contributions and transitions in, states that enter segments (in contributions' places) out
  bool led;                // the first segments have been walked; else what enters them is written too
  const float* init;
  const float* log_decay;
  const int32_t* cu;
  int num_seqs;
  int64_t total_tokens;
  int num_heads;
  int seg;
  int64_t unit0;           // first (sequence, head) of the launch (set by it)
};

// The walk back.
struct DeltaBackArgs {
  const void* q;
  const void* k;
  const void* v;
  const void* d_o;         // [T, H, 128]
  const char* blocks;      // the prep kernel's
  const float* e;          // DeltaSaveArgs::e
  const int32_t* cu;
  int num_seqs;
  int64_t total_tokens;
  int num_heads, qk_heads;
  bool bf16;
  int seg;
  bool segmented;
  int64_t unit0, units;
  const float* d_final;    // [N,H,128,128] or null (zero)
  float* d_initial;        // or null
  float* rstates;          // [segment slots][H][128,128]: states pass (written), else what reaches the segments' ends
  void* dv;
  void* ds;                // [chunk slots][H] images of what reaches the chunks' ends (written), as DeltaSaveArgs::s
  void* yh;                // (bf16) [T, H, 128] dv / beta as DeltaSaveArgs::u (written)
  int* exps;               // (bf16) as DeltaSaveArgs::exps (written)
  float* change;           // [8][H][T] v . dv (written)
  float* beta_part;        // [8][H][T] (written)
  float* anchors;          // as DeltaSaveArgs::anchors, of dS (written)
  int anchor;
  bool end_state;
};

struct DeltaBackScanArgs {
  float* rstates;          // contributions in, what reaches the segments' ends out
  const float* pairs;      // DeltaWalkArgs::pairs: the transitions
  const float* d_final;
  const int32_t* cu;
  int num_seqs;
  int64_t total_tokens;
  int num_heads;
  int seg;
  int64_t unit0;
};

struct DeltaGradArgs {
  const void* q;
  const void* k;
  const void* d_o;
  const void* u;           // the walks' results
  const void* dv;
  const void* yh;          // (bf16) dv / beta
  const void* s;
  const void* ds;
  const int* s_exps;
  const int* ds_exps;
  const char* blocks;      // the prep kernel's
  const int32_t* cu;
  int num_seqs;
  int64_t total_tokens;
  int num_heads, qk_heads;
  bool bf16;
  int64_t unit0;           // first (chunk slot, query and key head) of the launch (set by it)
  void* dq;
  void* dk;
};

struct DeltaDecodeArgs {
  float* state;            // [N,H,128,128], in place
  const void* q;           // [N, qk_heads, 128]
  const void* k;
  const void* v;           // [N, H, 128]
  const float* log_decay;  // [N, H]
  const float* beta;       // [N, H]
  void* o;
  int num_seqs;
  int num_heads;
  int qk_heads;
  bool bf16;
};

hipError_t launch_delta_prep(DeltaPrepArgs a, hipStream_t stream);
hipError_t launch_delta_walk(DeltaWalkArgs a, hipStream_t stream);
hipError_t launch_delta_save(DeltaWalkArgs a, hipStream_t stream);
// Segments: their own contributions and transitions, then the states that enter them.
hipError_t launch_delta_pairs(DeltaWalkArgs a, hipStream_t stream);
hipError_t launch_delta_scan(DeltaScanArgs a, hipStream_t stream);
hipError_t launch_delta_back(DeltaBackArgs a, hipStream_t stream);
hipError_t launch_delta_back_states(DeltaBackArgs a, hipStream_t stream);
hipError_t launch_delta_back_scan(DeltaBackScanArgs a, hipStream_t stream);
hipError_t launch_delta_grad(DeltaGradArgs a, hipStream_t stream);
hipError_t launch_delta_beta(const float* part, float* dbeta, const int32_t* cu, int num_seqs, int64_t total_tokens,
                             int num_heads, hipStream_t stream);
hipError_t launch_delta_decode(const DeltaDecodeArgs& a, hipStream_t stream);
// Checks the documented input ranges on `stream`, waits, and returns the
// KDA_CHECK_* bits that failed.
hipError_t run_delta_checks(const void* k, bool bf16, int64_t k_rows, const float* log_decay, const float* beta,
                            int64_t count, const int32_t* cu, int num_seqs, int64_t total_tokens, hipStream_t stream,
                            uint32_t* flags);

}  // namespace kda
