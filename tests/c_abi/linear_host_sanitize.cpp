// Host code of kda_linear_api.hip and kda_beam_api.hip under AddressSanitizer
// and UndefinedBehaviorSanitizer (CPU only): sizes from one token to the
// largest, every schedule, workspace queries that agree with the calls, and
// refusals.  The launch functions here only check what they are given against
// the workspace; the addresses are made up and never dereferenced.
#include <cstdint>
#include <cstdio>

#include "kda_beam.h"
#include "kda_beam_internal.h"
#include "kda_linear.h"
#include "kda_linear_internal.h"

static int failures = 0, launches = 0;
#define EXPECT(x)                                             \
  do {                                                        \
    if (!(x)) {                                               \
      std::fprintf(stderr, "line %d: %s\n", __LINE__, #x);    \
      ++failures;                                             \
    }                                                         \
  } while (0)

static char* const kWs = reinterpret_cast<char*>(0x600000000000ull);
static size_t ws_bytes = 0;
// [p, p + bytes) lies in the workspace
static void inside(const void* p, size_t bytes, int line) {
  const char* c = static_cast<const char*>(p);
  if (bytes > 0 && !(c >= kWs && c + bytes <= kWs + ws_bytes)) {
    std::fprintf(stderr, "line %d: outside the workspace\n", line);
    ++failures;
  }
}
#define inside(p, bytes) inside(p, bytes, __LINE__)
static const size_t kState = 128 * 128 * 4;

namespace kda {
bool debug_checks() { return false; }
void set_check_flags(uint32_t) {}
hipError_t run_linear_checks(const float*, int64_t, const int32_t*, int, int64_t, hipStream_t, uint32_t*) {
  return hipErrorUnknown;
}
hipError_t launch_linear_walk(const LinearWalkArgs& a, hipStream_t) {
  ++launches;
  if (a.segmented) {
    const size_t slots = (size_t)linear_slots(a.total_tokens, a.num_seqs, a.seg) * a.num_heads;
    EXPECT((size_t)a.units == slots);
    inside(a.snap, slots * kState);
  } else {
    EXPECT(a.units == (int64_t)a.num_seqs * a.num_heads);
  }
  return hipSuccess;
}
hipError_t launch_linear_states(const LinearWalkArgs& f, const LinearWalkArgs* r, hipStream_t) {
  ++launches;
  const size_t slots = (size_t)linear_slots(f.total_tokens, f.num_seqs, f.seg) * f.num_heads;
  EXPECT(f.segmented && (size_t)f.units == slots && (!r || (r->segmented && r->units == f.units && r->snap != f.snap)));
  inside(f.seg_decay, slots * 4);
  if (r) {
    inside(r->seg_decay, slots * 4);
    EXPECT(r->seg_decay >= f.seg_decay + slots);
  }
  return hipSuccess;
}
hipError_t launch_linear_scan(LinearScanArgs f, const LinearScanArgs* r, hipStream_t) {
  ++launches;
  const size_t slots = (size_t)linear_slots(f.total_tokens, f.num_seqs, f.seg) * f.num_heads;
  inside(f.snap, slots * kState);
  if (r) inside(r->snap, slots * kState);
  return hipSuccess;
}
hipError_t launch_linear_grad(const LinearGradArgs& a, hipStream_t) {
  ++launches;
  const LinearWalkArgs& w = a.dq;
  const size_t blocks = w.narrow ? 2 : 1, rows = (size_t)w.total_tokens * w.num_heads;
  EXPECT(a.dv_whole >= 0 && a.dv_whole <= w.num_heads);
  EXPECT(a.dv_whole == w.num_heads || (!w.narrow && !w.segmented && w.num_seqs == 1));
  if (a.decay_grad) {
    EXPECT(w.anchor % 64 == 0 && w.anchor > 0 && (!w.segmented || w.seg % w.anchor == 0));
    inside(w.change, blocks * rows * 4);
    inside(a.dk.change, blocks * rows * 4);
    const size_t states = w.anchors == w.snap
                              ? (size_t)linear_slots(w.total_tokens, w.num_seqs, w.anchor)
                              : (size_t)linear_boundaries(w.total_tokens, w.num_seqs, w.anchor, w.end_state);
    inside(w.anchors, states * w.num_heads * kState);
    inside(a.dk.anchors, states * w.num_heads * kState);
  }
  if (w.o_f32) {
    inside(w.o, rows * 512);
    inside(a.dk.o, rows * 512);
  }
  return hipSuccess;
}
hipError_t launch_linear_finish(LinearFinishArgs a, bool, hipStream_t) {
  ++launches;
  if (a.decay_blocks && a.decay.part) inside(a.decay.part, (size_t)linear_slots(a.decay.total_tokens, a.decay.num_seqs, a.decay.anchor) *
                                             a.decay.num_heads * 8);
  return hipSuccess;
}
hipError_t launch_linear_decay_sum(const double*, float*, int64_t, int, hipStream_t) { return hipSuccess; }
hipError_t launch_linear_decode(const LinearDecodeArgs&, hipStream_t) {
  ++launches;
  return hipSuccess;
}
hipError_t launch_beam_select(const BeamSelectArgs& a, hipStream_t) {
  ++launches;
  const size_t rows = (size_t)a.groups * a.beams, parts = rows * a.plan.slices * 256;
  inside(a.part_max, parts * 4);
  inside(a.part_at, parts * 4);
  inside(a.slice_max, rows * a.plan.slices * 4);
  inside(a.slice_sum, rows * a.plan.slices * 4);
  // the parts hold the row
  EXPECT((int64_t)a.plan.slices * 256 * a.plan.nv >= beam_vectors(a.vocab, a.plan.es) && a.plan.slices * 256 <= 2048);
  return hipSuccess;
}
hipError_t launch_beam_reorder(const BeamReorderArgs& a, int unit, hipStream_t) {
  ++launches;
  EXPECT(a.count >= 1 && a.count <= kBeamReorderMax && (unit == 16 || unit == 4 || unit == 1));
  return hipSuccess;
}
}  // namespace kda

// an address space of its own for every tensor
template <typename T = void>
static T* P(int i) {
  return reinterpret_cast<T*>(0x100000000000ull + (uint64_t)i * 0x20000000000ull);
}

int main() {
  const int seqs[] = {1, 2, 9, 1000}, heads[] = {1, 3, 8, 16, 48, 90, 96, 128, 300, 65535};
  const int64_t tokens[] = {0, 1, 63, 64, 4927, 8192, 131072, 3000000, 2147483647};
  const int segs[] = {-1, 0, 64, 192, 64 * 1021, 2147483584};
  for (int n : seqs)
    for (int h : heads)
      for (int64_t t : tokens)
        for (int seg : segs)
          for (int hq : {1, h})
            for (int dt : {0, 1}) {
              if ((double)t * h > 1e9) continue;  // (2 TiB between the tensors)
              const int32_t* cu = n > 1 ? P<int32_t>(20) : nullptr;
              ws_bytes = kda_linear_chunk_fwd_workspace_bytes(n, t, h, hq, 128, 128, (kda_dtype)dt, seg);
              if (ws_bytes < (1ull << 40)) {
                const int s = kda_linear_chunk_fwd(P(0), P(1), P(2), P<float>(3), nullptr, cu, n, t, h, hq, 0, 128, 128,
                                                   (kda_dtype)dt, seg, P(4), P<float>(5), kWs, ws_bytes, nullptr);
                EXPECT(s == KDA_OK || s == KDA_ERR_INVALID_ARG);
                if (s == KDA_OK && ws_bytes > 0)
                  EXPECT(kda_linear_chunk_fwd(P(0), P(1), P(2), P<float>(3), nullptr, cu, n, t, h, hq, 0, 128, 128,
                                              (kda_dtype)dt, seg, P(4), P<float>(5), kWs, ws_bytes - 1,
                                              nullptr) == KDA_ERR_WORKSPACE);
              }
              for (int f = 0; f < 8; ++f) {
                const int per_head = f & 1, need = f >> 1 & 1, last = f >> 2 & 1;
                ws_bytes = kda_linear_chunk_bwd_workspace_bytes(n, t, h, hq, per_head, need, last, 128, 128, (kda_dtype)dt,
                                                                seg);
                if (ws_bytes >= (1ull << 44)) continue;
                const int s = kda_linear_chunk_bwd(P(0), P(1), P(2), P<float>(3), nullptr, cu, P(6),
                                                   last ? P<float>(7) : nullptr, n, t, h, hq, per_head, 128, 128,
                                                   (kda_dtype)dt, seg, P(8), P(9), P(10), need ? P<float>(11) : nullptr,
                                                   P<float>(12), kWs, ws_bytes, nullptr);
                EXPECT(s == KDA_OK || s == KDA_ERR_INVALID_ARG);
              }
            }
  EXPECT(launches > 10000);
  for (int n : {1, 7, 4096, 100000, 16777215, 16777216, 2147483647})
    for (int h : {1, 96, 65535, 65536, 2147483647}) {
      const int s = kda_linear_decode_step(P<float>(0), P(1), P(2), P(3), P<float>(4), n, h, 1, 0, 128, 128,
                                           KDA_DTYPE_BF16, P(5), nullptr);
      EXPECT(s == ((double)n * h < 16777216.0 && h <= 65535 ? KDA_OK : KDA_ERR_INVALID_ARG) ||
             (double)n * h * 65536.0 > 2e12);  // (more than lies between the tensors)
    }
  for (int b : {1, 64, 1 << 20, 2147483647})
    for (int k : {1, 4, 16, 17, 2147483647})
      for (int v : {1, 7, 8, 17, 2047, 128003, 1 << 24, 2147483647})
        for (int dt : {0, 1, 2, -5}) {
          ws_bytes = kda_beam_select_workspace_bytes(b, k, v, (kda_dtype)dt);
          const int s = kda_beam_select(P(0), P<float>(1), nullptr, b, k, v, 0, (kda_dtype)dt, P<float>(2), P<int32_t>(3),
                                        P<int32_t>(4), nullptr, kWs, ws_bytes, nullptr);
          EXPECT((s == KDA_OK) == (ws_bytes > 0) || (double)b * k * v > 2e11);
        }
  void* st[8] = {P(0), P(1), P(2), P(3), P(4), P(5), P(6), P(7)};
  for (int64_t r : {(int64_t)0, (int64_t)1, (int64_t)4, (int64_t)6291456, (int64_t)1 << 31, (int64_t)1 << 40, INT64_MAX, (int64_t)-1})
    for (int b : {1, 64, 2147483647})
      for (int k : {1, 5, 16}) {
        const int64_t rows[8] = {r, r, 64, 12, 3, 0, 16, 1};
        const int s = kda_beam_reorder(st, rows, 8, P<int32_t>(9), b, k, nullptr);
        EXPECT(s == KDA_OK || s == KDA_ERR_INVALID_ARG);
      }
  std::printf("%d launches\n", launches);
  if (failures == 0) std::printf("linear host sanitizer checks passed\n");
  return failures != 0;
}
