// kda_beam.hip — beam search over recurrent states: selection of the best
// continuations, and the states' reordering.
//
// Selection.  Candidate (k, t) of a group of K beams over V tokens has the
// score c = s_k + x_kt - log sum_t' e^{x_kt'}; a finished beam has only its
// end token, at s_k.  The K largest c are wanted, ties to the lowest k V + t.
//
// Within a row c grows with x, so the row's K best are found on the logits
// themselves, exactly, whatever the rounding of the sum.  They need no second
// pass over the row and no sorting: cut a row in parts and note each part's
// largest element (ties to the lowest index).  If an element is among the K
// best, its part's largest is at least as good; were that part not among the
// K with the best largest elements, K elements would precede ours.  So the K
// best parts hold the K best elements.
//   beam_scan_kernel   reads every logit once: per thread the largest element
//                      of its part and, rescaled to the workgroup's maximum,
//                      the sum of exponentials (exponentials of differences
//                      to the thread's own maximum, fp32; the workgroup's
//                      threads are combined in fp64, and its sum kept in fp32:
//                      half a step, 6e-8, of what the score takes the log of).
//                      Bound by HBM (64 groups x 8 beams x 128003 bf16 logits:
//                      28 us, 4.7 TB/s).
//   beam_pick_kernel   one workgroup per group: the K best parts of each row,
//                      their elements read again (K x nv vectors), the row's
//                      K best; then the K best of the K x K candidates,
//                      compared as fp64 scores.  Bound by latency: a chain of
//                      dependent reads and counts (the same case: 13 us; one
//                      group of 4 beams x 32000: 7 us after a scan of 4.5).
// Nothing depends on the order in which workgroups run.
//
// Reordering.  Row n of a group's states becomes the row of its parent.  A
// thread owns the same few bytes of all the group's rows, reads what moves and
// then writes it, so the rows change in place with no copy of the states and
// no barrier, and rows that stay are not touched.  Bound by HBM (64 groups of 4
// beams, 96 heads of states and histories: 370 us, 5.7 TB/s of what moves).
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "kda_device.h"
#include "kda_beam_internal.h"

namespace kda {
namespace {

// Order of candidates in a row as one number: larger is better, a larger
// value before a smaller one, the lower index first among equals.
__device__ __forceinline__ uint64_t beam_key(float x, uint32_t at) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.f);  // -0 counts as 0
  const uint32_t o = (u & 0x80000000u) ? ~u : u | 0x80000000u;
  return (uint64_t)o << 32 | (uint32_t)~at;
}
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __builtin_bit_cast(float, (o & 0x80000000u) ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ uint32_t key_at(uint64_t key) { return ~(uint32_t)key; }

// Largest of a wave's numbers, in every lane (lane moves within rows of 16,
// then between them: no LDS).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t dpp_max(uint64_t x) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)x, CTRL, ROWS, 0xf, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(x >> 32), CTRL, ROWS, 0xf, false);
  const uint64_t o = (uint64_t)hi << 32 | lo;
  return o > x ? o : x;
}
__device__ __forceinline__ uint64_t wave_max(uint64_t x) {
  x = dpp_max<0x111, 0xf>(x);  // from the lane 1, 2, 4, 8 below
  x = dpp_max<0x112, 0xf>(x);
  x = dpp_max<0x114, 0xf>(x);
  x = dpp_max<0x118, 0xf>(x);
  x = dpp_max<0x142, 0xa>(x);  // from the last lane of the row below
  x = dpp_max<0x143, 0xc>(x);  // from the last lane of the lower half
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, 63);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(x >> 32), 63);
  return (uint64_t)hi << 32 | lo;
}
// NaN is a masked logit like -inf (the maximum of NaN and a number is the
// number); +inf counts as the largest finite number.
__device__ __forceinline__ float beam_logit(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX); }
template <typename E>
__device__ __forceinline__ float load_logit(const E* p) { return beam_logit(to_f32(*p)); }

// Where the vectors of a row start and how many there are.
struct BeamRow {
  int head;   // elements before the first vector
  int nvec;
};
template <typename E>
__device__ __forceinline__ BeamRow beam_row(const E* row, int vocab) {
  constexpr int U = 16 / (int)sizeof(E);
  const int off = (int)(reinterpret_cast<uintptr_t>(row) & 15) / (int)sizeof(E);
  BeamRow r;
  r.head = min((U - off) % U, vocab);
  r.nvec = (vocab - r.head) / U;
  return r;
}
// The element outside the vectors that thread t of the first slice takes, or -1.
template <typename E>
__device__ __forceinline__ int beam_extra(const BeamRow& r, int vocab, int t) {
  constexpr int U = 16 / (int)sizeof(E);
  if (t < r.head) return t;
  const int at = r.head + r.nvec * U + (t - U);
  return t >= U && t < 2 * U && at < vocab ? at : -1;
}

template <typename E>
__device__ __forceinline__ void load_vector(float (&x)[16 / sizeof(E)], const E* p) {
  const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  if constexpr (sizeof(E) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = beam_logit(__builtin_bit_cast(float, v[i] << 16));
      x[2 * i + 1] = beam_logit(__builtin_bit_cast(float, v[i] & 0xffff0000u));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = beam_logit(__builtin_bit_cast(float, (uint32_t)v[i]));
  }
}

// A row contributes logits unless its beam is finished or has no score.
__device__ __forceinline__ bool row_is_read(const BeamSelectArgs& a, int64_t row) {
  return a.scores[row] > -INFINITY && !(a.finished && a.finished[row]);
}

// e^x for x <= 0.  The product's rounding moves a term by |x| 2^-24 of it, and
// terms of large |x| are small: the sum's error stays near its own rounding.
__device__ __forceinline__ float beam_exp(float x) { return exp2_fast(x * 1.44269504f); }

// One workgroup per (row, slice).
template <typename E>
__global__ __launch_bounds__(kBeamThreads) void beam_scan_kernel(const BeamSelectArgs a) {
  constexpr int U = 16 / (int)sizeof(E);
  const int64_t row = blockIdx.x / a.plan.slices;
  const int slice = (int)(blockIdx.x % a.plan.slices);
  if (!row_is_read(a, row)) return;
  const int t = threadIdx.x, nv = a.plan.nv;
  const E* x = static_cast<const E*>(a.logits) + row * a.vocab;
  const BeamRow r = beam_row(x, a.vocab);
  float best = -INFINITY, sum = 0.f;
  int at = INT32_MAX;
  auto take = [&](float v, int i) {
    if (v > best || (v == best && i < at)) {
      best = v;
      at = i;
    }
  };
  // the exponentials are relative to the running maximum; a vector's are
  // summed once its own maximum is known
  float top = -INFINITY;
  auto fold = [&](float m) {
    if (m > top) {
      sum *= top > -INFINITY ? beam_exp(top - m) : 0.f;
      top = m;
    }
  };
  const int first = slice * kBeamThreads * nv + t;
  for (int i = 0; i < nv; ++i) {
    const int vec = first + i * kBeamThreads;
    if (vec >= r.nvec) break;
    const int e0 = r.head + vec * U;
    float v[U];
    load_vector<E>(v, x + e0);
    float m = v[0];
#pragma unroll
    for (int j = 1; j < U; ++j) m = fmaxf(m, v[j]);
    if (m > best) {  // the lowest index with the vector's maximum (vectors come in order)
      int k = U - 1;
#pragma unroll
      for (int j = U - 2; j >= 0; --j) k = v[j] == m ? j : k;
      best = m;
      at = e0 + k;
    }
    if (m > -INFINITY) {
      fold(m);
#pragma unroll
      for (int j = 0; j < U; ++j) sum += beam_exp(v[j] - top);
    } else if (at == INT32_MAX) {
      at = e0;
    }
  }
  if (slice == 0) {
    const int i = beam_extra<E>(r, a.vocab, t);
    if (i >= 0) {
      const float v = load_logit(x + i);
      take(v, i);
      if (v > -INFINITY) {
        fold(v);
        sum += beam_exp(v - top);
      }
    }
  }
  const int64_t parts = (int64_t)a.plan.slices * kBeamThreads;
  a.part_max[row * parts + slice * kBeamThreads + t] = best;
  a.part_at[row * parts + slice * kBeamThreads + t] = at;  // INT32_MAX: the part is empty
  // over the workgroup
  float m = top;
#pragma unroll
  for (int k = 32; k >= 1; k >>= 1) m = fmaxf(m, __shfl_xor(m, k));
  __shared__ float sm[4];
  __shared__ double ss[4];
  if ((t & 63) == 0) sm[t >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  double d = top > -INFINITY ? (double)sum * (double)beam_exp(top - m) : 0.0;
#pragma unroll
  for (int k = 32; k >= 1; k >>= 1) d += __shfl_xor(d, k);
  if ((t & 63) == 0) ss[t >> 6] = d;
  __syncthreads();
  if (t == 0) {
    a.slice_max[row * a.plan.slices + slice] = m;
    a.slice_sum[row * a.plan.slices + slice] = (float)(ss[0] + ss[1] + ss[2] + ss[3]);
  }
}

// Largest of a wave's numbers (not NaN), in every lane.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_fmax(float x) {
  const int o = __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, -INFINITY), __builtin_bit_cast(int, x), CTRL, ROWS,
                                            0xf, false);
  return fmaxf(x, __builtin_bit_cast(float, o));
}
__device__ __forceinline__ float wave_fmax(float x) {
  x = dpp_fmax<0x111, 0xf>(x);
  x = dpp_fmax<0x112, 0xf>(x);
  x = dpp_fmax<0x114, 0xf>(x);
  x = dpp_fmax<0x118, 0xf>(x);
  x = dpp_fmax<0x142, 0xa>(x);
  x = dpp_fmax<0x143, 0xc>(x);
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}

// One workgroup per group, wave k for beam k.
//   1. The C = min(K, V) best parts.  A lane holds up to 32; the C-th largest
//      of the lanes' own maxima is a bound that at least C parts reach, and
//      seldom many more: those move to one a lane and are sorted by counting.
//      (More than 64, which takes ties, go through C rounds of the wave's
//      maximum over all parts.)
//   2. Their largest elements are C elements of the row, so none below the
//      last of them is wanted.
//   3. The C parts are read again; where one holds another element that is
//      wanted (seldom), the list of the C best is formed anew with it.
// Then the waves place the K x C candidates by counting as well.
template <typename E>
__global__ __launch_bounds__(64 * kBeamMax) void beam_pick_kernel(const BeamSelectArgs a) {
  constexpr int U = 16 / (int)sizeof(E);
  constexpr int PL = kBeamMaxParts / 64;  // parts per lane
  const int K = a.beams, V = a.vocab;
  const int g = blockIdx.x, lane = threadIdx.x & 63;
  const int k = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = (int64_t)g * K + k;
  __shared__ uint64_t few_key[kBeamMax][64];
  __shared__ int few_id[kBeamMax][64];
  __shared__ double cand_score[kBeamMax * kBeamMax];
  __shared__ uint32_t cand_token[kBeamMax * kBeamMax];
  __shared__ uint8_t done[kBeamMax];
  const float score = a.scores[row];
  const bool fin = a.finished && a.finished[row];
  const int C = min(K, V);  // candidates of a row
  const int parts = a.plan.slices * kBeamThreads;
  {
    double mine = -INFINITY;  // lane i < C: the row's i-th best
    uint32_t token = 0;
    if (!row_is_read(a, row)) {
      // the end token if the beam is finished (a beam without a score ties at
      // -inf with everything), then the lowest tokens at -inf
      const bool ends = fin && score > -INFINITY && a.end_token >= 0 && a.end_token < V;
      int t = lane;
      if (ends) t = lane == 0 ? a.end_token : (lane - 1 < a.end_token ? lane - 1 : lane);
      if (ends && lane == 0) mine = (double)score;
      token = (uint32_t)t;
    } else {
      // all loads before the first use: they are in flight together
      const float* pm = a.part_max + row * parts;
      const int32_t* pa = a.part_at + row * parts;
      float top[PL];
      int where[PL];
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        const int p = min(64 * i + lane, parts - 1);
        top[i] = pm[p];
        where[i] = pa[p];
      }
      const int sl = min(lane, a.plan.slices - 1);
      const float sm = lane < a.plan.slices ? a.slice_max[row * a.plan.slices + sl] : -INFINITY;
      const float ssum = lane < a.plan.slices ? a.slice_sum[row * a.plan.slices + sl] : 0.f;
      // log of the row's sum of exponentials, relative to its largest logit
      // (which may be so large that the sum of the two is no more than itself)
      const float m = wave_fmax(sm);
      double sum = sm > -INFINITY ? (double)ssum * exp((double)sm - (double)m) : 0.0;
#pragma unroll
      for (int i = 32; i >= 1; i >>= 1) sum += __shfl_xor(sum, i);
      const double log_sum = log(sum);
      // a bound that C parts reach
      float most = -INFINITY;
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        if (64 * i + lane >= parts) where[i] = INT32_MAX;
        if (where[i] != INT32_MAX) most = fmaxf(most, top[i]);
      }
      float bound = -INFINITY;
      for (int c = 0; c < C;) {
        bound = wave_fmax(most);
        if (!(bound > -INFINITY)) break;
        c += __popcll(__ballot(most == bound));
        if (most == bound) most = -INFINITY;
      }
      int few = 0;
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        const bool in = where[i] != INT32_MAX && top[i] >= bound;
        const uint64_t mask = __ballot(in);
        if (mask != 0) {
          const int to = few + __popcll(mask & ((1ull << lane) - 1));
          if (in && to < 64) {
            few_key[k][to] = beam_key(top[i], (uint32_t)where[i]);
            few_id[k][to] = 64 * i + lane;
          }
          few += __popcll(mask);
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
      uint64_t list = 0;  // lane i < C: the i-th best element
      int part = -1;      // and the part it is from
      uint64_t least = 0;
      if (few <= 64) {
        // sorted by counting: a part's place is the number of better ones
        // (their keys differ, as the indices do)
        const uint64_t cur = lane < few ? few_key[k][lane] : 0;
        const int id = lane < few ? few_id[k][lane] : -1;
        int place = 0;
        for (int j = 0; j < few; ++j) place += few_key[k][j] > cur;
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        if (lane < few) {
          few_key[k][place] = cur;
          few_id[k][place] = id;
        }
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        if (lane < min(few, C)) {
          list = few_key[k][lane];
          part = few_id[k][lane];
        }
        if (few >= C) least = __shfl((unsigned long long)list, C - 1);
      } else {
        uint64_t before = ~0ull;
        for (int c = 0; c < C; ++c) {
          uint64_t cur = 0;
          int id = -1;
#pragma unroll
          for (int i = 0; i < PL; ++i) {
            const uint64_t key = where[i] != INT32_MAX ? beam_key(top[i], (uint32_t)where[i]) : 0;
            if (key < before && key > cur) {
              cur = key;
              id = 64 * i + lane;
            }
          }
          const uint64_t w = wave_max(cur);
          const int src = __ffsll((unsigned long long)__ballot(cur == w)) - 1;
          const int got = __builtin_amdgcn_readlane(id, src);
          if (lane == c) {
            list = w;
            part = got;
          }
          before = least = w;
        }
      }
      // their elements: vector j of part i is lane i nv + j (64 a turn)
      const E* x = static_cast<const E*>(a.logits) + row * V;
      const BeamRow r = beam_row(x, V);
      const int nv = a.plan.nv;
      for (int v0 = 0; v0 < C * nv; v0 += 64) {
        const int vid = v0 + lane;
        const int i = min(vid / nv, C - 1);
        const int owner = __shfl(part, i);
        uint64_t key[U + 1];
#pragma unroll
        for (int j = 0; j <= U; ++j) key[j] = 0;
        if (vid < C * nv && owner >= 0) {
          const int slice = owner / kBeamThreads, t = owner % kBeamThreads;
          const int vec = slice * kBeamThreads * nv + (vid % nv) * kBeamThreads + t;
          if (vec < r.nvec) {
            const int e0 = r.head + vec * U;
            float y[U];
            load_vector<E>(y, x + e0);
#pragma unroll
            for (int j = 0; j < U; ++j) key[j] = beam_key(y[j], (uint32_t)(e0 + j));
          }
          if (vid % nv == 0 && slice == 0) {
            const int e = beam_extra<E>(r, V, t);
            if (e >= 0) key[U] = beam_key(load_logit(x + e), (uint32_t)e);
          }
        }
        // wanted: better than the last of the list, and not in it already
#pragma unroll
        for (int j = 0; j <= U; ++j)
          if (key[j] <= least) key[j] = 0;
        for (int c = 0; c < C; ++c) {
          const uint64_t have = __shfl((unsigned long long)list, c);
#pragma unroll
          for (int j = 0; j <= U; ++j)
            if (key[j] == have) key[j] = 0;
        }
        bool wanted = false;
#pragma unroll
        for (int j = 0; j <= U; ++j) wanted |= key[j] != 0;
        if (!__any(wanted)) continue;
        uint64_t keep = 0;
        uint64_t before = ~0ull;
        for (int c = 0; c < C; ++c) {
          uint64_t b = list < before ? list : 0;
#pragma unroll
          for (int j = 0; j <= U; ++j)
            if (key[j] < before && key[j] > b) b = key[j];
          b = wave_max(b);
          if (lane == c) keep = b;
          before = b;
          if (b == 0) break;
        }
        list = keep;
        least = __shfl((unsigned long long)list, C - 1);
      }
      const float v = key_value(list);
      if (v > -INFINITY) mine = (double)score + (((double)v - (double)m) - log_sum);
      token = key_at(list);
    }
    if (!(mine == mine)) mine = -INFINITY;  // a score that is not a number
    if (lane < C) {
      cand_score[k * C + lane] = mine;
      cand_token[k * C + lane] = token;
    }
    if (lane == 0) done[k] = fin;
  }
  __syncthreads();
  // the K best of the K x C candidates (C = K, or V < K candidates a row): a
  // candidate's place is the number of better ones, the largest score first.
  // Among equal scores the lower beam comes first, and within a beam its list's
  // order, which is that of the logits: logits that differ may well have the
  // same score.  Wave k places its own row's, each by 8 lanes (4 with more than
  // 8 beams).
  const int sh = K > 8 ? 2 : 3, lanes = 1 << sh;
  const int c = lane >> sh;
  const int me = k * C + min(c, C - 1);
  const double ms = cand_score[me];
  int place = 0;
  for (int j = lane & (lanes - 1); j < K * C; j += lanes) {
    const double s = cand_score[j];
    place += s > ms || (s == ms && j < me);
  }
  for (int m = lanes >> 1; m >= 1; m >>= 1) place += __shfl_xor(place, m);
  if (c < C && (lane & (lanes - 1)) == 0 && place < K) {
    // (the clamp keeps a wrong candidate in range)
    const int token = (int)min(cand_token[me], (uint32_t)(V - 1));
    const int64_t o = (int64_t)g * K + place;
    a.out_scores[o] = (float)ms;
    a.out_tokens[o] = token;
    a.out_parents[o] = k;
    if (a.out_finished) a.out_finished[o] = done[k] || token == a.end_token;
  }
}

// ---------------------------------------------------------------------------
// Reordering: a thread owns one unit of every row of its group.
// ---------------------------------------------------------------------------
template <typename T, int KMAX>
__global__ __launch_bounds__(256) void beam_reorder_kernel(const BeamReorderArgs a) {
  const int64_t blk = blockIdx.x % a.blocks;
  const int64_t g = a.group0 + blockIdx.x / a.blocks;
  const int K = a.beams;
  int s = 0;
  while (s + 1 < a.count && blk >= a.block0[s + 1]) ++s;
  int from[KMAX];
#pragma unroll
  for (int i = 0; i < KMAX; ++i) {
    from[i] = i;
    if (i < K) {
      const int p = a.parents[g * K + i];
      if (p >= 0 && p < K) from[i] = p;  // a parent out of range leaves the row as it is
    }
  }
  const int64_t units = a.row_units[s];
  const int64_t at = (blk - a.block0[s]) * 256 + threadIdx.x;
  if (at >= units) return;
  T* base = static_cast<T*>(a.state[s]) + g * K * units + at;
  T v[KMAX];
#pragma unroll
  for (int i = 0; i < KMAX; ++i)
    if (from[i] != i) v[i] = __builtin_nontemporal_load(base + from[i] * units);
#pragma unroll
  for (int i = 0; i < KMAX; ++i)
    if (from[i] != i) __builtin_nontemporal_store(v[i], base + i * units);
}

template <typename E>
hipError_t launch_select_t(const BeamSelectArgs& a, hipStream_t stream) {
  const int64_t rows = (int64_t)a.groups * a.beams;
  hipLaunchKernelGGL(beam_scan_kernel<E>, dim3((unsigned)(rows * a.plan.slices)), dim3(kBeamThreads), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(beam_pick_kernel<E>, dim3((unsigned)a.groups), dim3(64 * a.beams), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_beam_select(const BeamSelectArgs& a, hipStream_t stream) {
  return a.bf16 ? launch_select_t<__bf16>(a, stream) : launch_select_t<float>(a, stream);
}

template <typename T>
static hipError_t launch_reorder_t(BeamReorderArgs a, hipStream_t stream) {
  a.blocks = 0;
  for (int s = 0; s < a.count; ++s) {
    a.block0[s] = a.blocks;
    a.blocks += (a.row_units[s] + 255) / 256;
  }
  if (a.blocks == 0) return hipSuccess;
  const int64_t most = UINT32_MAX / 256 / a.blocks;  // groups of a launch (below 2^32 threads)
  for (a.group0 = 0; a.group0 < a.groups; a.group0 += most) {
    const dim3 g((unsigned)(std::min(a.groups - a.group0, most) * a.blocks)), b(256);
    if (a.beams <= 4) hipLaunchKernelGGL((beam_reorder_kernel<T, 4>), g, b, 0, stream, a);
    else if (a.beams <= 8) hipLaunchKernelGGL((beam_reorder_kernel<T, 8>), g, b, 0, stream, a);
    else hipLaunchKernelGGL((beam_reorder_kernel<T, 16>), g, b, 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_beam_reorder(const BeamReorderArgs& a, int unit, hipStream_t stream) {
  if (unit == 16) return launch_reorder_t<u32x4>(a, stream);
  if (unit == 4) return launch_reorder_t<uint32_t>(a, stream);
  return launch_reorder_t<uint8_t>(a, stream);
}

}  // namespace kda
