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
//                      to the thread's own maximum, fp32; combined in fp64).
//                      Bound by HBM.
//   beam_pick_kernel   one workgroup per group, a wave per beam: the K best
//                      parts, their elements read again (K x nv vectors), the
//                      row's K best; then one wave takes the K best of the
//                      K x K candidates, compared as fp64 scores.
// Nothing depends on the order in which workgroups run.
//
// Reordering.  Row n of a group's states becomes the row of its parent.  A
// thread owns the same few bytes of all the group's rows, reads what moves and
// then writes it, so the rows change in place with no copy of the states and
// no barrier, and rows that stay are not touched.
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

__device__ __forceinline__ uint64_t wave_max(uint64_t x) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    const uint64_t o = __shfl_xor((unsigned long long)x, m);
    x = o > x ? o : x;
  }
  return x;
}

// NaN is a masked logit like -inf; +inf counts as the largest number.
__device__ __forceinline__ float beam_logit(float x) { return fminf(x == x ? x : -INFINITY, FLT_MAX); }
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
      sum *= top > -INFINITY ? __expf(top - m) : 0.f;
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
      for (int j = 0; j < U; ++j) sum += expf(v[j] - top);
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
        sum += expf(v - top);
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
  double d = top > -INFINITY ? (double)sum * (double)expf(top - m) : 0.0;
#pragma unroll
  for (int k = 32; k >= 1; k >>= 1) d += __shfl_xor(d, k);
  if ((t & 63) == 0) ss[t >> 6] = d;
  __syncthreads();
  if (t == 0) {
    a.slice_max[row * a.plan.slices + slice] = m;
    a.slice_sum[row * a.plan.slices + slice] = (float)(ss[0] + ss[1] + ss[2] + ss[3]);
  }
}

struct BeamCandidate {
  double score;
  uint64_t at;  // beam * vocab + token
};
__device__ __forceinline__ bool better(const BeamCandidate& a, const BeamCandidate& b) {
  return a.score > b.score || (a.score == b.score && a.at < b.at);
}

// One workgroup per group, wave k for beam k.
template <typename E>
__global__ __launch_bounds__(64 * kBeamMax) void beam_pick_kernel(const BeamSelectArgs a) {
  constexpr int U = 16 / (int)sizeof(E);
  constexpr int PL = kBeamMaxParts / 64;  // parts per lane
  const int K = a.beams, V = a.vocab;
  const int g = blockIdx.x, lane = threadIdx.x & 63;
  const int k = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = (int64_t)g * K + k;
  __shared__ BeamCandidate cand[kBeamMax * kBeamMax];
  __shared__ uint8_t done[kBeamMax];
  const float score = a.scores[row];
  const bool fin = a.finished && a.finished[row];
  if (lane == 0) done[k] = fin;
  const int C = min(K, V);  // candidates of a row
  BeamCandidate mine = {-INFINITY, 0};  // lane i < C: the row's i-th best
  if (!row_is_read(a, row)) {
    // the end token if the beam is finished (a beam without a score ties at
    // -inf with everything), then the lowest tokens at -inf
    const bool ends = fin && score > -INFINITY && a.end_token >= 0 && a.end_token < V;
    int t = lane;
    if (ends) t = lane == 0 ? a.end_token : (lane - 1 < a.end_token ? lane - 1 : lane);
    mine.score = ends && lane == 0 ? (double)score : -INFINITY;
    mine.at = (uint64_t)k * V + t;
  } else {
    // log of the row's sum of exponentials
    float m = -INFINITY;
    for (int s = lane; s < a.plan.slices; s += 64) m = fmaxf(m, a.slice_max[row * a.plan.slices + s]);
#pragma unroll
    for (int i = 32; i >= 1; i >>= 1) m = fmaxf(m, __shfl_xor(m, i));
    double sum = 0.0;
    if (m > -INFINITY)
      for (int s = lane; s < a.plan.slices; s += 64) {
        const float sm = a.slice_max[row * a.plan.slices + s];
        if (sm > -INFINITY) sum += (double)a.slice_sum[row * a.plan.slices + s] * exp((double)sm - (double)m);
      }
#pragma unroll
    for (int i = 32; i >= 1; i >>= 1) sum += __shfl_xor(sum, i);
    const double lse = (double)m + log(sum);
    // the C best parts
    const int64_t parts = (int64_t)a.plan.slices * kBeamThreads;
    uint64_t pk[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int64_t p = lane + 64 * i;
      pk[i] = 0;
      if (p < parts) {
        const int at = a.part_at[row * parts + p];
        if (at != INT32_MAX) pk[i] = beam_key(a.part_max[row * parts + p], (uint32_t)at);
      }
    }
    const E* x = static_cast<const E*>(a.logits) + row * V;
    const BeamRow r = beam_row(x, V);
    int part = -1;  // lane i < C: the i-th best part
    uint64_t last = ~0ull;
    for (int c = 0; c < C; ++c) {
      uint64_t b = 0;
      int bi = 0;
#pragma unroll
      for (int i = 0; i < PL; ++i)
        if (pk[i] < last && pk[i] > b) {
          b = pk[i];
          bi = i;
        }
      const uint64_t w = wave_max(b);
      if (w == 0) break;  // fewer parts than candidates
      const uint64_t who = __ballot(b == w);
      const int src = __ffsll((unsigned long long)who) - 1;
      const int got = __shfl(lane + 64 * bi, src);
      if (lane == c) part = got;
      last = w;
    }
    // their elements: vector j of part i is lane (64 a turn); the list of the
    // best so far stays with the lanes 0 .. C - 1
    uint64_t list = 0;
    auto merge = [&](const uint64_t* key, int count) {
      uint64_t keep = 0, before = ~0ull;
      for (int c = 0; c < C; ++c) {
        uint64_t b = list < before ? list : 0;
        for (int i = 0; i < count; ++i)
          if (key[i] < before && key[i] > b) b = key[i];
        b = wave_max(b);
        if (lane == c) keep = b;
        before = b;
        if (b == 0) break;
      }
      list = keep;
    };
    const int nv = a.plan.nv;
    for (int v0 = 0; v0 < C * nv; v0 += 64) {
      const int id = v0 + lane;
      const int owner = __shfl(part, min(id / nv, C - 1));
      uint64_t key[U + 1];
#pragma unroll
      for (int j = 0; j <= U; ++j) key[j] = 0;
      if (id < C * nv && owner >= 0) {
        const int slice = owner / kBeamThreads, t = owner % kBeamThreads;
        const int vec = slice * kBeamThreads * nv + (id % nv) * kBeamThreads + t;
        if (vec < r.nvec) {
          const int e0 = r.head + vec * U;
#pragma unroll
          for (int j = 0; j < U; ++j) key[j] = beam_key(load_logit(x + e0 + j), (uint32_t)(e0 + j));
        }
        if (id % nv == 0 && slice == 0) {
          const int i = beam_extra<E>(r, V, t);
          if (i >= 0) key[U] = beam_key(load_logit(x + i), (uint32_t)i);
        }
      }
      merge(key, U + 1);
    }
    const float v = key_value(list);
    mine.score = v > -INFINITY ? (double)score + ((double)v - lse) : -INFINITY;
    mine.at = (uint64_t)k * V + key_at(list);
  }
  if (lane < C) cand[k * C + lane] = mine;
  __syncthreads();
  if (k != 0) return;
  // the K best of the K x C candidates (C = K, or V < K candidates a row)
  constexpr int CL = kBeamMax * kBeamMax / 64;
  BeamCandidate own[CL];
#pragma unroll
  for (int i = 0; i < CL; ++i) {
    own[i].score = -INFINITY;
    own[i].at = ~0ull;
    if (lane + 64 * i < K * C) own[i] = cand[lane + 64 * i];
    if (!(own[i].score == own[i].score)) own[i].score = -INFINITY;  // a score that is not a number
  }
  BeamCandidate prev = {INFINITY, 0};
  bool any = false;
  for (int c = 0; c < K; ++c) {
    BeamCandidate b = {-INFINITY, ~0ull};
#pragma unroll
    for (int i = 0; i < CL; ++i)
      if ((!any || better(prev, own[i])) && better(own[i], b)) b = own[i];
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) {
      BeamCandidate o;
      o.score = __shfl_xor(b.score, m);
      o.at = __shfl_xor((unsigned long long)b.at, m);
      if (better(o, b)) b = o;
    }
    prev = b;
    any = true;
    if (lane == 0) {
      // (V K >= K candidates always exist; the guard keeps a wrong one in range)
      const uint64_t at = b.at < (uint64_t)K * V ? b.at : 0;
      const int parent = (int)(at / V), token = (int)(at % V);
      const int64_t o = (int64_t)g * K + c;
      a.out_scores[o] = (float)b.score;
      a.out_tokens[o] = token;
      a.out_parents[o] = parent;
      if (a.out_finished) a.out_finished[o] = done[parent] || token == a.end_token;
    }
  }
}

// ---------------------------------------------------------------------------
// Reordering: a thread owns one unit of every row of its group.
// ---------------------------------------------------------------------------
template <typename T, int KMAX>
__global__ __launch_bounds__(256) void beam_reorder_kernel(const BeamReorderArgs a) {
  const int64_t blk = blockIdx.x % a.blocks;
  const int64_t g = blockIdx.x / a.blocks;
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
  const int64_t grid = a.blocks * a.groups;
  if (grid == 0) return hipSuccess;
  const dim3 g((unsigned)grid), b(256);
  if (a.beams <= 4) hipLaunchKernelGGL((beam_reorder_kernel<T, 4>), g, b, 0, stream, a);
  else if (a.beams <= 8) hipLaunchKernelGGL((beam_reorder_kernel<T, 8>), g, b, 0, stream, a);
  else hipLaunchKernelGGL((beam_reorder_kernel<T, 16>), g, b, 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_beam_reorder(const BeamReorderArgs& a, int unit, hipStream_t stream) {
  if (unit == 16) return launch_reorder_t<u32x4>(a, stream);
  if (unit == 4) return launch_reorder_t<uint32_t>(a, stream);
  return launch_reorder_t<uint8_t>(a, stream);
}

}  // namespace kda
