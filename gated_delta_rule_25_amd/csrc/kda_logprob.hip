// kda_logprob.hip — log probabilities of given tokens, entropies and the most
// probable tokens of rows of logits, and their gradient.
//
// Forward, one workgroup per row and one pass over it.  With d = x - m and m a
// running maximum, a thread keeps s = sum e^d and w = sum d e^d; when the maximum
// moves by c = m - m' both are e^c (s, w + c s).  The row's z = m + log s, and
// the entropy is log s - w / s: no difference of large numbers, whatever the
// logits' size.  The K best of the row need no sorting and no second pass over
// it: a thread notes the largest element of its part (its vectors), and the K
// best parts hold the K best elements (were an element's part not among them,
// K others would precede it).  One wave picks those parts, K rounds of the
// largest, and reads their vectors again; what they hold above the last of the K
// is put into the list, which a row of lanes keeps in order.  Bound by HBM where
// there are many rows (2048 of 128003 bf16 with 8 alternatives: 117 us, 4.5 TB/s), by
// the chain of loads, reductions and reads where few (4 of 32000 fp32: 12 us).
//
// Backward: elementwise, one read and one write of the row (none where nothing
// reaches it; one more read where log s is lost beside the largest logit, below).
// Bound by HBM (4096 rows of 128003 bf16: 433 us, 4.8 TB/s).
#include <algorithm>

#include "kda_logits.h"
#include "kda_logprob_internal.h"

namespace kda {
namespace {

constexpr float kLog2e = 1.44269504f;
// Differences below this count as this: e^-150 is below the smallest fp32
// number, and -inf times zero would be NaN.
constexpr float kLeast = -150.f;

template <typename E, int THREADS>
__global__ __launch_bounds__(THREADS) void logprob_kernel(const LogprobArgs a) {
  constexpr int U = 16 / (int)sizeof(E);
  constexpr int WAVES = THREADS / 64, PL = THREADS / 64;  // parts a lane of the picking wave holds
  const int64_t row = blockIdx.x;
  const int t = threadIdx.x, lane = t & 63, V = a.vocab;
  const int wv = __builtin_amdgcn_readfirstlane(t >> 6);
  const E* x = static_cast<const E*>(a.logits) + row * a.row_stride;
  const BeamRow r = beam_row(x, V);
  const int token = a.tokens ? a.tokens[row] : -1;
  const bool scored = token >= 0 && token < V;
  const float given = scored ? load_logit(x + token) : 0.f;

  float best = -INFINITY, top = -INFINITY, s = 0.f, w = 0.f;
  int at = INT32_MAX;
  auto fold = [&](float m) {
    if (m > top) {
      const float c = fmaxf(top - m, kLeast);
      const float f = beam_exp(c);
      w = f * (w + c * s);
      s *= f;
      top = m;
    }
  };
  auto add = [&](float v) {
    const float d = fmaxf(v - top, kLeast);
    const float e = beam_exp(d);
    s += e;
    w += d * e;
  };
  auto take = [&](const float (&v)[U], int e0) {
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
      for (int j = 0; j < U; ++j) add(v[j]);
    } else if (at == INT32_MAX) {
      at = e0;
    }
  };
  // four vectors in flight
  int vec = t;
  for (; vec + 3 * THREADS < r.nvec; vec += 4 * THREADS) {
    float v[4][U];
#pragma unroll
    for (int i = 0; i < 4; ++i) load_vector<E>(v[i], x + r.head + (int64_t)(vec + i * THREADS) * U);
#pragma unroll
    for (int i = 0; i < 4; ++i) take(v[i], r.head + (vec + i * THREADS) * U);
  }
  for (; vec < r.nvec; vec += THREADS) {
    float v[U];
    load_vector<E>(v, x + r.head + (int64_t)vec * U);
    take(v, r.head + vec * U);
  }
  {
    const int i = beam_extra<E>(r, V, t);
    if (i >= 0) {
      const float v = load_logit(x + i);
      if (v > best || (v == best && i < at)) {
        best = v;
        at = i;
      }
      if (v > -INFINITY) {
        fold(v);
        add(v);
      }
    }
  }

  // over the workgroup
  __shared__ float sm[WAVES];
  __shared__ double ss[2][WAVES];
  __shared__ uint64_t keys[THREADS];
  const float wm = wave_fmax(top);
  if (lane == 0) sm[wv] = wm;
  if (a.top > 0) keys[t] = at == INT32_MAX ? 0 : beam_key(best, (uint32_t)at);
  __syncthreads();
  float m = sm[0];
#pragma unroll
  for (int i = 1; i < WAVES; ++i) m = fmaxf(m, sm[i]);
  {
    const float c = top > -INFINITY ? fmaxf(top - m, kLeast) : 0.f;
    const double f = (double)beam_exp(c);
    double ds = f * (double)s, dw = f * ((double)w + (double)c * (double)s);
#pragma unroll
    for (int k = 32; k >= 1; k >>= 1) {
      ds += __shfl_xor(ds, k);
      dw += __shfl_xor(dw, k);
    }
    if (lane == 0) {
      ss[0][wv] = ds;
      ss[1][wv] = dw;
    }
  }
  __syncthreads();
  if (wv != 0) return;
  double ds = 0.0, dw = 0.0;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) {
    ds += ss[0][i];
    dw += ss[1][i];
  }
  const bool any = m > -INFINITY;  // (else the row is masked throughout)
  const double log_s = any ? log(ds) : 0.0;
  auto logprob = [&](float v) {
    return v > -INFINITY ? (float)((double)v - (double)m - log_s) : -INFINITY;
  };
  if (lane == 0) {
    if (a.logprobs) a.logprobs[row] = scored ? logprob(given) : 0.f;
    if (a.log_sum) a.log_sum[row] = any ? (float)((double)m + log_s) : -INFINITY;
    if (a.entropy) a.entropy[row] = any ? (float)fmax(log_s - dw / ds, 0.0) : 0.f;
  }
  if (a.top == 0) return;

  // the best parts: lane i < K ends with the i-th of their largest elements
  const int K = a.top;
  uint64_t key[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) key[i] = keys[64 * i + lane];
  uint64_t list = 0;
  int part = -1;
  for (int k = 0; k < K; ++k) {
    uint64_t mine = key[0];
#pragma unroll
    for (int i = 1; i < PL; ++i) mine = key[i] > mine ? key[i] : mine;
    const uint64_t most = wave_max(mine);
    if (most == 0) break;  // (fewer parts than K)
    const uint64_t who = __ballot(mine == most);
    const int src = __builtin_ctzll(who);
    int slot = 0;
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (key[i] == most) {
        slot = i;
        if (lane == src) key[i] = 0;
      }
    const int p = 64 * __builtin_amdgcn_readlane(slot, src) + src;
    if (lane == k) {
      list = most;
      part = p;
    }
  }
  const int parts = __popcll(__ballot(part >= 0));
  const int first = part >= 0 ? (int)key_at(list) : -1;  // where the part's largest is
  // what else they hold that belongs into the list
  auto least_of = [&] {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(list >> 32), K - 1) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)list, K - 1);
  };
  uint64_t least = least_of();
  auto offer = [&](uint64_t c) {  // each lane's candidate (0: none)
    uint64_t who = __ballot(c > least);
    while (who) {
      const int src = __builtin_ctzll(who);
      const uint64_t n = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(c >> 32), src) << 32 |
                         (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)c, src);
      const int place = __popcll(__ballot(lane < K && list > n));
      const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)list, 0x111, 0xf, 0xf, true);
      const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(list >> 32), 0x111, 0xf, 0xf, true);
      if (lane < K) list = lane < place ? list : lane == place ? n : (uint64_t)hi << 32 | lo;
      least = least_of();
      if (lane == src) c = 0;
      who = __ballot(c > least);
    }
  };
  for (int i0 = 0; i0 * 64 < (r.nvec + THREADS - 1) / THREADS; ++i0) {
    // vector i0 * 64 + lane of each part, eight parts' loads in flight
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (8 * half >= parts) break;
      float v[8][U];
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const int of = __builtin_amdgcn_readlane(part, 8 * half + p);
        const int vec = (i0 * 64 + lane) * THREADS + of;
        if (8 * half + p < parts && vec < r.nvec) {
          load_vector<E>(v[p], x + r.head + (int64_t)vec * U);
        }
      }
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        if (8 * half + p >= parts) break;
        const int of = __builtin_amdgcn_readlane(part, 8 * half + p);
        const int vec = (i0 * 64 + lane) * THREADS + of;
        // (the part's largest is in the list already)
        const int known = __builtin_amdgcn_readlane(first, 8 * half + p) - (r.head + vec * U);
        const bool in = vec < r.nvec;
        const float bar = least == 0 ? -INFINITY : key_value(least);
        bool any_in = false;
#pragma unroll
        for (int j = 0; j < U; ++j) any_in |= in && j != known && v[p][j] >= bar;
        if (__ballot(any_in) == 0) continue;
#pragma unroll
        for (int j = 0; j < U; ++j) offer(in && j != known ? beam_key(v[p][j], (uint32_t)(r.head + vec * U + j)) : 0);
      }
    }
  }
  // the elements outside the vectors
  for (int p = 0; p < parts; ++p) {
    const int of = __builtin_amdgcn_readlane(part, p);
    const int i = beam_extra<E>(r, V, of);
    if (i < 0) continue;
    const bool known = i == __builtin_amdgcn_readlane(first, p);
    offer(lane == 0 && !known ? beam_key(load_logit(x + i), (uint32_t)i) : 0);
  }
  if (lane < K) {
    a.top_logprobs[row * K + lane] = logprob(key_value(list));
    a.top_tokens[row * K + lane] = (int32_t)key_at(list);
  }
}

// ---------------------------------------------------------------------------
// Gradient: `slices` workgroups per row.
// ---------------------------------------------------------------------------
constexpr int kGradThreads = 256;

// log p = x - z is off by half a step of z, and p by as much of itself: 2^-15 of it
// where |z| is below this, in bf16 (whose results are rounded to 2^-9) 2^-13.  Logits
// that are all as large as that are rare, and then one step of z may be more than
// log s: a row filled with its type's lowest value would get p = 1 for every token.
// Farther out one of a row's workgroups reads it once more, finds its largest m and
// log s, and takes it alone, as d_logits may be the logits: log p = (x - m) - log s.
// (4096 such rows of 128003 bf16: 1.30 ms, others 0.44; one row 35 us for 5.6.)
template <typename E>
constexpr float kFar = sizeof(E) == 2 ? 4096.f : 1024.f;

// m and log s of a row that is not masked throughout; every thread's reads have
// ended.  What they make is taken only if it is z: else z is what the caller wants.
template <typename E>
__device__ __forceinline__ void largest_and_sum(const E* x, const BeamRow& r, int V, float z, float& top, float& log_s) {
  constexpr int U = 16 / (int)sizeof(E), WAVES = kGradThreads / 64;
  const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
  float m = -INFINITY;
  double s = 0.0;
  // N vectors, or what there is of them
  auto take = [&](const auto& v) {
    constexpr int N = sizeof(v) / sizeof(float);
    const float* y = &v[0][0];
    float vm = y[0];
#pragma unroll
    for (int j = 1; j < N; ++j) vm = fmaxf(vm, y[j]);
    if (vm > m) {
      s *= (double)beam_exp(fmaxf(m - vm, kLeast));
      m = vm;
    }
    if (m == -INFINITY) return;
    float part = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) part += beam_exp(fmaxf(y[j] - m, kLeast));
    s += (double)part;
  };
  int vec = t;
  for (; vec + 3 * kGradThreads < r.nvec; vec += 4 * kGradThreads) {
    float v[4][U];
#pragma unroll
    for (int i = 0; i < 4; ++i) load_vector<E>(v[i], x + r.head + (int64_t)(vec + i * kGradThreads) * U);
    take(v);
  }
  for (; vec < r.nvec; vec += kGradThreads) {
    float v[1][U];
    load_vector<E>(v[0], x + r.head + (int64_t)vec * U);
    take(v);
  }
  const int i = beam_extra<E>(r, V, t);
  if (i >= 0) {
    const float v[1][1] = {{load_logit(x + i)}};
    take(v);
  }
  __shared__ float sm[WAVES];
  __shared__ double ss[WAVES];
  const float wm = wave_fmax(m);
  if (lane == 0) sm[wv] = wm;
  __syncthreads();
  float all = sm[0];
#pragma unroll
  for (int k = 1; k < WAVES; ++k) all = fmaxf(all, sm[k]);
  s *= m > -INFINITY ? (double)beam_exp(fmaxf(m - all, kLeast)) : 0.0;
#pragma unroll
  for (int k = 32; k >= 1; k >>= 1) s += __shfl_xor(s, k);
  if (lane == 0) ss[wv] = s;
  __syncthreads();
  s = 0.0;
#pragma unroll
  for (int k = 0; k < WAVES; ++k) s += ss[k];
  const double l = log(s);
  if (fabs((double)all + l - (double)z) <= fabs((double)z) * 0x1p-23) {
    top = all;
    log_s = (float)l;
  }
}

template <typename E>
__global__ __launch_bounds__(kGradThreads) void logprob_grad_kernel(const LogprobGradArgs a) {
  constexpr int U = 16 / (int)sizeof(E);
  const int64_t row = a.row0 + blockIdx.x / a.slices;
  int slice = (int)(blockIdx.x % a.slices);
  const int V = a.vocab;
  const E* x = static_cast<const E*>(a.logits) + row * a.row_stride;
  E* dx = static_cast<E*>(a.d_logits) + row * a.d_row_stride;
  const int token = a.tokens[row];
  const float z = a.log_sum[row];
  const bool any = z > -INFINITY;
  const bool scored = any && token >= 0 && token < V;
  const float g = scored ? a.d_logprobs[row] : 0.f;
  const float h = any && a.d_entropy ? a.d_entropy[row] : 0.f;
  // -p (g + h (log p + entropy))
  const float c = h != 0.f ? g + h * a.entropy[row] : g;
  float top = z, log_s = 0.f;  // z as a sum
  auto grad = [&](float v, int i) {
    const float d = fmaxf((v - top) - log_s, kLeast);
    const float y = -beam_exp(d) * (c + h * d);
    return i == token ? y + g : y;
  };
  const bool zero = g == 0.f && h == 0.f;
  const BeamRow r = beam_row(x, V);
  const bool same = ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(dx)) & 15) == 0;
  const bool far = !zero && fabsf(z) >= kFar<E>;
  const int stride = far ? kGradThreads : kGradThreads * a.slices;
  if (far) {
    // (another of each row's, for all XCDs to have their part)
    if (slice != (int)(row % a.slices)) return;
    slice = 0;
    largest_and_sum(x, r, V, z, top, log_s);
  }
  int vec = slice * kGradThreads + threadIdx.x;
  auto put = [&](float (&v)[U], int e0) {
    if (zero) {
#pragma unroll
      for (int j = 0; j < U; ++j) v[j] = 0.f;
    } else {
#pragma unroll
      for (int j = 0; j < U; ++j) v[j] = grad(v[j], e0 + j);
    }
    if (same) {
      u32x4 y;
      if constexpr (sizeof(E) == 2) {
        typedef __bf16 v8 __attribute__((ext_vector_type(8)));
        v8 b;
#pragma unroll
        for (int j = 0; j < U; ++j) b[j] = (__bf16)v[j];
        y = __builtin_bit_cast(u32x4, b);
      } else {
        const f32x4 b = {v[0], v[1], v[2], v[3]};
        y = __builtin_bit_cast(u32x4, b);
      }
      __builtin_nontemporal_store(y, reinterpret_cast<u32x4*>(dx + e0));
    } else {
#pragma unroll
      for (int j = 0; j < U; ++j) dx[e0 + j] = from_f32<E>(v[j]);
    }
  };
  // (one workgroup: four vectors in flight)
  if (far)
    for (; vec + 3 * kGradThreads < r.nvec; vec += 4 * kGradThreads) {
      float v[4][U];
#pragma unroll
      for (int i = 0; i < 4; ++i) load_vector<E>(v[i], x + r.head + (vec + i * kGradThreads) * U);
#pragma unroll
      for (int i = 0; i < 4; ++i) put(v[i], r.head + (vec + i * kGradThreads) * U);
    }
  for (; vec < r.nvec; vec += stride) {
    float v[U];
    if (!zero) load_vector<E>(v, x + r.head + vec * U);
    put(v, r.head + vec * U);
  }
  if (slice == 0) {
    const int i = beam_extra<E>(r, V, threadIdx.x);
    if (i >= 0) dx[i] = from_f32<E>(zero ? 0.f : grad(load_logit(x + i), i));
  }
}

template <typename E>
hipError_t launch_e(const LogprobArgs& a, int cus, hipStream_t stream) {
  // Few rows: as many loads in flight for each as a workgroup can have.  (256 units, bf16 of 128003 tokens: 64
  // rows 24.7 us with 1024 threads and 29.7 with 256, 256 rows 30 and 42, 512 rows 48 and 48, 640 rows 65 and 56.)
  if (a.rows <= 2 * (int64_t)cus)
    hipLaunchKernelGGL((logprob_kernel<E, 1024>), dim3((unsigned)a.rows), dim3(1024), 0, stream, a);
  else
    hipLaunchKernelGGL((logprob_kernel<E, 256>), dim3((unsigned)a.rows), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_logprob(const LogprobArgs& a, int cus, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  return a.bf16 ? launch_e<__bf16>(a, cus, stream) : launch_e<float>(a, cus, stream);
}

hipError_t launch_logprob_grad(LogprobGradArgs a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  const int64_t rows = a.rows;
  // eight vectors a thread
  const int64_t vectors = (int64_t)a.vocab * (a.bf16 ? 2 : 4) / 16;
  a.slices = (int)std::min<int64_t>(std::max<int64_t>((vectors + 8 * kGradThreads - 1) / (8 * kGradThreads), 1), 64);
  const int64_t most = ((int64_t)0xffffffff / kGradThreads) / a.slices;
  for (int64_t r0 = 0; r0 < rows; r0 += most) {
    a.row0 = r0;
    a.rows = std::min(rows - r0, most);
    const dim3 grid((unsigned)(a.rows * a.slices));
    if (a.bf16) hipLaunchKernelGGL(logprob_grad_kernel<__bf16>, grid, dim3(kGradThreads), 0, stream, a);
    else hipLaunchKernelGGL(logprob_grad_kernel<float>, grid, dim3(kGradThreads), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace kda
