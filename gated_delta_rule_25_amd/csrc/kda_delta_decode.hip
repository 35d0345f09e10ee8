// kda_delta_decode.hip — one token of the gated delta rule with one decay per
// head for many independent sequences, and the precondition checks of its calls.
//
//   S~ = a S,  u = beta (v - S~^T k),  S <- S~ + k u^T,  o = S^T q = S~^T q + (k . q) u
//
// One pass over the state: both column sums, S^T k and S^T q, come from the
// registers that the update is formed in.  Bound by HBM: 128 KiB of state per
// (sequence, head) and step against 7 x 128^2 flops; 256 sequences x 96 heads take
// 532 us, 6.1 TB/s.
#include "kda.h"
#include "kda_api_util.h"
#include "kda_delta_internal.h"
#include "kda_device.h"
#include "kda_internal.h"

namespace kda {
namespace {

// One 256-thread workgroup per (sequence, head, block of 128 / SPLIT value
// columns).  Thread t owns four columns and 16 / SPLIT consecutive rows.
template <typename E, int SPLIT>
__global__ __launch_bounds__(256) void delta_decode_kernel(const DeltaDecodeArgs p) {
  constexpr int CG = 32 / SPLIT;    // groups of four columns
  constexpr int RG = 256 / CG;      // row groups
  constexpr int R = D / RG;         // rows per thread
  const int64_t u = blockIdx.x / SPLIT;  // n * H + h
  const int cb = blockIdx.x % SPLIT;
  const int t = threadIdx.x, cg = t % CG, rg = t / CG;
  const int col = cb * (D / SPLIT) + 4 * cg;
  const int H = p.num_heads;
  const int h = (int)(u % H);
  const int64_t n = u / H;
  const int64_t uq = n * p.qk_heads + h / (H / p.qk_heads);

  float* S = p.state + u * (D * D) + (R * rg) * D + col;
  f32x4 st[R];
#pragma unroll
  for (int i = 0; i < R; ++i) st[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(S + i * D));
  const float a = __expf(p.log_decay[u]);
  const float beta = p.beta[u];
  // a zero drops the state, whatever it holds (infinities and NaN times zero
  // would be NaN)
  const bool keep = a != 0.f;
  const E* v = static_cast<const E*>(p.v) + u * D + col;
  const E* q = static_cast<const E*>(p.q) + uq * D + R * rg;
  const E* k = static_cast<const E*>(p.k) + uq * D + R * rg;
  const f32x4 vv = (f32x4){to_f32(v[0]), to_f32(v[1]), to_f32(v[2]), to_f32(v[3])};
  f32x4 x = {0.f, 0.f, 0.f, 0.f}, y = {0.f, 0.f, 0.f, 0.f};
  float kq = 0.f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    st[i] *= a;
#pragma unroll
    for (int j = 0; j < 4; ++j) st[i][j] = keep ? st[i][j] : 0.f;
    const float kk = to_f32(k[i]), qq = to_f32(q[i]);
    x += kk * st[i];
    y += qq * st[i];
    kq += kk * qq;
  }
  // sums over the row groups: the lanes of a wave that share columns, then the waves
#pragma unroll
  for (int m = 32; m >= CG; m >>= 1) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] += __shfl_xor(x[j], m);
      y[j] += __shfl_xor(y[j], m);
    }
    kq += __shfl_xor(kq, m);
  }
  __shared__ f32x4 part[2][4][CG];
  __shared__ float part_kq[4];
  if ((t & 63) < CG) {
    part[0][t >> 6][cg] = x;
    part[1][t >> 6][cg] = y;
  }
  if ((t & 63) == 0) part_kq[t >> 6] = kq;
  __syncthreads();
  x = part[0][0][cg];
  y = part[1][0][cg];
  kq = part_kq[0];
#pragma unroll
  for (int w = 1; w < 4; ++w) {
    x += part[0][w][cg];
    y += part[1][w][cg];
    kq += part_kq[w];
  }
  const f32x4 uu = beta * (vv - x);
#pragma unroll
  for (int i = 0; i < R; ++i)
    __builtin_nontemporal_store(st[i] + to_f32(k[i]) * uu, reinterpret_cast<f32x4*>(S + i * D));
  if (t < CG) {
    const f32x4 o = y + kq * uu;
    E* dst = static_cast<E*>(p.o) + u * D + col;
#pragma unroll
    for (int j = 0; j < 4; ++j) dst[j] = from_f32<E>(o[j]);
  }
}

template <typename E, int SPLIT>
hipError_t launch_decode_s(const DeltaDecodeArgs& a, hipStream_t stream) {
  const int64_t units = (int64_t)a.num_seqs * a.num_heads;
  hipLaunchKernelGGL((delta_decode_kernel<E, SPLIT>), dim3((unsigned)(units * SPLIT)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

// Four workgroups per state, on 32 of its columns each, while that adds loads in
// flight: 64 states 4.7 us for 6.5, 384 states 8.1 for 9.6; beyond, rows of 128
// bytes cost more than whole ones: 512 states 12.0 us for 10.4, 24576 616 for 533.
constexpr int64_t kSplitUnits = 448;

template <typename E>
hipError_t launch_decode_e(const DeltaDecodeArgs& a, hipStream_t stream) {
  const int64_t units = (int64_t)a.num_seqs * a.num_heads;
  return units <= kSplitUnits ? launch_decode_s<E, 4>(a, stream) : launch_decode_s<E, 1>(a, stream);
}

__device__ unsigned int g_delta_flags;

__global__ void delta_flags_clear_kernel() { g_delta_flags = 0; }

// One wave per key row (its length) and, by strides, the scalars.
template <typename E>
__global__ __launch_bounds__(256) void delta_check_kernel(const E* k, int64_t k_rows, const float* la, const float* beta,
                                                          int64_t count, const int32_t* cu, int num_seqs,
                                                          int64_t total_tokens) {
  unsigned int bad = 0;
  const int64_t step = (int64_t)gridDim.x * 256;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  for (int64_t r = at >> 6; r < k_rows; r += step >> 6) {
    const int lane = threadIdx.x & 63;
    const float a = to_f32(k[r * D + 2 * lane]), b = to_f32(k[r * D + 2 * lane + 1]);
    float s = a * a + b * b;
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) s += __shfl_xor(s, m);
    if (!(s <= 1.02f * 1.02f)) bad |= KDA_CHECK_K_NORM;
  }
  for (int64_t i = at; i < count; i += step) {
    if (!(la[i] <= 0.f)) bad |= KDA_CHECK_LOG_ALPHA;
    if (!(beta[i] >= 0.f && beta[i] <= 1.f)) bad |= KDA_CHECK_BETA;
  }
  if (cu)
    for (int64_t n = at; n < num_seqs; n += step) {
      if (cu[n + 1] < cu[n]) bad |= KDA_CHECK_CU_SEQLENS;
      if (n == 0 && (cu[0] != 0 || (int64_t)cu[num_seqs] != total_tokens)) bad |= KDA_CHECK_CU_SEQLENS;
    }
  if (bad) atomicOr(&g_delta_flags, bad);
}

}  // namespace

hipError_t launch_delta_decode(const DeltaDecodeArgs& a, hipStream_t stream) {
  return a.bf16 ? launch_decode_e<__bf16>(a, stream) : launch_decode_e<float>(a, stream);
}

hipError_t run_delta_checks(const void* k, bool bf16, int64_t k_rows, const float* log_decay, const float* beta,
                            int64_t count, const int32_t* cu, int num_seqs, int64_t total_tokens, hipStream_t stream,
                            uint32_t* flags) {
  const std::lock_guard<std::mutex> lock(checks_mutex());
  *flags = 0;
  void* dflag = nullptr;
  hipError_t e = hipGetSymbolAddress(&dflag, HIP_SYMBOL(g_delta_flags));
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(delta_flags_clear_kernel, dim3(1), dim3(1), 0, stream);
  if (bf16)
    hipLaunchKernelGGL(delta_check_kernel<__bf16>, dim3(1024), dim3(256), 0, stream, static_cast<const __bf16*>(k),
                       k_rows, log_decay, beta, count, cu, num_seqs, total_tokens);
  else
    hipLaunchKernelGGL(delta_check_kernel<float>, dim3(1024), dim3(256), 0, stream, static_cast<const float*>(k),
                       k_rows, log_decay, beta, count, cu, num_seqs, total_tokens);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  unsigned int host = 0;
  e = hipMemcpyAsync(&host, dflag, sizeof(host), hipMemcpyDeviceToHost, stream);
  if (e != hipSuccess) return e;
  e = hipStreamSynchronize(stream);
  if (e != hipSuccess) return e;
  *flags = host;
  return hipSuccess;
}

}  // namespace kda
