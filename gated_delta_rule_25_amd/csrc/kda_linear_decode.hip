// kda_linear_decode.hip — one token of per-head-decay linear attention for
// many independent sequences, and the precondition checks of its calls.
//
//   S <- a S + k v^T,   o = S^T q    (read after the token's write)
//
// One pass over the state: a thread scales its elements, adds k_i v_j, stores
// them and keeps the products with q_i; nothing of the new state depends on a
// sum over the old one, so stores follow their own loads with no barrier
// between.  Bound by HBM: 128 KiB of state per (sequence, head) and step
// against 4 x 128^2 flops (256 sequences x 96 heads: 550 us, 5.9 TB/s).
#include "kda.h"
#include "kda_device.h"
#include "kda_internal.h"
#include "kda_linear_internal.h"

namespace kda {
namespace {

// One 256-thread workgroup per (sequence, head, block of 128 / SPLIT value
// columns).  Thread t owns four columns and 16 / SPLIT consecutive rows.
template <typename E, int SPLIT>
__global__ __launch_bounds__(256) void linear_decode_kernel(const LinearDecodeArgs p) {
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
  const float a = __expf(p.decay_per_head ? p.log_decay[h] : p.log_decay[u]);
  // a zero drops the state, whatever it holds (infinities and NaN times zero
  // would be NaN); chosen element by element, as a branch would wait for all of
  // the state (256 sequences x 96 heads: 550 us, with a branch 572)
  const bool keep = a != 0.f;
  const E* v = static_cast<const E*>(p.v) + u * D + col;
  const E* q = static_cast<const E*>(p.q) + uq * D + R * rg;
  const E* k = static_cast<const E*>(p.k) + uq * D + R * rg;
  const f32x4 vv = (f32x4){to_f32(v[0]), to_f32(v[1]), to_f32(v[2]), to_f32(v[3])};
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < R; ++i) {
    f32x4 old = a * st[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) old[j] = keep ? old[j] : 0.f;
    const f32x4 ns = old + to_f32(k[i]) * vv;
    __builtin_nontemporal_store(ns, reinterpret_cast<f32x4*>(S + i * D));
    o += to_f32(q[i]) * ns;
  }
  // sum over the row groups: the lanes of a wave that share columns, then the waves
#pragma unroll
  for (int m = 32; m >= CG; m >>= 1)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] += __shfl_xor(o[j], m);
  __shared__ f32x4 part[4][CG];
  if ((t & 63) < CG) part[t >> 6][cg] = o;
  __syncthreads();
  if (t < CG) {
    o = part[0][t];
#pragma unroll
    for (int w = 1; w < 4; ++w) o += part[w][t];
    E* dst = static_cast<E*>(p.o) + u * D + col;
#pragma unroll
    for (int j = 0; j < 4; ++j) dst[j] = from_f32<E>(o[j]);
  }
}

template <typename E, int SPLIT>
hipError_t launch_decode_s(const LinearDecodeArgs& a, hipStream_t stream) {
  const int64_t units = (int64_t)a.num_seqs * a.num_heads;
  hipLaunchKernelGGL((linear_decode_kernel<E, SPLIT>), dim3((unsigned)(units * SPLIT)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

// Up to here the states fit the 256 MiB cache in front of HBM, and four
// workgroups for each keep more loads in flight (1 x 32 heads: 2.8 us now, 3.1
// against 5.1 when this was chosen; 4 x 96: 6.3 against 10.9; 32 x 96: 75 against 78); beyond, rows of 128
// bytes cost more than whole ones (256 x 96: 614 us against 568).
constexpr int64_t kSplitUnits = 4096;

template <typename E>
hipError_t launch_decode_e(const LinearDecodeArgs& a, hipStream_t stream) {
  const int64_t units = (int64_t)a.num_seqs * a.num_heads;
  return units <= kSplitUnits ? launch_decode_s<E, 4>(a, stream) : launch_decode_s<E, 1>(a, stream);
}

__device__ unsigned int g_linear_flags;

__global__ void linear_flags_clear_kernel() { g_linear_flags = 0; }

__global__ __launch_bounds__(256) void linear_check_kernel(const float* la, int64_t count, const int32_t* cu,
                                                           int num_seqs, int64_t total_tokens) {
  unsigned int bad = 0;
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += step)
    if (!(la[i] <= 0.f)) bad |= KDA_CHECK_LOG_ALPHA;
  if (cu)
    for (int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x; n < num_seqs; n += step) {
      if (cu[n + 1] < cu[n]) bad |= KDA_CHECK_CU_SEQLENS;
      if (n == 0 && (cu[0] != 0 || (int64_t)cu[num_seqs] != total_tokens)) bad |= KDA_CHECK_CU_SEQLENS;
    }
  if (bad) atomicOr(&g_linear_flags, bad);
}

}  // namespace

hipError_t launch_linear_decode(const LinearDecodeArgs& a, hipStream_t stream) {
  return a.bf16 ? launch_decode_e<__bf16>(a, stream) : launch_decode_e<float>(a, stream);
}

hipError_t run_linear_checks(const float* log_decay, int64_t count, const int32_t* cu, int num_seqs,
                             int64_t total_tokens, hipStream_t stream, uint32_t* flags) {
  *flags = 0;
  void* dflag = nullptr;
  hipError_t e = hipGetSymbolAddress(&dflag, HIP_SYMBOL(g_linear_flags));
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(linear_flags_clear_kernel, dim3(1), dim3(1), 0, stream);
  hipLaunchKernelGGL(linear_check_kernel, dim3(1024), dim3(256), 0, stream, log_decay, count, cu, num_seqs,
                     total_tokens);
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
