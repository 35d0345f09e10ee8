// kda_delta_prep.hip — what a chunk of the gated delta rule has to be solved
// for, token-parallel.
//
// Within a chunk of C tokens, with A_ij = (k_i . k_j) e^{G_i - G_j} for j < i
// (G: prefix sums of the log decays) and B = Diag(beta), the values that are
// written are u = B e with (1 + A B) e = r (kda_delta.hip).  Instead of the
// inverse the kernel forms
//   X = (1 + A B)^-1 A,   e = r - X B r,
// strictly lower triangular: the identity's part of the inverse stays exact,
// and of the transposed system, which the backward pass solves,
// (1 + B A)^-1 = 1 - B X is as near.  It solves (1 + A B) X = A in fp32: the
// diagonal 16 x 16 blocks by substitution, D_a = (1 + A B)_aa^-1 = 1 - X_aa B_a,
// and block column b downwards, X_ab = D_a (A_ab - sum_{b<=c<a} A_ac B_c X_cb),
// on fp32 matrix cores, whose result tile is the next product's operand.
//
// Near HBM's rate: 96 heads x 8192 tokens take 86 us for 16.5 KiB read and 11.5 KiB
// written per 64 tokens and head, 4.1 TB/s, with five workgroups a compute unit (as
// LDS allows).  With the rows of A read all before the solve, 170 registers a wave,
// there were three, and 111 us; before that two, and 144.
#include <algorithm>

#include "kda.h"
#include "kda_delta_util.h"

namespace kda {
namespace {

template <typename E>
struct PrepLayout {
  static constexpr int ES = (int)sizeof(E);
  static constexpr int C = 128 / ES, NT = C / 16, TILES = delta_tiles(C);
  static constexpr int PITCH = 20;                              // floats of a tile row
  static constexpr int KT = 0;                                  // E [C][128]
  static constexpr int A = C * D * ES;                          // float [TILES][16][PITCH]
  static constexpr int SUM = A + TILES * 16 * PITCH * 4;        // float [2][C]
  static constexpr int ROW = SUM + 2 * C * 4;                   // float [C] e^{G_i}
  static constexpr int WGT = ROW + C * 4;                       // float [C] e^{G_C - G_j}
  static constexpr int BETA = WGT + C * 4;                      // float [C]
  static constexpr int BROW = BETA + C * 4;                     // float [C] beta e^{G_i}
  static constexpr int GAM = BROW + C * 4;                      // float e^{G_C} (and three of padding)
  static constexpr int BYTES = GAM + 16;
  static constexpr int THREADS = 64 * NT;
};

// One workgroup of C / 16 waves per (chunk, head): wave a forms and solves row
// tile a's diagonal block, then solves block column a.
template <typename E>
__global__ __launch_bounds__(PrepLayout<E>::THREADS, 4) void delta_prep_kernel(const DeltaPrepArgs p) {
  using L = PrepLayout<E>;
  constexpr int C = L::C, NT = L::NT, ES = L::ES, TILES = L::TILES;
  __shared__ __align__(1024) unsigned char smem[L::BYTES];
  static_assert(delta_matrix_bytes(C) <= C * D * ES, "the result fits the key tile's place");
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)smem;
  float* sA = reinterpret_cast<float*>(smem + L::A);
  float* sSum = reinterpret_cast<float*>(smem + L::SUM);
  float* sBeta = reinterpret_cast<float*>(smem + L::BETA);
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int H = p.num_heads;
  const int64_t u = p.unit0 + blockIdx.x;
  const int h = (int)(u % H);
  const int64_t slot = u / H;

  // the sequence: the last one whose first slot is not behind this one
  int n = 0;
  if (p.cu) {
    int hi = p.num_seqs - 1;
    while (n < hi) {
      const int mid = (n + hi + 1) >> 1;
      if (clamp_cu(p.cu, mid, p.total_tokens) / C + mid <= slot) n = mid;
      else hi = mid - 1;
    }
  }
  int64_t bos, eos;
  seq_range(p.cu, n, p.total_tokens, bos, eos);
  const int64_t j = slot - (bos / C + n);
  const int64_t t0 = bos + j * C;
  if (j < 0 || t0 >= eos) return;
  const int nv = (int)min((int64_t)C, eos - t0);

  {
    const uint32_t stride = (uint32_t)p.qk_heads * (D * ES);
    const Rsrc rs = make_rsrc(static_cast<const char*>(p.k) + (size_t)t0 * stride + (size_t)(h / (H / p.qk_heads)) * (D * ES),
                              (uint32_t)(nv - 1) * stride + D * ES);
    constexpr int UR = D * ES / 16, RP = 64 / UR;  // 16-byte units per row, rows per KiB
    constexpr int PIECES = C * D * ES / 1024 / NT;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int piece = wv * PIECES + i;
      const int row = piece * RP + lane / UR;
      const uint32_t unit = (uint32_t)(((lane % UR) ^ swizzle<E, D>(row)) * 16);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)(smem + piece * 1024), 16,
                                               (int)((uint32_t)row * stride + unit), 0, 0, 0);
    }
  }
  if (wv == 0) {
    const bool on = lane < nv;
    const size_t at = (size_t)(t0 + lane) * H + h;
    const float la = on ? p.log_decay[at] : 0.f, b = on ? p.beta[at] : 0.f;
    const double s = prefix_sum<C>((double)fmaxf(la, kMinLogDecay) * kLog2e, lane);
    if (lane < C) {
      const float hi = (float)s;
      sSum[lane] = hi;
      sSum[C + lane] = (float)(s - (double)hi);
      sBeta[lane] = b;
      const double tot = read_lane(s, C - 1);
      const float row = exp2_sum(s);
      reinterpret_cast<float*>(smem + L::ROW)[lane] = row;
      reinterpret_cast<float*>(smem + L::BROW)[lane] = b * row;
      reinterpret_cast<float*>(smem + L::WGT)[lane] = exp2_sum(tot - s);
      if (lane < 4) reinterpret_cast<float*>(smem + L::GAM)[lane] = exp2_sum(tot);
    }
  }
  __builtin_amdgcn_s_waitcnt(vmcnt_wait(0));
  __syncthreads();

  // A, row tile wv: rows 16 wv + 4 g + i, column 16 b + l16
  constexpr uint32_t TILE = 16 * L::PITCH * 4;
  auto a_tile = [&](int a, int b) { return sA + (size_t)tile_no(a, b) * (16 * L::PITCH); };
  {
    const uint32_t at = lds0 + tile_at<E, D>(l16, 8 * g);
    Frag<E> fi[4];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) ld_row(fi[ks], at + 16 * wv * (D * ES), 32 * ks);
    const f32x4 gi = *reinterpret_cast<const f32x4*>(sSum + 16 * wv + 4 * g);
    const f32x4 gi_lo = *reinterpret_cast<const f32x4*>(sSum + C + 16 * wv + 4 * g);
    for (int b = 0; b <= wv; ++b) {
      Frag<E> fj[4];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) ld_row(fj[ks], at + 16 * b * (D * ES), 32 * ks);
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) acc = mma(acc, fi[ks], fj[ks]);
      const float gj = sSum[16 * b + l16], gj_lo = sSum[C + 16 * b + l16];
      float* dst = a_tile(wv, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool on = b < wv || l16 < 4 * g + i;
        const float d = (gi[i] - gj) + (gi_lo[i] - gj_lo);
        const float x = acc[i] * exp2_fast(d);
        dst[(4 * g + i) * L::PITCH + l16] = on ? x : 0.f;
      }
    }
  }
  // (a wave's own writes are in order)
  {
    // diagonal block: column l16 of X, x_i = A_ij - sum_{j<m<i} A_im beta_m x_m
    float* a = a_tile(wv, wv);
    uint32_t at = as_is(lds0 + L::A + (uint32_t)tile_no(wv, wv) * TILE), col = as_is(at + 4 * l16);
    uint32_t beta = as_is(lds0 + L::BETA + 64 * wv);
    float x[16], z[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[i] = lds_get<float>(col + i * L::PITCH * 4);
#pragma unroll
      for (int m = 0; m < i; m += 4) {
        const f32x4 r = lds_get<f32x4>(at + (i * L::PITCH + m) * 4);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (m + q < i) x[i] -= r[q] * z[m + q];
      }
      z[i] = lds_get<float>(beta + 4 * i) * x[i];
      // (rows to come are not read before: registers)
      if (i == 7 || i == 11 || i == 13) asm volatile("" : "+v"(at), "+v"(col), "+v"(beta) : "v"(z[i]));
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (g == 0)
#pragma unroll
      for (int i = 0; i < 16; ++i) a[i * L::PITCH + l16] = x[i];
  }
  __syncthreads();

  // block column wv, downwards; res[a] = X_{a, wv}: rows 4 g + i, column l16
  f32x4 res[NT];
  const uint32_t own = as_is(lds0 + L::A + wv * TILE + (4 * g * L::PITCH + l16) * 4);
  const uint32_t rows = as_is(lds0 + L::A + (l16 * L::PITCH + 4 * g) * 4), beta = as_is(lds0 + L::BETA + 16 * g);
#pragma unroll
  for (int a = 0; a < NT; ++a) {
    if (a < wv) continue;
    f32x4 acc;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = lds_get<float>(own + tile_no(a, 0) * TILE + i * L::PITCH * 4);
    if (a > wv) {
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        if (c < wv || c >= a) continue;
        Frag16<float> f, x;
        f.v = -lds_get<f32x4>(beta + 64 * c) * lds_get<f32x4>(rows + tile_no(a, c) * TILE);
        x.v = res[c];
        acc = mma16(acc, f, x);
      }
      // D_a = 1 - X_aa B_a
      Frag16<float> f, x;
      f.v = -lds_get<f32x4>(beta + 64 * a) * lds_get<f32x4>(rows + tile_no(a, a) * TILE);
      x.v = acc;
      acc = mma16(acc, f, x);
    }
    res[a] = acc;
  }
  // -X in two terms (the key tile is read by no wave any more)
#pragma unroll
  for (int a = 0; a < NT; ++a) {
    if (a < wv) continue;
    _Float16* tile = reinterpret_cast<_Float16*>(smem + tile_no(a, wv) * kDeltaTileBytes);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = -res[a][i];
      const _Float16 t = (_Float16)x;
      const uint32_t at = tile16_at(4 * g + i, l16 >> 2) / 2 + (l16 & 3);
      tile[at] = t;
      tile[at + TILES * (kDeltaTileBytes / 2)] = (_Float16)(x - (float)t);
    }
  }
  __syncthreads();
  constexpr int BYTES = delta_matrix_bytes(C);
  char* dst = p.blocks + (size_t)u * delta_block_bytes(C);
  for (int i = tid; i < BYTES / 16; i += L::THREADS)
    reinterpret_cast<u32x4*>(dst)[i] = reinterpret_cast<const u32x4*>(smem)[i];
  for (int i = tid; i < 6 * C / 4 + 1; i += L::THREADS)
    reinterpret_cast<f32x4*>(dst + BYTES)[i] = reinterpret_cast<const f32x4*>(sSum)[i];
}

template <typename E>
hipError_t launch_prep_e(DeltaPrepArgs a, hipStream_t stream) {
  using L = PrepLayout<E>;
  const int64_t units = delta_chunk_slots(a.total_tokens, a.num_seqs, L::C) * a.num_heads;
  constexpr int64_t MOST = kMaxThreads / L::THREADS;
  for (int64_t u = 0; u < units; u += MOST) {
    a.unit0 = u;
    hipLaunchKernelGGL(delta_prep_kernel<E>, dim3((unsigned)std::min(units - u, MOST)), dim3(L::THREADS), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_delta_prep(DeltaPrepArgs a, hipStream_t stream) {
  return a.bf16 ? launch_prep_e<__bf16>(a, stream) : launch_prep_e<float>(a, stream);
}

}  // namespace kda
