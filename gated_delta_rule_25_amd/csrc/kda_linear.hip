// kda_linear.hip — linear attention with one decay per head, chunked form.
//
// Per (sequence, head), with a 128 x 128 state S (rows = key channels):
//   S_t = a_t S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t,   a_t = exp(log_decay_t) <= 1.
// Over a chunk of C tokens with incoming state S and G_i = sum_{j<=i} log a_j:
//   o_i = sum_{j<=i} e^{G_i - G_j} (q_i . k_j) v_j + e^{G_i} S^T q_i
//   S  <- e^{G_C} S + sum_j e^{G_C - G_j} k_j v_j^T
// Every exponent that is taken is <= 0, whatever the decays; -inf (the state
// is dropped) included.  The decay is one scalar per token and head, so it
// scales rows of the products and never enters them: q, k and v reach the
// matrix cores as they are, exact in bf16.
//
// Gradients.  With dS_t the gradient that reaches S_t,
//   dq_t = S_t do_t,   dk_t = dS_t v_t,   dv_t = dS_t^T k_t,
// which are the same walk with the tensors in other roles (LinearWalkArgs),
// the last two backwards in time.  For the decays, d/d log a_t is what of the
// loss flows through a_t S_{t-1}, and that changes from token to token by
//   D_t = D_{t+1} + r_t - c_t,  r_t = q_t . dq_t,  c_t = k_t . dk_t
// (each without the token's own q_t . k_t term, which cancels), and at any
// token boundary equals <S, dS>.  The sum over t is restarted from that
// product at every segment boundary, so rounding cannot build up along the
// sequence.
//
// What is rounded.  bf16: the pair matrix (q_i . k_j) e^{..} and the state,
// as operands of the outputs' products, to one bf16 each (the output is bf16
// itself: measured 2.3e-3 of its norm off the 64-bit result, against 1.7e-3 for
// the output's own rounding).  The state's update takes e^{..} v_j as the sum
// of three bf16 terms (24 bits), because the state is an fp32 result; the
// part of r_t and c_t that comes through the state takes three terms of the
// state for the same reason.  Accumulation is fp32, prefix sums of the decays
// are fp64 (a difference of two sums decides every factor).
#include <algorithm>
#include <atomic>

#include "kda.h"
#include "kda_chunk_util.h"
#include "kda_linear_internal.h"

namespace kda {
namespace {

constexpr double kLog2e = 1.4426950408889634;
// log decays below this are taken as this: e^-120 is below the smallest fp32
// number, and sums of it keep their differences exact enough.
constexpr float kMinLogDecay = -120.f;

__device__ __forceinline__ int64_t clamp_cu(const int32_t* cu, int n, int64_t T) {
  const int64_t c = cu[n];
  return c < 0 ? 0 : (c > T ? T : c);
}

struct Segment {
  int n;              // sequence
  int j;              // segment within it
  int count;          // segments of the sequence
  int64_t bos, eos;   // the sequence's tokens
  bool ok;
};

// The segment in a slot.  cu_seqlens outside its preconditions gives some
// slot assignment or other, always within the buffers.
__device__ __forceinline__ Segment find_segment(const int32_t* cu, int N, int64_t T, int seg, int64_t slot) {
  Segment s;
  int lo = 0;
  if (cu) {
    int hi = N - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (clamp_cu(cu, mid, T) / seg + 2 * (int64_t)mid <= slot) lo = mid;
      else hi = mid - 1;
    }
  }
  s.n = lo;
  seq_range(cu, lo, T, s.bos, s.eos);
  s.count = (int)((s.eos - s.bos + seg - 1) / seg);
  const int64_t j = slot - (s.bos / seg + 2 * (int64_t)lo);
  s.j = (int)j;
  // an empty sequence has one segment with no tokens
  s.ok = j >= 0 && j < (s.count > 0 ? s.count : 1);
  return s;
}

__device__ __forceinline__ int64_t slot_of(int n, int64_t bos, int seg, int64_t j) {
  return bos / seg + 2 * (int64_t)n + j;
}

// ---- LDS tiles ------------------------------------------------------------
// A tile holds C tokens x 128 channels, row-major, its 16-byte units XOR-ed
// with the row (mod 16) so that the 16 rows a matrix-core operand reads at
// one channel fall on different banks.
template <typename E>
__device__ __forceinline__ int tile_at(int row, int ch) {
  constexpr int U = 16 / (int)sizeof(E);  // elements per unit
  return row * D + (((ch / U) ^ (row & 15)) * U) + (ch % U);
}

// operand with the channels ch .. ch+7 of a row
__device__ __forceinline__ void ld_row(Frag<__bf16>& f, const __bf16* t, int row, int ch) {
  f.v = *reinterpret_cast<const bf16x8*>(t + tile_at<__bf16>(row, ch));
}
__device__ __forceinline__ void ld_row(Frag<float>& f, const float* t, int row, int ch) {
  f.lo = *reinterpret_cast<const f32x4*>(t + tile_at<float>(row, ch));
  f.hi = *reinterpret_cast<const f32x4*>(t + tile_at<float>(row, ch + 4));
}

// operand of column ch (one per lane of 16) over the rows row .. row+7.
// bf16: the transposing LDS read hands each lane of 16 one column of a
// 4-row x 16-channel block, whose rows the lanes 4r .. 4r+3 address.
__device__ __forceinline__ void ld_col(Frag<__bf16>& f, const __bf16* t, int row, int ch0, int l16) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  const int r = row + (l16 >> 2), c = ch0 + 4 * (l16 & 3);
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(t + tile_at<__bf16>(r, c)));
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(t + tile_at<__bf16>(r + 4, c)));
  const bf16x4 x = __builtin_bit_cast(bf16x4, a), y = __builtin_bit_cast(bf16x4, b);
  f.v = (bf16x8){x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
}
__device__ __forceinline__ void ld_col(Frag<float>& f, const float* t, int row, int ch0, int l16) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.lo[i] = t[tile_at<float>(row + i, ch0 + l16)];
    f.hi[i] = t[tile_at<float>(row + 4 + i, ch0 + l16)];
  }
}

__device__ __forceinline__ float frag_get(const Frag<__bf16>& f, int i) { return (float)f.v[i]; }
__device__ __forceinline__ float frag_get(const Frag<float>& f, int i) { return i < 4 ? f.lo[i] : f.hi[i - 4]; }

// The pair matrix in LDS: C rows of 128 bytes, 16-byte units XOR-ed with the row (mod 8).
template <typename E, int C>
__device__ __forceinline__ int pair_at(int row, int col) {
  constexpr int U = 16 / (int)sizeof(E);
  return row * C + (((col / U) ^ (row & 7)) * U) + (col % U);
}
template <int C>
__device__ __forceinline__ void ld_pair(Frag<__bf16>& f, const __bf16* t, int row, int col) {
  f.v = *reinterpret_cast<const bf16x8*>(t + pair_at<__bf16, C>(row, col));
}
template <int C>
__device__ __forceinline__ void ld_pair(Frag<float>& f, const float* t, int row, int col) {
  f.lo = *reinterpret_cast<const f32x4*>(t + pair_at<float, C>(row, col));
  f.hi = *reinterpret_cast<const f32x4*>(t + pair_at<float, C>(row, col + 4));
}

// x as the sum of NS operands (bf16: NS terms of 8 bits each; fp32: itself).
template <int NS>
__device__ __forceinline__ void split(Frag<__bf16> (&f)[NS], const float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float r = x[i];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const __bf16 b = (__bf16)r;
      f[s].v[i] = b;
      r -= (float)b;
    }
  }
}
template <int NS>
__device__ __forceinline__ void split(Frag<float> (&f)[NS], const float (&x)[8]) {
  static_assert(NS == 1, "fp32 operands are exact");
  frag_from_f32(f[0], x);
}

template <typename E, int NX>
struct WalkLayout {
  static constexpr int C = sizeof(E) == 2 ? 64 : 32;
  static constexpr int TILE = C * D * (int)sizeof(E);  // 16 KiB
  static constexpr int NTILE = 3 + NX;                 // query, key, value[, x]
  static constexpr int PAIR = 2 * NTILE * TILE;        // two chunks in flight
  static constexpr int SUM = PAIR + C * C * (int)sizeof(E);  // double [2][C] prefix sums (log2)
  static constexpr int ROW = SUM + 2 * C * 8;          // float [2][C] factor of the state in row t
  static constexpr int WGT = ROW + 2 * C * 4;          // float [2][C] factor of token t in the state
  static constexpr int GAM = WGT + 2 * C * 4;          // float [2]
  static constexpr int ANC = GAM + 16;                 // float [2][4] <S, dS> by wave
  static constexpr int RX = ANC + 32;                  // float [2][4][C] state part . x by wave
  static constexpr int RR = RX + (NX ? 2 * 4 * C * 4 : 0);  // float [2][4][C] pair sums of the keys by wave
  static constexpr int RC = RR + (NX ? 2 * 4 * C * 4 : 0);  // float [2][2][C] pair sums of the queries
  static constexpr int BYTES = RC + (NX ? 2 * 2 * C * 4 : 0);
};

// ---------------------------------------------------------------------------
// The walk.  Four compute waves and a loader wave per (sequence or segment,
// head, block of 64 CT value columns).  Compute wave w owns 16 CT value
// columns and keeps its [128 x 16 CT] slice of the state in matrix-core
// accumulators (fp32) over the whole walk; accumulators of two stacked tiles
// are an operand of the next product as they are.  Per chunk:
//   1. the pair matrix: wave w forms the products of one 16-query tile with
//      the keys up to it, scales them by e^{G_i - G_j} and leaves them in LDS;
//   2. outputs, transposed (rows = value columns), so that a lane stores four
//      consecutive columns: S^T q, scaled by e^{G_i}, plus the pair matrix
//      times v;
//   3. S <- e^{G_C} S + k^T (e^{G_C - G_j} v_j), v read once for 2 and 3.
// The loader wave copies the next chunk's tiles from global memory straight
// into the other half of LDS and forms the decays' prefix sums, so that the
// compute waves never wait behind a copy of their own.  Two barriers per chunk.
// REV walks backwards in time: the pair matrix is upper triangular and the
// factors of rows and of tokens change places.
// DG (the decays' gradient): x is q in the dq walk and k in the dk walk.
// ---------------------------------------------------------------------------
template <typename E, int CT, bool REV, bool TR, bool OUT, bool DG>
__global__ __launch_bounds__(320) void linear_walk_kernel(const LinearWalkArgs p) {
  using L = WalkLayout<E, DG ? 1 : 0>;
  constexpr int C = L::C, NT = C / 16, KT = C / 32, ES = (int)sizeof(E);
  constexpr bool BF = ES == 2;
  constexpr int NSV = BF ? 3 : 1;              // terms of the weighted values
  constexpr int NSS = (BF && DG) ? 3 : 1;      // terms of the state in the outputs' product
  constexpr bool DK = DG && REV;               // dk walk: forms the decays' gradient
  static_assert(L::BYTES <= 160 * 1024, "LDS budget exceeded");
  extern __shared__ __align__(16) unsigned char smem[];
  double* sSum = reinterpret_cast<double*>(smem + L::SUM);
  float* sRow = reinterpret_cast<float*>(smem + L::ROW);
  float* sWgt = reinterpret_cast<float*>(smem + L::WGT);
  float* sGam = reinterpret_cast<float*>(smem + L::GAM);
  float* sAnc = reinterpret_cast<float*>(smem + L::ANC);
  float* sRX = reinterpret_cast<float*>(smem + L::RX);
  float* sRR = reinterpret_cast<float*>(smem + L::RR);
  float* sRC = reinterpret_cast<float*>(smem + L::RC);
  E* sP = reinterpret_cast<E*>(smem + L::PAIR);

  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, l16 = lane & 15, g = lane >> 4;
  constexpr int CB = 2 / CT;  // column blocks of a head
  // blocks b and b + 8 run on the same XCD: a head's column blocks share its L2
  const int64_t slot8 = blockIdx.x >> 3;
  const int cb = (int)(slot8 % CB);
  const int64_t u = (slot8 / CB) * 8 + (blockIdx.x & 7);
  if (u >= p.units) return;
  const int H = p.num_heads;
  const int h = (int)(u % H);
  const int64_t rank = u / H;
  // tokens [tb, te) of sequence n = tokens [bos, eos)
  int n;
  int64_t bos, eos, tb, te, slot;
  bool first, last;  // the item begins / ends its sequence
  if (p.segmented) {
    const Segment s = find_segment(p.cu, p.num_seqs, p.total_tokens, p.seg, rank);
    if (!s.ok) {
      if constexpr (DK)
        if (p.d_decay_part && tid == 0) p.d_decay_part[u] = 0.0;
      return;
    }
    n = s.n;
    bos = s.bos;
    eos = s.eos;
    slot = rank;
    tb = bos + (int64_t)s.j * p.seg;
    te = min(eos, tb + p.seg);
    first = s.j == 0;
    last = s.j + 1 >= s.count;
    if constexpr (!OUT)
      if (REV ? first : last) return;  // no segment follows that would read it
  } else {
    n = (int)rank;
    seq_range(p.cu, n, p.total_tokens, bos, eos);
    slot = slot_of(n, bos, p.seg, 0);
    tb = bos;
    te = eos;
    first = last = true;
  }
  const int nch = (int)((te - tb + C - 1) / C);
  const size_t nh = (size_t)n * H + h;
  auto chunk_of = [&](int ci) { return REV ? nch - 1 - ci : ci; };

  if (wv == 4) {
    // ---- loader wave ----
    auto copy_tile = [&](const void* src, int heads, int64_t t0, int nv, unsigned char* dst) {
      const int hh = h / (H / heads);
      const char* base = static_cast<const char*>(src) + ((size_t)t0 * heads + hh) * (D * ES);
      const size_t stride = (size_t)heads * (D * ES);
      constexpr int RP = 1024 / (D * ES);  // rows per 1 KiB piece
      constexpr int UR = 64 / RP;          // 16-byte units per row
#pragma unroll
      for (int i = 0; i < L::TILE / 1024; ++i) {
        const int row = i * RP + lane / UR;
        const int unit = (lane % UR) ^ (row & 15);
        // rows behind the end repeat the last one: their factors are zero
        const char* s = base + (size_t)min(row, nv - 1) * stride + unit * 16;
        __builtin_amdgcn_global_load_lds(s, (__attribute__((address_space(3))) void*)(dst + i * 1024), 16, 0, 0);
      }
    };
    auto copy_chunk = [&](int ci) {
      const int64_t t0 = tb + (int64_t)chunk_of(ci) * C;
      const int nv = (int)min((int64_t)C, te - t0);
      unsigned char* dst = smem + (ci & 1) * (L::NTILE * L::TILE);
      if (OUT) copy_tile(p.q, p.q_heads, t0, nv, dst);
      copy_tile(p.k, p.k_heads, t0, nv, dst + L::TILE);
      copy_tile(p.v, p.v_heads, t0, nv, dst + 2 * L::TILE);
      if constexpr (DG) copy_tile(p.x, p.x_heads, t0, nv, dst + 3 * L::TILE);
    };
    auto load_decay = [&](int ci) -> float {
      const int64_t t = tb + (int64_t)chunk_of(ci) * C + lane;
      if (lane >= C || t >= te) return 0.f;
      return p.decay_per_head ? p.log_decay[h] : p.log_decay[(size_t)t * H + h];
    };
    double log_total = 0.0;
    auto put_decay = [&](int ci, float la) {
      const int64_t t = tb + (int64_t)chunk_of(ci) * C + lane;
      double s = (double)fmaxf(la, kMinLogDecay) * kLog2e;
#pragma unroll
      for (int m = 1; m < C; m <<= 1) {
        const double o = __shfl_up(s, m);
        if (lane >= m) s += o;
      }
      const double tot = __shfl(s, C - 1);
      log_total += tot;
      const float head = exp2_fast((float)s), tail = exp2_fast((float)(tot - s));
      if (lane < C) {
        const int b = (ci & 1) * C + lane;
        sSum[b] = s;
        sRow[b] = REV ? tail : head;
        sWgt[b] = t < te ? (REV ? head : tail) : 0.f;
      }
      if (lane == 0) sGam[ci & 1] = exp2_fast((float)tot);
    };
    // the decays' gradient of chunk ci from the compute waves' sums
    double flow = 0.0;   // D behind the chunk
    double dsum = 0.0;
    auto finish = [&](int ci, float rdot) {
      if constexpr (DG) {
        const int64_t t0 = tb + (int64_t)chunk_of(ci) * C;
        const bool in = lane < C && t0 + lane < te;
        const int b = ci & 1;
        float part = 0.f;
        if (lane < C)
#pragma unroll
          for (int w = 0; w < 4; ++w) part += sRX[(b * 4 + w) * C + lane];
        if constexpr (!REV) {
          if (in) p.row_dot[(size_t)(t0 + lane) * H + h] = part;
        } else {
          float keys = 0.f, queries = 0.f;
          if (lane < C) {
#pragma unroll
            for (int w = 0; w < 4; ++w) keys += sRR[(b * 4 + w) * C + lane];
            queries = sRC[(b * 2 + 0) * C + lane] + (NT == 2 ? sRC[(b * 2 + 1) * C + lane] : 0.f);
          }
          const int64_t tend = min(te, t0 + C);
          if (tend == te || (tend - bos) % p.seg == 0)
            flow = (double)sAnc[b * 4] + (double)sAnc[b * 4 + 1] + (double)sAnc[b * 4 + 2] + (double)sAnc[b * 4 + 3];
          double s = in ? ((double)rdot + (double)keys) - ((double)part + (double)queries) : 0.0;
#pragma unroll
          for (int m = 1; m < C; m <<= 1) {
            const double o = __shfl_down(s, m);
            if (lane + m < C) s += o;
          }
          const double d = flow + s;
          if (in) {
            if (p.d_log_decay) p.d_log_decay[(size_t)(t0 + lane) * H + h] = (float)d;
            dsum += d;
          }
          flow += __shfl(s, 0);
        }
      }
    };
    auto load_rdot = [&](int ci) -> float {
      if constexpr (DK) {
        const int64_t t = tb + (int64_t)chunk_of(ci) * C + lane;
        if (lane < C && t < te) return p.row_dot[(size_t)t * H + h];
      }
      return 0.f;
    };
    if (nch > 0) {
      put_decay(0, load_decay(0));
      copy_chunk(0);
    }
    float la_next = nch > 1 ? load_decay(1) : 0.f;
    float rdot_cur = 0.f;
    for (int ci = 0; ci < nch; ++ci) {
      __builtin_amdgcn_s_waitcnt(vmcnt_wait(0));
      __syncthreads();  // chunk ci is in LDS; every wave is done with chunk ci - 1
      const float la = la_next;
      const float rdot_prev = rdot_cur;
      if (ci + 2 < nch) la_next = load_decay(ci + 2);
      rdot_cur = load_rdot(ci);
      if (ci + 1 < nch) {
        copy_chunk(ci + 1);
        put_decay(ci + 1, la);
      }
      if (ci > 0) finish(ci - 1, rdot_prev);
      if (OUT) __syncthreads();  // the pair matrix
    }
    if constexpr (DG) {
      __syncthreads();
      if (nch > 0) finish(nch - 1, rdot_cur);
      if constexpr (REV) {
        if (p.d_decay_part) {
#pragma unroll
          for (int m = 32; m >= 1; m >>= 1) dsum += __shfl_xor(dsum, m);
          if (lane == 0) p.d_decay_part[u] = dsum;
        }
      }
    }
    if (!OUT && lane == 0 && cb == 0) p.seg_decay[(size_t)slot * H + h] = exp2_fast((float)log_total);
    return;
  }

  // ---- compute waves ----
  const int col0 = cb * (64 * CT) + 16 * CT * wv;
  // state element (row, column) of this walk in a stored state
  auto state_at = [&](int row, int col) { return TR ? col * D + row : row * D + col; };
  auto load_state = [&](const float* src, f32x4 (&s)[CT][8]) {
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int rt = 0; rt < 8; ++rt) {
        const int row = 16 * rt + 4 * g, col = col0 + 16 * c + l16;
        if constexpr (TR) {
          s[c][rt] = *reinterpret_cast<const f32x4*>(src + state_at(row, col));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) s[c][rt][i] = src[state_at(row + i, col)];
        }
      }
  };
  auto store_state = [&](float* dst, const f32x4 (&s)[CT][8]) {
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int rt = 0; rt < 8; ++rt) {
        const int row = 16 * rt + 4 * g, col = col0 + 16 * c + l16;
        if constexpr (TR) {
          *reinterpret_cast<f32x4*>(dst + state_at(row, col)) = s[c][rt];
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) dst[state_at(row + i, col)] = s[c][rt][i];
        }
      }
  };
  constexpr size_t kState = (size_t)D * D;
  f32x4 accS[CT][8];
  {
    const float* src = nullptr;
    if (OUT) {
      // segmented: the scan has put the incoming state of every segment in its
      // slot, the first one's too, as `fin` may be `init`
      if (p.segmented && nch > 0) src = p.snap + ((size_t)slot * H + h) * kState;
      else if (p.init) src = p.init + nh * kState;
    }
    if (src) {
      load_state(src, accS);
    } else {
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int rt = 0; rt < 8; ++rt) accS[c][rt] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }
  }

  for (int ci = 0; ci < nch; ++ci) {
    const int64_t t0 = tb + (int64_t)chunk_of(ci) * C;
    const int nv = (int)min((int64_t)C, te - t0);
    const unsigned char* buf = smem + (ci & 1) * (L::NTILE * L::TILE);
    const E* sQ = reinterpret_cast<const E*>(buf);
    const E* sK = reinterpret_cast<const E*>(buf + L::TILE);
    const E* sV = reinterpret_cast<const E*>(buf + 2 * L::TILE);
    const E* sX = reinterpret_cast<const E*>(buf + 3 * L::TILE);
    const int b = ci & 1;

    // what the decays' gradient needs of the states at segment boundaries
    if constexpr (DG && !REV) {
      if (!p.segmented && (t0 - bos) % p.seg == 0)
        store_state(p.fwd_snap + ((size_t)(slot + (t0 - bos) / p.seg) * H + h) * kState, accS);
    }
    if constexpr (DK) {
      const int64_t tend = t0 + nv;
      if (tend == te || (tend - bos) % p.seg == 0) {
        const int64_t sl = slot_of(n, bos, p.seg, (tend - bos + p.seg - 1) / p.seg);
        const float* src = p.fwd_snap + ((size_t)sl * H + h) * kState;
        float dot = 0.f;
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
          for (int rt = 0; rt < 8; ++rt) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(src + state_at(16 * rt + 4 * g, col0 + 16 * c + l16));
#pragma unroll
            for (int i = 0; i < 4; ++i) dot += x[i] * accS[c][rt][i];
          }
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1) dot += __shfl_xor(dot, m);
        if (lane == 0) sAnc[b * 4 + wv] = dot;
      }
    }
    __syncthreads();  // chunk ci is in LDS

    const double* gs = sSum + b * C;
    if constexpr (OUT) {
      // ---- 1: pair matrix, keys in rows: lane = query, four consecutive keys ----
      const int rt = NT == 4 ? wv : wv >> 1;
      Frag<E> fq[4];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) ld_row(fq[ks], sQ, 16 * rt + l16, 32 * ks + 8 * g);
      Frag<E> fx[DK ? 4 : 1];
      if constexpr (DK)
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) ld_row(fx[ks], sX, 16 * rt + l16, 32 * ks + 8 * g);
      const int q = 16 * rt + l16;
      const double gq = gs[q];
      float csum = 0.f;
#pragma unroll
      for (int kk = 0; kk < (NT == 4 ? NT : 1); ++kk) {
        const int kt = NT == 4 ? kk : (wv & 1);
        // tiles beyond the triangle that share a 32-deep step with it are zero
        const bool tri = REV ? kt >= rt : kt <= rt;
        const bool use = REV ? kt >= (rt & ~1) : kt <= (rt | 1);
        f32x4 rsum = {0.f, 0.f, 0.f, 0.f};
        if (use) {
          f32x4 acc = {0.f, 0.f, 0.f, 0.f};
          if (tri) {
            f32x4 acc2 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
              Frag<E> fk;
              ld_row(fk, sK, 16 * kt + l16, 32 * ks + 8 * g);
              acc = mma(acc, fk, fq[ks]);
            }
            if constexpr (DK)
#pragma unroll
              for (int ks = 0; ks < 4; ++ks) {
                Frag<E> fv;
                ld_row(fv, sV, 16 * kt + l16, 32 * ks + 8 * g);
                acc2 = mma(acc2, fv, fx[ks]);
              }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int k = 16 * kt + 4 * g + i;
              const bool on = REV ? (k >= q && k < nv) : k <= q;
              const double gd = REV ? gs[k] - gq : gq - gs[k];
              const float x = on ? acc[i] * exp2_fast((float)gd) : 0.f;
              if constexpr (DK) {
                const float f = (on && k != q) ? x * acc2[i] : 0.f;
                rsum[i] = f;
                csum += f;
              }
              acc[i] = x;
            }
          }
          store_row4(sP + pair_at<E, C>(q, 16 * kt + 4 * g), acc);
        }
        if constexpr (DK) {
          // over the 16 queries of the tile
#pragma unroll
          for (int m = 8; m >= 1; m >>= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) rsum[i] += __shfl_xor(rsum[i], m);
          if (l16 == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) sRR[(b * 4 + wv) * C + 16 * kt + 4 * g + i] = rsum[i];
          }
        }
      }
      if constexpr (DK) {
        csum += __shfl_xor(csum, 16);
        csum += __shfl_xor(csum, 32);
        if (g == 0) sRC[(b * 2 + (NT == 2 ? (wv & 1) : 0)) * C + q] = csum;
        if constexpr (NT == 2) {
          // the key tile this wave has no products with
          if (lane < 16) sRR[(b * 4 + wv) * C + 16 * (1 - (wv & 1)) + lane] = 0.f;
        }
      }
      __syncthreads();  // pair matrix
    }

    // ---- 2: outputs (transposed: lane = token, four consecutive value columns) ----
    Frag<E> fv[CT][KT];
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) ld_col(fv[c][kt], sV, 32 * kt + 8 * g, col0 + 16 * c, l16);
    if constexpr (OUT) {
      f32x4 accO[CT][NT];
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int rt = 0; rt < NT; ++rt) accO[c][rt] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        Frag<E> fs[CT][NSS];
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          float x[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = accS[c][2 * ks][i];
            x[4 + i] = accS[c][2 * ks + 1][i];
          }
          split<NSS>(fs[c], x);
        }
#pragma unroll
        for (int rt = 0; rt < NT; ++rt) {
          Frag<E> fq;
          ld_frag_pair(fq, sQ + tile_at<E>(16 * rt + l16, 32 * ks + 4 * g),
                       sQ + tile_at<E>(16 * rt + l16, 32 * ks + 16 + 4 * g));
#pragma unroll
          for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int s = 0; s < NSS; ++s) accO[c][rt] = mma(accO[c][rt], fs[c][s], fq);
        }
      }
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) {
        const float f = sRow[b * C + 16 * rt + l16];
        float dot = 0.f;
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          accO[c][rt] *= f;
          if constexpr (DG) {
            Frag16<E> fx;
            ld_frag16(fx, sX + tile_at<E>(16 * rt + l16, col0 + 16 * c + 4 * g));
            const f32x4 x = frag16_to_f32(fx);
#pragma unroll
            for (int i = 0; i < 4; ++i) dot += x[i] * accO[c][rt][i];
          }
        }
        if constexpr (DG) {
          dot += __shfl_xor(dot, 16);
          dot += __shfl_xor(dot, 32);
          if (g == 0) sRX[(b * 4 + wv) * C + 16 * rt + l16] = dot;
        }
      }
#pragma unroll
      for (int rt = 0; rt < NT; ++rt)
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
          if (REV ? kt < rt / 2 : kt > rt / 2) continue;
          Frag<E> fp;
          ld_pair<C>(fp, sP, 16 * rt + l16, 32 * kt + 8 * g);
#pragma unroll
          for (int c = 0; c < CT; ++c) accO[c][rt] = mma(accO[c][rt], fv[c][kt], fp);
        }
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) {
        if (16 * rt + l16 >= nv) continue;
        const size_t at = ((size_t)(t0 + 16 * rt + l16) * H + h) * D + col0 + 4 * g;
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          if (p.o_f32) store_row4(static_cast<float*>(p.o) + at + 16 * c, accO[c][rt]);
          else store_row4(static_cast<E*>(p.o) + at + 16 * c, accO[c][rt]);
        }
      }
    }

    // ---- 3: state ----
    const float gam = sGam[b];
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int rt = 0; rt < 8; ++rt) accS[c][rt] *= gam;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      const f32x4 w0 = *reinterpret_cast<const f32x4*>(sWgt + b * C + 32 * kt + 8 * g);
      const f32x4 w1 = *reinterpret_cast<const f32x4*>(sWgt + b * C + 32 * kt + 8 * g + 4);
      Frag<E> fw[CT][NSV];
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = frag_get(fv[c][kt], i) * (i < 4 ? w0[i & 3] : w1[i & 3]);
        split<NSV>(fw[c], x);
      }
#pragma unroll
      for (int rt = 0; rt < 8; ++rt) {
        Frag<E> fk;
        ld_col(fk, sK, 32 * kt + 8 * g, 16 * rt, l16);
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
          for (int s = 0; s < NSV; ++s) accS[c][rt] = mma(accS[c][rt], fk, fw[c][s]);
      }
    }
  }
  if constexpr (DG) __syncthreads();  // the last chunk's sums
  if (OUT) {
    if (p.fin && (REV ? first : last)) store_state(p.fin + nh * kState, accS);
    if constexpr (DG && !REV)
      if (last && nch > 0)
        store_state(p.fwd_snap + ((size_t)slot_of(n, bos, p.seg, (eos - bos + p.seg - 1) / p.seg) * H + h) * kState, accS);
  } else {
    store_state(p.snap + ((size_t)slot * H + h) * kState, accS);
  }
}

template <typename E, int CT, bool REV, bool TR, bool OUT, bool DG>
hipError_t launch_walk_t(const LinearWalkArgs& a, hipStream_t stream) {
  using L = WalkLayout<E, DG ? 1 : 0>;
  constexpr int CB = 2 / CT;
  const int64_t blocks = (a.units + 7) / 8 * 8 * CB;
  static std::atomic<bool> set[64];
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= 64 || !set[dev].load(std::memory_order_relaxed)) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(linear_walk_kernel<E, CT, REV, TR, OUT, DG>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
    if (e != hipSuccess) return e;
    if (dev >= 0 && dev < 64) set[dev].store(true, std::memory_order_relaxed);
  }
  hipLaunchKernelGGL((linear_walk_kernel<E, CT, REV, TR, OUT, DG>), dim3((unsigned)blocks), dim3(320), L::BYTES, stream, a);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_walk_e(const LinearWalkArgs& a, hipStream_t stream) {
  if (!a.write_o)
    return a.reverse ? launch_walk_t<E, 2, true, false, false, false>(a, stream)
                     : launch_walk_t<E, 2, false, false, false, false>(a, stream);
  if (a.transposed) {
    if (a.reverse)
      return a.with_decay_grad ? launch_walk_t<E, 2, true, true, true, true>(a, stream)
                               : launch_walk_t<E, 2, true, true, true, false>(a, stream);
    return a.with_decay_grad ? launch_walk_t<E, 2, false, true, true, true>(a, stream)
                             : launch_walk_t<E, 2, false, true, true, false>(a, stream);
  }
  if (a.reverse) return launch_walk_t<E, 2, true, false, true, false>(a, stream);
  return a.narrow ? launch_walk_t<E, 1, false, false, true, false>(a, stream)
                  : launch_walk_t<E, 2, false, false, true, false>(a, stream);
}

// ---------------------------------------------------------------------------
// Incoming state of every segment: the segments' contributions composed in
// order, elementwise (the decay of a segment is one scalar).  A thread owns
// four elements of one (sequence, head)'s state and reads the next segment's
// contribution while it composes this one.
// ---------------------------------------------------------------------------
template <bool REV>
__global__ __launch_bounds__(256) void linear_scan_kernel(const LinearScanArgs a) {
  constexpr size_t kState = (size_t)D * D;
  const int H = a.num_heads;
  const int64_t nh = blockIdx.x >> 4;
  const int at = ((int)(blockIdx.x & 15) * 256 + threadIdx.x) * 4;
  const int n = (int)(nh / H), h = (int)(nh % H);
  int64_t bos, eos;
  seq_range(a.cu, n, a.total_tokens, bos, eos);
  const int count = (int)((eos - bos + a.seg - 1) / a.seg);
  const int64_t base = slot_of(n, bos, a.seg, 0);
  auto where = [&](int j) { return ((size_t)(base + (REV ? count - 1 - j : j)) * H + h); };
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (a.init) s = *reinterpret_cast<const f32x4*>(a.init + (size_t)nh * kState + at);
  f32x4 next = {0.f, 0.f, 0.f, 0.f};
  float dec = 0.f;
  if (count > 1) {
    next = *reinterpret_cast<const f32x4*>(a.snap + where(0) * kState + at);
    dec = a.seg_decay[where(0)];
  }
  for (int j = 0; j < count; ++j) {
    const f32x4 add = next;
    const float d = dec;
    if (j + 2 < count) {  // the last segment's own contribution is not needed
      next = *reinterpret_cast<const f32x4*>(a.snap + where(j + 1) * kState + at);
      dec = a.seg_decay[where(j + 1)];
    }
    *reinterpret_cast<f32x4*>(a.snap + where(j) * kState + at) = s;
    s = s * d + add;
  }
}

// ---------------------------------------------------------------------------
// Gradients of shared query and key heads: the sum over the value heads that
// share one, in order.  Four consecutive channels per thread.
// ---------------------------------------------------------------------------
template <typename E>
__global__ __launch_bounds__(256) void linear_share_sum_kernel(const float* __restrict__ src, E* __restrict__ dst,
                                                               int64_t rows, int share) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = i >> 5;
  const int ch = (int)(i & 31) * 4;
  if (row >= rows) return;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < share; ++j) s += *reinterpret_cast<const f32x4*>(src + (row * share + j) * D + ch);
  store_row4(dst + row * D + ch, s);
}

__global__ __launch_bounds__(64) void linear_decay_sum_kernel(const double* __restrict__ part, float* __restrict__ dst,
                                                              int64_t units, int H) {
  const int h = blockIdx.x;
  double s = 0.0;
  for (int64_t u = h + (int64_t)threadIdx.x * H; u < units; u += (int64_t)64 * H) s += part[u];
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) s += __shfl_xor(s, m);
  if (threadIdx.x == 0) dst[h] = (float)s;
}

}  // namespace

hipError_t launch_linear_walk(const LinearWalkArgs& a, hipStream_t stream) {
  return a.bf16 ? launch_walk_e<__bf16>(a, stream) : launch_walk_e<float>(a, stream);
}

hipError_t launch_linear_scan(const LinearScanArgs& a, hipStream_t stream) {
  const int64_t blocks = (int64_t)a.num_seqs * a.num_heads * 16;
  if (a.reverse)
    hipLaunchKernelGGL(linear_scan_kernel<true>, dim3((unsigned)blocks), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL(linear_scan_kernel<false>, dim3((unsigned)blocks), dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_linear_share_sum(const float* src, void* dst, int64_t rows, int share, bool bf16,
                                   hipStream_t stream) {
  const int64_t blocks = (rows * 32 + 255) / 256;
  if (blocks == 0) return hipSuccess;
  if (bf16)
    hipLaunchKernelGGL(linear_share_sum_kernel<__bf16>, dim3((unsigned)blocks), dim3(256), 0, stream, src,
                       static_cast<__bf16*>(dst), rows, share);
  else
    hipLaunchKernelGGL(linear_share_sum_kernel<float>, dim3((unsigned)blocks), dim3(256), 0, stream, src,
                       static_cast<float*>(dst), rows, share);
  return hipGetLastError();
}

hipError_t launch_linear_decay_sum(const double* part, float* dst, int64_t units, int num_heads, hipStream_t stream) {
  hipLaunchKernelGGL(linear_decay_sum_kernel, dim3((unsigned)num_heads), dim3(64), 0, stream, part, dst, units,
                     num_heads);
  return hipGetLastError();
}

}  // namespace kda
