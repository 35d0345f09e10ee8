// kda_delta_bwd.hip — gradients of the gated delta rule with one decay per head.
//
// With the notation of kda_delta.hip, f_i = e^{G_i}, w_j = e^{G_C - G_j},
// Gam_ij = e^{G_i - G_j}, e = u / beta (as it is computed, not divided for), and
// per chunk the state S that enters it and the gradient dS' that reaches its end:
//   du = P^T do + w k dS',   P_ij = (q_i . k_j) Gam_ij (j <= i)
//   y = (1 + B A)^-T du = du - X^T (B du),   dv = B y,   dbeta = e . y
//   dS = e^{G_C} dS' + (f q)^T do - (f k)^T dv
// which does not depend on the forward states.  The rest is per chunk:
//   dq_i = f_i S do_i + sum_{j<=i} (do_i . u_j) Gam_ij k_j
//   dk_j = w_j dS' u_j - f_j S dv_j + sum_{i>=j} (do_i . u_j) Gam_ij q_i
//          - sum_{i<j} (dv_j . u_i) Gam_ji k_i - sum_{i>j} (dv_i . u_j) Gam_ij k_i
// For the decays, d/d log a_t is what of the loss flows through S~_t, and that
// changes from token to token by
//   D_t = D_{t+1} + o_t . do_t - v_t . dv_t,
// and behind any token equals <S, dS>: the sum is restarted from that at every
// boundary of `anchor` tokens, so that rounding cannot build up.
//
// Steps: the prep kernel; the forward walk that leaves S, u and e of every
// chunk and o . do (delta_save_kernel); the walk back (delta_back_kernel), which
// writes dv, y, dS' of every chunk, v . dv and the terms of dbeta; the chunks'
// gradients, token-parallel (delta_grad_h_kernel, delta_grad_f_kernel); and the
// sums over the value columns and the tokens (linear_finish_kernel,
// delta_beta_kernel).  96 heads x 8192 tokens in bf16 take 86 + 556 + 630 + 424 +
// 81 + 10 us.
//
// What is rounded.  dv before it is rounded to its type, d_initial_state, dbeta
// and the decays' gradient are formed from products of 22 bits, as the forward
// states are.  For bf16 inputs, dq and dk take S, dS', u and y rounded to fp16 as
// operands, which are written and read again at half the bytes of fp32, and pairs
// of two bf16 terms.  With independent keys they are off by their own rounding only
// (1.68e-3 in norm for 1.66e-3; with bf16 operands and pairs 2.9e-3).  Where a chunk's
// keys are nearly the same each u replaces what the ones before left, and the
// roundings of all of them add up: at most 1.97e-3 and 1.81e-3 (the same key 2048
// times, beta 0.9, decays of 0.98 and 1).  In fp32 the products are fp32.
#include <type_traits>

#include "kda.h"
#include "kda_delta_walk.h"

namespace kda {
namespace {

// Sum over the 16 lanes of a row of sixteen values at once: lane l gets that of
// value l.  (The lanes are paired by exchanging 15, 7, 2 and 1 in their number.)
template <int N>
__device__ __forceinline__ float sum_rows(float (&x)[N], int l16) {
  if constexpr (N == 16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[i] + dpp_move_f32<0x140>(x[i]), b = x[i + 8] + dpp_move_f32<0x140>(x[i + 8]);
      x[i] = l16 & 8 ? b : a;
    }
  } else {
    // (eight values: both halves of the row get the same ones)
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] += dpp_move_f32<0x140>(x[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = x[i] + dpp_move_f32<0x141>(x[i]), b = x[i + 4] + dpp_move_f32<0x141>(x[i + 4]);
    x[i] = l16 & 4 ? b : a;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float a = x[i] + dpp_move_f32<0x4e>(x[i]), b = x[i + 2] + dpp_move_f32<0x4e>(x[i + 2]);
    x[i] = l16 & 2 ? b : a;
  }
  const float a = x[0] + dpp_move_f32<0xb1>(x[0]), b = x[1] + dpp_move_f32<0xb1>(x[1]);
  return l16 & 1 ? b : a;
}

// ---------------------------------------------------------------------------
// The walk back, in the roles of the forward one; values: d_o.  Bound as that is:
// 96 heads x 8192 tokens, bf16: 630 us, 10600 cycles a chunk, matrix cores 23 % busy,
// vector issue 48 %; without the stores of dS' 20 us less.
// BACK_STATES: what a segment adds to the gradient that reaches its first token.
// ---------------------------------------------------------------------------
template <typename E, Walk W>
__device__ __forceinline__ void delta_back(const DeltaBackArgs& p, unsigned char* smem, int64_t u, int cb) {
  constexpr int IT = Num<E>::IT, NS = 2, PT = 2;
  constexpr bool OUT = W == Walk::BACK;
  using L = DeltaLayout<E, PT>;
  constexpr int C = L::C, NT = L::NT, ES = L::ES;
  constexpr int KS = C / 32;
  static_assert(L::BYTES <= 160 * 1024, "LDS budget exceeded");
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)smem;
  int* sCol = reinterpret_cast<int*>(smem + L::COL);

  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int H = p.num_heads;
  const Item it = find_item<C>(p, smem, u);
  if (!it.ok) return;
  if constexpr (!OUT)
    if (it.first) return;  // nothing reads it
  const Chunks<C, true> ch{it};
  const int h = it.h, hq = h / (H / p.qk_heads), nch = it.nch;
  const size_t nh = (size_t)it.n * H + h;

  if (wv >= 4) {
    const HelperArgs ha{p.q, p.k, p.d_o, p.blocks, H, p.qk_heads, hq, cb, false};
    return prepare_chunks<E, L, PT, W>(it, smem, ha, wv - 4);
  }

  // ---- compute ----
  __builtin_amdgcn_s_setprio(2);
  const int vc0 = 16 * wv;
  const int col0 = cb * kVW + vc0;
  constexpr size_t kState = (size_t)D * D;
  f32x4 accS[8];
  int col_exp = 0;
  bool moved = false;  // col_exp, since it was last noted in LDS
  {
    const float* src = nullptr;
    if (OUT) {
      if (p.segmented && nch > 0) src = p.rstates + ((size_t)it.slot * H + h) * kState;
      else if (p.d_final) src = p.d_final + nh * kState;
    }
#pragma unroll
    for (int rt = 0; rt < 8; ++rt)
#pragma unroll
      for (int i = 0; i < 4; ++i) accS[rt][i] = src ? src[(16 * rt + 4 * g + i) * D + col0 + l16] : 0.f;
  }
  const uint32_t q_at = tile_at<__bf16, D>(l16, 4 * g);
  const uint32_t k_at = tile_at<__bf16, D>(4 * g + (l16 >> 2), 4 * (l16 & 3));
  const uint32_t t_at = tile16_at(4 * g + (l16 >> 2), l16 & 3);
  const uint32_t o_row = (uint32_t)H * (D * ES);
  const uint32_t o_at = (uint32_t)l16 * o_row + (uint32_t)((col0 + 4 * g) * ES);
  f16x8 ident[2];
  ident[0] = identity_h(0, l16, g);
  ident[1] = identity_h(1, l16, g);
  const int ct = cb * 4 + wv;  // column tile
  // v's rows in the layout of the stores of dv, and e, from memory a chunk ahead
  using Raw = std::conditional_t<ES == 2, u32x2, f32x4>;
  Raw v[OUT ? NT : 1];
  f32x4 e[OUT ? NT : 1];
  auto load_next = [&](int ci) {
    if constexpr (OUT) {
      const Rsrc rs = chunk_rows<E>(p.v, H, h, ch, ci, D * ES);
      const Rsrc re = make_rsrc(p.e + (((size_t)(ci < nch ? ch.slot(ci) : 0) * H + h) * 8 + cb * 4 + wv) * (NT * 256),
                                ci < nch ? NT * 1024 : 0);
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) {
        const int off = (int)(o_at + 16 * rt * o_row);
        if constexpr (ES == 2) v[rt] = __builtin_amdgcn_raw_buffer_load_b64(rs, off, 0, 0);
        else v[rt] = __builtin_bit_cast(f32x4, buf_ld16(rs, (uint32_t)off, 0));
        e[rt] = __builtin_bit_cast(f32x4, buf_ld16(re, (uint32_t)(rt * 1024 + lane * 16), 0));
      }
    }
  };
  load_next(0);
  if (g == 0) sCol[wv * 16 + l16] = 0;
  auto store_state = [&](float* to) {
#pragma unroll
    for (int rt = 0; rt < 8; ++rt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        to[(16 * rt + 4 * g + i) * D + col0 + l16] = __builtin_amdgcn_ldexpf(accS[rt][i], col_exp);
  };
  chunk_barrier();
  chunk_barrier();

  for (int ci = 0; ci < nch; ++ci) {
    if constexpr (OUT) {
      // the gradient of the state at the boundaries of the decays' gradient
      const int64_t done = min(ch.begin(ci) + C, it.te) - it.bos;
      const bool at_end = done == it.eos - it.bos;
      if (p.anchors && (at_end ? p.end_state : done % p.anchor == 0)) {
        const int64_t j = (done + p.anchor - 1) / p.anchor;
        store_state(p.anchors + ((size_t)boundary_of(it.n, it.bos, p.anchor, p.end_state, j) * H + h) * kState);
      }
    }
    chunk_barrier();
    const int b = ci % 3, b2 = ci & 1;
    const uint32_t base = lds0 + (uint32_t)b2 * L::SET;
    const uint32_t vbase = lds0 + L::VALS + b * L::VTILE;
    const uint32_t x_at = as_is(lds0 + L::XS + b * L::XBYTES + t_at);
    const uint32_t p_at = as_is(lds0 + L::PAIR + b2 * (PT * L::PTERM) + t_at);
    const unsigned char* factors = smem + L::XS + b * L::XBYTES;
    const float* sRow = reinterpret_cast<const float*>(factors + L::ROW);
    const float* sWgt = reinterpret_cast<const float*>(factors + L::WGT);
    const float* sBeta = reinterpret_cast<const float*>(factors + L::BETA);
    const float gam = *reinterpret_cast<const float*>(factors + L::GAM);
    const int* sExp = reinterpret_cast<const int*>(smem + L::EXPS) + b2 * C;
    f16x8 fk[2][NT][IT];
    auto read_k = [&](int ks) {
#pragma unroll
      for (int rt = 0; rt < NT; ++rt)
#pragma unroll
        for (int t = 0; t < IT; ++t) fk[ks & 1][rt][t] = ld_row_h(base + L::K + t * L::HALF + q_at, 32 * ks, 16 * rt);
    };
    read_k(0);

    // d_o with the query rows' scale: rows 16 rt + 4 g + i of this lane's column
    f32x4 val[NT];
    read_column<E, L>(val, vbase, vc0, l16, g);
#pragma unroll
    for (int rt = 0; rt < NT; ++rt) {
      const i32x4 eq = *reinterpret_cast<const i32x4*>(sExp + 16 * rt + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) val[rt][i] = __builtin_amdgcn_ldexpf(val[rt][i], eq[i]);
    }
    bool live;
    {
      // the columns' scale
      float ms = 0.f, mv = 0.f;
#pragma unroll
      for (int rt = 0; rt < 8; ++rt)
#pragma unroll
        for (int i = 0; i < 4; ++i) ms = fmaxf(ms, fabsf(accS[rt][i]));
#pragma unroll
      for (int rt = 0; rt < NT; ++rt)
#pragma unroll
        for (int i = 0; i < 4; ++i) mv = fmaxf(mv, fabsf(val[rt][i]));
      // (a row of q is below 2^kQueryExpBack, its length below 12 times that: what 64 tokens add to a
      // du stays below 2^14)
      const int e = column_exp(ms, col_exp, mv, kQueryExpBack + 4);
      live = e > kNoExp;
      const bool off = live && (e - col_exp > kMostExp || e - col_exp < kLeastExp);
      if (__ballot(off) || moved) {
        const int de = off ? e - col_exp - kScaledExp : 0;
        col_exp += de;
#pragma unroll
        for (int rt = 0; rt < 8; ++rt)
#pragma unroll
          for (int i = 0; i < 4; ++i) accS[rt][i] = __builtin_amdgcn_ldexpf(accS[rt][i], -de);
        if (g == 0) sCol[wv * 16 + l16] = col_exp;
      }
#pragma unroll
      for (int rt = 0; rt < NT; ++rt)
#pragma unroll
        for (int i = 0; i < 4; ++i) val[rt][i] = __builtin_amdgcn_ldexpf(val[rt][i], -col_exp);
    }
    const size_t unit = (size_t)ch.slot(ci) * H + h;
    const i32x4 ce = *reinterpret_cast<const i32x4*>(sCol + wv * 16 + 4 * g);

    __builtin_amdgcn_sched_barrier(0);
    // du = w k dS' + P^T do.  Each region below first issues the LDS reads of the next one.
    f32x4 acc[NT];
#pragma unroll
    for (int rt = 0; rt < NT; ++rt) acc[rt] = (f32x4){0.f, 0.f, 0.f, 0.f};
    f16x8 fs[2][NS], fp[NT][KS][PT];
    split_op(fs[0], accS[0], accS[1]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      if (ks < 3) {
        read_k(ks + 1);
        split_op(fs[(ks + 1) & 1], accS[2 * ks + 2], accS[2 * ks + 3]);
      } else {
#pragma unroll
        for (int rt = 0; rt < NT; ++rt)
#pragma unroll
          for (int s = rt / 2; s < KS; ++s)
#pragma unroll
            for (int t = 0; t < PT; ++t) fp[rt][s][t] = ld_tiles_t(p_at + t * L::PTERM, rt, s);
      }
      if constexpr (OUT) store_turned((const E*)nullptr, p.ds, unit, ct, ks, fs[ks & 1][0], accS, ident, ce, lane);
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) acc[rt] = mma_terms(acc[rt], fk[ks & 1][rt], fs[ks & 1]);
      __builtin_amdgcn_sched_barrier(0);
    }
    // dS, of which the queries' part does not wait for dv.  Where the chunk's first decay
    // leaves little of everything that reaches it, the operands are scaled by that: all
    // factors come relative to the first token's.
    const float first = sRow[0];
    const int ef = first > 0.f ? max(__builtin_amdgcn_readfirstlane(__builtin_amdgcn_frexp_expf(first)), -120) : 0;
    const float up = __builtin_amdgcn_ldexpf(1.f, -ef);
#pragma unroll
    for (int rt = 0; rt < 8; ++rt) accS[rt] *= up * gam;
    auto queries = [&](int s) {
      f16x8 fq[NS];
      const f32x4 f0 = up * *reinterpret_cast<const f32x4*>(sRow + 32 * s + 4 * g);
      const f32x4 f1 = up * *reinterpret_cast<const f32x4*>(sRow + 32 * s + 16 + 4 * g);
      split_op(fq, f0 * val[2 * s], f1 * val[2 * s + 1]);
#pragma unroll
      for (int rt = 0; rt < 8; ++rt) {
        f16x8 f[IT];
#pragma unroll
        for (int t = 0; t < IT; ++t) f[t] = ld_col_h(base + L::Q + t * L::HALF, k_at, 16 * rt, 32 * s);
        accS[rt] = mma_terms(accS[rt], f, fq);
      }
    };
    f32x4 beta[NT];
#pragma unroll
    for (int rt = 0; rt < NT; ++rt) beta[rt] = *reinterpret_cast<const f32x4*>(sBeta + 16 * rt + 4 * g);
    {
      f16x8 fd[KS][IT];
#pragma unroll
      for (int s = 0; s < KS; ++s) split_op(fd[s], val[2 * s], val[2 * s + 1]);
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) acc[rt] *= exp2i(-Num<E>::KEXP) * *reinterpret_cast<const f32x4*>(sWgt + 16 * rt + 4 * g);
#pragma unroll
      for (int s = KS - 1; s >= 0; --s)
#pragma unroll
        for (int rt = 0; rt <= 2 * s + 1; ++rt) acc[rt] = mma_terms(acc[rt], fp[rt][s], fd[s]);
      queries(0);
    }
    // y = du - X^T (B du); (the block holds -X)
    f16x8 fx[NT][KS][NS];
#pragma unroll
    for (int rt = 0; rt < NT; ++rt)
#pragma unroll
      for (int s = rt / 2; s < KS; ++s)
#pragma unroll
        for (int t = 0; t < NS; ++t) fx[rt][s][t] = ld_tiles_t(x_at + t * L::XTERM, rt, s);
    __builtin_amdgcn_sched_barrier(0);
    {
      f16x8 fb[KS][NS];
#pragma unroll
      for (int s = 0; s < KS; ++s) split_op(fb[s], beta[2 * s] * acc[2 * s], beta[2 * s + 1] * acc[2 * s + 1]);
#pragma unroll
      for (int s = KS - 1; s >= 0; --s)
#pragma unroll
        for (int rt = 0; rt <= 2 * s + 1; ++rt) acc[rt] = mma_terms(acc[rt], fx[rt][s], fb[s]);
      if constexpr (KS == 2) queries(1);
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (OUT) {
      // dbeta over this wave's columns
      float x[4 * NT];
#pragma unroll
      for (int rt = 0; rt < NT; ++rt)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[4 * rt + i] = __builtin_amdgcn_ldexpf(e[rt][i], col_exp) * acc[rt][i];
      const float sum = sum_rows(x, l16);
      const int at = l16 & (4 * NT - 1), row = 16 * (at >> 2) + 4 * g + (at & 3);
      if (p.beta_part && l16 < 4 * NT && row < ch.rows(ci))
        p.beta_part[((size_t)(cb * 4 + wv) * H + h) * p.total_tokens + ch.begin(ci) + row] = sum;
    }
    // dv = B y: y, which is not small where beta is, is turned over and handed on
    if constexpr (OUT) {
      const Rsrc rs = chunk_rows<E>(p.dv, H, h, ch, ci, D * ES);
      const Rsrc rh = ES == 2 ? chunk_rows<E>(p.yh, H, h, ch, ci, D * ES) : rs;
      f16x8 fv[KS][NS];
#pragma unroll
      for (int s = 0; s < KS; ++s) split_op(fv[s], acc[2 * s], acc[2 * s + 1]);
      float dot[NT];
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) {
        f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = NS - 1; t >= 0; --t) y = mma_h(y, fv[rt / 2][t], ident[rt & 1]);
        Frag16<E> f;
        f.v = __builtin_bit_cast(decltype(f.v), v[rt]);
        const f32x4 x = frag16_to_f32(f);
        if constexpr (ES == 2) store_cols_h(rh, (int)(o_at + 16 * rt * o_row), y);
        y *= sBeta[16 * rt + l16];
        dot[rt] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) dot[rt] += x[i] * __builtin_amdgcn_ldexpf(y[i], ce[i]);
        store_cols<E>(rs, (int)(o_at + 16 * rt * o_row), y, ce);
      }
      if (ES == 2 && g == 0) p.exps[unit * D + col0 + l16] = live ? col_exp : kNoExp;
      int tile;
      const float sum = sum_groups(dot, g, tile);
      if (p.change && tile >= 0 && 16 * tile + l16 < ch.rows(ci))
        p.change[((size_t)(cb * 4 + wv) * H + h) * p.total_tokens + ch.begin(ci) + 16 * tile + l16] = sum;
      load_next(ci + 1);
    }
#pragma unroll
    for (int rt = 0; rt < NT; ++rt) acc[rt] *= beta[rt];
    moved = ef != 0;
    col_exp += ef;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      f16x8 fv[NS];
      {
        constexpr float ks = -exp2i(-Num<E>::KEXP);
        const f32x4 f0 = ks * up * *reinterpret_cast<const f32x4*>(sRow + 32 * s + 4 * g);
        const f32x4 f1 = ks * up * *reinterpret_cast<const f32x4*>(sRow + 32 * s + 16 + 4 * g);
        split_op(fv, f0 * acc[2 * s], f1 * acc[2 * s + 1]);
      }
#pragma unroll
      for (int rt = 0; rt < 8; ++rt) {
        f16x8 f[IT];
#pragma unroll
        for (int t = 0; t < IT; ++t) f[t] = ld_col_h(base + L::K + t * L::HALF, k_at, 16 * rt, 32 * s);
        accS[rt] = mma_terms(accS[rt], f, fv);
      }
    }
  }
  float* dst = nullptr;
  if (!OUT) dst = p.rstates + ((size_t)it.slot * H + h) * kState;
  else if (p.d_initial && it.first) dst = p.d_initial + nh * kState;
  if (dst) store_state(dst);
}

template <typename E, Walk W>
__global__ __launch_bounds__(kWalkThreads) void delta_back_kernel(const DeltaBackArgs p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  int part;
  const int64_t u = delta_unit<2>(p.unit0, p.num_heads, p.qk_heads, blockIdx.x, part);
  if (u < p.units) delta_back<E, W>(p, smem, u, part);
}

template <typename E, Walk W>
hipError_t launch_back_e(const DeltaBackArgs& a, hipStream_t stream) {
  constexpr int LDS = DeltaLayout<E, 2>::BYTES;
  static std::atomic<bool> set[64];
  const hipError_t e = allow_lds(delta_back_kernel<E, W>, LDS, set);
  if (e != hipSuccess) return e;
  return launch_delta_parts<2>(a, [&](const DeltaBackArgs& part, unsigned blocks) {
    hipLaunchKernelGGL((delta_back_kernel<E, W>), dim3(blocks), dim3(kWalkThreads), LDS, stream, part);
  });
}

// ---------------------------------------------------------------------------
// The gradient that reaches every segment's end, from the last segment back:
// D_end(j - 1) = M_j^T D_end(j) + B'_j, with the forward transitions M_j.  As
// delta_scan_kernel; D_end(j) takes B'_j's place.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void delta_back_scan_kernel(const DeltaBackScanArgs a) {
  constexpr size_t kState = (size_t)D * D;
  const int H = a.num_heads;
  const int ct = blockIdx.x & 7;
  const int64_t nh = a.unit0 + (blockIdx.x >> 3);
  const int n = (int)(nh / H), h = (int)(nh % H);
  const int tid = threadIdx.x, wv = tid >> 6, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
  const int col = 16 * ct + l16;
  int64_t bos, eos;
  seq_range(a.cu, n, a.total_tokens, bos, eos);
  const int count = (int)((eos - bos + a.seg - 1) / a.seg);
  if (count == 0) return;
  const int64_t base = slot_of(n, bos, a.seg, 0);
  __shared__ f32x4 sS[8][64];
  auto row_of = [&](int q, int i) { return 16 * (2 * wv + q) + 4 * g + i; };
  f32x4 mine[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
#pragma unroll
    for (int i = 0; i < 4; ++i) mine[q][i] = a.d_final ? a.d_final[(size_t)nh * kState + row_of(q, i) * D + col] : 0.f;
    sS[2 * wv + q][lane] = mine[q];
  }
  __syncthreads();
  for (int j = count - 1; j >= 0; --j) {
    float* Bj = a.rstates + ((size_t)(base + j) * H + h) * kState;
    const float* Mj = a.pairs + (((size_t)(base + j) * H + h) * 2 + 1) * kState;
    f32x4 acc[2];
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float* at = Bj + row_of(q, i) * D + col;
        if (j > 0) acc[q][i] = *at;  // (the first segment's is not formed)
        *at = mine[q][i];
      }
    if (j == 0) break;
#pragma unroll
    for (int kt = 0; kt < 8; ++kt) {
      Frag16<float> sf, mf;
      sf.v = sS[kt][lane];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
#pragma unroll
        for (int i = 0; i < 4; ++i) mf.v[i] = Mj[(size_t)(16 * kt + 4 * g + i) * D + 16 * (2 * wv + q) + l16];
        acc[q] = mma16(acc[q], mf, sf);
      }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      mine[q] = acc[q];
      sS[2 * wv + q][lane] = acc[q];
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// dq and dk of a chunk, for the value heads that share a query and key head in
// turn.  Four waves per (chunk, query and key head); wave w owns 32 key channels
// of both.  First the products with S and dS', whose operands come straight
// from memory (a wave's own rows), and the pairs do . u and dv . u, shared out
// by tiles; then, with those in LDS, their products with k and q.  Bound by the
// traffic of the states between the walks and this kernel (178 KB a chunk and head
// in bf16, 452 us for 96 heads x 8192 tokens at a copy's rate; they take 424, as the
// cache holds some of it).  Two workgroups a compute unit, as registers allow: with
// one, all operands of a phase held, 590 us.
//   dq = f do S^T + tril(do u^T decays) k
//   dk = -f dv S^T + w u dS'^T + tril(do u^T decays)^T q - sym(dv u^T decays) k
// ---------------------------------------------------------------------------
constexpr int kGradThreads = 256;

// The chunk of a workgroup: its first token and rows; none: rows = 0.
template <int C>
__device__ __forceinline__ void grad_chunk(const DeltaGradArgs& p, int64_t slot, int64_t& t0, int& rows) {
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
  t0 = bos + j * C;
  rows = j < 0 || t0 >= eos ? 0 : (int)min((int64_t)C, eos - t0);
}

// Copies a chunk's rows of one head ([C][128], swizzled), and the prep kernel's
// factors, straight into LDS.
template <typename E, int C>
__device__ __forceinline__ void copy_rows(unsigned char* dst, const void* src, int heads, int head, int64_t t0, int rows,
                                          int wv, int lane) {
  constexpr int ES = (int)sizeof(E), UR = D * ES / 16, RP = 64 / UR, PIECES = C * D * ES / 1024 / 4;
  const uint32_t stride = (uint32_t)heads * (D * ES);
  const Rsrc rs = make_rsrc(static_cast<const char*>(src) + (size_t)t0 * stride + (size_t)head * (D * ES),
                            (uint32_t)(rows - 1) * stride + D * ES);
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int piece = wv * PIECES + i, row = piece * RP + lane / UR;
    const uint32_t unit = (uint32_t)(((lane % UR) ^ swizzle<E, D>(row)) * 16);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)(dst + piece * 1024), 16,
                                             (int)((uint32_t)row * stride + unit), 0, 0, 0);
  }
}
template <int C>
__device__ __forceinline__ void copy_factors(unsigned char* dst, const char* blocks, size_t unit, int wv, int lane) {
  constexpr int PIECES = delta_factor_bytes(C) / 1024;
  const Rsrc rs = make_rsrc(blocks + unit * delta_block_bytes(C) + delta_matrix_bytes(C), delta_factor_bytes(C));
  if (wv < PIECES)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)(dst + wv * 1024), 16,
                                             wv * 1024 + lane * 16, 0, 0, 0);
}

// rows 16 rt + 4 g + i, channels 32 wv + 16 c + l16: through LDS for whole rows
template <typename E, int C>
__device__ __forceinline__ void store_grads(const DeltaGradArgs& p, unsigned char* smem, const f32x4 (&dq)[C / 16][2],
                                            const f32x4 (&dk)[C / 16][2], int hq, int64_t t0, int rows) {
  constexpr int ES = (int)sizeof(E), TILE = C * D * ES;
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4, wv = tid >> 6;
  __syncthreads();
#pragma unroll
  for (int which = 0; which < 2; ++which) {
#pragma unroll
    for (int rt = 0; rt < C / 16; ++rt)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<E*>(smem + which * TILE + tile_at<E, D>(16 * rt + 4 * g + i, 32 * wv + 16 * c + l16)) =
              from_f32<E>((which ? dk : dq)[rt][c][i]);
  }
  __syncthreads();
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    constexpr int UR = D * ES / 16;
    char* dst = static_cast<char*>(which ? p.dk : p.dq) + ((size_t)t0 * p.qk_heads + hq) * (D * ES);
    for (int i = tid; i < rows * UR; i += kGradThreads) {
      const int row = i / UR, unit = i % UR;
      const u32x4 y = *reinterpret_cast<const u32x4*>(smem + which * TILE + row * (D * ES) + ((unit ^ swizzle<E, D>(row)) * 16));
      *reinterpret_cast<u32x4*>(dst + (size_t)row * p.qk_heads * (D * ES) + unit * 16) = y;
    }
  }
}

// ---- bf16 inputs.  S, u and dS', y = dv / beta come in fp16, their value columns
// scaled by the walks: 2^cs and 2^cb.  The products over value columns take
//   do' = do 2^(cs - e), e the row's largest exponent, and
//   y' = y 2^(cs + cb - m) and dS' so with u, m the largest cs + cb,
// whose powers of two leave the sum again, as beta joins it.  Pairs are bf16 in two
// terms: their magnitudes differ from row to row, and so do those of k and q.  bf16 operands
// throughout made dq and dk 1.7 times as far off as their own rounding is. ----
struct GradHLayout {
  static constexpr int C = 64, TILES = delta_tiles(C);
  static constexpr int TILE = C * D * 2;                 // a [C][128] tile
  static constexpr int DO = 0, U = TILE, DV = 2 * TILE;  // first; then k and q
  static constexpr int KT = 0, QT = TILE;
  static constexpr int PTERM = TILES * kDeltaTileBytes;
  static constexpr int PO = 3 * TILE;                    // [2] terms of do . u
  static constexpr int PV = PO + 2 * PTERM;              // [2] terms of -dv . u, below the diagonal
  static constexpr int FACT = PV + 2 * PTERM;            // the prep kernel's factors
  static constexpr int EXPS = FACT + delta_factor_bytes(C);  // int [C] e
  static constexpr int SCALE = EXPS + C * 4;             // fp16 [128] 2^(cs + cb - m)
  static constexpr int BYTES = SCALE + D * 2;
};

__device__ __forceinline__ void store_pair_b(unsigned char* tiles, int rt, int kt, int l16, int g, f32x4 x) {
  bf16x4 hi, lo;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    hi[i] = (__bf16)x[i];
    lo[i] = (__bf16)(x[i] - (float)hi[i]);
  }
  unsigned char* to = tiles + tile_no(rt, kt) * kDeltaTileBytes + tile16_at(l16, g);
  *reinterpret_cast<u32x2*>(to) = __builtin_bit_cast(u32x2, hi);
  *reinterpret_cast<u32x2*>(to + GradHLayout::PTERM) = __builtin_bit_cast(u32x2, lo);
}

// A sum that is formed here (the compiler would put it off and keep its parts).
__device__ __forceinline__ void formed(f32x4& x) { asm volatile("" : "+v"(x)); }

__global__ __launch_bounds__(kGradThreads, 2) void delta_grad_h_kernel(const DeltaGradArgs p) {
  using L = GradHLayout;
  constexpr int C = L::C, NT = C / 16, FACT = delta_matrix_bytes(C);
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)smem;
  using W = DeltaLayout<__bf16, 2>;
  const float* sSum = reinterpret_cast<const float*>(smem + L::FACT + W::SUM - FACT);
  const float* sRow = reinterpret_cast<const float*>(smem + L::FACT + W::ROW - FACT);
  const float* sWgt = reinterpret_cast<const float*>(smem + L::FACT + W::WGT - FACT);
  const float* sBeta = reinterpret_cast<const float*>(smem + L::FACT + W::BETA - FACT);
  int* sExp = reinterpret_cast<int*>(smem + L::EXPS);
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int H = p.num_heads, Hq = p.qk_heads, share = H / Hq;
  const int64_t wg = p.unit0 + blockIdx.x;
  const int hq = (int)(wg % Hq);
  const int64_t slot = wg / Hq;
  int64_t t0;
  int nv;
  grad_chunk<C>(p, slot, t0, nv);
  if (nv == 0) return;

  // a thread's rows 16 wv + 4 i + g and channels 8 l16 ..
  auto load_rows = [&](u32x4 (&raw)[4], const void* src, int heads, int head) {
    const uint32_t stride = (uint32_t)heads * (D * 2);
    const Rsrc rs = make_rsrc(static_cast<const char*>(src) + (size_t)t0 * stride + (size_t)head * (D * 2),
                              (uint32_t)(nv - 1) * stride + D * 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) raw[i] = buf_ld16(rs, (uint32_t)(16 * wv + 4 * i + g) * stride + l16 * 16, 0);
  };
  auto row_at = [&](int tile, int i) -> u32x4* {
    return reinterpret_cast<u32x4*>(smem + tile + tile_at<__bf16, D>(16 * wv + 4 * i + g, 8 * l16));
  };
  const uint32_t a_at = tile_at<__bf16, D>(l16, 4 * g);
  f32x4 dq[NT][2], dk[NT][2];
#pragma unroll
  for (int rt = 0; rt < NT; ++rt)
#pragma unroll
    for (int c = 0; c < 2; ++c) dq[rt][c] = dk[rt][c] = (f32x4){0.f, 0.f, 0.f, 0.f};

  for (int hs = 0; hs < share; ++hs) {
    const int h = hq * share + hs;
    const size_t unit = (size_t)slot * H + h;
    if (hs > 0) __syncthreads();
    copy_factors<C>(smem + L::FACT, p.blocks, unit, wv, lane);
    copy_rows<__bf16, C>(smem + L::U, p.u, H, h, t0, nv, wv, lane);
    __builtin_amdgcn_sched_barrier(0);
    u32x4 raw[4], rawv[4];
    i32x4 cs[2], cb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      cs[i] = *reinterpret_cast<const i32x4*>(p.s_exps + unit * D + 8 * l16 + 4 * i);
      cb[i] = *reinterpret_cast<const i32x4*>(p.ds_exps + unit * D + 8 * l16 + 4 * i);
    }
    load_rows(raw, p.d_o, H, h);
    load_rows(rawv, p.yh, H, h);
    __builtin_amdgcn_sched_barrier(0);
    // this wave's rows of S and dS'
    const u32x2* si = static_cast<const u32x2*>(p.s) + unit * 4096 + lane;
    const u32x2* di = static_cast<const u32x2*>(p.ds) + unit * 4096 + lane;
    auto load_state = [&](f16x8 (&f)[4][2], const u32x2* img) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const u32x2* at = img + ((2 * wv + c) * 8 + 2 * s) * 64;
          const u32x2 x = __builtin_nontemporal_load(at), y = __builtin_nontemporal_load(at + 64);
          f[s][c] = __builtin_bit_cast(f16x8, (u32x4){x[0], x[1], y[0], y[1]});
        }
    };
    f16x8 fs[4][2], fd[4][2];
    load_state(fs, si);
    load_state(fd, di);
    __builtin_amdgcn_sched_barrier(0);

    // scales
    int most = INT32_MIN;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cb[i / 4][i % 4] += cs[i / 4][i % 4];
      most = max(most, cb[i / 4][i % 4]);
    }
    most = max(most, __builtin_amdgcn_update_dpp(0, most, 0x128, 0xf, 0xf, true));
    most = max(most, __builtin_amdgcn_update_dpp(0, most, 0x124, 0xf, 0xf, true));
    most = max(most, __builtin_amdgcn_update_dpp(0, most, 0x122, 0xf, 0xf, true));
    most = max(most, __builtin_amdgcn_update_dpp(0, most, 0x121, 0xf, 0xf, true));
    const int em = __builtin_amdgcn_readfirstlane(most);
    f16x8 scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) scale[i] = (_Float16)__builtin_amdgcn_ldexpf(1.f, cb[i / 4][i % 4] - em);
    if (wv == 0 && g == 0) *reinterpret_cast<f16x8*>(smem + L::SCALE + 16 * l16) = scale;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x[8];
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w = raw[i][j];
        x[2 * j] = __builtin_amdgcn_ldexpf(__builtin_bit_cast(float, w << 16), cs[j / 2][2 * (j & 1)]);
        x[2 * j + 1] = __builtin_amdgcn_ldexpf(__builtin_bit_cast(float, w & 0xffff0000u), cs[j / 2][2 * (j & 1) + 1]);
        m = fmaxf(m, fmaxf(fabsf(x[2 * j]), fabsf(x[2 * j + 1])));
      }
      m = max_row(m);
      const int e = m > 0.f ? __builtin_amdgcn_frexp_expf(m) : 0;
      if (l16 == 0) sExp[16 * wv + 4 * i + g] = e;
      u32x4 y;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        y[j] = __builtin_bit_cast(uint32_t, cvt_h2(__builtin_amdgcn_ldexpf(x[2 * j], -e), __builtin_amdgcn_ldexpf(x[2 * j + 1], -e)));
      *row_at(L::DO, i) = y;
      *row_at(L::DV, i) = __builtin_bit_cast(u32x4, __builtin_bit_cast(f16x8, rawv[i]) * scale);
    }
    // (the copies into LDS have landed: the states' loads came behind them)
    __builtin_amdgcn_s_waitcnt(vmcnt_wait(32));
    __syncthreads();

    uint32_t at = as_is(lds0 + a_at);
    // dq += f do S^T, dk -= f dv S^T; by key channels, as registers allow
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      f32x4 aq[NT], ak[NT];
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) aq[rt] = ak[rt] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        f16x8 fo[NT], fv[NT];
#pragma unroll
        for (int rt = 0; rt < NT; ++rt) {
          fo[rt] = ld_row_h(at + L::DO, 32 * s, 16 * rt);
          fv[rt] = ld_row_h(at + L::DV, 32 * s, 16 * rt);
        }
#pragma unroll
        for (int rt = 0; rt < NT; ++rt) {
          aq[rt] = mma_h(aq[rt], fo[rt], fs[s][c]);
          ak[rt] = mma_h(ak[rt], fv[rt], fs[s][c]);
        }
        at = after(at, fo[0]);
      }
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) {
        const f32x4 f = *reinterpret_cast<const f32x4*>(sRow + 16 * rt + 4 * g);
        const f32x4 b = *reinterpret_cast<const f32x4*>(sBeta + 16 * rt + 4 * g);
        const i32x4 e = *reinterpret_cast<const i32x4*>(sExp + 16 * rt + 4 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dq[rt][c][i] += f[i] * __builtin_amdgcn_ldexpf(aq[rt][i], e[i]);
          dk[rt][c][i] -= f[i] * b[i] * __builtin_amdgcn_ldexpf(ak[rt][i], em);
        }
        formed(dq[rt][c]);
        formed(dk[rt][c]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // k and q, for later
    u32x4 rawk[4];
    load_rows(rawk, p.k, Hq, hq);
    load_rows(raw, p.q, Hq, hq);
    // dk += w u dS'^T
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const u32x2 x = *reinterpret_cast<const u32x2*>(smem + L::SCALE + 2 * (32 * s + 4 * g));
      const u32x2 y = *reinterpret_cast<const u32x2*>(smem + L::SCALE + 2 * (32 * s + 16 + 4 * g));
      const f16x8 sc = __builtin_bit_cast(f16x8, (u32x4){x[0], x[1], y[0], y[1]});
#pragma unroll
      for (int c = 0; c < 2; ++c) fd[s][c] *= sc;
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      f32x4 ak[NT];
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) ak[rt] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        f16x8 fu[NT];
#pragma unroll
        for (int rt = 0; rt < NT; ++rt) fu[rt] = ld_row_h(at + L::U, 32 * s, 16 * rt);
#pragma unroll
        for (int rt = 0; rt < NT; ++rt) ak[rt] = mma_h(ak[rt], fu[rt], fd[s][c]);
        at = after(at, fu[0]);
      }
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) {
        const f32x4 w = *reinterpret_cast<const f32x4*>(sWgt + 16 * rt + 4 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) dk[rt][c][i] += w[i] * __builtin_amdgcn_ldexpf(ak[rt][i], em);
        formed(dk[rt][c]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }

    // pairs: column = the later token i, rows = four earlier ones
    for (int no = wv; no < L::TILES; no += 4) {
      int rt = 0;
      while (tile_no(rt + 1, 0) <= no) ++rt;
      const int kt = no - tile_no(rt, 0);
      f32x4 ao = {0.f, 0.f, 0.f, 0.f}, av = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const f16x8 fu = ld_row_h(at + L::U + 16 * kt * (D * 2), 32 * s, 0);
        ao = mma_h(ao, fu, ld_row_h(at + L::DO + 16 * rt * (D * 2), 32 * s, 0));
        av = mma_h(av, fu, ld_row_h(at + L::DV + 16 * rt * (D * 2), 32 * s, 0));
      }
      const int i = 16 * rt + l16;
      const float gi = sSum[i], gi_lo = sSum[C + i];
      const f32x4 gj = *reinterpret_cast<const f32x4*>(sSum + 16 * kt + 4 * g);
      const f32x4 gj_lo = *reinterpret_cast<const f32x4*>(sSum + C + 16 * kt + 4 * g);
      const int ei = sExp[i];
      const float bi = -sBeta[i];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int jj = 16 * kt + 4 * g + x;
        const float d = exp2_fast((gi - gj[x]) + (gi_lo - gj_lo[x]));
        ao[x] = jj <= i ? __builtin_amdgcn_ldexpf(ao[x], ei) * d : 0.f;
        av[x] = jj < i ? bi * __builtin_amdgcn_ldexpf(av[x], em) * d : 0.f;
      }
      store_pair_b(smem + L::PO, rt, kt, l16, g, ao);
      store_pair_b(smem + L::PV, rt, kt, l16, g, av);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      *row_at(L::KT, i) = rawk[i];
      *row_at(L::QT, i) = raw[i];
    }
    __syncthreads();

    // contractions over the tokens 32 s ..
    const uint32_t c_at = tile_at<__bf16, D>(4 * g + (l16 >> 2), 4 * (l16 & 3));
    const uint32_t t_at = tile16_at(l16, g), tt_at = tile16_at(4 * g + (l16 >> 2), l16 & 3);
    auto mma_b = [](f32x4 acc, f16x8 a, f16x8 b) {
      Frag<__bf16> x, y;
      x.v = __builtin_bit_cast(bf16x8, a);
      y.v = __builtin_bit_cast(bf16x8, b);
      return mma(acc, x, y);
    };
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      f16x8 fk[2], fq[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        fk[c] = ld_col_h(lds0 + L::KT, c_at, 32 * wv + 16 * c, 32 * s);
        fq[c] = ld_col_h(lds0 + L::QT, c_at, 32 * wv + 16 * c, 32 * s);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint32_t po = lds0 + L::PO + t * L::PTERM, pv = lds0 + L::PV + t * L::PTERM;
#pragma unroll
        for (int rt = 0; rt < NT; ++rt) {
          if (s <= rt / 2) {
            const f16x8 fo = ld_tiles(po + t_at, rt, s), fv = ld_tiles(pv + t_at, rt, s);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              dq[rt][c] = mma_b(dq[rt][c], fo, fk[c]);
              dk[rt][c] = mma_b(dk[rt][c], fv, fk[c]);
            }
          }
          if (s >= rt / 2) {
            const f16x8 fo = ld_tiles_t(po + tt_at, rt, s), fv = ld_tiles_t(pv + tt_at, rt, s);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              dk[rt][c] = mma_b(dk[rt][c], fo, fq[c]);
              dk[rt][c] = mma_b(dk[rt][c], fv, fk[c]);
            }
          }
        }
      }
    }
  }
  store_grads<__bf16, C>(p, smem, dq, dk, hq, t0, nv);
}

// ---- fp32 inputs: fp32 throughout. ----
struct GradFLayout {
  static constexpr int C = 32, NT = C / 16, TILES = delta_tiles(C);
  static constexpr int TILE = C * D * 4;
  static constexpr int PTILE = 16 * 16 * 4;      // a pair tile
  static constexpr int DO = 0, U = TILE, DV = 2 * TILE;  // first; then k and q
  static constexpr int KT = 0, QT = TILE;
  static constexpr int PO = 3 * TILE;            // [TILES] do . u
  static constexpr int PV = PO + TILES * PTILE;  // [NT][NT] -dv . u, symmetric
  static constexpr int FACT = PV + NT * NT * PTILE;  // the prep kernel's factors
  static constexpr int BYTES = FACT + delta_factor_bytes(C);
};

// 16 x 16 tiles of pairs: rows of 64 bytes, their 16-byte units turned by the row.
__device__ __forceinline__ uint32_t ptile_at(int row, int piece) {
  return (uint32_t)(row * 64 + ((piece ^ ((row >> 1) & 3)) << 4));
}
// operand rows (lane = row l16, four columns 4 g ..), and of the transposed tile
__device__ __forceinline__ void ld_ptile(Frag16<float>& f, uint32_t base, int l16, int g) {
  f.v = lds_get<f32x4>(base + ptile_at(l16, g));
}
__device__ __forceinline__ void ld_ptile_t(Frag16<float>& f, uint32_t base, int l16, int g) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f.v[i] = lds_get<float>(base + ptile_at(4 * g + i, l16 >> 2) + 4 * (l16 & 3));
}
// operand over the tokens t0 + 4 g .. of channel ch0 + l16 of a [C][128] tile
__device__ __forceinline__ void ld_tok(Frag16<float>& f, uint32_t base, int ch0, int t0, int l16, int g) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f.v[i] = lds_get<float>(base + tile_at<float, D>(t0 + 4 * g + i, ch0 + l16));
}

__global__ __launch_bounds__(kGradThreads, 2) void delta_grad_f_kernel(const DeltaGradArgs p) {
  using L = GradFLayout;
  constexpr int C = L::C, NT = L::NT, FACT = delta_matrix_bytes(C);
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)smem;
  using W = DeltaLayout<float, 2>;
  const float* sSum = reinterpret_cast<const float*>(smem + L::FACT + W::SUM - FACT);
  const float* sRow = reinterpret_cast<const float*>(smem + L::FACT + W::ROW - FACT);
  const float* sWgt = reinterpret_cast<const float*>(smem + L::FACT + W::WGT - FACT);
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int H = p.num_heads, Hq = p.qk_heads, share = H / Hq;
  const int64_t wg = p.unit0 + blockIdx.x;
  const int hq = (int)(wg % Hq);
  const int64_t slot = wg / Hq;
  int64_t t0;
  int nv;
  grad_chunk<C>(p, slot, t0, nv);
  if (nv == 0) return;

  const uint32_t a_at = tile_at<float, D>(l16, 4 * g);
  f32x4 dq[NT][2], dk[NT][2];
#pragma unroll
  for (int rt = 0; rt < NT; ++rt)
#pragma unroll
    for (int c = 0; c < 2; ++c) dq[rt][c] = dk[rt][c] = (f32x4){0.f, 0.f, 0.f, 0.f};

  for (int hs = 0; hs < share; ++hs) {
    const int h = hq * share + hs;
    const size_t unit = (size_t)slot * H + h;
    if (hs > 0) __syncthreads();
    copy_factors<C>(smem + L::FACT, p.blocks, unit, wv, lane);
    copy_rows<float, C>(smem + L::DO, p.d_o, H, h, t0, nv, wv, lane);
    copy_rows<float, C>(smem + L::U, p.u, H, h, t0, nv, wv, lane);
    copy_rows<float, C>(smem + L::DV, p.dv, H, h, t0, nv, wv, lane);
    // this wave's rows of S and dS'
    const f32x4* si = static_cast<const f32x4*>(p.s) + unit * 4096 + lane;
    const f32x4* di = static_cast<const f32x4*>(p.ds) + unit * 4096 + lane;
    __builtin_amdgcn_s_waitcnt(vmcnt_wait(0));
    __syncthreads();

    // dq += f do S^T, dk -= f dv S^T, dk += w u dS'^T
    f32x4 aq[NT][2], av[NT][2], au[NT][2];
#pragma unroll
    for (int rt = 0; rt < NT; ++rt)
#pragma unroll
      for (int c = 0; c < 2; ++c) aq[rt][c] = av[rt][c] = au[rt][c] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      Frag<float> fs[2], fd[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int at = ((2 * wv + c) * 8 + 2 * s) * 64;
        fs[c].lo = __builtin_nontemporal_load(si + at);
        fs[c].hi = __builtin_nontemporal_load(si + at + 64);
        fd[c].lo = __builtin_nontemporal_load(di + at);
        fd[c].hi = __builtin_nontemporal_load(di + at + 64);
      }
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) {
        Frag<float> fo, fv, fu;
        ld_row_acc(fo, lds0 + L::DO + a_at, 32 * s, 16 * rt);
        ld_row_acc(fv, lds0 + L::DV + a_at, 32 * s, 16 * rt);
        ld_row_acc(fu, lds0 + L::U + a_at, 32 * s, 16 * rt);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          aq[rt][c] = mma(aq[rt][c], fo, fs[c]);
          av[rt][c] = mma(av[rt][c], fv, fs[c]);
          au[rt][c] = mma(au[rt][c], fu, fd[c]);
        }
      }
    }
#pragma unroll
    for (int rt = 0; rt < NT; ++rt) {
      const f32x4 f = *reinterpret_cast<const f32x4*>(sRow + 16 * rt + 4 * g);
      const f32x4 w = *reinterpret_cast<const f32x4*>(sWgt + 16 * rt + 4 * g);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        dq[rt][c] += f * aq[rt][c];
        dk[rt][c] += w * au[rt][c] - f * av[rt][c];
      }
    }

    // pairs: column = the later token i, rows = four earlier ones
    for (int t = wv; t < 2 * L::TILES; t += 4) {
      const bool of_v = t >= L::TILES;
      const int no = of_v ? t - L::TILES : t;
      int rt = 0;
      while (tile_no(rt + 1, 0) <= no) ++rt;
      const int kt = no - tile_no(rt, 0);
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        Frag<float> fu, fx;
        ld_row_acc(fu, lds0 + L::U + a_at + 16 * kt * (D * 4), 32 * s, 0);
        ld_row_acc(fx, lds0 + (of_v ? L::DV : L::DO) + a_at + 16 * rt * (D * 4), 32 * s, 0);
        acc = mma(acc, fu, fx);
      }
      const int i = 16 * rt + l16;
      const float gi = sSum[i], gi_lo = sSum[C + i];
      const f32x4 gj = *reinterpret_cast<const f32x4*>(sSum + 16 * kt + 4 * g);
      const f32x4 gj_lo = *reinterpret_cast<const f32x4*>(sSum + C + 16 * kt + 4 * g);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int jj = 16 * kt + 4 * g + x;
        const float d = (gi - gj[x]) + (gi_lo - gj_lo[x]);
        const float y = acc[x] * exp2_fast(d);
        acc[x] = of_v ? (jj < i ? -y : 0.f) : (jj <= i ? y : 0.f);
      }
      if (!of_v) {
        *reinterpret_cast<f32x4*>(smem + L::PO + no * L::PTILE + ptile_at(l16, g)) = acc;
      } else {
        // both halves of a symmetric matrix
        unsigned char* lower = smem + L::PV + (rt * NT + kt) * L::PTILE;
        unsigned char* upper = smem + L::PV + (kt * NT + rt) * L::PTILE;
        if (rt != kt) *reinterpret_cast<f32x4*>(lower + ptile_at(l16, g)) = acc;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int r = 4 * g + x;  // (of the earlier token)
          float* up = reinterpret_cast<float*>(upper + ptile_at(r, l16 >> 2)) + (l16 & 3);
          float* lo = reinterpret_cast<float*>(lower + ptile_at(l16, r >> 2)) + (r & 3);
          if (rt != kt || r < l16) *up = acc[x];
          if (rt == kt && r <= l16) *lo = acc[x];  // (zero on the diagonal)
        }
      }
    }
    __syncthreads();
    copy_rows<float, C>(smem + L::KT, p.k, Hq, hq, t0, nv, wv, lane);
    copy_rows<float, C>(smem + L::QT, p.q, Hq, hq, t0, nv, wv, lane);
    __builtin_amdgcn_s_waitcnt(vmcnt_wait(0));
    __syncthreads();

#pragma unroll
    for (int kt = 0; kt < NT; ++kt) {
      // contraction over the tokens of tile kt
      Frag16<float> fk[2], fq[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        ld_tok(fk[c], lds0 + L::KT, 32 * wv + 16 * c, 16 * kt, l16, g);
        ld_tok(fq[c], lds0 + L::QT, 32 * wv + 16 * c, 16 * kt, l16, g);
      }
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) {
        Frag16<float> f;
        if (kt <= rt) {
          ld_ptile(f, lds0 + L::PO + tile_no(rt, kt) * L::PTILE, l16, g);
#pragma unroll
          for (int c = 0; c < 2; ++c) dq[rt][c] = mma16(dq[rt][c], f, fk[c]);
        }
        if (kt >= rt) {
          ld_ptile_t(f, lds0 + L::PO + tile_no(kt, rt) * L::PTILE, l16, g);
#pragma unroll
          for (int c = 0; c < 2; ++c) dk[rt][c] = mma16(dk[rt][c], f, fq[c]);
        }
        ld_ptile(f, lds0 + L::PV + (rt * NT + kt) * L::PTILE, l16, g);
#pragma unroll
        for (int c = 0; c < 2; ++c) dk[rt][c] = mma16(dk[rt][c], f, fk[c]);
      }
    }
  }
  store_grads<float, C>(p, smem, dq, dk, hq, t0, nv);
}

template <typename L>
hipError_t launch_grad(void (*kernel)(DeltaGradArgs), std::atomic<bool> (&set)[64], DeltaGradArgs a, hipStream_t stream) {
  hipError_t e = allow_lds(kernel, L::BYTES, set);
  if (e != hipSuccess) return e;
  const int64_t units = delta_chunk_slots(a.total_tokens, a.num_seqs, L::C) * a.qk_heads;
  constexpr int64_t MOST = kMaxThreads / kGradThreads;
  for (int64_t u = 0; u < units; u += MOST) {
    a.unit0 = u;
    hipLaunchKernelGGL(kernel, dim3((unsigned)std::min(units - u, MOST)), dim3(kGradThreads), L::BYTES, stream, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// dbeta [T, H] from its terms by column tiles, [8][H][T]: 64 tokens x 32 heads a
// workgroup, turned over through LDS.  Rows behind the last sequence stay as they are.
__global__ __launch_bounds__(256) void delta_beta_kernel(const float* part, float* dbeta, const int32_t* cu, int num_seqs,
                                                         int64_t T, int64_t block0, int H) {
  __shared__ float tile[32][65];
  const int64_t t0 = (block0 + blockIdx.x) * 64;
  const int64_t rows = cu ? clamp_cu(cu, num_seqs, T) : T;
  const int h0 = blockIdx.y * 32;
  const int t = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int h = w; h < 32; h += 4) {
    float s = 0.f;
    if (t0 + t < rows && h0 + h < H)
      for (int c = 0; c < 8; ++c) s += part[((size_t)c * H + h0 + h) * T + t0 + t];
    tile[h][t] = s;
  }
  __syncthreads();
  const int h = threadIdx.x & 31;
  for (int r = threadIdx.x >> 5; r < 64; r += 8)
    if (t0 + r < rows && h0 + h < H) dbeta[(size_t)(t0 + r) * H + h0 + h] = tile[h][r];
}

}  // namespace

hipError_t launch_delta_back(DeltaBackArgs a, hipStream_t stream) {
  return a.bf16 ? launch_back_e<__bf16, Walk::BACK>(a, stream) : launch_back_e<float, Walk::BACK>(a, stream);
}

hipError_t launch_delta_back_states(DeltaBackArgs a, hipStream_t stream) {
  return a.bf16 ? launch_back_e<__bf16, Walk::BACK_STATES>(a, stream) : launch_back_e<float, Walk::BACK_STATES>(a, stream);
}

hipError_t launch_delta_back_scan(DeltaBackScanArgs a, hipStream_t stream) {
  const int64_t units = (int64_t)a.num_seqs * a.num_heads;
  constexpr int64_t MOST = kMaxThreads / 256 / 8;
  for (int64_t u = 0; u < units; u += MOST) {
    a.unit0 = u;
    hipLaunchKernelGGL(delta_back_scan_kernel, dim3((unsigned)(std::min(units - u, MOST) * 8)), dim3(256), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_delta_grad(DeltaGradArgs a, hipStream_t stream) {
  static std::atomic<bool> set_h[64], set_f[64];
  return a.bf16 ? launch_grad<GradHLayout>(delta_grad_h_kernel, set_h, a, stream)
                : launch_grad<GradFLayout>(delta_grad_f_kernel, set_f, a, stream);
}

hipError_t launch_delta_beta(const float* part, float* dbeta, const int32_t* cu, int num_seqs, int64_t total_tokens,
                             int num_heads, hipStream_t stream) {
  // (as many token blocks as a launch of fewer than 2^32 threads holds: 2^25 of 64 tokens and 2048 of heads)
  const unsigned hb = (unsigned)((num_heads + 31) / 32);
  const int64_t blocks = (total_tokens + 63) / 64, most = kMaxThreads / 256 / hb;
  for (int64_t b = 0; b < blocks; b += most) {
    hipLaunchKernelGGL(delta_beta_kernel, dim3((unsigned)std::min(blocks - b, most), hb), dim3(256), 0, stream, part,
                       dbeta, cu, num_seqs, total_tokens, b, num_heads);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace kda
