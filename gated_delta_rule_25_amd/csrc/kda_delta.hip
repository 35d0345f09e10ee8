// kda_delta.hip — the gated delta rule with one decay per head, chunked form.
//
// Per (sequence, head), with a 128 x 128 state S (rows = key channels):
//   S~_t = a_t S_{t-1},  u_t = beta_t (v_t - S~_t^T k_t),  S_t = S~_t + k_t u_t^T,  o_t = S_t^T q_t.
// Over a chunk of C tokens with incoming state S, G_i = sum_{j<=i} log a_j,
// B = Diag(beta) and X of the prep kernel (kda_delta_prep.hip):
//   r_i = v_i - e^{G_i} S^T k_i,   u = B (r - X B r)
//   o_i = e^{G_i} S^T q_i + sum_{j<=i} (q_i . k_j) e^{G_i - G_j} u_j
//   S  <- e^{G_C} S + sum_j k_j (e^{G_C - G_j} u_j)^T
// Every exponent that is taken is <= 0, whatever the decays; -inf included.
//
// What is rounded.  The state is an fp32 result, and S^T k, X B r and the
// state's update are what it is made of, and what an output is made of may be
// larger than the output: all products take both fp16 terms of what is not exact
// in one (kda_delta_util.h).  With one term of the state, the pairs and u in bf16
// outputs these were off by 2.4e-3 (norm) instead of their own rounding's 1.7e-3.
// Accumulation is fp32, prefix sums of the decays fp64.
#include <algorithm>

#include "kda.h"
#include "kda_delta_walk.h"

namespace kda {
namespace {

// ---------------------------------------------------------------------------
// The walk.  Eight waves per (sequence or segment, head, 64 value columns),
// meeting at one barrier per chunk: four compute waves, of which wave w owns 16
// value columns and keeps its [128 x 16] slice of the state in matrix-core
// accumulators, and four that prepare the chunks to come (prepare_chunks).  A
// state is a chain of chunks, and 64 columns with all that is prepared for them
// take 146 of the 160 KiB of LDS, so one workgroup fills a compute unit: 96 heads
// fill 192 of 256.
// Bound by the length of a chunk, 6500 cycles, in which matrix cores work 35 %,
// vector instructions issue 58 % and LDS delivers 37 % of the time (96 heads x 8192
// tokens, bf16: 427 us, then 0.97 GB of HBM traffic; of 484 us before the operands'
// order, the compute waves alone took 341 and the preparing ones alone 270).
// Twelve waves, eight of them preparing: 447 us; S^T q after S^T k instead of beside
// it: 471 (446 then); bf16 terms: 536.
// STATES: the segment's own contribution to the state (which = 0) and its
// transition (which = 1: from the identity, without values); M = 2: both, walked
// side by side by the same waves, with the keys read and prepared once.
// SAVE: instead of the outputs, what the backward pass needs (DeltaSaveArgs).
// ---------------------------------------------------------------------------
template <typename E, Walk W, int M = 1>
__device__ __forceinline__ void delta_walk(const DeltaWalkArgs& p, unsigned char* smem, const Item& it, int cb, int which = 0) {
  constexpr bool SAVE = W == Walk::SAVE, PAIRS = W == Walk::OUT || SAVE;
  constexpr int IT = Num<E>::IT, NS = 2;
  constexpr int PT = 2;                        // terms of the pair matrix
  using L = DeltaLayout<E, PT>;
  constexpr int C = L::C, NT = L::NT, ES = L::ES;
  constexpr int KS = C / 32;                   // token steps
  static_assert(L::BYTES <= 160 * 1024, "LDS budget exceeded");
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)smem;
  int* sCol = reinterpret_cast<int*>(smem + L::COL);

  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int H = p.num_heads;
  const Chunks<C, false> ch{it};
  const int h = it.h, hq = h / (H / p.qk_heads), nch = it.nch;
  const size_t nh = (size_t)it.n * H + h;

  if (wv >= 4) {
    const HelperArgs ha{p.q, p.k, p.v, p.blocks, H, p.qk_heads, hq, cb, M == 1 && which == 1};
    return prepare_chunks<E, L, PT, W>(it, smem, ha, wv - 4);
  }

  // ---- compute: the longer of the two (its priority measured 470 -> 446 us, 96 heads x 8192 tokens) ----
  __builtin_amdgcn_s_setprio(2);
  const int vc0 = 16 * wv;                // first value column within the block
  const int col0 = cb * kVW + vc0;        // and within the head
  const int ct = cb * 4 + wv;             // column tile
  constexpr size_t kState = (size_t)D * D;
  // tile rt: rows 16 rt + 4 g + i of column col0 + l16; the state is 2^col_exp times this
  f32x4 accS[M][8];
  int col_exp[M] = {};
  {
    const float* src = nullptr;
    if (W != Walk::STATES) {
      if (p.segmented && !(W == Walk::OUT && p.led && it.first)) {
        // from the scan, the first segment's too: `fin` may be `init`, and a sequence's segments, the last of
        // which writes `fin`, are walked in any order
        src = p.pairs + ((size_t)it.entry * H + h) * 2 * kState;
      } else {
        if (p.init) src = p.init + nh * kState;
        // a first decay that leaves nothing of the state drops it, whatever it holds
        if (src && nch > 0 && exp2_sum((double)fmaxf(p.log_decay[(size_t)it.tb * H + h], kMinLogDecay) * kLog2e) == 0.f)
          src = nullptr;
      }
    }
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int rt = 0; rt < 8; ++rt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 16 * rt + 4 * g + i;
          accS[m][rt][i] = src ? src[row * D + col0 + l16] : which + m == 1 && row == col0 + l16 ? 1.f : 0.f;
        }
  }
  const uint32_t q_at = tile_at<__bf16, D>(l16, 4 * g);
  const uint32_t k_at = tile_at<__bf16, D>(4 * g + (l16 >> 2), 4 * (l16 & 3));
  const uint32_t t_at = tile16_at(l16, g);
  const uint32_t o_row = (uint32_t)H * (D * ES);
  const uint32_t o_at = (uint32_t)l16 * o_row + (uint32_t)((col0 + 4 * g) * ES);
#pragma unroll
  for (int m = 0; m < M; ++m)
    if (g == 0) sCol[m * 64 + wv * 16 + l16] = 0;
  // SAVE: d_o's rows in the outputs' layout, from memory a chunk ahead
  using Raw = std::conditional_t<ES == 2, u32x2, f32x4>;
  Raw d_o[SAVE ? NT : 1];
  auto load_d_o = [&](int ci) {
    if constexpr (SAVE) {
      const Rsrc rs = chunk_rows<E>(p.save.d_o, H, h, ch, ci, D * ES);
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) {
        const int off = (int)(o_at + 16 * rt * o_row);
        if constexpr (ES == 2) d_o[rt] = __builtin_amdgcn_raw_buffer_load_b64(rs, off, 0, 0);
        else d_o[rt] = __builtin_bit_cast(f32x4, buf_ld16(rs, (uint32_t)off, 0));
      }
    }
  };
  load_d_o(0);
  f16x8 ident[2];
  if constexpr (SAVE) {
    ident[0] = identity_h(0, l16, g);
    ident[1] = identity_h(1, l16, g);
  }
  auto store_state = [&](float* to, int m) {
#pragma unroll
    for (int rt = 0; rt < 8; ++rt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        to[(16 * rt + 4 * g + i) * D + col0 + l16] = __builtin_amdgcn_ldexpf(accS[m][rt][i], col_exp[m]);
  };
  chunk_barrier();
  chunk_barrier();

  for (int ci = 0; ci < nch; ++ci) {
    chunk_barrier();
    const int b = ci % 3, b2 = ci & 1;
    const uint32_t base = lds0 + (uint32_t)b2 * L::SET;
    const uint32_t vbase = lds0 + L::VALS + b * L::VTILE;
    const uint32_t x_at = as_is(lds0 + L::XS + b * L::XBYTES + t_at);
    const uint32_t p_at = as_is(lds0 + L::PAIR + b2 * (PT * L::PTERM) + t_at);
    const unsigned char* factors = smem + L::XS + b * L::XBYTES;
    const float* sRow = reinterpret_cast<const float*>(factors + L::ROW);
    const float* sKRow = reinterpret_cast<const float*>(factors + (SAVE ? L::ROW : L::BROW));
    const float* sWgt = reinterpret_cast<const float*>(factors + L::WGT);
    const float* sBeta = reinterpret_cast<const float*>(factors + L::BETA);
    const float gam = *reinterpret_cast<const float*>(factors + L::GAM);
    const int* sExp = reinterpret_cast<const int*>(smem + L::EXPS) + b2 * C;

    // keys and queries of channel steps ks and ks + 1 are held at a time
    f16x8 fk[2][NT][IT], fq[2][PAIRS ? NT : 1][IT];
    auto read_kq = [&](int ks) {
#pragma unroll
      for (int rt = 0; rt < NT; ++rt)
#pragma unroll
        for (int t = 0; t < IT; ++t) fk[ks & 1][rt][t] = ld_row_h(base + L::K + t * L::HALF + q_at, 32 * ks, 16 * rt);
      if constexpr (PAIRS)
#pragma unroll
        for (int rt = 0; rt < NT; ++rt)
#pragma unroll
          for (int t = 0; t < IT; ++t)
            fq[ks & 1][rt][t] = ld_row_h(base + L::Q + t * L::HALF + q_at, 32 * ks, 16 * rt);
    };
    read_kq(0);
    // beta v (SAVE: v): rows 16 rt + 4 g + i of this lane's column
    f32x4 val[NT], beta[NT];
    auto read_beta = [&] {
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) beta[rt] = *reinterpret_cast<const f32x4*>(sBeta + 16 * rt + 4 * g);
    };
    read_beta();
    read_column<E, L>(val, vbase, vc0, l16, g);
    if constexpr (!SAVE)
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) val[rt] *= beta[rt];
    bool live;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      // the columns' scale
      float ms = 0.f, mv = 0.f;
#pragma unroll
      for (int rt = 0; rt < 8; ++rt)
#pragma unroll
        for (int i = 0; i < 4; ++i) ms = fmaxf(ms, fabsf(accS[m][rt][i]));
      if (m == 0)
#pragma unroll
        for (int rt = 0; rt < NT; ++rt)
#pragma unroll
          for (int i = 0; i < 4; ++i) mv = fmaxf(mv, fabsf(SAVE ? beta[rt][i] * val[rt][i] : val[rt][i]));
      const int e = column_exp(ms, col_exp[m], mv, 0);
      live = e > kNoExp;
      const bool off = live && (e - col_exp[m] > kMostExp || e - col_exp[m] < kLeastExp);
      if (__ballot(off)) {
        const int de = off ? e - col_exp[m] - kScaledExp : 0;
        col_exp[m] += de;
#pragma unroll
        for (int rt = 0; rt < 8; ++rt)
#pragma unroll
          for (int i = 0; i < 4; ++i) accS[m][rt][i] = __builtin_amdgcn_ldexpf(accS[m][rt][i], -de);
        if (g == 0) sCol[m * 64 + wv * 16 + l16] = col_exp[m];
      }
    }
#pragma unroll
    for (int rt = 0; rt < NT; ++rt)
#pragma unroll
      for (int i = 0; i < 4; ++i) val[rt][i] = __builtin_amdgcn_ldexpf(val[rt][i], -col_exp[0]);
    const size_t unit = (size_t)ch.slot(ci) * H + h;
    const i32x4 ce = *reinterpret_cast<const i32x4*>(sCol + wv * 16 + 4 * g);

    __builtin_amdgcn_sched_barrier(0);
    // S^T k and S^T q.  Each region below first issues the LDS reads of the next one.
    f32x4 accX[M][NT], accO[NT];
#pragma unroll
    for (int rt = 0; rt < NT; ++rt) {
      accO[rt] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int m = 0; m < M; ++m) accX[m][rt] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }
    f16x8 fs[M][2][NS], fx[NT][KS][NS];
    f32x4 krow[NT];
    auto read_x = [&] {
#pragma unroll
      for (int rt = 0; rt < NT; ++rt)
#pragma unroll
        for (int s = 0; s <= rt / 2; ++s)
#pragma unroll
          for (int t = 0; t < NS; ++t) fx[rt][s][t] = ld_tiles(x_at + t * L::XTERM, rt, s);
    };
#pragma unroll
    for (int m = 0; m < M; ++m) split_op(fs[m][0], accS[m][0], accS[m][1]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      if (ks < 3) {
        read_kq(ks + 1);
#pragma unroll
        for (int m = 0; m < M; ++m) split_op(fs[m][(ks + 1) & 1], accS[m][2 * ks + 2], accS[m][2 * ks + 3]);
      } else {
#pragma unroll
        for (int rt = 0; rt < NT; ++rt) krow[rt] = *reinterpret_cast<const f32x4*>(sKRow + 16 * rt + 4 * g);
        // (not held through the products above: registers)
        asm volatile("" ::: "memory");
        read_beta();
        read_x();
      }
      if constexpr (SAVE) store_turned((const E*)nullptr, p.save.s, unit, ct, ks, fs[0][ks & 1][0], accS[0], ident, ce, lane);
#pragma unroll
      for (int rt = 0; rt < NT; ++rt)
#pragma unroll
        for (int m = 0; m < M; ++m) accX[m][rt] = mma_terms(accX[m][rt], fk[ks & 1][rt], fs[m][ks & 1]);
      if constexpr (PAIRS)
#pragma unroll
        for (int rt = 0; rt < NT; ++rt) accO[rt] = mma_terms(accO[rt], fs[0][ks & 1], fq[ks & 1][rt]);
      if constexpr (ES == 2 && W == Walk::OUT) mix<16, 4 * NT, 2>();
      else __builtin_amdgcn_sched_barrier(0);
    }
    // B r (SAVE: r), then u = B r - B X (B r); (the block holds -X)
    f16x8 fp[PAIRS ? NT : 1][KS][PT];
    auto read_pairs = [&] {
      if constexpr (PAIRS)
#pragma unroll
        for (int rt = 0; rt < NT; ++rt)
#pragma unroll
          for (int s = 0; s <= rt / 2; ++s)
#pragma unroll
            for (int t = 0; t < PT; ++t) fp[rt][s][t] = ld_tiles(p_at + t * L::PTERM, rt, s);
    };
#pragma unroll
    for (int rt = 0; rt < NT; ++rt) {
      const f32x4 fk = Num<E>::KEXP ? exp2i(-Num<E>::KEXP) * krow[rt] : krow[rt];
      accX[0][rt] = val[rt] - fk * accX[0][rt];
      if constexpr (M == 2) accX[1][rt] *= -fk;
    }
    f16x8 fr[M][KS][NS];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        if constexpr (SAVE) split_op(fr[m][s], beta[2 * s] * accX[m][2 * s], beta[2 * s + 1] * accX[m][2 * s + 1]);
        else split_op(fr[m][s], accX[m][2 * s], accX[m][2 * s + 1]);
      }
    __builtin_amdgcn_sched_barrier(0);
    // the state's update takes the keys by columns
    f16x8 fc[8][IT];
    auto read_cols = [&](int s, int first, int count) {
#pragma unroll
      for (int rt = 0; rt < 8; ++rt)
        if (rt >= first && rt < first + count)
#pragma unroll
          for (int t = 0; t < IT; ++t) fc[rt][t] = ld_col_h(base + L::K + t * L::HALF, k_at, 16 * rt, 32 * s);
    };
    f32x4 wgt[NT];
#pragma unroll
    for (int rt = 0; rt < NT; ++rt) {
      wgt[rt] = *reinterpret_cast<const f32x4*>(sWgt + 16 * rt + 4 * g);
      if constexpr (Num<E>::KEXP) wgt[rt] *= exp2i(-Num<E>::KEXP);
    }
    f32x4 accZ[M][NT];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) accZ[m][rt] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int rt = 2 * s; rt < NT; ++rt)
#pragma unroll
        for (int m = 0; m < M; ++m) accZ[m][rt] = mma_terms(accZ[m][rt], fx[rt][s], fr[m][s]);
    if constexpr (PAIRS)
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) accO[rt] *= sRow[16 * rt + l16];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int rt = 0; rt < 8; ++rt) accS[m][rt] *= gam;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int rt = 0; rt < NT; ++rt) {
      if constexpr (SAVE) {
        // e = r - X B r, as it is; then u
        accX[0][rt] += accZ[0][rt];
        f32x4 e;
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = __builtin_amdgcn_ldexpf(accX[0][rt][i], col_exp[0]);
        __builtin_nontemporal_store(e, reinterpret_cast<f32x4*>(p.save.e) + (unit * 8 + ct) * (NT * 64) + rt * 64 + lane);
        accX[0][rt] *= beta[rt];
      } else {
#pragma unroll
        for (int m = 0; m < M; ++m) accX[m][rt] += beta[rt] * accZ[m][rt];
      }
    }
    read_pairs();
    f16x8 fw[M][KS][NS];
    if constexpr (PAIRS) {
      // outputs, transposed: lane = token, four consecutive value columns
      f16x8 fe[KS][NS];
#pragma unroll
      for (int s = 0; s < KS; ++s) split_op(fe[s], accX[0][2 * s], accX[0][2 * s + 1]);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (SAVE) {
        // u, turned over likewise
        const Rsrc rs = chunk_rows<E>(p.save.u, H, h, ch, ci, D * ES);
#pragma unroll
        for (int rt = 0; rt < NT; ++rt) {
          if constexpr (ES == 2) {
            store_cols_h(rs, (int)(o_at + 16 * rt * o_row), mma_h((f32x4){0.f, 0.f, 0.f, 0.f}, fe[rt / 2][0], ident[rt & 1]));
          } else {
            Frag16<float> f;
            f.v = accX[0][rt];
            store_cols<E>(rs, (int)(o_at + 16 * rt * o_row), turn(f), ce);
          }
        }
        if (ES == 2 && g == 0) p.save.exps[unit * D + col0 + l16] = live ? col_exp[0] : kNoExp;
      }
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int rt = 2 * s; rt < NT; ++rt) accO[rt] = mma_terms(accO[rt], fe[s], fp[rt][s]);
    }
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int s = 0; s < KS; ++s) split_op(fw[m][s], wgt[2 * s] * accX[m][2 * s], wgt[2 * s + 1] * accX[m][2 * s + 1]);
    read_cols(0, 0, 8);
    __builtin_amdgcn_sched_barrier(0);
    // the state
#pragma unroll
    for (int rt = 0; rt < 8; ++rt)
#pragma unroll
      for (int m = 0; m < M; ++m) accS[m][rt] = mma_terms(accS[m][rt], fc[rt], fw[m][0]);
    if constexpr (KS == 2) {
      read_cols(1, 0, 8);
      if constexpr (IT == 1) {
        // (as the first step's keys come free)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, M * NS, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int rt = 0; rt < 8; ++rt)
#pragma unroll
        for (int m = 0; m < M; ++m) accS[m][rt] = mma_terms(accS[m][rt], fc[rt], fw[m][1]);
    }
    if constexpr (W == Walk::OUT) {
      const Rsrc rs = chunk_rows<E>(p.o, H, h, ch, ci, D * ES);
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) store_cols<E>(rs, (int)(o_at + 16 * rt * o_row), accO[rt], ce + sExp[16 * rt + l16]);
    }
    if constexpr (SAVE) {
      // o . d_o over this wave's columns
      float dot[NT];
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) {
        Frag16<E> f;
        f.v = __builtin_bit_cast(decltype(f.v), d_o[rt]);
        const f32x4 x = frag16_to_f32(f);
        const int eq = sExp[16 * rt + l16];
        dot[rt] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) dot[rt] += x[i] * __builtin_amdgcn_ldexpf(accO[rt][i], ce[i] + eq);
      }
      int tile;
      const float sum = sum_groups(dot, g, tile);
      if (p.save.change && tile >= 0 && 16 * tile + l16 < ch.rows(ci))
        p.save.change[((size_t)ct * H + h) * p.total_tokens + ch.begin(ci) + 16 * tile + l16] = sum;
      load_d_o(ci + 1);
      // the state at the boundaries of the decays' gradient
      const int64_t done = min(ch.begin(ci) + C, it.te) - it.bos;
      const bool at_end = done == it.eos - it.bos;
      if (p.save.anchors && (at_end ? p.save.end_state : done % p.save.anchor == 0)) {
        const int64_t j = (done + p.save.anchor - 1) / p.save.anchor;
        store_state(p.save.anchors + ((size_t)boundary_of(it.n, it.bos, p.save.anchor, p.save.end_state, j) * H + h) * kState, 0);
      }
    }
  }
  if constexpr (W == Walk::STATES) {
#pragma unroll
    for (int m = 0; m < M; ++m) store_state(p.pairs + (((size_t)it.slot * H + h) * 2 + which + m) * kState, m);
  } else if (!it.last) {
    // (the first segment's, walked before the scan, which goes on from it)
    if (W == Walk::OUT && p.led && it.first) store_state(p.pairs + ((size_t)it.slot * H + h) * 2 * kState, 0);
  } else if (p.fin) {
    store_state(p.fin + nh * kState, 0);
  }
}

template <typename E>
__global__ __launch_bounds__(kWalkThreads) void delta_walk_kernel(const DeltaWalkArgs p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  int part;
  const int64_t u = delta_unit<2>(p.unit0, p.num_heads, p.qk_heads, blockIdx.x, part);
  if (u >= p.units) return;
  const Item it = find_item<delta_chunk(sizeof(E) == 2)>(p, smem, u);
  if (it.ok && !(p.led && it.first)) delta_walk<E, Walk::OUT>(p, smem, it, part);
}

// What comes before the scan over segments: contributions and transitions, which
// the last segments do without; and, where that is wanted, the first segments'
// outputs.
template <typename E, int M>
__global__ __launch_bounds__(kWalkThreads) void delta_pairs_kernel(const DeltaWalkArgs p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  int part;
  const int64_t u = delta_unit<4 / M>(p.unit0, p.num_heads, p.qk_heads, blockIdx.x, part);
  if (u >= p.units) return;
  const Item it = find_item<delta_chunk(sizeof(E) == 2)>(p, smem, u);
  if (!it.ok) return;
  const int cb = part & 1, which = part >> 1;
  if (p.led && it.first) {
    if (which == 0) delta_walk<E, Walk::OUT>(p, smem, it, cb);
  } else if (p.all_pairs || !it.last) {
    delta_walk<E, Walk::STATES, M>(p, smem, it, cb, which);
  }
}

template <typename E>
__global__ __launch_bounds__(kWalkThreads) void delta_save_kernel(const DeltaWalkArgs p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  int part;
  const int64_t u = delta_unit<2>(p.unit0, p.num_heads, p.qk_heads, blockIdx.x, part);
  if (u >= p.units) return;
  const Item it = find_item<delta_chunk(sizeof(E) == 2)>(p, smem, u);
  if (it.ok) delta_walk<E, Walk::SAVE>(p, smem, it, part);
}

template <typename E>
hipError_t launch_walk_e(const DeltaWalkArgs& a, hipStream_t stream) {
  constexpr int LDS = DeltaLayout<E, 2>::BYTES;
  static std::atomic<bool> set[64];
  const hipError_t e = allow_lds(delta_walk_kernel<E>, LDS, set);
  if (e != hipSuccess) return e;
  return launch_delta_parts<2>(a, [&](const DeltaWalkArgs& part, unsigned blocks) {
    hipLaunchKernelGGL(delta_walk_kernel<E>, dim3(blocks), dim3(kWalkThreads), LDS, stream, part);
  });
}

template <typename E, int M>
hipError_t launch_pairs_e(const DeltaWalkArgs& a, hipStream_t stream) {
  constexpr int LDS = DeltaLayout<E, 2>::BYTES;
  static std::atomic<bool> set[64];
  const hipError_t e = allow_lds(delta_pairs_kernel<E, M>, LDS, set);
  if (e != hipSuccess) return e;
  return launch_delta_parts<4 / M>(a, [&](const DeltaWalkArgs& part, unsigned blocks) {
    hipLaunchKernelGGL((delta_pairs_kernel<E, M>), dim3(blocks), dim3(kWalkThreads), LDS, stream, part);
  });
}

template <typename E>
hipError_t launch_save_e(const DeltaWalkArgs& a, hipStream_t stream) {
  constexpr int LDS = DeltaLayout<E, 2>::BYTES;
  static std::atomic<bool> set[64];
  const hipError_t e = allow_lds(delta_save_kernel<E>, LDS, set);
  if (e != hipSuccess) return e;
  return launch_delta_parts<2>(a, [&](const DeltaWalkArgs& part, unsigned blocks) {
    hipLaunchKernelGGL(delta_save_kernel<E>, dim3(blocks), dim3(kWalkThreads), LDS, stream, part);
  });
}

// ---------------------------------------------------------------------------
// Incoming state of every segment, S_in(j+1) = M_j S_in(j) + B_j, by column
// tiles of 16 (a state's columns evolve on their own).  One workgroup of four
// waves per (sequence, head, column tile); wave w owns row tiles 2 w and 2 w + 1
// in the layout of an fp32 result tile, which is the next product's operand;
// the 128 x 16 tile goes through LDS after each step, and the next segment's M
// and B are fetched while one step runs.  S_in(j+1) takes B_j's place; that of
// segment 1 is there already where the first segments have been walked (led), else
// S_in(0), which the walk reads here as `fin` may be `init`, takes the place of the
// last segment's contribution, which nothing reads.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void delta_scan_kernel(const DeltaScanArgs a) {
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
  const int from = a.led ? 1 : 0;
  if (a.led && count <= from + 1) return;
  const int64_t base = slot_of(n, bos, a.seg, 0);
  auto pair = [&](int j) { return a.pairs + ((size_t)(base + j) * H + h) * 2 * kState; };
  __shared__ f32x4 sS[8][64];
  auto row_of = [&](int q, int i) { return 16 * (2 * wv + q) + 4 * g + i; };
  const float* start = a.led ? pair(0) : a.init ? a.init + (size_t)nh * kState : nullptr;
  // (the first decay may drop the state, whatever it holds)
  if (!a.led && count > 0 && exp2_sum((double)fmaxf(a.log_decay[(size_t)bos * H + h], kMinLogDecay) * kLog2e) == 0.f)
    start = nullptr;
  float* entry = pair(max(count, 1) - 1);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    f32x4 s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i] = start ? start[row_of(q, i) * D + col] : 0.f;
      if (!a.led) entry[row_of(q, i) * D + col] = s[i];
    }
    sS[2 * wv + q][lane] = s;
  }
  if (count <= from + 1) return;
  __syncthreads();
  Frag16<float> mf[2][8];
  f32x4 bj[2];
  auto fetch = [&](int j) {
    const float* Bj = pair(j);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
      for (int kt = 0; kt < 8; ++kt)
        ld_frag16(mf[q][kt], Bj + kState + (size_t)(16 * (2 * wv + q) + l16) * D + 16 * kt + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) bj[q][i] = Bj[row_of(q, i) * D + col];
    }
  };
  fetch(from);
  for (int j = from; j + 1 < count; ++j) {  // (the last segment forms neither)
    float* Bj = pair(j);
    f32x4 acc[2];
    Frag16<float> mcur[2][8];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      acc[q] = bj[q];
#pragma unroll
      for (int kt = 0; kt < 8; ++kt) mcur[q][kt] = mf[q][kt];
    }
    if (j + 2 < count) fetch(j + 1);
#pragma unroll
    for (int kt = 0; kt < 8; ++kt) {
      Frag16<float> sf;
      sf.v = sS[kt][lane];
#pragma unroll
      for (int q = 0; q < 2; ++q) acc[q] = mma16(acc[q], mcur[q][kt], sf);
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      sS[2 * wv + q][lane] = acc[q];
#pragma unroll
      for (int i = 0; i < 4; ++i) Bj[row_of(q, i) * D + col] = acc[q][i];
    }
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_delta_walk(DeltaWalkArgs a, hipStream_t stream) {
  return a.bf16 ? launch_walk_e<__bf16>(a, stream) : launch_walk_e<float>(a, stream);
}

hipError_t launch_delta_pairs(DeltaWalkArgs a, hipStream_t stream) {
  if (a.both) return a.bf16 ? launch_pairs_e<__bf16, 2>(a, stream) : launch_pairs_e<float, 2>(a, stream);
  return a.bf16 ? launch_pairs_e<__bf16, 1>(a, stream) : launch_pairs_e<float, 1>(a, stream);
}

hipError_t launch_delta_save(DeltaWalkArgs a, hipStream_t stream) {
  return a.bf16 ? launch_save_e<__bf16>(a, stream) : launch_save_e<float>(a, stream);
}

hipError_t launch_delta_scan(DeltaScanArgs a, hipStream_t stream) {
  const int64_t units = (int64_t)a.num_seqs * a.num_heads;
  constexpr int64_t MOST = kMaxThreads / 256 / 8;
  for (int64_t u = 0; u < units; u += MOST) {
    a.unit0 = u;
    hipLaunchKernelGGL(delta_scan_kernel, dim3((unsigned)(std::min(units - u, MOST) * 8)), dim3(256), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace kda
