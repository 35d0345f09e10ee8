// kda_delta_walk.h — the walk of a state of the gated delta rule over the chunks
// of a sequence or segment: its LDS, and the roles of the waves that prepare
// chunks for the compute waves (kda_delta.hip forwards, kda_delta_bwd.hip
// backwards in time).
#pragma once

#include <algorithm>
#include <type_traits>

#include "kda_delta_util.h"

namespace kda {
namespace {

constexpr int kVW = 64;        // value columns of a workgroup: half a head
constexpr int kWalkThreads = 64 * 8;

// PT: terms of the pair matrix.
template <typename E, int PT>
struct DeltaLayout {
  static constexpr int ES = (int)sizeof(E);
  static constexpr int C = 128 / ES, NT = C / 16, TILES = delta_tiles(C);
  static constexpr int HALF = C * D * 2;                     // one term of a key or query tile
  static constexpr int TILE = HALF * Num<E>::IT;
  static constexpr int K = 0, Q = TILE, SET = 2 * TILE;      // [2] sets
  static constexpr int VTILE = C * kVW * ES;
  static constexpr int VALS = 2 * SET;                       // [3] value tiles
  static constexpr int XTERM = TILES * kDeltaTileBytes;
  static constexpr int XBYTES = delta_block_bytes(C);
  static constexpr int XS = VALS + 3 * VTILE;                // [3] blocks of the prep kernel
  static constexpr int SUM = delta_matrix_bytes(C);          // and in them: float [2][C] prefix sums,
  static constexpr int ROW = SUM + 2 * C * 4;                // [C] e^{G_i},
  static constexpr int WGT = ROW + C * 4;                    // [C] e^{G_C - G_j},
  static constexpr int BETA = WGT + C * 4;                   // [C] beta,
  static constexpr int BROW = BETA + C * 4;                  // [C] beta e^{G_i},
  static constexpr int GAM = BROW + C * 4;                   // e^{G_C}
  static constexpr int PTERM = TILES * kDeltaTileBytes;
  static constexpr int PAIR = XS + 3 * XBYTES;               // [2][PT] pair matrices
  static constexpr int COL = PAIR + 2 * PT * PTERM;          // int [2][4][16] exponents of the states' columns
  static constexpr int EXPS = COL + 2 * 4 * 16 * 4;          // int [2][C] exponents of the queries
  static constexpr int SYNC = EXPS + 2 * C * 4;              // int: rows converted
  static constexpr int BYTES = SYNC + 16;
};

// The scaled maximum of a column of the state and of beta v is kept from 2 to
// 2^8 and set to 2^5 .. 2^6 when it leaves that: u then stays below 2^15 for keys
// of unit length (|S| + 64 |beta v| at most), and the lo terms' smallest step is
// 2^-25 of the maximum.
constexpr int kMostExp = 8, kLeastExp = 2;  // (2^(e - 1) .. 2^e)
constexpr int kScaledExp = 6;
constexpr int kNoExp = -1000;  // of a column of zeros, where the walks note exponents
// Rows of q are scaled to 2^(kQueryExp - 1) .. 2^kQueryExp, so that the second terms
// of the pairs are normal numbers in fp16.  (The backward walk divides the gradients
// it multiplies with q by their scale.)
constexpr int kQueryExp = 8, kQueryExpBack = 2;

// Exponent of a column: of the largest of the state, held as 2^col_exp times s,
// and of the values, v times 2^more; kNoExp: all are zero.  (Exponents, as one side
// may be out of the other's range.)
__device__ __forceinline__ int column_exp(float s, int col_exp, float v, int more) {
  const int es = s > 0.f ? __builtin_amdgcn_frexp_expf(s) + col_exp : kNoExp;
  const int ev = v > 0.f ? __builtin_amdgcn_frexp_expf(v) + more : kNoExp;
  return (int)max_groups((float)max(es, ev));
}

typedef int i32x4 __attribute__((ext_vector_type(4)));

// What a walk is for.
enum class Walk {
  OUT,     // forwards: outputs
  STATES,  // forwards: a segment's own contribution to the state, or its transition
  SAVE,    // forwards: what the backward pass needs of a chunk
  BACK,    // backwards: gradients
  BACK_STATES,
};
constexpr bool is_back(Walk w) { return w == Walk::BACK || w == Walk::BACK_STATES; }

// A (sequence or segment, head): tokens [tb, te) of sequence n = [bos, eos).
struct Item {
  int h, n;
  int64_t bos, eos, tb, te, slot;
  int64_t entry;     // segments: the slot in which delta_scan_kernel leaves the state that enters this one
  bool first, last;  // it begins / ends its sequence
  bool ok;
  int nch;           // chunks
};
template <int C, typename A>
__device__ __forceinline__ Item find_item(const A& p, unsigned char* smem, int64_t u) {
  Item it;
  const int H = p.num_heads;
  it.h = (int)(u % H);
  const int64_t rank = u / H;
  it.ok = true;
  if (p.segmented) {
    const Segment s = find_segment(p.cu, p.num_seqs, p.total_tokens, p.seg, rank);
    it.ok = s.ok;
    it.n = s.n;
    it.bos = s.bos;
    it.eos = s.eos;
    it.slot = rank;
    it.tb = s.bos + (int64_t)s.j * p.seg;
    it.te = min(s.eos, it.tb + p.seg);
    it.first = s.j == 0;
    it.last = s.j + 1 >= s.count;
    it.entry = it.first ? rank + max(s.count, 1) - 1 : rank - 1;
  } else {
    it.n = longest_first<kWalkThreads>(reinterpret_cast<int*>(smem), p.cu, p.num_seqs, p.total_tokens, (int)rank);
    seq_range(p.cu, it.n, p.total_tokens, it.bos, it.eos);
    it.slot = it.entry = 0;
    it.tb = it.bos;
    it.te = it.eos;
    it.first = it.last = true;
  }
  it.nch = (int)((it.te - it.tb + C - 1) / C);
  return it;
}

// Chunk number ci of a walk: where it begins, its rows, and its slot.
template <int C, bool REV>
struct Chunks {
  const Item& it;
  __device__ __forceinline__ int of(int ci) const { return REV ? it.nch - 1 - ci : ci; }
  __device__ __forceinline__ int64_t begin(int ci) const { return it.tb + (int64_t)of(ci) * C; }
  __device__ __forceinline__ int rows(int ci) const { return (int)min((int64_t)C, it.te - begin(ci)); }
  __device__ __forceinline__ int64_t slot(int ci) const { return it.bos / C + it.n + (it.tb - it.bos) / C + of(ci); }
};

// Rows of a [T, heads, 128] tensor, one head, from a chunk's first on; a chunk
// behind the walk's end is an empty view.
template <typename E, typename CH>
__device__ __forceinline__ Rsrc chunk_rows(const void* src, int heads, int head, const CH& ch, int ci, int bytes) {
  const uint32_t stride = (uint32_t)heads * (D * (int)sizeof(E));
  return make_rsrc(static_cast<const char*>(src) + (size_t)ch.begin(ci) * stride + (size_t)head * (D * sizeof(E)),
                   ci < ch.it.nch ? (uint32_t)(ch.rows(ci) - 1) * stride + bytes : 0);
}

// Four consecutive columns (16 kt + 4 g ..) of row 16 rt + l16 of a matrix in tiles.
template <int PT>
__device__ __forceinline__ void store_pair(unsigned char* tiles, int term, int rt, int kt, int l16, int g, f32x4 x) {
  uint32_t a[PT], b[PT];
  split2<PT>(a, x[0], x[1]);
  split2<PT>(b, x[2], x[3]);
#pragma unroll
  for (int t = 0; t < PT; ++t)
    *reinterpret_cast<u32x2*>(tiles + t * term + tile_no(rt, kt) * kDeltaTileBytes + tile16_at(l16, g)) =
        (u32x2){a[t], b[t]};
}

struct HelperArgs {
  const void* q;
  const void* k;
  const void* vals;         // the tensor of the value tiles
  const char* blocks;       // the prep kernel's
  int heads, qk_heads, hq, cb;
  bool no_values;
};

// ---- The four waves that prepare chunks, where conversions, scales and pairs would
// wait in turn with the compute waves' products (270 us of their own, 96 heads x 8192
// tokens; rows loaded one chunk ahead instead of two: a walk of 484 us was 536).  In iteration ci (from -2), meeting
// the compute waves, which work on chunk ci, at its beginning, each takes a
// quarter of
//   the keys' and queries' rows of chunk ci + 1, from registers that were loaded
//   two iterations before, into LDS as fp16;
//   the copies of the value tile and the prep kernel's block of chunk ci + 2
//   straight into LDS;
//   and, once all four have their rows in place, the tiles of chunk ci + 1's pair
//   matrix (keys in rows: lane = query, four consecutive keys).
// ----
template <typename E, typename L, int PT, Walk W>
__device__ __forceinline__ void prepare_chunks(const Item& it, unsigned char* smem, const HelperArgs& p, int hw) {
  constexpr int C = L::C, NT = L::NT, ES = L::ES, IT = Num<E>::IT;
  constexpr bool PAIRS = W != Walk::STATES;
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)smem;
  const Chunks<C, is_back(W)> ch{it};
  const int nch = it.nch;
  int* sSync = reinterpret_cast<int*>(smem + L::SYNC);

  // copies of 1 KiB, 16 bytes a lane; rows behind the end lie outside the buffer
  // views and arrive as zeros
  constexpr int VP = L::VTILE / 1024 / 4, XP = (L::XBYTES / 1024 + 3) / 4;
  auto copy = [&](int ci) {
    const uint32_t stride = (uint32_t)p.heads * (D * ES);
    unsigned char* dst = smem + L::VALS + (ci % 3) * L::VTILE;
    const Rsrc rs = make_rsrc(static_cast<const char*>(p.vals) + (size_t)ch.begin(ci) * stride +
                                  ((size_t)it.h * D + (size_t)p.cb * kVW) * ES,
                              p.no_values ? 0 : (uint32_t)(ch.rows(ci) - 1) * stride + kVW * ES);
    constexpr int UR = kVW * ES / 16, RP = 64 / UR;
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      const int piece = hw * VP + i, row = piece * RP + lane / UR;
      const uint32_t unit = (uint32_t)(((lane % UR) ^ swizzle<E, kVW>(row)) * 16);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)(dst + piece * 1024), 16,
                                               (int)((uint32_t)row * stride + unit), 0, 0, 0);
    }
    const Rsrc rx = make_rsrc(p.blocks + ((size_t)ch.slot(ci) * p.heads + it.h) * L::XBYTES, L::XBYTES);
    unsigned char* dx = smem + L::XS + (ci % 3) * L::XBYTES;
#pragma unroll
    for (int i = 0; i < XP; ++i) {
      // (the same number of copies in every wave: the last ones twice)
      const int piece = min(hw * XP + i, L::XBYTES / 1024 - 1);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (__attribute__((address_space(3))) void*)(dx + piece * 1024), 16,
                                               piece * 1024 + lane * 16, 0, 0, 0);
    }
  };

  // rows
  constexpr int UR = D * ES / 16, RP = 64 / UR;   // lanes per row, rows per load
  constexpr int LOADS = C / 4 / RP;
  const int row0 = hw * (C / 4) + lane / UR;
  const uint32_t qk_stride = (uint32_t)p.qk_heads * (D * ES);
  u32x4 raw_k[2][LOADS], raw_q[2][LOADS];         // of even and odd chunks
  auto load_rows = [&](u32x4 (&raw)[LOADS], const void* src, int ci) {
    const Rsrc rs = chunk_rows<E>(src, p.qk_heads, p.hq, ch, ci, D * ES);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) raw[i] = buf_ld16(rs, (uint32_t)(row0 + i * RP) * qk_stride + (lane % UR) * 16, 0);
  };
  auto put_row = [&](unsigned char* dst, int row, const float (&x)[16 / ES]) {
    if constexpr (ES == 2) {
      uint32_t y[4][1];
#pragma unroll
      for (int j = 0; j < 4; ++j) split2<1>(y[j], x[2 * j], x[2 * j + 1]);
      *reinterpret_cast<u32x4*>(dst + tile_at<__bf16, D>(row, 8 * (lane % UR))) = (u32x4){y[0][0], y[1][0], y[2][0], y[3][0]};
    } else {
      uint32_t a[2], b[2];
      split2<2>(a, x[0], x[1]);
      split2<2>(b, x[2], x[3]);
#pragma unroll
      for (int t = 0; t < 2; ++t)
        *reinterpret_cast<u32x2*>(dst + t * L::HALF + tile_at<__bf16, D>(row, 4 * (lane % UR))) = (u32x2){a[t], b[t]};
    }
  };
  auto values_of = [&](float (&x)[16 / ES], const u32x4& raw) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w = raw[j];  // (a bit cast of the element itself reads the first one)
      if constexpr (ES == 2) {
        x[2 * j] = __builtin_bit_cast(float, w << 16);
        x[2 * j + 1] = __builtin_bit_cast(float, w & 0xffff0000u);
      } else {
        x[j] = __builtin_bit_cast(float, w);
      }
    }
  };
  auto put_keys = [&](const u32x4 (&raw)[LOADS], unsigned char* dst) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      float x[16 / ES];
      values_of(x, raw[i]);
      if constexpr (Num<E>::KEXP)
#pragma unroll
        for (float& y : x) y *= exp2i(Num<E>::KEXP);
      put_row(dst, row0 + i * RP, x);
    }
  };
  auto put_queries = [&](const u32x4 (&raw)[LOADS], unsigned char* dst, int* exps) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      float x[16 / ES];
      values_of(x, raw[i]);
      float m = fabsf(x[0]);
#pragma unroll
      for (int j = 1; j < 16 / ES; ++j) m = fmaxf(m, fabsf(x[j]));
      m = max_row(m);
      if constexpr (UR == 32) m = fmaxf(m, __shfl_xor(m, 16));
      const int e = m > 0.f ? __builtin_amdgcn_frexp_expf(m) - (is_back(W) ? kQueryExpBack : kQueryExp) : 0;
      if (lane % UR == 0) exps[row0 + i * RP] = e;
#pragma unroll
      for (float& y : x) y = __builtin_amdgcn_ldexpf(y, -e);
      put_row(dst, row0 + i * RP, x);
    }
  };

  // a tile of the pair matrix
  const uint32_t r_at = tile_at<__bf16, D>(l16, 8 * g);
  auto put_pair = [&](int c, int rt, int kt) {
    const uint32_t base = lds0 + (uint32_t)(c & 1) * L::SET + r_at;
    const float* gs = reinterpret_cast<const float*>(smem + L::XS + (c % 3) * L::XBYTES + L::SUM);
    auto ld = [&](uint32_t at, int row, int ks) {
      Frag<__bf16> f;
      ld_row(f, at + row * (D * 2), 32 * ks);
      return __builtin_bit_cast(f16x8, f.v);
    };
    f16x8 fq[4][IT], fk[4][IT];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
      for (int t = 0; t < IT; ++t) {
        fq[ks][t] = ld(base + L::Q + t * L::HALF, 16 * rt, ks);
        fk[ks][t] = ld(base + L::K + t * L::HALF, 16 * kt, ks);
      }
    const float gq = gs[16 * rt + l16], gq_lo = gs[C + 16 * rt + l16];
    const f32x4 gk = *reinterpret_cast<const f32x4*>(gs + 16 * kt + 4 * g);
    const f32x4 gk_lo = *reinterpret_cast<const f32x4*>(gs + C + 16 * kt + 4 * g);
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) acc = mma_terms(acc, fk[ks], fq[ks]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool on = kt < rt || 4 * g + i <= l16;
      const float d = (gq - gk[i]) + (gq_lo - gk_lo[i]);
      float x = acc[i] * exp2_fast(d);
      if constexpr (Num<E>::KEXP) x *= exp2i(-Num<E>::KEXP);
      acc[i] = on ? x : 0.f;
    }
    store_pair<PT>(smem + L::PAIR + (c & 1) * (PT * L::PTERM), L::PTERM, rt, kt, l16, g, acc);
  };

  load_rows(raw_k[0], p.k, 0);
  if constexpr (PAIRS) load_rows(raw_q[0], p.q, 0);
  if (hw == 0 && lane == 0) *sSync = 0;
  int synced = 0;
  // an iteration, with the registers of chunk ci + 1 (par: its parity)
  auto step = [&](int ci, auto par_) {
    constexpr int par = decltype(par_)::value;
    // The copies of chunk ci + 1 have landed, whose factors the pairs take: behind
    // them this wave issued rows only.
    constexpr int ROWS = (PAIRS ? 2 : 1) * LOADS;
    __builtin_amdgcn_s_waitcnt(vmcnt_wait(ROWS));
    chunk_barrier();
    if (ci + 2 < nch) copy(ci + 2);
    const int c = ci + 1;
    if (c >= 0 && c < nch) {
      unsigned char* set = smem + (c & 1) * L::SET;
      put_keys(raw_k[par], set + L::K);
      if constexpr (PAIRS) put_queries(raw_q[par], set + L::Q, reinterpret_cast<int*>(smem + L::EXPS) + (c & 1) * C);
    }
    // (before the first chunk: of the second one)
    load_rows(raw_k[par], p.k, c + 2);
    if constexpr (PAIRS) {
      load_rows(raw_q[par], p.q, c + 2);
      if (c < 0 || c >= nch) return;
      // every wave's rows are in place (each adds one, in every such iteration)
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (lane == 0) __hip_atomic_fetch_add(sSync, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
      synced += 4;
      while (__hip_atomic_load(sSync, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP) < synced)
        __builtin_amdgcn_s_sleep(1);
      asm volatile("" ::: "memory");
      if constexpr (NT == 4) {
        if (hw == 0) {
          put_pair(c, 0, 0);
          put_pair(c, 3, 0);
          put_pair(c, 3, 1);
        } else if (hw == 1) {
          put_pair(c, 1, 0);
          put_pair(c, 1, 1);
          put_pair(c, 3, 2);
        } else if (hw == 2) {
          put_pair(c, 2, 0);
          put_pair(c, 2, 1);
        } else {
          put_pair(c, 2, 2);
          put_pair(c, 3, 3);
        }
      } else {
        if (hw == 0) put_pair(c, 0, 0);
        else if (hw == 1) put_pair(c, 1, 0);
        else if (hw == 2) put_pair(c, 1, 1);
      }
    }
  };
  for (int ci = -2; ci < nch; ci += 2) {
    step(ci, std::integral_constant<int, 1>{});
    if (ci + 1 < nch) step(ci + 1, std::integral_constant<int, 0>{});
  }
}

// Order of a region's instructions: `reads` LDS reads, then n times a matrix
// instruction and v vector ones.  (Left alone the compiler puts every read right
// before its use, and the one compute wave of a SIMD waits for each.)
template <int READS, int M, int V>
__device__ __forceinline__ void mix() {
  if constexpr (READS > 0) __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
#pragma unroll
  for (int i = 0; i < M; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x002, V, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
}

// A chunk's tile of values as four rows 16 rt + 4 g .. of this lane's column
// (vc0 + l16), in fp32.
template <typename E, typename L>
__device__ __forceinline__ void read_column(f32x4 (&x)[L::NT], uint32_t base, int vc0, int l16, int g) {
#pragma unroll
  for (int rt = 0; rt < L::NT; ++rt) {
    if constexpr (L::ES == 2) {
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      const uint32_t at = base + tile_at<E, kVW>(16 * rt + 4 * g + (l16 >> 2), vc0 + 4 * (l16 & 3));
      const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[rt][2 * i] = __builtin_bit_cast(float, y[i] << 16);
        x[rt][2 * i + 1] = __builtin_bit_cast(float, y[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[rt][i] = lds_get<float>(base + tile_at<E, kVW>(16 * rt + 4 * g + i, vc0 + l16));
    }
  }
}

// Operand over 32 tokens, 4 g .. and 16 + 4 g .., of a column block of 16 x 16
// tiles (the transposed matrix's row tile ct): tiles (2 s, ct) and (2 s + 1, ct); at =
// tile16_at(4 g + l16 / 4, l16 % 4).
__device__ __forceinline__ f16x8 ld_tiles_t(uint32_t at, int ct, int s) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  s16x4 a = {0, 0, 0, 0};
  if (2 * s >= ct)
    a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + tile_no(2 * s, ct) * kDeltaTileBytes));
  const s16x4 b =
      __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + tile_no(2 * s + 1, ct) * kDeltaTileBytes));
  const u32x2 x = __builtin_bit_cast(u32x2, a), y = __builtin_bit_cast(u32x2, b);
  return __builtin_bit_cast(f16x8, (u32x4){x[0], x[1], y[0], y[1]});
}

// The identity's columns of token tile `half` (0, 1) of 32 tokens: a product with
// it turns a result's rows and columns over.
__device__ __forceinline__ f16x8 identity_h(int half, int l16, int g) {
  f16x8 f;
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = (_Float16)((j >> 2) == half && 4 * g + (j & 3) == l16 ? 1.f : 0.f);
  return f;
}

// Four value columns of a row, y times powers of two, in the I/O dtype.
template <typename E>
__device__ __forceinline__ void store_cols(const Rsrc& rs, int off, f32x4 y, i32x4 e) {
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = __builtin_amdgcn_ldexpf(y[i], e[i]);
  if constexpr (sizeof(E) == 4) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y), rs, off, 0, 0);
  } else {
    const bf16x4 z = (bf16x4){(__bf16)y[0], (__bf16)y[1], (__bf16)y[2], (__bf16)y[3]};
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, z), rs, off, 0, 0);
  }
}

// Four value columns of a row in fp16, as they are scaled.
__device__ __forceinline__ void store_cols_h(const Rsrc& rs, int off, f32x4 y) {
  const u32x2 z = {__builtin_bit_cast(uint32_t, cvt_h2(y[0], y[1])), __builtin_bit_cast(uint32_t, cvt_h2(y[2], y[3]))};
  __builtin_amdgcn_raw_buffer_store_b64(z, rs, off, 0, 0);
}

// A state slice (16 value columns ct of all key rows), turned over: a lane holds
// four value columns of one key row, as the gradients' kernel takes it.  Image of
// a chunk and head: [key tile][column tile][lane][4].  bf16 inputs: the leading
// terms f of key rows 32 ks .., as they are scaled; ident: the identity.
__device__ __forceinline__ void store_turned(const __bf16*, void* image, size_t unit, int ct, int ks, f16x8 f,
                                             const f32x4 (&)[8], const f16x8 (&ident)[2], i32x4, int lane) {
  u32x2* dst = static_cast<u32x2*>(image) + (unit * 64 + ct) * 64 + lane;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const f32x4 y = mma_h((f32x4){0.f, 0.f, 0.f, 0.f}, f, ident[half]);
    const u32x2 z = {__builtin_bit_cast(uint32_t, cvt_h2(y[0], y[1])), __builtin_bit_cast(uint32_t, cvt_h2(y[2], y[3]))};
    __builtin_nontemporal_store(z, dst + (2 * ks + half) * (8 * 64));
  }
}
// A 16 x 16 tile's rows and columns turned over, in fp32.
__device__ __forceinline__ f32x4 turn(const Frag16<float>& f) {
  const int l16 = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
  Frag16<float> one;
#pragma unroll
  for (int i = 0; i < 4; ++i) one.v[i] = 4 * g + i == l16 ? 1.f : 0.f;
  return mma16((f32x4){0.f, 0.f, 0.f, 0.f}, f, one);
}
// (fp32: exact, from the state itself; ce: the exponents of the columns 4 g ..)
__device__ __forceinline__ void store_turned(const float*, void* image, size_t unit, int ct, int ks, f16x8,
                                             const f32x4 (&s)[8], const f16x8 (&)[2], i32x4 ce, int lane) {
  f32x4* dst = static_cast<f32x4*>(image) + (unit * 64 + ct) * 64 + lane;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    Frag16<float> f;
    f.v = s[2 * ks + half];
    f32x4 y = turn(f);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __builtin_amdgcn_ldexpf(y[i], ce[i]);
    __builtin_nontemporal_store(y, dst + (2 * ks + half) * (8 * 64));
  }
}

// Blocks b and b + 8 run on the same XCD: what the parts of a head and the
// heads that share a key head read comes from its L2 after the first.
template <int PER>
__device__ __forceinline__ int64_t delta_unit(int64_t unit0, int heads, int qk_heads, int64_t block, int& part) {
  const int share = heads / qk_heads, per = share * PER;
  const int64_t slot8 = block >> 3;
  part = (int)(slot8 % PER);
  return unit0 + (slot8 / per * 8 + (block & 7)) * share + slot8 % per / PER;
}

// Calls launch(part, blocks) for parts of a.units whose blocks make fewer than
// 2^32 threads.
template <int PER, typename A, typename F>
hipError_t launch_delta_parts(const A& a, const F& launch) {
  const int64_t group = 8 * (a.num_heads / a.qk_heads);  // units that go to the XCDs together
  const int64_t most = std::max(kMaxThreads / kWalkThreads / (group * PER), (int64_t)1) * group;
  for (int64_t u = 0; u < a.units; u += most) {
    A part = a;
    part.unit0 = u;
    part.units = std::min(a.units, u + most);
    launch(part, (unsigned)((part.units - u + group - 1) / group * group * PER));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace
}  // namespace kda
