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
// token boundary equals <S, dS>.  The dq walk leaves the r_t and the dk walk
// the c_t, and both the states at every boundary of `anchor` tokens; the sum
// over t is restarted from their product there, so that rounding cannot build
// up along the sequence (decay_grad, in linear_finish_kernel).
//
// What is rounded.  bf16: the pair matrix (q_i . k_j) e^{..} and the state,
// as operands of the outputs' products, to one bf16 each (the output is bf16
// itself: measured 2.3e-3 of its norm off the 64-bit result, against 1.7e-3 for
// the output's own rounding; a second term of each does not fit LDS in the
// walks of whole heads).  The state's update takes e^{..} v_j as the sum
// of three bf16 terms (24 bits), because the state is an fp32 result, and in
// every walk, so that no output's bits depend on whether the state is asked
// for; the part of r_t and c_t that comes through the state takes three terms
// of the state for the same reason (and with it dq and dk where the decays'
// gradient is wanted, else they take one).  Accumulation is fp32, prefix sums of the decays
// are fp64 (a difference of two sums decides every factor).
#include <algorithm>
#include <atomic>
#include <type_traits>

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
__device__ __forceinline__ int64_t boundary_of(int n, int64_t bos, int anchor, bool ends, int64_t j) {
  return bos / anchor + (ends ? n : 0) + j - 1;
}

// Sequence of rank r when the sequences are ordered longest first (ties by
// index), so that the longest walks start first.  Every thread of the
// workgroup calls it.  Up to 256 sequences; more keep their order.
constexpr int kRankedSeqs = 256;
template <int THREADS>
__device__ __forceinline__ int longest_first(int* lds, const int32_t* cu, int N, int64_t T, int r) {
  if (!cu || N == 1 || N > kRankedSeqs) return r;
  for (int i = threadIdx.x; i < N; i += THREADS) {
    int64_t bos, eos;
    seq_range(cu, i, T, bos, eos);
    lds[i] = (int)(eos - bos);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < N; i += THREADS) {
    const int mine = lds[i];
    int rank = 0;
    for (int m = 0; m < N; ++m) rank += lds[m] > mine || (lds[m] == mine && m < i);
    if (rank == r) lds[kRankedSeqs] = i;
  }
  __syncthreads();
  const int n = __builtin_amdgcn_readfirstlane(lds[kRankedSeqs]);
  __syncthreads();  // the LDS is used for tiles from here on
  return n;
}

// ---- LDS tiles ------------------------------------------------------------
// A tile holds C tokens x W channels, row-major, its 16-byte units XOR-ed
// with a function of the row so that what one instruction reads falls on
// different banks.  In bytes, element (row, ch) is at
//   row W ES + ((ch ES) ^ 16 swizzle(row)),
// so with the lane's part of ch in an offset `at`, the rest of ch (which has
// no bit in common with it) is one more XOR on the address, and 16 more rows
// are an addition.
//
// What one LDS cycle serves (measured with the conflict counter): 32
// consecutive lanes of an 8-byte read, the lanes 0-3, 12-15, 20-27 (and so on)
// of a 16-byte read.  bf16, rows of 256 bytes: 16 rows read at one channel
// need 16 different units; a transposing read takes two neighbouring units of
// the rows 8 g .. 8 g + 3 for two g, so the upper three bits of the swizzle
// have to tell those eight rows apart; a 16-byte read takes unit u of the rows
// 0-3, 12-15 and unit u ^ 1 of the rows 4-11, so each of these two sets has to
// fill whole pairs of units.  Rows of half a tile (128 bytes, two to a turn of
// the banks) are only read transposing.  fp32: 16 lanes of a column read take
// four neighbouring units, and half a wave two rows that differ in bit 2: the
// row itself.
template <typename E, int W>
__device__ __forceinline__ int swizzle(int row) {
  if constexpr (sizeof(E) == 4) return row & 15;
  else if constexpr (W == D) return ((row ^ (row << 1)) & 8) | ((row & 3) << 1) | ((row >> 2) & 1);
  else return ((row >> 1) & 4) | (row & 2) | ((row >> 2) & 1);
}
template <typename E, int W>
__device__ __forceinline__ uint32_t tile_at(int row, int ch) {
  return (uint32_t)(row * W * (int)sizeof(E) + ((ch * (int)sizeof(E)) ^ (swizzle<E, W>(row) << 4)));
}
// Reads at a byte address of LDS (a number rather than a pointer, so that the
// XORs are on it and its constant parts stay in the instruction).
template <typename T>
__device__ __forceinline__ T lds_get(uint32_t at) {
  return *reinterpret_cast<const __attribute__((address_space(3))) T*>(at);
}
// The same for 8-byte halves of an operand: volatile, or two rows' halves are
// fetched by one instruction into registers that moves have to sort again.
template <typename T>
__device__ __forceinline__ T lds_get_half(uint32_t at) {
  return *reinterpret_cast<const volatile __attribute__((address_space(3))) T*>(at);
}

// operand with the channels ch .. ch+7 of a row; `at` = the lane's 8 g, ch0 = 32 ks
__device__ __forceinline__ void ld_row(Frag<__bf16>& f, uint32_t at, int ch0) {
  f.v = lds_get<bf16x8>(at ^ (uint32_t)(ch0 * 2));
}
__device__ __forceinline__ void ld_row(Frag<float>& f, uint32_t at, int ch0) {
  f.lo = lds_get<f32x4>(at ^ (uint32_t)(ch0 * 4));
  f.hi = lds_get<f32x4>(at ^ (uint32_t)(ch0 * 4 + 16));
}
// operand with the channels ch0 + 4 g .. and ch0 + 16 + 4 g .. of a row (what
// two stacked accumulator tiles hold); `at` = the lane's 4 g
__device__ __forceinline__ void ld_row_acc(Frag<__bf16>& f, uint32_t at, int ch0, int rows) {
  const u32x2 a = lds_get_half<u32x2>((at ^ (uint32_t)(ch0 * 2)) + rows * (D * 2));
  const u32x2 b = lds_get_half<u32x2>((at ^ (uint32_t)(ch0 * 2 + 32)) + rows * (D * 2));
  f.v = __builtin_bit_cast(bf16x8, (u32x4){a[0], a[1], b[0], b[1]});
}
__device__ __forceinline__ void ld_row_acc(Frag<float>& f, uint32_t at, int ch0, int rows) {
  f.lo = lds_get<f32x4>((at ^ (uint32_t)(ch0 * 4)) + rows * (D * 4));
  f.hi = lds_get<f32x4>((at ^ (uint32_t)(ch0 * 4 + 64)) + rows * (D * 4));
}

// Operands whose contraction runs over a chunk's tokens: 32 deep in bf16
// (eight tokens a lane, the tokens 8 g ..), 16 deep in fp32 (four, 4 g ..).
template <typename E>
struct Tok;
template <>
struct Tok<__bf16> {
  using F = Frag<__bf16>;
  static constexpr int N = 8;      // tokens a lane holds
  static constexpr int READS = 2;  // LDS reads of a column
};
template <>
struct Tok<float> {
  using F = Frag16<float>;
  static constexpr int N = 4;
  static constexpr int READS = 4;
};
__device__ __forceinline__ f32x4 mma_tok(f32x4 acc, const Frag<__bf16>& a, const Frag<__bf16>& b) {
  return mma(acc, a, b);
}
__device__ __forceinline__ f32x4 mma_tok(f32x4 acc, const Frag16<float>& a, const Frag16<float>& b) {
  return mma16(acc, a, b);
}
// A column over the lane's tokens.  bf16: the transposing LDS read hands each
// lane of 16 one column of a 4-row x 16-channel block, whose rows the lanes
// 4r .. 4r+3 address.  col_at: the lane's offsets (two reads in bf16, four in
// fp32) at column 0 of a tile; ch0 is a multiple of 16.
template <int W>
__device__ __forceinline__ void col_at(uint32_t (&at)[2], const __bf16*, int ch, int l16, int g) {
  const int r = 8 * g + (l16 >> 2), c = ch + 4 * (l16 & 3);
  at[0] = tile_at<__bf16, W>(r, c);
  at[1] = tile_at<__bf16, W>(r + 4, c);
}
template <int W>
__device__ __forceinline__ void col_at(uint32_t (&at)[4], const float*, int ch, int l16, int g) {
#pragma unroll
  for (int i = 0; i < 4; ++i) at[i] = tile_at<float, W>(4 * g + i, ch + l16);
}
__device__ __forceinline__ void ld_col(Frag<__bf16>& f, uint32_t base, const uint32_t (&at)[2], int ch0) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)((base + at[0]) ^ (uint32_t)(ch0 * 2)));
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)((base + at[1]) ^ (uint32_t)(ch0 * 2)));
  const bf16x4 x = __builtin_bit_cast(bf16x4, a), y = __builtin_bit_cast(bf16x4, b);
  f.v = (bf16x8){x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
}
__device__ __forceinline__ void ld_col(Frag16<float>& f, uint32_t base, const uint32_t (&at)[4], int ch0) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f.v[i] = lds_get<float>((base + at[i]) ^ (uint32_t)(ch0 * 4));
}
// the same from memory (raw buffer view, byte offset)
__device__ __forceinline__ void buf_row(Frag<__bf16>& f, const Rsrc& rs, uint32_t off) {
  f.v = __builtin_bit_cast(bf16x8, buf_ld16(rs, off, 0));
}
__device__ __forceinline__ void buf_row(Frag<float>& f, const Rsrc& rs, uint32_t off) {
  f.lo = __builtin_bit_cast(f32x4, buf_ld16(rs, off, 0));
  f.hi = __builtin_bit_cast(f32x4, buf_ld16(rs, off, 16));
}
// The pair matrix: rows of RB = 64 or 128 bytes, their 16-byte units XOR-ed so
// that the rows of a 16-byte read (above) fall on all banks.  pair_at: the
// byte offset of unit u; the tokens of step kt are the units 4 kt ...
template <int RB>
__device__ __forceinline__ uint32_t pair_at(int row, int u) {
  static_assert(RB == 64 || RB == 128, "two row lengths");
  const int b3 = (row >> 3) & 1, b2 = (row >> 2) & 1, b1 = (row >> 1) & 1;
  const int x = RB == 64 ? (b3 ^ b2) << 1 | b3 : (b3 ^ b2) << 2 | b1 << 1 | b3;
  return (uint32_t)(row * RB + ((u ^ x) << 4));
}
// a row over the lane's tokens (unit g)
__device__ __forceinline__ void ld_pair(Frag<__bf16>& f, uint32_t at) { f.v = lds_get<bf16x8>(at); }
__device__ __forceinline__ void ld_pair(Frag16<float>& f, uint32_t at) { f.v = lds_get<f32x4>(at); }
__device__ __forceinline__ float frag_get(const Frag<__bf16>& f, int i) { return (float)f.v[i]; }
__device__ __forceinline__ float frag_get(const Frag16<float>& f, int i) { return f.v[i]; }

// x as the sum of NS operands.  bf16, one term: rounded to nearest.  Three
// terms: the 24 significant bits cut in three (each subtraction is exact; two
// terms: the first 16), the high halves of two words packed by one byte permutation.  fp32: itself.
template <int NS>
__device__ __forceinline__ void split(Frag<__bf16> (&f)[NS], const float (&x)[8]) {
  if constexpr (NS == 1) {
    frag_from_f32(f[0], x);
  } else {
    static_assert(NS == 2 || NS == 3, "one to three terms");
    uint32_t t[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      t[0][i] = __builtin_bit_cast(uint32_t, x[i]);
      const float r = x[i] - __builtin_bit_cast(float, t[0][i] & 0xffff0000u);
      t[1][i] = __builtin_bit_cast(uint32_t, r);
      t[2][i] = __builtin_bit_cast(uint32_t, r - __builtin_bit_cast(float, t[1][i] & 0xffff0000u));
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __builtin_amdgcn_perm(t[s][2 * i + 1], t[s][2 * i], 0x07060302u);
      f[s].v = __builtin_bit_cast(bf16x8, w);
    }
  }
}
template <int NS>
__device__ __forceinline__ void split(Frag<float> (&f)[NS], const float (&x)[8]) {
  static_assert(NS == 1, "fp32 operands are exact");
  frag_from_f32(f[0], x);
}
template <int NS>
__device__ __forceinline__ void split(Frag16<float> (&f)[NS], const float (&x)[4]) {
  static_assert(NS == 1, "fp32 operands are exact");
  f[0].v = (f32x4){x[0], x[1], x[2], x[3]};
}

// Every wave's LDS writes land before any wave goes on.  (Not __syncthreads():
// its fence would also wait for the copies into LDS that the loader wave has
// in flight for later chunks.)
__device__ __forceinline__ void chunk_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Moves of a double between the lanes of a row of 16, without LDS: lane l
// gets lane l - N (shr) or l + N (shl), zero where there is none.
template <int CTRL>
__device__ __forceinline__ double dpp_move(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xf, 0xf, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xf, 0xf, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <int CTRL>
__device__ __forceinline__ float dpp_move_f32(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ double read_lane(double x, int l) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, l);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), l);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Sums over the lanes of a column (lane mod 16): of four values at a time, each
// row of 16 lanes ending with one of them (`tile` says which), or of two, every
// other row ending with one (tile -1: none).
__device__ __forceinline__ float swap_add32(float a, float b) {  // lower half: a's, upper half: b's sums of halves
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
                                                  false, false);
  const uint32_t lo = r[0], hi = r[1];
  return __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
}
__device__ __forceinline__ float swap_add16(float a, float b) {  // even rows: a's, odd rows: b's sums of row pairs
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
                                                  false, false);
  const uint32_t lo = r[0], hi = r[1];
  return __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
}
__device__ __forceinline__ float sum_groups(const float (&x)[4], int g, int& tile) {
  tile = (g & 1) << 1 | g >> 1;
  return swap_add16(swap_add32(x[0], x[1]), swap_add32(x[2], x[3]));
}
__device__ __forceinline__ float sum_groups(const float (&x)[2], int g, int& tile) {
  const float s = swap_add32(x[0], x[1]);
  tile = g & 1 ? -1 : g >> 1;
  return swap_add16(s, s);
}
// Sum over the 16 lanes of a row, in every one of them.
__device__ __forceinline__ float sum_row(float x) {
  x += dpp_move_f32<0x128>(x);
  x += dpp_move_f32<0x124>(x);
  x += dpp_move_f32<0x122>(x);
  x += dpp_move_f32<0x121>(x);
  return x;
}
// Sums over the lanes 0 .. lane (prefix) and lane .. C - 1 (suffix) of C lanes.
template <int C>
__device__ __forceinline__ double prefix_sum(double x, int lane) {
  x += dpp_move<0x111>(x);
  x += dpp_move<0x112>(x);
  x += dpp_move<0x114>(x);
  x += dpp_move<0x118>(x);
  double low = 0.0;
#pragma unroll
  for (int r = 16; r < C; r += 16) {
    const double t = read_lane(x, r - 1);
    low += lane >= r ? t : 0.0;
  }
  return x + low;
}
template <int C>
__device__ __forceinline__ double suffix_sum(double x, int lane) {
  x += dpp_move<0x101>(x);
  x += dpp_move<0x102>(x);
  x += dpp_move<0x104>(x);
  x += dpp_move<0x108>(x);
  double high = 0.0;
#pragma unroll
  for (int r = C - 16; r > 0; r -= 16) {
    const double t = read_lane(x, r);
    high += lane < r ? t : 0.0;
  }
  return x + high;
}

// NW compute waves of 16 value columns each: 4 (half a head) or 8 (a head).
// Chunks of 64 tokens (32 in fp32), query and key tiles of three chunks and
// value tiles of two in LDS.  All walks take the same chunks: what r_t counts
// as coming through the state (dq walk) is what the dk walk (DK) does not
// count as a pair.
template <typename E, int NW, bool DG, bool DK>
struct WalkLayout {
  static constexpr int ES = (int)sizeof(E);
  static constexpr int C = 128 / ES;
  static constexpr int TILE = C * D * ES;              // a query or key tile
  static constexpr int VW = 16 * NW;                   // value columns of the workgroup
  static constexpr int VTILE = C * VW * ES;
  static constexpr int K = TILE, SET = 2 * TILE;       // tiles that arrive together
  static constexpr int NBUF = 3;
  static constexpr int VALS = NBUF * SET;              // [2] value tiles
  static constexpr int RB = C * ES;                    // bytes of a pair matrix row
  static constexpr int PAIR = VALS + 2 * VTILE;        // E [2][C][C]
  static constexpr int SUM = PAIR + 2 * C * RB;        // float [4][2][C] prefix sums (log2), high and low part
  static constexpr int ROW = SUM + 4 * 2 * C * 4;      // float [4][C] factor of the state in row t
  static constexpr int WGT = ROW + 4 * C * 4;          // float [4][C] factor of token t in the state
  static constexpr int GAM = WGT + 4 * C * 4;          // float [4] factor of the state over the chunk
  static constexpr int RX = GAM + 16;                  // float [2][NW][C] state part . x by compute wave
  static constexpr int RR = RX + (DG ? 2 * NW * C * 4 : 0);  // float [2][2][C] pair sums of the keys by pair wave
  static constexpr int RC = RR + (DK ? 4 * C * 4 : 0);       // float [2][C] pair sums of the queries
  static constexpr int BYTES = RC + (DK ? 2 * C * 4 : 0);
};

// 2^x of a sum of decays.  Its whole part goes into the exponent, as fp32 would
// keep an x of 30 to 2^-19 only (1.3e-6 of the factor; the hardware's own
// rounding is 2^-23).
__device__ __forceinline__ float exp2_sum(double x) {
  const double whole = __builtin_rint(fmax(x, -1000.0));  // (below 2^-1000 nothing is left in fp32)
  return __builtin_amdgcn_ldexpf(exp2_fast((float)(fmax(x, -1000.0) - whole)), (int)whole);
}

// The state is kept as 2^s times what the accumulators hold, so that a chunk's
// decay need not scale them: the decay wave moves it into s, and with it into
// the factors of rows and tokens, until s falls below this (the factors stay
// below 2^30) or the state itself is wanted.
constexpr double kScaleFloor = -30.0;

// ---------------------------------------------------------------------------
// The walk.  NW + 4 waves per (sequence or segment, head, block of 16 NW value
// columns), in four roles, meeting at one barrier per chunk:
//   NW compute waves: wave w owns 16 value columns and keeps its [128 x 16]
//              slice of the state in matrix-core accumulators (fp32) over the
//              whole walk; accumulators of two stacked tiles are an operand of
//              the next product as they are.  For chunk c: the outputs,
//              transposed (rows = value columns), so that a lane stores four
//              consecutive columns: S^T q, scaled by e^{G_i}, plus the pair
//              matrix times v; then S <- e^{G_C} S + k^T (e^{G_C - G_j} v_j).
//   two pair waves: the pair matrix of chunk c + 1 in 16-query tiles, the
//              products with the keys up to them scaled by e^{G_i - G_j}
//   a decay wave: prefix sums and factors of chunk c + 2; with DG the r_t or c_t
//              of chunk c - 1
//   a loader:  copies tiles from global memory straight into LDS, queries and
//              keys two chunks ahead of the compute waves, values one
// A compute wave is bound by its own chain of instructions, not by the matrix
// cores (a wave issues at most one vector instruction in 4 cycles, and waits
// for LDS in between): a whole head takes eight waves of 16 columns rather than
// four of 32, chunks are as long as LDS allows, and what can be is left to the
// other waves.
// Measured, bf16, 96 heads x 8192 tokens.  Forward, half heads: 225 us, 3.6
// TB/s of the 4.8 that a large copy reaches here; copies and compute waves take
// about 3500 cycles a chunk each.  Backward, whole heads: a dk, dq, dv walk of
// 128 chunks takes 610, 590, 400 us side by side, 8700 cycles a chunk with the
// decays' gradient where its matrix instructions take 3600 of a SIMD.  The
// three walks fetch 2.3 GB and write 0.72 GB, 620 us at a large copy's rate: at
// 650-685 us the launch is as near to that bound as to the waves' own.
// REV walks backwards in time: the pair matrix is upper triangular and the
// factors of rows and of tokens change places.
// DG (the decays' gradient): x is q in the dq walk and k in the dk walk.
// ---------------------------------------------------------------------------
template <typename E, int NW, bool REV, bool TR, bool OUT, bool DG>
__device__ __forceinline__ void walk(const LinearWalkArgs& p, unsigned char* smem, int64_t u, int cb) {
  constexpr bool DK = DG && REV;               // dk walk: forms the decays' gradient
  using L = WalkLayout<E, NW, DG, DK>;
  using TF = typename Tok<E>::F;
  constexpr int TN = Tok<E>::N;
  constexpr int C = L::C, NT = C / 16, ES = L::ES, NBUF = L::NBUF;
  constexpr bool BF = ES == 2;
  constexpr int NSV = BF ? 3 : 1;              // terms of the weighted values
  constexpr int NSS = (BF && DG) ? 3 : 1;      // terms of the state in the outputs' product
  static_assert(L::BYTES <= 160 * 1024, "LDS budget exceeded");
  constexpr int KT = C / (4 * TN);             // token steps per chunk
  constexpr int TPS = NT / KT;                 // 16-token tiles per token step
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)smem;
  float* sSum = reinterpret_cast<float*>(smem + L::SUM);
  float* sRow = reinterpret_cast<float*>(smem + L::ROW);
  float* sWgt = reinterpret_cast<float*>(smem + L::WGT);
  float* sGam = reinterpret_cast<float*>(smem + L::GAM);
  float* sRX = reinterpret_cast<float*>(smem + L::RX);
  float* sRR = reinterpret_cast<float*>(smem + L::RR);
  float* sRC = reinterpret_cast<float*>(smem + L::RC);

  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int H = p.num_heads;
  const int h = (int)(u % H);
  const int64_t rank = u / H;
  // tokens [tb, te) of sequence n = tokens [bos, eos)
  int n;
  int64_t bos, eos, tb, te, slot;
  bool first, last;  // the item begins / ends its sequence
  if (p.segmented) {
    const Segment s = find_segment(p.cu, p.num_seqs, p.total_tokens, p.seg, rank);
    if (!s.ok) return;
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
    n = longest_first<64 * (NW + 4)>(reinterpret_cast<int*>(smem), p.cu, p.num_seqs, p.total_tokens, (int)rank);
    seq_range(p.cu, n, p.total_tokens, bos, eos);
    slot = 0;
    tb = bos;
    te = eos;
    first = last = true;
  }
  const int nch = (int)((te - tb + C - 1) / C);
  const size_t nh = (size_t)n * H + h;
  auto chunk_of = [&](int ci) { return REV ? nch - 1 - ci : ci; };
  // Boundaries where the decays' gradient takes the state from memory or leaves
  // it there (an item begins at one): chunks from one to the next, and from the
  // walk's start to the first behind it.
  const int stretch = DG ? p.anchor / C : 0;
  const int stretch0 = DG && REV ? (nch + stretch - 1) % stretch + 1 : stretch;
  // Iteration ci (from -1): compute waves on chunk ci, pair waves on ci + 1,
  // decay wave on ci + 2 and back on ci - 1.

  // The SIMDs serve their oldest wave first; what the compute waves wait for
  // at the next barrier goes ahead of them.
  if (wv >= NW) __builtin_amdgcn_s_setprio(2);

  if (wv == NW + 3) {
    // ---- loader ----
    // 1 KiB pieces, 16 bytes a lane; the lanes' offsets are the same in every
    // chunk.  Rows behind the end lie outside the buffer view and arrive as
    // zeros.
    // the tensors from this head's rows on
    struct Rows {
      const char* base;
      uint32_t stride;
    };
    auto rows_of = [&](const void* src, int heads) {
      return Rows{static_cast<const char*>(src) + (size_t)(h / (H / heads)) * (D * ES), (uint32_t)heads * (D * ES)};
    };
    const Rows rq = rows_of(p.q, p.q_heads), rk = rows_of(p.k, p.k_heads), rv = rows_of(p.v, p.v_heads);
    auto copy_tile = [&](auto width, const Rows& src, int ch0, int ci, unsigned char* dst) {
      constexpr int W = decltype(width)::value;
      constexpr int NPC = C * W * ES / 1024;   // pieces
      constexpr int UR = W * ES / 16;          // 16-byte units per row
      constexpr int RP = 64 / UR;              // rows per piece
      const int64_t t0 = tb + (int64_t)chunk_of(ci) * C;
      const int nv = (int)min((int64_t)C, te - t0);
      const uint32_t stride = src.stride;
      const Rsrc rs = make_rsrc(src.base + (size_t)t0 * stride, (uint32_t)(nv - 1) * stride + D * ES);
      uint32_t row = (uint32_t)(lane / UR) * stride + ch0 * ES;
#pragma unroll
      for (int i = 0; i < NPC; ++i) {
        const uint32_t unit = (uint32_t)(((lane % UR) ^ swizzle<E, W>(i * RP + lane / UR)) * 16);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)(dst + i * 1024), 16,
                                                 (int)(row + unit), 0, 0, 0);
        row += RP * stride;
      }
    };
    using Whole = std::integral_constant<int, D>;
    using Block = std::integral_constant<int, L::VW>;
    auto copy_set = [&](int ci) {
      if (ci >= nch) return;
      unsigned char* dst = smem + (ci % NBUF) * L::SET;
      if (OUT) copy_tile(Whole{}, rq, 0, ci, dst);
      copy_tile(Whole{}, rk, 0, ci, dst + L::K);
    };
    copy_set(0);
    for (int ci = -1; ci < nch; ++ci) {
      __builtin_amdgcn_s_waitcnt(vmcnt_wait(0));
      chunk_barrier();
      copy_set(ci + 2);
      if (ci + 1 < nch)
        copy_tile(Block{}, rv, cb * L::VW, ci + 1, smem + L::VALS + ((ci + 1) & 1) * L::VTILE);
    }
    if constexpr (DG) chunk_barrier();
    return;
  }

  if (wv == NW + 2) {
    // ---- decays ----
    // rows behind the end lie outside the buffer view and read zero
    auto load_rows = [&](const float* src, int ci) -> float {
      const int64_t t0 = tb + (int64_t)chunk_of(ci) * C;
      const int nv = (int)min((int64_t)C, te - t0);
      const Rsrc rs = make_rsrc(src + (size_t)t0 * H + h, ci >= 0 && ci < nch ? (uint32_t)((nv - 1) * H + 1) * 4 : 0);
      return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, lane < C ? lane * H * 4 : -4, 0, 0));
    };
    const float la_head = p.decay_per_head ? p.log_decay[h] : 0.f;
    auto load_decay = [&](int ci) -> float {
      if (!p.decay_per_head) return load_rows(p.log_decay, ci);
      return lane < C && tb + (int64_t)chunk_of(ci) * C + lane < te ? la_head : 0.f;
    };
    double log_total = 0.0;
    double scale = 0.0;  // s: the state is 2^s times the accumulators
    int boundary = stretch0;
    auto put_decay = [&](int ci, float la) {
      const int64_t t = tb + (int64_t)chunk_of(ci) * C + lane;
      const double s = prefix_sum<C>((double)fmaxf(la, kMinLogDecay) * kLog2e, lane);
      const double tot = read_lane(s, C - 1);
      log_total += tot;
      const double before = scale;
      scale += tot;
      float gam = 1.f;
      const bool at_boundary = DG && --boundary == 0;  // the state behind the chunk is wanted
      if (at_boundary) boundary = stretch;
      if (scale < kScaleFloor || ci == nch - 1 || at_boundary) {
        gam = exp2_sum(scale);
        scale = 0.0;
      }
      const float row = exp2_sum(before + (REV ? tot - s : s));
      const float wgt = exp2_sum((REV ? s : tot - s) - scale);
      const int b = ci & 3;
      if (lane < C) {
        const float hi = (float)s;
        sSum[b * 2 * C + lane] = hi;
        sSum[b * 2 * C + C + lane] = (float)(s - (double)hi);
        sRow[b * C + lane] = row;
        sWgt[b * C + lane] = t < te ? wgt : 0.f;
      }
      if (lane == 0) sGam[b] = gam;
    };
    // what this walk's columns say of the decays' gradient at a chunk's tokens
    auto finish = [&](int ci) {
      const int64_t t0 = tb + (int64_t)chunk_of(ci) * C;
      if (lane >= C || t0 + lane >= te) return;
      float part = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) part += sRX[((ci & 1) * NW + w) * C + lane];
      if constexpr (DK) {
        // pairs within the chunk, as queries (c) and as keys (r)
        part += sRC[(ci & 1) * C + lane];
#pragma unroll
        for (int w = 0; w < 2; ++w) part -= sRR[((ci & 1) * 2 + w) * C + lane];
      }
      p.change[((size_t)cb * H + h) * p.total_tokens + t0 + lane] = part;
    };
    if (nch > 0) put_decay(0, load_decay(0));
    // two iterations ahead of their use, one in flight over a barrier
    float la_next = load_decay(1);
    for (int ci = -1; ci < nch; ++ci) {
      chunk_barrier();
      const float la = la_next;
      la_next = load_decay(ci + 3);
      if (ci + 2 < nch) put_decay(ci + 2, la);
      if constexpr (DG)
        if (ci > 0) finish(ci - 1);
    }
    if constexpr (DG) {
      chunk_barrier();
      if (nch > 0) finish(nch - 1);
    }
    if (!OUT && lane == 0 && cb == 0) p.seg_decay[(size_t)slot * H + h] = exp2_sum(log_total);
    return;
  }

  if (wv >= NW) {
    // ---- pair matrix of chunk ci + 1, keys in rows: lane = query, four consecutive keys ----
    const uint32_t k_at = tile_at<E, D>(l16, 8 * g);
    // query tiles RA and RB (RB < 0: none) by pair wave PW
    auto pairs = [&](auto pw_, auto ra_, auto rb_) {
      constexpr int PW = decltype(pw_)::value, RA = decltype(ra_)::value, RBT = decltype(rb_)::value;
      constexpr int ROWS = RBT >= 0 ? 2 : 1;
      (void)PW;
      constexpr int rts[2] = {RA, RBT};
      auto in_triangle = [](int kt, int rt) { return REV ? kt >= rt : kt <= rt; };
      // DK: a chunk later, when its values have come, the pairs' products with
      // (v . x) over the block's columns, summed by query and by key.  x comes
      // from memory a chunk ahead.
      constexpr int XS = L::VW / 32;
      Frag<E> fx[DK ? ROWS : 1][DK ? XS : 1];
      f32x4 held[DK ? ROWS : 1][DK ? NT : 1];
      const uint32_t v_at = tile_at<E, L::VW>(l16, 8 * g);
      auto fetch_x = [&](int ci) {
        if constexpr (DK) {
          const int64_t t0 = tb + (int64_t)chunk_of(ci) * C;
          const int nv = (int)min((int64_t)C, te - t0);
          const uint32_t stride = (uint32_t)p.x_heads * (D * ES);
          const Rsrc rs = make_rsrc(static_cast<const char*>(p.x) + ((size_t)t0 * p.x_heads + h / (H / p.x_heads)) * (D * ES),
                                    ci < nch ? (uint32_t)(nv - 1) * stride + D * ES : 0);
#pragma unroll
          for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int ks = 0; ks < XS; ++ks)
              buf_row(fx[r][ks], rs, (uint32_t)(16 * rts[r] + l16) * stride + (cb * L::VW + 32 * ks + 8 * g) * ES);
        }
      };
      auto sum_pairs = [&](int ci) {
        if constexpr (DK) {
          const uint32_t vbase = lds0 + L::VALS + (ci & 1) * L::VTILE + v_at;
          const int nv = (int)min((int64_t)C, te - (tb + (int64_t)chunk_of(ci) * C));
          float csum[ROWS];
#pragma unroll
          for (int r = 0; r < ROWS; ++r) csum[r] = 0.f;
#pragma unroll
          for (int kt = 0; kt < NT; ++kt) {
            f32x4 rsum = {0.f, 0.f, 0.f, 0.f};
            Frag<E> fv[XS];
#pragma unroll
            for (int ks = 0; ks < XS; ++ks) ld_row(fv[ks], vbase + 16 * kt * (L::VW * ES), 32 * ks);
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
              if (!in_triangle(kt, rts[r])) continue;
              f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int ks = 0; ks < XS; ++ks) acc = mma(acc, fv[ks], fx[r][ks]);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int k = 16 * kt + 4 * g + i, q = 16 * rts[r] + l16;
                // (the token's own pair cancels)
                const float f = k > q && k < nv ? held[r][kt][i] * acc[i] : 0.f;
                rsum[i] += f;
                csum[r] += f;
              }
            }
            // over the 16 queries of the tiles
#pragma unroll
            for (int i = 0; i < 4; ++i) rsum[i] = sum_row(rsum[i]);
            if (l16 == 0) *reinterpret_cast<f32x4*>(sRR + ((ci & 1) * 2 + PW) * C + 16 * kt + 4 * g) = rsum;
          }
#pragma unroll
          for (int r = 0; r < ROWS; ++r) {
            csum[r] = swap_add32(csum[r], csum[r]);
            csum[r] = swap_add16(csum[r], csum[r]);
            if (g == 0) sRC[(ci & 1) * C + 16 * rts[r] + l16] = csum[r];
          }
        }
      };
      if (DK && nch > 0) fetch_x(0);
      for (int ci = -1; ci < nch; ++ci) {
        chunk_barrier();
        if (DK && ci >= 0) {
          sum_pairs(ci);
          fetch_x(ci + 1);
        }
        if (!OUT || ci + 1 >= nch) continue;
        const uint32_t base = lds0 + (uint32_t)((ci + 1) % NBUF) * L::SET;
        unsigned char* pair = smem + L::PAIR + ((ci + 1) & 1) * (C * L::RB);
        const int b = (ci + 1) & 3;
        const int64_t t0 = tb + (int64_t)chunk_of(ci + 1) * C;
        const int nv = (int)min((int64_t)C, te - t0);
        const float* gs = sSum + b * 2 * C;
        Frag<E> fq[ROWS][4];
        float gq[ROWS], gq_lo[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) ld_row(fq[r][ks], base + k_at + 16 * rts[r] * (D * ES), 32 * ks);
          gq[r] = gs[16 * rts[r] + l16];
          gq_lo[r] = gs[C + 16 * rts[r] + l16];
        }
#pragma unroll
        for (int kt = 0; kt < NT; ++kt) {
          Frag<E> fk[4];
          f32x4 gk, gk_lo;
          if (in_triangle(kt, RA) || (ROWS > 1 && in_triangle(kt, RBT))) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) ld_row(fk[ks], base + L::K + k_at + 16 * kt * (D * ES), 32 * ks);
            gk = *reinterpret_cast<const f32x4*>(gs + 16 * kt + 4 * g);
            gk_lo = *reinterpret_cast<const f32x4*>(gs + C + 16 * kt + 4 * g);
          }
#pragma unroll
          for (int r = 0; r < ROWS; ++r) {
            const int rt = rts[r];
            const bool tri = in_triangle(kt, rt);
            // a tile beyond the triangle that shares a token step with it is zero
            if (!tri && kt / TPS != rt / TPS) continue;
            const int q = 16 * rt + l16;
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
            if (tri) {
#pragma unroll
              for (int ks = 0; ks < 4; ++ks) acc = mma(acc, fk[ks], fq[r][ks]);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int k = 16 * kt + 4 * g + i;
                // (keys behind the end are zeros; backwards, so are their factors' uses)
                const bool on = kt != rt || (REV ? k >= q : k <= q);
                const float d = (gq[r] - gk[i]) + (gq_lo[r] - gk_lo[i]);
                const float x = acc[i] * exp2_fast(REV ? -d : d);
                acc[i] = on && (!REV || k < nv) ? x : 0.f;
              }
              if constexpr (DK) held[r][kt] = acc;
            }
            const uint32_t at = BF ? pair_at<L::RB>(q, 2 * kt + (g >> 1)) + 8 * (g & 1) : pair_at<L::RB>(q, 4 * kt + g);
            store_row4(reinterpret_cast<E*>(pair + at), acc);
          }
        }
      }
      if constexpr (DG) chunk_barrier();
    };
    // one tile from each end of the triangle
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using None = std::integral_constant<int, -1>;
    if (wv == NW) {
      if constexpr (NT == 4) pairs(I0{}, I0{}, std::integral_constant<int, 3>{});
      else pairs(I0{}, I0{}, None{});
    } else {
      if constexpr (NT == 4) pairs(I1{}, I1{}, std::integral_constant<int, 2>{});
      else pairs(I1{}, I1{}, None{});
    }
    return;
  }

  // ---- compute ----
  const int vc0 = 16 * wv;               // first value column within the block
  const int col0 = cb * L::VW + vc0;     // and within the head
  // The state slice: tile rt holds rows 16 rt + 4 g + i of column col0 + l16;
  // TR: of the transpose of what is stored.
  auto load_state = [&](const float* src, f32x4 (&s)[8]) {
#pragma unroll
    for (int rt = 0; rt < 8; ++rt) {
      const int row = 16 * rt + 4 * g, col = col0 + l16;
      if constexpr (TR) {
        s[rt] = *reinterpret_cast<const f32x4*>(src + col * D + row);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[rt][i] = src[(row + i) * D + col];
      }
    }
  };
  auto store_state = [&](float* dst, const f32x4 (&s)[8]) {
#pragma unroll
    for (int rt = 0; rt < 8; ++rt) {
      const int row = 16 * rt + 4 * g, col = col0 + l16;
      if constexpr (TR) {
        *reinterpret_cast<f32x4*>(dst + col * D + row) = s[rt];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) dst[(row + i) * D + col] = s[rt][i];
      }
    }
  };
  constexpr size_t kState = (size_t)D * D;
  // what the decays' gradient needs of the state (S in the dq walk, dS in the
  // dk walk) at boundary j of the sequence's stretches of `anchor` tokens
  const int64_t stretches = DG ? (eos - bos + p.anchor - 1) / p.anchor : 0;
  auto leave_state = [&](int64_t j, const f32x4 (&s)[8]) {
    if (j == 0 || (j == stretches && !p.end_state)) return;
    const int64_t at = p.anchors == p.snap ? slot_of(n, bos, p.anchor, j)
                                           : boundary_of(n, bos, p.anchor, p.end_state, j);
    store_state(p.anchors + ((size_t)at * H + h) * kState, s);
  };
  f32x4 accS[8];
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
      for (int rt = 0; rt < 8; ++rt) accS[rt] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }
  }
  // lane offsets within the tiles and the output rows
  uint32_t k_at[Tok<E>::READS], v_at[Tok<E>::READS];
  col_at<D>(k_at, static_cast<const E*>(nullptr), 0, l16, g);
  col_at<L::VW>(v_at, static_cast<const E*>(nullptr), vc0, l16, g);
  const uint32_t q_at = tile_at<E, D>(l16, 4 * g);
  uint32_t p_at[KT];
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) p_at[kt] = pair_at<L::RB>(l16, 4 * kt + g);
  const int oes = TR && p.o_f32 ? 4 : ES;
  const uint32_t o_row = (uint32_t)H * (D * oes);
  const uint32_t o_at = (uint32_t)l16 * o_row + (uint32_t)((col0 + 4 * g) * oes);
  // queries of the channel steps ks and ks + 1 are held at a time
  Frag<E> fq[OUT ? 2 : 1][NT];
  auto read_q = [&](uint32_t at, int ks) {
    if constexpr (OUT)
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) ld_row_acc(fq[ks & 1][rt], at + q_at, 32 * ks, 16 * rt);
  };
  // x of a chunk's rows, in the layout of the outputs, from memory a chunk ahead
  using Raw = std::conditional_t<BF, u32x2, f32x4>;
  Raw xr[DG ? NT : 1];
  auto load_x = [&](int ci) {
    if constexpr (DG) {
      const int64_t t0 = tb + (int64_t)chunk_of(ci) * C;
      const int nv = (int)min((int64_t)C, te - t0);
      const uint32_t stride = (uint32_t)p.x_heads * (D * ES);
      const Rsrc rs = make_rsrc(static_cast<const char*>(p.x) + ((size_t)t0 * p.x_heads + h / (H / p.x_heads)) * (D * ES),
                                ci < nch ? (uint32_t)(nv - 1) * stride + D * ES : 0);
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) {
        const int off = (int)((16 * rt + l16) * stride + (col0 + 4 * g) * ES);
        if constexpr (BF) xr[rt] = __builtin_amdgcn_raw_buffer_load_b64(rs, off, 0, 0);
        else xr[rt] = __builtin_bit_cast(f32x4, buf_ld16(rs, (uint32_t)off, 0));
      }
    }
  };
  load_x(0);
  chunk_barrier();  // iteration -1: the pair matrix of the first chunk is being formed

  uint32_t base = lds0;  // of the chunk's query and key tiles
  read_q(base, 0);
  read_q(base, 1);
  int boundary = 0;  // chunks to the next one
  int64_t stretch_at = DG ? (REV ? (te - bos + p.anchor - 1) / p.anchor : (tb - bos) / p.anchor) : 0;
  for (int ci = 0; ci < nch; ++ci) {
    const int64_t t0 = tb + (int64_t)chunk_of(ci) * C;
    const int nv = (int)min((int64_t)C, te - t0);
    const int b = ci & 3;

    if constexpr (DG) {
      if (boundary == 0) {
        if (p.anchors != p.snap) leave_state(stretch_at, accS);
        stretch_at += REV ? -1 : 1;
        boundary = ci == 0 ? stretch0 : stretch;
      }
      --boundary;
    }
    chunk_barrier();

    // The LDS reads run a few operands ahead of the products, in the order of
    // use (at most 15 can be waited for one by one); the vector arithmetic
    // fills the gaps between products.
    if (NW == 8 && wv >= 4) __builtin_amdgcn_s_setprio(1);
    const uint32_t base_next = base + L::SET == lds0 + NBUF * L::SET ? lds0 : base + L::SET;
    const uint32_t vbase = lds0 + L::VALS + (ci & 1) * L::VTILE;
    // (in a scalar register)
    const float gam = __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, sGam[b])));
    float w[KT][TN];
    TF fv[KT], fk[8];
    auto read_values = [&](int kt) {
#pragma unroll
      for (int i = 0; i < TN; i += 4) {
        const f32x4 y = *reinterpret_cast<const f32x4*>(sWgt + b * C + 4 * TN * kt + TN * g + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[kt][i + j] = y[j];
      }
      ld_col(fv[kt], vbase + kt * (4 * TN * L::VW * ES), v_at, 0);
    };
    if constexpr (!DG) {
      read_values(0);
      read_values(1);
    }
    auto read_k = [&](int kt, int first, int count) {
#pragma unroll
      for (int rt = 0; rt < 8; ++rt)
        if (rt >= first && rt < first + count) ld_col(fk[rt], base + L::K + kt * (4 * TN * D * ES), k_at, 16 * rt);
    };
    // values times their factors, in the terms of the state's update
    TF fw[KT][NSV];
    auto weigh_values = [&](int kt) {
      float x[TN];
#pragma unroll
      for (int i = 0; i < TN; ++i) x[i] = frag_get(fv[kt], i) * w[kt][i];
      split<NSV>(fw[kt], x);
    };
    auto add_to_state = [&](int kt) {
#pragma unroll
      for (int s = 0; s < NSV; ++s)
#pragma unroll
        for (int rt = 0; rt < 8; ++rt) accS[rt] = mma_tok(accS[rt], fk[rt], fw[kt][s]);
    };
    f32x4 accO[OUT ? NT : 1];
    if constexpr (OUT) {
      // outputs (transposed: lane = token, four consecutive value columns)
      float row[NT];
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) row[rt] = sRow[b * C + 16 * rt + l16];
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) accO[rt] = (f32x4){0.f, 0.f, 0.f, 0.f};
      Frag<E> fs[2][NSS];
      auto split_state = [&](int ks) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = accS[2 * ks][i];
          x[4 + i] = accS[2 * ks + 1][i];
        }
        split<NSS>(fs[ks & 1], x);
      };
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        if (ks == 0) split_state(0);
        if (ks < 3) split_state(ks + 1);
        if (DG && ks == 3) read_values(0);
#pragma unroll
        for (int s = 0; s < NSS; ++s)
#pragma unroll
          for (int rt = 0; rt < NT; ++rt) accO[rt] = mma(accO[rt], fs[ks & 1][s], fq[ks & 1][rt]);
        if constexpr (NSS > 1) {
          // the next step's operands are cut between this one's products
#pragma unroll
          for (int i = 0; i < NSS * NT; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
          }
        }
        if (ks < 2) read_q(base, ks + 2);
        else if (!DG) read_k(0, 2 * (ks - 2), 2);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (DG) {  // (no registers for them earlier)
        read_values(1);
        read_k(0, 0, 4);
      }
      weigh_values(0);
      TF fp[NT][KT];
#pragma unroll
      for (int rt = 0; rt < NT; ++rt)
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
          if (REV ? kt >= rt / TPS : kt <= rt / TPS)
            ld_pair(fp[rt][kt], lds0 + L::PAIR + (ci & 1) * (C * L::RB) + p_at[kt] + 16 * rt * L::RB);
      if constexpr (!DG) read_k(0, 4, 4);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) accO[rt] *= row[rt];
      if (gam == 0.f) {
        // the state is dropped in this chunk: rows behind that do not see it,
        // whatever it holds (infinities and NaN times zero would be NaN)
#pragma unroll
        for (int rt = 0; rt < NT; ++rt)
#pragma unroll
          for (int i = 0; i < 4; ++i) accO[rt][i] = row[rt] == 0.f ? 0.f : accO[rt][i];
      }
      if constexpr (DG) {
        float dot[NT];
#pragma unroll
        for (int rt = 0; rt < NT; ++rt) {
          Frag16<E> fx;
          fx.v = __builtin_bit_cast(decltype(fx.v), xr[rt]);
          const f32x4 x = frag16_to_f32(fx);
          dot[rt] = x[0] * accO[rt][0];
#pragma unroll
          for (int i = 1; i < 4; ++i) dot[rt] += x[i] * accO[rt][i];
        }
        int tile;
        const float sum = sum_groups(dot, g, tile);
        if (tile >= 0) sRX[((ci & 1) * NW + wv) * C + 16 * tile + l16] = sum;
      }
      if constexpr (DG) {
        load_x(ci + 1);
        read_k(0, 4, 4);
      }
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int rt = 0; rt < NT; ++rt)
          if (REV ? kt >= rt / TPS : kt <= rt / TPS) accO[rt] = mma_tok(accO[rt], fv[kt], fp[rt][kt]);
    } else {
      read_k(0, 0, 8);
      weigh_values(0);
    }
    if (NW == 8 && wv >= 4) __builtin_amdgcn_s_setprio(0);
    // the state's scale, when the decays have run far enough (decay wave)
    if (gam != 1.f) {
#pragma unroll
      for (int rt = 0; rt < 8; ++rt) accS[rt] *= gam;
      if (gam == 0.f) {
#pragma unroll
        for (int rt = 0; rt < 8; ++rt) accS[rt] = (f32x4){0.f, 0.f, 0.f, 0.f};
      }
    }
    // State.  The first step's products cover the second one's weighted values
    // and, as its keys come free, their reads; the second step's cover the
    // outputs' stores and the reads of the next chunk's queries (its tiles are
    // in LDS already; the last chunk reads what is there and drops it).
    static_assert(KT == 2, "two token steps a chunk");
    add_to_state(0);
    weigh_values(1);
    read_k(1, 0, 8);
    if constexpr (BF) {
#pragma unroll
      for (int i = 0; i < 8 * NSV; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
        if (i >= 8 * (NSV - 1)) __builtin_amdgcn_sched_group_barrier(0x100, Tok<E>::READS, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (OUT) {
      // rows behind the end fall outside the buffer view and are dropped
      const Rsrc orb = make_rsrc(static_cast<char*>(p.o) + ((size_t)t0 * H + h) * (D * oes),
                                 (uint32_t)(nv - 1) * o_row + D * oes);
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) {
        const int off = (int)(o_at + 16 * rt * o_row);
        if (!BF || (TR && p.o_f32)) {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, accO[rt]), orb, off, 0, 0);
        } else {
          const f32x4 t = accO[rt];
          const bf16x4 y = (bf16x4){(__bf16)t[0], (__bf16)t[1], (__bf16)t[2], (__bf16)t[3]};
          __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, y), orb, off, 0, 0);
        }
      }
    }
    add_to_state(1);
    read_q(base_next, 0);
    read_q(base_next, 1);
    base = base_next;
  }
  if constexpr (DG) chunk_barrier();  // the last chunk's sums
  if (OUT) {
    if (p.fin && (REV ? first : last)) store_state(p.fin + nh * kState, accS);
    if constexpr (DG && !REV)
      if (last && nch > 0) leave_state(stretches, accS);
  } else {
    store_state(p.snap + ((size_t)slot * H + h) * kState, accS);
  }
}

// Blocks b and b + 8 run on the same XCD: what the column blocks of a head and
// the heads that share a key head read comes from its L2 after the first.
template <int CB>
__device__ __forceinline__ int64_t unit_of(const LinearWalkArgs& p, int64_t block, int& cb) {
  const int share = p.num_heads / p.k_heads, per = share * CB;
  const int64_t slot8 = block >> 3;
  cb = (int)(slot8 % CB);
  return p.unit0 + (slot8 / per * 8 + (block & 7)) * share + slot8 % per / CB;
}

template <typename E, int NW>
__global__ __launch_bounds__(64 * (NW + 4)) void linear_walk_kernel(const LinearWalkArgs p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  int cb;
  const int64_t u = unit_of<8 / NW>(p, blockIdx.x, cb);
  if (u < p.units) walk<E, NW, false, false, true, false>(p, smem, u, cb);
}

// Every segment's own contribution to the state, forwards and, in the second
// half of the blocks if there are any, backwards.
template <typename E>
__global__ __launch_bounds__(64 * (8 + 4)) void linear_states_kernel(const LinearWalkArgs f, const LinearWalkArgs r,
                                                                    unsigned forward_blocks) {
  extern __shared__ __align__(1024) unsigned char smem[];
  int cb;
  if (blockIdx.x < forward_blocks) {
    const int64_t u = unit_of<1>(f, blockIdx.x, cb);
    if (u < f.units) walk<E, 8, false, false, false, false>(f, smem, u, cb);
  } else {
    const int64_t u = unit_of<1>(r, blockIdx.x - forward_blocks, cb);
    if (u < r.units) walk<E, 8, true, false, false, false>(r, smem, u, cb);
  }
}

// The three gradients' walks of every work item: per sequence (or segment) the
// dq and dk walks of all heads, which take longer, then the dv walks, those of
// the heads from dv_whole on by half heads.
template <typename E, int NW, bool DG>
__global__ __launch_bounds__(64 * (NW + 4)) void linear_grad_kernel(const LinearGradArgs p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  constexpr int CB = 8 / NW;
  const GradGrid grid(p.dq.num_heads, CB, p.dv_whole);
  const int H = p.dq.num_heads;
  const int64_t item = p.item0 + blockIdx.x / grid.blocks;
  int at = blockIdx.x % grid.blocks;  // b and b + 8 run on the same XCD
  auto head = [&](int cbs, int& part) {
    part = (at >> 3) % cbs;
    return (at >> 3) / cbs * 8 + (at & 7);
  };
  int part;
  if (at < grid.heavy) {
    const int h = head(2 * CB, part);
    if (h >= H) return;
    if (part < CB) walk<E, NW, true, true, true, DG>(p.dk, smem, item * H + h, part);
    else walk<E, NW, false, true, true, DG>(p.dq, smem, item * H + h, part - CB);
    return;
  }
  at -= grid.heavy;
  if (at < grid.whole) {
    const int h = head(CB, part);
    if (h < p.dv_whole) walk<E, NW, true, false, true, false>(p.dv, smem, item * H + h, part);
  } else if constexpr (NW == 8) {
    at -= grid.whole;
    const int h = p.dv_whole + head(2, part);
    if (h < H && threadIdx.x < 64 * (4 + 4)) walk<E, 4, true, false, true, false>(p.dv, smem, item * H + h, part);
  }
}

// A launch has fewer than 2^32 threads.
constexpr int64_t kMaxThreads = 0xffffffffll;

// Dynamic LDS above 64 KiB has to be asked for, once per device.
template <typename K>
hipError_t allow_lds(K kernel, int bytes, std::atomic<bool> (&set)[64]) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const bool known = dev >= 0 && dev < 64;
  if (known && set[dev].load(std::memory_order_relaxed)) return hipSuccess;
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess && known) set[dev].store(true, std::memory_order_relaxed);
  return e;
}

// Calls launch(first unit, units behind the last, blocks) for parts of a.units
// whose blocks make no more than `most_blocks`.
template <int CB, typename F>
hipError_t launch_parts(const LinearWalkArgs& a, int64_t most_blocks, const F& launch) {
  const int64_t group = 8 * (a.num_heads / a.k_heads);  // units that go to the XCDs together
  const int64_t most = std::max(most_blocks / (group * CB), (int64_t)1) * group;
  for (int64_t u = 0; u < a.units; u += most) {
    const int64_t end = std::min(a.units, u + most);
    launch(u, end, (unsigned)((end - u + group - 1) / group * group * CB));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename E, int NW>
hipError_t launch_walk_t(const LinearWalkArgs& a, hipStream_t stream) {
  constexpr int LDS = WalkLayout<E, NW, false, false>::BYTES, THREADS = 64 * (NW + 4);
  static std::atomic<bool> set[64];
  hipError_t e = allow_lds(linear_walk_kernel<E, NW>, LDS, set);
  if (e != hipSuccess) return e;
  return launch_parts<8 / NW>(a, kMaxThreads / THREADS, [&](int64_t u, int64_t end, unsigned blocks) {
    LinearWalkArgs part = a;
    part.unit0 = u;
    part.units = end;
    hipLaunchKernelGGL((linear_walk_kernel<E, NW>), dim3(blocks), dim3(THREADS), LDS, stream, part);
  });
}

template <typename E>
hipError_t launch_states_e(const LinearWalkArgs& forward, const LinearWalkArgs* reverse, hipStream_t stream) {
  constexpr int LDS = WalkLayout<E, 8, false, false>::BYTES, THREADS = 64 * (8 + 4);
  static std::atomic<bool> set[64];
  hipError_t e = allow_lds(linear_states_kernel<E>, LDS, set);
  if (e != hipSuccess) return e;
  return launch_parts<1>(forward, kMaxThreads / THREADS / 2, [&](int64_t u, int64_t end, unsigned blocks) {
    LinearWalkArgs f = forward, r = reverse ? *reverse : forward;
    f.unit0 = r.unit0 = u;
    f.units = r.units = end;
    hipLaunchKernelGGL(linear_states_kernel<E>, dim3(reverse ? 2 * blocks : blocks), dim3(THREADS), LDS, stream, f, r,
                       blocks);
  });
}

template <typename E, int NW, bool DG>
hipError_t launch_grad_t(const LinearGradArgs& a, hipStream_t stream) {
  constexpr int LDS = std::max({WalkLayout<E, NW, DG, DG>::BYTES, WalkLayout<E, NW, DG, false>::BYTES,
                                WalkLayout<E, NW, false, false>::BYTES, WalkLayout<E, 4, false, false>::BYTES});
  static std::atomic<bool> set[64];
  hipError_t e = allow_lds(linear_grad_kernel<E, NW, DG>, LDS, set);
  if (e != hipSuccess) return e;
  constexpr int THREADS = 64 * (NW + 4);
  const int64_t items = a.dq.units / a.dq.num_heads;
  const int per = GradGrid(a.dq.num_heads, 8 / NW, a.dv_whole).blocks;
  const int64_t most = kMaxThreads / THREADS / per;  // items of a launch (65535 heads: 28, by half heads 21)
  LinearGradArgs part = a;
  for (part.item0 = 0; part.item0 < items; part.item0 += most) {
    const int64_t blocks = std::min(items - part.item0, most) * per;
    hipLaunchKernelGGL((linear_grad_kernel<E, NW, DG>), dim3((unsigned)blocks), dim3(THREADS), LDS, stream, part);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename E>
hipError_t launch_grad_e(const LinearGradArgs& a, hipStream_t stream) {
  if (a.dq.narrow) return a.decay_grad ? launch_grad_t<E, 4, true>(a, stream) : launch_grad_t<E, 4, false>(a, stream);
  return a.decay_grad ? launch_grad_t<E, 8, true>(a, stream) : launch_grad_t<E, 8, false>(a, stream);
}

// ---------------------------------------------------------------------------
// The decays' gradient of one (stretch of `anchor` tokens, head):
//   D_t = <S, dS> at the stretch's end + sum over t' >= t of r_t' - c_t',
// in fp64, from the stretch's end on, 1024 tokens a turn (four a thread).  Bound
// by the states it reads (96 heads x 8192 tokens, stretches of 1024: 31 us for
// 107 MB).
// ---------------------------------------------------------------------------
__device__ __forceinline__ void decay_grad(const LinearDecayGradArgs& a) {
  constexpr size_t kState = (size_t)D * D;
  const int H = a.num_heads;
  const int h = (int)(blockIdx.x % H);
  const int64_t slot = blockIdx.x / H;
  const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
  __shared__ double part[4];
  auto block_sum = [&](double x) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m);
    if (lane == 0) part[wv] = x;
    __syncthreads();
    const double y = ((part[0] + part[1]) + part[2]) + part[3];
    __syncthreads();
    return y;
  };
  const Segment s = find_segment(a.cu, a.num_seqs, a.total_tokens, a.anchor, slot);
  double total = 0.0;
  if (s.ok && s.count > 0) {
    const int64_t tb = s.bos + (int64_t)s.j * a.anchor, te = min(s.eos, tb + (int64_t)a.anchor);
    double flow = 0.0;
    if (s.j + 1 < s.count || a.has_d_final) {
      const int64_t at = boundary_of(s.n, s.bos, a.anchor, a.has_d_final, s.j + 1);
      // (segments: what enters the next one, and what enters this one backwards)
      const float* S = a.s_anchors + ((size_t)(a.own ? at : slot + 1) * H + h) * kState;
      const float* M = a.ds_anchors + ((size_t)(a.own ? at : slot) * H + h) * kState;
      double d = 0.0;
      for (int i = 0; i < 16; ++i) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(S + i * 1024 + 4 * t);
        const f32x4 y = *reinterpret_cast<const f32x4*>(M + i * 1024 + 4 * t);
#pragma unroll
        for (int j = 0; j < 4; ++j) d += (double)x[j] * (double)y[j];
      }
      flow = block_sum(d);
    }
    const size_t half = (size_t)H * a.total_tokens;
    for (int64_t b = tb + (te - 1 - tb) / 1024 * 1024; b >= tb; b -= 1024) {
      double x[4];
      double mine = 0.0;
#pragma unroll
      for (int j = 3; j >= 0; --j) {
        const int64_t at = b + 4 * t + j;
        double c = 0.0;
        if (at < te) {
          const size_t i = (size_t)h * a.total_tokens + at;
          for (int k = 0; k < a.blocks; ++k) c += (double)a.r[k * half + i] - (double)a.c[k * half + i];
        }
        mine += c;
        x[j] = mine;  // from token at to the last of this thread's
      }
      // what the threads behind this one sum to
      double w = mine;
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) {
        const double o = __shfl_down(w, m);
        if (lane + m < 64) w += o;
      }
      if (lane == 0) part[wv] = w;
      __syncthreads();
      double behind = w - mine, all = 0.0;
#pragma unroll
      for (int k = 3; k >= 0; --k) {
        if (k > wv) behind += part[k];
        all += part[k];
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t at = b + 4 * t + j;
        if (at < te) {
          const double d = flow + behind + x[j];
          if (a.d_log_decay) a.d_log_decay[(size_t)at * H + h] = (float)d;
          total += d;
        }
      }
      flow += all;
    }
  }
  if (a.part) {
    const double y = block_sum(total);
    if (t == 0) a.part[blockIdx.x] = y;
  }
}

// ---------------------------------------------------------------------------
// Incoming state of every segment: the segments' contributions composed in
// order, elementwise (the decay of a segment is one scalar).  A thread owns
// four elements of one (sequence, head)'s state and reads the next segment's
// contribution while it composes this one.
// ---------------------------------------------------------------------------
template <bool REV>
__device__ __forceinline__ void scan(const LinearScanArgs& a, int64_t block) {
  constexpr size_t kState = (size_t)D * D;
  const int H = a.num_heads;
  const int64_t nh = a.unit0 + (block >> 4);
  const int at = ((int)(block & 15) * 256 + threadIdx.x) * 4;
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
    s = d == 0.f ? add : s * d + add;  // (a dropped state may hold anything)
  }
}

__global__ __launch_bounds__(256) void linear_scan_kernel(const LinearScanArgs f, const LinearScanArgs r,
                                                          unsigned forward_blocks) {
  if (blockIdx.x < forward_blocks) scan<false>(f, blockIdx.x);
  else scan<true>(r, blockIdx.x - forward_blocks);
}

// ---------------------------------------------------------------------------
// What follows the gradients' walks, in one launch: the decays' gradient, and
// the gradients of shared query and key heads, summed over the value heads that
// share one, in order (four consecutive channels per thread).
// ---------------------------------------------------------------------------
template <typename E>
__global__ __launch_bounds__(256) void linear_finish_kernel(const LinearFinishArgs a) {
  int64_t b = blockIdx.x;
  if (b < a.decay_blocks) {
    decay_grad(a.decay);
    return;
  }
  b -= a.decay_blocks;
  const bool of_dk = b >= a.share_blocks;
  if (of_dk) b -= a.share_blocks;
  const LinearDecayGradArgs& d = a.decay;
  const int64_t T = d.cu ? clamp_cu(d.cu, d.num_seqs, d.total_tokens) : d.total_tokens;
  const int share = d.num_heads / a.qk_heads;
  const float* src = a.share + (of_dk ? (size_t)d.total_tokens * d.num_heads * D : 0);
  E* dst = static_cast<E*>(of_dk ? a.dk : a.dq);
  const int64_t rows = T * a.qk_heads;
  for (int64_t i = b * 256 + threadIdx.x; (i >> 5) < rows; i += a.share_blocks * 256) {
    const int64_t row = i >> 5;
    const int ch = (int)(i & 31) * 4;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < share; ++j) s += *reinterpret_cast<const f32x4*>(src + (row * share + j) * D + ch);
    store_row4(dst + row * D + ch, s);
  }
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
  if (a.narrow) return a.bf16 ? launch_walk_t<__bf16, 4>(a, stream) : launch_walk_t<float, 4>(a, stream);
  return a.bf16 ? launch_walk_t<__bf16, 8>(a, stream) : launch_walk_t<float, 8>(a, stream);
}

hipError_t launch_linear_states(const LinearWalkArgs& f, const LinearWalkArgs* r, hipStream_t stream) {
  return f.bf16 ? launch_states_e<__bf16>(f, r, stream) : launch_states_e<float>(f, r, stream);
}

hipError_t launch_linear_grad(const LinearGradArgs& a, hipStream_t stream) {
  return a.dq.bf16 ? launch_grad_e<__bf16>(a, stream) : launch_grad_e<float>(a, stream);
}

// Workgroups for the sums of dq, and as many for dk, over shared heads (they go
// on by strides): with the 14 * 2^20 stretches that a call may have at most
// (kda_linear_api.hip), 2^24 - 2 of 256 threads.
constexpr int64_t kMostShareBlocks = ((int64_t)1 << 20) - 1;
static_assert((((int64_t)14 << 20) + 2 * kMostShareBlocks) * 256 <= kMaxThreads, "one launch holds both");

hipError_t launch_linear_finish(LinearFinishArgs a, bool bf16, hipStream_t stream) {
  const LinearDecayGradArgs& d = a.decay;
  a.decay_blocks = a.decay_blocks ? linear_slots(d.total_tokens, d.num_seqs, d.anchor) * d.num_heads : 0;
  a.share_blocks = a.share ? std::min((d.total_tokens * a.qk_heads * 32 + 255) / 256, kMostShareBlocks) : 0;
  const int64_t blocks = a.decay_blocks + 2 * a.share_blocks;
  if (blocks == 0) return hipSuccess;
  if (bf16) hipLaunchKernelGGL(linear_finish_kernel<__bf16>, dim3((unsigned)blocks), dim3(256), 0, stream, a);
  else hipLaunchKernelGGL(linear_finish_kernel<float>, dim3((unsigned)blocks), dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_linear_scan(LinearScanArgs f, const LinearScanArgs* reverse, hipStream_t stream) {
  const int64_t units = (int64_t)f.num_seqs * f.num_heads;
  constexpr int64_t MOST = kMaxThreads / 256 / 32;
  LinearScanArgs r = reverse ? *reverse : f;
  for (int64_t u = 0; u < units; u += MOST) {
    f.unit0 = r.unit0 = u;
    const unsigned blocks = (unsigned)(std::min(units - u, MOST) * 16);
    hipLaunchKernelGGL(linear_scan_kernel, dim3(reverse ? 2 * blocks : blocks), dim3(256), 0, stream, f, r, blocks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_linear_decay_sum(const double* part, float* dst, int64_t units, int num_heads, hipStream_t stream) {
  hipLaunchKernelGGL(linear_decay_sum_kernel, dim3((unsigned)num_heads), dim3(64), 0, stream, part, dst, units,
                     num_heads);
  return hipGetLastError();
}

}  // namespace kda
