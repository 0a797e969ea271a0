// The gated delta rule, 64 tokens at a time.
//
// With G_i the sum of g up to token i of a chunk (in a tree: down its path) and "before" the tokens before (ancestors of) one,
//   (I + A) U = diag(beta) (V - diag(e^G) K S),   A_ij = beta_i e^(G_i - G_j) k_i . k_j   for j before i,
//   out = scale (diag(e^G) Q S + (e^(G_i - G_j) q_i . k_j) U),    S' = e^G_last S + sum_j e^(G_last - G_j) k_j u_j^T.
// k_delta_terms makes what does not depend on S, for all chunks at once: T = (I + A)^-1, the factors P of out and the rows'
// scalars.  k_delta_scan walks through a sequence's chunks with 16 columns of S in a wave's registers.
//
// Matrix instructions: 16x16x32 BF16.  Their results (a lane: one column, 4 neighbouring rows) are the next ones' right operand
// (a lane: one column, 8 of the summed index) without a move: where a result's rows are tokens, T and P are laid out in
// the order that this gives, and where they are S's, the rows of S are numbered so that it is the order of K in memory.
// k, q and v are BF16 and exact; what is FP32 (S, R, T, U, P) goes in as two BF16 values (hi + lo, off by 2^-16 at most; of T R and P U
// without the product of the two lows).  So the states keep nearly all of FP32 (2.7e-6 of their norm after 4096 tokens; the recurrence in
// FP32 1e-7), and out is off by its rounding to BF16 alone (0.0017 of its norm; with S and U as one value each 0.0026, and a tree's outputs
// further from those of its tokens one by one than their rounding).  T is made in FP32 throughout: 16 x 16 blocks by substitution (which
// does not cancel as powers of A would), joined by FP32 matrix instructions.
//
// Measured, 48 heads of 128 x 128 over 16 of keys: a prompt of 4096 186 us (terms 46, scan 143: 64 chunks, one after another, on 96 of 256
// compute units), a tree of 63 nodes 16 (10 and 6), 16 trees of 24 nodes 47, seven prompts of 21834 tokens together, 32 heads, 405.  The scan
// is bound by the waves that carry S: of a chunk's 5600 cycles, with the cycle counter noted, K S and S's split are 1700 to 2000, U 1000, the
// search for values that are no numbers 500, S' 1500.  Hence the waves for loads and outputs beside them, whose traffic in LDS they
// wait for: with S and U as one value each for out, half of that, the times were 159, 16, 45 and 363 us.  32 columns a work-group
// were faster then for a prompt alone (142 against 158) and slower where work-groups fill the chip (467 against 346).  The terms wait for their
// loads and for one another's phases, at 5 work-groups a compute unit.
#include "w12_delta_chunk.h"
#include "w12_delta_steps.h"
#include "w12_gemm_common.h"
#include "w12_lanes.h"
#include "w12_kernels.h"
#include "w12_rows.h"
#include "w12_sequences.h"

#include <algorithm>

namespace w12 {

typedef float f32x4v __attribute__((ext_vector_type(4)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

constexpr int kChunkThreads = 256;

__device__ __forceinline__ f32x4v mma(bf8 a, bf8 b, f32x4v c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ f32x4v mma32(float a, float b, f32x4v c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }
// a 16 x 16 product of FP32: a holds A[row][4 g .. 4 g + 3] of the lane's row, b a result (its column, rows 4 g .. 4 g + 3)
__device__ __forceinline__ f32x4v mma_block(f32x4v a, f32x4v b, f32x4v c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c = mma32(a[i], b[i], c);
  return c;
}

__device__ __forceinline__ bool finite(float v) { return fabsf(v) < INFINITY; }

// v where bit b of m is set, else 0; one of four.  By bits: choices between values become branches here.
__device__ __forceinline__ float where_bit(uint32_t m, int b, float v) {
  return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v) & (uint32_t)__builtin_amdgcn_sbfe((int)m, b, 1));
}
__device__ __forceinline__ float pick(int i, float a, float b, float c, float d) {
  const uint32_t m = 1u << i;
  return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, where_bit(m, 0, a)) | __builtin_bit_cast(uint32_t, where_bit(m, 1, b)) |
                                       __builtin_bit_cast(uint32_t, where_bit(m, 2, c)) | __builtin_bit_cast(uint32_t, where_bit(m, 3, d)));
}

// Eight FP32 values as BF16, and what that leaves over as BF16.
__device__ __forceinline__ bf8 high(f32x4v a, f32x4v b) {
  const u32x4v r = {bf16_pair(a[0], a[1]), bf16_pair(a[2], a[3]), bf16_pair(b[0], b[1]), bf16_pair(b[2], b[3])};
  return __builtin_bit_cast(bf8, r);
}
__device__ __forceinline__ bf8 low(f32x4v a, f32x4v b, bf8 hi) {
  const u32x4v h = __builtin_bit_cast(u32x4v, hi);
  u32x4v r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = i < 2 ? a[2 * i] : b[2 * i - 4], y = i < 2 ? a[2 * i + 1] : b[2 * i - 3];
    float xh;
    asm("v_lshlrev_b32 %0, 16, %1" : "=v"(xh) : "v"(h[i]));      // written as a shift it becomes a second conversion, and the shift
    r[i] = bf16_pair(x - xh, y - __builtin_bit_cast(float, h[i] & 0xFFFF0000u));
  }
  return __builtin_bit_cast(bf8, r);
}

// Rows of keys or queries in LDS: 16-byte pieces, swizzled by row so that neither the reads of a column of pieces (16 rows; taken
// as lanes 0-3, 12-15 and 20-27, and their like) nor, with 16 pieces, the turning reads of 4 pieces of 4 rows meet in a bank.
template <int DK>
__device__ __forceinline__ int piece_at(int row, int piece) {
  constexpr int P = DK / 8;
  const int q = row >> 2 & 3;
  const int s = P == 16 ? (row & 3) << 2 | ((q ^ q >> 1) & 1) << 1 | q >> 1 : row >> 1 & 7;
  return (row * P + (piece ^ s)) * 16;
}
// A lane's operand of rows 16 rt .. + 15 (row lane % 16) and values 32 ks + 8 (lane / 16) .. + 7.
template <int DK>
__device__ __forceinline__ bf8 rows_operand(const char* m, int rt, int ks) {
  const int lane = threadIdx.x & 63;
  return *reinterpret_cast<const bf8*>(m + piece_at<DK>(16 * rt + (lane & 15), 4 * ks + (lane >> 4)));
}

// Whether a sequence's tokens are taken 64 at a time, which goes by their own number (and the form) alone: between 8 (48 heads of 128, 1 / 4 /
// 16 / 64 sequences: 13 / 18 / 41 / 131 us token by token, 15 / 24 / 60 / 212 in chunks) and 16 (21 / 29 / 65 / 215 and 15 / 25 / 59 / 216).
__device__ __forceinline__ bool taken_in_chunks(const w12_sequences& s, const Range& r) { return s.tree_mask || r.n >= W12_DELTA_CHUNK_FROM; }

// Sequence number j of those; false where there are fewer.  A wave looks at 64 at a time.
__device__ __forceinline__ bool find_long(const w12_sequences& s, int j, int& b, Range& r) {
  if (s.tree_mask) {
    b = j;
    if (j < s.count) r = range_of(s, b);
    return j < s.count;
  }
  for (int b0 = 0; b0 < s.count; b0 += 64) {
    const int i = b0 + (threadIdx.x & 63);
    Range mine = {0, 0};
    if (i < s.count) mine = range_of(s, i);
    uint64_t longs = __ballot(taken_in_chunks(s, mine));
    const int n = __builtin_popcountll(longs);
    if (j < n) {
      while (j-- > 0) longs &= longs - 1;
      const int l = __builtin_ctzll(longs);
      b = b0 + l;
      r.start = __builtin_amdgcn_readlane(mine.start, l);
      r.n = __builtin_amdgcn_readlane(mine.n, l);
      return true;
    }
    j -= n;
  }
  return false;
}

// ------------------------------------------------------------------------------------------- terms

// Work-groups from `pieces` on have no chunk: they take the short sequences, beside the others.
template <int DK>
__global__ __launch_bounds__(kChunkThreads, 4) void k_delta_terms(w12_delta_args a, w12_sequences s, char* ws, int pieces) {
  static_assert(kChunkThreads == kDeltaThreads, "a work-group takes either");
  constexpr int KS = DK / 32;
  // keys, and once they are used the inverses of A's diagonal blocks
  union Shared {
    char k[kChunk * DK * 2];
    struct {
      f32x4v d[4][64];                           // a lane's column, rows 4 g .. + 3
      float turn[4][16][20];
    } inverse;
  };
  __shared__ __attribute__((aligned(16))) Shared lds;
  __shared__ f32x4v ablk[10][64];                // A's blocks (r, s), r >= s: a lane's column, rows 4 g .. + 3
  __shared__ __attribute__((aligned(16))) float rk[kChunk], rq[kChunk], beta[kChunk], br[kChunk], gh[kChunk], gl[kChunk];
  __shared__ __attribute__((aligned(16))) uint32_t anc[2][kChunk];      // lower and upper halves
  __shared__ int found[2];
  const int tid = threadIdx.x, lane = tid & 63, w = wave_id(), c16 = lane & 15, g4 = lane >> 4;
  const int h = blockIdx.y, hk = h / (a.v_heads / a.k_heads);
  if ((int)blockIdx.x >= pieces) {
    const int i = blockIdx.x - pieces, blocks = a.dv / kGroupColumns;
    delta_steps<DK>(a, s, i / blocks, h, i % blocks, W12_DELTA_CHUNK_FROM - 1);
    return;
  }
  if (blockIdx.x == 0 && h == 0 && tid < kZeroBytes / 16) reinterpret_cast<uint4*>(ws)[tid] = make_uint4(0, 0, 0, 0);
  int b, chunk;
  Range r;
  if (!find_piece(s, blockIdx.x, kChunk, found, b, r, chunk)) return;
  const int first = chunk * kChunk, m = min(kChunk, r.n - first);
  if (m <= 0 || !taken_in_chunks(s, r)) return;
  auto row_at = [&](int i) { return i < m ? row_of(s, r.start + first + i) : -1; };
  auto operand = [&](const uint16_t* p, int64_t ld, int row, bf8 x[KS]) {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      u32x4v u = {0, 0, 0, 0};
      if (row >= 0) u = *reinterpret_cast<const u32x4v*>(p + row * ld + hk * DK + 32 * ks + 8 * g4);
      x[ks] = __builtin_bit_cast(bf8, u);
    }
  };
  // Tile w of K, the tiles of Q that this wave's fragments are of, and (all waves) decays and strengths of every row.
  bf8 kt[KS], qt[2][KS];
  const int krow = row_at(16 * w + c16);
  operand(a.k, a.ldk, krow, kt);
  const int q0 = w == 0 ? 0 : w == 1 ? 2 : 3;
  const int qrow = a.q ? row_at(16 * q0 + c16) : -1, qrow1 = a.q && w == 0 ? row_at(16 + c16) : -1;
  operand(a.q, a.ldq, qrow, qt[0]);
  if (w == 0) operand(a.q, a.ldq, qrow1, qt[1]);
  const int lrow = row_at(lane);
  float gv = 0.0f, bv = 0.0f;
  if (lrow >= 0) {
    gv = a.g[lrow * a.ldg + h];
    bv = a.beta[lrow * a.ldbeta + h];
  }
  const uint64_t path = lane < m ? ancestors(s, r.start + first, lane) : 0;
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) *reinterpret_cast<bf8*>(lds.k + piece_at<DK>(16 * w + c16, 4 * ks + g4)) = kt[ks];
  // (the barriers from here on are for LDS alone: stores to memory take their time beside them)
  // squares of the norms: the diagonal of a tile with itself, which lanes of 4 g + i = c16 hold
  auto square = [&](const bf8 x[KS]) {
    f32x4v t = {0, 0, 0, 0};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) t = mma(x[ks], x[ks], t);
    return pick(c16 & 3, t[0], t[1], t[2], t[3]);
  };
  const bool diagonal = g4 == c16 >> 2;
  auto over_norm = [&](float squares) {
    const float sum = squares + a.eps;
    return !a.l2norm ? 1.0f : has_norm(sum) ? __builtin_amdgcn_rsqf(sum) : NAN;
  };
  const float kk = square(kt);
  if (diagonal) rk[16 * w + c16] = krow < 0 ? 0.0f : finite(kk) ? over_norm(kk) : NAN;
  if (a.q) {
    const float qq = square(qt[0]);
    if (diagonal && w < 3) rq[16 * q0 + c16] = qrow < 0 ? 0.0f : a.scale * over_norm(qq);
    if (w == 0) {
      const float qq1 = square(qt[1]);
      if (diagonal) rq[16 + c16] = qrow1 < 0 ? 0.0f : a.scale * over_norm(qq1);
    }
  }
  lds_barrier();
  // A row whose key, decay or strength is no number is left out here, and made up for where the results are stored.  -inf is a number for
  // a decay: like anything below -1e4 it clears the state.
  const float ikl = rk[lane];
  const bool bad = !finite(ikl) || !(gv < INFINITY) || !finite(bv);
  const uint64_t bads = __ballot(bad);
  const double g1 = bad ? 0.0 : (double)fmaxf(gv, -1e4f) * 1.4426950408889634;
  double gsum;
  if (s.tree_mask) {
    if (w == 0) *reinterpret_cast<double*>(&ablk[0][lane]) = g1;
    lds_barrier();
    gsum = g1;
    for (uint64_t p = path; p; p &= p - 1) gsum += *reinterpret_cast<const double*>(&ablk[0][__builtin_ctzll(p)]);
  } else {
    gsum = sum_up(g1);
  }
  const uint64_t gbits = __builtin_bit_cast(uint64_t, gsum);
  const double last = __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(gbits >> 32), 63) << 32 |
                                                     (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)gbits, 63));
  Terms out(ws + kZeroBytes, (int64_t)blockIdx.x * a.v_heads + h);
  const float rkl = bad ? 0.0f : ikl;
  if (w == 0) {
    const float hi = (float)gsum;
    gh[lane] = hi;
    gl[lane] = (float)(gsum - hi);
    beta[lane] = bad ? 0.0f : bv;
    br[lane] = bad ? 0.0f : bv * ikl;
    const uint64_t mine = bad ? 0 : path & ~bads;
    anc[0][lane] = (uint32_t)mine;
    anc[1][lane] = (uint32_t)(mine >> 32);
  } else if (w == 1) {
    const float grown = __builtin_amdgcn_exp2f((float)gsum);
    float* rows = out.rows();
    rows[kTaken + lane] = grown * rkl;
    rows[kLeft + lane] = __builtin_amdgcn_exp2f((float)(last - gsum)) * rkl;
    if (lane == 0) {
      rows[kGrown] = __builtin_amdgcn_exp2f((float)last);
      reinterpret_cast<uint64_t*>(rows)[kBad / 2] = bads;
    }
  } else if (w == 2 && a.q) {
    out.out_rows()[lane] = __builtin_amdgcn_exp2f((float)gsum) * rq[lane];
  }
  lds_barrier();
  // This wave's fragments of P (rt, ks): (0, 0) and (1, 0), (2, 0) and (2, 1), (3, 0), (3, 1), tile by tile; and the same tiles of A.
  // A: a lane's column, 4 neighbouring rows; P turned: a lane's row, 4 neighbouring columns.  A loop: where work-groups are few, a kernel
  // that runs through its code once waits for the code.
#pragma unroll 1
  for (int j = 0; j < (w < 2 ? 4 : 2); ++j) {
    const int rt = w == 0 ? j >> 1 : w == 1 ? 2 : 3, t = w == 0 ? j & 1 : w == 3 ? 2 + j : j, half = t >> 1;
    if (w == 0 && j == 2) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) qt[0][ks] = qt[1][ks];
    }
    f32x4v pt = {0, 0, 0, 0};
    if (t <= rt) {
      f32x4v kk = {0, 0, 0, 0}, kq = kk;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const bf8 x = rows_operand<DK>(lds.k, t, ks);
        kk = mma(rows_operand<DK>(lds.k, rt, ks), x, kk);
        kq = mma(x, qt[0][ks], kq);
      }
      // A: column 16 t + c16, rows 16 rt + 4 g4 ..; P: row 16 rt + c16, columns 16 t + 4 g4 ..
      const int bit = 16 * (t & 1), arow = 16 * rt + 4 * g4, acol = 16 * t + c16, prow = 16 * rt + c16, pcol = 16 * t + 4 * g4;
      const auto at4 = [](const float* p) { return *reinterpret_cast<const f32x4v*>(p); };
      const f32x4v ha = at4(gh + arow), la = at4(gl + arow), ba = at4(br + arow), hp = at4(gh + pcol), lp = at4(gl + pcol), rp = at4(rk + pcol);
      const u32x4v ma = *reinterpret_cast<const u32x4v*>(anc[half] + arow);
      const float hc = gh[acol], lc = gl[acol], rc = rk[acol], hr = gh[prow], lr = gl[prow], rr = rq[prow];
      const uint32_t self = prow >> 5 == half ? 1u << (prow & 31) : 0u;
      const uint32_t sees = (anc[half][prow] | self) & ~(uint32_t)(bads >> 32 * half);
      f32x4v ab;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e = __builtin_amdgcn_exp2f((ha[i] - hc) + (la[i] - lc));
        ab[i] = where_bit(ma[i], bit + c16, ba[i] * rc * e * kk[i]);
        const float f = __builtin_amdgcn_exp2f((hr - hp[i]) + (lr - lp[i]));
        pt[i] = where_bit(sees, bit + 4 * g4 + i, rr * rp[i] * f * kq[i]);
      }
      ablk[block_of(rt, t)][lane] = ab;
    }
    if (a.q) {
      const uint2 hi = make_uint2(bf16_pair(pt[0], pt[1]), bf16_pair(pt[2], pt[3]));
      const auto over = [](float x, float y, uint32_t h) { return bf16_pair(x - bf16_float(h), y - __builtin_bit_cast(float, h & 0xFFFF0000u)); };
      const int f = fragment_of(rt, half);
      reinterpret_cast<uint2*>(out.p(f) + lane)[t & 1] = hi;
      reinterpret_cast<uint2*>(out.p_low(f) + lane)[t & 1] = make_uint2(over(pt[0], pt[1], hi.x), over(pt[2], pt[3], hi.y));
    }
  }
  lds_barrier();
  // the inverse of diagonal block w: a lane's column by substitution (the four groups of lanes do the same)
  float d[16];
  {
    const f32x4v* const blk = ablk[block_of(w, w)];      // [16 (row / 4) + column], row % 4
#pragma unroll
    for (int i = 0; i < 16; ++i) d[i] = i == c16 ? 1.0f : 0.0f;
#pragma unroll
    for (int j = 0; j < 15; ++j)
#pragma unroll
      for (int q = j / 4; q < 4; ++q) {
        const f32x4v x = blk[16 * q + j];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * q + i > j) d[4 * q + i] -= x[i] * d[j];
      }
  }
  f32x4v mine;
#pragma unroll
  for (int i = 0; i < 4; ++i) mine[i] = pick(g4, d[i], d[4 + i], d[8 + i], d[12 + i]);
  lds.inverse.d[w][lane] = mine;
#pragma unroll
  for (int i = 0; i < 4; ++i) lds.inverse.turn[w][4 * g4 + i][c16] = mine[i];
  lds_barrier();
  // block row w of T, turned: X_w = D_w^T, X_t = -D_t^T sum_{t < u <= w} A_ut^T X_u
  f32x4v x[4];
#pragma unroll
  for (int t = 3; t >= 0; --t) {
    x[t] = f32x4v{0, 0, 0, 0};
    if (t == w) x[t] = *reinterpret_cast<const f32x4v*>(&lds.inverse.turn[w][c16][4 * g4]);
    if (t >= w) continue;
    f32x4v sum = {0, 0, 0, 0};
#pragma unroll
    for (int u = 3; u > t; --u)
      if (u <= w) sum = mma_block(ablk[block_of(u, t)][lane], x[u], sum);
    const f32x4v none = {0, 0, 0, 0};
    x[t] = none - mma_block(lds.inverse.d[t][lane], sum, none);
  }
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    if (ks > w >> 1) continue;
    const int f = fragment_of(w, ks);
#pragma unroll
    for (int t = 2 * ks; t < 2 * ks + 2; ++t) x[t] *= *reinterpret_cast<const f32x4v*>(beta + 16 * t + 4 * g4);
    const bf8 hi = high(x[2 * ks], x[2 * ks + 1]);
    out.t_high(f)[lane] = hi;
    out.t_low(f)[lane] = low(x[2 * ks], x[2 * ks + 1], hi);
  }
}

// -------------------------------------------------------------------------------------------- scan

// 16 bytes a lane from memory to the wave's 1 KB of LDS at `at`.  Not through the builtin: the compiler would wait for it before
// every read of LDS.
__device__ __forceinline__ void to_lds(const void* from, uint32_t at) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               : : "s"(__builtin_amdgcn_readfirstlane((int)at)), "v"(from) : "memory", "m0");
}
__device__ __forceinline__ void to_lds(uint64_t base, uint32_t off, uint32_t at) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               : : "s"(__builtin_amdgcn_readfirstlane((int)at)), "v"(off), "s"(base) : "memory", "m0");
}

// Waves of a work-group: one for every 16 columns of S, one on each SIMD; one for the outputs of two of those; the others for the
// loads (a wave starts one to LDS in 75 cycles or more, a chunk takes 44).
constexpr int kTiles = 4, kScanColumns = 16 * kTiles, kOuts = kTiles / 2, kScanThreads = 512, kLoaders = kScanThreads / 64 - kTiles - kOuts;

// What a chunk has in LDS.  A step has two barriers.  S before the chunk is written before the one in its middle and read after it, U the other
// way round, so that neither needs a second buffer, for which there would be no room.
template <int DK>
struct ScanLds {
  char k[3][kChunk * DK * 2];
  struct {
    char first[kFirstPages * 1024];              // terms
    char v[kChunk * kScanColumns * 2];
  } chunk[2];
  bf8 s[2][kTiles][DK / 32][64];                 // for the outputs: S before the chunk (high, low),
  bf8 u[2][kTiles][2][64];                       // U (high, low),
  uint64_t bad[kTiles][16];                      // and by column the tokens that were no numbers
  char second[2][kSecondPages * 1024];
};

// 16 bytes of LDS at an address.
__device__ __forceinline__ u32x4v lds_at(uint32_t at) { return *reinterpret_cast<__attribute__((address_space(3))) const u32x4v*>(at); }

__device__ __forceinline__ bf8 turned(uint32_t at, int further) {
  const i16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_i16x4*>(at));
  const i16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_i16x4*>(at + further));
  return __builtin_bit_cast(bf8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Asks the scheduler for N matrix instructions, each with so many vector instructions and reads of LDS behind it: they run beside it, if
// they stand there (a wave issues in order).
template <int N, int VECTOR, int READS>
__device__ __forceinline__ void beside_matrix() {
  if constexpr (N > 0) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (READS > 0) __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
    if constexpr (VECTOR > 0) __builtin_amdgcn_sched_group_barrier(0x002, VECTOR, 0);
    beside_matrix<N - 1, VECTOR, READS>();
  }
}

template <int DK, bool ROWS, bool MANY>
__global__ __launch_bounds__(kScanThreads) void k_delta_scan(w12_delta_args a, w12_sequences s, const char* ws) {
  constexpr int KS = DK / 32, RT = DK / 16;
  __shared__ __attribute__((aligned(1024))) ScanLds<DK> lds;
  const int lane = threadIdx.x & 63, w = wave_id(), c16 = lane & 15, g4 = lane >> 4;
  // the column blocks of a head read the same rows and terms: neighbours, on one XCD
  const int blocks = a.dv / kScanColumns;
  // (and every sequence on all of them: lengths differ)
  const int of = blocks * a.v_heads, at = (int)logical_wg(blockIdx.x % of, of);
  const int cb = at % blocks, h = at / blocks;
  const int hk = h / (a.v_heads / a.k_heads);
  const int col0 = cb * kScanColumns;
  // The sequences that are taken 64 at a time: this work-group's, one, or with MANY one after another.  Of LDS, what a sequence's waves read
  // last, the next one's write behind its first barrier.
  int number = blockIdx.x / of, b;
  Range r;
  bool there = find_long(s, number, b, r);
  auto next = [&] {
    if constexpr (!MANY) return false;
    number += gridDim.x / of;
    return find_long(s, number, b, r);
  };

  if (w >= kTiles + kOuts) {
    for (; there; there = next()) {
      const int chunks = (r.n + kChunk - 1) / kChunk;
      // ---- loads: of K and V a lane's places in a chunk, of the terms whole pages
      const int me = w - kTiles - kOuts;
      constexpr int kLanes = DK / 8, kRows = 64 / kLanes, kEach = kChunk / kRows / kLoaders;
      constexpr int kVLanes = kScanColumns / 8, kVRows = 64 / kVLanes, kVEach = kChunk / kVRows / kLoaders;
      const char* const zeros = ws;                // the first row of the workspace
      const char *kp[kEach], *vp[kVEach];
      auto row_in = [&](int i) { return (me * kEach + i) * kRows + lane / kLanes; };
      auto vrow_in = [&](int i) { return (me * kVEach + i) * kVRows + lane / kVLanes; };
      auto from = [&](const uint16_t* m, int64_t ld, int row, int64_t at) { return reinterpret_cast<const char*>(m + row * ld + at); };
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int piece = (piece_at<DK>(row_in(i), lane % kLanes) >> 4) % kLanes;      // that belongs in this place
        kp[i] = from(a.k, a.ldk, ROWS ? 0 : r.start + row_in(i), hk * DK + piece * 8);
      }
#pragma unroll
      for (int i = 0; i < kVEach; ++i)
        vp[i] = from(a.v, a.ldv, ROWS ? 0 : r.start + vrow_in(i), h * a.dv + col0 + lane % kVLanes * 8);
      const int64_t kstep = kChunk * 2 * a.ldk, vstep = kChunk * 2 * a.ldv;
      // `p`: of the chunk that is fetched; with rows, of row 0
      auto send = [&](const char*& p, int64_t step, int64_t ld, int chunk, int row, const char* to) {
        const char* x = p;
        const int token = chunk * kChunk + row;
        if constexpr (ROWS) {
          const int in = token < r.n ? row_of(s, r.start + token) : -1;
          x = in >= 0 ? p + in * (2 * ld) : zeros;
        } else {
          if ((chunk + 1) * kChunk > r.n) x = token < r.n ? p : zeros;
          p += step;
        }
        to_lds(x, lds_off(to));
      };
      auto fetch_k = [&](int chunk, int buf) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) send(kp[i], kstep, a.ldk, chunk, row_in(i), lds.k[buf] + (me * kEach + i) * 1024);
      };
      auto fetch_v = [&](int chunk) {
#pragma unroll
        for (int i = 0; i < kVEach; ++i) send(vp[i], vstep, a.ldv, chunk, vrow_in(i), lds.chunk[chunk & 1].v + (me * kVEach + i) * 1024);
      };
      const uint64_t terms = (uint64_t)(uintptr_t)ws + kZeroBytes + ((int64_t)first_piece(r, b, kChunk) * a.v_heads + h) * kTermsBytes;
      const uint64_t terms_step = (uint64_t)a.v_heads * kTermsBytes;
      auto fetch_pages = [&](uint64_t from, int pages, int mine, const char* to) {
#pragma unroll
        for (int i = 0; i < (kFirstPages + kLoaders - 1) / kLoaders; ++i) {
          const int page = i * kLoaders + mine;
          if (page < pages) to_lds(from, (uint32_t)(page * 1024 + lane * 16), lds_off(to) + page * 1024);
        }
      };
      auto fetch_first = [&](int chunk) { fetch_pages(terms + chunk * terms_step, kFirstPages, me, lds.chunk[chunk & 1].first); };
      if (chunks) {
        fetch_k(0, 0);
        fetch_first(0);
        fetch_v(0);
      }
      if (chunks > 1) fetch_k(1, 1);
      wait_vm_all();
      barrier();
      int k2 = 2;
      for (int c = 0; c < chunks; ++c) {
        if (c + 1 < chunks) {
          fetch_first(c + 1);
          fetch_v(c + 1);
        }
        if (a.q) fetch_pages(terms + c * terms_step + kFirstPages * 1024, kSecondPages, kLoaders - 1 - me, lds.second[c & 1]);
        if (c + 2 < chunks) fetch_k(c + 2, k2);
        k2 = k2 == 2 ? 0 : k2 + 1;
        barrier();
        wait_vm_all();
        barrier();
      }
    }
    return;
  }

  if (w >= kTiles) {
    for (; there; there = next()) {
      const int chunks = (r.n + kChunk - 1) / kChunk;
      // ---- outputs, half of the tokens a wave (tiles 0 and 3, or 1 and 2: 3 fragments of P each), turned: a lane's token (of each 16), and of
      // every two tiles 8 neighbouring columns, so that it stores 16 bytes.
      const int half = w - kTiles, tile[2] = {half, 3 - half};
      bf8 q[KS][2], pl[3];
      const char* const terms = ws + kZeroBytes + ((int64_t)first_piece(r, b, kChunk) * a.v_heads + h) * kTermsBytes;
      // P's second matrix has no room in LDS
      auto read_p = [&](int chunk) {
        const Terms from(const_cast<char*>(terms), (int64_t)chunk * a.v_heads);
#pragma unroll
        for (int i = 0; i < 3; ++i) pl[i] = from.p_low(fragment_of(tile[(i + 1) / 2], i / 2))[lane];
      };
      // (of tokens that are not there any row will do: a token's query makes its own output only)
      auto read_q = [&](int chunk) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int token = min(chunk * kChunk + 16 * tile[j] + c16, r.n - 1);
          const int row = ROWS ? max(row_of(s, r.start + token), 0) : r.start + token;
          const u32x4v* p = reinterpret_cast<const u32x4v*>(a.q + row * a.ldq + hk * DK) + g4;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) q[ks][j] = __builtin_bit_cast(bf8, p[4 * ks]);
        }
      };
      if (a.q && chunks) {
        read_q(0);
        read_p(0);
      }
      barrier();
      f32x4v o[kTiles][2];
      bf8 sw[2][kTiles][KS];
      auto add_qs = [&](int part) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int n = 0; n < kTiles; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) o[n][j] = mma(sw[part][n][ks], q[ks][j], o[n][j]);
      };
      // The rest of the chunk's Q S, e^G of it, and P U (U first from LDS, which answers while the lows of S run).
      auto add_pu = [&](int chunk) {
        const char* const second = lds.second[chunk & 1];
        const bf8* const pf = reinterpret_cast<const bf8*>(second) + lane;
        const float* const rows = reinterpret_cast<const float*>(second + kFragments * 1024) + c16;
        bf8 uw[2][kTiles][2], p[3];       // p: of tile[0], of tile[1], and of its later tokens
        float scale[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) scale[j] = rows[16 * tile[j]];
#pragma unroll
        for (int i = 0; i < 3; ++i) p[i] = pf[fragment_of(tile[(i + 1) / 2], i / 2) * 64];
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int n = 0; n < kTiles; ++n) uw[part][n][ks] = lds.u[part][n][ks][lane];
        __builtin_amdgcn_sched_barrier(0);
        add_qs(1);
        if (chunk + 1 < chunks) read_q(chunk + 1);
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) o[n][j] *= scale[j];
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          const bf8(&x)[kTiles][2] = uw[part == 2];
          const bf8* const y = part == 1 ? pl : p;
#pragma unroll
          for (int n = 0; n < kTiles; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) o[n][j] = mma(x[n][0], y[j], o[n][j]);
#pragma unroll
          for (int n = 0; n < kTiles; ++n) o[n][1] = mma(x[n][1], y[2], o[n][1]);
        }
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
          const uint64_t* const bad = lds.bad[n];
          if (!__any(bad[c16] != 0)) continue;
          int token0 = c16;
          asm volatile("" : "+v"(token0));           // else what follows is made before the loop, and kept
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int in = 16 * tile[j] + token0;
            const uint64_t path = chunk * kChunk + in < r.n ? ancestors(s, r.start, in) | (uint64_t)1 << in : 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (path & bad[4 * g4 + i]) o[n][j][i] = NAN;
          }
        }
      };
      auto put = [&](int chunk) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int token = chunk * kChunk + 16 * tile[j] + c16;
          const int row = token < r.n ? (ROWS ? row_of(s, r.start + token) : r.start + token) : -1;
          if (row >= 0) {
            uint16_t* const to = a.out + row * a.ldo + h * a.dv + col0 + 8 * g4;
#pragma unroll
            for (int n = 0; n < kTiles; n += 2)
              *reinterpret_cast<bf8*>(to + 16 * n) = high(o[n][j], o[n + 1][j]);
          }
        }
      };
      for (int c = 0; c < chunks; ++c) {
        if (c > 0 && a.q) add_pu(c - 1);
        lds_barrier();                               // S is there, U has been read
        if (a.q) {
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
              for (int n = 0; n < kTiles; ++n) sw[part][n][ks] = lds.s[part][n][ks][lane];
          __builtin_amdgcn_sched_barrier(0);
          if (c > 0) {
            read_p(c);
            put(c - 1);
          }
#pragma unroll
          for (int n = 0; n < kTiles; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) o[n][j] = f32x4v{0, 0, 0, 0};
          add_qs(0);
        }
        lds_barrier();
      }
      if (chunks && a.q) {
        add_pu(chunks - 1);
        put(chunks - 1);
      }
    }
    return;
  }

  for (; there; there = next()) {
    const int chunks = (r.n + kChunk - 1) / kChunk;
    // ---- 16 columns of S through the chunks: what the kernel's time is made of.  Of every 8 columns, two waves have 4 each: so the outputs
    // have 8 neighbours in a lane.
    const int src = slot_of(s, s.src, b), dst = slot_of(s, s.dst, b);
    const int64_t state_at = ((int64_t)h * a.dv + col0 + (w >> 1) * 32 + (c16 >> 2) * 8 + (w & 1) * 4 + (c16 & 3)) * DK + 8 * g4;
    f32x4v st[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) st[i] = f32x4v{0, 0, 0, 0};
    if (src >= 0) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const f32x4v* p = reinterpret_cast<const f32x4v*>(a.state + src * a.slot_stride + state_at + 32 * ks);
        st[2 * ks] = p[0];
        st[2 * ks + 1] = p[1];
      }
    }
    bf8 k[KS][4];
    // A lane's places in the first buffer of K, of the operands of K S and of those of K turned (pieces 4 ks further lie where these bits
    // differ).  The compiler is not to know that they stay the same: it would keep every address made from them.
    uint32_t kplace = lds_off(lds.k[0]) + piece_at<DK>(c16, g4);
    uint32_t tplace = lds_off(lds.k[0]) + piece_at<DK>(4 * g4 + (c16 >> 2), c16 & 3);
    auto read_k = [&](int buf) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
          k[ks][rt] = __builtin_bit_cast(bf8, lds_at((kplace ^ (ks * 64)) + buf * (kChunk * DK * 2) + rt * 16 * DK * 2));
    };
    barrier();
    __builtin_amdgcn_s_setprio(2);
    if (chunks) read_k(0);
    int k0 = 0, k1 = 1;                            // the buffers of this chunk's K, and the next one's
    for (int c = 0; c < chunks; ++c) {
      asm volatile("" : "+v"(kplace), "+v"(tplace));
      const auto& here = lds.chunk[c & 1];
      const float* const rows = reinterpret_cast<const float*>(here.first + 2 * kFragments * 1024) + 4 * g4;
      const bf8* const tf = reinterpret_cast<const bf8*>(here.first) + lane;
      // K S, and beside it the rest of S's split, its decay, and what the next step reads from LDS
      const float grown = rows[kGrown - 4 * g4];
      uint64_t bad_col = reinterpret_cast<const uint64_t*>(here.first + 2 * kFragments * 1024)[kBad / 2];
      __builtin_amdgcn_sched_barrier(0);
      f32x4v taken[4];
      i16x4 v[4];
      bf8 t[2 * kFragments], sh[KS], sl[KS];
      // V turned: a lane's column of 4 neighbouring tokens
      const uint32_t vat = lds_off(here.v) + (4 * g4 + (c16 >> 2)) * (kScanColumns * 2) + (w >> 1) * 64 + (c16 & 3) * 16 + (w & 1) * 8;
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) {
        taken[rt] = *reinterpret_cast<const f32x4v*>(rows + kTaken + 16 * rt);
        v[rt] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_i16x4*>(vat + rt * 16 * kScanColumns * 2));
      }
      f32x4v x[4];
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) x[rt] = f32x4v{0, 0, 0, 0};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        sh[ks] = high(st[2 * ks], st[2 * ks + 1]);
        sl[ks] = low(st[2 * ks], st[2 * ks + 1], sh[ks]);
        lds.s[0][w][ks][lane] = sh[ks];
        lds.s[1][w][ks][lane] = sl[ks];
        st[2 * ks] *= grown;
        st[2 * ks + 1] *= grown;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) x[rt] = mma(k[ks][rt], sh[ks], x[rt]);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) x[rt] = mma(k[ks][rt], sl[ks], x[rt]);
        if (ks == KS / 2 - 1) {
          __builtin_amdgcn_sched_group_barrier(0x002, 24, 0);
          beside_matrix<4 * KS, 4, 1>();
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int i = 0; i < 2 * kFragments; ++i) t[i] = tf[i * 64];
        }
      }
      beside_matrix<4 * KS, 4, 1>();
      __builtin_amdgcn_sched_barrier(0);
      // R = V - e^G K S / |k|, U = T R, and beside them K turned: of tokens 32 ks + 4 g .. + 3 (and 16 further) the values that the rows
      // of S's tile i are
      bf8 kt[RT];
      auto read_turned = [&](int ks) {
#pragma unroll
        for (int i = 0; i < RT; ++i)
          kt[i] = turned((tplace ^ ((i >> 1) * 64)) + k0 * (kChunk * DK * 2) + ks * 32 * DK * 2 + (i & 1) * 8, 16 * DK * 2);
      };
      f32x4v left[4], u[4];
      bf8 uh, ul, first_high, first_low;             // scaled for S; of the first half as it is, for the outputs
      auto finish = [&](int ks) {
        u[2 * ks] *= left[2 * ks];
        u[2 * ks + 1] *= left[2 * ks + 1];
        uh = high(u[2 * ks], u[2 * ks + 1]);
        ul = low(u[2 * ks], u[2 * ks + 1], uh);
      };
      auto solve = [&] {
        bf8 rh[2], rl[2];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) u[rt] = f32x4v{0, 0, 0, 0};
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          rh[ks] = high(x[2 * ks], x[2 * ks + 1]);
          rl[ks] = low(x[2 * ks], x[2 * ks + 1], rh[ks]);
        }
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
          for (int part = 0; part < 3; ++part)
#pragma unroll
            for (int rt = 2 * ks; rt < 4; ++rt)
              u[rt] = mma(t[fragment_of(rt, ks) + (part == 2 ? kFragments : 0)], part == 1 ? rl[ks] : rh[ks], u[rt]);
        first_high = high(u[0], u[1]);
        first_low = low(u[0], u[1], first_high);
        finish(0);
      };
#pragma unroll
      for (int rt = 0; rt < 4; ++rt)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[rt][i] = __builtin_fmaf(-taken[rt][i], x[rt][i], bf16_float((uint16_t)v[rt][i]));
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) left[rt] = *reinterpret_cast<const f32x4v*>(rows + kLeft + 16 * rt);
      read_turned(0);
      solve();
      __builtin_amdgcn_sched_group_barrier(0x002, 40, 0);
      beside_matrix<12, 3, 2>();
      beside_matrix<6, 6, 0>();
      __builtin_amdgcn_sched_barrier(0);
      lds_barrier();                                 // the outputs have read the U before
      // Every row of the last tile takes every value of R, if only 0 times: one that is no number shows there.  It is taken out then, as
      // it would reach tokens that do not follow its own, and remembered.
      if (__any(!finite(u[3][0]))) {
        uint64_t mine = 0;
        int row0 = 4 * g4;
        asm volatile("" : "+v"(row0));               // else the bits of all rows are made before the loop, and kept
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!(fabsf(x[rt][i]) < 0x1.FFp127f)) {      // beyond BF16 is infinite too
              mine |= (uint64_t)1 << (16 * rt + row0 + i);
              x[rt][i] = 0.0f;
            }
        mine |= __shfl_xor(mine, 16);
        mine |= __shfl_xor(mine, 32);
        bad_col |= mine;
        solve();
      }
      auto put_u = [&] {
        const bf8 hi = high(u[2], u[3]);
        if (g4 == 0) lds.bad[w][c16] = bad_col;
        lds.u[0][w][0][lane] = first_high;
        lds.u[1][w][0][lane] = first_low;
        lds.u[0][w][1][lane] = hi;
        lds.u[1][w][1][lane] = low(u[2], u[3], hi);
      };
      if (dst < 0 && c + 1 == chunks) {              // nobody asks for what S has become
        put_u();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int rt = 0; rt < 4; ++rt) asm volatile("" : "=v"(k[ks][rt]));      // not needed again: else one is kept, in memory
        lds_barrier();
        break;
      }
      // S, half of the tokens at a time: the other half's split runs beside, and the reads of the next chunk's K
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < RT; ++i) st[i] = mma(kt[i], uh, st[i]);
#pragma unroll
      for (int i = 0; i < RT; ++i) st[i] = mma(kt[i], ul, st[i]);
      put_u();
      finish(1);
      read_turned(1);
      beside_matrix<2 * RT, 4, 2>();
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < RT; ++i) st[i] = mma(kt[i], uh, st[i]);
#pragma unroll
      for (int i = 0; i < RT; ++i) st[i] = mma(kt[i], ul, st[i]);
      read_k(k1);
      beside_matrix<2 * RT, 0, 1>();
      __builtin_amdgcn_sched_barrier(0);
      if (__any(bad_col != 0)) {
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) st[i][e] = bad_col ? NAN : st[i][e];
      }
      k0 = k1;
      k1 = k1 == 2 ? 0 : k1 + 1;
      lds_barrier();
    }
    if (dst >= 0) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        f32x4v* p = reinterpret_cast<f32x4v*>(a.state + dst * a.slot_stride + state_at + 32 * ks);
        p[0] = st[2 * ks];
        p[1] = st[2 * ks + 1];
      }
    }
  }
}

uint64_t delta_chunk_workspace_bytes(int32_t T, int32_t count, int32_t v_heads) {
  return kZeroBytes + (uint64_t)most_pieces(T, count, kChunk) * v_heads * kTermsBytes;
}

template <int DK>
static hipError_t chunk_launches(const w12_delta_args& a, const w12_sequences& s, char* ws, hipStream_t stream) {
  const int64_t pieces = most_pieces(s.T, s.count, kChunk), shorts = s.tree_mask ? 0 : (int64_t)s.count * (a.dv / kGroupColumns);
  k_delta_terms<DK><<<dim3((unsigned)(pieces + shorts), (unsigned)a.v_heads), kChunkThreads, 0, stream>>>(a, s, ws, (int)pieces);
  // A work-group for every long sequence there can be; where most are short, one round of the chip, which takes them in turn: a
  // work-group that finds none keeps a compute unit, for its LDS, as long as it takes to look.
  const int64_t of = a.v_heads * (a.dv / kScanColumns);
  const bool many = !s.tree_mask && s.T < (int64_t)W12_DELTA_CHUNK_FROM * s.count;
  const int64_t sequences = many ? std::min((int64_t)s.T / W12_DELTA_CHUNK_FROM, ceil_div(device_cus(), of)) : s.count;
  const unsigned scans = (unsigned)(sequences * of);
  if (many) s.rows ? k_delta_scan<DK, true, true><<<scans, kScanThreads, 0, stream>>>(a, s, ws)
                   : k_delta_scan<DK, false, true><<<scans, kScanThreads, 0, stream>>>(a, s, ws);
  else s.rows ? k_delta_scan<DK, true, false><<<scans, kScanThreads, 0, stream>>>(a, s, ws)
              : k_delta_scan<DK, false, false><<<scans, kScanThreads, 0, stream>>>(a, s, ws);
  return hipGetLastError();
}

hipError_t launch_delta_chunks(const w12_delta_args& a, const w12_sequences& s, void* ws, hipStream_t stream) {
  return a.dk == 64 ? chunk_launches<64>(a, s, static_cast<char*>(ws), stream) : chunk_launches<128>(a, s, static_cast<char*>(ws), stream);
}

}  // namespace w12
