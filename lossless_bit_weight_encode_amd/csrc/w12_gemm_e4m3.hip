// The 8-bit product with block scales: Y = (X sx) (W sw)^T, E4M3 operands, FP32 sums.
//
// The operands become BF16 (which holds every E4M3 value) on their way to the matrix instructions:
// the 8-bit ones line up the products of eight neighbouring k with the largest and drop what is below
// 2^-13 of it (measured), so they do not hold a sum in 32 bits; the BF16 ones do.  A step is one block
// of 128 k: its sum, from zero, is multiplied by the two scales and added in FP32.
//
// A work-group takes tiles of BN channels x BM rows of X; their steps, end to end, are cut into equal
// shares, one a work-group (so few tiles of a long k fill the chip).  The work-groups of a tile leave
// FP32 partial tiles, and the last one to arrive adds them in the order of the work-groups (bitwise the
// same every time).  Operands are loaded into registers DEPTH steps ahead.  They pass
// through LDS (double-buffered; W as it is, X widened to BF16 once for all waves), their pieces
// swizzled by row so that the operand reads, 32 rows of one piece, meet every bank equally; the next step's
// pieces are put there beside the matrix instructions.  For a few rows over a short W they load
// straight into operand registers: a wave's W is nobody else's, and no wave waits for another.
//
// Bound: few rows by the read of W (63 rows of 34816 x 5120, 178 MB: 57 us, 3.3 TB/s; a copy of the kernel that only reads
// W in this order took 38), many by the matrix instructions and what feeds them (512 rows: 216 to 226 us, 805 to 845
// TFLOP/s; a copy with the instructions alone took 120).
#include "w12_device.h"
#include "w12_gemm_common.h"
#include "w12_kernels.h"
#include "w12_rows.h"

namespace w12 {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4e __attribute__((ext_vector_type(4)));

constexpr int kStepK = 128;
constexpr int kScaleSteps = 32;

// Eight E4M3 bytes to BF16.
__device__ __forceinline__ uint4 widen8(uint32_t lo, uint32_t hi) {
  return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true)));
}

// The first n bytes of a piece, zeros after them (n may be past its ends).
__device__ __forceinline__ uint4 first_bytes(uint4 u, int n) {
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int left = n - 4 * i;
    w[i] = left >= 4 ? w[i] : left <= 0 ? 0 : w[i] & ((1u << (8 * left)) - 1);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

struct E4m3Args {
  const uint8_t *X, *W;
  const float *xs, *wsc;
  float* Y;
  uint32_t* counters;
  float* parts;
  uint32_t ldx, ldw, ldxs, x_bytes, w_bytes, xs_bytes;
  int64_t ldws, ldy;
  int M, N, K, steps, m_tiles;
  int64_t total, share;    // steps of all tiles, and of a share
  uint32_t part_bytes;
};

// WN x WM waves of NB x MB blocks of 32 channels x 32 rows; LDS: operands through LDS.
template <int WN_, int WM_, int NB_, int MB_, int DEPTH, int PER_CU, bool LDS>
struct E4m3Cfg {
  static constexpr int WN = WN_, WM = WM_, NB = NB_, MB = MB_, kDepth = DEPTH, kPerCu = PER_CU;
  static constexpr bool kLds = LDS;
  static constexpr int kWaves = WN * WM, kThreads = kWaves * 64;
  static constexpr int kBN = WN * NB * 32, kBM = WM * MB * 32;
  static constexpr int kWPieces = LDS ? kBN * 8 / kThreads : NB * 4;     // loads of a thread a step
  static constexpr int kXPieces = LDS ? kBM * 8 / kThreads : MB * 4;
  static constexpr int kPart = kBN * kBM;                                // floats of a partial tile
  static constexpr int kWavesPerSimd = kWaves * PER_CU / 4;
  static_assert(kWPieces >= 1 && kXPieces >= 1 && (LDS || DEPTH >= 2), "every thread loads; a slot is free before it is filled");
};

template <typename C>
__global__ __launch_bounds__(C::kThreads, C::kWavesPerSimd) void k_gemm_e4m3(E4m3Args g) {
  constexpr int NB = C::NB, MB = C::MB, DEPTH = C::kDepth;
  __shared__ uint4 lw[C::kLds ? 2 : 1][C::kLds ? C::kBN * 8 : 1];
  __shared__ uint4 lx[C::kLds ? 2 : 1][C::kLds ? C::kBM * 16 : 1];
  // scales of the next kScaleSteps steps, [step][row], and of the tile's blocks of 128 channels
  __shared__ float lxs[C::kLds ? kScaleSteps : 1][C::kLds ? C::kBM + 1 : 1];
  __shared__ float lws[C::kLds ? kScaleSteps : 1][C::kLds ? C::kBN / W12_QUANT_BLOCK : 1];
  __shared__ uint32_t s_last;
  const int t = threadIdx.x, lane = t & 63, wave = wave_id(), col = lane & 31, hi = lane >> 5;
  const int wn = wave % C::WN, wm = wave / C::WN;
  const int piece = t & 7, prow = t >> 3;      // this thread's part of the operands on their way to LDS
  constexpr int kRowsStep = C::kThreads / 8;
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(g.W, g.w_bytes), rx = make_rsrc(g.X, g.x_bytes);
  const __amdgpu_buffer_rsrc_t rp = make_rsrc(g.parts, g.part_bytes), rs = make_rsrc(g.xs, g.xs_bytes);
  // where this lane's operands are in LDS: its row, the piece that the swizzle gives k = 0
  const uint32_t wbase = (uint32_t)((wn * NB * 32 + col) * 128 + ((hi ^ (col >> 1 & 7)) * 16));
  const uint32_t xbase = (uint32_t)((wm * MB * 32 + col) * 256 + (((2 * hi) ^ (col & 15)) * 16));
  const int64_t me = logical_wg(blockIdx.x, gridDim.x);
  const int64_t r0 = me * g.share, r1 = min(r0 + g.share, g.total);
  int64_t at = r0;
  while (at < r1) {
    const int64_t tile = at / g.steps, c0 = tile * g.steps;
    const int first = (int)(at - c0), last = (int)min(r1 - c0, (int64_t)g.steps);
    at = c0 + last;
    const int n0 = (int)(tile / g.m_tiles) * C::kBN, m0 = (int)(tile % g.m_tiles) * C::kBM;

    // Byte offsets of this thread's pieces (rows past the end take the last row, whose results are not
    // stored), and of the scales of this lane's rows of X.
    uint32_t woff[C::kLds ? C::kWPieces : NB], xoff[C::kLds ? C::kXPieces : MB], xsoff[MB];
    if constexpr (C::kLds) {
#pragma unroll
      for (int i = 0; i < C::kWPieces; ++i) woff[i] = (uint32_t)min(n0 + prow + i * kRowsStep, g.N - 1) * g.ldw + piece * 16;
#pragma unroll
      for (int i = 0; i < C::kXPieces; ++i) xoff[i] = (uint32_t)min(m0 + prow + i * kRowsStep, g.M - 1) * g.ldx + piece * 16;
    } else {
#pragma unroll
      for (int a = 0; a < NB; ++a) woff[a] = (uint32_t)min(n0 + (wn * NB + a) * 32 + col, g.N - 1) * g.ldw + hi * 16;
#pragma unroll
      for (int b = 0; b < MB; ++b) xoff[b] = (uint32_t)min(m0 + (wm * MB + b) * 32 + col, g.M - 1) * g.ldx + hi * 16;
    }
#pragma unroll
    for (int b = 0; b < MB; ++b) xsoff[b] = (uint32_t)min(m0 + (wm * MB + b) * 32 + col, g.M - 1) * g.ldxs;
    const bool wave_on = m0 + wm * MB * 32 < g.M && n0 + wn * NB * 32 < g.N;
    const float* wrow = g.wsc + (int64_t)(min(n0 + wn * NB * 32, g.N - 1) / W12_QUANT_BLOCK) * g.ldws;

    // Operands on their way.  Straight to operand registers, piece j of a lane is k = 16 (2 j + hi) .. + 15 of
    // the step.  Pieces past the end of a row (in the last step) hold what follows it; they are cleared before use.
    uint4 wreg[DEPTH][C::kWPieces], xreg[DEPTH][C::kXPieces];
    float sreg[DEPTH][MB + 1];
    const bool tail = last * kStepK > g.K;
    const int whole = last - tail;
    auto fetch = [&](int step, int d) {
      const uint32_t k = (uint32_t)(step * kStepK);
#pragma unroll
      for (int i = 0; i < C::kWPieces; ++i)
        wreg[d][i] = C::kLds ? bload16(rw, woff[i] + k) : bload16(rw, woff[i / 4] + k + 32 * (i % 4));
#pragma unroll
      for (int i = 0; i < C::kXPieces; ++i)
        xreg[d][i] = C::kLds ? bload16(rx, xoff[i] + k) : bload16(rx, xoff[i / 4] + k + 32 * (i % 4));
    };
    // Scales.  A lane's are those of its rows of X, each in a line of memory of its own: with LDS they are brought there
    // for 32 steps at once (512 rows through 34816 x 5120: 20 us less than step by step); else they travel with the operands.
    auto fetch_scales = [&](int st, int d) {
#pragma unroll
      for (int b = 0; b < MB; ++b)
        sreg[d][b] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, (int)((xsoff[b] + (uint32_t)st) * 4u), 0, 0));
      sreg[d][MB] = wrow[st];
    };
    auto put_scales = [&](int step) {
      for (int i = t; i < C::kBM * kScaleSteps; i += C::kThreads) {
        const int r = i / kScaleSteps, j = i % kScaleSteps;
        const uint32_t at = (uint32_t)min(m0 + r, g.M - 1) * g.ldxs + (uint32_t)min(step + j, g.steps - 1);
        lxs[j][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, (int)(at * 4u), 0, 0));
      }
      for (int i = t; i < kScaleSteps * (C::kBN / W12_QUANT_BLOCK); i += C::kThreads) {
        const int j = i / (C::kBN / W12_QUANT_BLOCK), n = i % (C::kBN / W12_QUANT_BLOCK);
        lws[j][n] = g.wsc[(int64_t)min(n0 / W12_QUANT_BLOCK + n, (g.N - 1) / W12_QUANT_BLOCK) * g.ldws + min(step + j, g.steps - 1)];
      }
      lds_barrier();
    };
    // What does not belong to the row, in the last step of a k that is no multiple of 128: zeros.
    auto clear_tail = [&](int d) {
      const int end = g.K - (g.steps - 1) * kStepK;
#pragma unroll
      for (int i = 0; i < C::kWPieces; ++i)
        wreg[d][i] = first_bytes(wreg[d][i], end - 16 * (C::kLds ? piece : 2 * (i % 4) + hi));
#pragma unroll
      for (int i = 0; i < C::kXPieces; ++i)
        xreg[d][i] = first_bytes(xreg[d][i], end - 16 * (C::kLds ? piece : 2 * (i % 4) + hi));
    };
    // Part i of the kParts in which a step is put into its buffer.
    constexpr int kParts = C::kWPieces + C::kXPieces;
    auto put_part = [&](int i, int buf, int d) {
      if (i < C::kWPieces) {
        const int r = prow + i * kRowsStep;
        lw[buf][r * 8 + (piece ^ (r >> 1 & 7))] = wreg[d][i < C::kWPieces ? i : 0];
      } else {
        const int j = i - C::kWPieces, r = prow + j * kRowsStep;
        const uint4 x = xreg[d][j < 0 ? 0 : j];
        lx[buf][r * 16 + ((2 * piece) ^ (r & 15))] = widen8(x.x, x.y);
        lx[buf][r * 16 + ((2 * piece + 1) ^ (r & 15))] = widen8(x.z, x.w);
      }
    };
    auto put = [&](int buf, int d) {
#pragma unroll
      for (int i = 0; i < kParts; ++i) put_part(i, buf, d);
    };

    f32x16 acc[NB][MB];
#pragma unroll
    for (int a = 0; a < NB; ++a)
#pragma unroll
      for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.0f;

    // `beside(i)` stands behind the matrix instructions of the i-th of 8 parts: what is to run under them has to.  A step
    // past the last whole one counts nothing (its operands are that step's, so 0 times its sum is 0, or NaN where
    // the sum is NaN already).
    auto compute = [&](int buf, int d, int scales, bool counts, auto beside) {
      float sc[MB];
      if constexpr (C::kLds) {
        const float ws = lws[scales][wn * NB * 32 / W12_QUANT_BLOCK];
#pragma unroll
        for (int b = 0; b < MB; ++b) sc[b] = lxs[scales][(wm * MB + b) * 32 + col] * ws;
      } else {
#pragma unroll
        for (int b = 0; b < MB; ++b) sc[b] = sreg[d][b] * sreg[d][MB];
      }
#pragma unroll
      for (int b = 0; b < MB; ++b) sc[b] = counts ? sc[b] : 0.0f;
      f32x16 part[NB][MB];
#pragma unroll
      for (int a = 0; a < NB; ++a)
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) part[a][b][i] = 0.0f;
      // Eight instructions of 16 k a block; instruction 2 j + e takes half e of piece j.  Operands are read from
      // LDS kAhead of them before their use (left to itself the compiler reads them right before it).
      constexpr int kAhead = C::kLds ? (NB * MB >= 4 ? 1 : 2) : 0;
      uint4 w[2][NB], x[kAhead + 1][MB];
      auto operands = [&](int i) {
        const int j = i / 2, e = i % 2;
        if (e == 0) {
#pragma unroll
          for (int a = 0; a < NB; ++a) {
            if constexpr (C::kLds)
              w[j % 2][a] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(lw[buf]) + (wbase ^ (32u * j)) + a * 32 * 128);
            else
              w[j % 2][a] = wreg[d][a * 4 + j];
          }
        }
#pragma unroll
        for (int b = 0; b < MB; ++b) {
          if constexpr (C::kLds)
            x[i % (kAhead + 1)][b] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(lx[buf]) +
                                                                      (xbase ^ (64u * j + 16u * e)) + b * 32 * 256);
          else
            x[0][b] = e ? widen8(xreg[d][b * 4 + j].z, xreg[d][b * 4 + j].w) : widen8(xreg[d][b * 4 + j].x, xreg[d][b * 4 + j].y);
        }
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) operands(i);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i + kAhead < 8) operands(i + kAhead);
        if constexpr (C::kLds) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int a = 0; a < NB; ++a) {
          const uint4 u = w[i / 2 % 2][a];
          const bf16x8 wb = __builtin_bit_cast(bf16x8, i % 2 ? widen8(u.z, u.w) : widen8(u.x, u.y));
#pragma unroll
          for (int b = 0; b < MB; ++b)
            part[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wb, __builtin_bit_cast(bf16x8, x[i % (kAhead + 1)][b]), part[a][b], 0, 0, 0);
        }
        beside(i);
      }
#pragma unroll
      for (int a = 0; a < NB; ++a)
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[a][b][i] += part[a][b][i] * sc[b];
    };

    auto within = [&](int step) { return max(min(step, whole - 1), first); };
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      fetch(within(first + d), d);
      if constexpr (!C::kLds) fetch_scales(within(first + d), d);
    }
    if constexpr (C::kLds) {
      put(0, 0);
      fetch(within(first + DEPTH), 0);
      lds_barrier();
    }
    // Step s goes through the registers of slot (s - first) % DEPTH and, with LDS, buffer (s - first) % 2, into
    // which it is put while step s - 1 is computed.  There is no branch in a turn: where paths meet that a fetch
    // or its use was on one of, the compiler waits for more than is needed.  A step that k ends in is taken by itself below.
    constexpr int kTurn = DEPTH % 2 ? 2 * DEPTH : DEPTH;
    static_assert(kScaleSteps % kTurn == 0, "scales are renewed between turns");
    for (int s0 = first; s0 < whole; s0 += kTurn) {
      if constexpr (C::kLds) {
        if ((s0 - first) % kScaleSteps == 0) put_scales(s0);
      }
#pragma unroll
      for (int i = 0; i < kTurn; ++i) {
        const int d = i % DEPTH, next = (i + 1) % DEPTH, step = s0 + i;
        compute(i & 1, d, (s0 - first) % kScaleSteps + i, step < whole, [&](int part) {
          if constexpr (C::kLds) {
#pragma unroll
            for (int q = part * kParts / 8; q < (part + 1) * kParts / 8; ++q) put_part(q, (i + 1) & 1, next);
          }
        });
        if constexpr (C::kLds) {
          fetch(within(step + 1 + DEPTH), next);
          lds_barrier();
        } else {
          fetch(within(step + DEPTH), d);
          fetch_scales(within(step + DEPTH), d);
        }
      }
    }
    if (tail) {
      fetch(whole, 0);
      if constexpr (!C::kLds) fetch_scales(whole, 0);
      clear_tail(0);
      if constexpr (C::kLds) {
        put(0, 0);
        put_scales(whole);
      }
      compute(0, 0, 0, true, [](int) {});
      if constexpr (C::kLds) lds_barrier();      // the next tile goes to the same buffers
    }

    const int rows = min(g.M - m0, C::kBM), cols = min(g.N - n0, C::kBN);
    const bool vec = (g.ldy & 3) == 0 && (reinterpret_cast<uintptr_t>(g.Y) & 15) == 0;
    auto store_y = [&](int m, int n, const float v[4]) {      // four channels of a row of the tile
      float* y = g.Y + (m0 + m) * g.ldy + n0 + n;
      if (vec && n + 4 <= cols) {
        *reinterpret_cast<float4*>(y) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < cols) y[i] = v[i];
      }
    };
    if (first == 0 && last == g.steps) {
      if (wave_on) {
#pragma unroll
        for (int a = 0; a < NB; ++a)
#pragma unroll
          for (int b = 0; b < MB; ++b) {
            const int m = (wm * MB + b) * 32 + col;
            if (m >= rows) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float v[4] = {acc[a][b][4 * q], acc[a][b][4 * q + 1], acc[a][b][4 * q + 2], acc[a][b][4 * q + 3]};
              store_y(m, (wn * NB + a) * 32 + 8 * q + 4 * hi, v);
            }
          }
      }
      continue;
    }
    // A partial tile, device-coherent (sc1), as its reader may be on another XCD.  Tiles in registers
    // are laid out [row of X][channel], so that every thread adds (one row has few places, and many parts);
    // the others [wave][float4][lane], whole lines a store, and a lane adds what it holds.
    const uint32_t lane_part = (uint32_t)(wave * NB * MB * 4 * 64 + lane) * 16u;
    if (wave_on) {
      const uint32_t base = (uint32_t)((2 * me + (c0 > r0)) * (C::kPart * 4));
#pragma unroll
      for (int a = 0; a < NB; ++a)
#pragma unroll
        for (int b = 0; b < MB; ++b) {
          const int m = (wm * MB + b) * 32 + col;
          if (m >= rows) continue;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const u32x4e v = {__float_as_uint(acc[a][b][4 * q]), __float_as_uint(acc[a][b][4 * q + 1]),
                              __float_as_uint(acc[a][b][4 * q + 2]), __float_as_uint(acc[a][b][4 * q + 3])};
            const uint32_t off = C::kLds ? lane_part + (uint32_t)((a * MB + b) * 4 + q) * 1024u
                                         : (uint32_t)(m * C::kBN + (wn * NB + a) * 32 + 8 * q + 4 * hi) * 4u;
            __builtin_amdgcn_raw_buffer_store_b128(v, rp, (int)(base + off), 0, kCachePolicySc1);
          }
        }
    }
    wait_vm_all();      // the stores of this wave are complete
    __syncthreads();
    const int64_t g0 = c0 / g.share, g1 = (c0 + g.steps - 1) / g.share;
    if (t == 0) {
      // the tile's counter is its first work-group's
      const uint32_t prev = __hip_atomic_fetch_add(g.counters + g0, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      s_last = prev == (uint32_t)(g1 - g0);
      if (s_last) __hip_atomic_store(g.counters + g0, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    const bool mine = s_last != 0;
    __syncthreads();    // s_last may be written again
    if (!mine) continue;
    const int parts = (int)(g1 - g0) + 1;
    const uint32_t base0 = (uint32_t)((2 * g0 + (c0 > g0 * g.share)) * (C::kPart * 4));
    auto load_part = [&](int p, uint32_t off) {      // the tile is the first that the later work-groups hold
      const uint32_t base = p == 0 ? base0 : (uint32_t)(2 * (g0 + p) * (C::kPart * 4));
      return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rp, (int)(base + off), 0, kCachePolicySc1));
    };
    if constexpr (C::kLds) {
      if (!wave_on) continue;
#pragma unroll
      for (int a = 0; a < NB; ++a)
#pragma unroll
        for (int b = 0; b < MB; ++b) {
          const int m = (wm * MB + b) * 32 + col;
          if (m >= rows) continue;
          f32x4 sum[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) sum[q] = load_part(0, lane_part + (uint32_t)((a * MB + b) * 4 + q) * 1024u);
          for (int p = 1; p < parts; ++p) {
            f32x4 v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = load_part(p, lane_part + (uint32_t)((a * MB + b) * 4 + q) * 1024u);
#pragma unroll
            for (int q = 0; q < 4; ++q) sum[q] += v[q];
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float v[4] = {sum[q][0], sum[q][1], sum[q][2], sum[q][3]};
            store_y(m, (wn * NB + a) * 32 + 8 * q + 4 * hi, v);
          }
        }
    } else {
      const int quads = (cols + 3) / 4;
      for (int i = t; i < quads * rows; i += C::kThreads) {
        const int m = i / quads, n = i % quads * 4;
        const uint32_t off = (uint32_t)(m * C::kBN + n) * 4u;
        f32x4 sum = {0, 0, 0, 0};
        for (int p = 0; p < parts; p += 8) {      // eight parts in flight
          f32x4 v[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) v[u] = load_part(min(p + u, parts - 1), off);
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (p + u < parts) sum += v[u];
        }
        const float v[4] = {sum[0], sum[1], sum[2], sum[3]};
        store_y(m, n, v);
      }
    }
  }
}

struct E4m3Plan {
  int path;        // rows of X a tile: 32, 64 or 128
  int64_t tiles, m_tiles, steps, total, share, groups;
  uint64_t part_bytes;
};

// Which tile (us, both sides): up to 64 rows Rows64, 256 channels on 8 waves, where Rows128 pads (Rows64 / Rows128, 34816
// channels of 5120: 16 rows 46 / 55, 64 rows 57 / 63, 96 rows 76 / 70; 5120 of 17408: 64 rows 44 / 56, but 128 rows
// 50 / 70, which the rule does not take).  Up to 4 rows, a W of long rows and up to 128 MB goes straight into registers,
// with three small work-groups a compute unit and partial tiles of the real rows only (Rows32 / Rows64 in a graph:
// 5120 of 17408 with 1 row 32.2 / 36.2, 4 rows 34.7 / 36.0, 8 rows 37.0 / 33.4; 5120 of 5120 with 1 row 15.1 / 17.8; 2048 of
// 8192 10.6 / 17.2; 1024 of 16384 11.8 / 23.2; but 5120 of 34816 55.1 / 50.8, 10240 of 8192 33.9 / 31.1, 7168 of 5120
// 22.3 / 20.4, 34816 of 5120 58 / 44).  Both bounds lie between these shapes and are no more exact than that: 8192 of
// 8192 (29.1 / 25.3) is on the wrong side.  Tiles of 128 channels: with 256 and two work-groups a unit 5120 of 17408
// took 2 us more.
using E4m3Rows32 = E4m3Cfg<4, 1, 1, 1, 2, 3, false>;
using E4m3Rows64 = E4m3Cfg<8, 1, 1, 2, 2, 1, true>;
using E4m3Rows128 = E4m3Cfg<4, 2, 2, 2, 1, 1, true>;

template <typename C>
static void plan_with(E4m3Plan& p, int M, int N) {
  p.m_tiles = ceil_div(M, C::kBM);
  p.tiles = ceil_div(N, C::kBN) * p.m_tiles;
  p.total = p.tiles * p.steps;
  const int64_t slots = (int64_t)device_cus() * C::kPerCu;
  p.share = ceil_div(p.total, slots);
  if (p.share < 4) p.share = 4 < p.steps ? 4 : p.steps;
  p.groups = ceil_div(p.total, p.share);
  p.part_bytes = p.share % p.steps ? (uint64_t)(2 * p.groups) * C::kPart * 4 : 0;
}

static E4m3Plan plan_e4m3(int M, int N, int K) {
  E4m3Plan p{};
  p.steps = ceil_div(K, kStepK);
  p.path = M <= 4 && K >= N && (int64_t)N * K <= (int64_t(1) << 27) ? 32 : M <= 64 ? 64 : 128;
  if (p.path == 32) plan_with<E4m3Rows32>(p, M, N);
  else if (p.path == 64) plan_with<E4m3Rows64>(p, M, N);
  else plan_with<E4m3Rows128>(p, M, N);
  return p;
}

static uint64_t e4m3_call_bytes(const E4m3Plan& p) { return p.part_bytes ? kCounterBytes + p.part_bytes : 0; }

uint64_t gemm_e4m3_call_bytes(int32_t M, int32_t N, int32_t K) { return e4m3_call_bytes(plan_e4m3(M, N, K)); }

// Enough for every number of rows up to M.  Fewer rows may need more (whole tiles for each work-group leave no parts):
// what a call needs goes by its path and its tiles along M, so one M of each is looked at.
uint64_t gemm_e4m3_workspace_bytes(int32_t M, int32_t N, int32_t K) {
  uint64_t most = gemm_e4m3_call_bytes(M, N, K);
  if (M > 4) most = max(most, gemm_e4m3_call_bytes(4, N, K));
  if (M > 64) most = max(most, gemm_e4m3_call_bytes(64, N, K));
  for (int m = E4m3Rows128::kBM; m < M; m += E4m3Rows128::kBM) most = max(most, gemm_e4m3_call_bytes(m, N, K));
  return most;
}

hipError_t launch_gemm_e4m3(const uint8_t* X, int32_t M, int64_t ldx, const float* xs, int64_t ldxs, const uint8_t* W,
                            int32_t N, int32_t K, int64_t ldw, const float* wsc, int64_t ldws, float* Y, int64_t ldy,
                            void* ws, hipStream_t stream) {
  const E4m3Plan p = plan_e4m3(M, N, K);
  E4m3Args g;
  g.X = X;
  g.W = W;
  g.xs = xs;
  g.wsc = wsc;
  g.Y = Y;
  g.counters = static_cast<uint32_t*>(ws);
  g.parts = reinterpret_cast<float*>(static_cast<char*>(ws) + kCounterBytes);
  g.ldx = (uint32_t)ldx;
  g.ldw = (uint32_t)ldw;
  g.x_bytes = (uint32_t)(ceil_div((M - 1) * ldx + K, 16) * 16);
  g.w_bytes = (uint32_t)(ceil_div((N - 1) * ldw + K, 16) * 16);
  g.ldxs = (uint32_t)ldxs;
  g.xs_bytes = (uint32_t)(((M - 1) * ldxs + ceil_div(K, W12_QUANT_BLOCK)) * 4);
  g.ldws = ldws;
  g.ldy = ldy;
  g.M = M;
  g.N = N;
  g.K = K;
  g.steps = (int)p.steps;
  g.m_tiles = (int)p.m_tiles;
  g.total = p.total;
  g.share = p.share;
  g.part_bytes = (uint32_t)p.part_bytes;
  const dim3 grid((unsigned)p.groups);
  if (p.path == 32) hipLaunchKernelGGL(k_gemm_e4m3<E4m3Rows32>, grid, dim3(E4m3Rows32::kThreads), 0, stream, g);
  else if (p.path == 64) hipLaunchKernelGGL(k_gemm_e4m3<E4m3Rows64>, grid, dim3(E4m3Rows64::kThreads), 0, stream, g);
  else hipLaunchKernelGGL(k_gemm_e4m3<E4m3Rows128>, grid, dim3(E4m3Rows128::kThreads), 0, stream, g);
  return hipGetLastError();
}

}  // namespace w12
