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
// same every time).  Operands go global -> registers (DEPTH steps ahead) -> LDS (double-buffered): W as it is,
// X widened to BF16 once for all waves; 16-byte pieces are swizzled by row so that the operand
// reads, 32 rows of one piece, meet every bank equally.
#include "w12_device.h"
#include "w12_gemm_common.h"
#include "w12_kernels.h"
#include "w12_rows.h"

namespace w12 {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4e __attribute__((ext_vector_type(4)));

constexpr int kStepK = 128;
constexpr uint32_t kPastEnd = 0xFFFFFFF0u;   // a buffer offset past any operand: reads give 0

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
  uint32_t ldx, ldw, x_bytes, w_bytes;
  int64_t ldxs, ldws, ldy;
  int M, N, K, steps, m_tiles;
  int64_t total, share;    // steps of all tiles, and of a share
  uint32_t part_bytes;
};

// WN x WM waves of NB x MB blocks of 32 channels x 32 rows.
template <int WN, int WM, int NB, int MB, int DEPTH, int PER_CU>
struct E4m3Cfg {
  static constexpr int kWaves = WN * WM, kThreads = kWaves * 64;
  static constexpr int kBN = WN * NB * 32, kBM = WM * MB * 32;
  static constexpr int kWPieces = kBN * 8 / kThreads, kXPieces = kBM * 8 / kThreads;   // loads of a thread a step
  static constexpr int kPart = kBN * kBM;                                              // floats of a partial tile
  static constexpr int kDepth = DEPTH, kPerCu = PER_CU;
  static_assert(kWPieces >= 1 && kXPieces >= 1, "every thread loads");
  static constexpr int kWavesPerSimd = kWaves * PER_CU / 4;
};

template <typename C, int WN, int WM, int NB, int MB>
__global__ __launch_bounds__(C::kThreads, C::kWavesPerSimd) void k_gemm_e4m3(E4m3Args g) {
  __shared__ uint4 lw[2][C::kBN * 8];
  __shared__ uint4 lx[2][C::kBM * 16];
  __shared__ uint32_t s_last;
  const int t = threadIdx.x, lane = t & 63, wave = wave_id(), col = lane & 31, hi = lane >> 5;
  const int wn = wave % WN, wm = wave / WN;
  const int piece = t & 7, prow = t >> 3;
  constexpr int kRowsStep = C::kThreads / 8;
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(g.W, g.w_bytes), rx = make_rsrc(g.X, g.x_bytes);
  const __amdgpu_buffer_rsrc_t rp = make_rsrc(g.parts, g.part_bytes);
  const int64_t me = logical_wg(blockIdx.x, gridDim.x);
  const int64_t r0 = me * g.share, r1 = min(r0 + g.share, g.total);
  int64_t at = r0;
  while (at < r1) {
    const int64_t tile = at / g.steps, c0 = tile * g.steps;
    const int first = (int)(at - c0), last = (int)min(r1 - c0, (int64_t)g.steps);
    at = c0 + last;
    const int n0 = (int)(tile / g.m_tiles) * C::kBN, m0 = (int)(tile % g.m_tiles) * C::kBM;

    uint32_t woff[C::kWPieces], xoff[C::kXPieces];
#pragma unroll
    for (int i = 0; i < C::kWPieces; ++i) {
      const int n = n0 + prow + i * kRowsStep;
      woff[i] = n < g.N ? (uint32_t)n * g.ldw : kPastEnd;
    }
#pragma unroll
    for (int i = 0; i < C::kXPieces; ++i) {
      const int m = m0 + prow + i * kRowsStep;
      xoff[i] = m < g.M ? (uint32_t)m * g.ldx : kPastEnd;
    }
    uint4 wreg[C::kDepth][C::kWPieces], xreg[C::kDepth][C::kXPieces];
    auto fetch = [&](int step, uint4* w, uint4* x) {
      const int k = step * kStepK + piece * 16;
      const bool in = step < last && k < g.K;
#pragma unroll
      for (int i = 0; i < C::kWPieces; ++i) w[i] = bload16(rw, in && woff[i] != kPastEnd ? woff[i] + (uint32_t)k : kPastEnd);
#pragma unroll
      for (int i = 0; i < C::kXPieces; ++i) x[i] = bload16(rx, in && xoff[i] != kPastEnd ? xoff[i] + (uint32_t)k : kPastEnd);
    };
    auto put = [&](int step, int buf, uint4* w, uint4* x) {
      const int left = g.K - step * kStepK - piece * 16;      // bytes of this piece that belong to the row
      if ((step + 1) * kStepK > g.K) {
#pragma unroll
        for (int i = 0; i < C::kWPieces; ++i) w[i] = first_bytes(w[i], left);
#pragma unroll
        for (int i = 0; i < C::kXPieces; ++i) x[i] = first_bytes(x[i], left);
      }
#pragma unroll
      for (int i = 0; i < C::kWPieces; ++i) {
        const int r = prow + i * kRowsStep;
        lw[buf][r * 8 + (piece ^ (r & 7))] = w[i];
      }
#pragma unroll
      for (int i = 0; i < C::kXPieces; ++i) {
        const int r = prow + i * kRowsStep;
        lx[buf][r * 16 + ((2 * piece) ^ (r & 15))] = widen8(x[i].x, x[i].y);
        lx[buf][r * 16 + ((2 * piece + 1) ^ (r & 15))] = widen8(x[i].z, x[i].w);
      }
    };

    f32x16 acc[NB][MB];
#pragma unroll
    for (int a = 0; a < NB; ++a)
#pragma unroll
      for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.0f;
    const bool wave_on = m0 + wm * MB * 32 < g.M && n0 + wn * NB * 32 < g.N;
    const int nblk = (n0 + wn * NB * 32) / W12_QUANT_BLOCK;
    const float* xrow[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) xrow[b] = g.xs + (int64_t)min(m0 + (wm * MB + b) * 32 + col, g.M - 1) * g.ldxs;
    const float* wrow = g.wsc + nblk * g.ldws;

    auto compute = [&](int step, int buf) {
      float sc[MB];
      const float ws = wrow[step];
#pragma unroll
      for (int b = 0; b < MB; ++b) sc[b] = xrow[b][step] * ws;
      f32x16 part[NB][MB];
#pragma unroll
      for (int a = 0; a < NB; ++a)
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) part[a][b][i] = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // this lane's k: 16 from 16 (2 j + hi), in two instructions of 8
        uint4 w[NB];
#pragma unroll
        for (int a = 0; a < NB; ++a) {
          const int r = (wn * NB + a) * 32 + col;
          w[a] = lw[buf][r * 8 + ((2 * j + hi) ^ (r & 7))];
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint4 x[MB];
#pragma unroll
          for (int b = 0; b < MB; ++b) {
            const int r = (wm * MB + b) * 32 + col;
            x[b] = lx[buf][r * 16 + ((2 * (2 * j + hi) + e) ^ (r & 15))];
          }
#pragma unroll
          for (int a = 0; a < NB; ++a) {
            const bf16x8 wb = __builtin_bit_cast(bf16x8, e ? widen8(w[a].z, w[a].w) : widen8(w[a].x, w[a].y));
#pragma unroll
            for (int b = 0; b < MB; ++b)
              part[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wb, __builtin_bit_cast(bf16x8, x[b]), part[a][b], 0, 0, 0);
          }
        }
      }
#pragma unroll
      for (int a = 0; a < NB; ++a)
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[a][b][i] += part[a][b][i] * sc[b];
    };

    constexpr int DEPTH = C::kDepth;
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) fetch(first + d, wreg[d], xreg[d]);
    put(first, 0, wreg[0], xreg[0]);
    fetch(first + DEPTH, wreg[0], xreg[0]);
    __syncthreads();
    // step s is computed from buffer (s - first) % 2 while step s + 1 goes from its registers into the other
    for (int s0 = first; s0 < last; s0 += 2 * DEPTH) {
#pragma unroll
      for (int d = 0; d < 2 * DEPTH; ++d) {
        const int step = s0 + d;
        if (step < last) {
          if (wave_on) compute(step, d & 1);
          if (step + 1 < last) {
            put(step + 1, (d + 1) & 1, wreg[(d + 1) % DEPTH], xreg[(d + 1) % DEPTH]);
            fetch(step + 1 + DEPTH, wreg[(d + 1) % DEPTH], xreg[(d + 1) % DEPTH]);
          }
          __syncthreads();
        }
      }
    }

    const bool whole = first == 0 && last == g.steps;
    bool store = whole;
    if (!whole) {
      // partial tile [float4][lane] of each wave; device-coherent (sc1), as its reader may be on another XCD
      const uint32_t wbase = (uint32_t)wave * NB * MB * 4 * 64 * 16 + (uint32_t)lane * 16;
      if (wave_on) {
        const uint32_t base = (uint32_t)((2 * me + (c0 > r0)) * (C::kPart * 4)) + wbase;
#pragma unroll
        for (int a = 0; a < NB; ++a)
#pragma unroll
          for (int b = 0; b < MB; ++b)
            if (m0 + (wm * MB + b) * 32 + col < g.M) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const u32x4e v = {__float_as_uint(acc[a][b][4 * q]), __float_as_uint(acc[a][b][4 * q + 1]),
                                  __float_as_uint(acc[a][b][4 * q + 2]), __float_as_uint(acc[a][b][4 * q + 3])};
                __builtin_amdgcn_raw_buffer_store_b128(v, rp, (int)(base + (uint32_t)((a * MB + b) * 4 + q) * 1024u), 0,
                                                       kCachePolicySc1);
              }
            }
      }
      wait_vm_all();      // the stores of this wave are complete
      __syncthreads();
      const int64_t g0 = c0 / g.share, g1 = (c0 + g.steps - 1) / g.share;
      if (t == 0) {
        const uint32_t prev = __hip_atomic_fetch_add(g.counters + g0, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_last = prev == (uint32_t)(g1 - g0);
        if (s_last) __hip_atomic_store(g.counters + g0, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      __syncthreads();
      store = s_last != 0;
      __syncthreads();    // s_last may be written again
      if (store && wave_on) {
#pragma unroll
        for (int a = 0; a < NB; ++a)
#pragma unroll
          for (int b = 0; b < MB; ++b) {
            if (m0 + (wm * MB + b) * 32 + col >= g.M) continue;
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.0f;
            for (int64_t p = g0; p <= g1; ++p) {
              const uint32_t base = (uint32_t)((2 * p + (c0 > p * g.share)) * (C::kPart * 4)) + wbase;
              f32x4 v[4];
#pragma unroll
              for (int q = 0; q < 4; ++q)
                v[q] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                     rp, (int)(base + (uint32_t)((a * MB + b) * 4 + q) * 1024u), 0, kCachePolicySc1));
#pragma unroll
              for (int i = 0; i < 16; ++i) acc[a][b][i] += v[i >> 2][i & 3];
            }
          }
      }
    }
    if (store && wave_on) {
      const bool vec = (g.ldy & 3) == 0 && (reinterpret_cast<uintptr_t>(g.Y) & 15) == 0;
#pragma unroll
      for (int a = 0; a < NB; ++a)
#pragma unroll
        for (int b = 0; b < MB; ++b) {
          const int m = m0 + (wm * MB + b) * 32 + col;
          if (m >= g.M) continue;
          float* y = g.Y + m * g.ldy;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int n = n0 + (wn * NB + a) * 32 + 8 * q + 4 * hi;
            if (vec && n + 4 <= g.N) {
              *reinterpret_cast<float4*>(y + n) =
                  make_float4(acc[a][b][4 * q], acc[a][b][4 * q + 1], acc[a][b][4 * q + 2], acc[a][b][4 * q + 3]);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (n + i < g.N) y[n + i] = acc[a][b][4 * q + i];
            }
          }
        }
    }
  }
}

struct E4m3Plan {
  int path;        // rows of X a tile: 32, 64 or 128
  int64_t tiles, m_tiles, steps, total, share, groups;
  uint64_t part_bytes;
};

using E4m3Rows32 = E4m3Cfg<4, 1, 1, 1, 3, 3>;
using E4m3Rows64 = E4m3Cfg<4, 1, 1, 2, 2, 2>;
using E4m3Rows128 = E4m3Cfg<4, 2, 2, 2, 1, 1>;

template <typename C>
static void plan_with(E4m3Plan& p, int M, int N) {
  p.m_tiles = ceil_div(M, C::kBM);
  p.tiles = ceil_div(N, C::kBN) * p.m_tiles;
  p.total = p.tiles * p.steps;
  const int64_t slots = (int64_t)device_cus() * C::kPerCu;
  p.share = ceil_div(p.total, slots);
  if (p.share < 4) p.share = 4 < p.steps ? 4 : p.steps;
  if (C::kBM < 128 && 2 * p.share > p.steps) p.share = ceil_div(p.share, p.steps) * p.steps;
  p.groups = ceil_div(p.total, p.share);
  p.part_bytes = p.share % p.steps ? (uint64_t)(2 * p.groups) * C::kPart * 4 : 0;
}

static E4m3Plan plan_e4m3(int M, int N, int K) {
  E4m3Plan p;
  p.steps = ceil_div(K, kStepK);
  p.path = M <= 32 ? 32 : M <= 64 ? 64 : 128;
  if (p.path == 32) plan_with<E4m3Rows32>(p, M, N);
  else if (p.path == 64) plan_with<E4m3Rows64>(p, M, N);
  else plan_with<E4m3Rows128>(p, M, N);
  return p;
}

uint64_t gemm_e4m3_workspace_bytes(int32_t M, int32_t N, int32_t K) {
  const E4m3Plan p = plan_e4m3(M, N, K);
  return p.part_bytes ? kCounterBytes + p.part_bytes : 0;
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
  g.ldxs = ldxs;
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
  if (p.path == 32) hipLaunchKernelGGL((k_gemm_e4m3<E4m3Rows32, 4, 1, 1, 1>), grid, dim3(E4m3Rows32::kThreads), 0, stream, g);
  else if (p.path == 64) hipLaunchKernelGGL((k_gemm_e4m3<E4m3Rows64, 4, 1, 1, 2>), grid, dim3(E4m3Rows64::kThreads), 0, stream, g);
  else hipLaunchKernelGGL((k_gemm_e4m3<E4m3Rows128, 4, 2, 2, 2>), grid, dim3(E4m3Rows128::kThreads), 0, stream, g);
  return hipGetLastError();
}

}  // namespace w12
