// Short causal convolution of every channel over a sequence's rows, or over a tree's paths.
//
//   y_t[c] = act(bias[c] + sum_j weight[c][j] x_{t - (W - 1) + j}[c]),   x before the first row from the state.
//
// A work-group takes a tile of rows of one sequence and 8 neighbouring channels a thread.  In a sequence a thread
// walks down its rows with the window in registers, so that every value is read once but for a tile's first W - 1; in
// a tree each row gathers its window along its path (neighbouring rows share most of it, from the cache).
// The first tile alone reads the state, and writes the new one after it: in place, no other work-group sees either.
#include "w12_gemm_common.h"
#include "w12_kernels.h"
#include "w12_rows.h"
#include "w12_sequences.h"

namespace w12 {

constexpr int kConvThreads = 64;
constexpr int kConvRows = 16;      // rows of a tile

template <bool F32, int W>
__global__ __launch_bounds__(kConvThreads) void k_short_conv(w12_conv_args a, w12_sequences s) {
  constexpr int kPast = W - 1, kBytes = F32 ? 4 : 2;
  __shared__ int found[2];
  int b, tile;
  Range r;
  if (!find_piece(s, blockIdx.x, kConvRows, found, b, r, tile)) return;
  if (tile > 0 && !a.y) return;                      // only the first tile moves a state
  const int c = (blockIdx.y * kConvThreads + threadIdx.x) * 8;
  if (c >= a.channels) return;
  const int src = slot_of(s, s.src, b), dst = slot_of(s, s.dst, b);
  // a token of the past: -1 is the newest
  auto past = [&](int i, float v[8]) {
    if (src < 0 || i < -kPast) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.0f;
    } else {
      load8<F32>(static_cast<const char*>(a.state) + (src * a.slot_stride + (kPast + i) * a.tap_stride) * kBytes, c, a.channels, v);
    }
  };
  auto token = [&](int i, float v[8]) {
    const int row = i < 0 ? -1 : row_of(s, r.start + i);
    if (i < 0) {
      past(i, v);
    } else if (row < 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.0f;
    } else {
      load8<F32>(static_cast<const char*>(a.x) + row * a.ldx * kBytes, c, a.channels, v);
    }
  };
  if (a.y) {
    float w[8][W], bias[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int j = 0; j < W; ++j) w[e][j] = c + e < a.channels ? bf16_float(a.weight[(int64_t)(c + e) * W + j]) : 0.0f;
      bias[e] = a.bias && c + e < a.channels ? bf16_float(a.bias[c + e]) : 0.0f;
    }
    const int t0 = tile * kConvRows, t1 = min(t0 + kConvRows, r.n);
    float x[W][8];
    if (!s.tree_mask)
#pragma unroll
      for (int j = 1; j < W; ++j) token(t0 - W + j, x[j]);
    for (int t = t0; t < t1; ++t) {
      if (s.tree_mask) {
        uint64_t before = ancestors(s, r.start, t);
        int at = t, back = 0;                        // back: how far into the past
#pragma unroll
        for (int j = W - 1; j >= 0; --j) {
          token(at, x[j]);
          if (before) {
            at = 63 - __builtin_clzll(before);
            before &= ~((uint64_t)1 << at);
          } else {
            at = --back;
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) x[j][e] = x[j + 1][e];
        token(t, x[W - 1]);
      }
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] = bias[e];
#pragma unroll
        for (int j = 0; j < W; ++j) y[e] += w[e][j] * x[j][e];
        if (a.silu) y[e] = y[e] / (1.0f + __expf(-y[e]));
      }
      const int row = row_of(s, r.start + t);
      if (row >= 0) store8<false>(a.y + row * a.ldy, c, a.channels, y);
    }
  }
  if (tile == 0 && dst >= 0) {
    float x[kPast][8];
#pragma unroll
    for (int j = 0; j < kPast; ++j) token(r.n - kPast + j, x[j]);
#pragma unroll
    for (int j = 0; j < kPast; ++j)
      store8<F32>(static_cast<char*>(a.state) + (dst * a.slot_stride + j * a.tap_stride) * kBytes, c, a.channels, x[j]);
  }
}

template <bool F32>
static void conv_width(const w12_conv_args& a, const w12_sequences& s, dim3 grid, hipStream_t stream) {
  switch (a.width) {
    case 2: k_short_conv<F32, 2><<<grid, kConvThreads, 0, stream>>>(a, s); break;
    case 3: k_short_conv<F32, 3><<<grid, kConvThreads, 0, stream>>>(a, s); break;
    default: k_short_conv<F32, 4><<<grid, kConvThreads, 0, stream>>>(a, s); break;
  }
}

hipError_t launch_short_conv(const w12_conv_args& a, const w12_sequences& s, hipStream_t stream) {
  const dim3 grid((unsigned)most_pieces(s.T, s.count, kConvRows), (unsigned)ceil_div(a.channels, 8 * kConvThreads));
  if (a.dtype == W12_DTYPE_F32) conv_width<true>(a, s, grid, stream);
  else conv_width<false>(a, s, grid, stream);
  return hipGetLastError();
}

}  // namespace w12
