// Short causal convolution of every channel over a sequence's rows, or over a tree's paths.
//
//   y_t[c] = act(bias[c] + sum_j weight[c][j] x_{t - (W - 1) + j}[c]),   x before the first row from the state.
//
// A work-group takes a tile of rows of one sequence and 8 neighbouring channels a thread.  In a sequence a thread
// walks down its rows with the window in registers, so that every value is read once but for a tile's first W - 1; in
// a tree each row gathers its window along its path (neighbouring rows share most of it, from the cache).
// A sequence's first tile alone reads the state (no tile is shorter than a window's past), and writes the new one after it: in place,
// no other work-group sees either.
//
// Bound by memory where rows are many: 4096 rows of 10240 channels of FP32 take 58 us (252 MB, 4.3 TB/s; the norm's pass over as much reaches
// 5.1), in tiles of 32 rows with 4 rows' loads in flight (tiles of 16: 63).  63 nodes take 5.6 us in tiles of 2 (with the
// call 8.7; in tiles of 16 21): too few bytes to matter, the loads of a window follow the mask's.
#include "w12_gemm_common.h"
#include "w12_kernels.h"
#include "w12_rows.h"
#include "w12_sequences.h"

namespace w12 {

constexpr int kConvThreads = 64;
// Rows of a tile.  Short tiles make work for the chip of few rows, long ones read fewer rows twice.
constexpr int kTreeTile = 2, kShortTile = 4, kLongTile = 32;

// Weights of a thread's 8 channels.
template <int W>
__device__ __forceinline__ void load_weights(const w12_conv_args& a, int c, float w[8][W]) {
  const uint16_t* p = a.weight + (int64_t)c * W;
  if (c + 8 <= a.channels) {
    float v[8 * W];
#pragma unroll
    for (int i = 0; i < W; ++i) unpack_bf16x8(reinterpret_cast<const uint4*>(p)[i], v + 8 * i);
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int j = 0; j < W; ++j) w[e][j] = v[e * W + j];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int j = 0; j < W; ++j) w[e][j] = c + e < a.channels ? bf16_float(p[e * W + j]) : 0.0f;
  }
}

template <bool F32, int W, bool TREE, int TILE>
__global__ __launch_bounds__(kConvThreads) void k_short_conv(w12_conv_args a, w12_sequences s) {
  constexpr int kPast = W - 1, kBytes = F32 ? 4 : 2;
  static_assert(TREE || TILE >= kPast, "the second tile would read the state that the first one replaces");
  __shared__ int found[2];
  int b, tile;
  Range r;
  // long tiles: the blocks of a tile's channels are neighbours, so that work-groups at work together read whole rows
  constexpr bool kFlat = TILE == kLongTile;
  const int blocks = kFlat ? (a.channels + 8 * kConvThreads - 1) / (8 * kConvThreads) : 1;
  const int block = kFlat ? blockIdx.x % blocks : blockIdx.y;
  if (!find_piece(s, blockIdx.x / blocks, TILE, found, b, r, tile)) return;
  if (tile > 0 && !a.y) return;                      // only the first tile moves a state
  const int c = (block * kConvThreads + threadIdx.x) * 8;
  if (c >= a.channels) return;
  const int src = slot_of(s, s.src, b), dst = slot_of(s, s.dst, b);
  // a token of the sequence, or of its past: -1 is the newest; zeros where there is none
  auto token = [&](int i, float v[8]) {
    const char* from = nullptr;
    if (i < 0) {
      if (src >= 0 && i >= -kPast) from = static_cast<const char*>(a.state) + (src * a.slot_stride + (kPast + i) * a.tap_stride) * kBytes;
    } else if (i < r.n) {
      const int row = row_of(s, r.start + i);
      if (row >= 0) from = static_cast<const char*>(a.x) + row * a.ldx * kBytes;
    }
    if (from) {
      load8<F32>(from, c, a.channels, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.0f;
    }
  };
  if (a.y) {
    float w[8][W], bias[8];
    load_weights<W>(a, c, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) bias[e] = a.bias && c + e < a.channels ? bf16_float(a.bias[c + e]) : 0.0f;
    // the output of token t from its window, oldest first
    auto put = [&](int t, auto window) {
      if (t >= r.n) return;
      const int row = row_of(s, r.start + t);
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] = bias[e];
#pragma unroll
        for (int j = 0; j < W; ++j) y[e] += w[e][j] * window(j)[e];
        if (a.silu) y[e] *= __builtin_amdgcn_rcpf(1.0f + __expf(-y[e]));
      }
      if (row >= 0) store8<false>(a.y + row * a.ldy, c, a.channels, y);
    };
    const int t0 = tile * TILE;
    if constexpr (TREE) {
      for (int t = t0; t < t0 + TILE; t += 2) {
        float x[2][W][8];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint64_t before = t + k < r.n ? ancestors(s, r.start, t + k) : 0;
          int at = t + k < r.n ? t + k : r.n, back = 0;        // back: how far into the past
#pragma unroll
          for (int j = W - 1; j >= 0; --j) {
            token(at, x[k][j]);
            if (before) {
              at = 63 - __builtin_clzll(before);
              before &= ~((uint64_t)1 << at);
            } else {
              at = --back;
            }
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) put(t + k, [&](int j) { return x[k][j]; });
      }
    } else {
      constexpr int kAtOnce = 4;      // rows whose loads a thread has in flight
      float x[kPast + kAtOnce][8];
#pragma unroll
      for (int j = 0; j < kPast; ++j) token(t0 - kPast + j, x[j]);
      for (int t = t0; t < min(t0 + TILE, r.n); t += kAtOnce) {
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) token(t + k, x[kPast + k]);
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) put(t + k, [&](int j) { return x[k + j]; });
#pragma unroll
        for (int j = 0; j < kPast; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) x[j][e] = x[j + kAtOnce][e];
      }
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

template <bool F32, int W>
static void conv_tiles(const w12_conv_args& a, const w12_sequences& s, hipStream_t stream) {
  const int64_t blocks = ceil_div(a.channels, 8 * kConvThreads);
  // Two waves a SIMD at least: between 2048 rows of 10240 channels (short tiles 36 us, long ones 39) and 4096 of 8192 (54 and 51; of 10240 64 and 59).
  const bool longer = !s.tree_mask && s.T / kLongTile * blocks >= 2 * 4 * device_cus();
  const int tile = s.tree_mask ? kTreeTile : longer ? kLongTile : kShortTile;
  const int64_t pieces = most_pieces(s.T, s.count, tile);
  const dim3 grid((unsigned)(longer ? pieces * blocks : pieces), (unsigned)(longer ? 1 : blocks));
  if (s.tree_mask) k_short_conv<F32, W, true, kTreeTile><<<grid, kConvThreads, 0, stream>>>(a, s);
  else if (longer) k_short_conv<F32, W, false, kLongTile><<<grid, kConvThreads, 0, stream>>>(a, s);
  else k_short_conv<F32, W, false, kShortTile><<<grid, kConvThreads, 0, stream>>>(a, s);
}

hipError_t launch_short_conv(const w12_conv_args& a, const w12_sequences& s, hipStream_t stream) {
  const bool f32 = a.dtype == W12_DTYPE_F32;
  switch (a.width) {
    case 2: f32 ? conv_tiles<true, 2>(a, s, stream) : conv_tiles<false, 2>(a, s, stream); break;
    case 3: f32 ? conv_tiles<true, 3>(a, s, stream) : conv_tiles<false, 3>(a, s, stream); break;
    default: f32 ? conv_tiles<true, 4>(a, s, stream) : conv_tiles<false, 4>(a, s, stream); break;
  }
  return hipGetLastError();
}

}  // namespace w12
