// Verification of drafted tokens against the target's probabilities.
//
// With the weights w_i = exp((z_i - max z) / temperature) of a row, its token is the first i whose running sum passes u
// times the total.  A first kernel takes every row's logits once, in pieces, and leaves each piece's maximum and
// sum of weights; a second one, a work-group per row, finds the piece in which the running sum passes, and the token in
// it; the last of a request's work-groups to arrive walks down the tree.  A chain with the drafter's probabilities needs
// no row's token but one: its acceptances follow from the sums alone, and the row after which it was cut is gone over in
// pieces again, with the last work-group to arrive picking the token.
// Everything that decides is FP64 (which here runs at the rate of FP32), so that the token does not depend on how the sum was split:
// a border between two tokens is missed by 2^-40 of the total at the most.
//
// Measured: 266 rows of 131072 logits of FP32 take 53 us, 41 of them the first kernel (139 MB, 3.4 TB/s: the FP64 weights, 13 operations each,
// run partly beside the loads), 12 the second; 63 rows 21 us (14 and 8), a chain of 17 rows of 50257 with the drafter's
// probabilities 18 (4 and 14: acceptances, the cut row's pieces and the last arriver's pick, one after another).
#include <limits.h>

#include "w12_gemm_common.h"
#include "w12_lanes.h"
#include "w12_kernels.h"
#include "w12_rows.h"

namespace w12 {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWaves = kVerifyThreads / 64;
// Values of a piece: for each wave so many rounds of 256 neighbours.  Few rows take short pieces, which fill the chip (when the rule was measured,
// 17 rows of 50257: 19 us, with 4 rounds 24; 63 of 131072: 25 and 27), many rows longer ones, with less to do around them (266 of 131072: 65 and 60 us).
constexpr int kShortRounds = 2, kLongRounds = 4;
constexpr int64_t kLongFrom = 4096;                            // long pieces of a call, two rounds of the chip
constexpr int piece_values(int rounds) { return kVerifyThreads * 4 * rounds; }

// A piece's maximum, where it is first met, and the sum of its weights relative to it.
struct Piece {
  double sum;
  float max;
  int at;
};

struct Verify {
  w12_verify_draft_args a;
  Piece* pieces;         // [T][count]
  double* rest;          // [requests][count]: sums of max(p - q, 0) of a cut chain
  int32_t* taken;        // [T]: the rows' tokens
  uint32_t* arrived;     // [requests]
  int count;             // pieces of a row
};

struct Nodes {
  int start, n;
};
__device__ __forceinline__ Nodes nodes_of(const w12_verify_draft_args& a, int b, bool all = false) {
  Nodes r;
  r.start = min(max(a.node_ptr[b], 0), a.T);
  r.n = min(max(a.node_ptr[b + 1], r.start), a.T) - r.start;
  if (!all) r.n = min(r.n, W12_VERIFY_NODES);
  return r;
}
// The last request that starts at or before a row: a wave looks at 64 of them at once.
__device__ __forceinline__ int request_of_row(const w12_verify_draft_args& a, int row) {
  const int lane = threadIdx.x & 63;
  int b = 0;
  for (int i = 1; i < a.requests; i += 64) {
    const uint64_t at = __ballot(i + lane < a.requests && a.node_ptr[i + lane] <= row);
    b += __builtin_popcountll(at);
    if (at != ~(uint64_t)0) break;
  }
  return b;
}
__device__ __forceinline__ float temperature_of(const w12_verify_draft_args& a, int b) {
  const float t = a.temperature ? a.temperature[b] : 1.0f;
  return t > 0.0f ? t : 0.0f;
}
__device__ __forceinline__ int parent_of(const w12_verify_draft_args& a, int start, int i) {
  if (!a.tree_mask) return i - 1;
  const uint64_t* m = a.tree_mask + (int64_t)(start + i) * a.ld_mask;
  for (int w = min(i >> 6, a.mask_words - 1); w >= 0; --w) {
    uint64_t bits = m[w];
    if (w == i >> 6) bits &= ((uint64_t)1 << (i & 63)) - 1;
    if (bits) return w * 64 + 63 - __builtin_clzll(bits);
  }
  return -1;
}
__device__ __forceinline__ double random_of(const float* u, int row) {
  const float x = u[row];
  return (double)(x >= 0.0f ? min(x, 0.99999994f) : 0.0f);
}
__device__ __forceinline__ float no_nan(float z) { return z == z ? z : -INFINITY; }
template <bool F32>
__device__ __forceinline__ float logit(const w12_verify_draft_args& a, int64_t row, int i) {
  return no_nan(F32 ? static_cast<const float*>(a.logits)[row * a.ld_logits + i]
                    : bf16_float(static_cast<const uint16_t*>(a.logits)[row * a.ld_logits + i]));
}

// 2^t of t <= 0, to 2^-41.6 of itself: 2^f of the rest f in [-1/2, 1/2] by its series, whose first term left out is (ln 2 / 2)^11 / 11! =
// 2^-42.1, of 2^(-1/2) at the least.
// t is rounded by adding 3/2 2^52, which leaves the whole number in the low bits; it goes into the exponent as it is (rounding and
// scaling instructions of FP64 run at a part of the rate).  What is below 2^-1000 is 0.
__device__ __forceinline__ double power(double t) {
  constexpr double shift = 6755399441055744.0;
  const double n = t + shift, f = t - (n - shift);
  constexpr double l = 0.69314718055994530942;
  constexpr double c2 = l * l / 2, c3 = c2 * l / 3, c4 = c3 * l / 4, c5 = c4 * l / 5, c6 = c5 * l / 6, c7 = c6 * l / 7, c8 = c7 * l / 8,
                   c9 = c8 * l / 9, c10 = c9 * l / 10;
  double p = fma(f, c10, c9);
  p = fma(f, p, c8);
  p = fma(f, p, c7);
  p = fma(f, p, c6);
  p = fma(f, p, c5);
  p = fma(f, p, c4);
  p = fma(f, p, c3);
  p = fma(f, p, c2);
  p = fma(f, p, l);
  p = fma(f, p, 1.0);
  const uint64_t bits = __builtin_bit_cast(uint64_t, p);
  const uint32_t whole = (uint32_t)__builtin_bit_cast(uint64_t, n) << 20;
  const double r = __builtin_bit_cast(double, (uint64_t)((uint32_t)(bits >> 32) + whole) << 32 | (uint32_t)bits);
  return t > -1000.0 ? r : 0.0;
}
// log2(e) / temperature
__device__ __forceinline__ double steepness(float t) { return 1.4426950408889634074 / (double)t; }
// The weight of a logit beside the row's largest.  A row whose largest is +inf gives all to the first of them, a temperature of 0 to the
// first of the largest: those are told apart by the place alone.
__device__ __forceinline__ double weight(float z, float top, double steep) { return power(((double)z - (double)top) * steep); }

// A wave's, and a work-group's, sums, and what was before each thread.
__device__ __forceinline__ double scan_wave(double v, double& before) {
  const double s = sum_up(v);
  before = s - v;
  const uint64_t u = __builtin_bit_cast(uint64_t, s);
  return __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), 63) << 32 |
                                        (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, 63));
}
__device__ __forceinline__ double scan_group(double v, double* lds, double& before) {
  const int w = threadIdx.x >> 6;
  const double mine = scan_wave(v, before);
  if ((threadIdx.x & 63) == 0) lds[w] = mine;
  __syncthreads();
  double off = 0.0, total = 0.0;
#pragma unroll
  for (int i = 0; i < kVerifyWaves; ++i) {
    if (i < w) off += lds[i];
    total += lds[i];
  }
  before += off;
  __syncthreads();
  return total;
}
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ int first_of(int a, int b) { return min(a, b); }
__device__ __forceinline__ int last_of(int a, int b) { return max(a, b); }
// The largest of a work-group's values, and where it is first met.
__device__ __forceinline__ void largest(float& top, int& at, float* ldsf, int* ldsi) {
  const float m = over_wave(top, larger);
  at = over_wave(top == m ? at : INT_MAX, first_of);
  top = m;
  if ((threadIdx.x & 63) == 0) ldsf[threadIdx.x >> 6] = top, ldsi[threadIdx.x >> 6] = at;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kVerifyWaves; ++i)
    if (ldsf[i] > top || (ldsf[i] == top && ldsi[i] < at)) top = ldsf[i], at = ldsi[i];
  __syncthreads();
}

struct VerifyLds {
  double d[kVerifyWaves], target;
  float f[kVerifyWaves];
  int i[kVerifyWaves], found, last;
  uint32_t place;
};

// A row's largest logit, its place (INT_MAX: there is none), and the sum of weights.
struct Row {
  float top;
  int at;
  double total, steep;
  bool one;              // the whole weight is in `at`
};

// A row of its pieces, by a work-group.  Threads take neighbouring pieces; `mine` is the weight of a thread's, `before` of those in front.
__device__ __forceinline__ int pieces_each(int count) { return (count + kVerifyThreads - 1) / kVerifyThreads; }
__device__ __forceinline__ double piece_weight(const Piece& p, const Row& r) { return p.at < 0 ? 0.0 : p.sum * weight(p.max, r.top, r.steep); }
__device__ __forceinline__ Row row_of_pieces(const Verify& v, int row, float t, VerifyLds& lds, double& mine, double& before) {
  Row r;
  r.top = -INFINITY;
  r.at = INT_MAX;
  const Piece* p = v.pieces + (int64_t)row * v.count;
  const int each = pieces_each(v.count), p0 = threadIdx.x * each, p1 = min(p0 + each, v.count);
  for (int i = p0; i < p1; ++i)
    if (p[i].at >= 0 && (r.at == INT_MAX || p[i].max > r.top)) r.top = p[i].max, r.at = p[i].at;
  largest(r.top, r.at, lds.f, lds.i);
  r.one = t == 0.0f || r.top == INFINITY;
  r.steep = r.one ? 1.0 : steepness(t);
  mine = 0.0;
  if (r.at != INT_MAX && !r.one)
    for (int i = p0; i < p1; ++i) mine += piece_weight(p[i], r);
  r.total = scan_group(mine, lds.d, before);
  return r;
}
// The same by 16 lanes, for a row of their own; the sum alone.
__device__ __forceinline__ Row row_of_lanes(const Verify& v, int row, float t) {
  Row r;
  r.top = -INFINITY;
  r.at = INT_MAX;
  const Piece* p = v.pieces + (int64_t)row * v.count;
  const int lane = threadIdx.x & 15;
  for (int i = lane; i < v.count; i += 16)
    if (p[i].at >= 0 && (r.at == INT_MAX || p[i].max > r.top)) r.top = p[i].max, r.at = p[i].at;
  const float m = over_row(r.top, larger);
  r.at = over_row(r.top == m ? r.at : INT_MAX, first_of);
  r.top = m;
  r.one = t == 0.0f || r.top == INFINITY;
  r.steep = r.one ? 1.0 : steepness(t);
  r.total = 0.0;
  if (r.at != INT_MAX && !r.one)
    for (int i = lane; i < v.count; i += 16) r.total += piece_weight(p[i], r);
  r.total = over_row(r.total, [](double a, double b) { return a + b; });
  return r;
}

// Of a work-group's threads with weights of their own and the weight before them: the first whose running sum passes `target`, and the
// last with a weight, should rounding leave none.  The thread then looks at its parts.  What is before a thread counts for nothing: it
// may be an ulp above the running sum of the thread in front, and a target between the two belongs to either.
template <typename F>
__device__ __forceinline__ void pass_to(double target, double mine, double before, VerifyLds& lds, F parts) {
  if (threadIdx.x == 0) lds.found = INT_MAX, lds.last = -1;
  __syncthreads();
  const bool has = mine > 0.0;
  const uint64_t any = __ballot(has), in = __ballot(has && target < before + mine);
  if ((threadIdx.x & 63) == 0) {
    if (in) atomicMin(&lds.found, (int)threadIdx.x + __builtin_ctzll(in));
    if (any) atomicMax(&lds.last, (int)threadIdx.x + 63 - __builtin_clzll(any));
  }
  __syncthreads();
  const int who = lds.found != INT_MAX ? lds.found : lds.last;
  if ((int)threadIdx.x == who) parts(target - before);
  __syncthreads();
}

// Where a thread's values of a piece are: 4 neighbours, every 256.
template <int R>
__device__ __forceinline__ int place_of(int piece, int round) {
  return piece * piece_values(R) + (int)(threadIdx.x >> 6) * (256 * R) + round * 256 + (int)(threadIdx.x & 63) * 4;
}
// Four neighbouring logits, -inf past the end.
template <bool F32>
__device__ __forceinline__ void logits4(const w12_verify_draft_args& a, int64_t row, int i, float z[4]) {
  if (i + 4 <= a.vocab) {
    if constexpr (F32) {
      const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + row * a.ld_logits + i);
      z[0] = x.x; z[1] = x.y; z[2] = x.z; z[3] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.logits) + row * a.ld_logits + i);
      z[0] = bf16_float(x.x); z[1] = __builtin_bit_cast(float, x.x & 0xFFFF0000u);
      z[2] = bf16_float(x.y); z[3] = __builtin_bit_cast(float, x.y & 0xFFFF0000u);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e] = no_nan(z[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e] = i + e < a.vocab ? logit<F32>(a, row, i + e) : -INFINITY;
  }
}

// The token of a piece in whose weights the running sum passes lds.target; weights4(i, w) gives those of places i .. i + 3.  By a whole work-group.
template <int R, typename F>
__device__ __forceinline__ int find_token(int piece, VerifyLds& lds, F weights4) {
  double w[R][4], round[R], sum = 0.0, before, unused;
#pragma unroll
  for (int j = 0; j < R; ++j) {
    weights4(place_of<R>(piece, j), w[j]);
    round[j] = w[j][0] + w[j][1] + w[j][2] + w[j][3];
    sum += round[j];
  }
  const double target = lds.target;
  const double wave = scan_wave(sum, unused);
  if ((threadIdx.x & 63) == 0) lds.d[threadIdx.x >> 6] = wave;
  if (threadIdx.x == 0) lds.found = INT_MAX, lds.last = -1;
  __syncthreads();
  double run = 0.0;
  for (int i = 0; i < (int)(threadIdx.x >> 6); ++i) run += lds.d[i];
  // every wave goes through its values; the first place that passes is the token
  int first = INT_MAX, last = -1;
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const double all = scan_wave(round[j], before);
    double at = run + before;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      at += w[j][e];
      if (w[j][e] > 0.0) {
        if (at > target) first = min(first, place_of<R>(piece, j) + e);
        last = place_of<R>(piece, j) + e;
      }
    }
    run += all;
  }
  // one lane for the wave: atomics on one place go one after another
  first = over_wave(first, first_of);
  last = over_wave(last, last_of);
  if ((threadIdx.x & 63) == 0) {
    atomicMin(&lds.found, first);
    atomicMax(&lds.last, last);
  }
  __syncthreads();
  const int token = lds.found != INT_MAX ? lds.found : lds.last;
  __syncthreads();
  return token;
}

// Whether this work-group is the last of `of` of a request to arrive.  What the others' first threads stored before, by atomics of the
// device's scope, is then there for loads of that scope.
__device__ __forceinline__ bool last_to_arrive(uint32_t* counter, uint32_t of, uint32_t* lds) {
  if (threadIdx.x == 0) *lds = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  const bool last = *lds == of - 1;
  __syncthreads();
  return last;
}

template <bool F32, int R>
__global__ __launch_bounds__(kVerifyThreads) void k_pieces(Verify v) {
  const w12_verify_draft_args& a = v.a;
  __shared__ VerifyLds lds;
  const int piece = blockIdx.y, row = blockIdx.x;
  float z[R][4];
#pragma unroll
  for (int j = 0; j < R; ++j) logits4<F32>(a, row, place_of<R>(piece, j), z[j]);
  if (row == 0 && piece == 0)
    for (int i = threadIdx.x; i < a.requests; i += kVerifyThreads) {
      v.arrived[i] = 0;
      if (nodes_of(a, i).n == 0) a.count[i] = 0, a.next_token[i] = -1;
    }
  const float t = temperature_of(a, request_of_row(a, row));
  float top = -INFINITY;
  int at = INT_MAX;
#pragma unroll
  for (int j = 0; j < R; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (z[j][e] > top) top = z[j][e], at = place_of<R>(piece, j) + e;
  largest(top, at, lds.f, lds.i);
  double sum = 0.0, before;
  if (t > 0.0f && at != INT_MAX && top != INFINITY) {
    const double steep = steepness(t);
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum += weight(z[j][e], top, steep);
  }
  sum = scan_group(sum, lds.d, before);
  if (threadIdx.x == 0) v.pieces[(int64_t)row * v.count + piece] = Piece{sum, top, at == INT_MAX ? -1 : at};
}

// The token that u takes from a row, by a whole work-group.
template <bool F32, int R>
__device__ __forceinline__ int take(const Verify& v, int row, float t, VerifyLds& lds) {
  const w12_verify_draft_args& a = v.a;
  double mine, before;
  const Row r = row_of_pieces(v, row, t, lds, mine, before);
  if (r.at == INT_MAX) return -1;
  if (r.one) return r.at;
  const Piece* p = v.pieces + (int64_t)row * v.count;
  pass_to(random_of(a.u, row) * r.total, mine, before, lds, [&](double target) {
    const int each = pieces_each(v.count), p0 = threadIdx.x * each, p1 = min(p0 + each, v.count);
    int in = p0;
    double run = 0.0, start = 0.0;
    for (int i = p0; i < p1; ++i) {
      const double w = piece_weight(p[i], r);
      if (w > 0.0) in = i, start = run;
      run += w;
      if (w > 0.0 && run > target) break;
    }
    lds.place = (uint32_t)in;
    lds.target = target - start;
  });
  const int piece = (int)lds.place;
  return find_token<R>(piece, lds, [&](int i, double w[4]) {
    float z[4];
    logits4<F32>(a, row, i, z);
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = weight(z[e], r.top, r.steep);
  });
}

// The token of every row, and the walk.
template <bool F32, int R>
__global__ __launch_bounds__(kVerifyThreads) void k_take(Verify v) {
  const w12_verify_draft_args& a = v.a;
  __shared__ VerifyLds lds;
  __shared__ int child[W12_VERIFY_NODES];
  const int row = blockIdx.x, b = request_of_row(a, row);
  const Nodes nodes = nodes_of(a, b);
  if (row < nodes.start || row >= nodes.start + nodes.n) return;
  const int token = take<F32, R>(v, row, temperature_of(a, b), lds);
  if (threadIdx.x == 0) __hip_atomic_store(&v.taken[row], token, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (!last_to_arrive(&v.arrived[b], (uint32_t)nodes.n, &lds.place)) return;
  for (int i = threadIdx.x; i < nodes.n; i += kVerifyThreads) child[i] = INT_MAX;
  __syncthreads();
  for (int i = 1 + threadIdx.x; i < nodes.n; i += kVerifyThreads) {
    const int up = parent_of(a, nodes.start, i), mine = a.tokens[nodes.start + i];
    if (up >= 0 && mine >= 0 && mine == __hip_atomic_load(&v.taken[nodes.start + up], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT))
      atomicMin(&child[up], i);
  }
  __syncthreads();
  const int all = nodes_of(a, b, true).n;
  if (threadIdx.x == 0) {
    int at = 0, n = 0;
    for (;;) {
      a.path[nodes.start + n++] = nodes.start + at;
      if (child[at] == INT_MAX) break;
      at = child[at];                     // children come after their parents, so this ends
    }
    a.count[b] = n;
    a.next_token[b] = __hip_atomic_load(&v.taken[nodes.start + at], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    lds.found = n;
  }
  __syncthreads();
  for (int i = lds.found + threadIdx.x; i < all; i += kVerifyThreads) a.path[nodes.start + i] = -1;
}

// A chain with the drafter's probabilities: acceptances, and the token after the cut.
template <bool F32, int R>
__global__ __launch_bounds__(kVerifyThreads) void k_chain(Verify v) {
  const w12_verify_draft_args& a = v.a;
  __shared__ VerifyLds lds;
  __shared__ int cut;
  const int piece = blockIdx.x, b = blockIdx.y;
  const Nodes nodes = nodes_of(a, b);
  if (nodes.n == 0) return;
  const float t = temperature_of(a, b);
  if (threadIdx.x == 0) cut = nodes.n;
  __syncthreads();
  for (int i0 = 1; i0 < nodes.n; i0 += kVerifyThreads / 16) {
    const int i = min(i0 + (int)(threadIdx.x >> 4), nodes.n - 1), row = nodes.start + i, x = a.tokens[row];
    const bool token = x >= 0 && x < a.vocab;
    const float z = token ? logit<F32>(a, row - 1, x) : 0.0f, qx = token ? a.q[row * a.ldq + x] : 0.0f;
    const Row r = row_of_lanes(v, row - 1, t);
    double p = 0.0;
    if (r.at != INT_MAX) p = r.one ? (x == r.at ? 1.0 : 0.0) : weight(z, r.top, r.steep) / r.total;
    const bool good = token && random_of(a.accept_u, row) * (double)qx < p;
    if (!good && (threadIdx.x & 15) == 0) atomicMin(&cut, i);
  }
  __syncthreads();
  const int n = cut, row = nodes.start + n - 1;
  const bool whole = n == nodes.n;
  double mine, before;
  const Row r = row_of_pieces(v, row, t, lds, mine, before);
  const double inverse = r.one || r.at == INT_MAX ? 0.0 : 1.0 / r.total;
  const float* const q = whole ? nullptr : a.q + (row + 1) * a.ldq;
  // what is left of p over q, which is all of p behind the last node
  auto rest4 = [&](int i, double w[4]) {
    float z[4];
    logits4<F32>(a, row, i, z);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      double p = 0.0;
      if (i + e < a.vocab && r.at != INT_MAX) p = r.one ? (i + e == r.at ? 1.0 : 0.0) : weight(z[e], r.top, r.steep) * inverse;
      if (!whole) {
        p = i + e < a.vocab ? p - (double)q[i + e] : 0.0;
        p = p > 0.0 ? p : 0.0;
      }
      w[e] = p;
    }
  };
  double sum = 0.0, w[4];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    rest4(place_of<R>(piece, j), w);
    sum += w[0] + w[1] + w[2] + w[3];
  }
  sum = scan_group(sum, lds.d, before);
  double* sums = v.rest + (int64_t)b * v.count;
  if (threadIdx.x == 0) __hip_atomic_store(&sums[piece], sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (!last_to_arrive(&v.arrived[b], (uint32_t)v.count, &lds.place)) return;
  const int each = pieces_each(v.count), p0 = threadIdx.x * each, p1 = min(p0 + each, v.count);
  auto sum_of = [&](int i) { return __hip_atomic_load(&sums[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
  mine = 0.0;
  for (int i = p0; i < p1; ++i) mine += sum_of(i);
  const double total = scan_group(mine, lds.d, before);
  int token;
  if (total > 0.0) {
    pass_to(random_of(a.u, row) * total, mine, before, lds, [&](double target) {
      int in = p0;
      double run = 0.0, start = 0.0;
      for (int i = p0; i < p1; ++i) {
        const double x = sum_of(i);
        if (x > 0.0) in = i, start = run;
        run += x;
        if (x > 0.0 && run > target) break;
      }
      lds.place = (uint32_t)in;
      lds.target = target - start;
    });
    const int in = (int)lds.place;
    token = find_token<R>(in, lds, rest4);
  } else {
    token = take<F32, R>(v, row, t, lds);      // nothing is left over: from p itself
  }
  if (threadIdx.x == 0) a.count[b] = n, a.next_token[b] = token;
  const int all = nodes_of(a, b, true).n;
  for (int i = threadIdx.x; i < all; i += kVerifyThreads) a.path[nodes.start + i] = i < n ? nodes.start + i : -1;
}

static uint64_t round16(uint64_t x) { return (x + 15) / 16 * 16; }

uint64_t verify_draft_workspace_bytes(int32_t T, int32_t requests, int32_t vocab) {
  const uint64_t count = ceil_div(vocab, piece_values(kShortRounds));
  return T * count * sizeof(Piece) + round16(requests * count * 8) + round16((uint64_t)T * 4) + round16((uint64_t)requests * 4);
}

template <bool F32, int R>
static void verify_launches(const Verify& v, hipStream_t stream) {
  k_pieces<F32, R><<<dim3((unsigned)v.a.T, (unsigned)v.count), kVerifyThreads, 0, stream>>>(v);
  if (v.a.q) k_chain<F32, R><<<dim3((unsigned)v.count, (unsigned)v.a.requests), kVerifyThreads, 0, stream>>>(v);
  else k_take<F32, R><<<(unsigned)v.a.T, kVerifyThreads, 0, stream>>>(v);
}

hipError_t launch_verify_draft(const w12_verify_draft_args& a, void* ws, hipStream_t stream) {
  const bool longer = a.T * ceil_div(a.vocab, piece_values(kLongRounds)) >= kLongFrom;
  Verify v;
  v.a = a;
  v.count = (int)ceil_div(a.vocab, piece_values(longer ? kLongRounds : kShortRounds));
  char* at = static_cast<char*>(ws);
  v.pieces = reinterpret_cast<Piece*>(at);
  at += (uint64_t)a.T * v.count * sizeof(Piece);
  v.rest = reinterpret_cast<double*>(at);
  at += round16((uint64_t)a.requests * v.count * 8);
  v.taken = reinterpret_cast<int32_t*>(at);
  at += round16((uint64_t)a.T * 4);
  v.arrived = reinterpret_cast<uint32_t*>(at);
  if (a.logits_dtype == W12_DTYPE_F32) longer ? verify_launches<true, kLongRounds>(v, stream) : verify_launches<true, kShortRounds>(v, stream);
  else longer ? verify_launches<false, kLongRounds>(v, stream) : verify_launches<false, kShortRounds>(v, stream);
  return hipGetLastError();
}

}  // namespace w12
