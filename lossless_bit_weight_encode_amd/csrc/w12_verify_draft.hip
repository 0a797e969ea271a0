// Verification of drafted tokens against the target's probabilities.
//
// With the weights w_i = exp((z_i - max z) / temperature) of a row, its token is the first i whose running sum passes u
// times the total.  A first kernel takes every row's logits once, in pieces, and leaves each piece's maximum and
// sum of weights; a second one, a work-group per row, finds the piece in which the running sum passes, and the token in
// it; the last of a request's work-groups to arrive walks down the tree.  A chain with the drafter's probabilities needs
// no row's token but one: its acceptances follow from the sums alone, and the row after which it was cut is gone over in
// pieces again, with the last work-group to arrive picking the token.
// Everything that decides is FP64, so that the token does not depend on how the sum was split (a border
// between two tokens is missed by 2^-40 of the total at the most).
#include <limits.h>

#include "w12_gemm_common.h"
#include "w12_kernels.h"
#include "w12_rows.h"

namespace w12 {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyValues = 32;                              // of a thread, neighbours
constexpr int kVerifyPiece = kVerifyThreads * kVerifyValues;   // values of a piece

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
// The last request that starts at or before a row.
__device__ __forceinline__ int request_of_row(const w12_verify_draft_args& a, int row) {
  int lo = 0, hi = a.requests;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.node_ptr[mid] <= row) lo = mid;
    else hi = mid;
  }
  return lo;
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
template <bool F32>
__device__ __forceinline__ float logit(const w12_verify_draft_args& a, int64_t row, int i) {
  const float z = F32 ? static_cast<const float*>(a.logits)[row * a.ld_logits + i]
                      : bf16_float(static_cast<const uint16_t*>(a.logits)[row * a.ld_logits + i]);
  return z == z ? z : -INFINITY;
}
// The weight of a logit beside the row's largest.  A row whose largest is +inf gives all to the first of them, a temperature of 0 to the
// first of the largest: those are told apart by the place alone.
__device__ __forceinline__ double weight(float z, float top, double inv_t) {
  return z == -INFINITY ? 0.0 : exp(((double)z - (double)top) * inv_t);
}

// A row's largest logit, its place, and the sum of weights (0: one place has it all, or there is none).
struct Row {
  float top;
  int at;
  double total, inv_t;
  bool one;              // the whole weight is in `at`
};

__device__ __forceinline__ Row row_of_pieces(const Verify& v, int row, float t) {
  Row r;
  r.top = -INFINITY;
  r.at = -1;
  const Piece* p = v.pieces + (int64_t)row * v.count;
  for (int i = 0; i < v.count; ++i)
    if (p[i].at >= 0 && (r.at < 0 || p[i].max > r.top)) r.top = p[i].max, r.at = p[i].at;
  r.one = t == 0.0f || r.top == INFINITY;
  r.inv_t = r.one ? 1.0 : 1.0 / (double)t;
  r.total = 0.0;
  if (r.at >= 0 && !r.one)
    for (int i = 0; i < v.count; ++i)
      if (p[i].at >= 0) r.total += p[i].sum * exp(((double)p[i].max - (double)r.top) * r.inv_t);
  return r;
}

// A work-group's sum, and each thread's sum of those before it.
__device__ __forceinline__ double scan_group(double v, double* lds, double& before) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  double s = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const double u = __shfl_up(s, o);
    if (lane >= o) s += u;
  }
  if (lane == 63) lds[w] = s;
  __syncthreads();
  double off = 0.0, total = 0.0;
  for (int i = 0; i < kVerifyThreads / 64; ++i) {
    if (i < w) off += lds[i];
    total += lds[i];
  }
  before = off + s - v;
  __syncthreads();
  return total;
}

template <bool F32>
__global__ __launch_bounds__(kVerifyThreads) void k_pieces(Verify v) {
  const w12_verify_draft_args& a = v.a;
  __shared__ float wmax[kVerifyThreads / 64];
  __shared__ int wat[kVerifyThreads / 64];
  __shared__ double lds[kVerifyThreads / 64];
  const int piece = blockIdx.y, row = blockIdx.x, lane = threadIdx.x & 63;
  if (row == 0 && piece == 0)
    for (int i = threadIdx.x; i < a.requests; i += kVerifyThreads) v.arrived[i] = 0;
  const int b = request_of_row(a, row);
  const float t = temperature_of(a, b);
  const int i0 = piece * kVerifyPiece + threadIdx.x * kVerifyValues;
  float z[kVerifyValues];
  float m = -INFINITY;
  int at = INT_MAX;
#pragma unroll
  for (int i = 0; i < kVerifyValues; ++i) {
    z[i] = i0 + i < a.vocab ? logit<F32>(a, row, i0 + i) : -INFINITY;
    if (z[i] > m) m = z[i], at = i0 + i;
  }
  float top = m;
  int first = at;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const float om = __shfl_xor(top, o);
    const int oa = __shfl_xor(first, o);
    if (om > top || (om == top && oa < first)) top = om, first = oa;
  }
  if (lane == 0) wmax[threadIdx.x >> 6] = top, wat[threadIdx.x >> 6] = first;
  __syncthreads();
  for (int i = 0; i < kVerifyThreads / 64; ++i)
    if (wmax[i] > top || (wmax[i] == top && wat[i] < first)) top = wmax[i], first = wat[i];
  double sum = 0.0, before;
  if (t > 0.0f && first != INT_MAX && top != INFINITY) {
    const double inv_t = 1.0 / (double)t;
#pragma unroll
    for (int i = 0; i < kVerifyValues; ++i) sum += weight(z[i], top, inv_t);
  }
  sum = scan_group(sum, lds, before);
  if (threadIdx.x == 0) v.pieces[(int64_t)row * v.count + piece] = Piece{sum, top, first == INT_MAX ? -1 : first};
}

// The place in a piece whose running sum of weights passes `target`; values(i) is the weight of place i of the row, where it is.  If rounding leaves
// none, the last place with a weight.
template <typename F>
__device__ __forceinline__ int find_place(int piece, double target, int* best, double* lds, F value) {
  const int i0 = piece * kVerifyPiece + threadIdx.x * kVerifyValues;
  if (threadIdx.x == 0) best[0] = INT_MAX, best[1] = -1;
  double sum = 0.0, before;
  int last = -1;
  for (int i = 0; i < kVerifyValues; ++i) {
    const double w = value(i0 + i);
    sum += w;
    if (w > 0.0) last = i0 + i;
  }
  scan_group(sum, lds, before);
  double run = before;
  for (int i = 0; i < kVerifyValues; ++i) {
    const double w = value(i0 + i);
    run += w;
    if (w > 0.0 && run > target) {
      atomicMin(&best[0], i0 + i);
      break;
    }
  }
  if (last >= 0) atomicMax(&best[1], last);
  __syncthreads();
  return best[0] != INT_MAX ? best[0] : best[1];
}

// Which piece the running sum passes `target` in, and the sum before it; the last with a weight if rounding leaves none.
template <typename F>
__device__ __forceinline__ int find_in(int count, double& target, F sum_of) {
  double run = 0.0;
  int last = -1;
  double last_before = 0.0;
  for (int i = 0; i < count; ++i) {
    const double s = sum_of(i);
    if (s > 0.0) {
      if (run + s > target) {
        target -= run;
        return i;
      }
      last = i;
      last_before = run;
    }
    run += s;
  }
  target -= last_before;
  return last;
}

// Whether this work-group is the last of `of` of a request to arrive; what the others wrote before is then visible.
__device__ __forceinline__ bool last_to_arrive(uint32_t* counter, uint32_t of, uint32_t* lds) {
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) *lds = atomicAdd(counter, 1u);
  __syncthreads();
  const bool last = *lds == of - 1;
  if (last) __threadfence();
  return last;
}

// The token of every row, and the walk.
template <bool F32>
__global__ __launch_bounds__(kVerifyThreads) void k_take(Verify v) {
  const w12_verify_draft_args& a = v.a;
  __shared__ double lds[kVerifyThreads / 64];
  __shared__ int best[2];
  __shared__ uint32_t place;
  __shared__ int child[W12_VERIFY_NODES];
  const int row = blockIdx.x, b = request_of_row(a, row);
  const Nodes nodes = nodes_of(a, b);
  if (row < nodes.start || row >= nodes.start + nodes.n) return;
  const Row r = row_of_pieces(v, row, temperature_of(a, b));
  int token = r.at;
  if (r.at >= 0 && !r.one) {
    double target = random_of(a.u, row) * r.total;
    const Piece* p = v.pieces + (int64_t)row * v.count;
    const int piece = find_in(v.count, target, [&](int i) {
      return p[i].at >= 0 ? p[i].sum * exp(((double)p[i].max - (double)r.top) * r.inv_t) : 0.0;
    });
    if (piece >= 0)
      token = find_place(piece, target, best, lds, [&](int i) { return i < a.vocab ? weight(logit<F32>(a, row, i), r.top, r.inv_t) : 0.0; });
  }
  if (threadIdx.x == 0) __hip_atomic_store(&v.taken[row], token, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (!last_to_arrive(&v.arrived[b], (uint32_t)nodes.n, &place)) return;
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
    best[0] = n;
  }
  __syncthreads();
  for (int i = best[0] + threadIdx.x; i < all; i += kVerifyThreads) a.path[nodes.start + i] = -1;
}

// A chain with the drafter's probabilities: acceptances, and the token after the cut.
template <bool F32>
__global__ __launch_bounds__(kVerifyThreads) void k_chain(Verify v) {
  const w12_verify_draft_args& a = v.a;
  __shared__ double lds[kVerifyThreads / 64];
  __shared__ int best[2], cut;
  __shared__ uint32_t place;
  const int piece = blockIdx.x, b = blockIdx.y;
  const Nodes nodes = nodes_of(a, b);
  if (nodes.n == 0) return;
  const float t = temperature_of(a, b);
  if (threadIdx.x == 0) cut = nodes.n;
  __syncthreads();
  for (int i = 1 + threadIdx.x; i < nodes.n; i += kVerifyThreads) {
    const int row = nodes.start + i, x = a.tokens[row];
    bool good = false;
    if (x >= 0 && x < a.vocab) {
      const Row r = row_of_pieces(v, row - 1, t);
      double p = 0.0;
      if (r.at >= 0) p = r.one ? (x == r.at ? 1.0 : 0.0) : weight(logit<F32>(a, row - 1, x), r.top, r.inv_t) / r.total;
      good = random_of(a.accept_u, row) * (double)a.q[row * a.ldq + x] < p;
    }
    if (!good) atomicMin(&cut, i);
  }
  __syncthreads();
  const int n = cut, row = nodes.start + n - 1;
  const bool whole = n == nodes.n;
  const Row r = row_of_pieces(v, row, t);
  const float* q = whole ? nullptr : a.q + (row + 1) * a.ldq;
  auto p_of = [&](int i) -> double {
    if (i >= a.vocab || r.at < 0) return 0.0;
    return r.one ? (i == r.at ? 1.0 : 0.0) : weight(logit<F32>(a, row, i), r.top, r.inv_t) / r.total;
  };
  auto rest_of = [&](int i) -> double {
    if (i >= a.vocab) return 0.0;
    const double d = p_of(i) - (double)q[i];
    return d > 0.0 ? d : 0.0;
  };
  double sum = 0.0, before;
  for (int i = 0; i < kVerifyValues; ++i) {
    const int at = piece * kVerifyPiece + threadIdx.x * kVerifyValues + i;
    sum += whole ? p_of(at) : rest_of(at);
  }
  sum = scan_group(sum, lds, before);
  double* sums = v.rest + (int64_t)b * v.count;
  if (threadIdx.x == 0) __hip_atomic_store(&sums[piece], sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (!last_to_arrive(&v.arrived[b], (uint32_t)v.count, &place)) return;
  auto sum_of = [&](int i) { return __hip_atomic_load(&sums[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
  double total = 0.0;
  for (int i = 0; i < v.count; ++i) total += sum_of(i);
  int token = -1;
  const double u = random_of(a.u, row);
  if (total > 0.0) {
    double target = u * total;
    const int in = find_in(v.count, target, sum_of);
    token = find_place(in, target, best, lds, [&](int i) { return whole ? p_of(i) : rest_of(i); });
  } else if (r.at >= 0) {
    // nothing is left over: from p itself
    token = r.at;
    if (!r.one) {
      const Piece* p = v.pieces + (int64_t)row * v.count;
      double target = u * r.total;
      const int in = find_in(v.count, target, [&](int i) {
        return p[i].at >= 0 ? p[i].sum * exp(((double)p[i].max - (double)r.top) * r.inv_t) : 0.0;
      });
      token = find_place(in, target / r.total, best, lds, p_of);
    }
  }
  if (threadIdx.x == 0) a.count[b] = n, a.next_token[b] = token;
  const int all = nodes_of(a, b, true).n;
  for (int i = threadIdx.x; i < all; i += kVerifyThreads) a.path[nodes.start + i] = i < n ? nodes.start + i : -1;
}

// Requests without nodes.
__global__ __launch_bounds__(kVerifyThreads) void k_empty(Verify v) {
  const int b = blockIdx.x * kVerifyThreads + threadIdx.x;
  if (b >= v.a.requests || nodes_of(v.a, b).n) return;
  v.a.count[b] = 0;
  v.a.next_token[b] = -1;
}

static uint64_t round16(uint64_t x) { return (x + 15) / 16 * 16; }

uint64_t verify_draft_workspace_bytes(int32_t T, int32_t requests, int32_t vocab) {
  const uint64_t count = ceil_div(vocab, kVerifyPiece);
  return T * count * sizeof(Piece) + round16(requests * count * 8) + round16((uint64_t)T * 4) + round16((uint64_t)requests * 4);
}

hipError_t launch_verify_draft(const w12_verify_draft_args& a, void* ws, hipStream_t stream) {
  Verify v;
  v.a = a;
  v.count = (int)ceil_div(a.vocab, kVerifyPiece);
  char* at = static_cast<char*>(ws);
  v.pieces = reinterpret_cast<Piece*>(at);
  at += (uint64_t)a.T * v.count * sizeof(Piece);
  v.rest = reinterpret_cast<double*>(at);
  at += round16((uint64_t)a.requests * v.count * 8);
  v.taken = reinterpret_cast<int32_t*>(at);
  at += round16((uint64_t)a.T * 4);
  v.arrived = reinterpret_cast<uint32_t*>(at);
  const bool f32 = a.logits_dtype == W12_DTYPE_F32;
  const dim3 grid((unsigned)a.T, (unsigned)v.count);
  if (f32) k_pieces<true><<<grid, kVerifyThreads, 0, stream>>>(v);
  else k_pieces<false><<<grid, kVerifyThreads, 0, stream>>>(v);
  k_empty<<<(unsigned)ceil_div(a.requests, kVerifyThreads), kVerifyThreads, 0, stream>>>(v);
  const dim3 chains((unsigned)v.count, (unsigned)a.requests);
  if (a.q) {
    if (f32) k_chain<true><<<chains, kVerifyThreads, 0, stream>>>(v);
    else k_chain<false><<<chains, kVerifyThreads, 0, stream>>>(v);
  } else {
    if (f32) k_take<true><<<(unsigned)a.T, kVerifyThreads, 0, stream>>>(v);
    else k_take<false><<<(unsigned)a.T, kVerifyThreads, 0, stream>>>(v);
  }
  return hipGetLastError();
}

}  // namespace w12
