// The gated delta rule, token by token.
//
//   S <- exp(g) S + k (beta (v - exp(g) S^T k))^T,  out = scale S^T q.
//
// The columns of S (one per element of v) do not depend on one another.  A column lies along the lanes of a wave,
// 8 values a lane, so that S^T k and S^T q are sums over 8 or 16 lanes (of the old state both: S'^T q = exp(g) S^T q + (k . q) u);
// a wave holds 16 columns in registers and walks through its tokens without a barrier.
//
// Single tokens are bound by the states, which are read and written once: 64 sequences of 48 heads of 128 x 128 take 85 us (405 MB, 4.8 TB/s,
// what a copy reaches here), one takes 5 us (6.3 MB).  Accepted paths (16 sequences, 40 us for 102 MB) pay for each token besides: 6 waves
// share a SIMD's vector instructions, and the sums over lanes follow one another (loads a token ahead: 42 before).
#include <limits.h>

#include "w12_delta_steps.h"
#include "w12_kernels.h"

namespace w12 {

template <int DK>
__global__ __launch_bounds__(kDeltaThreads) void k_delta_steps(w12_delta_args a, w12_sequences s) {
  delta_steps<DK>(a, s, blockIdx.x, blockIdx.y, blockIdx.z, INT_MAX);
}

// Rows a sequence has, on average, from which a call has to have the workspace.  With lens the host does not know how many count; accepted
// paths are far shorter than the trees that they lead through.
static bool many_rows(const w12_sequences& s) {
  return s.tree_mask || s.T >= (int64_t)(s.lens ? W12_DELTA_CHUNK_FROM_LENS : W12_DELTA_CHUNK_FROM) * s.count;
}
// Whether some sequence can be long among short ones: 64 tokens beside 10 single ones (48 heads of 128) take 27 us so and 88 one by one, 700 beside
// 63 single ones 119 and 4040.  A call that has no long one after all pays 2 to 6 us (16 sequences of 8 tokens 45 instead of 40, 64 of 2
// tokens 90 instead of 88), hence 64 tokens and not the 12 from which a sequence gains.
static bool a_long_one(const w12_sequences& s) { return !s.lens && s.T - s.count + 1 >= W12_DELTA_CHUNK_LONG; }

uint64_t gated_delta_workspace_bytes(int32_t T, int32_t count, int32_t v_heads, int32_t dk, int32_t dv) {
  return delta_chunk_workspace_bytes(T, count, v_heads);
}
uint64_t gated_delta_call_bytes(const w12_sequences& s, int32_t v_heads) {
  return many_rows(s) ? delta_chunk_workspace_bytes(s.T, s.count, v_heads) : 0;
}

hipError_t launch_gated_delta(const w12_delta_args& a, const w12_sequences& s, void* ws, uint64_t ws_bytes, hipStream_t stream) {
  if (many_rows(s) || (a_long_one(s) && ws && ws_bytes >= delta_chunk_workspace_bytes(s.T, s.count, a.v_heads)))
    return launch_delta_chunks(a, s, ws, stream);
  const dim3 grid((unsigned)s.count, (unsigned)a.v_heads, (unsigned)(a.dv / kGroupColumns));
  if (a.dk == 64) k_delta_steps<64><<<grid, kDeltaThreads, 0, stream>>>(a, s);
  else k_delta_steps<128><<<grid, kDeltaThreads, 0, stream>>>(a, s);
  return hipGetLastError();
}

}  // namespace w12
