// Sequences of rows, shared by the operators that carry a state: which rows a sequence has, the tree
// that they form, and the work-groups' way from an index to a sequence.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/w12.h"

namespace w12 {

// A sequence's range of tokens, cut to what is there.
struct Range {
  int start, n;
};

__device__ __forceinline__ Range range_of(const w12_sequences& s, int b) {
  Range r;
  r.start = min(max(s.ptr[b], 0), s.T);
  r.n = min(max(s.ptr[b + 1], r.start), s.T) - r.start;
  if (s.lens) r.n = min(r.n, max(s.lens[b], 0));
  if (s.tree_mask) r.n = min(r.n, W12_TREE_NODES);
  return r;
}

// The row of token t (a place in ptr's numbering), or -1 where it names none.
__device__ __forceinline__ int row_of(const w12_sequences& s, int t) {
  if (!s.rows) return t;
  const int r = s.rows[t];
  return (uint32_t)r < (uint32_t)s.T ? r : -1;
}

// Slots of a sequence's old and new state, or -1.
__device__ __forceinline__ int slot_of(const w12_sequences& s, const int32_t* which, int b) {
  if (!which) return -1;
  const int i = which[b];
  return (uint32_t)i < (uint32_t)s.slots ? i : -1;
}

// Of up to 64 tokens from `start` on, those before token i: all of them, or in a tree its ancestors.
__device__ __forceinline__ uint64_t ancestors(const w12_sequences& s, int start, int i) {
  const uint64_t below = ((uint64_t)1 << i) - 1;
  return s.tree_mask ? s.tree_mask[(int64_t)(start + i) * s.ld_mask] & below : below;
}

// Whether a sum of squares (with eps) has a norm in FP32: not one of zeros or of what is too small for the type, nor one past it or NaN.
__device__ __forceinline__ bool has_norm(float sum) { return sum >= 0x1p-126f && sum < INFINITY; }

// Pieces of `step` rows: sequence b's are numbered from start / step + b on, which keeps the numbers of
// different sequences apart without a sum over their lengths; T / step + count numbers are enough for all.
__host__ __device__ inline int64_t most_pieces(int64_t T, int64_t count, int step) { return T / step + count; }
__device__ __forceinline__ int first_piece(const Range& r, int b, int step) { return r.start / step + b; }

// The sequence of a piece and its place there; false where the number belongs to none.  Called by a whole
// work-group; `found` is two ints of LDS.  Every thread looks at sequences of its own, so the search takes one round of
// loads for up to blockDim sequences.
__device__ __forceinline__ bool find_piece(const w12_sequences& s, int piece, int step, int* found, int& b, Range& r, int& at) {
  if (threadIdx.x == 0) found[0] = -1;
  __syncthreads();
  for (int i = threadIdx.x; i < s.count; i += blockDim.x) {
    const Range ri = range_of(s, i);
    const int p = piece - first_piece(ri, i, step);
    // a sequence without rows has one piece all the same: its state has to be copied
    if (p >= 0 && p < max(1, (ri.n + step - 1) / step)) found[0] = i;
  }
  __syncthreads();
  b = __builtin_amdgcn_readfirstlane(found[0]);
  if (b < 0) return false;
  r = range_of(s, b);
  at = piece - first_piece(r, b, step);
  return true;
}

}  // namespace w12
