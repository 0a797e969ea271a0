// What the two kernels of the chunked gated delta rule hand over, by chunk and value head.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w12 {

constexpr int kChunk = 64;

// Operands of rows 16 rt .. and tokens 32 ks .. of a lower triangular 64 x 64 matrix: of those that are not all zero, the number.
__host__ __device__ constexpr int fragment_of(int rt, int ks) { return rt < 2 ? rt : 2 * rt - 2 + ks; }
constexpr int kFragments = 6;
// Its 16 x 16 blocks (r, s), r >= s.
__host__ __device__ constexpr int block_of(int r, int s) { return r * (r + 1) / 2 + s; }

// The workspace starts with a row of zeros, in place of tokens that are not there.
constexpr int kZeroBytes = 256;

// T = (I + A)^-1 diag(beta) as two BF16 matrices (each fragment 16 bytes a lane) and 256 words: e^G / |k| and e^(G_last - G) / |k|
// of the rows, e^G_last, and a bit for each row that is no number; then P's first BF16 matrix and scale e^G / |q|; then P's second.
constexpr int kFirstPages = 2 * kFragments + 1, kSecondPages = kFragments + 1;      // of 1 KB
constexpr int kTermsBytes = (kFirstPages + kSecondPages + kFragments) * 1024;
struct Terms {
  char* at;
  typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
  __device__ Terms(char* ws, int64_t i) : at(ws + i * kTermsBytes) {}
  __device__ bf8* t_high(int f) const { return reinterpret_cast<bf8*>(at + f * 1024); }
  __device__ bf8* t_low(int f) const { return t_high(kFragments + f); }
  __device__ float* rows() const { return reinterpret_cast<float*>(at + 2 * kFragments * 1024); }
  __device__ char* second() const { return at + kFirstPages * 1024; }
  __device__ bf8* p(int f) const { return reinterpret_cast<bf8*>(second() + f * 1024); }
  __device__ bf8* p_low(int f) const { return reinterpret_cast<bf8*>(second() + (kSecondPages + f) * 1024); }
  __device__ float* out_rows() const { return reinterpret_cast<float*>(second() + kFragments * 1024); }
};
// Words of rows().
constexpr int kTaken = 0, kLeft = 64, kGrown = 128, kBad = 130;

}  // namespace w12
