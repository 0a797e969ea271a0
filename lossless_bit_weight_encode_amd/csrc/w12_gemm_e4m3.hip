// The 8-bit product with block scales: Y = (X sx) (W sw)^T, E4M3 operands, FP32 sums.
//
// One wave takes 16 channels x 16 rows of X and goes over k in blocks of 128: four 16x16x32
// matrix instructions sum a block, whose result is scaled and added in FP32.  The operands become
// BF16 (which holds every E4M3 value): the 8-bit matrix instructions line up the products of eight
// neighbouring k with the largest and drop what is below 2^-13 of it (measured), so they do not
// hold a sum in 32 bits; the BF16 ones do.
#include "w12_device.h"
#include "w12_gemm_common.h"
#include "w12_kernels.h"

namespace w12 {

// Bytes k .. k + 7 of a row of K (zeros past K; the row is 16-byte aligned, k a multiple of 8).
__device__ __forceinline__ long load_k8(const uint8_t* row, int k, int K) {
  if (k + 8 <= K) return *reinterpret_cast<const long*>(row + k);
  unsigned long v = 0;
  for (int j = 0; j < 8; ++j)
    if (k + j < K) v |= (unsigned long)row[k + j] << (8 * j);
  return (long)v;
}

// Eight E4M3 bytes to BF16.
__device__ __forceinline__ bf16x8 e4m3_bf16x8(long v) {
  const uint32_t w[2] = {(uint32_t)(unsigned long)v, (uint32_t)((unsigned long)v >> 32)};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, false));
    r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, true));
  }
  return __builtin_bit_cast(bf16x8, make_uint4(r[0], r[1], r[2], r[3]));
}

__global__ __launch_bounds__(64) void k_gemm_e4m3(const uint8_t* X, int M, int64_t ldx, const float* xs, int64_t ldxs,
                                                  const uint8_t* W, int N, int K, int64_t ldw, const float* wsc,
                                                  int64_t ldws, float* Y, int64_t ldy) {
  const int lane = threadIdx.x, r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16;
  const int n = min(n0 + r, N - 1), m = min(m0 + r, M - 1);
  const uint8_t* w = W + (int64_t)n * ldw;
  const uint8_t* x = X + (int64_t)m * ldx;
  f32x4 sum = {0, 0, 0, 0};
  for (int k0 = 0; k0 < K; k0 += 128) {
    f32x4 part = {0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int k = k0 + s * 32 + q * 8;
      part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(e4m3_bf16x8(load_k8(w, k, K)), e4m3_bf16x8(load_k8(x, k, K)), part, 0, 0, 0);
    }
    sum += part * (xs[m * ldxs + k0 / 128] * wsc[(n0 / 128) * ldws + k0 / 128]);
  }
  if (m0 + r < M)
    for (int i = 0; i < 4; ++i)
      if (n0 + q * 4 + i < N) Y[(m0 + r) * ldy + n0 + q * 4 + i] = sum[i];
}

uint64_t gemm_e4m3_workspace_bytes(int32_t, int32_t, int32_t) { return 0; }

hipError_t launch_gemm_e4m3(const uint8_t* X, int32_t M, int64_t ldx, const float* xs, int64_t ldxs, const uint8_t* W,
                            int32_t N, int32_t K, int64_t ldw, const float* wsc, int64_t ldws, float* Y, int64_t ldy,
                            void*, hipStream_t stream) {
  const dim3 g((unsigned)ceil_div(N, 16), (unsigned)ceil_div(M, 16));
  hipLaunchKernelGGL(k_gemm_e4m3, g, dim3(64), 0, stream, X, M, ldx, xs, ldxs, W, N, K, ldw, wsc, ldws, Y, ldy);
  return hipGetLastError();
}

}  // namespace w12
