// Residual addition and RMS norm, with outputs in BF16 and / or in E4M3 with a scale per 128.
//
// r = residual + delta;  y = r / sqrt(mean(r^2) + eps) * weight;  scale_b = max|y| / 448 over a block.
// One work-group takes one row and keeps it in registers between the sum of squares and the
// outputs, so every value is read once and written once; the bound is memory traffic.  A lane
// holds V pieces of eight values; 16 neighbouring lanes hold a block of 128, whose largest
// magnitude they find among themselves.  4096 rows of 5120 from FP32 to FP32 and E4M3 (273 MB): 54 us, 5.1 TB/s (a plain
// copy: 4.7); up to 64 rows: 2.7 to 4.6 us in a call of 7.5 to 7.9.
#include "w12_gemm_common.h"
#include "w12_kernels.h"
#include "w12_rows.h"

namespace w12 {

constexpr int kNormMaxThreads = 1024;

__device__ __forceinline__ float wave_sum(float s) {
#pragma unroll
  for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o);
  return s;
}

template <int V, bool RF32, bool DF32>
__global__ __launch_bounds__(kNormMaxThreads) void k_add_rmsnorm(w12_norm_args a) {
  __shared__ float part[kNormMaxThreads / 64];
  const int64_t m = blockIdx.x;
  const int t = threadIdx.x, threads = blockDim.x, N = a.N;
  const char* res = static_cast<const char*>(a.residual) + m * a.ld_residual * (RF32 ? 4 : 2);
  const char* del = static_cast<const char*>(a.delta) + m * a.ld_delta * (DF32 ? 4 : 2);
  char* out = static_cast<char*>(a.residual_out) + m * a.ld_residual_out * (RF32 ? 4 : 2);
  float r[V][8];
  float ss = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = (t + j * threads) * 8;
    load8<RF32>(res, i, N, r[j]);
    if (a.delta) {
      float d[8];
      load8<DF32>(del, i, N, d);
#pragma unroll
      for (int e = 0; e < 8; ++e) r[j][e] += d[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) ss += r[j][e] * r[j][e];
    if (a.residual_out) store8<RF32>(out, i, N, r[j]);
  }
  ss = wave_sum(ss);
  if ((t & 63) == 0) part[t >> 6] = ss;
  __syncthreads();
  ss = 0.0f;
  for (int w = 0; w < threads / 64; ++w) ss += part[w];
  const float inv = 1.0f / sqrtf(ss / (float)N + a.eps);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = (t + j * threads) * 8;
    float w[8], y[8];
    load8<false>(a.weight, i, N, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = r[j][e] * inv * w[e];
    if (a.y) store8<false>(a.y + m * a.ldy, i, N, y);
    if (a.yq) {
      // magnitudes as integers order NaN above infinity above every number
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __builtin_bit_cast(uint32_t, y[e]) & 0x7FFFFFFFu);
#pragma unroll
      for (int o = 8; o; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
      const float amax = __builtin_bit_cast(float, top);
      // of a block of zeros, or one so small that the quotient leaves the subnormal range, 0: a scale of 1 rounds it to zeros
      const float least = amax / kE4M3Max;
      const float scale = least == 0.0f ? 1.0f : least;
      if ((t & 15) == 0 && i < N) a.yq_scale[m * a.ld_scale + i / W12_QUANT_BLOCK] = scale;
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] /= scale;
      store8_e4m3(a.yq + m * a.ldyq, i, N, y);
    }
  }
}

template <int V>
static void norm_types(const w12_norm_args& a, int threads, hipStream_t stream) {
  const dim3 g((unsigned)a.M), b((unsigned)threads);
  const bool rf = a.residual_dtype == W12_DTYPE_F32, df = a.delta && a.delta_dtype == W12_DTYPE_F32;
  if (rf && df) hipLaunchKernelGGL((k_add_rmsnorm<V, true, true>), g, b, 0, stream, a);
  else if (rf) hipLaunchKernelGGL((k_add_rmsnorm<V, true, false>), g, b, 0, stream, a);
  else if (df) hipLaunchKernelGGL((k_add_rmsnorm<V, false, true>), g, b, 0, stream, a);
  else hipLaunchKernelGGL((k_add_rmsnorm<V, false, false>), g, b, 0, stream, a);
}

hipError_t launch_add_rmsnorm(const w12_norm_args& a, hipStream_t stream) {
  const int pieces = (int)ceil_div(a.N, 8);
  int v = 1;
  while (pieces > v * kNormMaxThreads) v *= 2;
  const int threads = (int)ceil_div(ceil_div(pieces, v), 64) * 64;
  switch (v) {
    case 1: norm_types<1>(a, threads, stream); break;
    case 2: norm_types<2>(a, threads, stream); break;
    case 4: norm_types<4>(a, threads, stream); break;
    default: norm_types<8>(a, threads, stream); break;
  }
  return hipGetLastError();
}

}  // namespace w12
