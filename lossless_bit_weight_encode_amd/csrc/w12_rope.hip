// Rotary positions and the write into the paged cache.
//
// Pair i of a head turns by theta = positions[axis(i)][t] * inv_freq[i]:
//   (a, b) -> (a cos theta - b sin theta, a sin theta + b cos theta).
// The angle is formed in FP64 as a number of turns and reduced there to half a turn either way,
// so a far position loses nothing; its sine and cosine are FP32.
#include "w12_gemm_common.h"
#include "w12_kernels.h"
#include "w12_rows.h"

namespace w12 {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = 128;

__device__ __forceinline__ float rope_src(const w12_rope_args& a, int64_t row, int i) {
  if (a.src_dtype == W12_DTYPE_F32) return static_cast<const float*>(a.qkv)[row * a.ld_qkv + i];
  return bf16_float(static_cast<const uint16_t*>(a.qkv)[row * a.ld_qkv + i]);
}

__global__ __launch_bounds__(kRopeThreads) void k_rope_append(w12_rope_args a, w12_kv_cache c) {
  __shared__ float cs[kRopeMaxPairs], sn[kRopeMaxPairs];
  const int64_t t = blockIdx.x;
  const int half = a.rot_dim / 2, D = c.dim;
  for (int i = threadIdx.x; i < half; i += kRopeThreads) {
    const int ax = a.axis ? min((int)a.axis[i], a.axes - 1) : 0;
    const double turns = (double)a.positions[ax * a.ld_positions + t] * a.inv_freq[i] * 0.15915494309189533577;
    const float x = (float)(2.0 * (turns - rint(turns)));
    sincospif(x, &sn[i], &cs[i]);
  }
  __syncthreads();
  const int64_t slot = a.slots[t];
  const bool put = slot >= 0 && slot / c.page_size < c.pages;
  const int64_t base = put ? slot / c.page_size * c.page_stride + slot % c.page_size * c.token_stride : 0;
  const int total = (a.q_heads + 2 * c.heads) * D;
  for (int i = threadIdx.x; i < total; i += kRopeThreads) {
    const int h = i / D, e = i % D;
    float v = rope_src(a, t, i);
    if (h < a.q_heads + c.heads && e < a.rot_dim) {
      const int pair = a.adjacent ? e / 2 : e % half;
      const bool second = a.adjacent ? e & 1 : e >= half;
      const float o = rope_src(a, t, i + (a.adjacent ? (second ? -1 : 1) : (second ? -half : half)));
      v = second ? o * sn[pair] + v * cs[pair] : v * cs[pair] - o * sn[pair];
    }
    if (h < a.q_heads) {
      a.q[t * a.ldq + i] = (uint16_t)bf16_pair(v, v);
    } else if (put) {
      const int kv = h - a.q_heads;
      const bool is_v = kv >= c.heads;
      const int hh = is_v ? kv - c.heads : kv;
      const int64_t at = base + hh * c.head_stride + e;
      void* dst = is_v ? c.v : c.k;
      if (c.dtype == W12_DTYPE_BF16) {
        static_cast<uint16_t*>(dst)[at] = (uint16_t)bf16_pair(v, v);
      } else {
        v /= (is_v ? c.v_scale : c.k_scale)[hh];
        static_cast<uint8_t*>(dst)[at] = (uint8_t)e4m3_quad(v, v, v, v);
      }
    }
  }
}

hipError_t launch_rope_append(const w12_rope_args& a, const w12_kv_cache& c, hipStream_t stream) {
  hipLaunchKernelGGL(k_rope_append, dim3((unsigned)a.T), dim3(kRopeThreads), 0, stream, a, c);
  return hipGetLastError();
}

}  // namespace w12
