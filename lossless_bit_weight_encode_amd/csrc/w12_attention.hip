// Attention of drafted tokens over a paged cache.
//
// One work-group takes one row and query head.  It goes over the tokens in tiles of 256 with the
// running maximum m and sum l of the softmax: scores of a tile (one token a thread), then
// l = l e^(m - m') + sum p, o = o e^(m - m') + sum p v (one element of the head a thread).
#include "w12_gemm_common.h"
#include "w12_kernels.h"
#include "w12_rows.h"

namespace w12 {

constexpr int kAttnThreads = 256;

template <bool E4M3>
__device__ __forceinline__ float cache_at(const void* p, int64_t i) {
  if constexpr (E4M3) return __builtin_amdgcn_cvt_f32_fp8((int)static_cast<const uint8_t*>(p)[i], 0);
  else return bf16_float(static_cast<const uint16_t*>(p)[i]);
}

template <bool E4M3>
__global__ __launch_bounds__(kAttnThreads) void k_tree_attention(w12_attention_args a, w12_kv_cache c) {
  __shared__ float q[256], p[kAttnThreads], red[4];
  __shared__ int64_t at[kAttnThreads];
  const int64_t row = blockIdx.x;
  const int h = blockIdx.y, D = c.dim, t = threadIdx.x, kvh = h / (a.q_heads / c.heads);
  // the row's request: the last one that starts at or before it
  int b = 0, start = 0, end = 0;
  for (b = 0; b < a.requests; ++b) {
    start = min(max(a.node_ptr[b], 0), a.T);
    end = min(max(a.node_ptr[b + 1], start), a.T);
    if (row >= start && row < end) break;
  }
  if (b == a.requests) return;
  const int node = (int)row - start;
  const int ctx = (int)min((int64_t)max(a.ctx_len[b], 0), (int64_t)a.max_pages * c.page_size);
  const int len = (int)min((int64_t)ctx + end - start, (int64_t)a.max_pages * c.page_size);
  if (t < D) q[t] = bf16_float(a.q[row * a.ldq + h * D + t]);
  const float scale = a.scale * 1.4426950408889634f * (E4M3 ? c.k_scale[kvh] : 1.0f);
  float m = -INFINITY, l = 0.0f, o = 0.0f;
  for (int t0 = 0; t0 < len; t0 += kAttnThreads) {
    const int j = t0 + t;
    bool sees = j < len;
    int64_t where = -1;
    if (sees && j >= ctx) {
      const int n = j - ctx;
      sees = a.tree_mask ? (n < 64 * a.mask_words && (a.tree_mask[row * a.ld_mask + n / 64] >> (n % 64) & 1)) : n <= node;
    }
    if (sees) {
      const int page = a.page_table[b * a.ld_table + j / c.page_size];
      sees = page >= 0 && page < c.pages;
      where = (int64_t)page * c.page_stride + (int64_t)(j % c.page_size) * c.token_stride + (int64_t)kvh * c.head_stride;
    }
    __syncthreads();
    float s = -INFINITY;
    if (sees) {
      s = 0.0f;
      for (int e = 0; e < D; ++e) s += q[e] * cache_at<E4M3>(c.k, where + e);
      s *= scale;
    }
    at[t] = sees ? where : -1;
    float top = s;
#pragma unroll
    for (int x = 32; x; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
    if ((t & 63) == 0) red[t >> 6] = top;
    __syncthreads();
    const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float base = mn == -INFINITY ? 0.0f : mn, corr = exp2f(m - base);
    p[t] = exp2f(s - base);
    __syncthreads();
    l *= corr;
    o *= corr;
    m = mn;
    for (int x = 0; x < min(kAttnThreads, len - t0); ++x) {
      if (at[x] < 0) continue;
      l += p[x];
      if (t < D) o += p[x] * cache_at<E4M3>(c.v, at[x] + t);
    }
  }
  if (t < D) {
    const float v = l == 0.0f ? 0.0f : o * (E4M3 ? c.v_scale[kvh] : 1.0f) / l;
    a.out[row * a.ldo + h * D + t] = (uint16_t)bf16_pair(v, v);
  }
  if (a.lse && t == 0) a.lse[row * a.ld_lse + h] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

uint64_t attention_workspace_bytes(int32_t, int32_t, int32_t, const w12_kv_cache&) { return 0; }

hipError_t launch_tree_attention(const w12_attention_args& a, const w12_kv_cache& c, void*, hipStream_t stream) {
  const dim3 g((unsigned)a.T, (unsigned)a.q_heads), b(kAttnThreads);
  if (c.dtype == W12_DTYPE_E4M3) hipLaunchKernelGGL(k_tree_attention<true>, g, b, 0, stream, a, c);
  else hipLaunchKernelGGL(k_tree_attention<false>, g, b, 0, stream, a, c);
  return hipGetLastError();
}

}  // namespace w12
