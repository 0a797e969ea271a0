// Rotary positions and the write into the paged cache.
//
// Pair i of a head turns by theta = positions[axis(i)][t] * inv_freq[i]:
//   (a, b) -> (a cos theta - b sin theta, a sin theta + b cos theta).
// The angle is formed in FP64 as a number of turns and reduced there to half a turn either way,
// so a far position loses nothing; its sine and cosine are FP32.  Bound: the launch, then positions -> sines -> the
// turn one after another (512 rows of 56 heads of 128 into an E4M3 cache, 21 MB: 7.7 us; 4096 into a BF16 one, 176 MB:
// 37.6, 4.7 TB/s, a copy's rate; one row: 2.7, in a call of 7.7).
#include "w12_gemm_common.h"
#include "w12_kernels.h"
#include "w12_rows.h"

namespace w12 {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = 128;

// One work-group takes `heads` of a row's heads (of Q, then K, then V), a thread 8 neighbouring values at a time:
// with PIECES, pairs lie 8 by 8 (or, adjacent, inside a piece), so a thread turns a piece with its
// partner's, read beside it (the two threads of a pair read the same lines); otherwise value by value.
// The loads start before the sines, which wait for positions and frequencies.
template <bool F32, bool PIECES>
__global__ __launch_bounds__(kRopeThreads) void k_rope_append(w12_rope_args a, w12_kv_cache c, int heads, int dim_bits) {
  __shared__ float cs[kRopeMaxPairs], sn[kRopeMaxPairs];
  const int64_t t = blockIdx.x;
  const int half = a.rot_dim / 2, D = 1 << dim_bits, all = a.q_heads + 2 * c.heads;
  const int h0 = blockIdx.y * heads, pieces = min(heads, all - h0) << (dim_bits - 3);
  const char* src = static_cast<const char*>(a.qkv) + t * a.ld_qkv * (F32 ? 4 : 2);
  const int64_t slot = a.slots[t];
  int p = threadIdx.x;
  float x[8], y[8];
  // piece p and the piece that holds its partners (the same piece where there are none)
  auto load = [&](int i) {
    const int h = h0 + (i >> (dim_bits - 3)), e = (i & (D / 8 - 1)) * 8, at = (h << dim_bits) + e;
    const bool turned = PIECES && h < a.q_heads + c.heads && e < a.rot_dim && !a.adjacent;
    load8<F32>(src, at, 1 << 30, x);
    load8<F32>(src, turned ? (e < half ? at + half : at - half) : at, 1 << 30, y);
  };
  if (p < pieces) load(p);
  for (int i = threadIdx.x; i < half; i += kRopeThreads) {
    const int ax = a.axis ? min((int)a.axis[i], a.axes - 1) : 0;
    const double turns = (double)a.positions[ax * a.ld_positions + t] * a.inv_freq[i] * 0.15915494309189533577;
    sincospif((float)(2.0 * (turns - rint(turns))), &sn[i], &cs[i]);
  }
  __syncthreads();
  const int page_bits = 31 - __builtin_clz(c.page_size);
  const bool put = slot >= 0 && (slot >> page_bits) < c.pages;
  const int64_t base = put ? (slot >> page_bits) * c.page_stride + (slot & (c.page_size - 1)) * c.token_stride : 0;
  for (; p < pieces; p += kRopeThreads) {
    if (p != (int)threadIdx.x) load(p);
    const int h = h0 + (p >> (dim_bits - 3)), e = (p & (D / 8 - 1)) * 8;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = x[i];
    if (h < a.q_heads + c.heads && e < a.rot_dim) {
      if constexpr (PIECES) {
        if (a.adjacent) {
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float co = cs[(e + i) / 2], si = sn[(e + i) / 2];
            v[i] = x[i] * co - x[i + 1] * si;
            v[i + 1] = x[i] * si + x[i + 1] * co;
          }
        } else {
          const int pair = e < half ? e : e - half;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float co = cs[pair + i], si = sn[pair + i];
            v[i] = e < half ? x[i] * co - y[i] * si : y[i] * si + x[i] * co;
          }
        }
      } else {
        const int at = h << dim_bits;
        for (int i = 0; i < 8 && e + i < a.rot_dim; ++i) {
          const int k = e + i;
          const bool second = a.adjacent ? k & 1 : k >= half;
          const int pair = a.adjacent ? k / 2 : second ? k - half : k;
          const int other = at + (a.adjacent ? k ^ 1 : second ? k - half : k + half);
          const float o = F32 ? reinterpret_cast<const float*>(src)[other] : bf16_float(reinterpret_cast<const uint16_t*>(src)[other]);
          v[i] = second ? o * sn[pair] + v[i] * cs[pair] : v[i] * cs[pair] - o * sn[pair];
        }
      }
    }
    if (h < a.q_heads) {
      store8<false>(a.q + t * a.ldq, (h << dim_bits) + e, 1 << 30, v);
    } else if (put) {
      const bool is_v = h >= a.q_heads + c.heads;
      const int hh = h - a.q_heads - (is_v ? c.heads : 0);
      const int64_t at = base + hh * c.head_stride + e;
      void* dst = is_v ? c.v : c.k;
      if (c.dtype == W12_DTYPE_BF16) {
        store8<false>(static_cast<uint16_t*>(dst) + at, 0, 8, v);
      } else {
        const float scale = (is_v ? c.v_scale : c.k_scale)[hh];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] /= scale;
        store8_e4m3(static_cast<uint8_t*>(dst) + at, 0, 8, v);
      }
    }
  }
}

hipError_t launch_rope_append(const w12_rope_args& a, const w12_kv_cache& c, hipStream_t stream) {
  const int dim_bits = 31 - __builtin_clz(c.dim), all = a.q_heads + 2 * c.heads;
  // pieces of a row over as many work-groups as leave each thread one piece, up to two rows a compute unit (us of 56 heads
  // of 128, split / whole: 64 rows 3.3 / 5.3, 256 rows 4.7 / 6.0, 512 rows 8.0 / 9.9, 1024 rows 12.8 / 12.5, 4096 rows 38.4 / 37.7)
  const int64_t pieces = (int64_t)all << (dim_bits - 3);
  const int64_t groups = a.T >= 2 * device_cus() ? 1 : ceil_div(pieces, kRopeThreads);
  const int heads = (int)ceil_div(all, groups);
  const dim3 g((unsigned)a.T, (unsigned)ceil_div(all, heads)), b(kRopeThreads);
  const bool f32 = a.src_dtype == W12_DTYPE_F32;
  // pairs of whole pieces: both halves (or, adjacent, the part that turns) end where pieces do
  if (a.rot_dim % (a.adjacent ? 8 : 16) == 0) {
    if (f32) hipLaunchKernelGGL((k_rope_append<true, true>), g, b, 0, stream, a, c, heads, dim_bits);
    else hipLaunchKernelGGL((k_rope_append<false, true>), g, b, 0, stream, a, c, heads, dim_bits);
  } else {
    if (f32) hipLaunchKernelGGL((k_rope_append<true, false>), g, b, 0, stream, a, c, heads, dim_bits);
    else hipLaunchKernelGGL((k_rope_append<false, false>), g, b, 0, stream, a, c, heads, dim_bits);
  }
  return hipGetLastError();
}

}  // namespace w12
