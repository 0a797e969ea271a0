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
#include "w12_gemm_common.h"
#include "w12_kernels.h"
#include "w12_rows.h"
#include "w12_sequences.h"

namespace w12 {

constexpr int kDeltaThreads = 256;
constexpr int kWaveColumns = 16;
constexpr int kGroupColumns = kWaveColumns * kDeltaThreads / 64;

// The sum over the L lanes (8 or 16) that share a column; every lane gets it.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
template <int L>
__device__ __forceinline__ float lane_sum(float v) {
  v = dpp_add<0xB1>(v);       // lanes 1 away
  v = dpp_add<0x4E>(v);       // 2 away
  v = dpp_add<0x141>(v);      // the other four of eight
  if constexpr (L == 16) v = dpp_add<0x140>(v);   // the other eight
  return v;
}

// A token of one value head: this lane's piece of k and q, its columns' values, and the scalars, as they are in memory.
template <int PASSES>
struct Token {
  uint4 k, q;
  uint16_t v[PASSES];
  float g, beta;
};

template <int DK>
__global__ __launch_bounds__(kDeltaThreads) void k_delta_steps(w12_delta_args a, w12_sequences s) {
  constexpr int L = DK / 8, P = 64 / L, PASSES = kWaveColumns / P;
  const int lane = threadIdx.x & 63, h = blockIdx.y, hk = h / (a.v_heads / a.k_heads);
  const int col = blockIdx.z * kGroupColumns + wave_id() * kWaveColumns + lane / L, piece = lane % L * 8;
  const int b = blockIdx.x;
  const Range r = range_of(s, b);
  const int src = slot_of(s, s.src, b), dst = slot_of(s, s.dst, b);
  float st[PASSES][8];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    if (src >= 0) {
      const float4* at = reinterpret_cast<const float4*>(a.state + src * a.slot_stride + ((int64_t)h * a.dv + col + p * P) * DK + piece);
      const float4 x = at[0], y = at[1];
      st[p][0] = x.x; st[p][1] = x.y; st[p][2] = x.z; st[p][3] = x.w;
      st[p][4] = y.x; st[p][5] = y.y; st[p][6] = y.z; st[p][7] = y.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) st[p][e] = 0.0f;
    }
  }
  auto load = [&](int row, Token<PASSES>& t) {
    if (row < 0) {
      t.k = t.q = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int p = 0; p < PASSES; ++p) t.v[p] = 0;
      t.g = t.beta = 0.0f;
      return;
    }
    t.k = *reinterpret_cast<const uint4*>(a.k + row * a.ldk + hk * DK + piece);
    if (a.q) t.q = *reinterpret_cast<const uint4*>(a.q + row * a.ldq + hk * DK + piece);
#pragma unroll
    for (int p = 0; p < PASSES; ++p) t.v[p] = a.v[row * a.ldv + h * a.dv + col + p * P];
    t.g = a.g[row * a.ldg + h];
    t.beta = a.beta[row * a.ldbeta + h];
  };
  // a token's loads run beside the one before it, and its row's number beside the one before that
  Token<PASSES> next;
  int next_row = -1, row_after = -1;
  if (r.n > 0) {
    next_row = row_of(s, r.start);
    load(next_row, next);
  }
  if (r.n > 1) row_after = row_of(s, r.start + 1);
  for (int i = 0; i < r.n; ++i) {
    const int row = next_row;
    const Token<PASSES> t = next;
    if (i + 1 < r.n) {
      next_row = row_after;
      load(next_row, next);
      if (i + 2 < r.n) row_after = row_of(s, r.start + i + 2);
    }
    float k[8], q[8];
    unpack_bf16x8(t.k, k);
    if (a.q) unpack_bf16x8(t.q, q);
    float kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      kk += k[e] * k[e];
      if (a.q) {
        qq += q[e] * q[e];
        kq += k[e] * q[e];
      }
    }
    kk = lane_sum<L>(kk);
    float rk = 1.0f, rq = a.scale;
    // zeros that stand for no row stay zeros, with eps 0 too; a key whose squares are past FP32 is no number
    if (a.l2norm && row >= 0) rk = has_norm(kk + a.eps) ? 1.0f / sqrtf(kk + a.eps) : NAN;
    if (!(kk < INFINITY)) rk = NAN;
    if (a.q) {
      qq = lane_sum<L>(qq);
      kq = lane_sum<L>(kq);
      if (a.l2norm) rq *= has_norm(qq + a.eps) ? 1.0f / sqrtf(qq + a.eps) : NAN;
    }
    const float grown = expf(t.g);
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      float sk = 0.0f, sq = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sk += st[p][e] * k[e];
        if (a.q) sq += st[p][e] * q[e];
      }
      sk = lane_sum<L>(sk);
      const float u = t.beta * (bf16_float(t.v[p]) - grown * rk * sk);
#pragma unroll
      for (int e = 0; e < 8; ++e) st[p][e] = grown * st[p][e] + rk * k[e] * u;
      if (a.q) {
        sq = lane_sum<L>(sq);
        const float o = rq * (grown * sq + rk * kq * u);
        if (lane % L == 0 && row >= 0)
          a.out[row * a.ldo + h * a.dv + col + p * P] = (uint16_t)bf16_pair(o, o);
      }
    }
  }
  if (dst >= 0) {
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      float4* at = reinterpret_cast<float4*>(a.state + dst * a.slot_stride + ((int64_t)h * a.dv + col + p * P) * DK + piece);
      at[0] = make_float4(st[p][0], st[p][1], st[p][2], st[p][3]);
      at[1] = make_float4(st[p][4], st[p][5], st[p][6], st[p][7]);
    }
  }
}

// Tokens a sequence has, on average, from which they are taken 64 at a time: between 8 (48 heads of 128, 1 / 4 / 16 / 64 sequences: 14 / 19 /
// 42 / 144 us token by token, 16 / 25 / 56 / 200 in chunks) and 16 (25 / 31 / 67 / 226 and 16 / 25 / 57 / 205).  With lens the host does
// not know how many count; accepted paths are far shorter than the trees that they lead through.
static bool in_chunks(const w12_sequences& s) {
  return s.tree_mask || s.T >= (int64_t)(s.lens ? W12_DELTA_CHUNK_FROM_LENS : W12_DELTA_CHUNK_FROM) * s.count;
}

uint64_t gated_delta_workspace_bytes(int32_t T, int32_t count, int32_t v_heads, int32_t dk, int32_t dv) {
  return delta_chunk_workspace_bytes(T, count, v_heads);
}
uint64_t gated_delta_call_bytes(const w12_sequences& s, int32_t v_heads) {
  return in_chunks(s) ? delta_chunk_workspace_bytes(s.T, s.count, v_heads) : 0;
}

hipError_t launch_gated_delta(const w12_delta_args& a, const w12_sequences& s, void* ws, hipStream_t stream) {
  if (in_chunks(s)) return launch_delta_chunks(a, s, ws, stream);
  const dim3 grid((unsigned)s.count, (unsigned)a.v_heads, (unsigned)(a.dv / kGroupColumns));
  if (a.dk == 64) k_delta_steps<64><<<grid, kDeltaThreads, 0, stream>>>(a, s);
  else k_delta_steps<128><<<grid, kDeltaThreads, 0, stream>>>(a, s);
  return hipGetLastError();
}

}  // namespace w12
