// The gated delta rule, token by token: what the kernel for single tokens does, and the work-groups for short sequences of a call that has
// long ones too.
#pragma once

#include "w12_gemm_common.h"
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

// Sequence b's tokens, for 64 columns of head h, by a work-group; a sequence of more than `most` tokens is left.  Multiplications and additions
// are fused where it says so and nowhere else: two kernels have this code, and a sequence is to be the same in both.
template <int DK>
__device__ __forceinline__ void delta_steps(const w12_delta_args& a, const w12_sequences& s, int b, int h, int block, int most) {
#pragma clang fp contract(off)
  constexpr int L = DK / 8, P = 64 / L, PASSES = kWaveColumns / P;
  const int lane = threadIdx.x & 63, hk = h / (a.v_heads / a.k_heads);
  const int col = block * kGroupColumns + wave_id() * kWaveColumns + lane / L, piece = lane % L * 8;
  const Range r = range_of(s, b);
  if (r.n > most) return;
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
      kk = fmaf(k[e], k[e], kk);
      if (a.q) {
        qq = fmaf(q[e], q[e], qq);
        kq = fmaf(k[e], q[e], kq);
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
        sk = fmaf(st[p][e], k[e], sk);
        if (a.q) sq = fmaf(st[p][e], q[e], sq);
      }
      sk = lane_sum<L>(sk);
      const float u = t.beta * fmaf(-(grown * rk), sk, bf16_float(t.v[p])), ku = rk * u;
#pragma unroll
      for (int e = 0; e < 8; ++e) st[p][e] = fmaf(k[e], ku, grown * st[p][e]);
      if (a.q) {
        sq = lane_sum<L>(sq);
        const float o = rq * fmaf(grown, sq, kq * ku);
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

}  // namespace w12
