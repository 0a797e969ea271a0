// Row vectors shared by the operators around the products: eight neighbouring values of a row are
// one lane's piece (16 bytes of BF16, 32 of FP32, 8 of E4M3), with conversions that round once.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w12 {

constexpr float kE4M3Max = 448.0f;

__device__ __forceinline__ float bf16_float(uint32_t bits) { return __builtin_bit_cast(float, bits << 16); }
// Two floats to BF16 pairs, to nearest even (one instruction; NaN stays NaN).
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef __bf16 v2 __attribute__((ext_vector_type(2)));
  v2 r;
  r[0] = (__bf16)a;
  r[1] = (__bf16)b;
  return __builtin_bit_cast(uint32_t, r);
}

// Cut off at the largest E4M3 value, which the conversion instruction does not do; NaN passes.
__device__ __forceinline__ float e4m3_clamp(float v) {
  v = v > kE4M3Max ? kE4M3Max : v;
  return v < -kE4M3Max ? -kE4M3Max : v;
}
// Four floats to E4M3 bytes, to nearest even.
__device__ __forceinline__ uint32_t e4m3_quad(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_clamp(a), e4m3_clamp(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(e4m3_clamp(c), e4m3_clamp(d), r, true);
}

__device__ __forceinline__ void unpack_bf16x8(uint4 u, float v[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_float(w[i]);
    v[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
  }
}

// Values i .. i + 7 of a row of n (zeros past n; the row is 16-byte aligned and i a multiple of 8).
template <bool F32>
__device__ __forceinline__ void load8(const void* row, int i, int n, float v[8]) {
  if (i + 8 <= n) {
    if constexpr (F32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(row) + i);
      const float4 a = p[0], b = p[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      unpack_bf16x8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + i), v);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = 0.0f;
      if (i + j < n) {
        if constexpr (F32) v[j] = static_cast<const float*>(row)[i + j];
        else v[j] = bf16_float(static_cast<const uint16_t*>(row)[i + j]);
      }
    }
  }
}

template <bool F32>
__device__ __forceinline__ void store8(void* row, int i, int n, const float v[8]) {
  if (i + 8 <= n) {
    if constexpr (F32) {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(row) + i);
      p[0] = make_float4(v[0], v[1], v[2], v[3]);
      p[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(row) + i) =
          make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) {
        if constexpr (F32) static_cast<float*>(row)[i + j] = v[j];
        else static_cast<uint16_t*>(row)[i + j] = (uint16_t)bf16_pair(v[j], v[j]);
      }
  }
}

__device__ __forceinline__ void store8_e4m3(uint8_t* row, int i, int n, const float v[8]) {
  const uint32_t lo = e4m3_quad(v[0], v[1], v[2], v[3]), hi = e4m3_quad(v[4], v[5], v[6], v[7]);
  if (i + 8 <= n) {
    *reinterpret_cast<uint2*>(row + i) = make_uint2(lo, hi);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) row[i + j] = (uint8_t)((j < 4 ? lo : hi) >> (8 * (j & 3)));
  }
}

}  // namespace w12
