// Sums over the lanes of a wave by moves between them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w12 {

// The sum of a wave's values up to each lane's.
template <int CTRL, int ROWS>
__device__ __forceinline__ double lanes_before(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, ROWS, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double sum_up(double v) {
  v += lanes_before<0x111, 0xF>(v);      // 1, 2, 4 and 8 lanes down, in rows of 16
  v += lanes_before<0x112, 0xF>(v);
  v += lanes_before<0x114, 0xF>(v);
  v += lanes_before<0x118, 0xF>(v);
  v += lanes_before<0x142, 0xA>(v);      // the last of the row below, into rows 1 and 3
  v += lanes_before<0x143, 0xC>(v);      // and of the lower half, into the upper
  return v;
}

}  // namespace w12
