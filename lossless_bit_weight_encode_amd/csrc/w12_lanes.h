// Sums and extremes over the lanes of a wave by moves between them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w12 {

template <int V>
struct Const {
  static constexpr int value = V;
};

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

// f over all lanes' values, for every lane; f(x, x) has to be x.
template <typename T, typename F>
__device__ __forceinline__ T over_wave(T v, F f) {
  const auto with = [&](auto ctrl, auto rows) {
    const int i = __builtin_bit_cast(int, v);
    v = f(v, __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(i, i, decltype(ctrl)::value, decltype(rows)::value, 0xF, false)));
  };
  with(Const<0x111>{}, Const<0xF>{});      // as in sum_up
  with(Const<0x112>{}, Const<0xF>{});
  with(Const<0x114>{}, Const<0xF>{});
  with(Const<0x118>{}, Const<0xF>{});
  with(Const<0x142>{}, Const<0xA>{});
  with(Const<0x143>{}, Const<0xC>{});
  return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}
// f over 16 neighbouring lanes' values (of 4 bytes or 8), for each of them.
template <typename T, typename F>
__device__ __forceinline__ T over_row(T v, F f) {
  const auto with = [&](auto ctrl) {
    T other;
    if constexpr (sizeof(T) == 8) {
      const uint64_t u = __builtin_bit_cast(uint64_t, v);
      const uint32_t lo = __builtin_amdgcn_mov_dpp((int)(uint32_t)u, decltype(ctrl)::value, 0xF, 0xF, true);
      const uint32_t hi = __builtin_amdgcn_mov_dpp((int)(u >> 32), decltype(ctrl)::value, 0xF, 0xF, true);
      other = __builtin_bit_cast(T, (uint64_t)hi << 32 | lo);
    } else {
      other = __builtin_bit_cast(T, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), decltype(ctrl)::value, 0xF, 0xF, true));
    }
    v = f(v, other);
  };
  with(Const<0xB1>{});       // lanes 1 away
  with(Const<0x4E>{});       // 2 away
  with(Const<0x141>{});      // the other four of eight
  with(Const<0x140>{});      // the other eight
  return v;
}

}  // namespace w12
