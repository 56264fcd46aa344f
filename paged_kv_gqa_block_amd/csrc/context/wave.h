// Sums and maxima over the 64 lanes of a wave, by moves between lanes (DPP).
#pragma once

#include "device_common.h"

namespace pkv {

constexpr int kDppRowShr = 0x110;      // + k: from the lane k below, in rows of 16
constexpr int kDppRowBcast15 = 0x142;  // a row's last lane to the next row
constexpr int kDppRowBcast31 = 0x143;  // lane 31 to the upper half

// x of the lane that CTRL names, 0 where there is none; rows outside ROWS get 0.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ int moved(int x) {
  return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, false);
}

// Inclusive sum.
__device__ __forceinline__ int wave_scan(int x) {
  x += moved<kDppRowShr + 1>(x);
  x += moved<kDppRowShr + 2>(x);
  x += moved<kDppRowShr + 4>(x);
  x += moved<kDppRowShr + 8>(x);
  x += moved<kDppRowBcast15, 0xa>(x);
  x += moved<kDppRowBcast31, 0xc>(x);
  return x;
}

// Maximum of x >= 0, in every lane.
__device__ __forceinline__ int wave_max(int x) {
  x = max(x, moved<kDppRowShr + 1>(x));
  x = max(x, moved<kDppRowShr + 2>(x));
  x = max(x, moved<kDppRowShr + 4>(x));
  x = max(x, moved<kDppRowShr + 8>(x));
  x = max(x, moved<kDppRowBcast15, 0xa>(x));
  x = max(x, moved<kDppRowBcast31, 0xc>(x));
  return __builtin_amdgcn_readlane(x, 63);
}

}  // namespace pkv
