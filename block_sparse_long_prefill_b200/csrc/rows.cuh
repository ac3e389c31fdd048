// rows.cuh -- rows of D bf16 values spread over lanes, 8 values (16 bytes) a lane.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace moba {

constexpr uint32_t kFull = 0xffffffffu;

// Lanes of a row and rows of a warp (d = 80: 3 rows of 10 lanes, two lanes idle).
template <int D>
struct RowLanes {
  static constexpr int LPR = D / 8;
  static constexpr int RPW = 32 / LPR;
};

// Sum over the row's lanes, the same in each of them.  base: the row's first lane.
template <int D>
__device__ __forceinline__ float row_sum(float x, int base, int v) {
  constexpr int LPR = RowLanes<D>::LPR;
  if constexpr ((LPR & (LPR - 1)) == 0) {
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) x += __shfl_xor_sync(kFull, x, o);
    return x;
  } else {
    // 10 lanes: lanes v and v + 5 add up, then the five sums in one order.
    const int half = LPR / 2;
    const float t = x + __shfl_sync(kFull, x, base + (v + half) % LPR);
    float s = __shfl_sync(kFull, t, base);
#pragma unroll
    for (int o = 1; o < half; ++o) s += __shfl_sync(kFull, t, base + o);
    return s;
  }
}

__device__ __forceinline__ void unpack8(const uint4 &a, float (&x)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(w[e] << 16);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}

}  // namespace moba
