// attend.cuh -- what the attention kernels over the paged 8-bit cache share.
#pragma once

#include "kv.cuh"

namespace qmv {

// 2^x (ex2.approx: 2 ulp over the range; 2^-inf = 0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;

}  // namespace qmv
