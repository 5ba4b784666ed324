// Reductions over a wavefront and over a workgroup, in a fixed order.
#pragma once

#include "wave.h"

namespace skg {

// The larger of two, NaN if either is (v_maximum3_f32, as quick as v_max3_f32).
__device__ __forceinline__ float max_or_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

template <int OFF>
__device__ __forceinline__ float xred_max(float v) {
  if constexpr (OFF >= 16) {
    int x = __float_as_int(v);
    auto p = (OFF == 32) ? __builtin_amdgcn_permlane32_swap(x, x, false, false)
                         : __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return max_or_nan(__int_as_float(p[0]), __int_as_float(p[1]));
  } else {
    return max_or_nan(v, __int_as_float(xshfl_dpp<OFF>(__float_as_int(v))));
  }
}

// The largest of a wave's 64 values, in every lane (NaN if one is).
__device__ __forceinline__ float butterfly_max(float v) {
  v = xred_max<32>(v);
  v = xred_max<16>(v);
  v = xred_max<8>(v);
  v = xred_max<4>(v);
  v = xred_max<2>(v);
  v = xred_max<1>(v);
  return v;
}

// The largest of a wave's 64 unsigned values, in every lane.
template <int OFF>
__device__ __forceinline__ uint32_t xred_umax(uint32_t v) {
  if constexpr (OFF >= 16) {
    auto p = (OFF == 32) ? __builtin_amdgcn_permlane32_swap((int)v, (int)v, false, false)
                         : __builtin_amdgcn_permlane16_swap((int)v, (int)v, false, false);
    return max((uint32_t)p[0], (uint32_t)p[1]);
  } else {
    return max(v, (uint32_t)xshfl_dpp<OFF>((int)v));
  }
}
__device__ __forceinline__ uint32_t butterfly_umax(uint32_t v) {
  v = xred_umax<32>(v);
  v = xred_umax<16>(v);
  v = xred_umax<8>(v);
  v = xred_umax<4>(v);
  v = xred_umax<2>(v);
  return xred_umax<1>(v);
}

// The sum of `a` and the largest `b` (NaN if one is) over a workgroup of up to 16
// waves, in every thread. `part` holds 32 floats of LDS that nobody else uses until the
// next barrier after this call.
__device__ __forceinline__ void block_sum_max(float& a, float& b, float* part) {
  a = butterfly_sum(a);
  b = butterfly_max(b);
  const int waves = (int)(blockDim.x >> 6);
  if (waves == 1) return;
  const int wave = (int)(threadIdx.x >> 6);
  if ((threadIdx.x & 63) == 0) {
    part[wave] = a;
    part[16 + wave] = b;
  }
  __syncthreads();
  a = part[0];
  b = part[16];
  for (int i = 1; i < waves; ++i) {
    a += part[i];
    b = max_or_nan(b, part[16 + i]);
  }
}

}  // namespace skg
