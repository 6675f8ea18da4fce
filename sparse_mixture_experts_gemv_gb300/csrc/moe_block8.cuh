// Device helpers of the 8-bit floating-point operators: a block of 128 values, sixteen in each of eight neighbouring
// lanes, to its scale and E4M3.
#pragma once

#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_int8.cuh"

namespace moe {
namespace block8 {

// The quotients of 16 values of a block by its scale, rounded to the nearest fp32 each: the product with the correctly
// rounded reciprocal is off by two steps at most, one correction by its exact remainder by less than one, and from
// there a second one is the rounded quotient (Markstein, IBM Journal of Research and Development 34, 1990). Remainders
// are exact while nothing leaves the normal range: scales beyond 2^+-90 (or NaN) take the division. Values below 2^-10
// of the scale, whose remainder may, are 0 in E4M3 either way. The remainder is q scale - v, and its
// correction taken off: where it is 0, that adds -0, and a quotient of -0 stays one.
MOE_DEV void divide(float (&v)[16], float scale) {
  if (scale >= 0x1p-90f && scale <= 0x1p90f) {
    const float inv = 1.f / scale;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float q = v[i] * inv;
      q = fmaf(-fmaf(q, scale, -v[i]), inv, q);
      v[i] = fmaf(-fmaf(q, scale, -v[i]), inv, q);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __fdiv_rn(v[i], scale);
  }
}

// The larger of two magnitudes; NaN if one of them is.
MOE_DEV float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// The block's scale, by all lanes of the warp.
MOE_DEV float block_scale(const float (&v)[16]) {
  float top = fabsf(v[0]);
#pragma unroll
  for (int j = 1; j < 16; ++j) top = max_nan(top, fabsf(v[j]));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  const float scale = top * (1.f / 448.f);
  if (!(top <= 3.402823466e38f)) return __uint_as_float(0x7FC00000u);
  return scale == 0.f ? 1.f : scale;
}
MOE_DEV uint4 to_e4m3(float (&v)[16], float scale) {
  divide(v, scale);
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * j], v[4 * j + 1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * j + 2], v[4 * j + 3]), __NV_SATFINITE, __NV_E4M3);
    w[j] = lo | hi << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace block8
}  // namespace moe
