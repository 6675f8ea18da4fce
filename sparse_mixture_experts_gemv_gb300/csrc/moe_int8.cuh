// Device helpers of the 8-bit integer operators: loads by type, the quantization
// of a row, the stores of results.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_common.cuh"
#include "moe_layer.h"

namespace moe {
namespace int8 {

// 16 consecutive elements (16-byte aligned) as fp32.
template <int DT>
MOE_DEV void load16(const void* p, int64_t i, float (&v)[16]) {
  if constexpr (DT == MOE_DTYPE_F32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float4 f = __ldg(q + c);
      v[4 * c] = f.x; v[4 * c + 1] = f.y; v[4 * c + 2] = f.z; v[4 * c + 3] = f.w;
    }
  } else {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint4 u = __ldg(q + c);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (DT == MOE_DTYPE_BF16) {
          v[8 * c + 2 * j] = bf16_lo(w[j]);
          v[8 * c + 2 * j + 1] = bf16_hi(w[j]);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
          v[8 * c + 2 * j] = f.x;
          v[8 * c + 2 * j + 1] = f.y;
        }
      }
    }
  }
}
// The same for fp32 written earlier in this call (by a kernel this one may overlap).
MOE_DEV void load16_cg(const float* p, float (&v)[16]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint4 u = ldg_cg(p + 4 * c);
    v[4 * c] = __uint_as_float(u.x); v[4 * c + 1] = __uint_as_float(u.y);
    v[4 * c + 2] = __uint_as_float(u.z); v[4 * c + 3] = __uint_as_float(u.w);
  }
}

// max of the bit patterns of |v|: an infinity or a NaN stays above every finite
// value, so that a row's largest pattern also says whether the row is finite.
template <int N>
MOE_DEV uint32_t amax_bits(const float (&v)[N]) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) a = max(a, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return a;
}

// How a row is quantized, from amax_bits over it: the scale, its reciprocal, and
// whether the quotients need the division (scale below the normal range's middle,
// where the reciprocal overflows or loses bits). The scale is a product with the
// rounded 1/127, not the rounded quotient (4.7% of rows differ by a step): so does
// PyTorch divide a tensor on the GPU by a number, and a caller who quantizes with
// amax / 127 there has the same integers and scales as the call.
struct RowScale {
  float scale, inv;
};
MOE_DEV RowScale row_scale(uint32_t bits) {
  RowScale r;
  const float amax = __uint_as_float(bits);
  if (bits >= 0x7F800000u) r.scale = __uint_as_float(0x7FC00000u);   // NaN: the whole row
  else r.scale = bits ? amax * (1.f / 127.f) : 1.f;   // the constant rounded to fp32, then the product
  r.inv = r.scale >= 0x1p-100f ? 1.f / r.scale : 0.f;   // 0: divide (also for NaN)
  return r;
}

// x / scale to the nearest whole number, halves to the even one, decided on the real
// quotient: a row's half of the largest value is a tie but for the scale's rounding.
// The product with the reciprocal is off by less than 1e-5, and adding 3 * 2^22 rounds it
// to a whole number: at most one off, and only where the exact remainder x - q * scale
// (one rounding, far below what it is compared with) reaches half a scale. That is rare,
// so that the values of a chunk are looked at together.
constexpr float kRound = 12582912.f;
template <int N>
MOE_DEV void quantize(const float (&v)[N], const RowScale r, float (&q)[N]) {
  if (r.inv != 0.f) {
    const float half = 0.5f * r.scale;
    float worst = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      q[i] = fmaf(v[i], r.inv, kRound) - kRound;
      worst = fmaxf(worst, fabsf(fmaf(-q[i], r.scale, v[i])));
    }
    if (worst >= half) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float d = fmaf(-q[i], r.scale, v[i]);
        const bool odd = (int)q[i] & 1;
        if (d > half || (d == half && odd)) q[i] += 1.f;
        else if (d < -half || (d == -half && odd)) q[i] -= 1.f;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {   // 0 for a scale that underflowed, and for NaN
      const float t = r.scale > 0.f ? rintf(v[i] / r.scale) : 0.f;
      q[i] = fminf(fmaxf(t, -127.f), 127.f);
    }
  }
}

// The low byte of q + 3 * 2^22 is q's.
MOE_DEV uint32_t pack4(const float* q) {
  const uint32_t a = __float_as_uint(q[0] + kRound), b = __float_as_uint(q[1] + kRound),
                 c = __float_as_uint(q[2] + kRound), d = __float_as_uint(q[3] + kRound);
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
MOE_DEV uint4 quantize16(const float (&v)[16], const RowScale r) {
  float q[16];
  quantize(v, r, q);
  return make_uint4(pack4(q), pack4(q + 4), pack4(q + 8), pack4(q + 12));
}

MOE_DEV int dot16(const uint4 w, const uint4 x, int acc) {
  acc = __dp4a((int)w.x, (int)x.x, acc);
  acc = __dp4a((int)w.y, (int)x.y, acc);
  acc = __dp4a((int)w.z, (int)x.z, acc);
  return __dp4a((int)w.w, (int)x.w, acc);
}

// One value, rounded to nearest even (a NaN stays one).
MOE_DEV uint16_t to_16(int dtype, float f) {
  if (dtype == MOE_DTYPE_F16) return __half_as_ushort(__float2half_rn(f));
  return __bfloat16_as_ushort(__float2bfloat16_rn(f));
}
MOE_DEV void store(void* out, int dtype, int64_t i, float f) {
  if (dtype == MOE_DTYPE_F32) static_cast<float*>(out)[i] = f;
  else static_cast<uint16_t*>(out)[i] = to_16(dtype, f);
}

}  // namespace int8
}  // namespace moe
