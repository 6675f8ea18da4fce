// Routing to experts from given logits, and its gradient.
//
//   s[e]   = softmax(l)[e] or 1 / (1 + exp(-l[e]))
//   key[e] = s[e] + bias[e]                          (the bias only chooses)
//   group g's score = the sum of its `group_top` largest keys; the `top_groups`
//   groups of the largest scores stay, equal ones by index
//   idx    = the k largest keys of the groups that stay, descending, equal ones by index
//   w[j]   = scale * s[idx[j]] (/ sum_i s[idx[i]])
// A logit of -inf or NaN turns its expert off for the token: it ranks below every
// expert that is on, and its weight is 0; +inf counts as the largest finite value.
//
// One warp serves one token; lane l holds the NPL consecutive experts l * NPL ...
// so that a row is read with 16-byte loads, a lower lane means a lower index, and
// (for the usual group sizes) a group is a run of whole lanes.
//
// Which experts are chosen must not depend on how a score was rounded. Without a
// bias and groups the keys are the logits themselves (both scores increase with
// the logit), so the choice is exact. Otherwise scores are computed in 32 bits,
// and a choice is kept only if the keys it separates are further apart than the
// 32-bit errors can reach; a token with a closer pair is decided again with all
// its scores in 64 bits.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kRouteWarps = 4;

struct RouteParams {
  const void* logits;
  const float* bias;
  int64_t stride;   // elements between rows
  int T, E, k, groups, per, top_groups, group_top, renormalise, sigmoid;
  float scale;
  int* idx;
  float* weights;
};

template <int DT>
MOE_DEV float load_one(const void* p, int64_t i) {
  if (DT == MOE_DTYPE_F32) return __ldg(static_cast<const float*>(p) + i);
  const uint16_t v = __ldg(static_cast<const uint16_t*>(p) + i);
  if (DT == MOE_DTYPE_BF16) return __uint_as_float((uint32_t)v << 16);
  return __half2float(__ushort_as_half(v));
}

// The lane's NPL logits of a row; experts past E are off. VEC: rows start on
// 16-byte boundaries and E is a multiple of what one 16-byte load holds.
template <int DT, int NPL, bool VEC>
MOE_DEV void load_logits(const void* logits, int64_t row0, int E, int lane, float (&x)[NPL]) {
  constexpr int per16 = DT == MOE_DTYPE_F32 ? 4 : 8;
  if constexpr (VEC && NPL % per16 == 0) {
    const char* p = static_cast<const char*>(logits) + (row0 + lane * NPL) * (16 / per16);
#pragma unroll
    for (int c = 0; c < NPL / per16; ++c) {
      uint32_t w[4] = {0, 0, 0, 0};
      const bool in = lane * NPL + c * per16 < E;
      if (in) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + c);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (DT == MOE_DTYPE_F32) {
          x[4 * c + i] = in ? __uint_as_float(w[i]) : -INFINITY;
        } else if (DT == MOE_DTYPE_BF16) {
          x[(8 * c + 2 * i) % NPL] = in ? bf16_lo(w[i]) : -INFINITY;
          x[(8 * c + 2 * i + 1) % NPL] = in ? bf16_hi(w[i]) : -INFINITY;
        } else {
          x[(8 * c + 2 * i) % NPL] = in ? __half2float(__ushort_as_half((uint16_t)w[i])) : -INFINITY;
          x[(8 * c + 2 * i + 1) % NPL] = in ? __half2float(__ushort_as_half((uint16_t)(w[i] >> 16))) : -INFINITY;
        }
      }
    }
  } else {
#pragma unroll
    for (int q = 0; q < NPL; ++q) {
      const int e = lane * NPL + q;
      x[q] = e < E ? load_one<DT>(logits, row0 + e) : -INFINITY;
    }
  }
#pragma unroll
  for (int q = 0; q < NPL; ++q) {
    if (isnan(x[q])) x[q] = -INFINITY;
    x[q] = fminf(x[q], FLT_MAX) + 0.0f;   // -0 becomes +0: equal logits have equal keys
  }
}

MOE_DEV float warp_max(float v) {
  return f32_from_order_key(__reduce_max_sync(0xFFFFFFFFu, f32_order_key(v)));
}
MOE_DEV double warp_sum64(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Order-preserving map of a double to uint64; 0 is below every number.
MOE_DEV unsigned long long f64_order_key(double d) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(d + 0.0);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

// ---------------------------------------------------------------- 64-bit decision
// The k choices of one token with every score in 64 bits. keys: E doubles of this
// warp in shared memory. Rare (see the file's head), so written for size.
template <int NPL>
MOE_DEV void route_exact(const RouteParams& p, const float (&x)[NPL], double* keys, int lane, int* out_e) {
  double sum = 1.0, top = 0.0;
  if (!p.sigmoid) {
    float m = -INFINITY;
#pragma unroll
    for (int q = 0; q < NPL; ++q) m = fmaxf(m, x[q]);
    top = (double)warp_max(m);
    double z = 0.0;
#pragma unroll 1
    for (int q = 0; q < NPL; ++q) {
      float v = x[0];
#pragma unroll
      for (int i = 1; i < NPL; ++i) if (i == q) v = x[i];
      if (v != -INFINITY) z += exp((double)v - top);
    }
    sum = warp_sum64(z);
  }
#pragma unroll 1
  for (int q = 0; q < NPL; ++q) {
    float v = x[0];
#pragma unroll
    for (int i = 1; i < NPL; ++i) if (i == q) v = x[i];
    const int e = lane * NPL + q;
    if (e < p.E) {
      double key = -(double)INFINITY;
      if (v != -INFINITY) {
        key = p.sigmoid ? 1.0 / (1.0 + exp(-(double)v)) : exp((double)v - top) / sum;
        if (p.bias) key += (double)__ldg(p.bias + e);
      }
      keys[e] = key;
    }
  }
  __syncwarp();
  if (p.groups > 1) {
    // lane g scores group g
    unsigned long long gk = 0;
    if (lane < p.groups) {
      double a = -(double)INFINITY, b = a;
      for (int i = 0; i < p.per; ++i) {
        const double v = keys[lane * p.per + i];
        if (v > a) { b = a; a = v; } else if (v > b) { b = v; }
      }
      // an expert that is off adds nothing; a group with none on stays at -inf
      gk = f64_order_key(p.group_top == 2 && b != -(double)INFINITY ? a + b : a);
    }
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
      const unsigned long long o = __shfl_sync(0xFFFFFFFFu, gk, g);
      rank += (o > gk || (o == gk && g < lane)) ? 1 : 0;
    }
    const uint32_t kept = __ballot_sync(0xFFFFFFFFu, lane < p.groups && rank < p.top_groups);
    for (int e = lane; e < p.E; e += 32)
      if (!(kept >> (e / p.per) & 1u)) keys[e] = __longlong_as_double(0x7FF8000000000000ll);   // NaN: out
    __syncwarp();
  }
#pragma unroll 1
  for (int r = 0; r < p.k; ++r) {
    unsigned long long best = 0;
    int be = 0;
    for (int q = 0; q < NPL; ++q) {
      const int e = lane * NPL + q;
      if (e >= p.E) break;
      const double v = keys[e];
      const unsigned long long kk = isnan(v) ? 0ull : f64_order_key(v);
      if (kk > best) { best = kk; be = e; }
    }
    const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(best >> 32));
    const uint32_t lo = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
    const uint32_t who = __ballot_sync(0xFFFFFFFFu, (uint32_t)(best >> 32) == hi && (uint32_t)best == lo);
    const int src = __ffs(who) - 1;
    const int e = __shfl_sync(0xFFFFFFFFu, be, src);
    if (lane == r) *out_e = e;
    if (lane == src) keys[e] = __longlong_as_double(0x7FF8000000000000ll);
    __syncwarp();
  }
}

// ---------------------------------------------------------------------- forward
template <int DT, int NPL, bool VEC>
__global__ void __launch_bounds__(32 * kRouteWarps) route_experts_kernel(const RouteParams p) {
  __shared__ double s_keys[kRouteWarps][32 * NPL];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* s_f = reinterpret_cast<float*>(s_keys[warp]);
  const bool keyed = p.bias != nullptr || p.groups > 1;
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp; t < p.T; t += (int64_t)gridDim.x * kRouteWarps) {
    float x[NPL];
    load_logits<DT, NPL, VEC>(p.logits, t * p.stride, p.E, lane, x);
    float m = x[0];
#pragma unroll
    for (int q = 1; q < NPL; ++q) m = fmaxf(m, x[q]);
    float z = 1.f;
    if (!p.sigmoid && (keyed || !p.renormalise)) {
      m = warp_max(m);
      z = 0.f;
#pragma unroll
      for (int q = 0; q < NPL; ++q) z += x[q] == -INFINITY ? 0.f : expf(x[q] - m);
      z = warp_sum(z);
    }

    int my_e = 0;        // lane r: the r-th choice
    bool close = false;
    uint32_t key[NPL];   // 0: not to be chosen (any more)
    if (!keyed) {
#pragma unroll
      for (int q = 0; q < NPL; ++q) key[q] = lane * NPL + q < p.E ? f32_order_key(x[q]) : 0u;
    } else {
      float smax = 0.f, cmax = 0.f;
#pragma unroll
      for (int q = 0; q < NPL; ++q) {
        const int e = lane * NPL + q;
        float c = -INFINITY;
        if (x[q] != -INFINITY) {
          const float s = p.sigmoid ? 1.f / (1.f + expf(-x[q])) : expf(x[q] - m) / z;
          c = p.bias ? s + __ldg(p.bias + e) : s;
          smax = fmaxf(smax, s);
          cmax = fmaxf(cmax, fabsf(c));
        }
        key[q] = e < p.E ? f32_order_key(c + 0.f) : 0u;
      }
      // A sigmoid is within 2^-21 of itself (exp to two units in the last place, the sum's and the
      // quotient's roundings); a softmax has its row's sum besides (16 + 5 additions: 2^-19.6). A
      // group's score adds two keys, and a difference has two sides: four times that, and the
      // roundings of the keys' own sums.
      const float near = warp_max(smax) * (p.sigmoid ? 0x1p-19f : 0x1p-17f) + warp_max(cmax) * 0x1p-21f;
      if (p.groups > 1) {
        __syncwarp();
#pragma unroll
        for (int q = 0; q < NPL; ++q)
          if (lane * NPL + q < p.E) s_f[lane * NPL + q] = f32_from_order_key(key[q]);
        __syncwarp();
        float g = 0.f;
        uint32_t gk = 0u;
        if (lane < p.groups) {
          float a = -INFINITY, b = a;
          for (int i = 0; i < p.per; ++i) {
            const float v = s_f[lane * p.per + i];
            if (v > a) { b = a; a = v; } else if (v > b) { b = v; }
          }
          g = p.group_top == 2 && b != -INFINITY ? a + b : a;
          gk = f32_order_key(g + 0.f);
        }
        int rank = 0;
        for (int o = 0; o < p.groups; ++o) {
          const uint32_t v = __shfl_sync(0xFFFFFFFFu, gk, o);
          rank += (v > gk || (v == gk && o < lane)) ? 1 : 0;
        }
        const bool stays = lane < p.groups && rank < p.top_groups;
        const uint32_t kept = __ballot_sync(0xFFFFFFFFu, stays);
        if (p.top_groups < p.groups) {   // the last group that stays against the first that goes
          const float last = __shfl_sync(0xFFFFFFFFu, g, __ffs(__ballot_sync(0xFFFFFFFFu, lane < p.groups && rank == p.top_groups - 1)) - 1);
          const float next = __shfl_sync(0xFFFFFFFFu, g, __ffs(__ballot_sync(0xFFFFFFFFu, lane < p.groups && rank == p.top_groups)) - 1);
          close = next != -INFINITY && last - next <= near;
        }
#pragma unroll
        for (int q = 0; q < NPL; ++q) {
          const int e = lane * NPL + q;
          if (e < p.E && !(kept >> (e / p.per) & 1u)) key[q] = 0u;
        }
      }
      // one round more than k, to see how far the first that is left out lies
      float before = INFINITY;
      uint32_t work[NPL];
#pragma unroll
      for (int q = 0; q < NPL; ++q) work[q] = key[q];
#pragma unroll 1
      for (int r = 0; r <= p.k; ++r) {
        uint32_t bk = 0u;
#pragma unroll
        for (int q = 0; q < NPL; ++q) bk = max(bk, work[q]);
        const uint32_t gmax = __reduce_max_sync(0xFFFFFFFFu, bk);
        if (gmax == 0u) break;
        const float v = f32_from_order_key(gmax);
        if (v == -INFINITY) {
          if (r == p.k) break;
        } else {
          close |= before - v <= near;
        }
        before = v;
        const int src = __ffs(__ballot_sync(0xFFFFFFFFu, bk == gmax)) - 1;
        int wq = 0;
        bool got = false;
#pragma unroll
        for (int q = 0; q < NPL; ++q)
          if (!got && work[q] == gmax) { wq = q; got = true; if (lane == src) work[q] = 0u; }
        const int e = src * NPL + __shfl_sync(0xFFFFFFFFu, wq, src);
        if (lane == r && r < p.k) my_e = e;
      }
    }
    if (!keyed) {
#pragma unroll 1
      for (int r = 0; r < p.k; ++r) {
        uint32_t bk = 0u;
#pragma unroll
        for (int q = 0; q < NPL; ++q) bk = max(bk, key[q]);
        const uint32_t gmax = __reduce_max_sync(0xFFFFFFFFu, bk);
        const int src = __ffs(__ballot_sync(0xFFFFFFFFu, bk == gmax)) - 1;
        int wq = 0;
        bool got = false;
#pragma unroll
        for (int q = 0; q < NPL; ++q)
          if (!got && key[q] == gmax) { wq = q; got = true; if (lane == src) key[q] = 0u; }
        const int e = src * NPL + __shfl_sync(0xFFFFFFFFu, wq, src);
        if (lane == r) my_e = e;
      }
    } else if (close) {
      __syncwarp();
      route_exact<NPL>(p, x, s_keys[warp], lane, &my_e);
    }

    // the chosen logits, from the row itself (it is in L1)
    const bool mine = lane < p.k;
    float v = mine ? load_one<DT>(p.logits, t * p.stride + my_e) : -INFINITY;
    if (isnan(v)) v = -INFINITY;
    v = fminf(v, FLT_MAX);
    const bool on = v != -INFINITY;
    float w;
    if (p.renormalise) {
      // the scores' ratios alone count: e^(a - max a) / c with s = e^a / c, which no logit over- or underflows
      const float a = p.sigmoid ? fminf(v, 0.f) : v;
      const float top = warp_max(a);
      float s = on ? expf(a - top) : 0.f;
      if (p.sigmoid) s /= 1.f + expf(-fabsf(v));
      const float sum = warp_sum(s);
      w = sum > 0.f ? p.scale * (s / sum) : 0.f;
    } else {
      w = p.scale * (on ? (p.sigmoid ? 1.f / (1.f + expf(-v)) : expf(v - m) / z) : 0.f);
    }
    if (mine) {
      p.idx[t * p.k + lane] = my_e;
      p.weights[t * p.k + lane] = w;
    }
  }
}

// --------------------------------------------------------------------- backward
// d_w[j] -> d_logits. With d = scale * d_w and s the scores of the chosen:
//   renormalised:  ds[j] = (d[j] - sum_i d[i] s[i] / S) / S,  S = sum_i s[i]
//   otherwise:     ds[j] = d[j]
//   softmax:       dl[e] = s[e] (ds[e] - sum_j ds[j] s[j]);  sigmoid: dl[e] = s[e] (1 - s[e]) ds[e]
// For the renormalised softmax the last sum is 0 and s[e] ds[e] = r[e] (d[e] - sum_i d[i] r[i]) with
// the ratios r = s / S, and for the renormalised sigmoid dl = r (1 - s) (d - sum d r): only the chosen
// logits are read then. All rows are written whole.
struct RouteBackParams {
  const void* logits;
  int64_t stride;
  const int* idx;
  const float* d_weights;
  void* d_logits;   // contiguous [T][E]
  int T, E, k, renormalise, sigmoid;
  float scale;
};

template <int DT>
MOE_DEV void store_one(void* p, int64_t i, float v) {
  if (DT == MOE_DTYPE_F32) static_cast<float*>(p)[i] = v;
  else if (DT == MOE_DTYPE_BF16) static_cast<uint16_t*>(p)[i] = f32_to_bf16_rne(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

template <int DT, int NPL, bool VEC>
__global__ void __launch_bounds__(32 * kRouteWarps) route_backward_kernel(const RouteBackParams p) {
  __shared__ float s_row[kRouteWarps][32 * NPL];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* row = s_row[warp];
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp; t < p.T; t += (int64_t)gridDim.x * kRouteWarps) {
    const int e = lane < p.k ? p.idx[t * p.k + lane] : -1;
    const bool mine = e >= 0 && e < p.E;
    float v = mine ? load_one<DT>(p.logits, t * p.stride + e) : -INFINITY;
    if (isnan(v)) v = -INFINITY;
    v = fminf(v, FLT_MAX);
    const bool on = v != -INFINITY;
    const float d = mine ? p.scale * p.d_weights[t * p.k + lane] : 0.f;
    __syncwarp();
    for (int i = lane; i < p.E; i += 32) row[i] = 0.f;
    __syncwarp();
    float m = 0.f, z = 1.f, dot = 0.f;
    if (p.renormalise) {
      const float a = p.sigmoid ? fminf(v, 0.f) : v;
      const float top = warp_max(a);
      float s = on ? expf(a - top) : 0.f;
      if (p.sigmoid) s /= 1.f + expf(-fabsf(v));
      const float sum = warp_sum(s);
      const float r = sum > 0.f ? s / sum : 0.f;
      float g = r * (d - warp_sum(on ? d * r : 0.f));
      if (p.sigmoid) g *= 1.f / (1.f + expf(v));   // 1 - s
      if (mine && on) row[e] = g;
    } else if (p.sigmoid) {
      if (mine && on) row[e] = d * (1.f / (1.f + expf(-v))) * (1.f / (1.f + expf(v)));
    } else {
      if (mine && on) row[e] = d;
    }
    __syncwarp();
    float x[NPL];
    const bool full = !p.renormalise && !p.sigmoid;
    if (full) {
      load_logits<DT, NPL, VEC>(p.logits, t * p.stride, p.E, lane, x);
      m = x[0];
#pragma unroll
      for (int q = 1; q < NPL; ++q) m = fmaxf(m, x[q]);
      m = warp_max(m);
      z = 0.f;
#pragma unroll
      for (int q = 0; q < NPL; ++q) {
        x[q] = x[q] == -INFINITY ? 0.f : expf(x[q] - m);
        z += x[q];
      }
      z = warp_sum(z);
      dot = warp_sum(on ? d * (expf(v - m) / z) : 0.f);   // on: z >= 1
#pragma unroll
      for (int q = 0; q < NPL; ++q) {
        const int i = lane * NPL + q;
        if (i < p.E) row[i] = z > 0.f ? x[q] / z * (row[i] - dot) : 0.f;
      }
      __syncwarp();
    }
    if (VEC) {
      constexpr int per16 = DT == MOE_DTYPE_F32 ? 4 : 8;
      uint4* dst = reinterpret_cast<uint4*>(static_cast<char*>(p.d_logits) + t * p.E * (16 / per16));
      for (int c = lane; c < p.E / per16; c += 32) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (DT == MOE_DTYPE_F32) {
            w[i] = __float_as_uint(row[4 * c + i]);
          } else {
            const float lo = row[8 * c + 2 * i], hi = row[8 * c + 2 * i + 1];
            w[i] = DT == MOE_DTYPE_BF16
                       ? (uint32_t)f32_to_bf16_rne(lo) | ((uint32_t)f32_to_bf16_rne(hi) << 16)
                       : (uint32_t)__half_as_ushort(__float2half_rn(lo)) |
                             ((uint32_t)__half_as_ushort(__float2half_rn(hi)) << 16);
          }
        }
        dst[c] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {
      for (int i = lane; i < p.E; i += 32) store_one<DT>(p.d_logits, t * p.E + i, row[i]);
    }
  }
}

// ------------------------------------------------------------------------- host
template <class P>
using RouteKernel = void (*)(const P);

template <int DT, int NPL, bool VEC>
RouteKernel<RouteParams> pick_kernel(const RouteParams&) { return route_experts_kernel<DT, NPL, VEC>; }
template <int DT, int NPL, bool VEC>
RouteKernel<RouteBackParams> pick_kernel(const RouteBackParams&) { return route_backward_kernel<DT, NPL, VEC>; }

template <int DT, bool VEC, class P>
RouteKernel<P> by_experts(const P& p) {
  if (p.E <= 64) return pick_kernel<DT, 2, VEC>(p);
  if (p.E <= 128) return pick_kernel<DT, 4, VEC>(p);
  if (p.E <= 256) return pick_kernel<DT, 8, VEC>(p);
  return pick_kernel<DT, 16, VEC>(p);
}

template <class P>
cudaError_t launch_route(const P& p, int dtype, bool vec, cudaStream_t s) {
  RouteKernel<P> f;
  if (dtype == MOE_DTYPE_F32) f = vec ? by_experts<MOE_DTYPE_F32, true>(p) : by_experts<MOE_DTYPE_F32, false>(p);
  else if (dtype == MOE_DTYPE_BF16) f = vec ? by_experts<MOE_DTYPE_BF16, true>(p) : by_experts<MOE_DTYPE_BF16, false>(p);
  else f = vec ? by_experts<MOE_DTYPE_F16, true>(p) : by_experts<MOE_DTYPE_F16, false>(p);
  const int64_t blocks = ((int64_t)p.T + kRouteWarps - 1) / kRouteWarps;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks < 152 * 16 ? blocks : 152 * 16));
  cfg.blockDim = dim3(32 * kRouteWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, f, p);
}

moe_status_t check_route(const moe_route_config_t* c, const void* logits, int32_t dtype, int64_t stride, int32_t T) {
  if (!c || T < 0) return MOE_ERR_INVALID_ARG;
  if (c->num_experts < 1 || c->top_k < 1 || c->groups < 1 || c->top_groups < 1 || c->top_groups > c->groups)
    return MOE_ERR_INVALID_ARG;
  if (c->num_experts % c->groups || c->top_k > c->num_experts / c->groups * c->top_groups) return MOE_ERR_INVALID_ARG;
  if (c->group_top != 1 && c->group_top != 2) return MOE_ERR_INVALID_ARG;
  if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (!isfinite(c->scale)) return MOE_ERR_INVALID_ARG;
  if (c->num_experts > MOE_ROUTE_MAX_EXPERTS || c->top_k > MOE_ROUTE_MAX_TOP_K || c->groups > MOE_ROUTE_MAX_GROUPS)
    return MOE_ERR_UNSUPPORTED;
  if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16) return MOE_ERR_INVALID_ARG;
  if (stride < c->num_experts) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!logits || ((uintptr_t)logits & (dtype == MOE_DTYPE_F32 ? 3 : 1)))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// Rows of `stride` elements from `base` can be read 16 bytes at a time.
bool rows_16(const void* base, int dtype, int64_t stride, int E) {
  const int size = dtype == MOE_DTYPE_F32 ? 4 : 2;
  return !((uintptr_t)base & 15) && stride * size % 16 == 0 && E * size % 16 == 0;
}

}  // namespace
}  // namespace moe

extern "C" {

moe_status_t moe_route_experts(const moe_route_config_t* cfg, const void* logits_dev, int32_t logits_dtype,
                               int64_t row_stride, const float* bias_dev, int32_t T, int32_t* idx_dev,
                               float* weights_dev, void* stream) {
  const moe_status_t st = moe::check_route(cfg, logits_dev, logits_dtype, row_stride, T);
  if (st != MOE_OK || T == 0) return st;
  if (!idx_dev || !weights_dev || ((uintptr_t)idx_dev & 3) || ((uintptr_t)weights_dev & 3) || ((uintptr_t)bias_dev & 3))
    return MOE_ERR_INVALID_ARG;
  moe::RouteParams p = {};
  p.logits = logits_dev;
  p.bias = bias_dev;
  p.stride = row_stride;
  p.T = T;
  p.E = cfg->num_experts;
  p.k = cfg->top_k;
  p.groups = cfg->top_groups < cfg->groups ? cfg->groups : 1;   // all groups stay: none is scored
  p.per = p.E / p.groups;
  p.top_groups = p.groups > 1 ? cfg->top_groups : 1;
  p.group_top = cfg->group_top;
  p.renormalise = cfg->renormalise != 0;
  p.sigmoid = cfg->score == MOE_SCORE_SIGMOID;
  p.scale = cfg->scale;
  p.idx = idx_dev;
  p.weights = weights_dev;
  const cudaError_t e = moe::launch_route(p, logits_dtype, moe::rows_16(logits_dev, logits_dtype, row_stride, p.E),
                                          (cudaStream_t)stream);
  return e == cudaSuccess ? MOE_OK : moe::record_cuda_failure(e, "moe_route_experts");
}

moe_status_t moe_route_experts_backward(const moe_route_config_t* cfg, const void* logits_dev, int32_t logits_dtype,
                                        int64_t row_stride, const int32_t* idx_dev, const float* d_weights_dev,
                                        int32_t T, void* d_logits_dev, void* stream) {
  const moe_status_t st = moe::check_route(cfg, logits_dev, logits_dtype, row_stride, T);
  if (st != MOE_OK || T == 0) return st;
  if (!idx_dev || !d_weights_dev || !d_logits_dev || ((uintptr_t)idx_dev & 3) || ((uintptr_t)d_weights_dev & 3) ||
      ((uintptr_t)d_logits_dev & (logits_dtype == MOE_DTYPE_F32 ? 3 : 1)))
    return MOE_ERR_INVALID_ARG;
  moe::RouteBackParams p = {};
  p.logits = logits_dev;
  p.stride = row_stride;
  p.idx = idx_dev;
  p.d_weights = d_weights_dev;
  p.d_logits = d_logits_dev;
  p.T = T;
  p.E = cfg->num_experts;
  p.k = cfg->top_k;
  p.renormalise = cfg->renormalise != 0;
  p.sigmoid = cfg->score == MOE_SCORE_SIGMOID;
  p.scale = cfg->scale;
  const bool vec = moe::rows_16(logits_dev, logits_dtype, row_stride, p.E) &&
                   moe::rows_16(d_logits_dev, logits_dtype, p.E, p.E);
  const cudaError_t e = moe::launch_route(p, logits_dtype, vec, (cudaStream_t)stream);
  return e == cudaSuccess ? MOE_OK : moe::record_cuda_failure(e, "moe_route_experts_backward");
}

}  // extern "C"
