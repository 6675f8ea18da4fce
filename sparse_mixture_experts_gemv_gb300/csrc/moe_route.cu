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
// 32-bit errors can reach; where a pair is closer, the keys are taken in 64 bits.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "moe_common.cuh"
#include "moe_int8.h"
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

// The lane's NPL logits of a row; -inf for experts past E. VEC: rows start on
// 16-byte boundaries and E is a multiple of what one 16-byte load holds.
template <int DT, int NPL, bool VEC>
MOE_DEV void load_raw(const void* logits, int64_t row0, int E, int lane, float (&x)[NPL]) {
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
}

// The same with NaN as -inf and +inf as the largest finite value.
template <int DT, int NPL, bool VEC>
MOE_DEV void load_logits(const void* logits, int64_t row0, int E, int lane, float (&x)[NPL]) {
  load_raw<DT, NPL, VEC>(logits, row0, E, lane, x);
#pragma unroll
  for (int q = 0; q < NPL; ++q) {
    if (isnan(x[q])) x[q] = -INFINITY;
    x[q] = fminf(x[q], FLT_MAX) + 0.0f;   // -0 becomes +0: equal logits have equal keys
  }
}

// The same for rows of finite logits, as they are; false where the lane has one that is not.
template <int DT, int NPL, bool VEC>
MOE_DEV bool load_finite(const void* logits, int64_t row0, int E, int lane, float (&x)[NPL]) {
  load_raw<DT, NPL, VEC>(logits, row0, E, lane, x);
  float zero = 0.f;
#pragma unroll
  for (int q = 0; q < NPL; ++q) zero = fmaf(lane * NPL + q < E ? x[q] : 0.f, 0.f, zero);   // NaN from inf and NaN
  return zero == 0.f;
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
// 1 / (1 + e^-x) by the approximate exponential and reciprocal. The exponential's argument is
// rounded to |x| 2^-23 or so, which s (1 - s) |x| <= 0.23 bounds in the result: within 2^-21
// of the sigmoid, absolutely, for every x.
MOE_DEV float key_sigmoid(float x) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
  return s;
}

// A pair of keys closer than this may be in either order. A sigmoid is within 2^-21 of what it
// stands for, a softmax, which has its row's sum besides (16 + 5 additions: 2^-19.6), within 2^-19
// of the row's largest, 1 / z. A group's score adds two keys, and a difference has two sides: four
// times that, and the roundings of sums that reach 1 + the largest bias.
MOE_DEV float near_of(const RouteParams& p, float z, float largest_bias) {
  return (p.sigmoid ? 0x1p-19f : 0x1p-17f / z) + (1.f + largest_bias) * 0x1p-21f;
}

// The top_groups largest of the lanes' scores below `lanes` that are a group's, as a mask of lanes; close:
// the last of them and the first that goes lie within `near`. score: -inf where no expert is on.
MOE_DEV uint32_t choose_groups(const RouteParams& p, float score, bool is_group, float near, int lane, bool& close) {
  uint32_t left = is_group ? f32_order_key(score + 0.f) : 0u, kept = 0u;
  float before = INFINITY;
  for (int r = 0; r <= p.top_groups; ++r) {
    const uint32_t g = __reduce_max_sync(0xFFFFFFFFu, left);
    const uint32_t first = __ballot_sync(0xFFFFFFFFu, left == g);
    const float v = f32_from_order_key(g);
    if (r == p.top_groups) {
      close = g != 0u && v != -INFINITY && before - v <= near;
      break;
    }
    before = v;
    kept |= first & (0u - first);
    if (lane == __ffs(first) - 1) left = 0u;
  }
  return kept;
}

// Rows that the short list does not serve: logits that are not finite, too many equal keys, too few
// lanes with an expert on, groups or (softmax) experts too close to tell apart in 32 bits. All keys
// one at a time, and in 64 bits where it takes that. Lane r returns the r-th choice.
template <int DT, int NPL, bool VEC, bool KEYED>
__device__ __noinline__ int route_slowly(const RouteParams& p, int64_t t, double* keys, int lane) {
  float x[NPL], c[NPL];
  load_logits<DT, NPL, VEC>(p.logits, t * p.stride, p.E, lane, x);
  int my_e = 0;
  uint32_t key[NPL];   // 0: not to be chosen (any more)
  bool close = KEYED;
  if (!KEYED) {
#pragma unroll
    for (int q = 0; q < NPL; ++q) key[q] = lane * NPL + q < p.E ? f32_order_key(x[q]) : 0u;
  } else if (p.groups == 1) {
    float m = x[0], z = 1.f, top = 0.f;
    if (!p.sigmoid) {
#pragma unroll
      for (int q = 1; q < NPL; ++q) m = fmaxf(m, x[q]);
      m = warp_max(m);
      z = 0.f;
#pragma unroll
      for (int q = 0; q < NPL; ++q) z += x[q] == -INFINITY ? 0.f : expf(x[q] - m);
      z = fmaxf(warp_sum(z), 1.f);   // at least the largest's 1, where one is on
    }
#pragma unroll
    for (int q = 0; q < NPL; ++q) {
      const int e = lane * NPL + q;
      const float b = e < p.E && p.bias ? __ldg(p.bias + e) : 0.f;
      top = fmaxf(top, fabsf(b));
      c[q] = x[q] == -INFINITY ? -INFINITY : (p.sigmoid ? key_sigmoid(x[q]) : expf(x[q] - m) / z) + b;
      key[q] = e < p.E ? f32_order_key(c[q] + 0.f) : 0u;
    }
    const float near = near_of(p, z, warp_max(top));
    // as below, but without taking anything off: only to see whether the choice is firm
    uint32_t left[NPL];
#pragma unroll
    for (int q = 0; q < NPL; ++q) left[q] = key[q];
    float before = INFINITY;
    close = false;
#pragma unroll 1
    for (int r = 0; r <= p.k; ++r) {
      uint32_t bk = 0u;
#pragma unroll
      for (int q = 0; q < NPL; ++q) bk = max(bk, left[q]);
      const uint32_t g = __reduce_max_sync(0xFFFFFFFFu, bk);
      const float v = f32_from_order_key(g);
      if (g == 0u || v == -INFINITY) break;   // experts that are off go by index: nothing to tell apart
      close |= before - v <= near;
      before = v;
      const int src = __ffs(__ballot_sync(0xFFFFFFFFu, bk == g)) - 1;
      bool got = false;
#pragma unroll
      for (int q = 0; q < NPL; ++q)
        if (lane == src && !got && left[q] == g) { left[q] = 0u; got = true; }
    }
  }
  if (close) {
    __syncwarp();
    route_exact<NPL>(p, x, keys, lane, &my_e);
    return my_e;
  }
#pragma unroll 1
  for (int r = 0; r < p.k; ++r) {
    uint32_t bk = 0u;
#pragma unroll
    for (int q = 0; q < NPL; ++q) bk = max(bk, key[q]);
    const uint32_t g = __reduce_max_sync(0xFFFFFFFFu, bk);
    const int src = __ffs(__ballot_sync(0xFFFFFFFFu, bk == g)) - 1;
    int wq = 0;
    bool got = false;
#pragma unroll
    for (int q = 0; q < NPL; ++q)
      if (!got && key[q] == g) { wq = q; got = true; if (lane == src) key[q] = 0u; }
    const int e = src * NPL + __shfl_sync(0xFFFFFFFFu, wq, src);
    if (lane == r) my_e = e;
  }
  return my_e;
}

// Nearly all rows: the k-th largest of the lanes' largest keys is at most the k-th largest key, and few
// keys lie above it (about 10 for k = 8). These, each in a lane of its own and in the order of their
// indexes, are ranked by counting; with a bias or groups, keys closer than `near` are ranked again in
// 64 bits, one evaluation a lane.
// Bound by its instructions, some 500 a row of 512 (65,536 rows of 512 bf16 logits: see the launch).
template <int DT, int NPL, bool VEC, bool KEYED>
__global__ void __launch_bounds__(32 * kRouteWarps, NPL == 16 ? 6 : 8) route_experts_kernel(const RouteParams p) {
  __shared__ double s_keys[kRouteWarps][32 * NPL];
  __shared__ int s_list[kRouteWarps][32];
  __shared__ float s_sorted[kRouteWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* s_f = reinterpret_cast<float*>(s_keys[warp]);
  pdl_wait();
  pdl_launch_dependents();
  float bias[NPL], largest_bias = 0.f;
  if (KEYED) {
#pragma unroll
    for (int q = 0; q < NPL; ++q) {
      const int e = lane * NPL + q;
      bias[q] = e >= p.E ? -INFINITY : p.bias ? __ldg(p.bias + e) : 0.f;   // -inf: never among the chosen
      if (e < p.E) largest_bias = fmaxf(largest_bias, fabsf(bias[q]));
    }
    largest_bias = warp_max(largest_bias);
  }
  // lanes a group has, where it is a run of 1, 2, 4, ... whole lanes
  const int run = p.per % NPL == 0 && ((p.per / NPL) & (p.per / NPL - 1)) == 0 ? p.per / NPL : 0;
  const uint32_t kOff = 0x007FFFFFu;   // the order key of -inf

  for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp; t < p.T; t += (int64_t)gridDim.x * kRouteWarps) {
    float c[NPL];
    const bool finite = load_finite<DT, NPL, VEC>(p.logits, t * p.stride, p.E, lane, c);
    bool slow = __any_sync(0xFFFFFFFFu, !finite);
    float m = 0.f, z = 1.f, near = 0.f;
    if (!p.sigmoid && (KEYED || !p.renormalise)) {   // c becomes the numerators; experts past E give 0
      m = c[0];
#pragma unroll
      for (int q = 1; q < NPL; ++q) m = fmaxf(m, c[q]);
      m = warp_max(slow ? 0.f : m);
      z = 0.f;
#pragma unroll
      for (int q = 0; q < NPL; ++q) {
        const float e = expf(c[q] - m);
        z += e;
        if (KEYED) c[q] = e;
      }
      z = warp_sum(z);
    }
    if (KEYED) {
      near = near_of(p, z, largest_bias);
      if (p.sigmoid) {
#pragma unroll
        for (int q = 0; q < NPL; ++q) c[q] = key_sigmoid(c[q]) + bias[q];
      } else {
        const float scale = 1.f / z;
#pragma unroll
        for (int q = 0; q < NPL; ++q) c[q] = fmaf(c[q], scale, bias[q]);
      }
    }

    float top = c[0];   // the lane's largest key among those that may be chosen
    if (KEYED && p.groups > 1) {
      float a = c[0], b = -INFINITY;   // the two largest keys
      bool close;
      if (run) {
#pragma unroll
        for (int q = 1; q < NPL; ++q) {
          b = fmaxf(b, fminf(a, c[q]));
          a = fmaxf(a, c[q]);
        }
        top = a;
        for (int o = 1; o < run; o <<= 1) {
          const float oa = __shfl_xor_sync(0xFFFFFFFFu, a, o), ob = __shfl_xor_sync(0xFFFFFFFFu, b, o);
          b = fmaxf(fmaxf(b, ob), fminf(a, oa));
          a = fmaxf(a, oa);
        }
        const float score = p.group_top == 2 && p.per > 1 ? a + b : a;
        const uint32_t kept = choose_groups(p, score, lane % run == 0 && lane / run < p.groups, near, lane, close);
        if (!(kept >> (lane - lane % run) & 1u)) top = -INFINITY;
      } else {
        __syncwarp();
#pragma unroll
        for (int q = 0; q < NPL; ++q)
          if (lane * NPL + q < p.E) s_f[lane * NPL + q] = c[q];
        __syncwarp();
        a = -INFINITY;
        if (lane < p.groups)
          for (int i = 0; i < p.per; ++i) {
            const float v = s_f[lane * p.per + i];
            b = fmaxf(b, fminf(a, v));
            a = fmaxf(a, v);
          }
        const float score = p.group_top == 2 && p.per > 1 ? a + b : a;
        const uint32_t kept = choose_groups(p, score, lane < p.groups, near, lane, close);
        top = -INFINITY;
#pragma unroll
        for (int q = 0; q < NPL; ++q) {
          const int e = lane * NPL + q;
          if (e >= p.E || !(kept >> (e / p.per) & 1u)) c[q] = -INFINITY;
          top = fmaxf(top, c[q]);
        }
      }
      slow |= close;
    } else {
#pragma unroll
      for (int q = 1; q < NPL; ++q) top = fmaxf(top, c[q]);
    }

    // the short list
    uint32_t left = f32_order_key(top + 0.f), bound = 0u;
    for (int r = 0; r < p.k; ++r) {
      bound = __reduce_max_sync(0xFFFFFFFFu, left);
      if (lane == __ffs(__ballot_sync(0xFFFFFFFFu, left == bound)) - 1) left = 0u;
    }
    const float least = f32_from_order_key(max(bound, kOff)) - near;
    uint32_t listed = 0u;
#pragma unroll
    for (int q = 0; q < NPL; ++q) listed |= c[q] >= least ? 1u << q : 0u;
    if (!(top >= least)) listed = 0u;
    const int count = __popc(listed);
    int at = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, at, o);
      if (lane >= o) at += v;
    }
    const int n = __shfl_sync(0xFFFFFFFFu, at, 31);
    slow |= bound <= kOff || n > 32;

    int e = 0, rank = lane;   // the lane's expert, and its place among the chosen
    if (!slow) {
      at -= count;
      __syncwarp();
      while (listed) {
        s_list[warp][at++] = lane * NPL + __ffs(listed) - 1;
        listed &= listed - 1;
      }
      __syncwarp();
      float key = -INFINITY, b = 0.f, v = 0.f;
      if (lane < n) {
        e = s_list[warp][lane];
        v = load_one<DT>(p.logits, t * p.stride + e) + 0.f;   // the row is in L1
        if (KEYED && p.bias) b = __ldg(p.bias + e);
        key = !KEYED ? v : p.sigmoid ? key_sigmoid(v) + b : fmaf(expf(v - m), 1.f / z, b);
      }
      rank = lane < n ? 0 : 32;
#pragma unroll 4
      for (int o = 0; o < n; ++o) {
        const float w = __shfl_sync(0xFFFFFFFFu, key, o);
        if (lane < n) rank += (w > key || (w == key && o < lane)) ? 1 : 0;
      }
      if (KEYED) {
        __syncwarp();
        if (lane < n) s_sorted[warp][rank] = key;
        __syncwarp();
        const bool close = lane < p.k && lane + 1 < n && s_sorted[warp][lane] - s_sorted[warp][lane + 1] <= near;
        if (__any_sync(0xFFFFFFFFu, close)) {
          if (p.sigmoid) {
            const unsigned long long exact =
                lane < n ? f64_order_key(1.0 / (1.0 + exp(-(double)v)) + (double)b) : 0ull;
            rank = lane < n ? 0 : 32;
            for (int o = 0; o < n; ++o) {
              const unsigned long long w = __shfl_sync(0xFFFFFFFFu, exact, o);
              if (lane < n) rank += (w > exact || (w == exact && o < lane)) ? 1 : 0;
            }
          } else {   // the row's sum has to be exact too
            slow = true;
          }
        }
      }
    }
    if (slow) {
      e = route_slowly<DT, NPL, VEC, KEYED>(p, t, s_keys[warp], lane);
      rank = lane;
      if (!p.renormalise && !p.sigmoid) {   // the sums, of the experts that are on
        float x[NPL];
        load_logits<DT, NPL, VEC>(p.logits, t * p.stride, p.E, lane, x);
        m = x[0];
#pragma unroll
        for (int q = 1; q < NPL; ++q) m = fmaxf(m, x[q]);
        m = warp_max(m);
        z = 0.f;
#pragma unroll
        for (int q = 0; q < NPL; ++q) z += x[q] == -INFINITY ? 0.f : expf(x[q] - m);
        z = warp_sum(z);
      }
    }

    const bool mine = rank < p.k;
    float v = mine ? load_one<DT>(p.logits, t * p.stride + e) : -INFINITY;
    if (isnan(v)) v = -INFINITY;
    v = fminf(v, FLT_MAX);
    const bool on = v != -INFINITY;
    float w;
    if (p.renormalise) {
      // the scores' ratios alone count: e^(a - max a) / c with s = e^a / c, which no logit over- or underflows
      const float a = p.sigmoid ? fminf(v, 0.f) : v;
      const float most = warp_max(a);
      float s = on ? expf(a - most) : 0.f;
      if (p.sigmoid) s /= 1.f + expf(-fabsf(v));
      const float sum = warp_sum(s);
      w = sum > 0.f ? p.scale * (s / sum) : 0.f;
    } else {
      w = p.scale * (on ? (p.sigmoid ? 1.f / (1.f + expf(-v)) : expf(v - m) / z) : 0.f);
    }
    if (mine) {
      p.idx[t * p.k + rank] = e;
      p.weights[t * p.k + rank] = w;
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
__global__ void __launch_bounds__(32 * kRouteWarps, NPL == 16 ? 6 : 8) route_backward_kernel(const RouteBackParams p) {
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
RouteKernel<RouteParams> pick_kernel(const RouteParams& p) {
  return p.bias || p.groups > 1 ? route_experts_kernel<DT, NPL, VEC, true> : route_experts_kernel<DT, NPL, VEC, false>;
}
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
  const int num_sms = int8::device_sms();
  RouteKernel<P> f;
  if (dtype == MOE_DTYPE_F32) f = vec ? by_experts<MOE_DTYPE_F32, true>(p) : by_experts<MOE_DTYPE_F32, false>(p);
  else if (dtype == MOE_DTYPE_BF16) f = vec ? by_experts<MOE_DTYPE_BF16, true>(p) : by_experts<MOE_DTYPE_BF16, false>(p);
  else f = vec ? by_experts<MOE_DTYPE_F16, true>(p) : by_experts<MOE_DTYPE_F16, false>(p);
  // no more CTAs than are resident at once: each warp keeps its experts' biases, and a second wave of a
  // few CTAs would run alone
  const int64_t blocks = ((int64_t)p.T + kRouteWarps - 1) / kRouteWarps;
  const int per_sm = p.E > 256 ? 6 : 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks < num_sms * per_sm ? blocks : num_sms * per_sm));
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
