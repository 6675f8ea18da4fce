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
// A bias is read the same way, and so a key is a finite number or -inf, never NaN:
// comparisons of keys, and differences of finite ones, always say something.
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
#include <cuda_bf16.h>
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

// The lane's NPL logits of a row as they are, -inf for experts past E; false where one is not
// finite. VEC: rows start on 16-byte boundaries and E is a multiple of what one 16-byte load holds.
template <int DT, int NPL, bool VEC>
MOE_DEV bool load_raw(const void* logits, int64_t row0, int E, int lane, float (&x)[NPL]) {
  constexpr int per16 = DT == MOE_DTYPE_F32 ? 4 : 8;
  constexpr uint32_t kOffPair = DT == MOE_DTYPE_F32 ? 0xFF800000u : DT == MOE_DTYPE_BF16 ? 0xFF80FF80u : 0xFC00FC00u;
  float zero = 0.f;   // NaN from infinities and NaN
  if constexpr (VEC && NPL % per16 == 0) {
    const char* p = static_cast<const char*>(logits) + (row0 + lane * NPL) * (16 / per16);
#pragma unroll
    for (int c = 0; c < NPL / per16; ++c) {
      uint4 v = make_uint4(kOffPair, kOffPair, kOffPair, kOffPair);
      const bool in = lane * NPL + c * per16 < E;
      if (in) v = __ldg(reinterpret_cast<const uint4*>(p) + c);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      float y[per16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (DT == MOE_DTYPE_F32) {
          y[i] = __uint_as_float(w[i]);
        } else if (DT == MOE_DTYPE_BF16) {
          y[(2 * i) % per16] = bf16_lo(w[i]);
          y[(2 * i + 1) % per16] = bf16_hi(w[i]);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
          y[(2 * i) % per16] = f.x;
          y[(2 * i + 1) % per16] = f.y;
        }
      }
      float chunk = 0.f;
#pragma unroll
      for (int i = 0; i < per16; ++i) {
        chunk = fmaf(y[i], 0.f, chunk);
        x[c * per16 + i] = y[i];
      }
      if (in) zero += chunk;
    }
  } else {
#pragma unroll
    for (int q = 0; q < NPL; ++q) {
      const int e = lane * NPL + q;
      x[q] = e < E ? load_one<DT>(logits, row0 + e) : -INFINITY;
      zero = fmaf(e < E ? x[q] : 0.f, 0.f, zero);
    }
  }
  return zero == 0.f;
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

// The bias of expert e: NaN as -inf, +inf as the largest finite value.
MOE_DEV float load_bias(const float* bias, int e) {
  const float b = __ldg(bias + e);
  return isnan(b) ? -INFINITY : fminf(b, FLT_MAX);
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
// The k choices of one token, lane r's being the r-th, with every key in 64 bits (the logits
// themselves where nothing else is asked for). keys: E doubles of this warp in shared memory. It
// serves the rows that the short list does not: too few lanes with an expert on, too many equal
// keys, groups or (softmax) experts too close to tell apart in 32 bits. With sigmoid scores, or a
// bias of distinct values, that is under 1% of rows, and so it is fetched cold: rolled loops, as
// little code as can be (unrolled, its fetch alone took some 50 us of a call). It is not rare where
// a softmax has equal keys, as 16-bit logits often are under groups or under one bias for several
// experts: 6% (fp16) to 50% (bf16) of rows, and 65,536 x 512 take 0.6 to 2.7 ms. Nor where one
// finite bias is very large (-1e9), by which all rows' keys count as close: 3.3 to 4.6 ms (-inf: 57 us).
template <int DT>
__device__ __noinline__ int route_exact(const RouteParams& p, int64_t t, bool keyed, double* keys, int lane) {
  const double kNone = -(double)INFINITY, kOut = __longlong_as_double(0x7FF8000000000000ll);   // off; NaN: out
  double sum = 1.0, top = 0.0;
  const bool softmax = keyed && !p.sigmoid;
  __syncwarp();
  float m = -INFINITY;
#pragma unroll 1
  for (int e = lane; e < p.E; e += 32) {
    float v = load_one<DT>(p.logits, t * p.stride + e);
    v = isnan(v) ? -INFINITY : fminf(v, FLT_MAX) + 0.f;
    m = fmaxf(m, v);
    keys[e] = (double)v;
  }
  if (softmax) {
    top = (double)warp_max(m);
    sum = 0.0;
#pragma unroll 1
    for (int e = lane; e < p.E; e += 32) sum += keys[e] == kNone ? 0.0 : exp(keys[e] - top);
    sum = warp_sum64(sum);
  }
#pragma unroll 1
  for (int e = lane; keyed && e < p.E; e += 32) {
    const double v = keys[e];
    if (v == kNone) continue;
    const double u = exp(softmax ? v - top : -v);
    keys[e] = (softmax ? u / sum : 1.0 / (1.0 + u)) + (p.bias ? (double)load_bias(p.bias, e) : 0.0);
  }
  __syncwarp();
  if (p.groups > 1) {
    unsigned long long gk = 0;   // lane g scores group g
    if (lane < p.groups) {
      double a = kNone, b = kNone;
#pragma unroll 1
      for (int i = 0; i < p.per; ++i) {
        const double v = keys[lane * p.per + i];
        if (v > a) { b = a; a = v; } else if (v > b) { b = v; }
      }
      // an expert that is off adds nothing; a group with none on stays at -inf
      gk = f64_order_key(p.group_top == 2 && b != kNone ? a + b : a);
    }
    int rank = 0;
#pragma unroll 1
    for (int g = 0; g < p.groups; ++g) {
      const unsigned long long o = __shfl_sync(0xFFFFFFFFu, gk, g);
      rank += (o > gk || (o == gk && g < lane)) ? 1 : 0;
    }
    const uint32_t kept = __ballot_sync(0xFFFFFFFFu, lane < p.groups && rank < p.top_groups);
#pragma unroll 1
    for (int e = lane; e < p.E; e += 32)
      if (!(kept >> (e / p.per) & 1u)) keys[e] = kOut;
    __syncwarp();
  }
  int mine = 0;
#pragma unroll 1
  for (int r = 0; r < p.k; ++r) {
    unsigned long long best = 0;
    uint32_t be = 0;
#pragma unroll 1
    for (int e = lane; e < p.E; e += 32) {
      const double v = keys[e];
      const unsigned long long kk = isnan(v) ? 0ull : f64_order_key(v);
      if (kk > best) { best = kk; be = e; }
    }
    const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(best >> 32));
    const bool high = (uint32_t)(best >> 32) == hi;
    const uint32_t lo = __reduce_max_sync(0xFFFFFFFFu, high ? (uint32_t)best : 0u);
    const uint32_t e = __reduce_min_sync(0xFFFFFFFFu, high && (uint32_t)best == lo ? be : 0xFFFFFFFFu);
    if (lane == r) mine = (int)e;
    if (lane == (int)(e & 31u)) keys[e] = kOut;
    __syncwarp();
  }
  return mine;
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

// A key with its last 5 bits replaced by the lane: distinct, so that a warp's largest also says whose
// it is. Off by less than 2^-18 of itself.
MOE_DEV uint32_t lane_key(float v, int lane) { return (f32_order_key(v) & ~31u) | (uint32_t)lane; }

// The top_groups largest of the scores that the lanes below p.groups hold, as a mask; close: the last
// of them and the first that goes lie within `near`. score: -inf where no expert is on.
MOE_DEV uint32_t choose_groups(const RouteParams& p, float score, float near, int lane, bool& close) {
  uint32_t left = lane < p.groups ? f32_order_key(score + 0.f) : 0u, kept = 0u, g = 0u, last = 0u;
  for (int r = 0; r <= p.top_groups; ++r) {
    last = g;
    g = __reduce_max_sync(0xFFFFFFFFu, left);
    const uint32_t first = __ballot_sync(0xFFFFFFFFu, left == g);
    if (r < p.top_groups) kept |= first & (0u - first);
    if (lane == __ffs(first) - 1) left = 0u;
  }
  const float a = f32_from_order_key(last), b = f32_from_order_key(g);
  close = b != -INFINITY && a - b <= near;
  return kept;
}

// The same in 64 bits for sigmoid scores, where 32 were too few: of each group's keys, those that can be
// among its two largest, one a lane. keys: the warp's keys; second: lane g's group's second largest; list
// and sums: 32 of shared memory each. false: more than 32 such keys.
template <int DT>
__device__ __noinline__ bool choose_groups_exactly(const RouteParams& p, int64_t t, const float* keys, float second,
                                                   float near, int lane, int* list, double* sums, uint32_t* kept) {
  int n = 0;
  __syncwarp();
#pragma unroll 1
  for (int e0 = 0; e0 < p.E; e0 += 32) {
    const int e = e0 + lane, g = min(e / p.per, 31);
    const float b = __shfl_sync(0xFFFFFFFFu, second, g);
    const bool take = e < p.E && keys[e] != -INFINITY && keys[e] >= b - near;
    const uint32_t who = __ballot_sync(0xFFFFFFFFu, take);
    const int at = n + __popc(who & ((1u << lane) - 1));
    if (take && at < 32) list[at] = e;
    n += __popc(who);
  }
  if (n > 32) return false;
  sums[lane] = -(double)INFINITY;
  __syncwarp();
  double key = -(double)INFINITY;
  int g = -1;
  if (lane < n) {
    const int e = list[lane];
    const float v = fminf(load_one<DT>(p.logits, t * p.stride + e), FLT_MAX);
    key = 1.0 / (1.0 + exp(-(double)v)) + (p.bias ? (double)load_bias(p.bias, e) : 0.0);
    g = e / p.per;
  }
  int rank = 0;
  double runner_up = 0.0;   // of the lane's group, for its first
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
    for (int o = 0; o < n; ++o) {
      const double w = __shfl_sync(0xFFFFFFFFu, key, o);
      const int og = __shfl_sync(0xFFFFFFFFu, g, o), orank = __shfl_sync(0xFFFFFFFFu, rank, o);
      if (og != g) continue;
      if (pass == 0) rank += (w > key || (w == key && o < lane)) ? 1 : 0;
      else if (orank == 1 && p.group_top == 2) runner_up = w;
    }
  }
  if (lane < n && rank == 0) sums[g] = key + runner_up;
  __syncwarp();
  const unsigned long long score = lane < p.groups ? f64_order_key(sums[lane]) : 0ull;
  int place = 0;
#pragma unroll 1
  for (int o = 0; o < p.groups; ++o) {
    const unsigned long long w = __shfl_sync(0xFFFFFFFFu, score, o);
    place += (w > score || (w == score && o < lane)) ? 1 : 0;
  }
  *kept = __ballot_sync(0xFFFFFFFFu, lane < p.groups && place < p.top_groups);
  __syncwarp();
  return true;
}

MOE_DEV float rcp(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Nearly all rows: the k-th largest of the lanes' largest keys is at most the k-th largest key, and few
// keys lie above it (about 10 for k = 8). These, each in a lane of its own and in the order of their
// indexes, are ranked by counting; with a bias or groups, keys closer than `near` are ranked again in
// 64 bits, one evaluation a lane.
// What bounds it is its instructions, a warp's per row, not what it reads: 65,536 rows of 512 bf16 logits
// with a bias and groups take 75 us, 910 instructions a row with 68% of the issue slots busy (all keys through k
// rounds of a warp: 457 us); 4,096 rows of 256 without 6 us.
template <int DT, int NPL, bool VEC, bool KEYED>
__global__ void __launch_bounds__(32 * kRouteWarps, 8) route_experts_kernel(const RouteParams p) {
  __shared__ double s_keys[kRouteWarps][32 * NPL];
  constexpr int kVec = NPL < 4 ? NPL : 4;
  __shared__ __align__(16) float s_bias[KEYED ? 32 * NPL : 4];   // [q / kVec][lane][kVec]
  __shared__ int s_list[kRouteWarps][32];
  __shared__ float s_sorted[kRouteWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* s_f = reinterpret_cast<float*>(s_keys[warp]);
  pdl_wait();
  pdl_launch_dependents();
  float largest_bias = 0.f;
  if (KEYED) {
    for (int i = threadIdx.x; i < 32 * NPL; i += 32 * kRouteWarps) {
      const int e = (i / kVec & 31) * NPL + i / (32 * kVec) * kVec + i % kVec;
      s_bias[i] = e >= p.E ? -INFINITY : p.bias ? load_bias(p.bias, e) : 0.f;   // past E: never chosen
    }
    __syncthreads();
    for (int i = lane; i < 32 * NPL; i += 32)
      if (s_bias[i] != -INFINITY) largest_bias = fmaxf(largest_bias, fabsf(s_bias[i]));
    largest_bias = warp_max(largest_bias);
  }
  // lanes a group has, where it is a run of 1, 2, 4, ... whole lanes
  const int run = p.per % NPL == 0 && ((p.per / NPL) & (p.per / NPL - 1)) == 0 ? p.per / NPL : 0;
  const uint32_t kOff = 0x007FFFFFu;   // the order key of -inf

  for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp; t < p.T; t += (int64_t)gridDim.x * kRouteWarps) {
    float c[NPL];
    const bool odd = __any_sync(0xFFFFFFFFu, !load_raw<DT, NPL, VEC>(p.logits, t * p.stride, p.E, lane, c));
    if (odd) load_logits<DT, NPL, VEC>(p.logits, t * p.stride, p.E, lane, c);
    bool slow = false;
    float m = 0.f, z = 1.f, near = 0.f;
    if (!p.sigmoid && (KEYED || !p.renormalise)) {   // c becomes the numerators; what is off or past E gives 0
      m = c[0];
#pragma unroll
      for (int q = 1; q < NPL; ++q) m = fmaxf(m, c[q]);
      m = fmaxf(warp_max(m), -FLT_MAX);   // also where nothing is on
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
      float bias[NPL];
#pragma unroll
      for (int q = 0; q < NPL; q += kVec) {
        const float* b = s_bias + (q * 32 + lane * kVec);
        if constexpr (kVec == 4) *reinterpret_cast<float4*>(bias + q) = *reinterpret_cast<const float4*>(b);
        else *reinterpret_cast<float2*>(bias + q) = *reinterpret_cast<const float2*>(b);
      }
      if (p.sigmoid) {
#pragma unroll
        for (int q = 0; q < NPL; ++q) c[q] = key_sigmoid(c[q]) + bias[q];
      } else {
        const float scale = 1.f / z;
#pragma unroll
        for (int q = 0; q < NPL; ++q) c[q] = fmaf(c[q], scale, bias[q]);
      }
      if (odd) {
        float x[NPL];
        load_logits<DT, NPL, VEC>(p.logits, t * p.stride, p.E, lane, x);
#pragma unroll
        for (int q = 0; q < NPL; ++q)
          if (x[q] == -INFINITY) c[q] = -INFINITY;
      }
    }

    float top = c[0];   // the lane's largest key among those that may be chosen
    if (!KEYED || p.groups == 1) {
#pragma unroll
      for (int q = 1; q < NPL; ++q) top = fmaxf(top, c[q]);
    } else {
      float a = -INFINITY, b = -INFINITY;   // lane g: the two largest keys of group g
      if (run) {
        a = c[0];
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
        a = __shfl_sync(0xFFFFFFFFu, a, (lane * run) & 31);
        b = __shfl_sync(0xFFFFFFFFu, b, (lane * run) & 31);
      } else {
        __syncwarp();
#pragma unroll
        for (int q = 0; q < NPL; ++q) s_f[lane * NPL + q] = c[q];
        __syncwarp();
        if (lane < p.groups)
          for (int i = 0; i < p.per; ++i) {
            const float v = s_f[lane * p.per + i];
            b = fmaxf(b, fminf(a, v));
            a = fmaxf(a, v);
          }
      }
      // a key of -inf adds nothing; two of the largest or lowest values leave no infinity, whose differences
      // from another are none
      const float score = p.group_top == 2 && b != -INFINITY ? fminf(fmaxf(a + b, -FLT_MAX), FLT_MAX) : a;
      bool close;
      uint32_t kept = choose_groups(p, score, near, lane, close);
      if (close) {
        slow = true;
        if (p.sigmoid) {
          if (run) {
            __syncwarp();
#pragma unroll
            for (int q = 0; q < NPL; ++q) s_f[lane * NPL + q] = c[q];
          }
          slow = !choose_groups_exactly<DT>(p, t, s_f, b, near, lane, s_list[warp], s_keys[warp] + 16 * NPL, &kept);
        }
      }
      if (run) {
        if (!(kept >> (lane / run) & 1u)) top = -INFINITY;
      } else {
        top = -INFINITY;
#pragma unroll
        for (int q = 0; q < NPL; ++q) {
          const int e = lane * NPL + q;
          if (e >= p.E || !(kept >> (e / p.per) & 1u)) c[q] = -INFINITY;
          top = fmaxf(top, c[q]);
        }
      }
    }

    // the short list
    uint32_t left = lane_key(top + 0.f, lane), bound = 0u;
    for (int r = 0; r < p.k; ++r) {
      bound = __reduce_max_sync(0xFFFFFFFFu, left);
      if (left == bound) left = 0u;
    }
    const float least = f32_from_order_key(max(bound & ~31u, kOff)) - near;
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
    slow |= (bound & ~31u) <= kOff || n > 32;

    int e = 0, rank = lane;   // the lane's expert, and its place among the chosen
    float v = 0.f;            // its logit
    if (!slow) {
      at -= count;
      __syncwarp();
      while (listed) {
        s_list[warp][at++] = lane * NPL + __ffs(listed) - 1;
        listed &= listed - 1;
      }
      __syncwarp();
      float key = -INFINITY, b = 0.f;
      rank = 32;
      if (lane < n) {
        e = s_list[warp][lane];
        v = fminf(load_one<DT>(p.logits, t * p.stride + e), FLT_MAX) + 0.f;   // the row is in L1
        if (KEYED) b = s_bias[(e % NPL / kVec * 32 + e / NPL) * kVec + e % kVec];
        key = !KEYED ? v : p.sigmoid ? key_sigmoid(v) + b : fmaf(expf(v - m), 1.f / z, b);
        rank = 0;
      }
#pragma unroll 4
      for (int o = 0; o < n; ++o) {
        const float w = __shfl_sync(0xFFFFFFFFu, key, o);
        rank += (w > key || (w == key && o < lane)) ? 1 : 0;   // lanes past n stay at 32 and more
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
#pragma unroll 1
            for (int o = 0; o < n; ++o) {
              const unsigned long long w = __shfl_sync(0xFFFFFFFFu, exact, o);
              rank += (w > exact || (w == exact && o < lane)) ? 1 : 0;
            }
          } else {   // the row's sum has to be exact too
            slow = true;
          }
        }
      }
    }
    if (slow) {
      e = route_exact<DT>(p, t, KEYED, s_keys[warp], lane);
      rank = lane;
      v = lane < p.k ? load_one<DT>(p.logits, t * p.stride + e) : 0.f;
      v = isnan(v) ? -INFINITY : fminf(v, FLT_MAX);
    }

    const bool mine = rank < p.k, on = mine && v != -INFINITY;
    float s = 0.f, w;
    if (p.renormalise) {
      // the scores' ratios alone count: e^(a - max a) / d with s = e^a / d, which no logit over- or underflows
      // (reciprocals by the approximate instruction, one unit in the last place off: weights within some 1e-7, about
      // twice what divisions leave, for fewer of the instructions that bound this kernel)
      const float a = on ? p.sigmoid ? fminf(v, 0.f) : v : -INFINITY;
      const float most = warp_max(a);
      if (on) s = expf(a - most);
      if (p.sigmoid) s *= rcp(1.f + expf(-fabsf(v)));
      const float sum = warp_sum(s);
      w = sum > 0.f ? p.scale * (s * rcp(sum)) : 0.f;
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
// logits are read then. All rows are written whole. 8,191 rows of 256 fp32: 7 us, most of it the rows'
// way through shared memory.
struct RouteBackParams {
  const void* logits;
  int64_t stride;
  const int* idx;
  const float* d_weights;
  void* d_logits;   // contiguous [T][E]
  int T, E, k, renormalise, sigmoid;
  float scale;
};

// Rounded to 16 bits, to nearest even; a NaN stays one.
template <int DT>
MOE_DEV uint32_t to_half(float v) {
  return DT == MOE_DTYPE_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}
template <int DT>
MOE_DEV void store_one(void* p, int64_t i, float v) {
  if (DT == MOE_DTYPE_F32) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = (uint16_t)to_half<DT>(v);
}

template <int DT, int NPL, bool VEC>
__global__ void __launch_bounds__(32 * kRouteWarps, 8) route_backward_kernel(const RouteBackParams p) {
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
      uint32_t off = 0u;   // they get 0 whatever the others' sum is
#pragma unroll
      for (int q = 0; q < NPL; ++q) {
        off |= x[q] == -INFINITY ? 1u << q : 0u;
        x[q] = x[q] == -INFINITY ? 0.f : expf(x[q] - m);
        z += x[q];
      }
      z = warp_sum(z);
      dot = warp_sum(on ? d * (expf(v - m) / z) : 0.f);   // on: z >= 1
#pragma unroll
      for (int q = 0; q < NPL; ++q) {
        const int i = lane * NPL + q;
        if (i < p.E) row[i] = off >> q & 1u ? 0.f : x[q] / z * (row[i] - dot);
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
            w[i] = to_half<DT>(row[8 * c + 2 * i]) | (to_half<DT>(row[8 * c + 2 * i + 1]) << 16);
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
  const int per_sm = 8;
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
