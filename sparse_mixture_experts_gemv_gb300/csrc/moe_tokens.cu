// Tokens in the order of their experts and back: dispatch, the weighted sum of the
// experts' results, and the gradients of both.
//
//   rows[pos[t, j]] = x[t]                       pos: a stable sort of the T k choices by expert
//   out[t] = sum_j w[t, j] y[pos[t, j]]
//   d_x[t] = sum_j d_rows[pos[t, j]]
//   d_y[pos[t, j]] = w[t, j] d_out[t],   d_w[t, j] = <d_out[t], y[pos[t, j]]>
//
// A choice of no expert (outside [0, E)) takes a place behind the last expert's rows, and
// pos holds ~place for it: so each of the T k rows belongs to one choice, every row of
// rows and d_y is written by the choice that owns it (with zeros, where there is no
// expert), and nothing has to be cleared. All of it moves bytes: memory bounds it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_common.cuh"
#include "moe_int8.h"
#include "moe_internal.h"

namespace moe {
namespace tokens {
namespace {

// ------------------------------------------------------------------------------- places
constexpr int kPlanThreads = 512;              // = choices of a segment
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanCtas = 8;                   // of the cluster that places many choices
constexpr int kBuckets = MOE_DISPATCH_MAX_EXPERTS + 1;   // the last one: no expert
constexpr int kFusedChoices = 2048;            // so many are placed by every CTA for itself

struct PlanShared {
  int hist[kBuckets];                          // choices of this CTA's part by expert
  int cursor[kBuckets];                        // the expert's next row
  uint8_t count[kPlanWarps][kBuckets + 3];     // a segment's choices by warp and expert
  int sums[kPlanWarps];
  int pos[kFusedChoices];
};

MOE_DEV int bucket_of(int e, int E) { return e >= 0 && e < E ? e : E; }

MOE_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
MOE_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
}
// The int at the same place of another CTA's shared memory.
MOE_DEV int remote(const int* p, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return (int)v;
}

// The rows of choices [a0, a1), which are this CTA's part of n: put(choice, row). Counts by expert, their sums over
// the parts and experts before, and then 512 choices at a time: a choice's rank is that within its warp (the lanes
// of the same expert below) plus the counts of the warps before it, a byte each, which keeps the order of the
// choices without a sort. CLUSTER: the parts are those of a cluster's CTAs.
template <bool CLUSTER, class Put>
MOE_DEV void place(PlanShared& s, const int* idx, int a0, int a1, int E, int* offsets, Put put) {
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
  for (int e = i; e <= E; e += kPlanThreads) s.hist[e] = 0;
  for (int c = i; c < (int)sizeof(s.count) / 4; c += kPlanThreads) reinterpret_cast<int*>(s.count)[c] = 0;
  __syncthreads();
#pragma unroll 8
  for (int a = a0 + i; a < a1; a += kPlanThreads) atomicAdd(&s.hist[bucket_of(__ldg(idx + a), E)], 1);
  if (CLUSTER) cluster_sync();
  else __syncthreads();
  // three consecutive experts a thread at most
  const int per = (E + kPlanThreads) / kPlanThreads, e0 = i * per;
  int total[3] = {}, before[3] = {}, sum = 0;
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    if (q >= per || e0 + q > E) continue;
    if constexpr (CLUSTER) {
      const uint32_t rank = cluster_rank();
#pragma unroll
      for (uint32_t r = 0; r < kPlanCtas; ++r) {
        const int v = remote(&s.hist[e0 + q], r);
        total[q] += v;
        before[q] += r < rank ? v : 0;
      }
    } else {
      total[q] = s.hist[e0 + q];
    }
    sum += total[q];
  }
  int upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) s.sums[warp] = upto;
  __syncthreads();
  int base = upto - sum;
  for (int w = 0; w < warp; ++w) base += s.sums[w];
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    if (q >= per || e0 + q > E) continue;
    s.cursor[e0 + q] = base + before[q];
    if (offsets) offsets[e0 + q] = base;       // offsets[E]: where the choices of no expert begin
    base += total[q];
  }
  if (CLUSTER) cluster_sync();                 // no CTA leaves while its counts are read
  else __syncthreads();
  for (int a = a0; a < a1; a += kPlanThreads) {
    const int at = a + i;
    const int e = at < a1 ? bucket_of(__ldg(idx + at), E) : -1;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
    const bool first = e >= 0 && (same & ((1u << lane) - 1)) == 0;
    if (first) s.count[warp][e] = (uint8_t)__popc(same);
    __syncthreads();
    if (e >= 0) {
      int row = s.cursor[e] + __popc(same & ((1u << lane) - 1));
      for (int w = 0; w < warp; ++w) row += s.count[w][e];
      put(at, e < E ? row : ~row);
    }
    __syncthreads();
    if (first) {
      atomicAdd(&s.cursor[e], __popc(same));
      s.count[warp][e] = 0;
    }
    __syncthreads();
  }
}

struct DispatchParams {
  const uint8_t* x;
  int64_t x_stride, row;     // bytes
  const float* x_scale;      // [T][scales] or NULL
  int scales;
  const int* idx;
  int T, k, E;
  uint8_t* rows;
  float* row_scale;
  int* offsets;
  int* pos;
};

// A vector of a row to its k places. `at`: the place of choice `lane`, ~place where there is no expert.
template <class V>
MOE_DEV void copy_piece(const DispatchParams& p, int64_t t, int64_t piece, int at, int lane) {
  constexpr int kU = sizeof(V) == 16 ? 4 : 8;
  const int64_t n = p.row / (int64_t)sizeof(V), v0 = piece * 32 * kU + lane;
  const V* src = reinterpret_cast<const V*>(p.x + t * p.x_stride);
  V v[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u)
    if (v0 + 32 * u < n) v[u] = __ldg(src + v0 + 32 * u);
  for (int j = 0; j < p.k; ++j) {
    const int r = __shfl_sync(0xFFFFFFFFu, at, j);
    V* dst = reinterpret_cast<V*>(p.rows + (int64_t)(r >= 0 ? r : ~r) * p.row);
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (v0 + 32 * u < n) dst[v0 + 32 * u] = r >= 0 ? v[u] : V{};
  }
  if (piece == 0 && p.x_scale)
    for (int c = lane; c - lane < p.scales; c += 32) {
      const float f = c < p.scales ? __ldg(p.x_scale + t * p.scales + c) : 0.f;
      for (int j = 0; j < p.k; ++j) {
        const int r = __shfl_sync(0xFFFFFFFFu, at, j);
        if (c < p.scales) p.row_scale[(int64_t)(r >= 0 ? r : ~r) * p.scales + c] = r >= 0 ? f : 0.f;
      }
    }
}
template <class V>
__host__ __device__ int64_t pieces_of(int64_t row) {
  const int64_t v = 32 * (sizeof(V) == 16 ? 4 : 8) * (int64_t)sizeof(V);
  return row > v ? (row + v - 1) / v : 1;
}

// Few choices: every CTA places all of them and copies its share of the rows.
template <class V>
__global__ void __launch_bounds__(kPlanThreads) dispatch_fused_kernel(const DispatchParams p) {
  __shared__ PlanShared s;
  pdl_wait();
  pdl_launch_dependents();
  const bool tells = blockIdx.x == 0;
  place<false>(s, p.idx, 0, p.T * p.k, p.E, tells ? p.offsets : nullptr, [&](int a, int row) {
    s.pos[a] = row;
    if (tells) p.pos[a] = row;
  });
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const int64_t pieces = pieces_of<V>(p.row), units = p.T * pieces;
  for (int64_t u = (int64_t)blockIdx.x * kPlanWarps + (threadIdx.x >> 5); u < units; u += (int64_t)gridDim.x * kPlanWarps) {
    const int64_t t = u / pieces;
    copy_piece<V>(p, t, u - t * pieces, lane < p.k ? s.pos[t * p.k + lane] : 0, lane);
  }
}

// Many choices: one cluster places them, each CTA an eighth.
__global__ void __launch_bounds__(kPlanThreads) __cluster_dims__(kPlanCtas, 1, 1) dispatch_plan_kernel(const DispatchParams p) {
  __shared__ PlanShared s;
  pdl_wait();
  pdl_launch_dependents();
  const int n = p.T * p.k, part = (n + kPlanCtas - 1) / kPlanCtas;
  const int a0 = min(n, (int)blockIdx.x * part), a1 = min(n, a0 + part);
  place<true>(s, p.idx, a0, a1, p.E, blockIdx.x == 0 ? p.offsets : nullptr, [&](int a, int row) { p.pos[a] = row; });
}

constexpr int kCopyThreads = 256;

// The rows, each token's read once.
template <class V>
__global__ void __launch_bounds__(kCopyThreads) dispatch_copy_kernel(const DispatchParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t pieces = pieces_of<V>(p.row), units = p.T * pieces;
  constexpr int kW = kCopyThreads / 32;
  for (int64_t u = (int64_t)blockIdx.x * kW + (threadIdx.x >> 5); u < units; u += (int64_t)gridDim.x * kW) {
    const int64_t t = u / pieces;
    copy_piece<V>(p, t, u - t * pieces, lane < p.k ? ldg_cg_s32(p.pos + t * p.k + lane) : 0, lane);
  }
}

// ------------------------------------------------------------------------ sums and gradients
// N consecutive values of type DT as fp32, and back, rounded once.
template <int DT, int N>
struct Pack {
  static constexpr int kBytes = N * (DT == MOE_DTYPE_F32 ? 4 : 2);
  uint32_t w[kBytes >= 4 ? kBytes / 4 : 1];
  MOE_DEV void load(const void* p, int64_t i) {
    const char* c = static_cast<const char*>(p) + i * (kBytes / N);
    if constexpr (kBytes == 16) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(c));
      w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    } else if constexpr (kBytes == 4) {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(c));
    } else {
      w[0] = __ldg(reinterpret_cast<const uint16_t*>(c));
    }
  }
  MOE_DEV void store(void* p, int64_t i) const {
    char* c = static_cast<char*>(p) + i * (kBytes / N);
    if constexpr (kBytes == 16) *reinterpret_cast<uint4*>(c) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (kBytes == 4) *reinterpret_cast<uint32_t*>(c) = w[0];
    else *reinterpret_cast<uint16_t*>(c) = (uint16_t)w[0];
  }
  MOE_DEV float get(int i) const {
    if constexpr (DT == MOE_DTYPE_F32) return __uint_as_float(w[i]);
    else if constexpr (DT == MOE_DTYPE_BF16) return i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    else return __half2float(__ushort_as_half((uint16_t)(w[i / 2] >> (16 * (i & 1)))));
  }
  MOE_DEV void set(const float (&f)[N]) {
    if constexpr (DT == MOE_DTYPE_F32) {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = __float_as_uint(f[i]);
    } else {
      uint16_t h[N];
#pragma unroll
      for (int i = 0; i < N; ++i)
        h[i] = DT == MOE_DTYPE_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(f[i])) : __half_as_ushort(__float2half_rn(f[i]));
      if constexpr (N == 1) w[0] = h[0];
      else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) w[i] = h[2 * i] | ((uint32_t)h[2 * i + 1] << 16);
      }
    }
  }
};

struct CombineParams {
  const void* y;             // [T k][H], row stride y_stride
  int64_t y_stride;
  const int* pos;
  const float* weights;      // NULL: 1
  void* out;
  const void* d_out;         // backward
  int64_t d_stride;
  void* d_y;                 // NULL: not wanted, likewise
  float* d_weights;
  int T, k, H;
};

constexpr int kMaxThreads = 256;
constexpr int kTogether = 8;   // choices whose rows are on their way at once

// out[t] = sum_j w y[pos], in 32 bits and in the order of the choices. One CTA a token.
template <int DT, int N>
__global__ void __launch_bounds__(kMaxThreads) combine_kernel(const CombineParams p) {
  __shared__ int s_at[MOE_ROUTE_MAX_TOP_K];
  __shared__ float s_w[MOE_ROUTE_MAX_TOP_K];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t rows = (int64_t)p.T * p.k;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    __syncthreads();
    for (int j = threadIdx.x; j < p.k; j += blockDim.x) {
      const int at = ldg_cg_s32(p.pos + t * p.k + j);
      s_at[j] = at < rows ? at : -1;
      s_w[j] = p.weights ? ldg_cg_f32(p.weights + t * p.k + j) : 1.f;
    }
    __syncthreads();
    for (int c = threadIdx.x * N; c < p.H; c += blockDim.x * N) {
      float acc[N] = {};
      for (int j0 = 0; j0 < p.k; j0 += kTogether) {
        Pack<DT, N> v[kTogether];
#pragma unroll
        for (int q = 0; q < kTogether; ++q)
          if (j0 + q < p.k && s_at[j0 + q] >= 0) v[q].load(p.y, s_at[j0 + q] * p.y_stride + c);
#pragma unroll
        for (int q = 0; q < kTogether; ++q)
          if (j0 + q < p.k && s_at[j0 + q] >= 0) {
            const float w = s_w[j0 + q];
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = fmaf(w, v[q].get(i), acc[i]);
          }
      }
      Pack<DT, N> o;
      o.set(acc);
      o.store(p.out, t * p.H + c);
    }
  }
}

// d_y[pos] = w d_out[t] and d_w = <d_out[t], y[pos]>, eight choices at a time: each thread adds up its columns, then
// the CTA adds the threads' sums, in a fixed order.
template <int DT, int N>
__global__ void __launch_bounds__(kMaxThreads) combine_backward_kernel(const CombineParams p) {
  __shared__ int s_at[MOE_ROUTE_MAX_TOP_K];
  __shared__ float s_w[MOE_ROUTE_MAX_TOP_K];
  __shared__ float s_sum[kMaxThreads / 32][kTogether];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t rows = (int64_t)p.T * p.k;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    __syncthreads();
    for (int j = threadIdx.x; j < p.k; j += blockDim.x) {
      const int at = ldg_cg_s32(p.pos + t * p.k + j);
      s_at[j] = at < rows && ~at < rows ? at : INT32_MAX;   // INT32_MAX: no row of y at all
      s_w[j] = p.weights ? ldg_cg_f32(p.weights + t * p.k + j) : 1.f;
    }
    __syncthreads();
    for (int j0 = 0; j0 < p.k; j0 += kTogether) {
      float dot[kTogether] = {};
      for (int c = threadIdx.x * N; c < p.H; c += blockDim.x * N) {
        Pack<DT, N> d, v[kTogether];
        d.load(p.d_out, t * p.d_stride + c);
        if (p.d_weights) {
#pragma unroll
          for (int q = 0; q < kTogether; ++q)
            if (j0 + q < p.k && (unsigned)s_at[j0 + q] < (unsigned)INT32_MAX) v[q].load(p.y, s_at[j0 + q] * p.y_stride + c);
        }
#pragma unroll
        for (int q = 0; q < kTogether; ++q) {
          if (j0 + q >= p.k) break;
          const int at = s_at[j0 + q];
          if (at == INT32_MAX) continue;
          if (p.d_weights && at >= 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) dot[q] = fmaf(d.get(i), v[q].get(i), dot[q]);
          }
          if (p.d_y) {
            const float w = s_w[j0 + q];
            float f[N];
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = at >= 0 ? w * d.get(i) : 0.f;
            Pack<DT, N> o;
            o.set(f);
            o.store(p.d_y, (int64_t)(at >= 0 ? at : ~at) * p.H + c);
          }
        }
      }
      if (!p.d_weights) continue;
#pragma unroll
      for (int q = 0; q < kTogether; ++q) {
        const float sum = warp_sum(dot[q]);
        if (lane == 0) s_sum[warp][q] = sum;
      }
      __syncthreads();
      if (threadIdx.x < kTogether && j0 + threadIdx.x < p.k) {
        float sum = 0.f;
        for (int w = 0; w < (int)blockDim.x / 32; ++w) sum += s_sum[w][threadIdx.x];
        p.d_weights[t * p.k + j0 + threadIdx.x] = sum;
      }
      __syncthreads();
    }
  }
}

// ------------------------------------------------------------------------------------ host
template <class K, class P>
cudaError_t launch(K kernel, int64_t grid, int block, cudaStream_t s, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(block);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <class V>
cudaError_t launch_dispatch(const DispatchParams& p, int sms, cudaStream_t s) {
  const int64_t units = p.T * pieces_of<V>(p.row);
  if ((int64_t)p.T * p.k <= kFusedChoices) {
    int64_t grid = (units + kPlanWarps - 1) / kPlanWarps;
    if (grid > 2 * sms) grid = 2 * sms;
    return launch(dispatch_fused_kernel<V>, grid < 1 ? 1 : grid, kPlanThreads, s, p);
  }
  cudaError_t e = launch(dispatch_plan_kernel, kPlanCtas, kPlanThreads, s, p);
  if (e != cudaSuccess) return e;
  constexpr int kW = kCopyThreads / 32;
  const int64_t want = (units + kW - 1) / kW, most = 8 * (int64_t)sms;
  return launch(dispatch_copy_kernel<V>, want < most ? want : most, kCopyThreads, s, p);
}

template <int DT, int N>
cudaError_t launch_combine(const CombineParams& p, bool backward, int sms, cudaStream_t s) {
  int threads = (int)((p.H + 32 * N - 1) / (32 * N)) * 32;
  if (threads > kMaxThreads) threads = kMaxThreads;
  const int64_t most = (int64_t)sms * 2048 / threads, grid = p.T < most ? p.T : most;
  return backward ? launch(combine_backward_kernel<DT, N>, grid, threads, s, p)
                  : launch(combine_kernel<DT, N>, grid, threads, s, p);
}
template <int DT>
cudaError_t launch_combine_dt(const CombineParams& p, bool wide, bool backward, cudaStream_t s) {
  const int sms = int8::device_sms();
  constexpr int kWide = DT == MOE_DTYPE_F32 ? 4 : 8;
  return wide ? launch_combine<DT, kWide>(p, backward, sms, s) : launch_combine<DT, 1>(p, backward, sms, s);
}
cudaError_t launch_combine_any(const CombineParams& p, int dtype, bool wide, bool backward, cudaStream_t s) {
  switch (dtype) {
    case MOE_DTYPE_F32: return launch_combine_dt<MOE_DTYPE_F32>(p, wide, backward, s);
    case MOE_DTYPE_BF16: return launch_combine_dt<MOE_DTYPE_BF16>(p, wide, backward, s);
    default: return launch_combine_dt<MOE_DTYPE_F16>(p, wide, backward, s);
  }
}

bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}
// Whether a call's counts are in range; *st is what it returns if not.
bool in_range(int32_t T, int32_t k, int64_t row, moe_status_t* st) {
  *st = T < 0 || k < 1 || row < 1 ? MOE_ERR_INVALID_ARG
        : k > MOE_ROUTE_MAX_TOP_K || (int64_t)T * k > INT32_MAX / 2 ? MOE_ERR_UNSUPPORTED : MOE_OK;
  return *st == MOE_OK;
}

}  // namespace
}  // namespace tokens
}  // namespace moe

extern "C" {

moe_status_t moe_dispatch_tokens(const void* x_dev, int64_t row_bytes, int64_t row_stride, const float* x_scale_dev,
                                 int32_t scales, const int32_t* idx_dev, int32_t T, int32_t k, int32_t E, void* rows_dev,
                                 float* row_scale_dev, int32_t* offsets_dev, int32_t* pos_dev, void* stream) {
  using namespace moe::tokens;
  moe_status_t st;
  if (!in_range(T, k, row_bytes, &st)) return st;
  if (E < 1 || scales < 0 || (T && ((scales > 0) != (x_scale_dev != nullptr) || (scales > 0) != (row_scale_dev != nullptr))))
    return MOE_ERR_INVALID_ARG;
  if (E > MOE_DISPATCH_MAX_EXPERTS || row_bytes > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
  if (!offsets_dev || (T && (!x_dev || !idx_dev || !rows_dev || !pos_dev || row_stride < row_bytes))) return MOE_ERR_INVALID_ARG;
  if (((uintptr_t)idx_dev | (uintptr_t)offsets_dev | (uintptr_t)pos_dev | (uintptr_t)x_scale_dev | (uintptr_t)row_scale_dev) & 3)
    return MOE_ERR_INVALID_ARG;
  const int64_t n = (int64_t)T * k;
  if (T && (overlap(x_dev, (T - 1) * row_stride + row_bytes, rows_dev, n * row_bytes) || overlap(idx_dev, n * 4, pos_dev, n * 4)))
    return MOE_ERR_INVALID_ARG;
  const DispatchParams p = {(const uint8_t*)x_dev, row_stride, row_bytes, x_scale_dev, scales, idx_dev, T, k, E,
                            (uint8_t*)rows_dev, row_scale_dev, offsets_dev, pos_dev};
  // the widest vector that every row starts and ends on
  const uint64_t a = (uintptr_t)x_dev | (uintptr_t)rows_dev | (uint64_t)row_bytes | (T > 1 ? (uint64_t)row_stride : 0);
  const int sms = moe::int8::device_sms();
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = !(a & 15) ? launch_dispatch<uint4>(p, sms, s) : !(a & 7) ? launch_dispatch<uint2>(p, sms, s)
                        : !(a & 3) ? launch_dispatch<uint32_t>(p, sms, s) : !(a & 1) ? launch_dispatch<uint16_t>(p, sms, s)
                        : launch_dispatch<uint8_t>(p, sms, s);
  return e == cudaSuccess ? MOE_OK : moe::record_cuda_failure(e, "moe_dispatch_tokens");
}

moe_status_t moe_combine_tokens(const void* y_dev, int32_t dtype, int64_t y_stride, const int32_t* pos_dev,
                                const float* weights_dev, int32_t T, int32_t k, int32_t H, void* out_dev, void* stream) {
  using namespace moe::tokens;
  moe_status_t st;
  if (!in_range(T, k, H, &st)) return st;
  if (dtype < MOE_DTYPE_F32 || dtype > MOE_DTYPE_F16) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  const int size = dtype == MOE_DTYPE_F32 ? 4 : 2;
  if (!y_dev || !pos_dev || !out_dev || y_stride < H) return MOE_ERR_INVALID_ARG;
  if (((uintptr_t)y_dev | (uintptr_t)out_dev) & (size - 1) || ((uintptr_t)pos_dev | (uintptr_t)weights_dev) & 3)
    return MOE_ERR_INVALID_ARG;
  if (overlap(y_dev, (((int64_t)T * k - 1) * y_stride + H) * size, out_dev, (int64_t)T * H * size)) return MOE_ERR_INVALID_ARG;
  CombineParams p = {};
  p.y = y_dev;
  p.y_stride = y_stride;
  p.pos = pos_dev;
  p.weights = weights_dev;
  p.out = out_dev;
  p.T = T;
  p.k = k;
  p.H = H;
  const bool wide = !(((uintptr_t)y_dev | (uintptr_t)out_dev | (uint64_t)(y_stride * size) | (uint64_t)((int64_t)H * size)) & 15);
  const cudaError_t e = launch_combine_any(p, dtype, wide, false, (cudaStream_t)stream);
  return e == cudaSuccess ? MOE_OK : moe::record_cuda_failure(e, "moe_combine_tokens");
}

moe_status_t moe_combine_tokens_backward(const void* d_out_dev, int64_t d_stride, const void* y_dev, int32_t dtype,
                                         int64_t y_stride, const int32_t* pos_dev, const float* weights_dev, int32_t T,
                                         int32_t k, int32_t H, void* d_y_dev, float* d_weights_dev, void* stream) {
  using namespace moe::tokens;
  moe_status_t st;
  if (!in_range(T, k, H, &st)) return st;
  if (dtype < MOE_DTYPE_F32 || dtype > MOE_DTYPE_F16) return MOE_ERR_INVALID_ARG;
  if (T == 0 || (!d_y_dev && !d_weights_dev)) return MOE_OK;
  const int size = dtype == MOE_DTYPE_F32 ? 4 : 2;
  if (!d_out_dev || !pos_dev || d_stride < H || (d_weights_dev && (!y_dev || y_stride < H))) return MOE_ERR_INVALID_ARG;
  if (((uintptr_t)d_out_dev | (uintptr_t)y_dev | (uintptr_t)d_y_dev) & (size - 1) ||
      ((uintptr_t)pos_dev | (uintptr_t)weights_dev | (uintptr_t)d_weights_dev) & 3)
    return MOE_ERR_INVALID_ARG;
  const int64_t n = (int64_t)T * k, dy = n * H * size;
  if (overlap(d_out_dev, ((T - 1) * d_stride + H) * size, d_y_dev, dy) ||
      (d_weights_dev && overlap(y_dev, ((n - 1) * y_stride + H) * size, d_y_dev, dy)))
    return MOE_ERR_INVALID_ARG;
  CombineParams p = {};
  p.y = y_dev;
  p.y_stride = y_stride;
  p.pos = pos_dev;
  p.weights = weights_dev;
  p.d_out = d_out_dev;
  p.d_stride = d_stride;
  p.d_y = d_y_dev;
  p.d_weights = d_weights_dev;
  p.T = T;
  p.k = k;
  p.H = H;
  uint64_t a = (uintptr_t)d_out_dev | (uintptr_t)d_y_dev | (uint64_t)(d_stride * size) | (uint64_t)((int64_t)H * size);
  if (d_weights_dev) a |= (uintptr_t)y_dev | (uint64_t)(y_stride * size);
  const cudaError_t e = launch_combine_any(p, dtype, !(a & 15), true, (cudaStream_t)stream);
  return e == cudaSuccess ? MOE_OK : moe::record_cuda_failure(e, "moe_combine_tokens_backward");
}

}  // extern "C"
