// Products and SwiGLU experts in 8-bit integers, for few tokens: the weights are
// streamed once and multiplied on the integer dot-product units.
//
//   out[t, n] = (sum_k q[t, k] w[n, k]) x_scale[t] w_scale[n]
//
// With few tokens a weight byte meets few activations, so reading the weights is
// what bounds these kernels. Every CTA quantizes the tokens for itself (a few KB
// from L2) and keeps them in shared memory as bytes; a warp then takes four rows of
// weights at a time in 16-byte loads that bypass L1, four dp4a a load and token,
// and adds the lanes' integer sums with one redux a row and token: exact.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "moe_int8.cuh"
#include "moe_internal.h"

namespace moe {
namespace int8 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxStreamT = 8;                // tokens of a CTA
constexpr int kRows = 4;                      // weight rows of a warp at a time
constexpr size_t kMaxTokenSmem = 96 * 1024;   // quantized tokens of a CTA

template <int DT>
MOE_DEV void quantize_rows_to_smem(const void* x, int64_t stride, const float* x_scale, int T, int K, uint4* q,
                                   float* scale, uint32_t (*red)[kMaxStreamT]) {
  const int nch = K / 16;
  if constexpr (DT == MOE_DTYPE_S8) {
    for (int t = 0; t < T; ++t)
      for (int c = threadIdx.x; c < nch; c += kThreads)
        q[t * nch + c] = __ldg(reinterpret_cast<const uint4*>(static_cast<const int8_t*>(x) + t * stride) + c);
    if (threadIdx.x < T) scale[threadIdx.x] = x_scale[threadIdx.x];
  } else {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float v[16];
    for (int t = 0; t < T; ++t) {
      uint32_t a = 0;
      for (int c = threadIdx.x; c < nch; c += kThreads) {
        load16<DT>(x, t * stride + 16 * c, v);
        a = max(a, amax_bits(v));
      }
      a = __reduce_max_sync(0xFFFFFFFFu, a);
      if (lane == 0) red[warp][t] = a;
    }
    __syncthreads();
    for (int t = 0; t < T; ++t) {
      uint32_t a = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) a = max(a, red[w][t]);
      const RowScale r = row_scale(a);
      for (int c = threadIdx.x; c < nch; c += kThreads) {
        load16<DT>(x, t * stride + 16 * c, v);
        q[t * nch + c] = quantize16(v, r);
      }
      if (threadIdx.x == 0) scale[t] = r.scale;
    }
  }
}

// Integer sums of `R` rows (p[r], K bytes each) with T tokens in shared memory,
// complete in every lane.
template <int T, int R>
MOE_DEV void dot_rows(const int8_t* const (&p)[R], const uint4* q, int nch, int lane, int (&acc)[R][T]) {
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < T; ++t) acc[r][t] = 0;
#pragma unroll 2
  for (int c = lane; c < nch; c += 32) {
    uint4 w[R];
#pragma unroll
    for (int r = 0; r < R; ++r) w[r] = ldg_stream(p[r] + 16 * c);
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const uint4 xv = q[t * nch + c];
#pragma unroll
      for (int r = 0; r < R; ++r) acc[r][t] = dot16(w[r], xv, acc[r][t]);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < T; ++t) acc[r][t] = __reduce_add_sync(0xFFFFFFFFu, acc[r][t]);
}

// ------------------------------------------------------------------ dense product
struct StreamParams {
  const void* x;
  int64_t x_stride;
  const float* x_scale;
  const int8_t* w;
  int64_t w_stride;
  const float* w_scale;
  void* out;
  int out_dtype, T, N, K;
};

template <int DT, int T>
__global__ void __launch_bounds__(kThreads, T >= 4 ? 2 : 3) int8_stream_kernel(const StreamParams p) {
  extern __shared__ uint4 q[];   // [T][K / 16]
  __shared__ uint32_t red[kWarps][kMaxStreamT];
  __shared__ float s_scale[kMaxStreamT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = blockIdx.y * T, nt = min(T, p.T - t0);
  const int nch = p.K / 16;
  pdl_wait();
  pdl_launch_dependents();
  const int size = DT == MOE_DTYPE_S8 ? 1 : DT == MOE_DTYPE_F32 ? 4 : 2;
  quantize_rows_to_smem<DT>(static_cast<const char*>(p.x) + t0 * p.x_stride * size, p.x_stride,
                            p.x_scale ? p.x_scale + t0 : nullptr, nt, p.K, q, s_scale, red);
  for (int i = threadIdx.x + nt * nch; i < T * nch; i += kThreads) q[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  for (int64_t n0 = ((int64_t)blockIdx.x * kWarps + warp) * kRows; n0 < p.N; n0 += (int64_t)gridDim.x * kWarps * kRows) {
    const int8_t* rows[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) rows[r] = p.w + min(n0 + r, (int64_t)p.N - 1) * p.w_stride;
    int acc[kRows][T];
    dot_rows<T, kRows>(rows, q, nch, lane, acc);
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int t = 0; t < T; ++t)
        if (lane == r * T + t && n0 + r < p.N && t < nt)
          store(p.out, p.out_dtype, (int64_t)(t0 + t) * p.N + n0 + r,
                (float)acc[r][t] * s_scale[t] * __ldg(p.w_scale + n0 + r));
  }
}

template <int DT, int T>
cudaError_t launch_stream_t(const StreamParams& p, int num_sms, cudaStream_t s) {
  const size_t smem = (size_t)T * p.K;
  static int allowed[64] = {};   // dynamic shared memory granted so far, by device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (smem > 40 * 1024 && (dev >= 64 || allowed[dev] < (int)smem)) {
    e = cudaFuncSetAttribute(int8_stream_kernel<DT, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(kMaxTokenSmem > smem ? kMaxTokenSmem : smem));
    if (e != cudaSuccess) return e;
    if (dev < 64) allowed[dev] = (int)(kMaxTokenSmem > smem ? kMaxTokenSmem : smem);
  }
  const int64_t blocks = (p.N + kWarps * kRows - 1) / (kWarps * kRows);
  const int chunks = (p.T + T - 1) / T;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks < num_sms * 4 ? blocks : num_sms * 4), chunks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, int8_stream_kernel<DT, T>, p);
}

template <int DT>
cudaError_t launch_stream_dt(const StreamParams& p, int num_sms, cudaStream_t s) {
  // tokens a CTA holds: as many as there are, up to 8, while they fit its shared memory
  int t = p.T >= 5 ? 8 : p.T >= 3 ? 4 : p.T;
  while (t > 1 && (size_t)t * p.K > kMaxTokenSmem) t /= 2;
  switch (t) {
    case 1: return launch_stream_t<DT, 1>(p, num_sms, s);
    case 2: return launch_stream_t<DT, 2>(p, num_sms, s);
    case 4: return launch_stream_t<DT, 4>(p, num_sms, s);
    default: return launch_stream_t<DT, 8>(p, num_sms, s);
  }
}

// ---------------------------------------------------------------------- experts
struct ExpertsParams {
  const void* x;
  const int* idx;
  const float* weights;
  const int8_t* gate_up;
  const float* gate_up_scale;
  const int8_t* down;
  const float* down_scale;
  void* out;
  float* h;      // fp32 [T * k][I]
  int T, k, E, H, I, out_dtype;
};

constexpr int kFeatures = 2 * kWarps;   // intermediate features of a CTA: two a warp (four rows)

// h of one choice (blockIdx.y) and kFeatures features.
template <int DT>
__global__ void __launch_bounds__(kThreads, 3) int8_experts_up_kernel(const ExpertsParams p) {
  extern __shared__ uint4 q[];   // [H / 16]
  __shared__ uint32_t red[kWarps][kMaxStreamT];
  __shared__ float s_scale[kMaxStreamT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t a = blockIdx.y; a < (int64_t)p.T * p.k; a += gridDim.y) {
    const int e = __ldg(p.idx + a);
    if (e < 0 || e >= p.E) continue;
    __syncthreads();
    quantize_rows_to_smem<DT>(static_cast<const uint16_t*>(p.x) + a / p.k * p.H, p.H, nullptr, 1, p.H, q, s_scale, red);
    __syncthreads();
    const int f0 = blockIdx.x * kFeatures + 2 * warp;
    if (f0 >= p.I) continue;
    const int f1 = min(f0 + 1, p.I - 1);
    const int64_t row0 = (int64_t)e * 2 * p.I;
    const int8_t* rows[4] = {p.gate_up + (row0 + f0) * p.H, p.gate_up + (row0 + p.I + f0) * p.H,
                             p.gate_up + (row0 + f1) * p.H, p.gate_up + (row0 + p.I + f1) * p.H};
    int acc[4][1];
    dot_rows<1, 4>(rows, q, p.H / 16, lane, acc);
    if (lane < 2 && f0 + lane < p.I) {
      const float* ws = p.gate_up_scale + row0 + f0 + lane;
      const float g = (float)(lane ? acc[2][0] : acc[0][0]) * s_scale[0] * __ldg(ws);
      const float u = (float)(lane ? acc[3][0] : acc[1][0]) * s_scale[0] * __ldg(ws + p.I);
      p.h[a * p.I + f0 + lane] = swiglu(g, u);
    }
  }
}

constexpr int kDownThreads = 128;
constexpr int kDownChannels = 2 * (kDownThreads / 32);
constexpr int kMaxChoices = MOE_ROUTE_MAX_TOP_K;

// out of one token (blockIdx.y) and kDownChannels channels, all its choices.
// Dynamic shared memory: `held` quantized rows of h.
__global__ void __launch_bounds__(kDownThreads, 6) int8_experts_down_kernel(const ExpertsParams p, int held) {
  extern __shared__ uint4 q[];   // [held][I / 16]
  __shared__ float s_scale[kMaxChoices];
  __shared__ int s_e[kMaxChoices];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nch = p.I / 16;
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t t = blockIdx.y; t < p.T; t += gridDim.y) {
    const int c0 = blockIdx.x * kDownChannels + 2 * warp, c1 = min(c0 + 1, p.H - 1);
    float sum0 = 0.f, sum1 = 0.f;
    for (int j0 = 0; j0 < p.k; j0 += held) {
      const int nj = min(held, p.k - j0);
      __syncthreads();
      for (int j = warp; j < nj; j += kDownThreads / 32) {
        const int64_t a = t * p.k + j0 + j;
        int e = __ldg(p.idx + a);
        if (e < 0 || e >= p.E) e = -1;
        if (e >= 0) {
          float v[16];
          uint32_t m = 0;
          for (int c = lane; c < nch; c += 32) {
            load16_cg(p.h + a * p.I + 16 * c, v);
            m = max(m, amax_bits(v));
          }
          const RowScale r = row_scale(__reduce_max_sync(0xFFFFFFFFu, m));
          for (int c = lane; c < nch; c += 32) {
            load16_cg(p.h + a * p.I + 16 * c, v);
            q[j * nch + c] = quantize16(v, r);
          }
          if (lane == 0) s_scale[j] = r.scale * __ldg(p.weights + a);
        }
        if (lane == 0) s_e[j] = e;
      }
      __syncthreads();
      if (c0 < p.H) {
        float ws0 = 0.f, ws1 = 0.f;   // lane j: the scales of choice j
        if (lane < nj && s_e[lane] >= 0) {
          ws0 = s_scale[lane] * __ldg(p.down_scale + (int64_t)s_e[lane] * p.H + c0);
          ws1 = s_scale[lane] * __ldg(p.down_scale + (int64_t)s_e[lane] * p.H + c1);
        }
#pragma unroll 4
        for (int j = 0; j < nj; ++j) {
          const int e = s_e[j];
          const float f0 = __shfl_sync(0xFFFFFFFFu, ws0, j), f1 = __shfl_sync(0xFFFFFFFFu, ws1, j);
          if (e < 0) continue;
          const int8_t* r0 = p.down + ((int64_t)e * p.H + c0) * p.I;
          const int8_t* r1 = p.down + ((int64_t)e * p.H + c1) * p.I;
          int a0 = 0, a1 = 0;
          for (int c = lane; c < nch; c += 32) {
            const uint4 w0 = ldg_stream(r0 + 16 * c), w1 = ldg_stream(r1 + 16 * c), xv = q[j * nch + c];
            a0 = dot16(w0, xv, a0);
            a1 = dot16(w1, xv, a1);
          }
          sum0 += (float)a0 * f0;
          sum1 += (float)a1 * f1;
        }
      }
    }
    sum0 = warp_sum(sum0);
    sum1 = warp_sum(sum1);
    if (lane < 2 && c0 + lane < p.H) store(p.out, p.out_dtype, t * p.H + c0 + lane, lane ? sum1 : sum0);
  }
}

template <class K, class... A>
cudaError_t launch_pdl(K kernel, dim3 grid, int block, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_experts_stream(const ExpertsParams& p, int x_dtype, cudaStream_t s) {
  const int64_t choices = (int64_t)p.T * p.k;
  const dim3 up((p.I + kFeatures - 1) / kFeatures, (unsigned)(choices < 65535 ? choices : 65535));
  cudaError_t e = x_dtype == MOE_DTYPE_BF16
                      ? launch_pdl(int8_experts_up_kernel<MOE_DTYPE_BF16>, up, kThreads, (size_t)p.H, s, p)
                      : launch_pdl(int8_experts_up_kernel<MOE_DTYPE_F16>, up, kThreads, (size_t)p.H, s, p);
  if (e != cudaSuccess) return e;
  int held = 32 * 1024 / p.I;   // rows of h a CTA keeps: 32 KB, so that several CTAs share an SM
  held = held < 1 ? 1 : held < p.k ? held : p.k;
  const dim3 down((p.H + kDownChannels - 1) / kDownChannels, (unsigned)(p.T < 65535 ? p.T : 65535));
  return launch_pdl(int8_experts_down_kernel, down, kDownThreads, (size_t)held * p.I, s, p, held);
}

int device_sms() {
  static int sms[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  if (!sms[dev] && cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 152;
  return sms[dev];
}

bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

int dtype_size(int d) { return d == MOE_DTYPE_S8 ? 1 : d == MOE_DTYPE_F32 ? 4 : 2; }
int64_t pad256(int64_t v) { return (v + 255) / 256 * 256; }

}  // namespace
}  // namespace int8
}  // namespace moe

extern "C" {

moe_status_t moe_quant_matmul_workspace(int32_t T, int32_t N, int32_t K, int32_t x_dtype, int64_t* bytes) {
  if (!bytes || T < 0 || N < 0 || K < 1 || x_dtype < MOE_DTYPE_F32 || x_dtype > MOE_DTYPE_S8) return MOE_ERR_INVALID_ARG;
  *bytes = 0;
  return MOE_OK;
}

moe_status_t moe_quant_matmul(const void* x_dev, int32_t x_dtype, int64_t x_stride, const float* x_scale_dev,
                             const int8_t* w_dev, int64_t w_stride, const float* w_scale_dev, void* out_dev,
                             int32_t out_dtype, int32_t T, int32_t N, int32_t K, void* workspace_dev,
                             int64_t workspace_bytes, void* stream) {
  using namespace moe::int8;
  (void)workspace_dev;
  (void)workspace_bytes;
  if (T < 0 || N < 0 || K < 1) return MOE_ERR_INVALID_ARG;
  if (x_dtype < MOE_DTYPE_F32 || x_dtype > MOE_DTYPE_S8 || out_dtype < MOE_DTYPE_F32 || out_dtype > MOE_DTYPE_F16)
    return MOE_ERR_INVALID_ARG;
  if (K % 16 || K > MOE_INT8_MAX_K) return MOE_ERR_UNSUPPORTED;
  if (T == 0 || N == 0) return MOE_OK;
  const int xs = dtype_size(x_dtype), os = dtype_size(out_dtype);
  if (!x_dev || !w_dev || !w_scale_dev || !out_dev || ((x_dtype == MOE_DTYPE_S8) != (x_scale_dev != nullptr)))
    return MOE_ERR_INVALID_ARG;
  if (((uintptr_t)x_dev | (uintptr_t)w_dev) & 15 || ((uintptr_t)w_scale_dev | (uintptr_t)x_scale_dev) & 3 ||
      (uintptr_t)out_dev & (os - 1))
    return MOE_ERR_INVALID_ARG;
  if (x_stride < K || w_stride < K || x_stride * xs % 16 || w_stride % 16) return MOE_ERR_INVALID_ARG;
  if (overlap(x_dev, ((T - 1) * x_stride + K) * xs, out_dev, (int64_t)T * N * os) ||
      overlap(w_dev, (N - 1) * w_stride + K, out_dev, (int64_t)T * N * os))
    return MOE_ERR_INVALID_ARG;
  const StreamParams p = {x_dev, x_stride, x_scale_dev, w_dev, w_stride, w_scale_dev, out_dev, out_dtype, T, N, K};
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  switch (x_dtype) {
    case MOE_DTYPE_F32: e = launch_stream_dt<MOE_DTYPE_F32>(p, device_sms(), s); break;
    case MOE_DTYPE_BF16: e = launch_stream_dt<MOE_DTYPE_BF16>(p, device_sms(), s); break;
    case MOE_DTYPE_F16: e = launch_stream_dt<MOE_DTYPE_F16>(p, device_sms(), s); break;
    default: e = launch_stream_dt<MOE_DTYPE_S8>(p, device_sms(), s); break;
  }
  return e == cudaSuccess ? MOE_OK : moe::record_cuda_failure(e, "moe_quant_matmul");
}

moe_status_t moe_quant_experts_workspace(const moe_int8_experts_config_t* c, int32_t T, int64_t* bytes) {
  using namespace moe::int8;
  if (!c || !bytes || T < 0) return MOE_ERR_INVALID_ARG;
  if (c->num_experts < 1 || c->top_k < 1 || c->hidden < 1 || c->intermediate < 1) return MOE_ERR_INVALID_ARG;
  if (c->hidden % 16 || c->intermediate % 16 || c->hidden > 16384 || c->intermediate > 16384 ||
      c->top_k > MOE_ROUTE_MAX_TOP_K || c->num_experts > MOE_INT8_MAX_EXPERTS)
    return MOE_ERR_UNSUPPORTED;
  *bytes = pad256((int64_t)T * c->top_k * c->intermediate * 4);
  return MOE_OK;
}

moe_status_t moe_quant_experts(const moe_int8_experts_config_t* c, const moe_int8_experts_weights_t* w,
                              const void* x_dev, int32_t x_dtype, const int32_t* idx_dev, const float* weights_dev,
                              void* out_dev, int32_t T, void* workspace_dev, int64_t workspace_bytes, void* stream) {
  using namespace moe::int8;
  int64_t need = 0;
  const moe_status_t st = moe_quant_experts_workspace(c, T, &need);
  if (st != MOE_OK) return st;
  if (x_dtype != MOE_DTYPE_BF16 && x_dtype != MOE_DTYPE_F16) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!w || !w->gate_up_dev || !w->gate_up_scale_dev || !w->down_dev || !w->down_scale_dev || !x_dev || !idx_dev ||
      !weights_dev || !out_dev || !workspace_dev || workspace_bytes < need)
    return MOE_ERR_INVALID_ARG;
  if (((uintptr_t)x_dev | (uintptr_t)out_dev | (uintptr_t)w->gate_up_dev | (uintptr_t)w->down_dev) & 15 ||
      ((uintptr_t)idx_dev | (uintptr_t)weights_dev | (uintptr_t)w->gate_up_scale_dev | (uintptr_t)w->down_scale_dev) & 3 ||
      (uintptr_t)workspace_dev & 255)
    return MOE_ERR_INVALID_ARG;
  const int64_t xb = (int64_t)T * c->hidden * 2;
  if (overlap(x_dev, xb, out_dev, xb)) return MOE_ERR_INVALID_ARG;
  ExpertsParams p = {};
  p.x = x_dev;
  p.idx = idx_dev;
  p.weights = weights_dev;
  p.gate_up = w->gate_up_dev;
  p.gate_up_scale = w->gate_up_scale_dev;
  p.down = w->down_dev;
  p.down_scale = w->down_scale_dev;
  p.out = out_dev;
  p.h = (float*)workspace_dev;
  p.T = T;
  p.k = c->top_k;
  p.E = c->num_experts;
  p.H = c->hidden;
  p.I = c->intermediate;
  p.out_dtype = x_dtype;
  const cudaError_t e = launch_experts_stream(p, x_dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? MOE_OK : moe::record_cuda_failure(e, "moe_quant_experts");
}

}  // extern "C"
