// 8-bit floating point (E4M3) with a scale for each block of 128: quantization of rows, a SwiGLU in the
// same pass if wanted, and the entry points of the products (moe_block8_gemm.cu).
//
//   scale[t, b] = amax over block b of row t times fp32(1/448), 1 where that is 0
//   q = E4M3(fp32(v / scale)),   v = x, or g / (1 + e^-g) u of the row's halves g and u
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_block8.cuh"
#include "moe_block8.h"
#include "moe_int8.h"
#include "moe_internal.h"

namespace moe {
namespace block8 {
namespace {

struct QuantizeParams {
  const void* x;
  int64_t stride;            // elements
  int T, K, blocks;
  uint8_t* q;                // [T][K]
  float* scale;              // [T][blocks]
};

constexpr int kThreads = 256;

// g / (1 + e^-g) * u. The quotient is the product with the approximate reciprocal, corrected once by the remainder (one
// step of Newton's; its sign as in divide(), for gates of -0): off by little more than its rounding. Below -80, where the
// reciprocal leaves the normal range, it is the division.
MOE_DEV void silu_mul(float (&g)[16], const float (&u)[16]) {
  float least = g[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) least = fminf(least, g[i]);
  if (least >= -80.f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float d = 1.f + expf(-g[i]);
      float y;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(d));
      const float q = g[i] * y;
      g[i] = fmaf(-fmaf(q, d, -g[i]), y, q) * u[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) g[i] = g[i] / (1.f + expf(-g[i])) * u[i];
  }
}

// Sixteen values a thread, eight threads a block of 128: its largest value comes from three exchanges, so that the
// rows are read once. The scale is a product with the rounded 1/448, and the quotient is rounded to fp32
// before E4M3: what elementary operations on tensors give, bit for bit. A block with an infinity or a NaN
// has the scale NaN, and with it NaN wherever it is used. Instructions bound it, 31 a value with SwiGLU: 32,768 x 512 bf16
// 22 us (with a division by the scale and one in the SwiGLU 28).
template <int DT, bool SWIGLU>
__global__ void __launch_bounds__(kThreads) block8_quantize_kernel(const QuantizeParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t per_row = (int64_t)p.blocks * 8, n = p.T * per_row;
  // whole warps take part in the exchanges: their last lanes may lie behind the end
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i - (threadIdx.x & 31) < n; i += (int64_t)gridDim.x * kThreads) {
    const int64_t t = n >> 32 ? i / per_row : (uint32_t)i / (uint32_t)per_row;   // a 64-bit division takes 100 instructions
    const int c = (int)(i - t * per_row) * 16;
    const bool in = i < n && c < p.K;
    float v[16] = {};
    if (in) {
      int8::load16<DT>(p.x, t * p.stride + c, v);
      if (SWIGLU) {
        float u[16];
        int8::load16<DT>(p.x, t * p.stride + p.K + c, u);
        silu_mul(v, u);
      }
    }
    const float scale = block_scale(v);
    if (!in) continue;
    *reinterpret_cast<uint4*>(p.q + t * p.K + c) = to_e4m3(v, scale);
    if (c % kBlock == 0) p.scale[t * p.blocks + c / kBlock] = scale;
  }
}

template <class K, class P>
cudaError_t launch(K kernel, int64_t grid, cudaStream_t s, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

cudaError_t launch_quantize(const QuantizeParams& p, int dtype, bool swiglu, cudaStream_t s) {
  const int64_t want = ((int64_t)p.T * p.blocks * 8 + kThreads - 1) / kThreads, most = 16 * (int64_t)int8::device_sms();
  const int64_t grid = want < most ? want : most;
  switch (dtype) {
    case MOE_DTYPE_F32:
      return swiglu ? launch(block8_quantize_kernel<MOE_DTYPE_F32, true>, grid, s, p)
                    : launch(block8_quantize_kernel<MOE_DTYPE_F32, false>, grid, s, p);
    case MOE_DTYPE_BF16:
      return swiglu ? launch(block8_quantize_kernel<MOE_DTYPE_BF16, true>, grid, s, p)
                    : launch(block8_quantize_kernel<MOE_DTYPE_BF16, false>, grid, s, p);
    default:
      return swiglu ? launch(block8_quantize_kernel<MOE_DTYPE_F16, true>, grid, s, p)
                    : launch(block8_quantize_kernel<MOE_DTYPE_F16, false>, grid, s, p);
  }
}

bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}
int size_of(int dtype) { return dtype == MOE_DTYPE_E4M3 ? 1 : dtype == MOE_DTYPE_F32 ? 4 : 2; }
int64_t pad256(int64_t v) { return (v + 255) / 256 * 256; }
int blocks_of(int n) { return tiles_of(n, kBlock); }
bool is_float(int dtype) { return dtype >= MOE_DTYPE_F32 && dtype <= MOE_DTYPE_F16; }

// Rows that come in another type are quantized to scratch: values, then scales. Few rows are quantized inside the product.
int64_t scratch(int64_t rows, int64_t K, int dtype) {
  return dtype == MOE_DTYPE_E4M3 || quantized_inside(rows, K) ? 0 : pad256(rows * K) + pad256(rows * blocks_of((int)K) * 4);
}

// rows, K and N in range, and whether there is anything to do (*st MOE_OK if it returns false)
moe_status_t check_product(int64_t rows, int K, int64_t N, int x_dtype, int out_dtype) {
  if (rows < 0 || N < 0 || K < 1 || (!is_float(x_dtype) && x_dtype != MOE_DTYPE_E4M3) || !is_float(out_dtype))
    return MOE_ERR_INVALID_ARG;
  return K % 16 || K > MOE_BLOCK_MAX_K ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe_status_t product(const void* x, int x_dtype, int64_t x_stride, const float* x_scale, GemmArgs& g, void* workspace,
                     int64_t workspace_bytes, void* stream, const char* what) {
  const int xs = size_of(x_dtype), os = size_of(g.out_dtype);
  const int64_t w_rows = (int64_t)g.groups * g.channels, out_bytes = (int64_t)g.rows * g.channels * os;
  if (!x || !g.w || !g.w_scale || !g.out || ((x_dtype == MOE_DTYPE_E4M3) != (x_scale != nullptr))) return MOE_ERR_INVALID_ARG;
  if (((uintptr_t)x | (uintptr_t)g.w) & 15 || ((uintptr_t)x_scale | (uintptr_t)g.w_scale | (uintptr_t)g.offsets) & 3 ||
      (uintptr_t)g.out & (os - 1))
    return MOE_ERR_INVALID_ARG;
  if (x_stride < g.K || g.w_stride < g.K || x_stride * xs % 16 || g.w_stride % 16) return MOE_ERR_INVALID_ARG;
  // a tensor map's strides have 40 bits, its extents 32; tiles are counted in 31
  if (x_stride * xs >= (int64_t)1 << 40 || g.w_stride >= (int64_t)1 << 40 || w_rows >= INT32_MAX ||
      ((int64_t)tiles_of(g.rows, 128) + g.groups) * tiles_of(g.channels, 64) >= INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  if (overlap(x, ((g.rows - 1) * x_stride + g.K) * xs, g.out, out_bytes) ||
      overlap(g.w, (w_rows - 1) * g.w_stride + g.K, g.out, out_bytes))
    return MOE_ERR_INVALID_ARG;
  const int64_t need = scratch(g.rows, g.K, x_dtype);
  if (need && (!workspace || workspace_bytes < need || (uintptr_t)workspace & 255)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  if (need) {
    QuantizeParams q = {};
    q.x = x;
    q.stride = x_stride;
    q.T = g.rows;
    q.K = g.K;
    q.blocks = blocks_of(g.K);
    q.q = (uint8_t*)workspace;
    q.scale = (float*)((uint8_t*)workspace + pad256((int64_t)g.rows * g.K));
    e = launch_quantize(q, x_dtype, false, s);
    g.early = 1;
    g.x_dtype = MOE_DTYPE_E4M3;
    g.x = q.q;
    g.x_stride = g.K;
    g.x_scale = q.scale;
  } else {
    g.x = x;
    g.x_dtype = x_dtype;
    g.x_stride = x_stride;
    g.x_scale = x_scale;
  }
  if (e == cudaSuccess) e = launch_gemm(g, int8::device_sms(), s);
  return e == cudaSuccess ? MOE_OK : record_cuda_failure(e, what);
}

}  // namespace
}  // namespace block8
}  // namespace moe

extern "C" {

moe_status_t moe_block_quantize(const void* x_dev, int32_t x_dtype, int64_t x_stride, int32_t swiglu, int32_t T, int32_t K,
                                void* q_dev, float* scale_dev, void* stream) {
  using namespace moe::block8;
  if (T < 0 || K < 1 || !is_float(x_dtype)) return MOE_ERR_INVALID_ARG;
  if (K % 16 || K > MOE_BLOCK_MAX_K) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  const int xs = size_of(x_dtype);
  const int64_t width = (int64_t)K * (swiglu ? 2 : 1);
  if (!x_dev || !q_dev || !scale_dev || ((uintptr_t)x_dev | (uintptr_t)q_dev) & 15 || (uintptr_t)scale_dev & 3 ||
      x_stride < width || x_stride * xs % 16)
    return MOE_ERR_INVALID_ARG;
  const int64_t xb = ((T - 1) * x_stride + width) * xs;
  if (overlap(x_dev, xb, q_dev, (int64_t)T * K) || overlap(x_dev, xb, scale_dev, (int64_t)T * blocks_of(K) * 4))
    return MOE_ERR_INVALID_ARG;
  const QuantizeParams p = {x_dev, x_stride, T, K, blocks_of(K), (uint8_t*)q_dev, scale_dev};
  const cudaError_t e = launch_quantize(p, x_dtype, swiglu != 0, (cudaStream_t)stream);
  return e == cudaSuccess ? MOE_OK : moe::record_cuda_failure(e, "moe_block_quantize");
}

moe_status_t moe_block_matmul_workspace(int32_t rows, int32_t K, int32_t x_dtype, int64_t* bytes) {
  using namespace moe::block8;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  const moe_status_t st = check_product(rows, K, 0, x_dtype, MOE_DTYPE_F32);
  if (st == MOE_OK) *bytes = scratch(rows, K, x_dtype);
  return st;
}

moe_status_t moe_block_matmul(const void* x_dev, int32_t x_dtype, int64_t x_stride, const float* x_scale_dev,
                              const void* w_dev, int64_t w_stride, const float* w_scale_dev, void* out_dev,
                              int32_t out_dtype, int32_t T, int32_t N, int32_t K, void* workspace_dev,
                              int64_t workspace_bytes, void* stream) {
  using namespace moe::block8;
  const moe_status_t st = check_product(T, K, N, x_dtype, out_dtype);
  if (st != MOE_OK || T == 0 || N == 0) return st;
  GemmArgs g = {};
  g.w = w_dev;
  g.w_stride = w_stride;
  g.w_scale = w_scale_dev;
  g.out = out_dev;
  g.out_dtype = out_dtype;
  g.rows = T;
  g.K = K;
  g.channels = N;
  g.groups = 1;
  return product(x_dev, x_dtype, x_stride, x_scale_dev, g, workspace_dev, workspace_bytes, stream, "moe_block_matmul");
}

moe_status_t moe_block_grouped_matmul(const void* x_dev, int32_t x_dtype, int64_t x_stride, const float* x_scale_dev,
                                      const int32_t* offsets_dev, const void* w_dev, const float* w_scale_dev,
                                      void* out_dev, int32_t out_dtype, int32_t M, int32_t E, int32_t N, int32_t K,
                                      void* workspace_dev, int64_t workspace_bytes, void* stream) {
  using namespace moe::block8;
  const moe_status_t st = check_product(M, K, N, x_dtype, out_dtype);
  if (st != MOE_OK) return st;
  if (E < 1) return MOE_ERR_INVALID_ARG;
  if (E > MOE_BLOCK_MAX_EXPERTS) return MOE_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return MOE_OK;
  if (!offsets_dev) return MOE_ERR_INVALID_ARG;
  GemmArgs g = {};
  g.w = w_dev;
  g.w_stride = K;
  g.w_scale = w_scale_dev;
  g.out = out_dev;
  g.out_dtype = out_dtype;
  g.rows = M;
  g.K = K;
  g.channels = N;
  g.groups = E;
  g.offsets = offsets_dev;
  return product(x_dev, x_dtype, x_stride, x_scale_dev, g, workspace_dev, workspace_bytes, stream, "moe_block_grouped_matmul");
}

void moe_block_test_force_wait_timeout(int32_t on) { moe::block8::test_withhold(on != 0); }

moe_status_t moe_block_sync_status(void* stream) {
  int code = 0;
  const cudaError_t e = moe::block8::gemm_status((cudaStream_t)stream, &code);
  if (e != cudaSuccess) return moe::record_cuda_failure(e, "moe_block_sync_status");
  return (moe_status_t)code;
}

}  // extern "C"
