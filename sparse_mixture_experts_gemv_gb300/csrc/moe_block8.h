// What the translation units of the 8-bit floating-point operators share on the host.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {
namespace block8 {

constexpr int kBlock = 128;   // values of a scale
constexpr int tiles_of(int n, int tile) { return (int)(((uint32_t)n + (uint32_t)tile - 1) / (uint32_t)tile); }   // any n >= 0

// Whether the product quantizes rows of other types itself, each CTA for itself: few values, which it keeps as an operand
// of 16 rows in shared memory. That saves a launch, some 5 us of a call, and takes 4 us for 32,768 values. GB300, us on the
// device and a call, inside / by a launch: 1 x 2,048 x 1,024 6.0, 11 / 7.2, 17; 1 x 2,560 x 157,184 64, 65 / 69, 68;
// 8 x 2,560 x 157,184 69, 69 / 69, 70; 16 x 2,048 x 4,096 10, 12 / 7, 17; 16 x 4,096 x 16,384 19, 19 / 12, 17.
constexpr bool quantized_inside(int64_t rows, int64_t K) { return rows <= 16 && K <= 4096 && rows * K <= 20480; }

// One launch of the product. Rows E4M3 [rows][K] with scales [rows][blocks of K]; weights E4M3
// [groups * channels][K] with scales [groups][blocks of channels][blocks of K]. Strides in
// elements.
struct GemmArgs {
  const void* x;
  int x_dtype;               // not E4M3: quantized_inside() rows, x_scale NULL
  int64_t x_stride;
  const float* x_scale;
  const void* w;
  int64_t w_stride;
  const float* w_scale;
  void* out;                 // [rows][channels] out_dtype
  int out_dtype;
  int rows, K, channels, groups;
  const int* offsets;        // [groups + 1] on the device, or NULL: one group of all rows
  int early;                 // the kernel before wrote x and x_scale, had waited for those before it, and nothing else
};
cudaError_t launch_gemm(const GemmArgs& a, int num_sms, cudaStream_t s);
void test_withhold(int on);   // test only: products launched by this thread get no rows
cudaError_t gemm_status(cudaStream_t s, int* code);   // synchronises; reads and clears the device's error word

}  // namespace block8
}  // namespace moe
