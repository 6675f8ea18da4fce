// What the translation units of the 8-bit floating-point operators share on the host.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {
namespace block8 {

constexpr int kBlock = 128;   // values of a scale
constexpr int tiles_of(int n, int tile) { return (int)(((uint32_t)n + (uint32_t)tile - 1) / (uint32_t)tile); }   // any n >= 0

// Whether the product quantizes rows of other types itself, each CTA for itself: few values, which it keeps as an operand
// of 16 rows in shared memory. That saves a launch, 6 us of a call that no graph holds, while that call is bound by its
// host; on the device it takes some 1.5 us for each 10,000 values, a launch of its own 1.5 to 2 us. GB300, bf16, us on the
// device (in a graph), inside / by a launch:
//   values   8,192  8 x 1,024 x 1,024 5.1 / 5.6      10,240  4 x 2,560 x 4,096 7.5 / 8.0
//           20,480  8 x 2,560 x 4,096 8.9 / 8.0, 16 x 1,280 x 1,024 7.4 / 6.2, 8 x 2,560 x 157,184 69 / 67
//           32,768  16 x 2,048 x 4,096 10.2 / 7.2    65,536  16 x 4,096 x 4,096 17.3 / 10.3
// and a call outside of graphs up to 16,384 channels 13-15 / 19-20 up to 32,768 values, 17-19 / 19-20 with 65,536. So the
// device alone would stop at some 10,000 values and the call past 32,768: the limit is between them, where a graph loses
// 1.4 us at most.
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
