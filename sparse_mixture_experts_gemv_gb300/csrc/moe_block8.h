// What the translation units of the 8-bit floating-point operators share on the host.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {
namespace block8 {

constexpr int kBlock = 128;   // values of a scale

// One launch of the product. Rows E4M3 [rows][K] with scales [rows][blocks of K]; weights E4M3
// [groups * channels][K] with scales [groups][blocks of channels][blocks of K]. Strides in bytes.
struct GemmArgs {
  const void* x;
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
