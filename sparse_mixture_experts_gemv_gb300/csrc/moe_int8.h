// What the 8-bit operators' translation units share on the host.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {
namespace int8 {

constexpr int kMaxBlock = 192;   // tokens of a tensor-core tile: two accumulators of so many columns
                                 // and two operand slots fill tensor memory

enum GemmKind { kDense = 0, kUp = 1, kDown = 2 };

// One launch of the tensor-core product. Weights [a_rows][K] bytes (row stride
// a_stride), tokens f16 [b_rows][K] whole numbers, each row padded with zeros to b_stride
// elements, a multiple of 64.
struct GemmArgs {
  const void* a;
  int64_t a_rows, a_stride;
  const void* b;
  int64_t b_rows, b_stride;
  int K;
  int channels;               // outputs of a group: N; I (up); H (down)
  int rows_per_group;         // weight rows of an expert (0 when dense)
  int block;                  // tokens of a tile at most, a multiple of 16
  // grouped: blocks of rows, written on the device: (expert, first row, rows, 0)
  const int4* blocks;
  const int* num_blocks;
  int max_blocks;
  int T;                      // dense: tokens
  const float* row_scale;     // dense, up: scale of each row of b
  const float* w_scale;       // dense: [N]; up: [E][2I]; down: [E][H]
  void* out;                  // dense: [T][N] out_dtype; up: fp32 h [rows][I]; down: fp32 y [rows][H]
  int out_dtype;              // dense
};
int device_sms();   // of the current device
cudaError_t launch_gemm(GemmKind kind, const GemmArgs& a, int num_sms, cudaStream_t s);
void test_withhold(int on);   // test only: products launched by this thread get no tokens
cudaError_t gemm_status(cudaStream_t s, int* code);   // synchronises; reads and clears the device's error word

}  // namespace int8
}  // namespace moe
