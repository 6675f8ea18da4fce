// Products and SwiGLU experts in 8-bit integers: the entry points, the kernels for few
// tokens, which stream the weights once through the integer dot-product units, and what
// goes around the tensor-core products of many tokens (moe_int8_gemm.cu).
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
#include "moe_int8.h"
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
#pragma unroll T == 1 ? 4 : 2
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

// CTAs an SM holds at once, by tokens: what their accumulators and loads in flight leave of the registers.
constexpr int stream_ctas(int tokens) { return tokens >= 4 ? 2 : 3; }

// 157,184 x 2,560 and one token: 58.6 us, 6.9 TB/s of weights and results, the rate of a copy; 1,024 x
// 2,048: 6 us, of which the launch and the token's quantization are most.
template <int DT, int T>
__global__ void __launch_bounds__(kThreads, stream_ctas(T)) int8_stream_kernel(const StreamParams p) {
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
  const int64_t resident = num_sms * stream_ctas(T);   // each quantizes the tokens once and takes many rows
  cfg.gridDim = dim3((unsigned)(blocks < resident ? blocks : resident), chunks);
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

// h of one choice (blockIdx.y) and kFeatures features. As soon as the expert is known its rows are
// requested into L2, two contiguous pieces: they come while the token is being quantized. Ling-shaped, T = 4:
// 24 us for 115 MB of distinct rows, 4.8 TB/s (31 us without the request); Qwen-shaped, T = 1: 8 us, latency.
template <int DT>
__global__ void __launch_bounds__(kThreads, 3) int8_experts_up_kernel(const ExpertsParams p) {
  extern __shared__ uint4 q[];   // [H / 16]
  __shared__ uint32_t red[kWarps][kMaxStreamT];
  __shared__ float s_scale[kMaxStreamT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t a = blockIdx.y;
  const int e = __ldg(p.idx + a);
  if (e < 0 || e >= p.E) return;
  const int64_t row0 = (int64_t)e * 2 * p.I;
  const int c0 = blockIdx.x * kFeatures;
  if (threadIdx.x < 2)
    prefetch_l2_bulk(p.gate_up + (row0 + (threadIdx.x ? p.I : 0) + c0) * p.H, (uint32_t)(min(kFeatures, p.I - c0) * p.H));
  quantize_rows_to_smem<DT>(static_cast<const uint16_t*>(p.x) + a / p.k * p.H, p.H, nullptr, 1, p.H, q, s_scale, red);
  __syncthreads();
  const int f0 = min(c0 + 2 * warp, p.I - 1), f1 = min(f0 + 1, p.I - 1);   // a warp past the end repeats the last
  const int8_t* rows[4] = {p.gate_up + (row0 + f0) * p.H, p.gate_up + (row0 + p.I + f0) * p.H,
                           p.gate_up + (row0 + f1) * p.H, p.gate_up + (row0 + p.I + f1) * p.H};
  int acc[4][1];
  dot_rows<1, 4>(rows, q, p.H / 16, lane, acc);
  if (lane < 2 && c0 + 2 * warp + lane < p.I) {
    const float* ws = p.gate_up_scale + row0 + f0 + lane;
    const float g = (float)(lane ? acc[2][0] : acc[0][0]) * s_scale[0] * __ldg(ws);
    const float u = (float)(lane ? acc[3][0] : acc[1][0]) * s_scale[0] * __ldg(ws + p.I);
    p.h[a * p.I + f0 + lane] = swiglu(g, u);
  }
}

constexpr int kMaxChoices = MOE_ROUTE_MAX_TOP_K;

// out of one token (blockIdx.y) and CH channels a warp, all its choices. Dynamic shared memory: `held`
// quantized rows of h; every CTA quantizes all of the token's, which more channels a warp keep from being
// most of the work. (Ling-shaped, T = 4: of 39 to 42 us for both kernels the tokens' quantization here is 5,
// the rows 13. Requesting the rows into L2 ahead of h, by this kernel or the one before, made it 3 and 4.5 more.)
// The chunks of all the held
// choices are one list: lane l takes chunks l, l + 32, ..., 8 / CH of them and CH channels at once, so that
// eight loads are in flight and a chunk's place and token values serve CH channels.
template <int CH>
__global__ void __launch_bounds__(kThreads, 3) int8_experts_down_kernel(const ExpertsParams p, int held) {
  extern __shared__ uint4 q[];   // [held][I / 16]
  __shared__ float s_scale[kMaxChoices];
  __shared__ int s_e[kMaxChoices];   // -1: none
  constexpr int kAtOnce = 8 / CH;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nch = p.I / 16;
  const int c0 = blockIdx.x * kWarps * CH, ch0 = c0 + warp * CH;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = blockIdx.y;
  float sum[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) sum[i] = 0.f;
  for (int j0 = 0; j0 < p.k; j0 += held) {
    const int nj = min(held, p.k - j0);
    __syncthreads();
    for (int j = warp; j < nj; j += kWarps) {
      const int64_t a = t * p.k + j0 + j;
      int e = __ldg(p.idx + a);
      if (e < 0 || e >= p.E) e = -1;
      if (e >= 0) {
        const float weight = __ldg(p.weights + a);
        const float* h = p.h + a * p.I;
        float v[16], u[16];   // the row's first 1024 values stay in registers
        uint32_t m = 0;
        if (lane < nch) {
          load16_cg(h + 16 * lane, v);
          m = amax_bits(v);
        }
        if (lane + 32 < nch) {
          load16_cg(h + 16 * (lane + 32), u);
          m = max(m, amax_bits(u));
        }
        for (int c = lane + 64; c < nch; c += 32) {
          float w[16];
          load16_cg(h + 16 * c, w);
          m = max(m, amax_bits(w));
        }
        const RowScale r = row_scale(__reduce_max_sync(0xFFFFFFFFu, m));
        if (lane < nch) q[j * nch + lane] = quantize16(v, r);
        if (lane + 32 < nch) q[j * nch + lane + 32] = quantize16(u, r);
        for (int c = lane + 64; c < nch; c += 32) {
          load16_cg(h + 16 * c, v);
          q[j * nch + c] = quantize16(v, r);
        }
        if (lane == 0) s_scale[j] = r.scale * weight;
      }
      if (lane == 0) s_e[j] = e;
    }
    __syncthreads();
    if (ch0 < p.H) {
      float ws[CH];   // lane j: the scales of choice j
      const int my_e = lane < nj ? s_e[lane] : -1;
#pragma unroll
      for (int i = 0; i < CH; ++i)
        ws[i] = my_e >= 0 && ch0 + i < p.H ? s_scale[lane] * __ldg(p.down_scale + (int64_t)my_e * p.H + ch0 + i) : 0.f;
      int j = 0, c = lane;   // the lane's chunk: c of choice j
      while (c >= nch) { c -= nch; ++j; }
      for (int at = 0; at < nj * nch; at += 32 * kAtOnce) {
        uint4 w[kAtOnce][CH];
        int from[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          const int e = j < nj ? s_e[j] : -1;
          const int8_t* row = p.down + ((int64_t)max(e, 0) * p.H + ch0) * p.I + 16 * c;
          from[u] = e >= 0 ? j : -1;
#pragma unroll
          for (int i = 0; i < CH; ++i)
            w[u][i] = e >= 0 && ch0 + i < p.H ? ldg_stream(row + (int64_t)i * p.I) : make_uint4(0, 0, 0, 0);
          c += 32;
          while (c >= nch) { c -= nch; ++j; }
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          const int chunk = at + 32 * u + lane;
          const uint4 xv = from[u] >= 0 ? q[chunk] : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            const float f = __shfl_sync(0xFFFFFFFFu, ws[i], from[u] & 31);
            if (from[u] >= 0) sum[i] += (float)dot16(w[u][i], xv, 0) * f;
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const float f = warp_sum(sum[i]);
    if (lane == i && ch0 + i < p.H) store(p.out, p.out_dtype, t * p.H + ch0 + i, f);
  }
}

// ------------------------------------------------- around the tensor-core products
struct PrepareParams {
  const void* x;          // [rows][K], row stride `stride` elements
  int64_t stride;
  const float* x_scale;   // S8 alone
  int rows, K;
  const int* num_rows;    // rows there really are, or NULL
  int K64;                // K rounded up to 64
  __half* q;              // [rows][K64] whole numbers, zeros behind K
  float* scale;           // [rows]
};

// A row as a warp reads and writes it: pieces of 4 fp32, else 8 elements a lane, consecutive lanes
// next to each other in both, so that every access of the warp is one contiguous run.
template <int DT>
struct Piece {
  static constexpr int kN = DT == MOE_DTYPE_F32 ? 4 : 8;
  uint32_t w[DT == MOE_DTYPE_S8 ? 2 : 4];
  // elements i ... of x; fp32 was written earlier in this call
  MOE_DEV void load(const void* x, int64_t i) {
    if constexpr (DT == MOE_DTYPE_S8) {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const int8_t*>(x) + i));
      w[0] = u.x; w[1] = u.y;
    } else {
      const uint4 u = DT == MOE_DTYPE_F32 ? ldg_cg(static_cast<const float*>(x) + i)
                                          : __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + i));
      w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    }
  }
  MOE_DEV void values(float (&v)[kN]) const {
#pragma unroll
    for (int c = 0; c < (int)(sizeof(w) / 4); ++c) {
      if constexpr (DT == MOE_DTYPE_F32) {
        v[c] = __uint_as_float(w[c]);
      } else if constexpr (DT == MOE_DTYPE_BF16) {
        v[2 * c] = bf16_lo(w[c]);
        v[2 * c + 1] = bf16_hi(w[c]);
      } else if constexpr (DT == MOE_DTYPE_F16) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[c]));
        v[2 * c] = f.x;
        v[2 * c + 1] = f.y;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * c + i] = (float)(int8_t)(w[c] >> (8 * i));
      }
    }
  }
  // whole numbers as f16 pairs: kN / 2 words
  MOE_DEV void quantized(const RowScale s, uint32_t (&o)[kN / 2]) const {
    float v[kN], q[kN];
    values(v);
    if constexpr (DT == MOE_DTYPE_S8) {
#pragma unroll
      for (int i = 0; i < kN; ++i) q[i] = v[i];
    } else {
      quantize(v, s, q);
    }
#pragma unroll
    for (int c = 0; c < kN / 2; ++c) {
      const __half2 h = __floats2half2_rn(q[2 * c], q[2 * c + 1]);
      o[c] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
};
template <int W>
MOE_DEV void store_words(void* p, const uint32_t (&o)[W]) {
  if constexpr (W == 2) *static_cast<uint2*>(p) = make_uint2(o[0], o[1]);
  else *static_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
}

// The row of K elements at x + i, quantized by one warp and handed out piece by piece: put(element
// index, words) is called by whole warps, a lane past K64 with an index of -1. The first kKept pieces
// a lane stay in registers between the search for the largest value and the quantization.
template <int DT, class Put>
MOE_DEV float quantize_row(const void* x, int64_t i, int K, int K64, int lane, Put put) {
  constexpr int kN = Piece<DT>::kN, kKept = 8;
  Piece<DT> kept[kKept];
  RowScale s = {};
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < kKept; ++c) {
    const int at = (32 * c + lane) * kN;
    if (at < K) kept[c].load(x, i + at);
  }
  if constexpr (DT != MOE_DTYPE_S8) {
#pragma unroll
    for (int c = 0; c < kKept; ++c)
      if ((32 * c + lane) * kN < K) {
        float v[kN];
        kept[c].values(v);
        m = max(m, amax_bits(v));
      }
    for (int at = (32 * kKept + lane) * kN; at < K; at += 32 * kN) {
      Piece<DT> piece;
      float v[kN];
      piece.load(x, i + at);
      piece.values(v);
      m = max(m, amax_bits(v));
    }
    s = row_scale(__reduce_max_sync(0xFFFFFFFFu, m));
  }
#pragma unroll
  for (int c = 0; c < kKept; ++c) {
    const int at = (32 * c + lane) * kN;
    uint32_t o[kN / 2] = {};
    if (at < K) kept[c].quantized(s, o);
    if (32 * c * kN < K64) put(at < K64 ? at : -1, o);
  }
  for (int base = 32 * kKept * kN; base < K64; base += 32 * kN) {
    const int at = base + lane * kN;
    uint32_t o[kN / 2] = {};
    if (at < K) {
      Piece<DT> piece;
      piece.load(x, i + at);
      piece.quantized(s, o);
    }
    put(at < K64 ? at : -1, o);
  }
  return s.scale;
}

constexpr int kPrepareThreads = 256;

// Rows as whole numbers in f16, and their scales: one warp a row. 32,768 rows of 512 fp32: 21 us, 4.8 TB/s.
template <int DT>
__global__ void __launch_bounds__(kPrepareThreads) int8_prepare_kernel(const PrepareParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int rows = p.num_rows ? min(p.rows, ldg_cg_s32(p.num_rows)) : p.rows;
  constexpr int kW = kPrepareThreads / 32;
  for (int64_t r = (int64_t)blockIdx.x * kW + (threadIdx.x >> 5); r < rows; r += (int64_t)gridDim.x * kW) {
    __half* q = p.q + r * p.K64;
    const float scale = quantize_row<DT>(p.x, r * p.stride, p.K, p.K64, lane, [&](int at, const auto& o) {
      if (at >= 0) store_words(q + at, o);
    });
    if (lane == 0) p.scale[r] = DT == MOE_DTYPE_S8 ? p.x_scale[r] : scale;
  }
}

// Choices in the order of their experts, and each one's token as whole numbers in f16 in
// that order, k copies. Every CTA finds out for itself which rows its chunk of tokens takes:
// from all choices, or, where they are many, from their counts by expert and chunk that a
// launch before has taken. (At 32,768 choices both take some 3 us, a launch more for the counts.) Gathering the
// rows inside the product instead took a copy of four rows at a time, whose issue alone
// made the up product 683 us at T = 4096 (Qwen-shaped).
struct GroupParams {
  const void* x;             // [T][H]
  const int* idx;            // [T][k]
  int T, k, E, H, H64;       // H64: H rounded up to 64
  int chunk, chunks;         // tokens of a CTA
  int block, max_blocks;
  int* chunk_counts;         // [chunks][E]; NULL: count all choices
  __half* q;                 // [rows][H64], zeros behind H
  float* scale;              // [rows]
  int* pos;                  // [T][k]: grouped row, -1 where there is none
  int4* blocks;
  int* counts;               // [0]: blocks, [1]: grouped rows
};

constexpr int kGroupThreads = 1024;

__global__ void __launch_bounds__(kGroupThreads) int8_count_kernel(const GroupParams p) {
  __shared__ int count[MOE_INT8_MAX_EXPERTS];
  for (int e = threadIdx.x; e < p.E; e += kGroupThreads) count[e] = 0;
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  const int64_t a0 = (int64_t)blockIdx.x * p.chunk * p.k;
  const int64_t a1 = min(a0 + (int64_t)p.chunk * p.k, (int64_t)p.T * p.k);
  for (int64_t a = a0 + threadIdx.x; a < a1; a += kGroupThreads) {
    const int e = __ldg(p.idx + a);
    if (e >= 0 && e < p.E) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kGroupThreads) p.chunk_counts[(int64_t)blockIdx.x * p.E + e] = count[e];
}

// 4,096 tokens of 2,048, k = 8: 28 us, for 134 MB of rows written.
// An expert's rows are cut evenly into blocks of at most p.block. Within an expert and a
// chunk the order is the shared-memory atomics': every row is computed by itself, so no
// result depends on it.
template <int DT>
__global__ void __launch_bounds__(kGroupThreads, 1) int8_group_kernel(const GroupParams p) {
  static_assert(kGroupThreads >= MOE_INT8_MAX_EXPERTS, "one thread an expert");
  __shared__ int cursor[MOE_INT8_MAX_EXPERTS], all[MOE_INT8_MAX_EXPERTS], before[MOE_INT8_MAX_EXPERTS], sums[2][32];
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
  all[i] = 0;
  before[i] = 0;
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  // several threads an expert where there are few experts: part q of n takes chunks q, q + n, ...
  const int parts = max(1, kGroupThreads / p.E), part = i / p.E;
  if (!p.chunk_counts) {
    const int choices = p.T * p.k, first = blockIdx.x * p.chunk * p.k;
#pragma unroll 4
    for (int a = i; a < choices; a += kGroupThreads) {
      const int e = __ldg(p.idx + a);
      if (e >= 0 && e < p.E) {
        atomicAdd(&all[e], 1);
        if (a < first) atomicAdd(&before[e], 1);
      }
    }
  } else if (part < parts) {
    const int e = i - part * p.E;
    int sum = 0, own = 0;
#pragma unroll 8
    for (int c = part; c < p.chunks; c += parts) {
      const int n = ldg_cg_s32(p.chunk_counts + (int64_t)c * p.E + e);
      sum += n;
      own += c < (int)blockIdx.x ? n : 0;
    }
    atomicAdd(&all[e], sum);
    atomicAdd(&before[e], own);
  }
  __syncthreads();
  const int c = i < p.E ? all[i] : 0, nb = (c + p.block - 1) / p.block;
  int rows = c, blocks = nb;   // inclusive scans
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int r = __shfl_up_sync(0xFFFFFFFFu, rows, o), b = __shfl_up_sync(0xFFFFFFFFu, blocks, o);
    if (lane >= o) { rows += r; blocks += b; }
  }
  if (lane == 31) { sums[0][warp] = rows; sums[1][warp] = blocks; }
  __syncthreads();
  if (warp == 0) {
    int r = sums[0][lane], b = sums[1][lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, r, o), y = __shfl_up_sync(0xFFFFFFFFu, b, o);
      if (lane >= o) { r += x; b += y; }
    }
    sums[0][lane] = r;
    sums[1][lane] = b;
  }
  __syncthreads();
  if (warp > 0) { rows += sums[0][warp - 1]; blocks += sums[1][warp - 1]; }
  const int row0 = rows - c;
  cursor[i] = row0 + before[i];
  if (blockIdx.x == 0) {
    const int b0 = blocks - nb, size = nb ? ((c + nb - 1) / nb + 15) & ~15 : 0;
    for (int b = 0; b < nb; ++b)
      if (b0 + b < p.max_blocks) p.blocks[b0 + b] = make_int4(i, row0 + b * size, min(size, c - b * size), 0);
    if (i == kGroupThreads - 1) { p.counts[0] = blocks; p.counts[1] = rows; }
  }
  __syncthreads();
  const int t1 = min(p.T, ((int)blockIdx.x + 1) * p.chunk);
  for (int t = blockIdx.x * p.chunk + warp; t < t1; t += kGroupThreads / 32) {
    int at = -1;
    if (lane < p.k) {
      const int e = __ldg(p.idx + (int64_t)t * p.k + lane);
      if (e >= 0 && e < p.E) at = atomicAdd(&cursor[e], 1);
      p.pos[(int64_t)t * p.k + lane] = at;
    }
    const float scale = quantize_row<DT>(p.x, (int64_t)t * p.H, p.H, p.H64, lane, [&](int i, const auto& o) {
      for (int j = 0; j < p.k; ++j) {
        const int to = __shfl_sync(0xFFFFFFFFu, at, j);
        if (to >= 0 && i >= 0) store_words(p.q + (int64_t)to * p.H64 + i, o);
      }
    });
    if (at >= 0) p.scale[at] = scale;
  }
}

struct CombineParams {
  const float* y;            // [rows][H]: integer sums times the channel's scale
  const float* h_scale;      // [rows]
  const int* pos;            // grouped row of each choice, -1: none
  const float* weights;
  void* out;
  int T, k, H, out_dtype;
};

constexpr int kCombineThreads = 256;

// out[t] = sum_j weights[t, j] h_scale_j y_j, four channels a thread. Reading y bounds it: 4,096 tokens, k = 8,
// H = 2,048: 45 us, 6 TB/s.
__global__ void __launch_bounds__(kCombineThreads) int8_combine_kernel(const CombineParams p) {
  __shared__ float s_f[MOE_ROUTE_MAX_TOP_K];
  __shared__ int s_pos[MOE_ROUTE_MAX_TOP_K];
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    __syncthreads();
    if (threadIdx.x < p.k) {
      const int64_t a = t * p.k + threadIdx.x;
      const int at = ldg_cg_s32(p.pos + a);
      s_pos[threadIdx.x] = at;
      s_f[threadIdx.x] = at >= 0 ? __ldg(p.weights + a) * ldg_cg_f32(p.h_scale + at) : 0.f;
    }
    __syncthreads();
    for (int c = threadIdx.x * 4; c < p.H; c += kCombineThreads * 4) {
      float acc[4] = {};
#pragma unroll 8
      for (int j = 0; j < p.k; ++j) {
        const int at = s_pos[j];
        if (at < 0) continue;
        const float f = s_f[j];
        const uint4 y = ldg_cg(p.y + (int64_t)at * p.H + c);
        acc[0] += f * __uint_as_float(y.x);
        acc[1] += f * __uint_as_float(y.y);
        acc[2] += f * __uint_as_float(y.z);
        acc[3] += f * __uint_as_float(y.w);
      }
      const uint32_t lo = (uint32_t)to_16(p.out_dtype, acc[0]) | ((uint32_t)to_16(p.out_dtype, acc[1]) << 16);
      const uint32_t hi = (uint32_t)to_16(p.out_dtype, acc[2]) | ((uint32_t)to_16(p.out_dtype, acc[3]) << 16);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + t * p.H + c) = make_uint2(lo, hi);
    }
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

cudaError_t launch_experts_stream(const ExpertsParams& p, int x_dtype, int num_sms, cudaStream_t s) {
  const dim3 up((p.I + kFeatures - 1) / kFeatures, (unsigned)(p.T * p.k));
  cudaError_t e = x_dtype == MOE_DTYPE_BF16
                      ? launch_pdl(int8_experts_up_kernel<MOE_DTYPE_BF16>, up, kThreads, (size_t)p.H, s, p)
                      : launch_pdl(int8_experts_up_kernel<MOE_DTYPE_F16>, up, kThreads, (size_t)p.H, s, p);
  if (e != cudaSuccess) return e;
  int held = 32 * 1024 / p.I;   // rows of h a CTA keeps: 32 KB, so that several CTAs share an SM
  held = held < 1 ? 1 : held < p.k ? held : p.k;
  // as many channels a warp as leave two CTAs an SM
  const int64_t want = (int64_t)p.T * p.H / (2 * kWarps * num_sms);
  const auto down = [&](int ch) {
    return dim3((p.H + kWarps * ch - 1) / (kWarps * ch), (unsigned)p.T);
  };
  const size_t smem = (size_t)held * p.I;
  if (want < 2) return launch_pdl(int8_experts_down_kernel<1>, down(1), kThreads, smem, s, p, held);
  if (want < 4) return launch_pdl(int8_experts_down_kernel<2>, down(2), kThreads, smem, s, p, held);
  if (want < 8) return launch_pdl(int8_experts_down_kernel<4>, down(4), kThreads, smem, s, p, held);
  return launch_pdl(int8_experts_down_kernel<8>, down(8), kThreads, smem, s, p, held);
}

bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

int dtype_size(int d) { return d == MOE_DTYPE_S8 ? 1 : d == MOE_DTYPE_F32 ? 4 : 2; }
int64_t pad256(int64_t v) { return (v + 255) / 256 * 256; }
int64_t pad64(int64_t v) { return (v + 63) / 64 * 64; }

// Which of the two a product takes. The tensor cores cost a launch more (some 5 us) and are as fast with 64 tokens
// as with one; the dot-product units read the weights once for each eight tokens, and their time goes by the
// results, each of which a warp adds up. GB300, us a call, dot products / tensor cores, tokens x K x channels:
//   2 x 2,560 x 157,184  66 / 74     4 x 2,560 x 157,184  81 / 72      4 x 1,024 x 32,768   16 / 20
//   4 x 4,096 x 16,384   20 / 22     8 x 4,096 x 16,384   30 / 23     32 x 2,048 x 2,048    15 / 18
//  64 x 2,048 x 2,048    26 / 16   128 x 2,048 x 512      15 / 16    256 x 2,048 x 512      28 / 17
//  16 x 16,384 x 4,096   57 / 89   512 x 128 x 128        12 / 19  1,024 x 128 x 128        21 / 17
// More tokens than 65,535, the CTAs of a grid's second dimension, always go to the tensor cores: with a long K a
// CTA of the dot products holds one.
bool stream_matmul(int64_t T, int64_t N) { return T <= 2 || (T <= 65535 && T * N <= (T <= 4 ? 131072 : 65536)); }
// Experts: the dot-product kernels read an expert's rows for every choice of it, the second time from L2 (some 7 TB/s);
// the tensor cores read them once, and take three launches more, some 20 us. So few tokens stream, unless the choices
// beyond one an expert have 2^27 bytes and more to read again. GB300, us a call after a flush of L2, streamed / tensor
// cores, k of E, H x I, and the bytes read again:
//   8 of 256, 2,048 x 512   T 16  86 / 101 (0)        T 24 111 / 128    T 32 145 / 142
//   8 of 512, 2,560 x 768   T 16 141 / 159 (0)        T 24 201 / 208    T 32 244 / 243
//   8 of 128, 2,048 x 768   T 12  86 / 103 (0)        T 16 117 / 114 (0)
//   2 of  16, 2,048 x 512   T 16  29 /  42 (50 MB)    T 32  43 /  46
//   8 of  16, 2,048 x 512   T  4  33 /  44 (50 MB)    T  8  41 /  48 (151 MB)   T 16  66 / 50 (352 MB)
//  32 of  32, 2,048 x 512   T  2  61 /  67 (101 MB)   T  4  86 /  69 (302 MB)   T 16 223 / 93 (1.5 GB)
//  32 of  64, 1,024 x 256   T  4  45 /  46 (50 MB)    T  8  63 /  52 (151 MB)   T 16  94 / 60 (352 MB)
//   8 of   8, 1,024 x 512   T  8  35 /  32 (88 MB)    T 12  37 /  34 (138 MB)   T 16  47 / 34 (189 MB)
//   2 of   8, 4,096 x 2,048 T  4  53 /  79 (0)        T  8  78 /  83 (201 MB)   T 12  98 / 85 (403 MB)
bool stream_experts(const moe_int8_experts_config_t* c, int64_t T) {
  const int64_t again = T * c->top_k - c->num_experts;
  return T <= 16 && again * 3 * c->hidden * c->intermediate < (int64_t(1) << 27);
}

cudaError_t launch_prepare(const PrepareParams& p, int dtype, int num_sms, cudaStream_t s) {
  const int64_t blocks = ((int64_t)p.rows + kPrepareThreads / 32 - 1) / (kPrepareThreads / 32);
  const dim3 grid((unsigned)(blocks < 16 * num_sms ? blocks : 16 * num_sms));
  switch (dtype) {
    case MOE_DTYPE_F32: return launch_pdl(int8_prepare_kernel<MOE_DTYPE_F32>, grid, kPrepareThreads, 0, s, p);
    case MOE_DTYPE_BF16: return launch_pdl(int8_prepare_kernel<MOE_DTYPE_BF16>, grid, kPrepareThreads, 0, s, p);
    case MOE_DTYPE_F16: return launch_pdl(int8_prepare_kernel<MOE_DTYPE_F16>, grid, kPrepareThreads, 0, s, p);
    default: return launch_pdl(int8_prepare_kernel<MOE_DTYPE_S8>, grid, kPrepareThreads, 0, s, p);
  }
}

struct MatmulWorkspace {
  int64_t q, scale, bytes;
};
MatmulWorkspace matmul_workspace(int64_t T, int64_t N, int64_t K) {
  MatmulWorkspace w = {};
  if (stream_matmul(T, N)) return w;
  w.scale = pad256(T * pad64(K) * 2);
  w.bytes = w.scale + pad256(T * 4);
  return w;
}

cudaError_t launch_matmul_tensor(const StreamParams& p, int x_dtype, uint8_t* ws, int num_sms, cudaStream_t s) {
  const MatmulWorkspace w = matmul_workspace(p.T, p.N, p.K);
  PrepareParams a = {};
  a.x = p.x;
  a.stride = p.x_stride;
  a.x_scale = p.x_scale;
  a.rows = p.T;
  a.K = p.K;
  a.K64 = (int)pad64(p.K);
  a.q = (__half*)(ws + w.q);
  a.scale = (float*)(ws + w.scale);
  cudaError_t e = launch_prepare(a, x_dtype, num_sms, s);
  if (e != cudaSuccess) return e;
  GemmArgs g = {};
  g.a = p.w;
  g.a_rows = p.N;
  g.a_stride = p.w_stride;
  g.b = a.q;
  g.b_rows = p.T;
  g.b_stride = a.K64;
  g.K = p.K;
  g.channels = p.N;
  // token tiles of even size: as few as there can be, or as many as give every SM a tile
  const int fewest = (p.T + kMaxBlock - 1) / kMaxBlock, most = (p.T + 15) / 16;
  const int spread = num_sms / ((p.N + 127) / 128);
  const int tiles = spread < fewest ? fewest : spread < most ? spread : most;
  g.block = ((p.T + tiles - 1) / tiles + 15) / 16 * 16;
  g.T = p.T;
  g.row_scale = a.scale;
  g.w_scale = p.w_scale;
  g.out = p.out;
  g.out_dtype = p.out_dtype;
  return launch_gemm(kDense, g, num_sms, s);
}

// Whether a launch counts the choices of each chunk first.
bool count_first(int64_t choices) { return choices > 32768; }

// Scratch of the experts' call. y takes h's place, which is dead by then.
struct ExpertsWorkspace {
  int64_t h, q, x_scale, hq, h_scale, chunk_counts, pos, blocks, counts, bytes;
  int block, max_blocks, chunk, chunks;
};
ExpertsWorkspace experts_workspace(const moe_int8_experts_config_t* c, int64_t T) {
  ExpertsWorkspace w = {};
  const int64_t rows = T * c->top_k, H = c->hidden, I = c->intermediate;
  if (stream_experts(c, T)) {
    w.bytes = pad256(rows * I * 4);
    return w;
  }
  // blocks about one and a half times an expert's mean load: most experts are one block
  const int64_t touched = rows < c->num_experts ? rows : c->num_experts;
  const int64_t want = (rows * 3 / (2 * touched) + 15) / 16 * 16;
  w.block = (int)(want < 32 ? 32 : want > kMaxBlock ? kMaxBlock : want);
  w.max_blocks = (int)(touched + rows / w.block);
  // a warp a token and CTA at a time; no more CTAs than SMs
  w.chunk = (int)((T + 127) / 128 > 32 ? (T + 127) / 128 : 32);
  w.chunks = (int)((T + w.chunk - 1) / w.chunk);
  int64_t at = 0;
  const auto take = [&at](int64_t bytes) { const int64_t o = at; at += pad256(bytes); return o; };
  w.h = take(rows * (I > H ? I : H) * 4);
  w.q = take(rows * pad64(H) * 2);
  w.x_scale = take(rows * 4);
  w.hq = take(rows * pad64(I) * 2);
  w.h_scale = take(rows * 4);
  w.chunk_counts = take(count_first(rows) ? (int64_t)w.chunks * c->num_experts * 4 : 0);
  w.pos = take(rows * 4);
  w.blocks = take((int64_t)w.max_blocks * 16);
  w.counts = take(8);
  w.bytes = at;
  return w;
}

cudaError_t launch_experts_tensor(const ExpertsParams& p, const moe_int8_experts_config_t* cfg, int x_dtype,
                                  uint8_t* ws, int num_sms, cudaStream_t s) {
  const ExpertsWorkspace w = experts_workspace(cfg, p.T);
  const int rows = p.T * p.k;
  GroupParams a = {};
  a.x = p.x;
  a.idx = p.idx;
  a.T = p.T;
  a.k = p.k;
  a.E = p.E;
  a.H = p.H;
  a.H64 = (int)pad64(p.H);
  a.chunk = w.chunk;
  a.chunks = w.chunks;
  a.block = w.block;
  a.max_blocks = w.max_blocks;
  a.chunk_counts = count_first(rows) ? (int*)(ws + w.chunk_counts) : nullptr;
  a.q = (__half*)(ws + w.q);
  a.scale = (float*)(ws + w.x_scale);
  a.pos = (int*)(ws + w.pos);
  a.blocks = (int4*)(ws + w.blocks);
  a.counts = (int*)(ws + w.counts);
  cudaError_t e = cudaSuccess;
  if (a.chunk_counts) e = launch_pdl(int8_count_kernel, dim3(w.chunks), kGroupThreads, 0, s, a);
  if (e != cudaSuccess) return e;
  e = x_dtype == MOE_DTYPE_BF16 ? launch_pdl(int8_group_kernel<MOE_DTYPE_BF16>, dim3(w.chunks), kGroupThreads, 0, s, a)
                                : launch_pdl(int8_group_kernel<MOE_DTYPE_F16>, dim3(w.chunks), kGroupThreads, 0, s, a);
  if (e != cudaSuccess) return e;

  GemmArgs g = {};
  g.a = p.gate_up;
  g.a_rows = (int64_t)p.E * 2 * p.I;
  g.a_stride = p.H;
  g.b = a.q;
  g.b_rows = rows;
  g.b_stride = a.H64;
  g.K = p.H;
  g.channels = p.I;
  g.rows_per_group = 2 * p.I;
  g.block = w.block;
  g.blocks = a.blocks;
  g.num_blocks = a.counts;
  g.max_blocks = w.max_blocks;
  g.row_scale = a.scale;
  g.w_scale = p.gate_up_scale;
  g.out = ws + w.h;
  e = launch_gemm(kUp, g, num_sms, s);
  if (e != cudaSuccess) return e;

  PrepareParams b = {};
  b.x = ws + w.h;
  b.stride = p.I;
  b.rows = rows;
  b.K = p.I;
  b.K64 = (int)pad64(p.I);
  b.num_rows = a.counts + 1;
  b.q = (__half*)(ws + w.hq);
  b.scale = (float*)(ws + w.h_scale);
  e = launch_prepare(b, MOE_DTYPE_F32, num_sms, s);
  if (e != cudaSuccess) return e;

  g.a = p.down;
  g.a_rows = (int64_t)p.E * p.H;
  g.a_stride = p.I;
  g.b = b.q;
  g.b_rows = rows;
  g.b_stride = b.K64;
  g.K = p.I;
  g.channels = p.H;
  g.rows_per_group = p.H;
  g.w_scale = p.down_scale;
  g.out = ws + w.h;
  e = launch_gemm(kDown, g, num_sms, s);
  if (e != cudaSuccess) return e;

  CombineParams c = {};
  c.y = (const float*)(ws + w.h);
  c.h_scale = b.scale;
  c.pos = a.pos;
  c.weights = p.weights;
  c.out = p.out;
  c.T = p.T;
  c.k = p.k;
  c.H = p.H;
  c.out_dtype = p.out_dtype;
  return launch_pdl(int8_combine_kernel, dim3((unsigned)(p.T < num_sms * 8 ? p.T : num_sms * 8)), kCombineThreads, 0, s, c);
}

}  // namespace

int device_sms() {
  static int sms[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  if (!sms[dev] && cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 152;
  return sms[dev];
}

}  // namespace int8
}  // namespace moe

extern "C" {

moe_status_t moe_quant_matmul_workspace(int32_t T, int32_t N, int32_t K, int32_t x_dtype, int64_t* bytes) {
  if (!bytes || T < 0 || N < 0 || K < 1 || x_dtype < MOE_DTYPE_F32 || x_dtype > MOE_DTYPE_S8) return MOE_ERR_INVALID_ARG;
  *bytes = moe::int8::matmul_workspace(T, N, K).bytes;
  return MOE_OK;
}

moe_status_t moe_quant_matmul(const void* x_dev, int32_t x_dtype, int64_t x_stride, const float* x_scale_dev,
                             const int8_t* w_dev, int64_t w_stride, const float* w_scale_dev, void* out_dev,
                             int32_t out_dtype, int32_t T, int32_t N, int32_t K, void* workspace_dev,
                             int64_t workspace_bytes, void* stream) {
  using namespace moe::int8;
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
  const int64_t need = matmul_workspace(T, N, K).bytes;
  if (need && (!workspace_dev || workspace_bytes < need || (uintptr_t)workspace_dev & 255)) return MOE_ERR_INVALID_ARG;
  const StreamParams p = {x_dev, x_stride, x_scale_dev, w_dev, w_stride, w_scale_dev, out_dev, out_dtype, T, N, K};
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  if (need) e = launch_matmul_tensor(p, x_dtype, (uint8_t*)workspace_dev, device_sms(), s);
  else switch (x_dtype) {
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
  if ((int64_t)T * c->top_k > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
  *bytes = experts_workspace(c, T).bytes;
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
  if (((uintptr_t)x_dev | (uintptr_t)out_dev | (uintptr_t)w->gate_up_dev | (uintptr_t)w->down_dev |
       (uintptr_t)w->down_scale_dev) & 15 ||
      ((uintptr_t)idx_dev | (uintptr_t)weights_dev | (uintptr_t)w->gate_up_scale_dev) & 3 ||
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
  const cudaError_t e = stream_experts(c, T)
                            ? launch_experts_stream(p, x_dtype, device_sms(), (cudaStream_t)stream)
                            : launch_experts_tensor(p, c, x_dtype, (uint8_t*)workspace_dev, device_sms(),
                                                    (cudaStream_t)stream);
  return e == cudaSuccess ? MOE_OK : moe::record_cuda_failure(e, "moe_quant_experts");
}

void moe_quant_test_force_wait_timeout(int32_t on) { moe::int8::test_withhold(on != 0); }

moe_status_t moe_quant_sync_status(void* stream) {
  int code = 0;
  const cudaError_t e = moe::int8::gemm_status((cudaStream_t)stream, &code);
  if (e != cudaSuccess) return moe::record_cuda_failure(e, "moe_quant_sync_status");
  return (moe_status_t)code;
}

}  // extern "C"
