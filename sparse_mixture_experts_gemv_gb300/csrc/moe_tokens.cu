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
constexpr int kBuckets = MOE_DISPATCH_MAX_EXPERTS + 1;   // the last one: no expert
constexpr int kFusedThreads = 512;
constexpr int kThreads = 1024;
constexpr int kFusedChoices = 2048;            // so many are placed by every CTA for itself
constexpr int kCountedChoices = 32768;         // and so many counted

template <int THREADS>
struct PlanShared {
  int hist[kBuckets + 7];                      // choices by expert
  int cursor[kBuckets + 7];                    // before: of the chunks before this one; then the expert's next row
  alignas(16) uint8_t count[kBuckets][THREADS / 32];   // a segment's choices by expert and warp
  int sums[THREADS / 32];
};

MOE_DEV int bucket_of(int e, int E) { return e >= 0 && e < E ? e : E; }

// The rows of choices [a0, a1): put(choice, row). s.hist holds all choices by expert and s.cursor those before a0 (what
// is written before is seen behind a barrier in here). Experts follow each other, and within a segment of as many
// choices as threads a choice's rank is that within its warp (the lanes of the same expert below) plus the counts of
// the warps before it, a byte each and added up four an instruction: the order of the choices, without a sort.
template <int THREADS, class Put>
MOE_DEV void place(PlanShared<THREADS>& s, const int* idx, int64_t a0, int64_t a1, int E, int* offsets, Put put) {
  constexpr int kWarps = THREADS / 32, kPer = (kBuckets + THREADS - 1) / THREADS;
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
  int next = a0 + i < a1 ? __ldg(idx + a0 + i) : 0;
  for (int c = i; c < (E + 1) * kWarps / 4; c += THREADS) reinterpret_cast<int*>(s.count)[c] = 0;
  __syncthreads();
  int total[kPer], sum = 0;
  const int e0 = i * kPer;                     // consecutive experts a thread
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    total[q] = e0 + q <= E ? s.hist[e0 + q] : 0;
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
  // the sums of the warps before, by one exchange among the lanes
  int base = lane < warp ? s.sums[lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) base += __shfl_xor_sync(0xFFFFFFFFu, base, o);
  base += upto - sum;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    if (e0 + q > E) continue;
    s.cursor[e0 + q] += base;
    if (offsets) offsets[e0 + q] = base;       // offsets[E]: where the choices of no expert begin
    base += total[q];
  }
  const uint32_t below = (1u << lane) - 1;
  const int bits = 32 - __clz(E + 1);
  for (int64_t a = a0; a < a1; a += THREADS) {
    const int64_t at = a + i;
    const int e = at < a1 ? bucket_of(next, E) : E + 1;   // E + 1: behind the end
    if (at + THREADS < a1) next = __ldg(idx + at + THREADS);
    // the lanes of the same expert, a vote a bit (one match of all values takes some 2,000 cycles a segment)
    uint32_t same = 0xFFFFFFFFu;
    for (int b = 0; b < bits; ++b) {
      const uint32_t set = __ballot_sync(0xFFFFFFFFu, e >> b & 1);
      same &= e >> b & 1 ? set : ~set;
    }
    const bool first = e <= E && (same & below) == 0;
    if (first) s.count[e][warp] = (uint8_t)__popc(same);
    __syncthreads();
    if (e <= E) {
      uint32_t row = s.cursor[e] + __popc(same & below);
      const uint4* c = reinterpret_cast<const uint4*>(s.count[e]);
#pragma unroll
      for (int w = 0; w < kWarps; w += 16) {
        const uint4 u = c[w / 16];
        const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int l = 0; l < 4; ++l) {
          const int n = warp - w - 4 * l;      // of these four warps, those before this one
          row = __dp4a(v[l], n >= 4 ? 0x01010101u : n <= 0 ? 0u : 0x01010101u >> (32 - 8 * n), row);
        }
      }
      put(at, e < E ? (int)row : ~(int)row);
    }
    __syncthreads();
    if (a + THREADS < a1) {
      if (first) {
        atomicAdd(&s.cursor[e], __popc(same));
        s.count[e][warp] = 0;
      }
      __syncthreads();
    }
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
  uint16_t* counts;          // [chunks][stride]: choices by chunk and expert
  int chunk, chunks, stride;
};

// A piece of a row (16-byte vectors: 1 KB) to its k places, and the row's scales with the first. `at`: the place of
// choice `lane`, ~place where there is no expert.
template <class V>
constexpr int kVectors = sizeof(V) == 16 ? 2 : 8;   // of a lane
template <class V>
MOE_DEV void copy_piece(const DispatchParams& p, int64_t t, int64_t piece, int at, int lane) {
  constexpr int kU = kVectors<V>;
  const int64_t n = p.row / (int64_t)sizeof(V), v0 = piece * 32 * kU + lane;
  const V* src = reinterpret_cast<const V*>(p.x + t * p.x_stride);
  V v[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u)
    if (v0 + 32 * u < n) v[u] = __ldg(src + v0 + 32 * u);
  const bool scales = piece == 0 && p.x_scale;
  float f = scales && lane < p.scales ? __ldg(p.x_scale + t * p.scales + lane) : 0.f;
  for (int j = 0; j < p.k; ++j) {
    const int r = __shfl_sync(0xFFFFFFFFu, at, j);
    V* dst = reinterpret_cast<V*>(p.rows + (int64_t)(r >= 0 ? r : ~r) * p.row);
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (v0 + 32 * u < n) dst[v0 + 32 * u] = r >= 0 ? v[u] : V{};
  }
  if (!scales) return;
  for (int c = lane; c - lane < p.scales; c += 32) {
    if (c >= 32) f = c < p.scales ? __ldg(p.x_scale + t * p.scales + c) : 0.f;
    for (int j = 0; j < p.k; ++j) {
      const int r = __shfl_sync(0xFFFFFFFFu, at, j);
      if (c < p.scales) p.row_scale[(int64_t)(r >= 0 ? r : ~r) * p.scales + c] = r >= 0 ? f : 0.f;
    }
  }
}
template <class V>
__host__ __device__ int64_t pieces_of(int64_t row) {
  const int64_t v = 32 * kVectors<V> * (int64_t)sizeof(V);
  return row > v ? (row + v - 1) / v : 1;
}

template <class V, class Pos>
MOE_DEV void copy_tokens(const DispatchParams& p, int64_t t0, int64_t t1, int part, int parts, Pos pos) {
  const int lane = threadIdx.x & 31;
  const int64_t pieces = pieces_of<V>(p.row), units = (t1 - t0) * pieces;
  for (int64_t u = part; u < units; u += parts) {
    const int64_t t = t0 + u / pieces;
    copy_piece<V>(p, t, u % pieces, lane < p.k ? pos(t * p.k + lane) : 0, lane);
  }
}

// Few choices: every CTA counts and places all of them, and copies its share of the rows.
template <class V>
__global__ void __launch_bounds__(kFusedThreads) dispatch_fused_kernel(const DispatchParams p) {
  __shared__ PlanShared<kFusedThreads> s;
  __shared__ int s_pos[kFusedChoices];
  for (int e = threadIdx.x; e <= p.E; e += kFusedThreads) s.hist[e] = s.cursor[e] = 0;
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  const int n = p.T * p.k;
#pragma unroll 4
  for (int a = threadIdx.x; a < n; a += kFusedThreads) atomicAdd(&s.hist[bucket_of(__ldg(p.idx + a), p.E)], 1);
  const bool tells = blockIdx.x == 0;
  place(s, p.idx, 0, n, p.E, tells ? p.offsets : nullptr, [&](int64_t a, int row) {
    s_pos[a] = row;
    if (tells) p.pos[a] = row;
  });
  constexpr int kW = kFusedThreads / 32;
  copy_tokens<V>(p, 0, p.T, blockIdx.x * kW + (threadIdx.x >> 5), gridDim.x * kW, [&](int64_t a) { return s_pos[a]; });
}

// Many choices: their numbers by expert in each chunk of tokens first.
__global__ void __launch_bounds__(kThreads) dispatch_count_kernel(const DispatchParams p) {
  __shared__ int hist[kBuckets + 7];
  for (int e = threadIdx.x; e < p.stride; e += kThreads) hist[e] = 0;
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  const int64_t a0 = (int64_t)blockIdx.x * p.chunk * p.k, a1 = min(a0 + (int64_t)p.chunk * p.k, (int64_t)p.T * p.k);
#pragma unroll 4
  for (int64_t a = a0 + threadIdx.x; a < a1; a += kThreads) atomicAdd(&hist[bucket_of(__ldg(p.idx + a), p.E)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < p.stride; e += kThreads)
    p.counts[(int64_t)blockIdx.x * p.stride + e] = (uint16_t)hist[e];
}

// Then every CTA adds up all chunks' numbers and those before its own, eight experts a load, places its chunk and copies
// its rows. Up to kCountedChoices it counts them all for itself, four a load, which takes time with the choices, where a
// launch of the counts takes it with chunks and experts. 2,048 bytes a row, k = 8, us on the device (in a graph), by itself
// / by a launch, of 64, 256 and 1,024 experts: 8,192 choices 6.4 / 10.0, 6.6 / 10.4, 6.8 / 13.7; 32,768 14.1 / 16.8,
// 14.8 / 17.1, 15.1 / 20.4; 40,000 17.7 / 19.7, 18.2 / 20.0, 18.6 / 23.4; 65,536 33.7 / 34.4, 34.7 / 34.6, 35.0 / 37.9;
// 131,072 65 / 62, 66 / 62, 68 / 65. They cross at 65,536 choices and later with many experts, and from 32,768 up to there
// counting by itself would gain up to 2 us, 5 with 1,024 experts: the limit, past which callers bring a workspace, is below
// the crossing for every number of experts. 8,191 tokens of 5,120 bytes, k = 8: 69 us with the counts before it, 5.5 TB/s.
template <class V>
__global__ void __launch_bounds__(kThreads, 1) dispatch_chunk_kernel(const DispatchParams p) {
  __shared__ PlanShared<kThreads> s;
  for (int e = threadIdx.x; e < p.stride; e += kThreads) s.hist[e] = s.cursor[e] = 0;
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * p.chunk, t1 = min(t0 + p.chunk, (int64_t)p.T);
  const int groups = p.stride / 8, parts = kThreads / groups, part = threadIdx.x / groups, g = threadIdx.x % groups;
  if (!p.counts) {
    // the choices before the chunk into the one, the others into the other
    const int n = p.T * p.k, own = (int)t0 * p.k, fours = (uintptr_t)p.idx & 15 ? 0 : n / 4;
    const auto count = [&](int a, int e) { atomicAdd(a < own ? &s.cursor[bucket_of(e, p.E)] : &s.hist[bucket_of(e, p.E)], 1); };
#pragma unroll 4
    for (int f = threadIdx.x; f < fours; f += kThreads) {
      const int4 e = __ldg(reinterpret_cast<const int4*>(p.idx) + f);
      count(4 * f, e.x);
      count(4 * f + 1, e.y);
      count(4 * f + 2, e.z);
      count(4 * f + 3, e.w);
    }
#pragma unroll 4
    for (int a = 4 * fours + threadIdx.x; a < n; a += kThreads) count(a, __ldg(p.idx + a));
    __syncthreads();
    for (int e = threadIdx.x; e <= p.E; e += kThreads) s.hist[e] += s.cursor[e];
  } else if (part < parts) {
    int all[8] = {}, before[8] = {};
#pragma unroll 4
    for (int c = part; c < p.chunks; c += parts) {
      const uint4 u = ldg_cg(p.counts + (int64_t)c * p.stride + 8 * g);
      const uint32_t v[4] = {u.x, u.y, u.z, u.w};
      const bool own = c < (int)blockIdx.x;
#pragma unroll
      for (int l = 0; l < 8; ++l) {
        const int n = l & 1 ? v[l / 2] >> 16 : v[l / 2] & 0xFFFF;
        all[l] += n;
        before[l] += own ? n : 0;
      }
    }
#pragma unroll
    for (int l = 0; l < 8; ++l) {
      atomicAdd(&s.hist[8 * g + l], all[l]);
      atomicAdd(&s.cursor[8 * g + l], before[l]);
    }
  }
  place(s, p.idx, t0 * p.k, t1 * p.k, p.E, blockIdx.x == 0 ? p.offsets : nullptr,
        [&](int64_t a, int row) { p.pos[a] = row; });
  copy_tokens<V>(p, t0, t1, threadIdx.x >> 5, kThreads / 32, [&](int64_t a) { return ldg_cg_s32(p.pos + a); });
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
    } else if constexpr (N == 1) {
      w[0] = DT == MOE_DTYPE_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(f[0])) : __half_as_ushort(__float2half_rn(f[0]));
    } else {   // in pairs: single conversions are an eighth as fast
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        if constexpr (DT == MOE_DTYPE_BF16) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
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

// A token's places and weights, in shared memory by turns: the next token's are on their way while one is worked on.
struct Choices {
  int at[2][MOE_ROUTE_MAX_TOP_K];
  float w[2][MOE_ROUTE_MAX_TOP_K];
};
// Place and weight of choice threadIdx.x of token t; INT32_MAX: no row of y at all.
MOE_DEV void fetch(const CombineParams& p, int64_t t, int& at, float& w) {
  if (t < p.T && threadIdx.x < p.k) {
    at = ldg_cg_s32(p.pos + t * p.k + threadIdx.x);
    w = p.weights ? ldg_cg_f32(p.weights + t * p.k + threadIdx.x) : 1.f;
  }
}
MOE_DEV void keep(Choices& s, int turn, const CombineParams& p, int at, float w) {
  const int64_t rows = (int64_t)p.T * p.k;
  if (threadIdx.x < p.k) {
    s.at[turn][threadIdx.x] = at < rows && ~at < rows ? at : INT32_MAX;
    s.w[turn][threadIdx.x] = w;
  }
}

// out[t] = sum_j w y[pos], in 32 bits and in the order of the choices. One CTA a token, one barrier a token. Memory
// bounds it: 8,191 tokens of 2,048 bf16, k = 8: 48 us, 6.0 TB/s.
template <int DT, int N>
__global__ void __launch_bounds__(kMaxThreads) combine_kernel(const CombineParams p) {
  __shared__ Choices s;
  pdl_wait();
  pdl_launch_dependents();
  int at = 0, turn = 0;
  float w = 0.f;
  fetch(p, blockIdx.x, at, w);
  keep(s, 0, p, at, w);
  __syncthreads();
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, turn ^= 1) {
    fetch(p, t + gridDim.x, at, w);
    for (uint32_t c = threadIdx.x * N; c < (uint32_t)p.H; c += blockDim.x * N) {   // past 2^31 behind the last
      float acc[N] = {};
      for (int j0 = 0; j0 < p.k; j0 += kTogether) {
        Pack<DT, N> v[kTogether];
#pragma unroll
        for (int q = 0; q < kTogether; ++q)
          if (j0 + q < p.k && (unsigned)s.at[turn][j0 + q] < (unsigned)INT32_MAX)
            v[q].load(p.y, s.at[turn][j0 + q] * p.y_stride + c);
#pragma unroll
        for (int q = 0; q < kTogether; ++q)
          if (j0 + q < p.k && (unsigned)s.at[turn][j0 + q] < (unsigned)INT32_MAX) {
            const float f = s.w[turn][j0 + q];
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = fmaf(f, v[q].get(i), acc[i]);
          }
      }
      Pack<DT, N> o;
      o.set(acc);
      o.store(p.out, t * p.H + c);
    }
    keep(s, turn ^ 1, p, at, w);
    __syncthreads();
  }
}

// d_y[pos] = w d_out[t] and d_w = <d_out[t], y[pos]>, eight choices at a time: each thread adds up its columns, then
// the CTA adds the threads' sums, in a fixed order. 8,191 tokens of 2,048 bf16, k = 8: 87 us, 6.4 TB/s (80 registers a
// thread instead of 64, three CTAs an SM: 97; in 64 registers the 16-byte-wide kernels spill 12 bytes a thread).
template <int DT, int N>
__global__ void __launch_bounds__(kMaxThreads, 4) combine_backward_kernel(const CombineParams p) {
  __shared__ Choices s;
  __shared__ float s_sum[2][kMaxThreads / 32][kTogether];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int next_at = 0, turn = 0, side = 0;
  float next_w = 0.f;
  fetch(p, blockIdx.x, next_at, next_w);
  keep(s, 0, p, next_at, next_w);
  __syncthreads();
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, turn ^= 1) {
    fetch(p, t + gridDim.x, next_at, next_w);
    for (int j0 = 0; j0 < p.k; j0 += kTogether, side ^= 1) {
      float dot[kTogether] = {};
      for (uint32_t c = threadIdx.x * N; c < (uint32_t)p.H; c += blockDim.x * N) {   // past 2^31 behind the last
        Pack<DT, N> d, v[kTogether];
        d.load(p.d_out, t * p.d_stride + c);
        if (p.d_weights) {
#pragma unroll
          for (int q = 0; q < kTogether; ++q)
            if (j0 + q < p.k && (unsigned)s.at[turn][j0 + q] < (unsigned)INT32_MAX)
              v[q].load(p.y, s.at[turn][j0 + q] * p.y_stride + c);
        }
#pragma unroll
        for (int q = 0; q < kTogether; ++q) {
          if (j0 + q >= p.k) break;
          const int at = s.at[turn][j0 + q];
          if (at == INT32_MAX) continue;
          if (p.d_weights && at >= 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) dot[q] = fmaf(d.get(i), v[q].get(i), dot[q]);
          }
          if (p.d_y) {
            const float w = s.w[turn][j0 + q];
            float f[N];
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = at >= 0 ? w * d.get(i) : 0.f;
            Pack<DT, N> o;
            o.set(f);
            o.store(p.d_y, (int64_t)(at >= 0 ? at : ~at) * p.H + c);
          }
        }
      }
      if (p.d_weights) {
#pragma unroll
        for (int q = 0; q < kTogether; ++q) {
          const float sum = warp_sum(dot[q]);
          if (lane == 0) s_sum[side][warp][q] = sum;
        }
      }
      if (j0 + kTogether >= p.k) keep(s, turn ^ 1, p, next_at, next_w);
      __syncthreads();
      if (p.d_weights && threadIdx.x < kTogether && j0 + threadIdx.x < p.k) {   // the other side is written meanwhile
        float sum = 0.f;
        for (int w = 0; w < (int)blockDim.x / 32; ++w) sum += s_sum[side][w][threadIdx.x];
        p.d_weights[t * p.k + j0 + threadIdx.x] = sum;
      }
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

// Chunks of many choices: one an SM, but none of more choices than 16 bits count.
struct Chunks {
  int chunk, chunks, stride;
  int64_t bytes;
};
Chunks chunks_of(int64_t T, int64_t k, int64_t E) {
  Chunks c = {};
  if (T * k <= kFusedChoices) return c;
  const int sms = int8::device_sms();
  const int64_t most = 65535 / k, each = (T + sms - 1) / sms;
  c.chunk = (int)(each < most ? each : most);
  c.chunks = (int)((T + c.chunk - 1) / c.chunk);
  c.stride = (int)((E + 1 + 7) / 8 * 8);
  c.bytes = T * k <= kCountedChoices ? 0 : ((int64_t)c.chunks * c.stride * 2 + 255) / 256 * 256;
  return c;
}

template <class V>
cudaError_t launch_dispatch(const DispatchParams& p, int sms, cudaStream_t s) {
  if (!p.chunks) {
    constexpr int kW = kFusedThreads / 32;
    int64_t grid = (p.T * pieces_of<V>(p.row) + kW - 1) / kW;
    if (grid > 2 * sms) grid = 2 * sms;
    return launch(dispatch_fused_kernel<V>, grid < 1 ? 1 : grid, kFusedThreads, s, p);
  }
  const cudaError_t e = p.counts ? launch(dispatch_count_kernel, p.chunks, kThreads, s, p) : cudaSuccess;
  return e != cudaSuccess ? e : launch(dispatch_chunk_kernel<V>, p.chunks, kThreads, s, p);
}

template <int DT, int N>
cudaError_t launch_combine(const CombineParams& p, bool backward, int sms, cudaStream_t s) {
  // as many rounds as kMaxThreads take, each with the same threads
  const int64_t vectors = ((int64_t)p.H + N - 1) / N, rounds = (vectors + kMaxThreads - 1) / kMaxThreads;
  const int threads = (int)((vectors + rounds - 1) / rounds + 31) / 32 * 32;
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

moe_status_t moe_dispatch_tokens_workspace(int32_t T, int32_t k, int32_t E, int64_t* bytes) {
  using namespace moe::tokens;
  moe_status_t st;
  if (!bytes || E < 1) return MOE_ERR_INVALID_ARG;
  if (!in_range(T, k, 1, &st)) return st;
  if (E > MOE_DISPATCH_MAX_EXPERTS) return MOE_ERR_UNSUPPORTED;
  *bytes = chunks_of(T, k, E).bytes;
  return MOE_OK;
}

moe_status_t moe_dispatch_tokens(const void* x_dev, int64_t row_bytes, int64_t row_stride, const float* x_scale_dev,
                                 int32_t scales, const int32_t* idx_dev, int32_t T, int32_t k, int32_t E, void* rows_dev,
                                 float* row_scale_dev, int32_t* offsets_dev, int32_t* pos_dev, void* workspace_dev,
                                 int64_t workspace_bytes, void* stream) {
  using namespace moe::tokens;
  moe_status_t st;
  if (!in_range(T, k, row_bytes, &st)) return st;
  if (E < 1 || scales < 0 || (T && ((scales > 0) != (x_scale_dev != nullptr) || (scales > 0) != (row_scale_dev != nullptr))))
    return MOE_ERR_INVALID_ARG;
  if (E > MOE_DISPATCH_MAX_EXPERTS || row_bytes > INT32_MAX / 2 || scales > INT32_MAX / 8) return MOE_ERR_UNSUPPORTED;
  if (!offsets_dev || (T && (!x_dev || !idx_dev || !rows_dev || !pos_dev || row_stride < row_bytes))) return MOE_ERR_INVALID_ARG;
  if (((uintptr_t)idx_dev | (uintptr_t)offsets_dev | (uintptr_t)pos_dev | (uintptr_t)x_scale_dev | (uintptr_t)row_scale_dev) & 3)
    return MOE_ERR_INVALID_ARG;
  const int64_t n = (int64_t)T * k;
  if (T && (overlap(x_dev, (T - 1) * row_stride + row_bytes, rows_dev, n * row_bytes) || overlap(idx_dev, n * 4, pos_dev, n * 4)))
    return MOE_ERR_INVALID_ARG;
  const Chunks c = chunks_of(T, k, E);
  if (c.bytes && (!workspace_dev || workspace_bytes < c.bytes || (uintptr_t)workspace_dev & 255)) return MOE_ERR_INVALID_ARG;
  const DispatchParams p = {(const uint8_t*)x_dev, row_stride, row_bytes, x_scale_dev, scales, idx_dev, T, k, E,
                            (uint8_t*)rows_dev, row_scale_dev, offsets_dev, pos_dev, c.bytes ? (uint16_t*)workspace_dev : nullptr, c.chunk,
                            c.chunks, c.stride};
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
