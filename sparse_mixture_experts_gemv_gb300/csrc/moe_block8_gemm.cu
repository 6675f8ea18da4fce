// Products in 8-bit floating point (E4M3) with a scale for each block of 128, on the tensor cores:
// dense, and grouped by expert.
//
//   out[r, n] = sum_b x_scale[r, b] w_scale[n / 128, b] (sum_{k in block b} x[r, k] w[n, k])
//
// The MMA multiplies E4M3 by E4M3 into fp32 accumulators, but knows nothing of scales that are no
// powers of two. So each block of 128 of K is a product of its own in tensor memory, and eight
// epilogue warps add it, times its scale, to sums in registers while the tensor cores work on
// the next block in the other half of tensor memory. Rows are the lanes of tensor memory and
// channels its columns: then a thread's values of a block have one scale, its row's times the
// 128 channels', and an element costs one FMA. (Channels as lanes would let a tile have fewer rows than
// 128, but every element would need a scale of its own from shared memory. A tile with few
// rows wastes tensor time only where the weights' way from memory takes longer: 128 rows
// make 256 operations of a weight byte, and the tensor cores do some 500 in a byte's time.)
//
// One persistent CTA an SM, warp-specialised:
//   warp 0        rows and weights by TMA into a ring, a block of K a stage
//   warp 1        issues the MMAs
//   warps 4-11    epilogue: four warps for each half of the columns
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_block8.h"
#include "moe_internal.h"
#include "moe_sm100.cuh"
#include "moe_sm100_warp.cuh"
#include "moe_tensormap.h"

namespace moe {
namespace block8 {
namespace {

using namespace sm100;

constexpr int kRows = 128;                // rows of a tile = lanes of tensor memory
constexpr int kThreads = 384;
constexpr int kMaxStages = 16;
constexpr int kRingBytes = 192 * 1024;
constexpr int kTurnBytes = 8 * 2048;      // 32 rows x 64 bytes for each epilogue warp
constexpr int kMaxGroups = MOE_BLOCK_MAX_EXPERTS;
constexpr int kTableBytes = 2 * (kMaxGroups + 4) * 4;
constexpr int kFixedSmem = 1024 /*align*/ + kTurnBytes + kTableBytes + 1024 /*barriers*/;
// A stage of few rows holds only those; the MMA reads 128 all the same, into what lies behind (their results are not
// used): the buffers behind the last stage are as long as that.
static_assert(kTurnBytes >= kRows * kBlock, "the MMA reads past the last stage");

__device__ int g_gemm_error;              // MOE_ERR_TIMEOUT once a bounded wait ran out

struct Params {
  const int* offsets;
  int rows, channels, groups, K;
  int tiles_n;               // channel tiles of a group
  int blocks;                // of K
  int row_blocks;            // channels' blocks of 128
  int stages, stage_bytes, a_bytes;
  const float* x_scale;
  const float* w_scale;
  void* out;
  int out_dtype;
  int wide;                  // rows of out are 16-byte aligned
  int withhold;              // test only: no rows come, so that the waits for them run out
};

// Boxes of 16, 32, 64 and 128 rows: a tile fetches what it has, not its neighbours'.
struct Maps {
  CUtensorMap w;
  CUtensorMap x[4];
};
MOE_DEV int box_of(int rows) { return rows <= 16 ? 0 : rows <= 32 ? 1 : rows <= 64 ? 2 : 3; }

struct Tile {
  int e, n0, row0, rows;
};

// Tiles in the order of groups, channels, rows: CTAs that work at the same time share weights.
// `e` only grows: a warp looks from where it was, 32 groups at a time.
struct Finder {
  const int* first;          // [groups + 1] first tile of a group
  const int* row;            // [groups + 1] first row
  int e;
  template <int NT>
  MOE_DEV Tile find(const Params& p, int tile) {
    const int lane = threadIdx.x & 31;
    while (true) {
      const int at = min(e + 1 + lane, p.groups);
      const uint32_t past = __ballot_sync(0xFFFFFFFFu, first[at] <= tile && e + 1 + lane <= p.groups);
      e += __popc(past);
      if (past != 0xFFFFFFFFu) break;
    }
    Tile t;
    const int rows = row[e + 1] - row[e], tm = (rows + kRows - 1) / kRows, in = tile - first[e];
    t.e = e;
    t.n0 = in / tm * NT;
    t.row0 = row[e] + in % tm * kRows;
    t.rows = min(kRows, row[e + 1] - t.row0);
    return t;
  }
};

// D[tmem] (+)= A[smem] * B[smem]^T in E4M3, issued by one thread.
MOE_DEV void mma_e4m3(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
      :: "r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}

// First rows and first tiles of the groups, by all threads: offsets are held to [0, rows] and to growing, so that
// whatever they are, tiles lie within the rows and apart.
template <int NT>
MOE_DEV void make_tables(const Params& p, int* first, int* row, int* scratch) {
  constexpr int kPer = (kMaxGroups + kThreads) / kThreads;
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
  if (!p.offsets) {
    if (i == 0) {
      row[0] = 0;
      row[1] = p.rows;
      first[0] = 0;
      first[1] = (p.rows + kRows - 1) / kRows * p.tiles_n;
    }
    __syncthreads();
    return;
  }
  int at[kPer], top = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int e = i * kPer + q;
    at[q] = e <= p.groups ? min(max(ldg_cg_s32(p.offsets + e), 0), p.rows) : 0;
    top = max(top, at[q]);
  }
  int upto = top;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto = max(upto, v);
  }
  if (lane == 31) scratch[warp] = upto;
  __syncthreads();
  int before = __shfl_up_sync(0xFFFFFFFFu, upto, 1);
  if (lane == 0) before = 0;
  for (int w = 0; w < warp; ++w) before = max(before, scratch[w]);
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    before = max(before, at[q]);
    if (i * kPer + q <= p.groups) row[i * kPer + q] = before;
  }
  __syncthreads();
  int tiles[kPer], sum = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int e = i * kPer + q;
    tiles[q] = e < p.groups ? (row[e + 1] - row[e] + kRows - 1) / kRows * p.tiles_n : 0;
    sum += tiles[q];
  }
  upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) scratch[warp] = upto;
  __syncthreads();
  int base = upto - sum;
  for (int w = 0; w < warp; ++w) base += scratch[w];
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    if (i * kPer + q <= p.groups) first[i * kPer + q] = base;
    base += tiles[q];
  }
  __syncthreads();
}

template <int OUT>
MOE_DEV uint32_t pack2(float a, float b) {
  if (OUT == MOE_DTYPE_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 64 bytes of each of the warp's 32 rows, turned in shared memory so that eight rows leave at a time in 16-byte
// pieces. v: the lane's row, 16 words.
MOE_DEV void store_rows(uint8_t* turn, const uint32_t (&v)[16], const Params& p, int64_t row0, int rows, int ch0, int size) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < 4; ++c)   // chunk c of row r lies at c ^ (r / 2 % 4): no bank twice in either direction
    *reinterpret_cast<uint4*>(turn + lane * 64 + ((c ^ (lane >> 1 & 3)) << 4)) =
        make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
  __syncwarp();
  const int64_t ld = (int64_t)p.channels * size;
  uint8_t* out = static_cast<uint8_t*>(p.out) + row0 * ld + (int64_t)ch0 * size;
  const int n = min(64, (p.channels - ch0) * size);   // bytes of a row that there are
  if (p.wide) {
    const int c = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2);
      if (r < rows && 16 * c < n)
        *reinterpret_cast<uint4*>(out + r * ld + 16 * c) =
            *reinterpret_cast<const uint4*>(turn + r * 64 + ((c ^ (r >> 1 & 3)) << 4));
    }
  } else if (size == 4) {
    for (int i = lane >> 4; i < rows; i += 2) {
      const int b = (lane & 15) * 4;
      if (b < n)
        *reinterpret_cast<uint32_t*>(out + i * ld + b) =
            *reinterpret_cast<const uint32_t*>(turn + i * 64 + (((b >> 4) ^ (i >> 1 & 3)) << 4) + (b & 15));
    }
  } else {
    const int b = lane * 2;
    if (b < n)
      for (int i = 0; i < rows; ++i)
        *reinterpret_cast<uint16_t*>(out + i * ld + b) =
            *reinterpret_cast<const uint16_t*>(turn + i * 64 + (((b >> 4) ^ (i >> 1 & 3)) << 4) + (b & 15));
  }
  __syncwarp();
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 1) block8_gemm_kernel(const __grid_constant__ Maps maps, const Params p) {
  constexpr int kCols = NT / 2;             // of an epilogue warp
  constexpr uint32_t kTmem = 2 * NT;        // two products
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* s_turn = smem + p.stages * p.stage_bytes;
  int* first = reinterpret_cast<int*>(s_turn + kTurnBytes);
  int* row = first + kMaxGroups + 4;
  uint64_t* full = reinterpret_cast<uint64_t*>(row + kMaxGroups + 4);
  uint64_t* empty = full + kMaxStages;
  uint64_t* d_full = empty + kMaxStages;
  uint64_t* d_empty = d_full + 2;
  uint64_t* drain = d_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* scratch = reinterpret_cast<int*>(tmem_slot + 2);   // [kThreads / 32]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&d_full[a], 1);
      mbar_init(&d_empty[a], 8);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&maps.w);
  }
  if (warp == 1) tmem_alloc(tmem_slot, kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  pdl_wait();
  asm volatile("fence.proxy.async.global;" ::: "memory");   // rows written by the kernel before, read by TMA here
  pdl_launch_dependents();
  make_tables<NT>(p, first, row, scratch);
  const int total = first[p.groups];
  Finder finder = {first, row, 0};

  const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty), ring0 = smem_u32(smem);
  if (warp == 0) {
    // ---------------------------------------------------- rows and weights
    uint32_t it = 0;
    int s = 0, ph = 1;
    bool stop = p.withhold != 0;
    for (int tile = blockIdx.x; tile < total && !stop; tile += gridDim.x) {
      const Tile t = finder.find<NT>(p, tile);
      const int box = box_of(t.rows);
      const CUtensorMap* map = &maps.x[box];
      const uint32_t bytes = (uint32_t)((16 << box) + NT) * kBlock;
      for (int b = 0; b < p.blocks; ++b, ++it) {
        if (!warp_wait(empty0 + 8 * s, ph, &g_gemm_error, abort_flag)) { stop = true; break; }
        if (elect()) {
          const uint32_t bar = full0 + 8 * s, dst = ring0 + s * p.stage_bytes;
          expect_tx(bar, bytes);
          load_2d(dst + p.a_bytes, &maps.w, b * kBlock, t.e * p.channels + t.n0, bar);
          load_2d(dst, map, b * kBlock, t.row0, bar);
        }
        __syncwarp();
        if (++s == p.stages) { s = 0; ph ^= 1; }
      }
    }
    land(full, p.stages, it, &g_gemm_error, abort_flag);
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(NT >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
    const uint32_t d_full0 = smem_u32(d_full), d_empty0 = smem_u32(d_empty);
    int s = 0, ph = 0;
    uint32_t ab = 0, d_ph = 1;
    bool stop = false;
    for (int tile = blockIdx.x; tile < total && !stop; tile += gridDim.x) {
      for (int b = 0; b < p.blocks; ++b) {
        if (!warp_wait(d_empty0 + 8 * ab, d_ph, &g_gemm_error, abort_flag) ||
            !warp_wait(full0 + 8 * s, ph, &g_gemm_error, abort_flag)) {
          stop = true;
          break;
        }
        tc_fence_after();
        const uint32_t at = ring0 + s * p.stage_bytes, d = tmem + ab * NT;
        const uint64_t adesc = smem_desc_sw128(at), bdesc = smem_desc_sw128(at + p.a_bytes);
        if (elect()) {
#pragma unroll
          for (int kk = 0; kk < kBlock / 32; ++kk)   // 32 of K: 32 bytes, 2 in the descriptors
            mma_e4m3(d, adesc + 2 * kk, bdesc + 2 * kk, idesc, kk != 0 ? 1u : 0u);
          commit(empty0 + 8 * s);
          commit(d_full0 + 8 * ab);
        }
        __syncwarp();
        if (++s == p.stages) { s = 0; ph ^= 1; }
        ab ^= 1;
        d_ph ^= ab ^ 1;   // flips when the halves come round
      }
    }
    if (elect()) mma_commit(drain);   // all MMAs complete before tensor memory is released
    __syncwarp();
    mbar_wait(drain, 0, &g_gemm_error, abort_flag, 2000000000LL, false);
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int quad = warp & 3, half = (warp - 4) >> 2;
    uint8_t* turn = s_turn + (warp - 4) * 2048;
    const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + half * kCols;
    const uint32_t d_full0 = smem_u32(d_full), d_empty0 = smem_u32(d_empty);
    uint32_t ab = 0, ph = 0;
    bool stop = false;
    for (int tile = blockIdx.x; tile < total && !stop; tile += gridDim.x) {
      const Tile t = finder.find<NT>(p, tile);
      const int rows = min(32, t.rows - quad * 32);   // of this warp
      const int ch0 = t.n0 + half * kCols;
      const bool work = rows > 0 && ch0 < p.channels;
      const float* xs = p.x_scale + (int64_t)(t.row0 + min(quad * 32 + lane, t.rows - 1)) * p.blocks;
      const float* ws = p.w_scale + ((int64_t)t.e * p.row_blocks + min(ch0, p.channels - 1) / kBlock) * p.blocks;
      float acc[kCols];
#pragma unroll
      for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
      float x_next = ldg_cg_f32(xs), w_next = __ldg(ws);
      for (int b = 0; b < p.blocks; ++b) {
        const float scale = x_next * w_next;
        if (b + 1 < p.blocks) {
          x_next = ldg_cg_f32(xs + b + 1);
          w_next = __ldg(ws + b + 1);
        }
        if (!warp_wait(d_full0 + 8 * ab, ph, &g_gemm_error, abort_flag)) { stop = true; break; }
        tc_fence_after();
        if (work) {
#pragma unroll
          for (int c = 0; c < kCols; c += 32) {
            uint32_t v[32];
            tmem_ld32(taddr + ab * NT + c, v);
            if (c + 32 == kCols) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) arrive(d_empty0 + 8 * ab);
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[c + i] = fmaf(__uint_as_float(v[i]), scale, acc[c + i]);
          }
        } else if (lane == 0) {
          arrive(d_empty0 + 8 * ab);
        }
        ab ^= 1;
        ph ^= ab ^ 1;
      }
      if (stop || !work) continue;
      const int64_t row0 = t.row0 + quad * 32;
      const int size = p.out_dtype == MOE_DTYPE_F32 ? 4 : 2;
      if (size == 4) {
#pragma unroll
        for (int c = 0; c < kCols; c += 16) {
          uint32_t v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(acc[c + i]);
          if (ch0 + c < p.channels) store_rows(turn, v, p, row0, rows, ch0 + c, 4);
        }
      } else {
#pragma unroll
        for (int c = 0; c < kCols; c += 32) {
          uint32_t v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            v[i] = p.out_dtype == MOE_DTYPE_BF16 ? pack2<MOE_DTYPE_BF16>(acc[c + 2 * i], acc[c + 2 * i + 1])
                                                 : pack2<MOE_DTYPE_F16>(acc[c + 2 * i], acc[c + 2 * i + 1]);
          if (ch0 + c < p.channels) store_rows(turn, v, p, row0, rows, ch0 + c, 2);
        }
      }
    }
    // rows before the first group and behind the last one are zeros
    const int64_t ld = (int64_t)p.channels * (p.out_dtype == MOE_DTYPE_F32 ? 4 : 2) / 2;   // in 16-bit words
    const int64_t head = row[0] * ld, tail = row[p.groups] * ld, end = p.rows * ld;
    uint16_t* out = static_cast<uint16_t*>(p.out);
    const int64_t step = (int64_t)gridDim.x * 256, i0 = (int64_t)blockIdx.x * 256 + threadIdx.x - 128;
    for (int64_t i = i0; i < head; i += step) out[i] = 0;
    for (int64_t i = tail + i0; i < end; i += step) out[i] = 0;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmem);
  }
}

// ------------------------------------------------------------------------- host
cudaError_t encode(CUtensorMap* m, const void* base, int64_t rows, int K, int64_t stride, uint32_t box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride};
  const cuuint32_t box[2] = {kBlock, box_rows};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box);
}

thread_local int t_withhold = 0;

template <int NT>
cudaError_t launch_tile(const GemmArgs& a, int num_sms, cudaStream_t s) {
  Maps maps = {};
  cudaError_t e = encode(&maps.w, a.w, (int64_t)a.groups * a.channels, a.K, a.w_stride, NT);
  for (int i = 0; i < 4 && e == cudaSuccess; ++i) {
    e = encode(&maps.x[i], a.x, a.rows, a.K, a.x_stride, 16u << i);
    if (a.rows <= 16 << i) break;
  }
  if (e != cudaSuccess) return e;
  Params p = {};
  p.offsets = a.offsets;
  p.rows = a.rows;
  p.channels = a.channels;
  p.groups = a.groups;
  p.K = a.K;
  p.tiles_n = (a.channels + NT - 1) / NT;
  p.blocks = (a.K + kBlock - 1) / kBlock;
  p.row_blocks = (a.channels + kBlock - 1) / kBlock;
  const int box = a.rows <= 16 ? 16 : a.rows <= 32 ? 32 : a.rows <= 64 ? 64 : kRows;
  p.a_bytes = box * kBlock;
  p.stage_bytes = p.a_bytes + NT * kBlock;
  p.stages = kRingBytes / p.stage_bytes;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  p.x_scale = a.x_scale;
  p.w_scale = a.w_scale;
  p.out = a.out;
  p.out_dtype = a.out_dtype;
  p.wide = !(((uintptr_t)a.out | (uint64_t)a.channels * (a.out_dtype == MOE_DTYPE_F32 ? 4 : 2)) & 15);
  p.withhold = t_withhold;
  const size_t smem = (size_t)p.stages * p.stage_bytes + kFixedSmem;
  // at most one tile a group more than the rows fill
  int64_t tiles = (a.rows + kRows - 1) / kRows;
  if (a.offsets) tiles += a.groups < a.rows ? a.groups : a.rows;
  tiles *= p.tiles_n;
  const int grid = (int)(tiles < num_sms ? tiles : num_sms);

  static bool allowed[64] = {};
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !allowed[dev]) {
    e = cudaFuncSetAttribute(block8_gemm_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes + kFixedSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) allowed[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block8_gemm_kernel<NT>, maps, p);
}

}  // namespace

void test_withhold(int on) { t_withhold = on; }

cudaError_t launch_gemm(const GemmArgs& a, int num_sms, cudaStream_t s) {
  // the widest tile that still gives every SM one
  const int64_t groups = a.offsets ? (a.rows < a.groups ? a.rows : a.groups) : 1;
  const int64_t tm = a.offsets ? (a.rows / kRows > groups ? a.rows / kRows : groups) : (a.rows + kRows - 1) / kRows;
  if (tm * ((a.channels + 255) / 256) >= num_sms) return launch_tile<256>(a, num_sms, s);
  if (tm * ((a.channels + 127) / 128) >= num_sms) return launch_tile<128>(a, num_sms, s);
  return launch_tile<64>(a, num_sms, s);
}

cudaError_t gemm_status(cudaStream_t s, int* code) {
  const int zero = 0;
  cudaError_t e = cudaStreamSynchronize(s);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(code, g_gemm_error, sizeof(int));
  if (e == cudaSuccess && *code) e = cudaMemcpyToSymbol(g_gemm_error, &zero, sizeof(int));
  return e;
}

}  // namespace block8
}  // namespace moe
