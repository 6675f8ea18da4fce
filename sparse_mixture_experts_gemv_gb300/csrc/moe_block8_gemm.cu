// Products in 8-bit floating point (E4M3) with a scale for each block of 128, on the tensor cores:
// dense, and grouped by expert.
//
//   out[r, n] = sum_b x_scale[r, b] w_scale[n / 128, b] (sum_{k in block b} x[r, k] w[n, k])
//
// The MMA multiplies E4M3 by E4M3 into fp32 accumulators, but knows nothing of scales that are no
// powers of two. So each block of 128 of K is a product of its own in tensor memory, and eight
// epilogue warps add it, times its scale, to sums in registers while the tensor cores work on
// the next blocks in other columns of tensor memory. Rows are the lanes of tensor memory and
// channels its columns: then a thread's values of a block have one scale, its row's times the
// 128 channels', and an element costs one FMA. (Channels as lanes would let a tile have fewer rows than
// 128, but every element would need a scale of its own from shared memory. A tile with few
// rows wastes tensor time only where the weights' way from memory takes longer: 128 rows
// make 256 operations of a weight byte, and the tensor cores do some 500 in a byte's time.)
//
// One persistent CTA an SM, warp-specialised:
//   warp 0        weights by TMA into a ring, a block of K a stage
//   warp 1        issues the MMAs
//   warp 2        rows by TMA into the same ring (or, few rows of another type: they are quantized once, by warps 2-11,
//                 into an operand that stays in shared memory, and the ring holds weights alone)
//   warp 3        scales into a ring of their own, four blocks a slot
//   warps 4-11    epilogue: four warps for each half of the columns
//
// GB300, kernel alone: dense 4,096 x 2,048 x 4,096 36 us (1.9 PFLOP/s; operands come from L2 at 18 TB/s, without the sums
// of blocks at 20), 8,192 x 8,192 x 8,192 472 us (2.3); 32,768 rows of 256 experts, 2,048 x 1,024 114 us and 512 x 2,048
// 72 us (5.9 and 5.8 TB/s of memory); one row of 2,560 x 157,184 65 us (6.2 TB/s).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "moe_block8.cuh"
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
constexpr int kEpilogueWarps = 8;
constexpr int kThreads = 128 + kEpilogueWarps * 32;
constexpr int kMaxStages = 16;
constexpr int kDone = 16;                 // completions of blocks: no fewer than stages or products
constexpr int kMaxGroups = MOE_BLOCK_MAX_EXPERTS;
constexpr int kTableBytes = 2 * (kMaxGroups + 4) * 4;
constexpr int kScaleSlots = 4;            // of four blocks: each row's, and that of the tile's block of 128 channels
constexpr int kBlockFloats = kRows + 4;
constexpr int kSlotFloats = 4 * kBlockFloats;
constexpr int kFixedSmem = 1024 /*align*/ + kTableBytes + kScaleSlots * kSlotFloats * 4 + 512 /*barriers*/;
// A tile's results in 16 bits, in units of 32 rows x 64 bytes: they leave on their own while the next tile is computed.
// (Stored by the warps themselves they left all SMs at once, and the next tiles waited for them: 1.8 us a tile of
// 128 x 256.)
template <int NT>
constexpr int kTurnBytes = kRows * NT * 2;
template <int NT>
constexpr int kRingBytes = (232448 /*an SM's shared memory*/ - kFixedSmem - kTurnBytes<NT>) / 1024 * 1024;
// A stage of few rows holds only those; the MMA reads 128 all the same, into what lies behind (their results are not
// used): the buffers behind the last stage are as long as that.
static_assert(kTurnBytes<64> >= kRows * kBlock, "the MMA reads past the last stage");

__device__ int g_gemm_error;              // MOE_ERR_TIMEOUT once a bounded wait ran out

struct Params {
  const int* offsets;
  int rows, channels, groups;
  int tiles_n;               // channel tiles of a group
  int blocks;                // of K
  int row_blocks;            // channels' blocks of 128
  int stages, stage_bytes, a_bytes;
  const void* x;             // RAW: rows of x_dtype, x_stride elements apart
  int x_dtype, K, raw_bytes; // raw_bytes: the operand of 16 rows and their scales in shared memory
  int64_t x_stride;
  const float* x_scale;
  const float* w_scale;
  void* out;
  int out_dtype;
  int wide;                  // rows of out are 16-byte aligned
  int scales_wide;           // and those of x_scale
  int early;                 // see GemmArgs
  int withhold;              // test only: no rows come, so that the waits for them run out
};

// Boxes of 16, 32, 64 and 128 rows: a tile fetches what it has, not its neighbours'.
struct Maps {
  CUtensorMap w;
  CUtensorMap x[4];
  CUtensorMap out;           // units of results, where rows are 16-byte aligned
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
    const int rows = row[e + 1] - row[e], tm = tiles_of(rows, kRows), in = tile - first[e];
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
MOE_DEV void make_tables(const Params& p, int* first, int* row, int* scratch) {
  constexpr int kPer = (kMaxGroups + kThreads) / kThreads;
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
  if (!p.offsets) {
    if (i == 0) {
      row[0] = 0;
      row[1] = p.rows;
      first[0] = 0;
      first[1] = tiles_of(p.rows, kRows) * p.tiles_n;
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
    tiles[q] = e < p.groups ? tiles_of(row[e + 1] - row[e], kRows) * p.tiles_n : 0;
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

// 32 columns of the lane on their way from tensor memory, and the wait for them: r is used behind it.
MOE_DEV void tmem_request32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
MOE_DEV void tmem_arrived32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
        "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
        "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
        "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
      :: "memory");
}
// acc[i] += v[i] * scale for 32 values, two an instruction.
MOE_DEV void add32(float2* acc, const uint32_t* v, float scale) {
  const float2 s = make_float2(scale, scale);
#pragma unroll
  for (int i = 0; i < 16; ++i)
    acc[i] = __ffma2_rn(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), s, acc[i]);
}

MOE_DEV float shared_f32(uint32_t a) {
  float f;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(a) : "memory");
  return f;
}
// Where an epilogue lane finds its scales: its row's, and that of the tile's block of 128 channels.
struct Scales {
  uint32_t full, empty;      // first barriers
  uint32_t row, channels;    // addresses within a slot
  int at, ph;
};

// Four blocks' scales of a row, written by a kernel that this one may overlap; those past the end are not used.
MOE_DEV float4 four_scales(const Params& p, const float* xs, int b) {
  if (p.scales_wide) {
    const uint4 u = ldg_cg(xs + b);
    return make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
  }
  const int last = p.blocks - 1;
  return make_float4(ldg_cg_f32(xs + b), ldg_cg_f32(xs + min(b + 1, last)), ldg_cg_f32(xs + min(b + 2, last)),
                     ldg_cg_f32(xs + min(b + 3, last)));
}

// Where an epilogue warp is.
struct Ring {
  uint32_t done, empty;      // first barriers
  uint32_t block;
};

// One block of a warp's C chunks of 32 columns: acc += scale * product, 32 columns on their way while the 32 before them
// are added; the product is let go as soon as it has been read.
template <int C>
MOE_DEV void add_block(float2 (&acc)[16 * C], uint32_t taddr, uint32_t empty, bool first, float scale) {
  uint32_t v[2][32];
  tmem_request32(taddr, v[0]);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    tmem_arrived32(v[c & 1]);
    if (c + 1 < C) {
      tmem_request32(taddr + 32 * (c + 1), v[(c + 1) & 1]);
    } else {
      tc_fence_before();
      __syncwarp();
      if (first) arrive(empty);
    }
    add32(acc + 16 * c, v[c & 1], scale);
  }
}

// At constant distances from an address: in unrolled code sums of addresses are made ahead of their use, and their
// registers are missing then.
template <int AT>
MOE_DEV float shared_f32_at(uint32_t a) {
  float f;
  asm volatile("ld.shared.f32 %0, [%1+%2];" : "=f"(f) : "r"(a), "n"(AT) : "memory");
  return f;
}
template <int AT>
MOE_DEV void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0+%1];" :: "r"(bar), "n"(AT) : "memory");
}
template <int AT>
MOE_DEV void lane_wait_at(uint32_t bar, uint32_t parity, int* err, volatile int* abort) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1+%3], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok) : "r"(bar), "r"(parity), "n"(AT) : "memory");
  if (!ok) lane_wait(bar + AT, parity, err, abort);
  __syncwarp();
}
template <int AT>
MOE_DEV void tmem_request32_at(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32+%33];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr), "n"(AT));
}

// All blocks of a tile, which come in fours: four are unrolled, whose barriers, scales and products follow each other.
// With two chunks a block (C = 2) the next block's first is on its way while this one's last is added (the request behind
// the last block is not used; one under a condition would cost copies of its registers): 4,096 x 2,048 x 4,096 40 -> 38 us.
// With one it only waits for a product that is not there yet.
template <int C, int NT>
MOE_DEV void add_fours(float2 (&acc)[16 * C], Scales& scales, Ring& ring, uint32_t taddr, int blocks,
                       volatile int* abort_flag) {
  constexpr uint32_t kProducts = 512 / NT;
  Scales sc = scales;
  uint32_t block = ring.block;
  const bool first = (threadIdx.x & 31) == 0;
  uint32_t v[2][32];
  if constexpr (C == 2) {
    lane_wait(ring.done + 8 * (block % kDone), block / kDone & 1, &g_gemm_error, abort_flag);
    tc_fence_after();
    tmem_request32(taddr + block % kProducts * NT, v[0]);
  }
#pragma unroll 1
  for (int b0 = 0; b0 < blocks; b0 += 4) {
    lane_wait(sc.full + 8 * sc.at, sc.ph, &g_gemm_error, abort_flag);
    const uint32_t row = sc.row + sc.at * (kSlotFloats * 4), channels = sc.channels + sc.at * (kSlotFloats * 4);
    const uint32_t done = ring.done + 8 * (block % kDone), ph = block / kDone & 1, product = block % kProducts;
    const uint32_t to = taddr + product * NT, empty = ring.empty + 8 * product;
    block += 4;
    const auto one = [&](auto index) {
      constexpr int q = decltype(index)::value;
      const float scale = shared_f32_at<q * kBlockFloats * 4>(row) * shared_f32_at<q * kBlockFloats * 4>(channels);
      if constexpr (C == 2) {
        tmem_arrived32(v[0]);
        tmem_request32_at<q * NT + 32>(to, v[1]);
        add32(acc, v[0], scale);
      } else {
        lane_wait_at<8 * q>(done, ph, &g_gemm_error, abort_flag);
        tc_fence_after();
        tmem_request32_at<q * NT>(to, v[1]);
      }
      tmem_arrived32(v[1]);
      tc_fence_before();
      __syncwarp();
      if (first) arrive_at<8 * q>(empty);
      if constexpr (C == 2) {
        if constexpr (q < 3) {
          lane_wait_at<8 * (q + 1)>(done, ph, &g_gemm_error, abort_flag);
          tc_fence_after();
          tmem_request32_at<(q + 1) * NT>(to, v[0]);
        } else {
          if (b0 + 4 < blocks) lane_wait(ring.done + 8 * (block % kDone), block / kDone & 1, &g_gemm_error, abort_flag);
          tc_fence_after();
          tmem_request32(taddr + block % kProducts * NT, v[0]);
        }
      }
      add32(acc + 16 * (C - 1), v[1], scale);
    };
    one(std::integral_constant<int, 0>());
    one(std::integral_constant<int, 1>());
    one(std::integral_constant<int, 2>());
    one(std::integral_constant<int, 3>());
    __syncwarp();
    if (first) arrive(sc.empty + 8 * sc.at);
    if (++sc.at == kScaleSlots) { sc.at = 0; sc.ph ^= 1; }
  }
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");   // the last request's registers are others' next
  scales = sc;
  ring.block = block;
}

// All blocks of any tile. `there` false: no rows or channels, and the products are let go. (Parameters are held in
// registers: behind the barriers' memory clobbers they would be read again every time.)
template <int C, int NT>
MOE_DEV void add_blocks(float2 (&acc)[16 * C], Scales& scales, Ring& ring, uint32_t taddr, int blocks, bool there,
                        volatile int* abort_flag) {
  constexpr uint32_t kProducts = 512 / NT;
  Scales sc = scales;
  Ring r = ring;
  const bool first = (threadIdx.x & 31) == 0;
#pragma unroll 1
  for (int b0 = 0; b0 < blocks; b0 += 4) {
    lane_wait(sc.full + 8 * sc.at, sc.ph, &g_gemm_error, abort_flag);
    uint32_t row = sc.row + sc.at * (kSlotFloats * 4), channels = sc.channels + sc.at * (kSlotFloats * 4);
    const uint32_t last = row + min(4, blocks - b0) * (kBlockFloats * 4);
#pragma unroll 1
    do {
      const float scale = shared_f32(row) * shared_f32(channels);
      lane_wait(r.done + 8 * (r.block % kDone), r.block / kDone & 1, &g_gemm_error, abort_flag);
      tc_fence_after();
      const uint32_t product = r.block % kProducts;
      if (there) add_block<C>(acc, taddr + product * NT, r.empty + 8 * product, first, scale);
      else if (first) arrive(r.empty + 8 * product);
      ++r.block;
      row += kBlockFloats * 4;
      channels += kBlockFloats * 4;
    } while (row != last);
    __syncwarp();
    if (first) arrive(sc.empty + 8 * sc.at);
    if (++sc.at == kScaleSlots) { sc.at = 0; sc.ph ^= 1; }
  }
  scales = sc;
  ring = r;
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

// A unit of results in shared memory: the lane's row, 16 words. Chunk c of row r lies at c ^ (r / 2 % 4), the 64-byte
// swizzle.
MOE_DEV void put_unit(uint8_t* unit, const uint32_t (&v)[16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4*>(unit + lane * 64 + ((c ^ (lane >> 1 & 3)) << 4)) =
        make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}
MOE_DEV void store_2d(const CUtensorMap* map, int c0, int c1, const void* smem) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
               :: "l"(map), "r"(c0), "r"(c1), "r"(smem_u32(smem)) : "memory");
}
MOE_DEV void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
MOE_DEV void store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
MOE_DEV void store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// A unit of fewer rows than 32 (the others are another group's), or of rows off 16-byte boundaries, by the warp: rows
// from .. rows.
MOE_DEV void copy_unit(const uint8_t* unit, const Params& p, int64_t row0, int from, int rows, int ch0, int size) {
  const int lane = threadIdx.x & 31;
  const int64_t ld = (int64_t)p.channels * size;
  uint8_t* out = static_cast<uint8_t*>(p.out) + row0 * ld + (int64_t)ch0 * size;
  const int n = min(64 / size, p.channels - ch0) * size;   // bytes of a row that there are (all channels' pass 31 bits)
  if (p.wide) {
    const int c = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2);
      if (r >= from && r < rows && 16 * c < n)
        *reinterpret_cast<uint4*>(out + r * ld + 16 * c) =
            *reinterpret_cast<const uint4*>(unit + r * 64 + ((c ^ (r >> 1 & 3)) << 4));
    }
  } else if (size == 4) {
    const int b = (lane & 15) * 4;
    if (b < n)
      for (int i = from + (lane >> 4); i < rows; i += 2)
        *reinterpret_cast<uint32_t*>(out + i * ld + b) =
            *reinterpret_cast<const uint32_t*>(unit + i * 64 + (((b >> 4) ^ (i >> 1 & 3)) << 4) + (b & 15));
  } else {
    const int b = lane * 2;
    if (b < n)
      for (int i = from; i < rows; ++i)
        *reinterpret_cast<uint16_t*>(out + i * ld + b) =
            *reinterpret_cast<const uint16_t*>(unit + i * 64 + (((b >> 4) ^ (i >> 1 & 3)) << 4) + (b & 15));
  }
}

// N units of `step` channels from ch0 on leave.
template <int N>
MOE_DEV void store_units(uint8_t* turn, const CUtensorMap* map, const Params& p, int64_t row0, int from, int rows, int ch0,
                         int size) {
  const int step = 64 / size;
  if (p.wide && rows - from == 32) {
    fence_proxy_async_smem();
    __syncwarp();
    if (elect()) {
      for (int c = 0; c < N; ++c)
        if (ch0 + c * step < p.channels) store_2d(map, ch0 + c * step, (int)row0, turn + c * 2048);
      store_commit();
    }
  } else {
    __syncwarp();
    for (int c = 0; c < N; ++c)
      if (ch0 + c * step < p.channels) copy_unit(turn + c * 2048, p, row0, from, rows, ch0 + c * step, size);
  }
}

// Few rows of another type to the operand of 16 rows, blocks of 128 behind each other in the 128-byte swizzle, and their
// scales [block][16] behind that. Rows that there are not stay as they are: results go by rows.
template <int DT>
MOE_DEV void quantize_rows(const Params& p, uint8_t* operand, float* scales, int thread, int threads) {
  const int per_row = p.blocks * 8, n = p.rows * per_row;
  for (int i = thread; i - (thread & 31) < n; i += threads) {
    const int t = i / per_row, c = i % per_row, b = c >> 3;
    const bool in = i < n && c * 16 < p.K;
    float v[16] = {};
    if (in) int8::load16<DT>(p.x, t * p.x_stride + 16 * c, v);
    const float scale = block_scale(v);
    if (i >= n) continue;
    const uint4 q = in ? to_e4m3(v, scale) : make_uint4(0, 0, 0, 0);   // zeros behind K
    *reinterpret_cast<uint4*>(operand + b * 2048 + t * kBlock + (((c & 7) ^ (t & 7)) << 4)) = q;
    if ((c & 7) == 0) scales[b * 16 + t] = scale;
  }
}

// NT: channels of a tile. RAW: quantized_inside().
template <int NT, bool RAW>
__global__ void __launch_bounds__(kThreads, 1) block8_gemm_kernel(const __grid_constant__ Maps maps, const Params p) {
  constexpr int kProducts = 512 / NT;       // in tensor memory at once
  static_assert(kProducts <= kDone, "a completion each");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int raw_bytes = RAW ? p.raw_bytes : 0;
  uint8_t* s_turn = smem + raw_bytes + p.stages * p.stage_bytes;
  float* s_raw_scale = reinterpret_cast<float*>(smem + p.blocks * 2048);
  int* first = reinterpret_cast<int*>(s_turn + kTurnBytes<NT>);
  int* row = first + kMaxGroups + 4;
  float* s_scale = reinterpret_cast<float*>(row + kMaxGroups + 4);
  uint64_t* full = reinterpret_cast<uint64_t*>(s_scale + kScaleSlots * kSlotFloats);
  uint64_t* done = full + kMaxStages;
  uint64_t* d_empty = done + kDone;
  uint64_t* sc_full = d_empty + kProducts;
  uint64_t* sc_empty = sc_full + kScaleSlots;
  uint64_t* raw_ready = sc_empty + kScaleSlots;
  uint64_t* drain = raw_ready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* scratch = reinterpret_cast<int*>(tmem_slot + 2);   // [kThreads / 32]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) mbar_init(&full[s], RAW ? 1 : 2);
    for (int a = 0; a < kDone; ++a) mbar_init(&done[a], 1);
    for (int a = 0; a < kScaleSlots; ++a) {
      mbar_init(&sc_full[a], 1);
      mbar_init(&sc_empty[a], kEpilogueWarps);
    }
    for (int a = 0; a < kProducts; ++a) mbar_init(&d_empty[a], kEpilogueWarps);
    mbar_init(raw_ready, kThreads / 32 - 2);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&maps.w);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Behind the call's own quantization only rows and scales wait for it: what came before it is complete when it lets
  // this kernel start, so that weights are on their way meanwhile.
  if (!p.early) pdl_wait();
  asm volatile("fence.proxy.async.global;" ::: "memory");   // rows written by the kernel before, read by TMA here
  pdl_launch_dependents();
  make_tables(p, first, row, scratch);
  const int total = first[p.groups];
  Finder finder = {first, row, 0};

  // One completion a block, behind its MMAs: it frees the stage for the copies and hands the product to the epilogue.
  const uint32_t full0 = smem_u32(full), done0 = smem_u32(done), ring0 = smem_u32(smem) + raw_bytes;
  if (RAW && warp >= 2) {
    float* scales = s_raw_scale;
    const int thread = threadIdx.x - 64, threads = kThreads - 64;
    if (p.x_dtype == MOE_DTYPE_BF16) quantize_rows<MOE_DTYPE_BF16>(p, smem, scales, thread, threads);
    else if (p.x_dtype == MOE_DTYPE_F16) quantize_rows<MOE_DTYPE_F16>(p, smem, scales, thread, threads);
    else quantize_rows<MOE_DTYPE_F32>(p, smem, scales, thread, threads);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(raw_ready);
  }
  if (warp == 0 || (!RAW && warp == 2)) {
    // ------------------------------------------------ weights (0), rows (2)
    if (p.early && warp == 2) {
      pdl_wait();
      asm volatile("fence.proxy.async.global;" ::: "memory");
    }
    const int blocks = p.blocks, stages = p.stages;
    const uint32_t stage_bytes = p.stage_bytes;
    uint32_t it = 0;
    int s = 0;
    bool stop = p.withhold != 0;
    for (int tile = blockIdx.x; tile < total && !stop; tile += gridDim.x) {
      const Tile t = finder.find<NT>(p, tile);
      const int box = box_of(t.rows);
      const CUtensorMap* map = warp == 0 ? &maps.w : &maps.x[box];
      const uint32_t bytes = (uint32_t)(warp == 0 ? NT : 16 << box) * kBlock;
      const uint32_t to = ring0 + (warp == 0 ? p.a_bytes : 0);
      const int at = warp == 0 ? t.e * p.channels + t.n0 : t.row0;
      for (int b = 0; b < blocks; ++b, ++it) {
        const uint32_t was = it - stages;   // the block whose stage this is
        if (it >= (uint32_t)stages &&
            !warp_wait(done0 + 8 * (was % kDone), was / kDone & 1, &g_gemm_error, abort_flag)) {
          stop = true;
          break;
        }
        if (elect()) {
          expect_tx(full0 + 8 * s, bytes);
          load_2d(to + s * stage_bytes, map, b * kBlock, at, full0 + 8 * s);
        }
        __syncwarp();
        if (++s == stages) s = 0;
      }
    }
    land(full, p.stages, it, &g_gemm_error, abort_flag);
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    // What is done between two blocks, some 400 cycles, bounds it: so two blocks are issued at once where both are
    // there, their waits overlap, and one commit a block serves both sides.
    constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(NT >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
    const uint32_t d_empty0 = smem_u32(d_empty);
    const int blocks = p.blocks, stages = p.stages;
    const uint32_t stage_bytes = p.stage_bytes, a_bytes = p.a_bytes;
    int s = 0, ph = 0, ab = 0, d_ph = 1;
    uint32_t it = 0;
    bool stop = RAW && !warp_wait(smem_u32(raw_ready), 0, &g_gemm_error, abort_flag);
    const auto issue = [&](int s, int ab, uint32_t it, int b) {
      const uint32_t at = ring0 + s * stage_bytes, d = tmem + ab * NT;
      const uint64_t adesc = smem_desc_sw128(RAW ? smem_u32(smem) + b * 2048 : at), bdesc = smem_desc_sw128(at + a_bytes);
#pragma unroll
      for (int kk = 0; kk < kBlock / 32; ++kk)   // 32 of K: 32 bytes, 2 in the descriptors
        mma_e4m3(d, adesc + 2 * kk, bdesc + 2 * kk, idesc, kk != 0 ? 1u : 0u);
      commit(done0 + 8 * (it % kDone));
    };
    for (int tile = blockIdx.x; tile < total && !stop; tile += gridDim.x) {
      for (int b = 0; b < blocks;) {
        int s1 = s + 1, ph1 = ph, ab1 = ab + 1, d_ph1 = d_ph;
        if (s1 == stages) { s1 = 0; ph1 ^= 1; }
        if (ab1 == kProducts) { ab1 = 0; d_ph1 ^= 1; }
        const bool one = try_wait(d_empty0 + 8 * ab, d_ph) & try_wait(full0 + 8 * s, ph);
        const bool two = (b + 1 < blocks) & test_wait(d_empty0 + 8 * ab1, d_ph1) & test_wait(full0 + 8 * s1, ph1);
        const bool both = __all_sync(0xFFFFFFFFu, one & two);
        if (!both && !__all_sync(0xFFFFFFFFu, one) &&
            (!warp_wait(d_empty0 + 8 * ab, d_ph, &g_gemm_error, abort_flag) ||
             !warp_wait(full0 + 8 * s, ph, &g_gemm_error, abort_flag))) {
          stop = true;
          break;
        }
        tc_fence_after();
        if (elect()) {
          issue(s, ab, it, b);
          if (both) issue(s1, ab1, it + 1, b + 1);
        }
        __syncwarp();
        s = s1; ph = ph1; ab = ab1; d_ph = d_ph1;
        ++b;
        ++it;
        if (both) {
          if (++s == stages) { s = 0; ph ^= 1; }
          if (++ab == kProducts) { ab = 0; d_ph ^= 1; }
          ++b;
          ++it;
        }
      }
    }
    if (elect()) mma_commit(drain);   // all MMAs complete before tensor memory is released
    __syncwarp();
    mbar_wait(drain, 0, &g_gemm_error, abort_flag, 2000000000LL, false);
  } else if (warp == 3) {
    // -------------------------------------------------------------- scales
    if (p.early) pdl_wait();
    const uint32_t sc_full0 = smem_u32(sc_full), sc_empty0 = smem_u32(sc_empty);
    int at = 0, ph = 1;
    bool stop = RAW && !warp_wait(smem_u32(raw_ready), 0, &g_gemm_error, abort_flag);
    for (int tile = blockIdx.x; tile < total && !stop; tile += gridDim.x) {
      const Tile t = finder.find<NT>(p, tile);
      const float* ws = p.w_scale + ((int64_t)t.e * p.row_blocks + t.n0 / kBlock) * p.blocks;
      for (int b = 0; b < p.blocks; b += 4) {
        float4 x[4];
#pragma unroll
        for (int i = 0; i < (RAW ? 0 : 4); ++i)
          x[i] = four_scales(p, p.x_scale + (int64_t)(t.row0 + min(lane + 32 * i, t.rows - 1)) * p.blocks, b);
        const float w = __ldg(ws + min(b + (lane & 3), p.blocks - 1));
        if (!warp_wait(sc_empty0 + 8 * at, ph, &g_gemm_error, abort_flag)) { stop = true; break; }
        float* slot = s_scale + at * kSlotFloats;
        if (RAW) {
          for (int q = lane >> 4; q < 4 && b + q < p.blocks; q += 2)
            slot[q * kBlockFloats + (lane & 15)] = s_raw_scale[(b + q) * 16 + (lane & 15)];
        }
#pragma unroll
        for (int i = 0; i < (RAW ? 0 : 4); ++i) {
          slot[lane + 32 * i] = x[i].x;
          slot[kBlockFloats + lane + 32 * i] = x[i].y;
          slot[2 * kBlockFloats + lane + 32 * i] = x[i].z;
          slot[3 * kBlockFloats + lane + 32 * i] = x[i].w;
        }
        if (lane < 4) slot[lane * kBlockFloats + kRows] = w;
        __syncwarp();
        if (lane == 0) arrive(sc_full0 + 8 * at);
        if (++at == kScaleSlots) { at = 0; ph ^= 1; }
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    constexpr int kCols = NT / 2;             // of a warp
    const int quad = warp & 3, half = (warp - 4) >> 2, blocks = p.blocks;
    uint8_t* turn = s_turn + (warp - 4) * (kTurnBytes<NT> / kEpilogueWarps);
    const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + half * kCols;
    Ring ring = {done0, smem_u32(d_empty), 0};
    Scales sc = {smem_u32(sc_full), smem_u32(sc_empty), smem_u32(s_scale + quad * 32 + lane),
                 smem_u32(s_scale + kRows), 0, 0};
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
      const Tile t = finder.find<NT>(p, tile);
      // this warp's rows, from .. rows of row0 on (RAW: lanes are rows of x, whatever tile they belong to)
      const int from = RAW ? t.row0 : 0, rows = RAW ? (quad ? 0 : t.row0 + t.rows) : min(32, t.rows - quad * 32);
      const int ch0 = t.n0 + half * kCols;
      const bool there = rows > 0 && ch0 < p.channels;
      float2 acc[kCols / 2];
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) acc[i] = make_float2(0.f, 0.f);
      if (there && blocks % 4 == 0) add_fours<kCols / 32, NT>(acc, sc, ring, taddr, blocks, abort_flag);
      else add_blocks<kCols / 32, NT>(acc, sc, ring, taddr, blocks, there, abort_flag);
      if (!there) continue;
      const int64_t row0 = RAW ? 0 : t.row0 + quad * 32;
      constexpr int kUnits = kCols / 32;
      if (p.out_dtype == MOE_DTYPE_F32) {
#pragma unroll
        for (int part = 0; part < 2; ++part) {   // the buffer holds half of them
          if (elect()) store_wait_read();
          __syncwarp();
#pragma unroll
          for (int c = 0; c < kUnits; ++c) {
            uint32_t v[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              v[2 * i] = __float_as_uint(acc[8 * (kUnits * part + c) + i].x);
              v[2 * i + 1] = __float_as_uint(acc[8 * (kUnits * part + c) + i].y);
            }
            put_unit(turn + c * 2048, v);
          }
          store_units<kUnits>(turn, &maps.out, p, row0, from, rows, ch0 + part * kCols / 2, 4);
        }
      } else {
        if (elect()) store_wait_read();
        __syncwarp();
#pragma unroll
        for (int c = 0; c < kUnits; ++c) {
          uint32_t v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            v[i] = p.out_dtype == MOE_DTYPE_BF16 ? pack2<MOE_DTYPE_BF16>(acc[16 * c + i].x, acc[16 * c + i].y)
                                                 : pack2<MOE_DTYPE_F16>(acc[16 * c + i].x, acc[16 * c + i].y);
          put_unit(turn + c * 2048, v);
        }
        store_units<kUnits>(turn, &maps.out, p, row0, from, rows, ch0, 2);
      }
    }
    if (elect()) store_wait();
    __syncwarp();
    // rows before the first group and behind the last one are zeros, two bytes a lane, on which every row starts (32,768
    // rows of 1,024 in bf16 without any expert: 12 us, 5.5 TB/s; in fp32 22 us, 6.2 TB/s)
    const int64_t ld = (int64_t)p.channels * (p.out_dtype == MOE_DTYPE_F32 ? 4 : 2) / 2;   // in 16-bit words
    const int64_t head = row[0] * ld, tail = row[p.groups] * ld, end = p.rows * ld;
    uint16_t* out = static_cast<uint16_t*>(p.out);
    constexpr int kLanes = kEpilogueWarps * 32;
    const int64_t step = (int64_t)gridDim.x * kLanes, i0 = (int64_t)blockIdx.x * kLanes + threadIdx.x - 128;
    for (int64_t i = i0; i < head; i += step) out[i] = 0;
    for (int64_t i = tail + i0; i < end; i += step) out[i] = 0;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------------- host
cudaError_t encode(CUtensorMap* m, const void* base, int64_t rows, int K, int64_t stride, uint32_t box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride};
  const cuuint32_t box[2] = {kBlock, box_rows};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box);
}

cudaError_t encode_out(CUtensorMap* m, const GemmArgs& a, int size) {
  const CUtensorMapDataType type = a.out_dtype == MOE_DTYPE_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : a.out_dtype == MOE_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                                   : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const cuuint64_t dims[2] = {(cuuint64_t)a.channels, (cuuint64_t)a.rows}, strides[1] = {(cuuint64_t)a.channels * size};
  const cuuint32_t box[2] = {(cuuint32_t)(64 / size), 32};
  return encode_tensor_map(m, type, 2, a.out, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_64B);
}

thread_local int t_withhold = 0;

template <int NT, bool RAW>
cudaError_t launch_tile(const GemmArgs& a, int num_sms, cudaStream_t s) {
  Maps maps = {};
  cudaError_t e = encode(&maps.w, a.w, (int64_t)a.groups * a.channels, a.K, a.w_stride, NT);
  const int tail = (a.rows - 1) % kRows + 1;   // dense: rows of the last tile
  for (int i = 0; i < 4 && e == cudaSuccess && !RAW; ++i) {
    const bool used = a.offsets ? i == 0 || a.rows > 8 << i : (i == 3 && a.rows > 64) || (tail <= 16 << i && (i == 0 || tail > 8 << i));
    if (used) e = encode(&maps.x[i], a.x, a.rows, a.K, a.x_stride, 16u << i);
  }
  if (e != cudaSuccess) return e;
  const int size = a.out_dtype == MOE_DTYPE_F32 ? 4 : 2;
  Params p = {};
  p.wide = !(((uintptr_t)a.out | (uint64_t)a.channels * size) & 15);
  if (p.wide) e = encode_out(&maps.out, a, size);
  if (e != cudaSuccess) return e;
  p.offsets = a.offsets;
  p.rows = a.rows;
  p.channels = a.channels;
  p.groups = a.groups;
  p.tiles_n = tiles_of(a.channels, NT);
  p.blocks = tiles_of(a.K, kBlock);
  p.row_blocks = tiles_of(a.channels, kBlock);
  const int box = a.rows <= 16 ? 16 : a.rows <= 32 ? 32 : a.rows <= 64 ? 64 : kRows;
  p.a_bytes = RAW ? 0 : box * kBlock;
  p.x = a.x;
  p.x_dtype = a.x_dtype;
  p.x_stride = a.x_stride;
  p.K = a.K;
  p.raw_bytes = RAW ? (p.blocks * (2048 + 64) + 1023) / 1024 * 1024 : 0;
  p.stage_bytes = p.a_bytes + NT * kBlock;
  p.stages = (kRingBytes<NT> - p.raw_bytes) / p.stage_bytes;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  p.x_scale = a.x_scale;
  p.w_scale = a.w_scale;
  p.out = a.out;
  p.out_dtype = a.out_dtype;
  p.scales_wide = !((uintptr_t)a.x_scale & 15) && p.blocks % 4 == 0;
  p.early = a.early;
  p.withhold = t_withhold;
  const size_t smem = p.raw_bytes + (size_t)p.stages * p.stage_bytes + kTurnBytes<NT> + kFixedSmem;
  // at most one tile a group more than the rows fill
  int64_t tiles = tiles_of(a.rows, kRows);
  if (a.offsets) tiles += a.groups < a.rows ? a.groups : a.rows;
  tiles *= p.tiles_n;
  const int grid = (int)(tiles < num_sms ? tiles : num_sms);

  static bool allowed[64] = {};
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !allowed[dev]) {
    e = cudaFuncSetAttribute(block8_gemm_kernel<NT, RAW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kRingBytes<NT> + kTurnBytes<NT> + kFixedSmem);
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
  return cudaLaunchKernelEx(&cfg, block8_gemm_kernel<NT, RAW>, maps, p);
}

}  // namespace

void test_withhold(int on) { t_withhold = on; }

cudaError_t launch_gemm(const GemmArgs& a, int num_sms, cudaStream_t s) {
  // Narrow tiles while each has an SM of its own, wide ones beyond: a block of K takes a CTA some 270 ns with 128 channels
  // and 190 with 64, and rows fetched for 64 channels are fetched twice as often. GB300, us, 128 / 64: 333 x 2,560 x 1,537
  // 9.8 / 8.1; 32 rows of 512 experts, 2,560 x 1,536 25.8 / 27.5; 1 x 2,560 x 157,184 65 / 70; 4,096 x 2,048 x 4,096
  // 36 / 49; 32,768 rows of 256 experts, 2,048 x 1,024 113 / 138. (256 channels, before the epilogue's last steps: 16, 33,
  // 76, 41, 118: with 128 sums a lane the registers are full, and loads from tensor memory wait for the sums before.)
  const int64_t groups = a.offsets ? (a.rows < a.groups ? a.rows : a.groups) : 1;
  const int64_t tm = a.offsets ? (a.rows / kRows > groups ? a.rows / kRows : groups) : tiles_of(a.rows, kRows);
  const bool narrow = tm * tiles_of(a.channels, 64) <= num_sms;
  if (a.x_dtype != MOE_DTYPE_E4M3) return narrow ? launch_tile<64, true>(a, num_sms, s) : launch_tile<128, true>(a, num_sms, s);
  return narrow ? launch_tile<64, false>(a, num_sms, s) : launch_tile<128, false>(a, num_sms, s);
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
