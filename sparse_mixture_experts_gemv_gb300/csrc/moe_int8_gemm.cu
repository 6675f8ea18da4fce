// 8-bit integer products on the tensor cores, for many tokens: dense, and grouped by
// expert.
//
//   D[channel, token] = sum_k w[channel, k] q[token, k]
//
// The fifth-generation tensor cores have no 8-bit integer kind on this chip, and the
// older integer instructions run far below the f16 rate. Whole numbers of 8 bits are
// exact in f16, their products (at most 2^14) and sums (up to 2^24) in the fp32
// accumulators, so the products run as f16 x f16, and give the integers themselves as
// long as no partial sum passes 2^24: for every K up to 1,024, and for longer ones but
// where nearly all terms are large and of one sign. There every step rounds.
//
// The weights stay bytes in memory: each tile of 128 channels x 128 bytes comes in by
// TMA, eight converter warps turn it into f16 and write it straight into tensor memory,
// from where the MMA reads its A operand. (Through shared memory the f16 copy would
// be written and read there once more, and with the token operand that is what bounds
// the MMA.) The tokens, far fewer than weights or read many times, are f16 in memory
// already and are the B operand, up to 192 a tile in steps of 16: with few tokens of an
// expert the MMA does no more than they need, and the weight stream bounds it.
//
// One persistent CTA an SM, warp-specialised:
//   warp 0        weights by TMA              warp 2  tokens by TMA
//   warp 1        issues the MMAs             warp 3  idle
//   warps 4-11    converters: two groups of four, each half of a step's K
//   warps 12-15   epilogue of the previous tile while the next one accumulates
// A step is 128 of K: eight MMAs. What the issuing warp does between two steps (a wait,
// addresses, a commit) takes some 300 cycles, about what the MMAs in the queue cover: with
// 64 of K and two waits a step it bounded the kernel (dense 4,096 x 2,048 x 4,096 76 us).
// Tensor memory: two accumulators of 192 columns, two operand slots of 64.
//
// GB300: dense 4,096 x 2,048 x 4,096 50 us (1.37 PFLOP/s, tensor pipe 56% busy); up and down products of
// 32,768 choices of 256 experts (H 2,048, I 512) 148 and 98 us, 4.9 and 5.3 TB/s of memory traffic, their epilogues
// next: without its one the down product takes 83. (Its sums were f16 once, 85 us: an output channel whose scales lie
// far below its expert's largest lost them, and every output took 2^-11 of its terms along.)
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_int8.cuh"
#include "moe_int8.h"
#include "moe_layer.h"
#include "moe_sm100.cuh"
#include "moe_sm100_warp.cuh"
#include "moe_tensormap.h"

namespace moe {
namespace int8 {
namespace {

using namespace sm100;

constexpr int kChannels = 128;            // channels of a tile = lanes of tensor memory
constexpr int kStep = 128;                // K of a stage
constexpr int kRawBytes = kChannels * kStep;
constexpr int kMaxStages = 8;             // of either ring
constexpr int kSlots = 2;                 // f16 weight operands in tensor memory
constexpr int kSlotCols = kStep / 2;
constexpr int kSlotBase = 2 * kMaxBlock;  // their first column
constexpr int kGemmThreads = 512;
constexpr int kStageBudget = 208 * 1024;  // shared memory of both rings
constexpr int kFixedSmem = 1024 /*align*/ + 4 * kMaxBlock * 4 /*scales*/ + 4 * 2048 /*turned results*/ + 1024 /*barriers*/;

__device__ int g_gemm_error;              // MOE_ERR_TIMEOUT once a bounded wait ran out

struct Params {
  const int4* blocks;
  const int* num_blocks;
  int max_blocks;
  int tiles_m;               // channel tiles of a group
  int tiles_t;               // dense: token tiles
  int T, block, channels, rows_per_group;
  int steps;
  int raw_stages, b_stages, b_bytes;
  const float* row_scale;
  const float* w_scale;
  void* out;
  int out_dtype;
  int wide;                  // dense: 16-bit results whose rows are 16-byte aligned
  int withhold;              // test only: no tokens come, so that the waits for them run out
};

// A copy's issue costs about as much as 8 KB, so that every step is one copy of weights (up: two) and one
// of tokens: a map for each number of rows a tile can have.
struct Maps {
  CUtensorMap a;
  CUtensorMap b[kMaxBlock / 16];   // boxes of 16, 32, ... rows; those a launch can use are filled in
};

struct Tile {
  int e, mt, row0, rows, n;   // n: rows rounded up to 16
};

template <int KIND>
MOE_DEV Tile decode(const Params& p, int tile) {
  Tile t;
  if (KIND == kDense) {   // neighbouring CTAs share the weights of a channel tile
    t.e = 0;
    t.mt = tile / p.tiles_t;
    t.row0 = (tile % p.tiles_t) * p.block;
    t.rows = min(p.block, p.T - t.row0);
  } else {                // neighbouring CTAs share the rows of a block; an expert's blocks follow each other
    const uint4 b = ldg_cg(p.blocks + tile / p.tiles_m);
    t.e = (int)b.x;
    t.mt = tile % p.tiles_m;
    t.row0 = (int)b.y;
    t.rows = (int)b.z;
  }
  t.n = (t.rows + 15) & ~15;
  return t;
}

// Four bytes of signed integers -> two f16 pairs. 0x64uu is 1024 + uu; with the sign
// bit flipped uu = b + 128, so b = that minus 1152, exactly.
MOE_DEV void s8x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  asm volatile("sub.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
  asm volatile("sub.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
}

// silu(g) * u by the approximate exponential, whose relative error grows with its argument, and the approximate
// quotient: off by 2^-21 of itself for g >= 0, by (5 + 1.2 |g|) 2^-23 of itself below (2^-18 at -20), where silu
// falls off faster than that grows: in all by less than 2^-20 of the larger of |silu(g) u| and |u|. It is cut to 8 bits
// next. (0 below -87.3, where silu is under 1e-36.)
MOE_DEV float fast_swiglu(float g, float u) { return __fdividef(g, 1.f + __expf(-g)) * u; }

// 32 columns of this warp's 32 lanes of tensor memory.
MOE_DEV void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
      :: "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
         "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
         "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
         "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]),
         "r"(taddr)
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]^T, issued by one thread.
MOE_DEV void mma_f16_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
      :: "r"(d), "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}

template <int KIND>
__global__ void __launch_bounds__(kGemmThreads, 1)
int8_gemm_kernel(const __grid_constant__ Maps maps, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  // two rings: tokens (stages of 2 x block x 128 bytes, whole 1024-byte swizzle atoms), which the MMAs free,
  // and raw weights, which come from further away and are free as soon as they are converted
  uint8_t* s_b = smem;
  uint8_t* s_raw = smem + p.b_stages * p.b_bytes;
  float* s_scale = reinterpret_cast<float*>(s_raw + p.raw_stages * kRawBytes);   // [4][kMaxBlock]
  uint16_t* s_turn = reinterpret_cast<uint16_t*>(s_scale + 4 * kMaxBlock);   // [4][1024]
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(s_turn + 4 * 1024);
  uint64_t* raw_empty = raw_full + kMaxStages;
  uint64_t* b_full = raw_empty + kMaxStages;
  uint64_t* b_empty = b_full + kMaxStages;
  uint64_t* a_full = b_empty + kMaxStages;
  uint64_t* d_full = a_full + kSlots;
  uint64_t* d_empty = d_full + 2;
  uint64_t* drain = d_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.raw_stages; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], 8);
    }
    for (int s = 0; s < p.b_stages; ++s) {
      mbar_init(&b_full[s], 1);
      mbar_init(&b_empty[s], 1);
    }
    for (int s = 0; s < kSlots; ++s) mbar_init(&a_full[s], 8);
    for (int a = 0; a < 2; ++a) {
      mbar_init(&d_full[a], 1);
      mbar_init(&d_empty[a], 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&maps.a);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  pdl_wait();
  asm volatile("fence.proxy.async.global;" ::: "memory");   // tokens written by the kernel before, read by TMA here
  pdl_launch_dependents();

  int total;
  if (KIND == kDense) {
    total = p.tiles_m * p.tiles_t;
  } else {
    const int nb = ldg_cg_s32(p.num_blocks);
    total = (nb < 0 || nb > p.max_blocks ? 0 : nb) * p.tiles_m;
  }

  // A role keeps its place in a ring as a stage number and a parity.
  const uint32_t raw_full0 = smem_u32(raw_full), raw_empty0 = smem_u32(raw_empty), b_full0 = smem_u32(b_full),
                 b_empty0 = smem_u32(b_empty), a_full0 = smem_u32(a_full);
  const uint32_t b0 = smem_u32(s_b), raw0 = smem_u32(s_raw);

  if (warp == 0) {
    // ------------------------------------------------------------- weights
    uint32_t it = 0;
    int s = 0, ph = 1;
    bool stop = false;
    for (int tile = blockIdx.x; tile < total && !stop; tile += gridDim.x) {
      const Tile t = decode<KIND>(p, tile);
      const int r0 = t.e * p.rows_per_group + t.mt * (KIND == kUp ? 64 : kChannels);
      for (int ks = 0; ks < p.steps; ++ks, ++it) {
        if (!warp_wait(raw_empty0 + 8 * s, ph, &g_gemm_error, abort_flag)) { stop = true; break; }
        if (elect()) {
          const uint32_t bar = raw_full0 + 8 * s, dst = raw0 + s * kRawBytes;
          expect_tx(bar, kRawBytes);
          load_2d(dst, &maps.a, ks * kStep, r0, bar);
          if (KIND == kUp)   // 64 gate rows, then their up rows
            load_2d(dst + kRawBytes / 2, &maps.a, ks * kStep, r0 + p.channels, bar);
        }
        __syncwarp();
        if (++s == p.raw_stages) { s = 0; ph ^= 1; }
      }
    }
    land(raw_full, p.raw_stages, it, &g_gemm_error, abort_flag);
  } else if (warp == 2) {
    // -------------------------------------------------------------- tokens
    uint32_t it = 0;
    int s = 0, ph = 1;
    bool stop = p.withhold != 0;
    for (int tile = blockIdx.x; tile < total && !stop; tile += gridDim.x) {
      const Tile t = decode<KIND>(p, tile);
      const CUtensorMap* map = &maps.b[t.n / 16 - 1];
      for (int ks = 0; ks < p.steps; ++ks, ++it) {
        if (!warp_wait(b_empty0 + 8 * s, ph, &g_gemm_error, abort_flag)) { stop = true; break; }
        if (elect()) {
          expect_tx(b_full0 + 8 * s, (uint32_t)(t.n * kStep * 2));
          load_3d(b0 + s * p.b_bytes, map, 0, t.row0, ks * (kStep / 64), b_full0 + 8 * s);
        }
        __syncwarp();
        if (++s == p.b_stages) { s = 0; ph ^= 1; }
      }
    }
    land(b_full, p.b_stages, it, &g_gemm_error, abort_flag);
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    int s = 0, ph = 0;
    uint32_t slot = 0, slot_ph = 0, tc = 0;
    bool stop = false;
    const uint32_t d_full0 = smem_u32(d_full), d_empty0 = smem_u32(d_empty);
    for (int tile = blockIdx.x; tile < total && !stop; tile += gridDim.x, ++tc) {
      const Tile t = decode<KIND>(p, tile);
      // f16 x f16 -> fp32, both K-major, 128 x n
      const uint32_t idesc = (1u << 4) | ((uint32_t)(t.n >> 3) << 17) | ((uint32_t)(kChannels >> 4) << 24);
      const uint32_t ab = tc & 1, d = tmem + ab * kMaxBlock;
      const uint32_t half = (uint32_t)t.n * 8;   // the second 64 of K lie n x 128 bytes behind the first
      if (!warp_wait(d_empty0 + 8 * ab, ((tc >> 1) & 1) ^ 1, &g_gemm_error, abort_flag)) break;
      tc_fence_after();
      for (int ks = 0; ks < p.steps; ++ks) {
        if (!warp_wait(b_full0 + 8 * s, ph, &g_gemm_error, abort_flag) ||
            !warp_wait(a_full0 + 8 * slot, slot_ph, &g_gemm_error, abort_flag)) {
          stop = true;
          break;
        }
        tc_fence_after();
        const uint32_t a0 = tmem + kSlotBase + slot * kSlotCols;
        const uint64_t bdesc = smem_desc_sw128(b0 + s * p.b_bytes);
        if (elect()) {
#pragma unroll
          for (int kk = 0; kk < kStep / 16; ++kk)   // 16 of K: 8 columns, and 32 bytes (2 in the descriptor)
            mma_f16_ts(d, a0 + kk * 8, bdesc + (kk & 3) * 2 + (kk >> 2) * half, idesc, (ks | kk) != 0 ? 1u : 0u);
          commit(b_empty0 + 8 * s);   // frees the stage and, since the converters wait on it too, the slot
          if (ks == p.steps - 1) commit(d_full0 + 8 * ab);
        }
        __syncwarp();
        if (++s == p.b_stages) { s = 0; ph ^= 1; }
        slot ^= 1;
        slot_ph ^= slot ^ 1;   // flips when the slots come round
      }
    }
    if (elect()) mma_commit(drain);   // all MMAs complete before tensor memory is released
    __syncwarp();
    mbar_wait(drain, 0, &g_gemm_error, abort_flag, 2000000000LL, false);
  } else if (warp >= 4 && warp < 12) {
    // ---------------------------------------------------------- converters
    const int group = (warp - 4) >> 2, quad = warp & 3;
    // The lane's row of the raw tile. up: a warp's lower 16 lanes are gate rows, its upper
    // 16 the up rows of the same features, so that the epilogue pairs them by a shuffle.
    const int row = KIND == kUp ? (lane >> 4) * 64 + quad * 16 + (lane & 15) : quad * 32 + lane;
    const uint8_t* src0 = s_raw + row * kStep;
    const int sw = row & 7;   // 128-byte swizzle: 16-byte chunk c of row r lands at c ^ (r % 8)
    const uint32_t to = tmem + ((uint32_t)(quad * 32) << 16) + kSlotBase + group * (kSlotCols / 2);
    int s = 0, ph = 0;
    int es = p.b_stages - kSlots, eph = 1;   // tokens' stage of the step kSlots before, whose MMAs read this slot
    uint32_t slot = 0;
    bool stop = false, first = true;
    for (int tile = blockIdx.x; tile < total && !stop; tile += gridDim.x) {
      for (int ks = 0; ks < p.steps; ++ks) {
        if (!warp_wait(raw_full0 + 8 * s, ph, &g_gemm_error, abort_flag)) { stop = true; break; }
        const uint8_t* src = src0 + s * kRawBytes;
        uint32_t r[32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 w = *reinterpret_cast<const uint4*>(src + (((4 * group + c) ^ sw) << 4));
          s8x4_to_f16(w.x, r[8 * c], r[8 * c + 1]);
          s8x4_to_f16(w.y, r[8 * c + 2], r[8 * c + 3]);
          s8x4_to_f16(w.z, r[8 * c + 4], r[8 * c + 5]);
          s8x4_to_f16(w.w, r[8 * c + 6], r[8 * c + 7]);
        }
        // Free once its values have been used (the conversions are volatile and stay ahead of this): an arrival
        // right behind the loads could be seen before they have read.
        __syncwarp();
        if (lane == 0) arrive(raw_empty0 + 8 * s);
        if (es == 0) first = false;
        if (!first && !warp_wait(b_empty0 + 8 * es, eph, &g_gemm_error, abort_flag)) { stop = true; break; }
        tc_fence_after();
        tmem_st32(to + slot * kSlotCols, r);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive(a_full0 + 8 * slot);
        slot ^= 1;
        if (++s == p.raw_stages) { s = 0; ph ^= 1; }
        if (++es == p.b_stages) { es = 0; eph ^= 1; }
      }
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------------ epilogue
    const int quad = warp & 3;
    float* cs = s_scale + quad * kMaxBlock;   // the warp's copy of the tile's token scales
    uint16_t* turn = s_turn + quad * 1024;    // 32 tokens x 32 channels of 16 bits, or 16 x 32 of fp32
    const bool f16_out = p.out_dtype == MOE_DTYPE_F16;
    uint32_t tc = 0;
    const auto channel = [&](const Tile& t) {
      return KIND == kUp ? t.mt * 64 + quad * 16 + (lane & 15) : t.mt * kChannels + quad * 32 + lane;
    };
    // A tile and its lane's scales are loaded a tile ahead: on a short tile their latency would show.
    const auto scales = [&](const Tile& t, float& a, float& b) {
      const int ch = channel(t);
      const float* w = p.w_scale + (KIND == kDense ? 0 : (int64_t)t.e * p.rows_per_group) + ch;
      a = ch < p.channels ? __ldg(w) : 0.f;
      b = 1.f;
      if (KIND == kUp && ch < p.channels) b = __ldg(w + p.channels);
    };
    Tile next = {};
    float next0 = 0.f, next1 = 1.f;
    if ((int)blockIdx.x < total) {
      next = decode<KIND>(p, blockIdx.x);
      scales(next, next0, next1);
    }
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x, ++tc) {
      const Tile t = next;
      const float w0 = next0, w1 = next1;
      const uint32_t ab = tc & 1;
      __syncwarp();
      if (KIND != kDown) {
        for (int c = lane; c < t.rows; c += 32) cs[c] = ldg_cg_f32(p.row_scale + t.row0 + c);
      }
      if (tile + (int)gridDim.x < total) {
        next = decode<KIND>(p, tile + gridDim.x);
        scales(next, next0, next1);
      }
      const int ch = channel(t);
      const bool in = ch < p.channels;
      __syncwarp();
      if (!warp_wait(smem_u32(&d_full[ab]), (tc >> 1) & 1, &g_gemm_error, abort_flag)) break;
      tc_fence_after();
      const uint32_t taddr = tmem + ab * kMaxBlock + ((uint32_t)(quad * 32) << 16);
      for (int c0 = 0; c0 < t.rows; c0 += 32) {
        uint32_t v[32];
        tmem_ld32(taddr + c0, v);
        const int nc = min(32, t.rows - c0);
        if (KIND == kUp) {
          // lower lanes take the even columns, upper lanes the odd ones: each sends its partner the
          // other column's half of the pair
          float* dst = static_cast<float*>(p.out) + ((int64_t)t.row0 + c0 + (lane >> 4)) * p.channels + ch;
          const bool upper = lane >= 16;
          const float* xs = cs + c0 + (lane >> 4);
          float h[16];   // all of them before the first store: nothing of it waits for a branch
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float keep = __uint_as_float(upper ? v[2 * i + 1] : v[2 * i]);
            const float got = __shfl_xor_sync(0xFFFFFFFFu, __uint_as_float(upper ? v[2 * i] : v[2 * i + 1]), 16);
            const float x = xs[2 * i];
            h[i] = fast_swiglu((upper ? got : keep) * x * w0, (upper ? keep : got) * x * w1);
          }
          const int limit = in ? nc - (lane >> 4) : 0;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (2 * i < limit) *dst = h[i];
            dst += 2 * p.channels;
          }
        } else if (KIND == kDown) {
          // fp32, 16 tokens at a time turned in shared memory, so that a token's 32 channels leave in 16-byte
          // pieces (stored as they are, 4 bytes a lane, 30 us more). The rows' scales wait for the weighted sum:
          // their loads ahead of every tile took 36 us.
          float* turn4 = reinterpret_cast<float*>(turn);
          const int ch4 = t.mt * kChannels + quad * 32 + (lane & 7) * 4;
#pragma unroll
          for (int half = 0; half < 32; half += 16) {
            if (half >= nc) break;
#pragma unroll
            for (int i = 0; i < 16; ++i) turn4[i * 32 + lane] = __uint_as_float(v[half + i]) * w0;
            __syncwarp();
            float* dst = static_cast<float*>(p.out) + ((int64_t)t.row0 + c0 + half + (lane >> 3)) * p.channels + ch4;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (ch4 < p.channels && half + 4 * i + (lane >> 3) < nc)
                *reinterpret_cast<float4*>(dst + (int64_t)4 * i * p.channels) =
                    *reinterpret_cast<const float4*>(turn4 + (4 * i + (lane >> 3)) * 32 + (lane & 7) * 4);
            __syncwarp();
          }
        } else if (p.wide) {
          // 16-bit results: turned in shared memory, so that a token's 32 channels leave in 16-byte pieces
          // (stored as they are, 2 bytes a lane, a tile of 192 tokens took 26,000 cycles)
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 xs = *reinterpret_cast<const float4*>(cs + c0 + i);
            const float f[4] = {__uint_as_float(v[i]) * xs.x * w0, __uint_as_float(v[i + 1]) * xs.y * w0,
                                __uint_as_float(v[i + 2]) * xs.z * w0, __uint_as_float(v[i + 3]) * xs.w * w0};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              turn[(i + j) * 32 + lane] = f16_out ? __half_as_ushort(__float2half_rn(f[j]))
                                                  : __bfloat16_as_ushort(__float2bfloat16_rn(f[j]));
          }
          __syncwarp();
          const int ch8 = t.mt * kChannels + quad * 32 + (lane & 3) * 8;
          uint16_t* dst = static_cast<uint16_t*>(p.out) + ((int64_t)t.row0 + c0 + (lane >> 2)) * p.channels + ch8;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (ch8 < p.channels && 8 * i + (lane >> 2) < nc)
              *reinterpret_cast<uint4*>(dst + (int64_t)8 * i * p.channels) =
                  *reinterpret_cast<const uint4*>(turn + (8 * i + (lane >> 2)) * 32 + (lane & 3) * 8);
          __syncwarp();
        } else {
          const int64_t at = ((int64_t)t.row0 + c0) * p.channels + ch;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (in && i < nc) {
              const float f = __uint_as_float(v[i]) * cs[c0 + i] * w0;
              if (p.out_dtype == MOE_DTYPE_F32) static_cast<float*>(p.out)[at + (int64_t)i * p.channels] = f;
              else static_cast<uint16_t*>(p.out)[at + (int64_t)i * p.channels] = to_16(p.out_dtype, f);
            }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&d_empty[ab]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------------- host
// `box_rows` rows of a step's 128 bytes; zeros past the rows' ends.
cudaError_t encode_weights(CUtensorMap* m, const GemmArgs& a, uint32_t box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)a.K, (cuuint64_t)a.a_rows}, strides[1] = {(cuuint64_t)a.a_stride};
  const cuuint32_t box[2] = {kStep, box_rows};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.a, dims, strides, box);
}
// A step's tokens in one copy: two columns of n rows x 64 values, one behind the other.
// Rows are padded to 64 values, so that a column never reaches into the next row.
cudaError_t encode_tokens(CUtensorMap* m, const GemmArgs& a, uint32_t n) {
  const cuuint64_t dims[3] = {64, (cuuint64_t)a.b_rows, (cuuint64_t)(a.b_stride / 64)};
  const cuuint64_t strides[2] = {(cuuint64_t)a.b_stride * 2, 128};
  const cuuint32_t box[3] = {64, n, kStep / 64};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, a.b, dims, strides, box);
}

template <int KIND>
cudaError_t launch_kind(const Maps& maps, const Params& p, int grid, size_t smem, cudaStream_t s) {
  static bool allowed[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !allowed[dev]) {
    e = cudaFuncSetAttribute(int8_gemm_kernel<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kStageBudget + kFixedSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) allowed[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, int8_gemm_kernel<KIND>, maps, p);
}

thread_local int t_withhold = 0;

}  // namespace

void test_withhold(int on) { t_withhold = on; }

cudaError_t launch_gemm(GemmKind kind, const GemmArgs& a, int num_sms, cudaStream_t s) {
  Maps maps = {};
  cudaError_t e = encode_weights(&maps.a, a, kind == kUp ? 64 : kChannels);
  const int tail = kind == kDense ? ((a.T - 1) % a.block + 16) / 16 * 16 : 0;   // rows of the last tile
  for (int n = 16; n <= a.block && e == cudaSuccess; n += 16)
    if (kind != kDense || n == a.block || n == tail)
      e = encode_tokens(&maps.b[n / 16 - 1], a, n);
  if (e != cudaSuccess) return e;
  Params p = {};
  p.blocks = a.blocks;
  p.num_blocks = a.num_blocks;
  p.max_blocks = a.max_blocks;
  const int per_tile = kind == kUp ? 64 : kChannels;
  p.tiles_m = (a.channels + per_tile - 1) / per_tile;
  p.tiles_t = kind == kDense ? (a.T + a.block - 1) / a.block : 1;
  p.T = a.T;
  p.block = a.block;
  p.channels = a.channels;
  p.rows_per_group = a.rows_per_group;
  p.steps = (a.K + kStep - 1) / kStep;
  // Tokens come from L2 and wait for the MMAs, three stages of the largest; the rest is for the weights,
  // which come from memory. (One ring of three stages for both bounded the dense product at 50 us.)
  p.b_bytes = a.block * kStep * 2;
  p.b_stages = 3 * kMaxBlock * kStep * 2 / p.b_bytes;
  if (p.b_stages > 6) p.b_stages = 6;
  p.raw_stages = (kStageBudget - p.b_stages * p.b_bytes) / kRawBytes;
  if (p.raw_stages > kMaxStages) p.raw_stages = kMaxStages;
  p.row_scale = a.row_scale;
  p.w_scale = a.w_scale;
  p.out = a.out;
  p.out_dtype = a.out_dtype;
  p.withhold = t_withhold;
  p.wide = a.out_dtype != MOE_DTYPE_F32 && a.channels % 8 == 0 && !((uintptr_t)a.out & 15);
  const size_t smem = (size_t)p.b_stages * p.b_bytes + (size_t)p.raw_stages * kRawBytes + kFixedSmem;
  const int64_t tiles = (int64_t)p.tiles_m * (kind == kDense ? p.tiles_t : a.max_blocks);
  const int grid = (int)(tiles < num_sms ? tiles : num_sms);
  switch (kind) {
    case kDense: return launch_kind<kDense>(maps, p, grid, smem, s);
    case kUp: return launch_kind<kUp>(maps, p, grid, smem, s);
    default: return launch_kind<kDown>(maps, p, grid, smem, s);
  }
}

cudaError_t gemm_status(cudaStream_t s, int* code) {
  const int zero = 0;
  cudaError_t e = cudaStreamSynchronize(s);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(code, g_gemm_error, sizeof(int));
  if (e == cudaSuccess && *code) e = cudaMemcpyToSymbol(g_gemm_error, &zero, sizeof(int));
  return e;
}

}  // namespace int8
}  // namespace moe
