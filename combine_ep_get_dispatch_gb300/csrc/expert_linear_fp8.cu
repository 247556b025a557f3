// The experts' products with 8-bit weights on sm_103a: y_row = x_row W_e^T, both
// sides E4M3, with a scale for each 128 channels of a row of x and for each
// 128 x 128 block of W; or x_row W_e, for the gradient of the first.
//
// Mathematics: with steps k of 128 channels,
//   y[r, o] = sum_k (sx[r, k] sw[o / 128, k]) <x[r, k], w[o, k]>,
// the inner products on the tensor cores (E4M3 products are exact, their sums
// fp32). The scales are any fp32 numbers, so no step's sum can be added to
// another's in tensor memory: each step's 128 rows x 256 outputs are read from
// there, scaled by one product per row and 128 outputs, and added to fp32 sums
// in the registers of eight warps, while the tensor cores work on the next step
// in the other half of tensor memory. The rows are the product's 128-row side
// (the lanes of tensor memory), so that a thread holds one row: its scale is one
// number, and a gated output, a row's largest magnitude and its E4M3 codes are
// formed without other threads but one.
//
// The gradient reads the same weights along the other axis: a step's 128
// outputs x 256 inputs enter the product as its transposed operand.
//
// What bounds it: the weights, read once from HBM, until an expert has about
// 100 rows; then the way from a step's products to the next ones in the same half
// of tensor memory: 516 cycles of products, 540 in which eight warps read them, and
// 880 from one to the other and back (the products' end seen, the read's end seen,
// the next issued), of which two steps at a time are on their way: 970 a step where
// the products alone would take 516. Halves of that (four of 128 outputs) do not
// help: a product of 128 outputs takes 109 cycles, one of 256 takes 129. Pairs of
// blocks that share the weights (cta_group::2) add as much again to the way. Under
// a load of seconds power comes before all that: 1370 W, at 1.5 to 1.8 GHz.
//
// The work is a list of units, (expert, 256 outputs, tile of up to 128 rows), each a
// run of steps of 128 inputs; one block an SM (see Share). Loads, products,
// scales and results have warps of their own; the loading one finds the block's
// units and passes them on. A unit that several blocks share is joined by the last of
// them to finish, in the order of the steps: the result does not depend on which one
// that was.
//
// Measured (7168 inputs; copy rate 6.69 TB/s; in brackets bursts, before power holds
// the clock down): 256 experts of 4 rows, 2 x 2048 gated outputs in FP8, 1003 us,
// 7.4 TB/s; about 128 rows, 1430 us (1290, 6.1 TB/s); one token's eight experts 42 us;
// 32 experts of 2048 rows, 4096 outputs, 1700 us, 2.26 PFLOP/s (1520, 2.53); the
// gradient of 16 experts of 1537 rows, 4096 to 7168, 725 us, 1.99 PFLOP/s (690, 2.09).
#include <algorithm>

#include "common.cuh"
#include "expert_tiles.cuh"
#include "kernels.cuh"
#include "tensor.cuh"

namespace ep {

namespace {

constexpr int kStep = 128;              // inputs a step
constexpr int kTileRows = 128;          // rows of the product (lanes of tensor memory)
constexpr int kTileN = 256;             // its outputs: with GLU 128 gates and their ups
constexpr int kBlock = 128;             // outputs that share a scale
constexpr unsigned kTileBytes = kTileN * kStep;
constexpr int kRowMaps = kTileRows / 16;  // boxes of 16, 32 .. 128 rows
constexpr int kMaxBlocks = 160;         // blocks a workspace has room for
constexpr int kThreads = 384;           // loads, products, scales (four warps), results (eight)
constexpr int kResultThreads = 256;
constexpr int kFewRows = 8;             // rows of a tile that a warp each finishes
constexpr unsigned kFewBytes = kFewRows * kTileN * sizeof(float);
constexpr int kMaxStages = 8;
constexpr int kTmemCols = 512;          // two steps' sums
constexpr int kMinStages = 2;           // fewest steps worth a block of their own
constexpr int kMaxParts = 4;            // most blocks that share a unit
constexpr int kJobs = 4;                // jobs between the loads and the results
constexpr int kTakeAhead = 8;           // steps before a unit's end at which the next is taken
constexpr int kAhead = 4;               // steps' scales in flight
// The scales of step i are handed over once those of step i + kAhead - 1 are on
// their way, whose job has been passed on by then. It has if all loads before it
// have been issued, for which the products of step i + kAhead - 2 - stages and the
// results of step i + kAhead - 4 - stages have to be done, and if the results of job
// i + kAhead - 1 - kJobs are (a job may be one step): all before step i.
static_assert(kAhead <= kJobs && kAhead <= 4, "scales would be waited for by what they wait for");
// Registers of a thread: 168 at launch, of which four warps give 80 each to the
// eight that hold the sums (3 x 168 = 88 + 2 x 208).
constexpr int kLoadRegs = 88, kResultRegs = 208;

struct Params {
  ExpertLinearFp8Params p;
  int tile_rows;  // rows of a full tile
  int KS;         // steps of a unit: blocks of 128 inputs
  int MT;         // units of a tile: an expert's output tiles
  int stages;
  unsigned stage_bytes;
  int scale_rows, scale_cols;  // blocks of W in either direction
  unsigned* counters;          // [kMaxBlocks]: arrivals at a shared unit
  unsigned* taken;             // whole units that blocks have taken, and blocks that are done
  float* partial;              // [kMaxBlocks][2][tile_rows][kTileN]
};

// A run of steps of one unit, as the loading warp passes it on.
struct Job {
  int steps;        // 0: no more jobs
  int e, mt, s0;    // expert, output tile, first step
  int row, rows;    // the tile's rows: the first, in x, and how many
  int first, last;  // the blocks that share the unit
};

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t job_full[kJobs], job_empty[kJobs];
  Job job[kJobs];
  uint32_t tmem;
  int last;                            // this block is the last to finish its shared unit
  Scan<kThreads> scan;
  float scale[2][2][kTileRows];        // [step's half of tensor memory][128 outputs][row]
  float top[2][2][kTileRows];          // FP8 results: [warpgroup][128 outputs][row]
};

struct RowMaps {
  CUtensorMap box[kRowMaps];
};

// How the blocks share the units. As many as make full rounds of all blocks are
// taken whole, one after the other as blocks become free; so units that follow
// one another are worked on at the same time, and what they share (rows that read
// the same weights, outputs that read the same rows) comes from HBM once. The
// rest comes first, cut into equal runs of steps. (With every unit in one such cut
// the blocks were at different places of their units and of the list: 32 experts
// of 2048 rows, 7168 inputs, 4096 outputs took 2650 us. With a fixed list for each
// block they drifted apart: 256 experts of about 128 rows read 9.6 GB where 7.8 must
// be, and took 1498 us.)
struct Share {
  int units, KS, blocks;
  int cut, cutters;  // units that are cut, blocks that share them
  int at, end;       // this block's steps of them
  // few: the tiles have up to kFewRows rows on average.
  __device__ Share(int units, int KS, int blocks, int me, bool few) : units(units), KS(KS), blocks(blocks) {
    // With fewer units than blocks, cutting them saves a block three quarters of a
    // unit's steps (kMaxParts), or what the blocks at hand allow: half of them feed all
    // of HBM's rate, so that from blocks / 2 units on nothing is saved. The join costs
    // as much as 6 steps with few rows and 22 with more (a step is 0.36 us), and 10 and
    // 31 where the cuts fall unevenly on the units. (One expert's units, whole / cut, in us;
    // 7168 inputs, 1 row: 16 units 28.1 / 15.4, 38 28.8 / 19.5, 60 29.5 / 28.1, 68 29.7 / 29.9;
    // 128 rows: 16 30.8 / 24.9, 38 31.2 / 29.8, 48 32.1 / 36.3. 2048 inputs, 1 row: 16 12.6 / 11.2,
    // 38 13.1 / 12.9, 48 13.2 / 15.7; 32 rows: 16 12.7 / 16.8, 48 13.2 / 21.6. 1024 inputs, 1 row:
    // 4 8.6 / 8.5, 48 10.5 / 14.1. 16384 inputs, 9 rows: 56 57.1 / 52.3.)
    const bool even = kMaxParts * units <= blocks;
    const int saved = KS * (blocks - max(2 * units, blocks / 4)) / blocks;
    const int join = few ? (even ? 6 : 10) : even ? 22 : 31;
    cut = units < blocks && saved <= join ? 0 : units % blocks;
    // Every block that takes part has steps: the join counts on it. (Of 32 experts
    // of 128 rows 8 units are left to cut: in us, shared by 2, 4, 8, 16 and 19 blocks
    // each, 232, 229, 237, 260 and 273.)
    cutters = min(min(blocks, kMaxParts * cut), max(cut * KS / kMinStages, 1));
    at = end = 0;
    if (me < cutters) {
      at = begin(me);
      end = begin(me + 1);
    }
  }
  __device__ __forceinline__ int begin(int block) const {
    return cut * KS * block / cutters;  // (below 160 * 128 * 160)
  }
  // The block that has step i of the cut units.
  __device__ __forceinline__ int owner(int i) const {
    const int total = cut * KS;
    return ((i + 1) * cutters + total - 1) / total - 1;
  }
};

// Where a unit lies, by a whole warp. An expert's tiles share its rows evenly:
// blocks that work on tiles of different sizes drift apart (256 experts of about
// 128 rows: 1783 us with tiles of 128 rows and the rest, 1498 so).
__device__ __forceinline__ void locate(const Params& q, const Tables& tb, int unit, Job& j) {
  j.e = uniform(expert_of(tb.tile0, q.p.E, unit / q.MT));
  const int tile0 = uniform(tb.tile0[j.e]), tiles = uniform(tb.tile0[j.e + 1]) - tile0;
  const int u = unit - tile0 * q.MT;
  j.mt = u / tiles;
  const int rows = uniform(tb.rows[j.e]), per = (rows + tiles - 1) / tiles, row = (u - j.mt * tiles) * per;
  j.row = uniform(tb.slot0[j.e]) + row;
  j.rows = min(per, rows - row);
}

// A warp's place in the list of jobs.
struct Jobs {
  int at = 0;
  unsigned parity = 0;
  // Whether there is a next job, at job[at]; by a whole warp (false too if the wait
  // has run out). done() gives its place back.
  __device__ __forceinline__ bool next(Shared& sh, int32_t* status) {
    return mbar_wait_warp(&sh.job_full[at], parity, status) && uniform(sh.job[at].steps) > 0;
  }
  __device__ __forceinline__ void done(Shared& sh) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.job_empty[at]);
    advance();
  }
  __device__ __forceinline__ void advance() {
    if (++at == kJobs) {
      at = 0;
      parity ^= 1;
    }
  }
};

__device__ __forceinline__ void result_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Whether all of the results' threads go on: none may leave alone.
__device__ __forceinline__ bool results_agree(bool ok) {
  unsigned r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u)
      : "memory");
  return r != 0;
}

// 32 columns of tensor memory have arrived in r. (Each register is an operand: what
// reads one that is not may be moved in front of the wait.)
__device__ __forceinline__ void arrived(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// sums += s * r.
__device__ __forceinline__ void add_scaled(uint64_t* sums, const uint32_t (&r)[32], uint64_t s) {
#pragma unroll
  for (int i = 0; i < 16; ++i)
    sums[i] = fma_f32x2(pack_f32x2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), s, sums[i]);
}

// A scale of x: fp32, or the power of two that a UE8M0 byte stands for.
__device__ __forceinline__ float row_scale(const ExpertLinearFp8Params& p, int64_t at) {
  if (!p.x_ue8m0) return __ldg(static_cast<const float*>(p.x_scale) + at);
  const uint32_t b = __ldg(static_cast<const uint8_t*>(p.x_scale) + at);
  return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7FC00000u : b << 23);
}

// silu(g): the exponential within 2 ulp, the reciprocal within 1, and no branch.
// (With an IEEE division, whose rare cases are a call, a unit's 64 gates and 64
// quotients a thread took as long as the products of 30 steps.)
__device__ __forceinline__ float silu(float g) {
  const float e = expf(-fabsf(g));
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.0f + e));  // (of a number from 1 to 2)
  return g * (g < 0.0f ? e * y : y);
}

// Eight results to BF16.
__device__ __forceinline__ uint4 bf16x8(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// A row's 64 results, outputs o .. o + 63. (32 bytes a store, a whole sector: with
// 16 a unit's results took 7 us, in which the products of 18 steps could be made.)
__device__ __forceinline__ void store_bf16(const ExpertLinearFp8Params& p, const float (&v)[64], int64_t row, int o,
                                           int outs) {
  uint16_t* to = static_cast<uint16_t*>(p.y) + row * outs + o;
  const bool whole = (reinterpret_cast<uintptr_t>(to) & 31) == 0;
#pragma unroll
  for (int i = 0; i < 64; i += 16) {
    const uint4 a = bf16x8(v + i), b = bf16x8(v + i + 8);
    if (whole && o + i + 8 < outs) {
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + i), "r"(a.x), "r"(a.y), "r"(a.z),
                   "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                   : "memory");
    } else {
      if (o + i < outs) *reinterpret_cast<uint4*>(to + i) = a;
      if (o + i + 8 < outs) *reinterpret_cast<uint4*>(to + i + 8) = b;
    }
  }
}

// The largest magnitude of 64 results (a NaN is left out).
__device__ __forceinline__ float largest(const float (&v)[64]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 64; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}

// The scale of 128 results of which m is the largest magnitude, as the dispatch
// quantises rows, and where it goes.
__device__ __forceinline__ float scale_of(const ExpertLinearFp8Params& p, float m) {
  float sc = __fdiv_rn(m, 448.0f);
  if (p.out_pow2 && sc > 0.0f) sc = pow2_ceil(sc);
  if (p.out_ue8m0 && m > 0.0f) sc = fmaxf(sc, __uint_as_float(0x00400000u));  // 2^-127
  return sc;
}
__device__ __forceinline__ void store_scale(const ExpertLinearFp8Params& p, float sc, int64_t row, int block, int outs) {
  const int64_t at = row * (outs / kBlock) + block;
  if (p.out_ue8m0)
    static_cast<uint8_t*>(p.y_scale)[at] = ue8m0_byte(sc);
  else
    static_cast<float*>(p.y_scale)[at] = sc;
}

// v / sc in E4M3, 64 of them. kQuick: correctly rounded from one correctly rounded
// reciprocal y, by which the quotient t = v y is within an ulp, its remainder v - sc t
// exact by a fused multiply-add, and t + remainder y rounds to v / sc (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// IBM J. Res. Dev. 34(1), 1990), as long as the remainder does not underflow where a
// code is not a zero (sc >= 2^-92) and y is a normal number (sc <= 2^126).
template <bool kQuick>
__device__ __forceinline__ void store_codes(const float (&v)[64], float sc, uint8_t* to) {
  const float y = kQuick ? __frcp_rn(sc) : 0.0f;
  const uint64_t y2 = pack_f32x2(y, y), s2 = pack_f32x2(-sc, -sc);
#pragma unroll
  for (int i = 0; i < 64; i += 16) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
      const float x0 = v[i + j], x1 = v[i + j + 1];
      float u0, u1;
      if (kQuick) {
        const uint64_t x = pack_f32x2(x0, x1), t = mul_f32x2(x, y2);
        unpack_f32x2(fma_f32x2(fma_f32x2(s2, t, x), y2, t), u0, u1);
        // (a zero keeps its sign)
        u0 = __uint_as_float(__float_as_uint(u0) | (__float_as_uint(x0) & 0x80000000u));
        u1 = __uint_as_float(__float_as_uint(u1) | (__float_as_uint(x1) & 0x80000000u));
      } else {
        u0 = sc > 0.0f ? __fdiv_rn(x0, sc) : x0;
        u1 = sc > 0.0f ? __fdiv_rn(x1, sc) : x1;
      }
      w[j / 4] |= pack_e4m3x2(u0, u1) << (8 * (j & 2));
    }
    *reinterpret_cast<uint4*>(to + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ... and to E4M3, with the scale of the 128 results that they are part of.
__device__ __forceinline__ void store_fp8(const ExpertLinearFp8Params& p, const float (&v)[64], float m, int64_t row,
                                          int o, int outs, bool writes_scale) {
  const float sc = scale_of(p, m);
  uint8_t* to = static_cast<uint8_t*>(p.y) + row * outs + o;
  if (sc >= 0x1p-92f && sc <= 0x1p126f)
    store_codes<true>(v, sc, to);
  else
    store_codes<false>(v, sc, to);
  if (writes_scale) store_scale(p, sc, row, o / kBlock, outs);
}

// A row's results by a warp: lane l has outputs 4 l .. 4 l + 3 of either 128 (a, b).
__device__ __forceinline__ void finish_row(const ExpertLinearFp8Params& p, float4 a, float4 b, int64_t row, int mt,
                                           int outs) {
  const int lane = threadIdx.x & 31;
  const auto store = [&](const float4& v, int block) {
    const int o = block * kBlock + 4 * lane;
    if (!p.out_fp8) {
      if (o < outs)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + row * outs + o) =
            make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
      return;
    }
    if (block * kBlock >= outs) return;
    const float m = fmaxf(fmaxf(fmaxf(0.0f, fabsf(v.x)), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));  // (no NaN)
    const float sc = scale_of(p, __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m))));
    const float d = sc > 0.0f ? sc : 1.0f;
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.y) + row * outs + o) =
        pack_e4m3x2(__fdiv_rn(v.x, d), __fdiv_rn(v.y, d)) | pack_e4m3x2(__fdiv_rn(v.z, d), __fdiv_rn(v.w, d)) << 16;
    if (lane == 0) store_scale(p, sc, row, block, outs);
  };
  if (p.glu) {
    store(make_float4(silu(a.x) * b.x, silu(a.y) * b.y, silu(a.z) * b.z, silu(a.w) * b.w), mt);
  } else {
    store(a, 2 * mt);
    store(b, 2 * mt + 1);
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    expert_linear_fp8_kernel(const Params q, const __grid_constant__ CUtensorMap map,
                             const __grid_constant__ RowMaps maps) {
  extern __shared__ uint8_t dynamic[];
  // The stages start on a 1024-byte boundary (the swizzle's period).
  uint8_t* smem = dynamic + (1024 - (smem_addr(dynamic) & 1023)) % 1024;
  __shared__ Shared sh;
  const ExpertLinearFp8Params& p = q.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  const Tables tb(reinterpret_cast<int*>(smem + q.stages * q.stage_bytes + kFewBytes), p.E);
  if (tid == 0) {
    for (int i = 0; i < q.stages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.acc_full[i], 1 + 2);   // the products, two warps of scales
      mbar_init(&sh.acc_empty[i], kResultThreads / 32);
    }
    for (int i = 0; i < kJobs; ++i) {
      mbar_init(&sh.job_full[i], 1);
      mbar_init(&sh.job_empty[i], 1 + 2 + kResultThreads / 32);
    }
    fence_mbar_init();
  }
  if (tid == 32) prefetch_map(&map);
  if (tid >= 64 && tid < 64 + q.tile_rows / 16) prefetch_map(&maps.box[tid - 64]);
  grid_dependency_wait();
  // (Tensor memory only now: a kernel that this one waits for may still ask for some.)
  if (warp == 3) tmem_alloc(&sh.tmem, kTmemCols);
  tile_experts<true>(q, sh.scan, tb);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  launch_dependents();
  const uint32_t tmem = uniform(sh.tmem);
  const int outs = p.glu ? p.M / 2 : p.M;
  // A stage: rows of x, then weights (a product always reads 128 rows: with
  // fewer, the lanes behind them hold nothing that is looked at).
  const unsigned w_at = static_cast<unsigned>(q.tile_rows) * kStep;

  if (warp < 4) {
    give_registers<kLoadRegs>();
    if (warp == 0) {
      // Loads. This warp finds the block's jobs and passes them on.
      const int tiles = uniform(tb.tile0[p.E]);
      const unsigned rows =  // of all tiles, from their scan
          __reduce_add_sync(0xffffffffu, lane < kThreads / 32 ? static_cast<unsigned>(sh.scan.rows[lane]) : 0u);
      Share share(tiles * q.MT, q.KS, gridDim.x, blockIdx.x, rows <= static_cast<unsigned>(kFewRows * tiles));
      Ring r;
      Jobs jobs;
      bool again = false, jobs_again = false;  // the rings have been filled once
      int next = share.cut + blockIdx.x;       // the next whole unit, in the first lane
      uint64_t filled = 0x0808080808080808ull;  // boxes of rows that each stage may hold
      auto take = [&]() {
        if (lane == 0) next = share.cut + gridDim.x + static_cast<int>(atomicAdd(q.taken, 1u));
      };
      auto pass_on = [&](const Job& j) {
        if (jobs_again && !mbar_wait_warp(&sh.job_empty[jobs.at], jobs.parity ^ 1, p.status)) return false;
        if (lane == 0) {
          sh.job[jobs.at] = j;
          mbar_arrive(&sh.job_full[jobs.at]);
        }
        __syncwarp();
        jobs.advance();
        if (jobs.at == 0) jobs_again = true;
        return true;
      };
      auto load = [&](const Job& j, int take_at) {
        const int boxes = (j.rows + 15) / 16;
        const unsigned bytes = kTileBytes + boxes * 16 * kStep;
        const CUtensorMap* box = &maps.box[boxes - 1];
        for (int st = j.s0; st < j.s0 + j.steps; ++st) {
          if (st == take_at) take();
          if (again && !mbar_wait_warp(&sh.empty[r.stage], r.parity ^ 1, p.status)) return false;
          // Rows behind the tile's are products too. What an earlier tile left there is
          // cleared: products of zeros take less power, and under a steady load power
          // holds the clock down (256 experts of about 128 rows, at 1.6 GHz: 1607 us, so 1565).
          const int held = static_cast<int>(filled >> 8 * r.stage & 15);
          if (boxes < held) {
            uint4* rest = reinterpret_cast<uint4*>(smem + r.offset + boxes * 16 * kStep);
            for (int i = lane; i < (min(held, q.tile_rows / 16) - boxes) * kStep; i += 32) rest[i] = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
          }
          filled += static_cast<uint64_t>(boxes - held) << 8 * r.stage;
          if (elect_one()) {
            uint64_t* bar = &sh.full[r.stage];
            uint8_t* to = smem + r.offset;
            mbar_arrive_expect_tx(bar, bytes);
            if (p.transposed)
              tma_load_4d(to + w_at, &map, 0, st * kStep, j.mt * 2, j.e, bar);
            else
              tma_load_4d(to + w_at, &map, st * kStep, j.mt * (p.glu ? kBlock : kTileN), 0, j.e, bar);
            tma_load_2d(to, box, st * kStep, j.row, bar);
          }
          __syncwarp();
          r.advance(q);
          if (r.stage == 0) again = true;
        }
        return true;
      };
      bool ok = true;
      while (ok) {
        Job j;
        int take_at = -1;
        if (share.at < share.end) {
          const int unit = share.at / q.KS, at = unit * q.KS;
          locate(q, tb, unit, j);
          j.s0 = share.at - at;
          j.steps = min(q.KS - j.s0, share.end - share.at);
          j.first = share.owner(at);
          j.last = share.owner(at + q.KS - 1);
          share.at += j.steps;
        } else {
          const int unit = uniform(next);
          j.s0 = j.first = j.last = 0;
          j.steps = 0;
          if (unit < share.units) {
            locate(q, tb, unit, j);
            j.steps = q.KS;
            take_at = max(q.KS - kTakeAhead, 0);
          }
        }
        ok = pass_on(j) && load(j, take_at);
        if (j.steps == 0) break;
      }
      if (!ok) {  // given up: loads in flight land before the block ends
        for (int i = 0; i < q.stages; ++i) mbar_drain(&sh.full[i], i < r.stage ? r.parity : r.parity ^ 1);
      }
    } else if (warp == 1) {
      // Products.
      const uint32_t base = smem_addr(smem);
      const uint64_t a0 = desc_rows128(base);
      const uint64_t b0 = p.transposed ? desc_inputs128(base + w_at, kBlock * kStep) : desc_rows128(base + w_at);
      // 32 inputs on: 32 bytes of a row, or 32 rows of 128 bytes.
      const unsigned b_step = (p.transposed ? 32 * 128 : 32) >> 4;
      const uint32_t idesc = idesc_e4m3(kTileRows, kTileN, p.transposed);
      Jobs jobs;
      Ring r;
      unsigned i = 0;
      bool ok = true;
      while (ok && jobs.next(sh, p.status)) {
        const unsigned end = i + uniform(sh.job[jobs.at].steps);
        jobs.done(sh);
        for (; i < end; ++i) {
          const unsigned half = i & 1;
          if (!mbar_wait_warp(&sh.full[r.stage], r.parity, p.status)) {
            mbar_drain(&sh.full[r.stage], r.parity);
            ok = false;
            break;
          }
          if (i >= 2 && !mbar_wait_warp(&sh.acc_empty[half], (i / 2 - 1) & 1, p.status)) {
            ok = false;
            break;
          }
          tmem_fence_after();
          if (elect_one()) {
            const uint64_t a = a0 + (r.offset >> 4), b = b0 + (r.offset >> 4);
            const uint32_t d = tmem + half * kTileN;
#pragma unroll
            for (unsigned j = 0; j < kStep / 32; ++j) mma_e4m3(d, a + 2 * j, b + b_step * j, idesc, j > 0);
            mma_commit(&sh.empty[r.stage]);
            mma_commit(&sh.acc_full[half]);
          }
          __syncwarp();
          r.advance(q);
        }
      }
    } else {
      // Scales: each lane of the two warps the products of two rows' scales with
      // the weights' for 2 x 128 outputs. Their loads run kAhead steps ahead, across units.
      const int t = tid - 64;
      Jobs jobs;
      bool more = true;
      int left = 0, rows = 0;       // of the job: steps, rows
      int64_t xa = 0;               // the next step's first scale of x,
      const float* w = nullptr;     // and of the weights,
      int w_next = 0, w_second = 0; // how far the next and the second 128 outputs' are
      float x0[kAhead], x1[kAhead], w0[kAhead], w1[kAhead];
      unsigned fetched = 0;
      auto fetch = [&](int i) {
        if (!more) return;
        if (left == 0) {
          more = jobs.next(sh, p.status);
          if (!more) return;
          const Job& j = sh.job[jobs.at];
          left = j.steps;
          rows = j.rows;
          xa = static_cast<int64_t>(j.row + t) * q.KS + j.s0;
          w = p.w_scale + static_cast<int64_t>(j.e) * q.scale_rows * q.scale_cols;
          const int b = p.glu ? j.mt : 2 * j.mt;  // first of the unit's two blocks of outputs
          if (p.transposed) {
            w += static_cast<int64_t>(j.s0) * q.scale_cols + b;
            w_next = q.scale_cols;
            w_second = b + 1 < q.scale_cols ? 1 : 0;
          } else {
            w += static_cast<int64_t>(b) * q.scale_cols + j.s0;
            w_next = 1;
            w_second = p.glu ? q.scale_rows / 2 * q.scale_cols : b + 1 < q.scale_rows ? q.scale_cols : 0;
          }
          jobs.done(sh);
        }
        x0[i] = t < rows ? row_scale(p, xa) : 0.0f;
        x1[i] = t + 64 < rows ? row_scale(p, xa + 64 * static_cast<int64_t>(q.KS)) : 0.0f;
        w0[i] = __ldg(w);
        w1[i] = __ldg(w + w_second);
        ++xa;
        w += w_next;
        --left;
        ++fetched;
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) fetch(i);
      bool ok = true;
      for (unsigned i0 = 0; ok && i0 < fetched; i0 += kAhead) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const unsigned i = i0 + j, half = i & 1;
          if (!ok || i >= fetched) continue;
          if (i >= 2) ok = mbar_wait_warp(&sh.acc_empty[half], (i / 2 - 1) & 1, p.status);
          if (!ok) continue;
          sh.scale[half][0][t] = x0[j] * w0[j];
          sh.scale[half][1][t] = x0[j] * w1[j];
          sh.scale[half][0][t + 64] = x1[j] * w0[j];
          sh.scale[half][1][t + 64] = x1[j] * w1[j];
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.acc_full[half]);
          fetch(j);
        }
      }
    }
  } else {
    take_registers<kResultRegs>();
    // Results: a thread holds one row, of either 128 outputs of the unit the half
    // that its warpgroup has.
    const int group = (warp - 4) >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t mine = tmem + (static_cast<uint32_t>(warp & 3) << 21) + group * 64;
    Jobs jobs;
    unsigned step = 0;
    bool ok = true;  // a warp whose wait has run out goes on without waiting: the others meet it
    while (results_agree(jobs.next(sh, p.status))) {
      const Job& g = sh.job[jobs.at];
      uint64_t sums[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) sums[i] = 0;
      const bool live = (warp & 3) * 32 < g.rows;  // some row of this warp's
      const unsigned end = step + uniform(g.steps);
#pragma unroll 1
      for (; step < end; ++step) {
        const unsigned half = step & 1;
        if (ok) ok = mbar_wait_warp(&sh.acc_full[half], step / 2 & 1, p.status);
        uint32_t v[32], u[32];
        if (ok && live) {
          tmem_fence_after();
          const uint32_t at = mine + half * kTileN;
          tmem_load32(v, at);
          const float s0 = sh.scale[half][0][r], s1 = sh.scale[half][1][r];
          const uint64_t t0 = pack_f32x2(s0, s0), t1 = pack_f32x2(s1, s1);
          arrived(v);
          tmem_load32(u, at + 32);
          add_scaled(sums, v, t0);
          arrived(u);
          tmem_load32(v, at + kBlock);
          add_scaled(sums + 16, u, t0);
          arrived(v);
          tmem_load32(u, at + kBlock + 32);
          add_scaled(sums + 32, v, t1);
          arrived(u);
          tmem_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.acc_empty[half]);
          add_scaled(sums + 48, u, t1);
        } else if (lane == 0) {
          mbar_arrive(&sh.acc_empty[half]);
        }
      }
      // With few rows a lane would form 64 gated outputs alone, and join them alone: a
      // warp takes a row instead. (One token's eight experts 45.0 us, so 43.2; four rows,
      // 16 units in four parts each, 24.0, so 17.6.)
      const bool few = g.rows <= kFewRows;
      bool finishes = true;
      if (g.steps != q.KS) {
        // A shared unit: the last block to arrive adds the parts, in order.
        const int me = blockIdx.x, c_first = g.first, c_last = g.last;
        // Four sums of a row beside the next row's four.
        const int n = g.rows;
        auto parts = [&](int block, bool starts) {
          return reinterpret_cast<float4*>(q.partial) +
                 (static_cast<int64_t>(block) * 2 + (starts ? 1 : 0)) * (kTileN / 4) * q.tile_rows;
        };
        auto part = [&](int block, bool starts) { return parts(block, starts) + group * 32 * n + r; };
        if (r < n) {
          float4* to = part(me, g.s0 == 0);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float4 f;
            unpack_f32x2(sums[2 * i], f.x, f.y);
            unpack_f32x2(sums[2 * i + 1], f.z, f.w);
            __stcg(to, f);
            to += n;
          }
        }
        result_sync();
        if (tid == kThreads - kResultThreads) {
          unsigned* counter = q.counters + c_first;
          __threadfence();  // the block's writes, which the barrier has ordered before it
          const bool last = atomicAdd(counter, 1u) == static_cast<unsigned>(c_last - c_first);
          if (last) *counter = 0u;
          __threadfence();
          sh.last = last;
        }
        result_sync();
        const bool last = sh.last;
        if (last && few) {
          // A warp a row: all of a row's sums of all parts on their way at once.
          const int mine = warp - 4;
          if (mine < n) {
            float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = a;
#pragma unroll 4
            for (int first = c_first; first <= c_last; ++first) {
              const float4* from = parts(first, first == c_first) + (lane >> 4) * 32 * n + (lane & 15) * n + mine;
              const float4 x = __ldcg(from), y = __ldcg(from + 16 * n);
              a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
              b.x += y.x, b.y += y.y, b.z += y.z, b.w += y.w;
            }
            finish_row(p, a, b, g.row + mine, g.mt, outs);
          }
        } else if (last && r < n) {
          // (Of two parts this block has one at hand, and which comes first makes no difference.)
          const bool two = c_last == c_first + 1;
          if (!two) {
#pragma unroll
            for (int i = 0; i < 64; ++i) sums[i] = 0;
          }
#pragma unroll 1
          for (int b = c_first; b <= c_last; ++b) {
            if (two && b == me) continue;
            const float4* from = part(b, b == c_first);
#pragma unroll
            for (int i0 = 0; i0 < 32; i0 += 16) {  // (as many loads in flight as registers are free)
              float4 f[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) f[i] = __ldcg(from + i * n);
              from += 16 * n;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                uint64_t* to = sums + 2 * (i0 + i);
                to[0] = add_f32x2(to[0], pack_f32x2(f[i].x, f[i].y));
                to[1] = add_f32x2(to[1], pack_f32x2(f[i].z, f[i].w));
              }
              asm volatile("" ::: "memory");
            }
          }
        }
        result_sync();  // sh.last is free again
        finishes = last && !few;
      }
      if (finishes && few) {
        float4* rows = reinterpret_cast<float4*>(smem + q.stages * q.stage_bytes);
        if (r < g.rows) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float4 f;
            unpack_f32x2(sums[2 * i], f.x, f.y);
            unpack_f32x2(sums[2 * i + 1], f.z, f.w);
            rows[r * (kTileN / 4) + group * 16 + (i < 16 ? i : i + 16)] = f;
          }
        }
        result_sync();
        const int mine = warp - 4;
        if (mine < g.rows) {
          const float4 a = rows[mine * (kTileN / 4) + lane], b = rows[mine * (kTileN / 4) + 32 + lane];
          finish_row(p, a, b, g.row + mine, g.mt, outs);
        }
        result_sync();
      } else if (finishes) {
        // Finished sums: the first 128 outputs' half (with GLU the gates'), then the second's.
        const int64_t row = g.row + r;
        const bool writes = r < g.rows;
        float a[64], b[64];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          unpack_f32x2(sums[i], a[2 * i], a[2 * i + 1]);
          unpack_f32x2(sums[32 + i], b[2 * i], b[2 * i + 1]);
        }
        int o = g.mt * kTileN + group * 64;
        if (p.glu) {
          o = g.mt * kBlock + group * 64;
#pragma unroll
          for (int i = 0; i < 64; ++i) a[i] = silu(a[i]) * b[i];
        }
        if (p.out_fp8) {
          // The other half of a row's 128 outputs is in the other warpgroup.
          sh.top[group][0][r] = largest(a);
          if (!p.glu) sh.top[group][1][r] = largest(b);
          result_sync();
          if (writes) store_fp8(p, a, fmaxf(sh.top[0][0][r], sh.top[1][0][r]), row, o, outs, group == 0);
          if (writes && !p.glu && o + kBlock < outs)
            store_fp8(p, b, fmaxf(sh.top[0][1][r], sh.top[1][1][r]), row, o + kBlock, outs, group == 0);
          result_sync();
        } else if (writes) {
          store_bf16(p, a, row, o, outs);
          if (!p.glu) store_bf16(p, b, row, o + kBlock, outs);
        }
      }
      jobs.done(sh);
    }
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (warp == 3) {
    tmem_fence_after();
    tmem_free(tmem, kTmemCols);
  }
  if (tid == 0) {  // the last block leaves the list as it was
    __threadfence();
    if (atomicAdd(q.taken + 1, 1u) == gridDim.x - 1) q.taken[0] = q.taken[1] = 0u;
  }
}

// Rows of a full tile: enough for nearly every expert's rows in one tile (the
// mean and four standard deviations of a random routing), so that weights are
// not read again, and no more, since a smaller tile leaves room for more stages
// of weights in flight.
int tile_rows_for(int E, int64_t max_rows) {
  const int64_t active = std::max<int64_t>(1, std::min<int64_t>(E, max_rows));
  const int64_t mean = (max_rows + active - 1) / active;
  int64_t sd4 = 4;
  while (sd4 * sd4 < 16 * mean) ++sd4;
  for (int cap = 16; cap < kTileRows; cap *= 2)
    if (cap >= mean + sd4) return cap;
  return kTileRows;
}

size_t partial_bytes(int tile_rows) { return sizeof(float) * kMaxBlocks * 2 * tile_rows * kTileN; }

cudaError_t launch_products(const Params& q, const CUtensorMap& map, const RowMaps& maps, size_t smem, int dev, int sms,
                            cudaStream_t s) {
  const auto kernel = expert_linear_fp8_kernel;
  const cudaError_t err = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), dev, smem);
  if (err != cudaSuccess) return err;
  return launch_kernel(kernel, dim3(std::min(sms, kMaxBlocks)), dim3(kThreads), smem, s, /*dependent=*/true, q, map,
                       maps);
}

}  // namespace

bool expert_linear_fp8_units_ok(int E, int64_t max_rows, int M, bool glu) {
  const int64_t tiles = max_rows / tile_rows_for(E, max_rows) + E, outs = glu ? M / 2 : M;
  return tiles * (outs / (glu ? kBlock : kTileN) + 1) <= INT32_MAX;
}

size_t expert_linear_fp8_ws_bytes(int E, int64_t max_rows) { return 1024 + partial_bytes(tile_rows_for(E, max_rows)); }

cudaError_t launch_expert_linear_fp8(const ExpertLinearFp8Params& p, cudaStream_t s) {
  if (p.max_rows <= 0 || p.x_rows <= 0) return cudaSuccess;
  Params q{};
  q.p = p;
  q.tile_rows = tile_rows_for(p.E, p.max_rows);
  q.KS = p.K / kStep;
  q.MT = p.glu ? (p.M / 2 + kBlock - 1) / kBlock : (p.M + kTileN - 1) / kTileN;
  const int parts = p.glu ? 2 : 1;
  const int out_blocks = parts * ((p.M / parts + kBlock - 1) / kBlock);
  q.scale_rows = p.transposed ? q.KS : out_blocks;
  q.scale_cols = p.transposed ? out_blocks : q.KS;
  q.counters = reinterpret_cast<unsigned*>(p.ws);
  q.taken = q.counters + kMaxBlocks;
  q.partial = reinterpret_cast<float*>(p.ws + 1024);
  q.stage_bytes = kTileBytes + static_cast<unsigned>(q.tile_rows) * kStep;
  const unsigned tables = static_cast<unsigned>(table_bytes(p.E));
  const unsigned most = 227 * 1024 - sizeof(Shared) - 2048 - tables - kFewBytes;
  q.stages = std::min<int>(kMaxStages, most / q.stage_bytes);
  const size_t smem = static_cast<size_t>(q.stages) * q.stage_bytes + kFewBytes + tables + 1024;

  const EncodeTiled encode = encode_tiled();
  if (!encode) return cudaErrorNotSupported;
  CUtensorMap map;
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  // A step's weights in one load: 128 inputs of 256 outputs (of 128 gates and
  // 128 ups), or of the transposed product 128 inputs x two times 128 outputs.
  cuuint64_t dims[4], strides[3];
  cuuint32_t box[4] = {kStep, kBlock, 2, 1};
  const cuuint64_t K = p.K, M = p.M, E = p.E;
  if (p.transposed) {
    dims[0] = kBlock, dims[1] = K, dims[2] = M / kBlock, dims[3] = E;
    strides[0] = M, strides[1] = kBlock, strides[2] = K * M;
  } else {
    dims[0] = K, dims[1] = M / parts, dims[2] = parts, dims[3] = E;
    strides[0] = K, strides[1] = M / parts * K, strides[2] = M * K;
    if (!p.glu) box[1] = kTileN, box[2] = 1;
  }
  if (encode(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(p.w), dims, strides, box, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  RowMaps maps;
  const cuuint64_t xd[2] = {K, static_cast<cuuint64_t>(p.x_rows)};
  for (int i = 0; i < q.tile_rows / 16; ++i) {
    const cuuint32_t b[2] = {kStep, static_cast<cuuint32_t>(16 * (i + 1))};
    if (encode(&maps.box[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(static_cast<const void*>(p.x)), xd,
               &K, b, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  const int dev = current_device();
  const int sms = device_sms(dev);
  if (sms < 1) return cudaErrorInvalidDevice;
  return launch_products(q, map, maps, smem, dev, sms, s);
}

}  // namespace ep
