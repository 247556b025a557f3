// The experts' products with 4-bit weights on sm_103a: y_row = x_row W_e^T.
//
// Mathematics: W's E2M1 codes and UE8M0 scales (32 inputs each) are operands
// of the tensor cores as they are: the block-scaled product multiplies E2M1 by
// E4M3 exactly and applies both sides' power-of-two scales, so no weight is
// ever converted. The weights are the product's 128-row side, the rows of x
// its columns. An E4M3 x enters as it is. A BF16 x enters as two columns: with
// s the smallest power of two that has 448 s >= the largest magnitude of 32
// neighbours, h = e4m3(x / s) and l = e4m3(16 (x / s - h)) with the scale s / 16.
// h keeps 4 of x's 8 significant bits and l the rest down to its finest step,
// 2^-13 s: all of them from 2^-6 s on, which is under 2^-13 of the largest, and
// within 2^-14 s below, under 2^-21.8 of it. The two columns' sums are added at
// the end.
//
// What bounds it: the weights, read once from HBM (4.25 bits each), until an
// expert has about 100 rows. So the work is laid out as one stream of weights:
// every (expert, rows tile, 128 outputs) is a unit of in / 128 steps, and the
// blocks (one an SM) take equal runs of consecutive steps, whatever the
// experts' loads. A unit that several blocks share is joined by the last of
// them to finish: each leaves its fp32 sums in the workspace, and the last
// adds them in the order of the steps, so that the result does not depend on
// which one that was.
//
// Next after HBM comes shared memory: 4-bit codes lie there in 8-bit
// containers, so 256 inputs of 128 outputs are written (32 KB) and read (32 KB)
// at 128 bytes a cycle in 512 of the 750 cycles that HBM gives them; a product
// of 16 columns costs 75 cycles beside those writes, 43 alone, whatever the
// tensor cores could do. Loads ahead of the ring into L2 only cost (995 us
// where 783 were without: every load passes the same engine).
//
// With more rows the blocks' reads of x set the pace: each of an expert's
// output tiles needs all of its rows, and each block loads them for itself
// (x may lie in any memory that the device can read, so no load serves several
// blocks at once). The blocks then work on an expert's output tiles side by
// side, so that its rows come from L2 but for the first time (work_together).
//
// Measured (256 experts, 7168 inputs, 2 x 2048 gated outputs; copy rate 6.69
// TB/s): 4 BF16 rows an expert 637 us, 6.2 TB/s; 128 E4M3 rows 1054 us, 4.1
// TB/s and 1.83 PFLOP/s; one token's eight experts 34 us, of which 10 pass before
// the first weights have come and 4 after the last; 2048 inputs, 7168 outputs, 4
// BF16 rows an expert 330 us, 6.0 TB/s.
//
// Two launches: expert_rows_kernel splits BF16 rows into the tensor cores'
// shared-memory layout (of E4M3 rows it lays out the scales; their codes come
// by tiled loads as they are), expert_linear_kernel is its programmatic
// dependent and starts reading weights meanwhile.
#include <algorithm>

#include "common.cuh"
#include "expert_tiles.cuh"
#include "kernels.cuh"
#include "tensor.cuh"

namespace ep {

namespace {

constexpr int kStep = 128;                  // inputs a step
constexpr int kTileM = 128;                 // outputs a unit (with GLU: 64 gates, 64 ups)
constexpr int kTileBytes = kTileM * kStep;  // weights of a step in shared memory (8-bit containers)
constexpr int kTileTx = kTileBytes / 2;     // ... and as TMA counts them
constexpr int kMaxSteps = 2;                // most steps a stage holds
constexpr int kScaleBytes = 512;            // scale bytes of 128 rows for one step
constexpr int kMaxCols = 192;
constexpr int kRowMaps = kMaxCols / 8;      // boxes of 8, 16 .. kMaxCols rows
constexpr int kMaxBlocks = 160;             // blocks a workspace has room for
constexpr int kThreads = 256;
constexpr int kMaxStages = 12;
constexpr int kTmemCols = 512;              // two accumulators of kMaxCols, then scales
constexpr int kTmemScales = 2 * kMaxCols;
constexpr int kScaleGroups = 6;              // groups of four steps of the weights' scales in shared memory
constexpr int kMinStages = 2;               // fewest stages worth a block of their own
constexpr int kScaleCols = 12;              // columns a step: 4 of the weights', 8 of the rows'

struct Params {
  ExpertLinearParams p;
  int mult;         // columns a row: 2 for BF16, 1 for E4M3
  int tile_rows;    // rows of a full tile
  int cols_cap;     // its columns
  int KB;           // steps of a unit: K / 128
  int steps;        // of a stage, 1 or 2
  int KS;           // stages of a unit; the last one may hold one step of two
  int MT;           // units of a tile: an expert's output tiles
  int stages;
  unsigned stage_bytes;
  int scale_bytes;     // of a step's rows: 512 for each 128 columns that a tile can have
  unsigned* counters;  // [kMaxBlocks]
  float* partial;      // [kMaxBlocks][2][tile_rows][kTileM]
  uint8_t* image;      // rows of x, step by step as shared memory holds them: codes, then scales
};

// ---- rows of x -------------------------------------------------------------------
// Columns of a tile, and the bytes of the image in front of it.
__device__ __forceinline__ int tile_cols(const Params& q, int n, int tile) {
  return round8(min(q.tile_rows, n - tile * q.tile_rows)) * q.mult;
}
__device__ __forceinline__ int64_t image_at(const Params& q, int slot0, int tile0, int tile) {
  const int64_t scales = static_cast<int64_t>(tile0 + tile) * q.KB * q.scale_bytes;
  if (q.mult == 1) return scales;  // the codes of E4M3 rows are not in it
  return scales + (static_cast<int64_t>(slot0) + static_cast<int64_t>(tile) * q.tile_rows) * q.mult * q.p.K;
}

__device__ __forceinline__ unsigned scale_place(int col) {
  return static_cast<unsigned>((col >> 7) * kScaleBytes + (col & 31) * 16 + ((col >> 5) & 3) * 4);
}

constexpr int kRowSpan = 1024;  // inputs of an item

// Items: groups of eight rows, and spans of inputs of BF16 rows; a warp takes a
// row. (One scan of the counts a block; with a scan and a search for each item
// this kernel took 40 us of the 756 for 128 tokens x 256 experts.)
__global__ void __launch_bounds__(kThreads) expert_rows_kernel(const Params q) {
  extern __shared__ int tables[];
  __shared__ Scan<kThreads> sc;
  const ExpertLinearParams& p = q.p;
  const Tables tb(tables, p.E);
  grid_dependency_wait();
  launch_dependents();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  tile_experts(q, sc, tb);
  const int spans = q.mult == 2 ? (p.K + kRowSpan - 1) / kRowSpan : 1;
  const int64_t items = static_cast<int64_t>(tb.slot0[p.E] / 8) * spans;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int group = static_cast<int>(item / spans), part = static_cast<int>(item % spans);
    const int e = expert_of(tb.slot0, p.E, group * 8);
    const int n = tb.rows[e], slot0 = tb.slot0[e], tile0 = tb.tile0[e];
    const int row0 = group * 8 - slot0, j = row0 + w;  // row within the expert
    const int tile = row0 / q.tile_rows, r = j - tile * q.tile_rows;
    const int cols = tile_cols(q, n, tile), rows8 = cols / q.mult;
    uint8_t* image = q.image + image_at(q, slot0, tile0, tile);
    const bool live = j < n;
    const int64_t row = first_row(p, e) + j;
    if (q.mult == 1) {
      // E4M3: a scale byte serves a step's four groups of 32.
      for (int kb = lane; kb < q.KB; kb += 32) {
        const uint32_t s = live ? __ldg(p.x_scale + row * q.KB + kb) : 127u;
        *reinterpret_cast<uint32_t*>(image + static_cast<int64_t>(kb) * q.scale_bytes + scale_place(r)) = s * 0x01010101u;
      }
      continue;
    }
    // Of a stage's steps (the last one may hold one of two): their codes, then their scales.
    const int step = cols * kStep + q.scale_bytes;
    auto codes = [&](int kb) {
      const int h = kb % q.steps;
      return image + static_cast<int64_t>(kb - h) * step + h * cols * kStep;
    };
    auto scales = [&](int kb) {
      const int h = kb % q.steps, n = min(q.steps, q.KB - (kb - h));
      return image + static_cast<int64_t>(kb - h) * step + n * cols * kStep + h * q.scale_bytes;
    };
    // Column c of step kb, 16-byte piece `piece`.
    auto place = [&](int kb, int c, int piece) {
      return codes(kb) + (c >> 3) * 1024 + (c & 7) * 128 + ((piece ^ (c & 7)) << 4);
    };
    // A lane splits 8 inputs, four lanes share a scale. Both columns of a row:
    // its high terms at r, its low terms at rows8 + r.
    const int k1 = min(p.K, (part + 1) * kRowSpan);
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) + row * p.K);
    uint4 raw[kRowSpan / 256];
#pragma unroll
    for (int i = 0; i < kRowSpan / 256; ++i) {
      const int k = part * kRowSpan + i * 256 + lane * 8;
      raw[i] = live && k < k1 ? __ldg(src + k / 8) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kRowSpan / 256; ++i) {
      const int k = part * kRowSpan + i * 256 + lane * 8;
      const uint4 v = raw[i];
      float x[8] = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y),
                    bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w)};
      float m = 0.0f;
      bool finite[8];
#pragma unroll
      for (int a = 0; a < 8; ++a) {
        finite[a] = fabsf(x[a]) <= 3.4028234663852886e38f;
        if (finite[a]) m = fmaxf(m, fabsf(x[a]));
      }
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      // The exponent of the smallest power of two >= m / 448, kept so that the
      // low terms' scale, 2^-4 of it, is a normal number.
      const uint32_t up = (__float_as_uint(__fdiv_rn(m, 448.0f)) + 0x007FFFFFu) >> 23;
      const uint32_t b = up < 5u ? 5u : up;
      const float inv = __uint_as_float((254u - b) << 23);
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        hi[h] = lo[h] = 0;
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          const int at = 4 * h + 2 * a;
          const float nan = __int_as_float(0x7FC00000);
          const float x0 = x[at] * inv, x1 = x[at + 1] * inv;
          const uint32_t c = pack_e4m3x2(finite[at] ? x0 : nan, finite[at + 1] ? x1 : nan);
          uint32_t f2;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f2) : "h"(static_cast<uint16_t>(c)));
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&f2));
          hi[h] |= c << (16 * a);
          lo[h] |= pack_e4m3x2((x0 - f.x) * 16.0f, (x1 - f.y) * 16.0f) << (16 * a);
        }
      }
      // A step's four scale bytes, gathered into its first lane.
      uint32_t s = b;
#pragma unroll
      for (int a = 1; a < 4; ++a) s |= __shfl_down_sync(0xffffffffu, b, 4 * a) << (8 * a);
      if (k >= k1) continue;
      const int kb = k / kStep, piece = (k % kStep) >> 4, half = (k >> 3 & 1) * 8;
      *reinterpret_cast<uint2*>(place(kb, r, piece) + half) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(place(kb, rows8 + r, piece) + half) = make_uint2(lo[0], lo[1]);
      if ((lane & 15) == 0) {
        uint8_t* at = scales(kb);
        *reinterpret_cast<uint32_t*>(at + scale_place(r)) = s;
        *reinterpret_cast<uint32_t*>(at + scale_place(rows8 + r)) = s - 0x04040404u;
      }
    }
  }
}

// ---- the products ------------------------------------------------------------------
struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t scale_full[kScaleGroups], scale_empty[kScaleGroups];
  uint64_t acc_full[2], acc_empty[2];
  uint32_t tmem;
  int last;                       // this block is the last to finish its shared unit
  Scan<kThreads> scan;
  float swap[2][8][64];           // GLU: ups on their way to the gates' threads
};

// A run of steps of one unit.
struct Segment {
  int e, tile, mt;
  int s0, s1;     // stages
  int cols;       // columns of its tile
  int rows;       // rows of its tile
  int slot0, tile0;  // the expert's (see Shared)
  int64_t unit;
};

// Which unit comes v-th in the blocks' runs when experts are worked on together
// (work_together): the j-th unit of run a is the a-th of the units that the
// blocks take at the same time, so that the output tiles of an expert, which read
// the same rows, are worked on side by side. `length` is the units of a run,
// rounded; of the last of `runs`, `full` are left.
struct Order {
  unsigned length, runs, full;
  __device__ __forceinline__ Order(unsigned units, unsigned blocks) {
    length = max(1u, (units + blocks / 2) / blocks);
    runs = (units + length - 1) / length;
    full = units - (runs - 1) * length;
  }
  __device__ __forceinline__ int unit(int64_t v) const {
    const unsigned a = static_cast<unsigned>(v) / length, j = static_cast<unsigned>(v) - a * length;
    return static_cast<int>(j < full ? j * runs + a : full * runs + (j - full) * (runs - 1) + a);
  }
};

// A block's stages: positions [at, end) of units * KS. Behind a first unit
// that had to be looked for, the next ones are counted on.
struct Run {
  int64_t at, end;
  int e = -1;        // expert of the last unit, -1 before the first
  int tile0, tiles;  // its tiles before and in all
  int tile, mt;      // the unit's
};

__device__ __forceinline__ int64_t run_begin(int64_t total, int blocks, int c) { return total * c / blocks; }
// The block that owns position i.
__device__ __forceinline__ int owner_of(int64_t total, int blocks, int64_t i) {
  return static_cast<int>(((i + 1) * blocks + total - 1) / total) - 1;
}

// The next run of steps of one unit, by a whole warp. Tiles of one (expert,
// outputs) follow one another, so that its weights come from L2 after the first.
// (Each role passes here between two units: with divisions and a search each
// time the products of 2048 inputs, eight stages a unit, took 366 us, now 330.)
template <bool kTogether>
__device__ __forceinline__ bool next_segment(const Params& q, const Tables& tb, const Order& order, Run& run, Segment& s) {
  if (run.at >= run.end) return false;
  const int E = q.p.E;
  if (run.e < 0 || kTogether) {
    s.unit = run.at / q.KS;
    s.s0 = static_cast<int>(run.at - s.unit * q.KS);
    const int unit = kTogether ? order.unit(s.unit) : static_cast<int>(s.unit);
    run.e = uniform(expert_of(tb.tile0, E, unit / q.MT));
    run.tile0 = uniform(tb.tile0[run.e]);
    run.tiles = uniform(tb.tile0[run.e + 1]) - run.tile0;
    const int u = unit - run.tile0 * q.MT;
    run.mt = u / run.tiles;
    run.tile = u - run.mt * run.tiles;
  } else {
    ++s.unit;
    s.s0 = 0;
    if (++run.tile == run.tiles) {
      run.tile = 0;
      if (++run.mt == q.MT) {  // the next expert that has rows
        run.mt = 0;
        const int lane = threadIdx.x & 31;
        unsigned some = 0;
        int e = run.e + 1;
        for (; e < E; e += 32) {
          some = __ballot_sync(0xffffffffu, e + lane < E && tb.rows[e + lane] > 0);
          if (some) break;
        }
        run.e = min(E - 1, e + __ffs(some) - 1);
        run.tile0 = uniform(tb.tile0[run.e]);
        run.tiles = uniform(tb.tile0[run.e + 1]) - run.tile0;
      }
    }
  }
  s.s1 = static_cast<int>(min(static_cast<int64_t>(q.KS), s.s0 + (run.end - run.at)));
  run.at += s.s1 - s.s0;
  s.e = run.e;
  s.slot0 = uniform(tb.slot0[run.e]);
  s.tile0 = run.tile0;
  s.tile = run.tile;
  s.mt = run.mt;
  s.rows = min(q.tile_rows, uniform(tb.rows[run.e]) - s.tile * q.tile_rows);
  s.cols = round8(s.rows) * q.mult;
  return true;
}

__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// E4M3 rows: maps for boxes of 8, 16, .. rows.
struct RowMaps {
  CUtensorMap box[kRowMaps];
};

// kFp8: x in E4M3. kSteps: steps of a stage. kTogether: the units' order, see Order.
template <bool kFp8, int kSteps, bool kTogether>
__global__ void __launch_bounds__(kThreads)
    expert_linear_kernel(const Params q, const __grid_constant__ CUtensorMap map,
                         const __grid_constant__ RowMaps maps) {
  extern __shared__ uint8_t dynamic[];
  // The stages start on a 1024-byte boundary (the swizzle's period).
  uint8_t* smem = dynamic + (1024 - (smem_addr(dynamic) & 1023)) % 1024;
  __shared__ Shared sh;
  const ExpertLinearParams& p = q.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  const Tables tb(reinterpret_cast<int*>(smem + q.stages * q.stage_bytes + kScaleGroups * 4 * kScaleBytes), p.E);
  if (tid == 0) {
    for (int i = 0; i < q.stages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < kScaleGroups; ++i) {
      mbar_init(&sh.scale_full[i], 1);
      mbar_init(&sh.scale_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.acc_full[i], 1);
      mbar_init(&sh.acc_empty[i], 128);
    }
    fence_mbar_init();
  }
  if (warp == 3) tmem_alloc(&sh.tmem, kTmemCols);
  // The counts are older than the rows kernel, which released this one only
  // once everything before it had completed.
  tile_experts(q, sh.scan, tb);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = uniform(sh.tmem);
  const int64_t total = static_cast<int64_t>(uniform(tb.tile0[p.E])) * q.MT * q.KS;
  const int outs = p.glu ? p.M / 2 : p.M;
  // Every block that takes part has steps: the join counts on it.
  const int me = static_cast<int>(blockIdx.x);
  const int blocks = static_cast<int>(min(static_cast<int64_t>(gridDim.x), max(total / kMinStages, int64_t{1})));
  const Order order(static_cast<unsigned>(uniform(tb.tile0[p.E]) * q.MT), blocks);
  Run run{0, 0};
  if (me < blocks) run = Run{run_begin(total, blocks, me), run_begin(total, blocks, me + 1)};
  // A stage: weights, rows, the rows' scales. Behind the stages: the ring of
  // the weights' scales.
  constexpr unsigned x_at = kSteps * kTileBytes;
  const unsigned ws_at = q.stages * q.stage_bytes;
  // First output row of half h (64 rows) of a unit's weights.
  auto out_row = [&](int mt, int h) { return p.glu ? mt * 64 + h * outs : mt * kTileM + h * 64; };

  if (warp == 0) {
    // Loads. The rows' part waits for the rows kernel, the first stages'
    // weights do not. (The instructions of a stage are what this loop costs:
    // one load of weights, one of rows, addresses advanced, none computed anew.)
    auto load_w = [&](const Segment& g, int st, unsigned bytes, const Ring& r) {
      uint64_t* bar = &sh.full[r.stage];
      mbar_arrive_expect_tx(bar, bytes);
      tma_load_5d(smem + r.offset, &map, 0, out_row(g.mt, 0), 0, st * kSteps, g.e, bar);
    };
    auto steps_of = [&](int st) { return static_cast<unsigned>(min(kSteps, q.KB - st * kSteps)); };
    // Bytes of a step's rows: codes and scales.
    auto step_bytes = [&](const Segment& g) { return static_cast<unsigned>(g.cols) * kStep + q.scale_bytes; };
    const Run start = run;
    Segment g;
    Ring r;
    int ahead = 0;
    while (ahead < q.stages && next_segment<kTogether>(q, tb, order, run, g)) {
      for (int st = g.s0; st < g.s1 && ahead < q.stages; ++st, ++ahead) {
        if (elect_one()) load_w(g, st, kSteps * kTileTx + steps_of(st) * step_bytes(g), r);
        r.advance(q);
      }
    }
    grid_dependency_wait();
    run = start;
    r = Ring{};
    unsigned round = 0;  // passes over the ring
    unsigned empty = 0;  // asked a stage ahead
    bool ok = true;
    while (ok && next_segment<kTogether>(q, tb, order, run, g)) {
      const unsigned step = step_bytes(g), xcodes = step - q.scale_bytes;
      const unsigned image_step = kFp8 ? q.scale_bytes : step;
      const uint8_t* x =
          q.image + image_at(q, g.slot0, g.tile0, g.tile) + static_cast<int64_t>(g.s0) * kSteps * image_step;
      // E4M3 rows come straight from x, one box a step.
      const int row = static_cast<int>(uniform(first_row(p, g.e))) + g.tile * q.tile_rows;
      const CUtensorMap* box = &maps.box[g.cols / 8 - 1];
      for (int st = g.s0; st < g.s1; ++st) {
        const bool loaded = ahead > 0;
        if (loaded) {
          --ahead;
        } else if (round > 0 && !mbar_wait_asked(empty, &sh.empty[r.stage], r.parity ^ 1, p.status)) {
          ok = false;
          break;
        }
        const Ring at = r;
        r.advance(q);
        if (r.stage == 0) round = 1;
        empty = mbar_ask(&sh.empty[r.stage], r.parity ^ 1);
        const unsigned steps = steps_of(st);
        if (elect_one()) {
          uint64_t* bar = &sh.full[at.stage];
          if (!loaded) load_w(g, st, kSteps * kTileTx + steps * step, at);
          uint8_t* to = smem + at.offset;
          if (kFp8) {
            bulk_g2s(to + x_at + steps * xcodes, x, steps * q.scale_bytes, bar);
#pragma unroll
            for (int h = 0; h < kSteps; ++h)
              if (h < steps) tma_load_2d(to + x_at + h * xcodes, box, (st * kSteps + h) * kStep, row, bar);
          } else {
            bulk_g2s(to + x_at, x, steps * step, bar);
          }
        }
        __syncwarp();
        x += kSteps * image_step;
      }
    }
    if (!ok) {  // given up: loads in flight land before the block ends
      for (int i = 0; i < q.stages; ++i) mbar_drain(&sh.full[i], i < r.stage ? r.parity : r.parity ^ 1);
    }
  } else if (warp == 1) {
    // Products.
    Segment g;
    Ring r;
    int seg = 0, slot = 0;
    bool ok = true;
    const uint32_t base = smem_addr(smem);
    const uint64_t a0 = desc_rows128(base), b0 = desc_rows128(base + x_at);
    const uint64_t ws0 = desc_rows16(base + ws_at), xs0 = desc_rows16(base + x_at);
    int group = 0;             // place in the ring of the weights' scales
    unsigned group_parity = 0;
    // What the next stage needs is looked for before this one's products are
    // issued, so that the look costs no time between them.
    unsigned full = 0, scales = 0;
    while (ok && next_segment<kTogether>(q, tb, order, run, g)) {
      const int buf = seg & 1;
      if (seg >= 2 && !mbar_wait_warp(&sh.acc_empty[buf], (seg / 2 - 1) & 1, p.status)) break;
      tmem_fence_after();
      const uint32_t d = tmem + buf * kMaxCols;
      const uint32_t idesc = idesc_e2m1_e4m3(g.cols);
      const bool wide = kSteps == 1 && g.cols > 128;
      const unsigned x_step = static_cast<unsigned>(g.cols) * kStep >> 4, xs_step = q.scale_bytes >> 4;
      for (int st = g.s0; st < g.s1; ++st) {
        const int kb = st * kSteps;
        const bool group_start = st == g.s0 || (kb & 3) == 0;
        if ((group_start && !mbar_wait_asked(scales, &sh.scale_full[group], group_parity, p.status)) ||
            !mbar_wait_asked(full, &sh.full[r.stage], r.parity, p.status)) {
          mbar_drain(&sh.full[r.stage], r.parity);
          ok = false;
          break;
        }
        tmem_fence_after();
        const bool last = st + 1 == g.s1, group_end = (kb + kSteps & 3) == 0 || last;
        const unsigned at = r.offset >> 4;  // in the descriptors' units
        const int stage = r.stage, this_group = group;
        r.advance(q);
        if (group_end && ++group == kScaleGroups) {
          group = 0;
          group_parity ^= 1;
        }
        full = mbar_ask(&sh.full[r.stage], r.parity);
        scales = mbar_ask(&sh.scale_full[group], group_parity);
        const uint64_t ws = ws0 + (this_group * 4 + (kb & 3)) * (kScaleBytes / 16);
        const uint32_t sc = tmem + kTmemScales + slot * kMaxSteps * kScaleCols;
        const bool both = kSteps > 1 && kb + 1 < q.KB;
        const uint64_t xs = xs0 + at + (both ? 2 : 1) * x_step;
        // 32 inputs a product: 32 bytes on.
        auto step = [&](int h, bool accumulate) {
          const uint32_t c = sc + h * kScaleCols;
          tmem_copy_scales(c, ws + h * (kScaleBytes / 16));
          tmem_copy_scales(c + 4, xs + h * xs_step);
          if (wide) tmem_copy_scales(c + 8, xs + h * xs_step + kScaleBytes / 16);
          const uint64_t a = a0 + at + h * (kTileBytes / 16), b = b0 + at + h * x_step;
          mma_scaled(d, a, b, idesc, c, c + 4, accumulate);
#pragma unroll
          for (int i = 1; i < 4; ++i)
            mma_scaled(d, a + 2 * i, b + 2 * i, idesc_scale_byte(idesc, i), c, c + 4, true);
        };
        if (elect_one()) {
          step(0, st > g.s0);
          if (both) step(1, true);
          mma_commit(&sh.empty[stage]);
          if (group_end) mma_commit(&sh.scale_empty[this_group]);
          if (last) mma_commit(&sh.acc_full[buf]);
        }
        __syncwarp();
        slot ^= 1;
      }
      ++seg;
    }
  } else if (warp < 4) {
    // The weights' scales: four bytes a row and step, laid out for the copy to
    // tensor memory (row r: place r % 32, word r / 32). A lane reads 16 bytes
    // of a row, four steps, at once, and keeps kAhead such groups in flight,
    // across units: with four steps ahead the loads' latency alone set the
    // pace (128 tokens x 256 experts: 1513 us). Two warps take turns: one spent
    // 870 cycles a stage on it, as long as the products take.
    constexpr int kAhead = 3;
    const int64_t pitch = p.K / 32;
    const bool vec = q.KB % 4 == 0;
    uint32_t v[kAhead][4][4];  // [group][row][step]
    int lo[kAhead], hi[kAhead];
    Segment g;
    int next = 0;
    bool more = next_segment<kTogether>(q, tb, order, run, g);
    if (more) next = g.s0 * kSteps;
    auto advance = [&]() {  // to the next group
      if (!more) return;
      next = (next & ~3) + 4;
      if (next >= min(q.KB, g.s1 * kSteps)) {
        more = next_segment<kTogether>(q, tb, order, run, g);
        if (more) next = g.s0 * kSteps;
      }
    };
    // Steps [lo, hi) of one aligned group of four; lo == hi: none left.
    auto fetch = [&](uint32_t(&to)[4][4], int& from, int& upto) {
      from = upto = 0;
      if (!more) return;
      const int group = next & ~3;
      from = next - group;
      const int end = min(q.KB, g.s1 * kSteps);
      upto = min(4, end - group);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = out_row(g.mt, i / 2) + (i & 1) * 32 + lane;
        const uint8_t* src = p.w_scale + (static_cast<int64_t>(g.e) * p.M + m) * pitch + 4 * group;
        if (m >= p.M) {
#pragma unroll
          for (int j = 0; j < 4; ++j) to[i][j] = 0x7F7F7F7Fu;
        } else if (vec) {
          const uint4 w = __ldg(reinterpret_cast<const uint4*>(src));
          to[i][0] = w.x; to[i][1] = w.y; to[i][2] = w.z; to[i][3] = w.w;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            to[i][j] = j >= from && j < upto ? __ldg(reinterpret_cast<const uint32_t*>(src) + j) : 0;
        }
      }
      advance();
      advance();  // the other warp's
    };
    if (warp == 3) advance();
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(v[i], lo[i], hi[i]);
    int at = warp - 2;
    unsigned parity = 0, round = 0;
    bool ok = true;
    while (ok && hi[0] > lo[0]) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (!ok || lo[i] >= hi[i]) continue;
        if (round > 0) ok = mbar_wait_warp(&sh.scale_empty[at], parity ^ 1, p.status);
        if (!ok) continue;
        uint4* to = reinterpret_cast<uint4*>(smem + ws_at + at * 4 * kScaleBytes) + lane;
#pragma unroll
        for (int j = 0; j < 4; ++j) to[j * (kScaleBytes / 16)] = make_uint4(v[i][0][j], v[i][1][j], v[i][2][j], v[i][3][j]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.scale_full[at]);
        at += 2;
        if (at >= kScaleGroups) {
          at -= kScaleGroups;
          parity ^= 1;
          round = 1;
        }
        fetch(v[i], lo[i], hi[i]);
      }
    }
  } else if (warp >= 4) {
    // Results: thread m holds output row m of the unit's 128, a column a row of x.
    const int m = tid - 128;
    grid_dependency_wait();
    Segment g;
    int seg = 0;
    while (next_segment<kTogether>(q, tb, order, run, g)) {
      const int buf = seg & 1;
      if (!all_agree(mbar_wait(&sh.acc_full[buf], (seg / 2) & 1, p.status))) break;
      ++seg;
      tmem_fence_after();
      const uint32_t acc = tmem + buf * kMaxCols + (static_cast<uint32_t>(warp & 3) << 21);
      const int rows8 = round8(g.rows);
      const bool whole = g.s0 == 0 && g.s1 == q.KS;
      const int64_t row0 = first_row(p, g.e) + g.tile * q.tile_rows;
      const int o = p.glu ? g.mt * 64 + (m & 63) : g.mt * kTileM + m;
      auto slot = [&](int block, bool starts) {
        return q.partial + (static_cast<int64_t>(block) * 2 + (starts ? 1 : 0)) * q.tile_rows * kTileM;
      };
      // Eight finished sums of this thread's output row: to y.
      auto finish = [&](float* v, int c0) {
        if (p.glu) {
          float(*swap)[64] = sh.swap[(c0 >> 3) & 1];
          if (m >= 64) {
#pragma unroll
            for (int i = 0; i < 8; ++i) swap[i][m - 64] = v[i];
          }
          epilogue_sync();
          if (m >= 64) return;
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = v[i] / (1.0f + expf(-v[i])) * swap[i][m];
        }
        if (o >= outs) return;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c0 + i < g.rows)
            reinterpret_cast<__nv_bfloat16*>(p.y)[(row0 + c0 + i) * outs + o] = __float2bfloat16(v[i]);
      };
      float* mine = slot(me, g.s0 == 0);
      for (int c0 = 0; c0 < rows8; c0 += 8) {
        float v[8];
        tmem_load8(v, acc + c0);
        if (q.mult == 2) {
          float l[8];
          tmem_load8(l, acc + rows8 + c0);
          tmem_wait_load(v, l);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += l[i];
        } else {
          tmem_wait_load(v);
        }
        if (whole) {
          finish(v, c0);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) __stcg(mine + (c0 + i) * kTileM + m, v[i]);
        }
      }
      tmem_fence_before();
      mbar_arrive(&sh.acc_empty[buf]);
      if (whole) {
        if (p.glu) epilogue_sync();  // the swap buffers are free again
        continue;
      }
      // A shared unit: the last block to arrive adds the parts, in order.
      const int c_first = owner_of(total, blocks, g.unit * q.KS);
      const int c_last = owner_of(total, blocks, (g.unit + 1) * q.KS - 1);
      epilogue_sync();
      if (m == 0) {
        unsigned* counter = q.counters + c_first;
        __threadfence();  // the block's writes, which the barrier has ordered before it
        const bool last = atomicAdd(counter, 1u) == static_cast<unsigned>(c_last - c_first);
        if (last) *counter = 0u;
        __threadfence();
        sh.last = last;
      }
      epilogue_sync();
      if (sh.last) {
        for (int c0 = 0; c0 < rows8; c0 += 8) {
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = __ldcg(slot(c_first, true) + (c0 + i) * kTileM + m);
          for (int b = c_first + 1; b <= c_last; ++b) {
            const float* part = slot(b, false);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += __ldcg(part + (c0 + i) * kTileM + m);
          }
          finish(v, c0);
        }
      }
      epilogue_sync();  // sh.last and the swap buffers are free again
    }
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (warp == 3) {
    tmem_fence_after();
    tmem_free(tmem, kTmemCols);
  }
}

// Rows of a full tile: enough for nearly every expert's rows in one tile (the
// mean and four standard deviations of a random routing), so that weights are
// not read again, and no more, since a smaller tile leaves room for more
// stages of weights in flight.
int tile_rows_for(int E, int64_t max_rows, int mult) {
  const int64_t active = std::max<int64_t>(1, std::min<int64_t>(E, max_rows));
  const int64_t mean = (max_rows + active - 1) / active;
  int64_t sd4 = 4;
  while (sd4 * sd4 < 16 * mean) ++sd4;
  const int caps[] = {16, 32, 64, 128, kMaxCols};
  for (int cap : caps)
    if (cap / mult >= mean + sd4) return cap / mult;
  return kMaxCols / mult;
}

// Steps of a stage: two halve what a stage costs besides its bytes. With more
// than 64 columns they are large enough for it not to matter, and one step lets
// a tile have more than 128. In us with one / two steps, rows an expert (256
// experts, 7168 inputs, 2 x 2048 gated outputs): 4 BF16 733 / 667, 12 BF16 769 /
// 737, 4 E4M3 737 / 641, 24 E4M3 758 / 710; of more than 64 columns 24 BF16 843 /
// 864, 40 BF16 971 / 970, 48 E4M3 850 / 852, 72 E4M3 882 / 895.
int steps_for(int cols) { return cols <= 64 ? 2 : 1; }

// Whether the blocks work on an expert's output tiles side by side, so that its
// rows come from L2, or each on its own run of them. With more than 64 columns
// always: in runs all experts' rows are in use at once (235 MB at 128 rows of 256
// experts, and 12.2 GB came from HBM where 4.4 must). With fewer columns for long
// units alone, since each unit of this order has to be looked for. In us in runs /
// together (256 experts, 4096 outputs): 7168 inputs, about 128 E4M3 rows 1936 /
// 1070, 72 E4M3 1360 / 921, 40 BF16 1484 / 992, 384 inputs (1536 outputs), 128 E4M3
// 195 / 184; up to 64 columns, 4 BF16, 12 BF16, 4 E4M3 and 28 E4M3 rows: 7168 inputs
// 732, 889, 662, 891 / 661, 732, 641, 726; 5120 496, 564, 468, 563 / 483, 534, 466,
// 530; 4096 387, 433, 373, 434 / 395, 439, 383, 438; 1024 134, 141, 132, 168 / 170,
// 169, 163, 173.
bool work_together(int steps, int KB) { return steps == 1 || KB >= 40; }

struct Sizes {
  int tile_rows;
  size_t counters, partial, image, total;
};

Sizes sizes_of(int E, int64_t max_rows, int K, bool fp8) {
  const int mult = fp8 ? 1 : 2;
  Sizes z{};
  z.tile_rows = tile_rows_for(E, max_rows, mult);
  auto up = [](size_t v) { return (v + 1023) & ~static_cast<size_t>(1023); };
  const int64_t active = std::min<int64_t>(E, max_rows);
  const int64_t slots = max_rows + 7 * active;
  const int64_t tiles = max_rows / z.tile_rows + active;
  const int sb = z.tile_rows * mult > 128 ? 2 * kScaleBytes : kScaleBytes;
  z.counters = 0;
  z.partial = 1024;
  z.image = z.partial + up(sizeof(float) * kMaxBlocks * 2 * z.tile_rows * kTileM);
  z.total = z.image + up(static_cast<size_t>(tiles) * (K / kStep) * sb + (fp8 ? 0 : static_cast<size_t>(slots) * mult * K));
  return z;
}

}  // namespace

namespace {

template <bool kFp8, int kSteps, bool kTogether>
cudaError_t launch_products(const Params& q, const CUtensorMap& map, const RowMaps& maps, size_t smem, int dev, int sms,
                            cudaStream_t s) {
  const auto kernel = expert_linear_kernel<kFp8, kSteps, kTogether>;
  const void* fn = reinterpret_cast<const void*>(kernel);
  const cudaError_t err = ensure_dynamic_smem(fn, dev, smem);
  if (err != cudaSuccess) return err;
  // One block an SM.
  return launch_kernel(kernel, dim3(std::min(sms, kMaxBlocks)), dim3(kThreads), smem, s, /*dependent=*/true, q, map,
                       maps);
}

template <bool kFp8>
cudaError_t launch_steps(const Params& q, const CUtensorMap& map, const RowMaps& maps, size_t smem, int dev, int sms,
                         cudaStream_t s) {
  if (!work_together(q.steps, q.KB)) return launch_products<kFp8, 2, false>(q, map, maps, smem, dev, sms, s);
  return q.steps == 2 ? launch_products<kFp8, 2, true>(q, map, maps, smem, dev, sms, s)
                      : launch_products<kFp8, 1, true>(q, map, maps, smem, dev, sms, s);
}

}  // namespace

size_t expert_linear_ws_bytes(int E, int64_t max_rows, int K, bool fp8) { return sizes_of(E, max_rows, K, fp8).total; }

cudaError_t launch_expert_linear(const ExpertLinearParams& p, cudaStream_t s) {
  if (p.max_rows <= 0 || p.x_rows <= 0) return cudaSuccess;
  const bool fp8 = p.x_scale != nullptr;
  const Sizes z = sizes_of(p.E, p.max_rows, p.K, fp8);
  Params q{};
  q.p = p;
  q.mult = fp8 ? 1 : 2;
  q.tile_rows = z.tile_rows;
  q.cols_cap = z.tile_rows * q.mult;
  q.KB = p.K / kStep;
  q.steps = steps_for(q.cols_cap);
  q.KS = (q.KB + q.steps - 1) / q.steps;
  q.MT = p.glu ? (p.M / 2 + 63) / 64 : (p.M + kTileM - 1) / kTileM;
  q.counters = reinterpret_cast<unsigned*>(p.ws + z.counters);
  q.partial = reinterpret_cast<float*>(p.ws + z.partial);
  q.image = p.ws + z.image;
  q.scale_bytes = q.cols_cap > 128 ? 2 * kScaleBytes : kScaleBytes;
  q.stage_bytes = (q.steps * (kTileBytes + q.cols_cap * kStep + q.scale_bytes) + 1023) / 1024 * 1024;
  constexpr unsigned kRing = kScaleGroups * 4 * kScaleBytes;
  const unsigned tables = static_cast<unsigned>(table_bytes(p.E));
  const unsigned most = 227 * 1024 - sizeof(Shared) - 2048 - kRing - tables;
  q.stages = std::min<int>(kMaxStages, most / q.stage_bytes);
  const size_t smem = static_cast<size_t>(q.stages) * q.stage_bytes + kRing + tables + 1024;

  const EncodeTiled encode = encode_tiled();
  if (!encode) return cudaErrorNotSupported;
  CUtensorMap map;
  // Inputs in steps of 128, outputs in one part or two (gates, ups); a load
  // brings two steps of a unit's 128 outputs, each step's 128 x 128 together.
  const int parts = p.glu ? 2 : 1;
  const cuuint64_t row = static_cast<cuuint64_t>(p.K) / 2, rows = static_cast<cuuint64_t>(p.M) / parts;
  const cuuint64_t dims[5] = {kStep, rows, static_cast<cuuint64_t>(parts), static_cast<cuuint64_t>(q.KB),
                              static_cast<cuuint64_t>(p.E)};
  const cuuint64_t strides[4] = {row, rows * row, kStep / 2, p.M * row};
  const cuuint32_t box[5] = {kStep, static_cast<cuuint32_t>(kTileM / parts), static_cast<cuuint32_t>(parts),
                             static_cast<cuuint32_t>(q.steps), 1};
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  if (encode(&map, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 5, const_cast<uint8_t*>(p.w), dims, strides, box, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;

  RowMaps maps;
  if (fp8) {
    const cuuint64_t xd[2] = {static_cast<cuuint64_t>(p.K), static_cast<cuuint64_t>(p.x_rows)};
    const cuuint64_t xs[1] = {static_cast<cuuint64_t>(p.K)};
    for (int i = 0; i < q.cols_cap / 8; ++i) {
      const cuuint32_t b[2] = {kStep, static_cast<cuuint32_t>(8 * (i + 1))};
      if (encode(&maps.box[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p.x), xd, xs, b, ones,
                 CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    }
  }
  const int dev = current_device();
  const int sms = device_sms(dev);
  if (sms < 1) return cudaErrorInvalidDevice;
  // Items of the rows kernel: at most these.
  const int64_t groups = (p.max_rows + 7 * std::min<int64_t>(p.E, p.max_rows)) / 8;
  const int64_t items = groups * (fp8 ? 1 : (p.K + kRowSpan - 1) / kRowSpan);
  // The products' blocks need nearly all of an SM's shared memory: with an SM
  // set up for them from the start, they begin beside the rows kernel's
  // (8 experts, 2 tokens of 5376 inputs: 17.7 us, so 14.6).
  cudaError_t err = prefer_shared(reinterpret_cast<const void*>(expert_rows_kernel), dev);
  if (err != cudaSuccess) return err;
  err = launch_kernel(expert_rows_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(items, 6 * sms))), dim3(kThreads),
                      tables, s, /*dependent=*/true, q);
  if (err != cudaSuccess) return err;
  return fp8 ? launch_steps<true>(q, map, maps, smem, dev, sms, s)
             : launch_steps<false>(q, map, maps, smem, dev, sms, s);
}

}  // namespace ep
