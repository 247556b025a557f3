// Attention of a call's new tokens over the paged E4M3 cache on sm_103a.
//
// Mathematics: for a query row, s_j = scale <q, k_j> log2(e), running maximum m
// and sums: every chunk of keys rescales what was summed by 2^(m - m') and adds
// 2^(s_j - m') (and that times v_j). The blocks' scales never touch a code: a
// key block's scale multiplies its scores, and a value block's scale 2^ev moves
// into the exponent, p_j = 2^(s_j + ev - m) with m the maximum of s_j + ev, so
// that p stays in [0, 1] whatever the scales (taken times 2^15 in fp16, so that
// weights keep 11 bits down to 2^-29 of the largest); the normaliser sums p_j 2^(e0 - ev),
// e0 the first block's exponent, kept in [-26, 0]: its block may be one that no
// row sees, whose scale can be anything, and 2^(e0 - ev) stays in fp32's range for
// every ev in [-127, 100]. Codes and p enter the products as fp16 (an
// E4M3 value is exact in it, p keeps 11 bits); q as fp16 too, divided by a power
// of two that brings its row's largest magnitude to [1, 2).
//
// What bounds it: the cache, read once from HBM. With up to 16 query rows a
// key/value head (16 G FLOP a byte) the products are far from their limit, so
// they run as m16n8k16 on registers, the cache on the 16-row side and the query
// rows as columns: S^T = K Q^T, O^T = V^T P^T. Eight query heads then fill a
// product (with rows and columns exchanged half of it idled, and decode of 128
// x 8192 tokens took 400 us), and a converted code serves every column tile.
// S^T turns into the second product's operand by an 8 x 8 transposition between
// lanes. K and V fragments come from shared memory in 16-byte loads without
// conflicts: channels are assigned to a fragment's places so that a lane's are
// contiguous, and the tiled TMA load swizzles rows.
//
// Work: the rows of one (sequence, cache head), up to 8 kNT kRW of them, are a
// unit of chunks of 32 tokens. The blocks take equal runs of consecutive
// places over all units, whatever the sequences' lengths; a unit has a place
// for each chunk and unit_cost more in front, so that a block with many short
// sequences is not the last to finish (24 sequences of 4 to 30011 tokens, 4
// drafted each: 75 us without). In a block, one warp
// loads (pages, scales, descriptors of what comes), four compute: kRW of them
// hold 8 kNT rows each, 4 / kRW groups take turns with the chunks and are joined
// at the end of a unit. A unit of few chunks is one group's alone, while the others
// take the next ones: its cost is the latency of its steps (queries 1500 cycles, a
// chunk 1650, joining 1000, results 1100), not their work. 8 heads of 64 tokens x 200
// sequences 24.0 us together, 17.7 alone; 16 heads of 150 tokens (5 chunks) 49.6 and
// 42.0; 8 heads of 200 tokens (7 chunks) 33.5 and 36.0. A unit that several blocks share is joined by the last
// of them to finish, in the order of its chunks, so results do not depend on
// which one that was.
//
// Measured (head size 128): 128 sequences x 8192 tokens x 8 cache heads, 8 rows
// each, 331 us, 6.5 TB/s (copy rate 6.69); one sequence of 131072 tokens, 4 x 16
// rows, 37 us: 4 before its first chunk, 23 for the chunks, 10 for joining 76
// parts. 32 rows: the products' warps, not HBM, set the pace (20000 tokens x 24
// x 4 heads: 153 us, 88 with the computing left out). Tried there without gain:
// four column tiles a warp, two chunks at once, smaller tiles on more warps.
#include <cuda.h>

#include "common.cuh"
#include "kernels.cuh"
#include "tensor.cuh"

namespace ep {

namespace {

constexpr int kChunk = 32;       // tokens
constexpr int kWarps = 4;        // computing warps
constexpr int kThreads = 256;    // the computing warps, a loading one, and three that complete its warpgroup
constexpr int kComputeRegs = 216, kLoadRegs = 40;  // of the 2 x 128 a thread pair is launched with (400 us -> 331
                                                   // for 128 x 8192 tokens: nothing spills)
constexpr int kMaxBlocks = 320;  // blocks a workspace has room for
constexpr int kFan = 8;          // parts of a shared unit that one block joins at once
// Chunks that a unit costs besides its own: queries, joining, results. Chunks of
// 64 rows cost more themselves: in us with 6 / 4 / 3 / 2, 60 sequences of up to 3000
// tokens, 8 drafted, 8 heads of 64: 42.2 / 40.5 / 38.6 / 40.2, 30 of 300: 23.1 / 23.2 /
// 24.0 / 24.0, 20 of up to 20000, 5 drafted: 57.0 / 56.5 / 56.6 / 55.6. With 32 rows and
// fewer it depends on the lengths alone (32 rows, 6 / 4: 49.4 / 47.3, 24.3 / 24.7,
// 37.3 / 38.4; 9 / 6 / 4 / 2 with heads of 128: 60 sequences of up to 3000 tokens, 8
// heads of 8 rows 21.1 / 20.2 / 20.1 / 21.5, of 16 rows 30.7 / 31.1 / 32.3 / 36.1, 24 of up to
// 30000, 4 heads of 8 rows 25.8 / 27.5 / 28.8 / 27.9, of 16 rows 34.1 / 36.0 / 37.5 / 38.6).
constexpr int unit_cost(int row_warps) { return row_warps < 4 ? 6 : 4; }
constexpr int kUnits = 8;        // units whose descriptors are in flight
constexpr int kSolo = 5;         // most chunks of a unit that one group of warps takes alone
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kTop = 15.0f;    // the largest weight enters the products as 2^15

template <int kD, int kNT>
struct Shape {
  static constexpr int kStages = kD == 128 ? 8 : 12;
  static constexpr int kBlocksPerSM = 2;
  static constexpr int kSide = kChunk * kD;  // bytes of keys (or values) of a chunk
  static constexpr int kStage = 2 * kSide;
};

// What the loading warp says of a chunk.
struct ChunkHeader {
  float ks[2];    // scales of its (up to two) pages' keys
  int ev[2];      // exponents of their values' scales
  unsigned valid; // tokens that exist
};

// A run of chunks of one unit.
struct Unit {
  int b, h, rt;      // sequence, cache head, row tile
  int t0, n;         // its tokens in the call
  int tok0, head0;   // token and head (of the cache head's) of the tile's first row
  int len;           // sequence length
  int first;         // first token of chunk 0
  int c0, c1, total; // chunks [c0, c1) of `total`
  int it;            // the block's running number of chunk c0
  int first_block, last_block;  // the blocks that share its chunks
};

// A sequence's units.
struct Sequence {
  int t0, n, len;
  int first;   // token that chunk 0 starts with
  int chunks;  // of each of its units
  int tiles;   // row tiles
  bool ok;
  __device__ __forceinline__ int places(int cost) const { return chunks + cost; }  // of a unit
  __device__ __forceinline__ int64_t all(int heads, int cost) const { return static_cast<int64_t>(places(cost)) * tiles * heads; }
};

template <int kD, int kNT, int kRW>
struct Shared {
  static constexpr int kTW = kWarps / kRW;
  static constexpr int kStages = Shape<kD, kNT>::kStages;
  uint64_t full[kStages], empty[kStages];
  uint64_t unit_full[kUnits], unit_empty[kUnits];
  ChunkHeader header[kStages];
  Unit unit[kUnits];
  int more[kUnits];  // 0: no further unit
  long long sums[kThreads / 32];
  int find_b;
  long long find_at;
  Sequence find;
  int bad;
  int last;
  static constexpr int kJoin = kTW / 2 * kRW;  // warps that hand their sums over at once
  float4 join_o[kJoin ? kJoin : 1][kJoin ? kD / 16 * kNT : 1][32];
  float4 join_ml[kJoin ? kJoin : 1][2 * kNT][32];  // a row's references and sum
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two E4M3 codes (the low or high half of w) as two fp16.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(w)));
  return r;
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(w >> 16)));
  return r;
}

__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The 8 x 8 transposition of fp16 pairs between lanes: lane (g, j) gives
// elements (g, 2j), (g, 2j + 1) and gets (2j, g), (2j + 1, g).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

__device__ __forceinline__ void compute_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// ---- the division of the work -----------------------------------------------------
// Sequence b of the call: what its units look like.
__device__ __forceinline__ Sequence sequence_at(const KVAttentionParams& p, int b, int tile_rows) {
  const KVParams& c = p.c;
  Sequence s;
  s.ok = true;
  if (c.cu) {
    s.t0 = __ldg(c.cu + b);
    s.n = __ldg(c.cu + b + 1) - s.t0;
    if (s.t0 < 0 || s.n < 0 || s.n > c.N - s.t0) {
      s.ok = false;
      s.n = 0;
    }
  } else {
    s.t0 = b;
    s.n = 1;
  }
  s.len = __ldg(c.lens + b);
  const int64_t cap = static_cast<int64_t>(c.MP) * c.P;
  const int stop = s.len < cap ? max(s.len, 0) : static_cast<int>(cap);
  const int64_t low = p.window > 0 ? static_cast<int64_t>(s.len) - s.n - p.window + 1 : 0;
  s.first = low > 0 ? static_cast<int>(low) & ~(kChunk - 1) : 0;
  s.chunks = stop > s.first ? (stop - s.first - 1) / kChunk + 1 : 1;
  s.tiles = static_cast<int>((static_cast<int64_t>(s.n) * p.G + tile_rows - 1) / tile_rows);
  return s;
}

__device__ __forceinline__ int64_t run_begin(int64_t total, int blocks, int c) { return total * c / blocks; }
__device__ __forceinline__ int owner_of(int64_t total, int blocks, int64_t i) {
  return static_cast<int>(((i + 1) * blocks + total - 1) / total) - 1;
}

// ---- the kernel ---------------------------------------------------------------------
template <int kD, int kNT, int kRW>
__global__ void __launch_bounds__(kThreads, Shape<kD, kNT>::kBlocksPerSM)
    kv_attention_kernel(const KVAttentionParams p, float* partial, unsigned* counters,
                        const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  constexpr int kTW = kWarps / kRW;
  constexpr int kUnitCost = unit_cost(kRW);
  using S = Shape<kD, kNT>;
  constexpr int kRows = 8 * kNT * kRW;
  constexpr int kStages = S::kStages;
  constexpr int kTiles = kD / 16;       // value channel tiles
  constexpr int kSteps = kD / 16;       // score product steps
  constexpr int kRowBytes = kD;         // of a token of a head
  constexpr int kPart = kRows * (kD + 4);  // floats of a partial result
  extern __shared__ uint8_t dynamic[];
  uint8_t* smem = dynamic + (1024 - (smem_addr(dynamic) & 1023)) % 1024;
  using Sh = Shared<kD, kNT, kRW>;
  Sh& sh = *reinterpret_cast<Sh*>(smem + kStages * S::kStage);
  const KVParams& c = p.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh.full[i], 2);  // the loads, the header
      mbar_init(&sh.empty[i], kRW);
    }
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(&sh.unit_full[i], 1);
      mbar_init(&sh.unit_empty[i], kWarps);
    }
    fence_mbar_init();
    sh.bad = 0;
  }
  grid_dependency_wait();
  __syncthreads();

  // Chunks of all units, by sequences; each thread sums a stretch of them.
  const int per = (c.B + kThreads - 1) / kThreads;
  const int b0 = min(c.B, tid * per), b1 = min(c.B, b0 + per);
  long long mine = 0;
  const int64_t cap = static_cast<int64_t>(c.MP) * c.P;
  for (int b = b0; b < b1; ++b) {
    const Sequence s = sequence_at(p, b, kRows);
    mine += s.all(c.KH, kUnitCost);
    if (!s.ok) sh.bad = 1;
    if (blockIdx.x == 0) {
      if (!s.ok) flag(c.status, EP_ST_BAD_INDEX);
      if (s.len > cap) flag(c.status, EP_ST_CAPACITY);
    }
  }
  if (c.cu && tid == 0 && (__ldg(c.cu) != 0 || __ldg(c.cu + c.B) != c.N)) sh.bad = 1;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) sh.sums[warp] = incl;
  __syncthreads();
  long long total = 0, before = incl - mine;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sh.sums[w];
    total += sh.sums[w];
  }
  total = uniform(total);
  if (total == 0 && !sh.bad) return;
  const int blocks = static_cast<int>(min(static_cast<long long>(gridDim.x), total));
  const int64_t begin = blockIdx.x < blocks ? run_begin(total, blocks, blockIdx.x) : 0;
  const int64_t end = blockIdx.x < blocks ? run_begin(total, blocks, blockIdx.x + 1) : 0;
  if (begin < end && begin >= before && begin < before + mine) {
    long long at = before;
    for (int b = b0; b < b1; ++b) {
      const Sequence s = sequence_at(p, b, kRows);
      if (begin < at + s.all(c.KH, kUnitCost)) {
        sh.find_b = b;
        sh.find_at = at;
        sh.find = s;
        break;
      }
      at += s.all(c.KH, kUnitCost);
    }
  }
  if (sh.bad) {
    // cu_tokens out of order or not covering every token: the rest are empty rows.
    for (int t = blockIdx.x; t < c.N; t += gridDim.x) {
      bool covered = false;
      for (int b = tid; b < c.B; b += kThreads) {
        const Sequence s = sequence_at(p, b, kRows);
        covered |= s.ok && t >= s.t0 && t - s.t0 < s.n;
      }
      if (__syncthreads_or(covered)) continue;
      for (int i = tid; i < p.QH * kD; i += kThreads) p.out[static_cast<int64_t>(t) * p.QH * kD + i] = 0;
      if (p.lse)
        for (int i = tid; i < p.QH; i += kThreads) p.lse[static_cast<int64_t>(t) * p.QH + i] = -INFINITY;
    }
  }
  __syncthreads();
  if (begin >= end) return;

  if (warp >= kWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
    if (warp > kWarps) return;
    // ---- loads ----
    int b = uniform(sh.find_b);
    int64_t seq_at = uniform(sh.find_at);
    Sequence s = sh.find;
    int64_t at = begin;
    int it = 0, un = 0, stage = 0;
    unsigned parity = 0;
    bool ok = true;
    while (ok && at < end) {
      // The unit that holds place `at`.
      while (at >= seq_at + s.all(c.KH, kUnitCost)) {
        seq_at += s.all(c.KH, kUnitCost);
        s = sequence_at(p, ++b, kRows);
      }
      const int u = static_cast<int>((at - seq_at) / s.places(kUnitCost));
      const int64_t unit_at = seq_at + static_cast<int64_t>(u) * s.places(kUnitCost);
      const int from = max(0, static_cast<int>(at - unit_at) - kUnitCost);
      at = min(end, unit_at + s.places(kUnitCost));
      const int upto = static_cast<int>(at - unit_at) - kUnitCost;
      if (upto <= from) continue;  // only places in front of its chunks
      Unit d;
      d.b = b;
      d.rt = u % s.tiles;  // row tiles of a head follow one another: its cache comes from L2 after the first
      d.h = u / s.tiles;
      d.tok0 = d.rt * kRows / p.G;
      d.head0 = d.rt * kRows - d.tok0 * p.G;
      d.t0 = s.t0;
      d.n = s.n;
      d.len = s.len;
      d.first = s.first;
      d.total = s.chunks;
      d.first_block = owner_of(total, blocks, unit_at + kUnitCost);
      d.last_block = owner_of(total, blocks, unit_at + s.places(kUnitCost) - 1);
      d.c0 = from;
      d.c1 = upto;
      d.it = it;
      const int slot = un % kUnits;
      if (un >= kUnits && !mbar_wait_warp(&sh.unit_empty[slot], (un / kUnits - 1) & 1, c.status)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        sh.unit[slot] = d;
        sh.more[slot] = 1;
        mbar_arrive(&sh.unit_full[slot]);
      }
      ++un;
      // Pages in batches of 32: a lane holds one page's number and scales; the
      // next batch's are in flight. (A chunk of two 16-token pages starts at an
      // even one, so both are in a batch.)
      const int stop = static_cast<int>(min(static_cast<int64_t>(max(s.len, 0)), cap));
      const int pages = stop > 0 ? ((stop - 1) >> c.log2P) + 1 : 0;  // pages the sequence has
      const int32_t* table = c.table + static_cast<int64_t>(b) * c.MP;
      auto page_no = [&](int j) { return j < pages ? __ldg(table + j) : -1; };
      auto scale_of = [&](const float* from, int page) {
        return page >= 0 && page < c.pages ? __ldg(from + static_cast<int64_t>(page) * c.KH + d.h) : 1.0f;
      };
      int batch = (d.first + d.c0 * kChunk) >> c.log2P;
      int id = page_no(batch + lane), id1 = page_no(batch + 32 + lane);
      float ks = scale_of(c.k_scale, id), vs = scale_of(c.v_scale, id);
      float ks1 = scale_of(c.k_scale, id1), vs1 = scale_of(c.v_scale, id1);
      int id2 = page_no(batch + 64 + lane);
      for (int k = d.c0; k < d.c1; ++k, ++it) {
        const int tok = d.first + k * kChunk;
        const int j = tok >> c.log2P;
        if (j >= batch + 32) {
          batch += 32;
          id = id1;
          ks = ks1;
          vs = vs1;
          id1 = id2;
          ks1 = scale_of(c.k_scale, id1);
          vs1 = scale_of(c.v_scale, id1);
          id2 = page_no(batch + 64 + lane);
        }
        if (it >= kStages && !mbar_wait_warp(&sh.empty[stage], parity ^ 1, c.status)) {
          ok = false;
          break;
        }
        uint64_t* bar = &sh.full[stage];
        uint8_t* to = smem + stage * S::kStage;
        // Tokens that exist from `from` on, `most` at the most, in a page of
        // the cache; a page outside it is reported and read as masked.
        auto exist = [&](int page, int from, int most) {
          const int have = min(most, stop - from);
          if (have <= 0) return 0u;
          if (page < 0 || page >= c.pages) {
            if (lane == 0) flag(c.status, EP_ST_BAD_INDEX);
            return 0u;
          }
          return have >= 32 ? ~0u : (1u << have) - 1u;
        };
        auto exponent = [](float v) { return static_cast<int>(__float_as_uint(v) >> 23 & 255) - 127; };
        const int src = j - batch;
        const int page = __shfl_sync(0xffffffffu, id, src);
        ChunkHeader hd;
        // Loads first: they need the page's number alone. Scales of a page that
        // nobody may read stay out of the arithmetic.
        if (c.P > 16) {
          hd.valid = exist(page, tok, kChunk);
          if (elect_one()) {
            mbar_arrive_expect_tx(bar, hd.valid ? S::kStage : 0);
            if (hd.valid) {
              const int block = page * c.KH + d.h, row = tok & (c.P - 1);
              tma_load_3d(to, &map_k, 0, row, block, bar);
              tma_load_3d(to + S::kSide, &map_v, 0, row, block, bar);
            }
          }
          const float pk = __shfl_sync(0xffffffffu, ks, src), pv = __shfl_sync(0xffffffffu, vs, src);
          hd.ks[0] = hd.ks[1] = hd.valid ? pk : 1.0f;
          hd.ev[0] = hd.ev[1] = hd.valid ? exponent(pv) : 0;
        } else {
          const int src1 = src + 1 & 31;
          const int page1 = __shfl_sync(0xffffffffu, id, src1);
          const unsigned v0 = exist(page, tok, 16), v1 = exist(page1, tok + 16, 16);
          hd.valid = v0 | v1 << 16;
          if (elect_one()) {
            mbar_arrive_expect_tx(bar, (v0 ? S::kSide : 0) + (v1 ? S::kSide : 0));
            if (v0) {
              tma_load_3d(to, &map_k, 0, 0, page * c.KH + d.h, bar);
              tma_load_3d(to + S::kSide, &map_v, 0, 0, page * c.KH + d.h, bar);
            }
            if (v1) {
              tma_load_3d(to + 16 * kRowBytes, &map_k, 0, 0, page1 * c.KH + d.h, bar);
              tma_load_3d(to + S::kSide + 16 * kRowBytes, &map_v, 0, 0, page1 * c.KH + d.h, bar);
            }
          }
          const float pk = __shfl_sync(0xffffffffu, ks, src), pv = __shfl_sync(0xffffffffu, vs, src);
          const float pk1 = __shfl_sync(0xffffffffu, ks, src1), pv1 = __shfl_sync(0xffffffffu, vs, src1);
          hd.ks[0] = v0 ? pk : 1.0f;
          hd.ks[1] = v1 ? pk1 : 1.0f;
          hd.ev[0] = v0 ? exponent(pv) : v1 ? exponent(pv1) : 0;
          hd.ev[1] = v1 ? exponent(pv1) : hd.ev[0];
        }
        if (elect_one()) {
          sh.header[stage] = hd;
          mbar_arrive(bar);
        }
        __syncwarp();
        if (++stage == kStages) {
          stage = 0;
          parity ^= 1;
        }
      }
    }
    const int slot = un % kUnits;
    if (un < kUnits || mbar_wait_warp(&sh.unit_empty[slot], (un / kUnits - 1) & 1, c.status)) {
      if (lane == 0) {
        sh.more[slot] = 0;
        mbar_arrive(&sh.unit_full[slot]);
      }
    }
    // Every load has landed before the block ends, also if those who wait for it
    // (or this warp) have given up.
    for (int i = 0; i < kStages; ++i)
      if (i < stage || it >= kStages) mbar_drain(&sh.full[i], i < stage ? parity : parity ^ 1);
    return;
  }

  // ---- computing warps ----
  // (128 registers a thread at launch; the loading side's share goes to these.)
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kComputeRegs));
  const int rw = warp % kRW, tw = warp / kRW;
  const int g = lane >> 2, j = lane & 3;
  const uint32_t sbase = smem_addr(smem);
  for (int un = 0;; ++un) {
    const int slot = un % kUnits;
    // (The warps leave together: each votes once in every unit that has barriers,
    // and once more with a no, at the end of the units or when its wait for one
    // has run out, which is the answer to the others' next vote. So none of them
    // stands at a barrier that another will not reach.)
    if (!mbar_wait_warp(&sh.unit_full[slot], (un / kUnits) & 1, c.status)) {
      all_agree(false);
      break;
    }
    if (!sh.more[slot]) {
      all_agree(false);
      break;
    }
    const Unit d = sh.unit[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.unit_empty[slot]);
    // Few chunks: one group's work, while the others take the next units. (A warp
    // has left a unit before it waits for another: that one's descriptor may
    // only come once the other groups have consumed units in between, and they
    // might stand at this unit's barriers.)
    const bool whole = d.c0 == 0 && d.c1 == d.total;
    const bool solo = kTW > 1 && whole && d.total <= kSolo;
    if (solo && un % kTW != tw) continue;

    // This warp's rows. As columns of the score products: lane (g, j) holds
    // row 8 t + g of column tile t, channels of quad j; of the results it gets
    // rows 8 t + 2j and 8 t + 2j + 1.
    const int rows = min(kRows, d.n * p.G - d.rt * kRows);  // of the tile
    const int row_base = rw * 8 * kNT;
    // Row -> token and head: a division of at most 4096 + 64 by G, by its reciprocal,
    // which is exact in this range (with divisions 79 sequences of up to 31 tokens,
    // 48 rows each, took 16.0 us, now 13.8).
    auto over_g = [&](int x) { return static_cast<int>(__umulhi(2u * static_cast<unsigned>(x), p.g_inverse)); };
    auto token_of = [&](int row) { return d.tok0 + over_g(d.head0 + row); };
    auto position = [&](int row) { return row < rows ? d.len - d.n + token_of(row) : -1; };  // -1: no such row
    uint32_t qb[kNT][kSteps][2];
    float qf[kNT][2];   // score factors: scale log2(e) times the power of two taken from q
    int pos[kNT][2];
#pragma unroll
    for (int t = 0; t < kNT; ++t) {
      const int row = row_base + 8 * t + g;
      const int x0 = d.head0 + row, y0 = over_g(x0);
      const int i = d.tok0 + y0, head = d.h * p.G + x0 - y0 * p.G;
      const bool live = row < rows;
      constexpr int kMineCh = kD / 4;  // channels of a lane
      uint4 raw[kMineCh / 8];
      const uint4* src = reinterpret_cast<const uint4*>(p.q + static_cast<int64_t>(d.t0 + i) * p.q_stride +
                                                        static_cast<int64_t>(head) * kD + j * kMineCh);
      uint32_t top = 0;
#pragma unroll
      for (int x = 0; x < kMineCh / 8; ++x) {
        raw[x] = live ? __ldg(src + x) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {raw[x].x, raw[x].y, raw[x].z, raw[x].w};
#pragma unroll
        for (int y = 0; y < 4; ++y) top = max(top, max(w[y] & 0x7FFFu, w[y] >> 16 & 0x7FFFu));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // Exponent of the largest magnitude (a BF16's bits order like its value).
      const int e = min(253, max(1, static_cast<int>(top >> 7)));
      const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
      const float f = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(e) << 23);
#pragma unroll
      for (int x = 0; x < kMineCh / 8; ++x) {
        const uint32_t w[4] = {raw[x].x, raw[x].y, raw[x].z, raw[x].w};
#pragma unroll
        for (int y = 0; y < 4; ++y)
          qb[t][2 * x + y / 2][y & 1] = pack_f16x2(bf16_lo(w[y]) * down, bf16_hi(w[y]) * down);
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        qf[t][r] = __shfl_sync(0xffffffffu, f, 8 * j + 4 * r);
        pos[t][r] = position(row_base + 8 * t + 2 * j + r);
      }
    }
    // Positions of the warp's first and last row: what every row sees of a chunk.
    const int first_pos = d.len - d.n + token_of(row_base);
    const int last_row = min(rows, row_base + 8 * kNT) - 1;
    const int last_pos = last_row >= row_base ? d.len - d.n + token_of(last_row) : -1;

    float o[kTiles][kNT][4];
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int t = 0; t < kNT; ++t) o[i][t][0] = o[i][t][1] = o[i][t][2] = o[i][t][3] = 0.0f;
    float m[kNT][2], l[kNT][2];
#pragma unroll
    for (int t = 0; t < kNT; ++t) {
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.0f;
    }
    int e0 = 0;
    bool started = false;

    for (int it = d.it + (solo ? 0 : tw); it < d.it + d.c1 - d.c0; it += solo ? 1 : kTW) {  // the groups take turns
      const int stage = it % kStages;
      // (A wait that gives up leaves wrong results and says so; the warp stays
      // for the barriers below, and the loading warp ends the work.)
      if (!mbar_wait_warp(&sh.full[stage], (it / kStages) & 1, c.status)) {
        mbar_drain(&sh.full[stage], (it / kStages) & 1);
        break;
      }
      const ChunkHeader hd = sh.header[stage];
      const uint32_t kbuf = sbase + stage * S::kStage, vbuf = kbuf + S::kSide;
      const int tok = d.first + (d.c0 + it - d.it) * kChunk;
      if (!started) {
        e0 = min(0, max(-26, hd.ev[0]));
        started = true;
      }
      // Scores: tokens 16 h + g (and + 8) of the chunk, rows 8 t + 2j, + 1.
      float s[2][kNT][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < kNT; ++t) s[h][t][0] = s[h][t][1] = s[h][t][2] = s[h][t][3] = 0.0f;
#pragma unroll
      for (int k0 = 0; k0 < kSteps; k0 += 4) {  // four steps: 16 bytes of a token's keys a lane
        uint32_t w[2][2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t row = kbuf + (h * 16 + 8 * x + g) * kRowBytes;
            const uint4 a = lds128(row + (kD == 128 ? ((2 * j + k0 / 4) ^ g) << 4 : (j ^ (g >> 1)) << 4));
            w[h][x][0] = a.x; w[h][x][1] = a.y; w[h][x][2] = a.z; w[h][x][3] = a.w;
          }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a[4] = {codes_lo(w[h][0][k]), codes_lo(w[h][1][k]), codes_hi(w[h][0][k]), codes_hi(w[h][1][k])};
#pragma unroll
            for (int t = 0; t < kNT; ++t) mma16816(s[h][t], a, qb[t][k0 + k][0], qb[t][k0 + k][1]);
          }
        }
      }
      // In units of log2, the value block's exponent added.
      const bool masked = hd.valid != ~0u || tok + kChunk - 1 > first_pos ||
                          (p.window > 0 && tok <= last_pos - p.window) || last_pos < first_pos;
      const float el[2] = {static_cast<float>(hd.ev[0] - e0), static_cast<float>(hd.ev[1] - e0)};
      auto sees = [&](int at, int ps) {
        return (hd.valid >> at & 1) && tok + at <= ps && !(p.window > 0 && tok + at <= ps - p.window);
      };
      float alpha[kNT][2], shift[kNT][2];
      bool moved = false;
#pragma unroll
      for (int t = 0; t < kNT; ++t)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float mx = -INFINITY;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float& v = s[h][t][2 * x + r];
              v = fmaf(v, hd.ks[h] * qf[t][r], el[h]);
              if (masked && !sees(h * 16 + g + 8 * x, pos[t][r])) v = -INFINITY;
              mx = fmaxf(mx, v);
            }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float top = fmaxf(m[t][r], mx);
          const float ref = top == -INFINITY ? 0.0f : top;
          alpha[t][r] = ex2(m[t][r] - ref);
          moved |= top > m[t][r];
          m[t][r] = top;
          l[t][r] *= alpha[t][r];
          shift[t][r] = ref - kTop;
        }
      const float w0 = ex2(-el[0]), w1 = ex2(-el[1]);
      uint32_t pb[2][kNT][2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < kNT; ++t) {
#pragma unroll
          for (int x = 0; x < 4; ++x) s[h][t][x] = ex2(s[h][t][x] - shift[t][x & 1]);
          l[t][0] = fmaf(s[h][t][0] + s[h][t][2], h ? w1 : w0, l[t][0]);
          l[t][1] = fmaf(s[h][t][1] + s[h][t][3], h ? w1 : w0, l[t][1]);
          pb[h][t][0] = transpose8(pack_f16x2(s[h][t][0], s[h][t][1]));
          pb[h][t][1] = transpose8(pack_f16x2(s[h][t][2], s[h][t][3]));
        }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
          for (int t = 0; t < kNT; ++t)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[i][t][x] *= alpha[t][x & 1];
      }
      // Values: lane (g, j) takes tokens 2j, 2j + 1, 2j + 8, 2j + 9 of each 16.
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        constexpr int kWords = kD / 32;  // of four channels, a lane's share of a token
        uint32_t v[4][kWords];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int t = q * 16 + (x >> 1) * 8 + 2 * j + (x & 1);
          if (kD == 128) {
            const uint4 w = lds128(vbuf + t * kRowBytes + ((g ^ (t & 7)) << 4));
            v[x][0] = w.x; v[x][1] = w.y; v[x][kWords - 2] = w.z; v[x][kWords - 1] = w.w;
          } else {
            const uint2 w = lds64(vbuf + t * kRowBytes + (((g >> 1) ^ (t >> 1 & 3)) << 4) + (g & 1) * 8);
            v[x][0] = w.x; v[x][1] = w.y;
          }
        }
        if (masked) {
          // A code that some rows must not see can be a NaN, and 0 times NaN is
          // one: NaN codes leave the product, and the rows that see them get
          // theirs from a count of them.
          uint32_t nan[4][kWords], some = 0;
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
              nan[x][w] = ((v[x][w] & 0x7F7F7F7Fu) + 0x01010101u & 0x80808080u) >> 7;
              some |= nan[x][w];
              v[x][w] &= ~(nan[x][w] * 0xFFu);
            }
          if (__any_sync(0xffffffffu, some != 0)) {
#pragma unroll
            for (int t = 0; t < kNT; ++t) {
              // 1 where row 8 t + g sees the token.
              const int ps = position(row_base + 8 * t + g);
              uint32_t in[2];
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int at = q * 16 + 8 * x + 2 * j;
                in[x] = (sees(at, ps) ? 0x3C00u : 0u) | (sees(at + 1, ps) ? 0x3C000000u : 0u);
              }
#pragma unroll
              for (int i = 0; i < kTiles; ++i) {
                float cnt[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                auto one = [&](int x, int ch) { return nan[x][ch >> 2] >> (8 * (ch & 3)) & 1u ? 0x3C00u : 0u; };
                const uint32_t a[4] = {one(0, 2 * i) | one(1, 2 * i) << 16, one(0, 2 * i + 1) | one(1, 2 * i + 1) << 16,
                                       one(2, 2 * i) | one(3, 2 * i) << 16, one(2, 2 * i + 1) | one(3, 2 * i + 1) << 16};
                mma16816(cnt, a, in[0], in[1]);
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  if (cnt[x] > 0.0f) o[i][t][x] = __int_as_float(0x7FC00000);
              }
            }
          }
        }
#pragma unroll
        for (int w = 0; w < kWords; ++w)
#pragma unroll
          for (int y = 0; y < 2; ++y) {  // channels 4 w + 2 y and the next
            const uint32_t a = __byte_perm(v[0][w], v[1][w], y ? 0x7362 : 0x5140);
            const uint32_t b = __byte_perm(v[2][w], v[3][w], y ? 0x7362 : 0x5140);
            const uint32_t f[4] = {codes_lo(a), codes_hi(a), codes_lo(b), codes_hi(b)};
#pragma unroll
            for (int t = 0; t < kNT; ++t) mma16816(o[2 * w + y][t], f, pb[q][t][0], pb[q][t][1]);
          }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[stage]);
    }

    // ---- end of the run of chunks: join the groups ----
    float md[kNT][2];
#pragma unroll
    for (int t = 0; t < kNT; ++t)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        l[t][r] += __shfl_xor_sync(0xffffffffu, l[t][r], 4);
        l[t][r] += __shfl_xor_sync(0xffffffffu, l[t][r], 8);
        l[t][r] += __shfl_xor_sync(0xffffffffu, l[t][r], 16);
        // The numerator is 2^m o, the values' exponents in m; the normaliser 2^md l.
        md[t][r] = m[t][r] - kTop;
        m[t][r] = md[t][r] + static_cast<float>(e0);
      }
    // (Whole units of one group's have no barriers. From here on nobody leaves
    // this unit, and what was handed over in the one before has been read.)
    if (!solo && (kTW > 1 || !whole) && !all_agree(true)) break;
    // Half of the groups hands over to the other half, until one is left.
#pragma unroll
    for (int half = kTW / 2; half >= 1; half /= 2) {
      if (solo) break;
      if (half < kTW / 2) compute_sync();  // what was handed over before has been read
      if (tw >= half && tw < 2 * half) {
        const int w = (tw - half) * kRW + rw;
#pragma unroll
        for (int t = 0; t < kNT; ++t) {
#pragma unroll
          for (int i = 0; i < kTiles; ++i)
            sh.join_o[w][i * kNT + t][lane] = make_float4(o[i][t][0], o[i][t][1], o[i][t][2], o[i][t][3]);
#pragma unroll
          for (int r = 0; r < 2; ++r)
            sh.join_ml[w][2 * t + r][lane] = make_float4(m[t][r], md[t][r], l[t][r], 0.0f);
        }
      }
      compute_sync();
      if (tw < half) {
        const int w = tw * kRW + rw;
#pragma unroll
        for (int t = 0; t < kNT; ++t) {
          float f[2], fo[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float4 x = sh.join_ml[w][2 * t + r][lane];
            const float top = fmaxf(m[t][r], x.x), topd = fmaxf(md[t][r], x.y);
            const float rt = top == -INFINITY ? 0.0f : top, rd = topd == -INFINITY ? 0.0f : topd;
            f[r] = ex2(m[t][r] - rt);
            fo[r] = ex2(x.x - rt);
            l[t][r] = fmaf(ex2(x.y - rd), x.z, l[t][r] * ex2(md[t][r] - rd));
            m[t][r] = top;
            md[t][r] = topd;
          }
#pragma unroll
          for (int i = 0; i < kTiles; ++i) {
            const float4 y = sh.join_o[w][i * kNT + t][lane];
            o[i][t][0] = fmaf(fo[0], y.x, o[i][t][0] * f[0]);
            o[i][t][1] = fmaf(fo[1], y.y, o[i][t][1] * f[1]);
            o[i][t][2] = fmaf(fo[0], y.z, o[i][t][2] * f[0]);
            o[i][t][3] = fmaf(fo[1], y.w, o[i][t][3] * f[1]);
          }
        }
      }
    }
    auto out_of = [&](int row) {  // (token, head) of a row of the tile
      const int x = d.head0 + row, y = over_g(x);
      return static_cast<int64_t>(d.t0 + d.tok0 + y) * p.QH + d.h * p.G + x - y * p.G;
    };
    // Lane (g, j) holds rows 8 t + 2j and + 1, channels [g kD / 8, (g + 1) kD / 8).
    if (whole) {
      if (solo || tw == 0) {
#pragma unroll
        for (int t = 0; t < kNT; ++t)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int row = row_base + 8 * t + 2 * j + r;
            if (row >= rows) continue;
            const float f = l[t][r] > 0.0f ? ex2(m[t][r] - md[t][r]) / l[t][r] : (l[t][r] == 0.0f ? 0.0f : l[t][r]);
            const int64_t at = out_of(row);
            uint4* to = reinterpret_cast<uint4*>(p.out + at * kD + g * (kD / 8));
#pragma unroll
            for (int i = 0; i < kTiles; i += 4)
              to[i / 4] = make_uint4(pack_bf16x2(o[i][t][r] * f, o[i][t][2 + r] * f),
                                     pack_bf16x2(o[i + 1][t][r] * f, o[i + 1][t][2 + r] * f),
                                     pack_bf16x2(o[i + 2][t][r] * f, o[i + 2][t][2 + r] * f),
                                     pack_bf16x2(o[i + 3][t][r] * f, o[i + 3][t][2 + r] * f));
            if (p.lse && g == 0) p.lse[at] = (md[t][r] + log2f(l[t][r])) * kLn2;
          }
      }
      continue;
    }
    // ---- a unit that other blocks share ----
    // Parts are joined in groups of kFan blocks, then the groups, each time by
    // the last to arrive and in order: with one level a long sequence's last
    // block read 76 parts one after the other (82 us for 131072 tokens x 4
    // cache heads).
    const int c_first = d.first_block, c_last = d.last_block;
    auto part = [&](int block, bool starts) {
      return partial + (static_cast<int64_t>(block) * 2 + (starts ? 1 : 0)) * kPart;
    };
    // One block's arrival on a counter that expects `n`: whether it is the last.
    auto arrive = [&](unsigned* counter, int n) {
      compute_sync();
      if (tid == 0) {
        __threadfence();  // the block's writes, which the barrier has ordered before it
        const bool last = atomicAdd(counter, 1u) == static_cast<unsigned>(n - 1);
        if (last) *counter = 0u;
        __threadfence();
        sh.last = last;
      }
      compute_sync();
      return sh.last != 0;
    };
    // Join parts first, first + step, ... below stop (the unit's first one lies in its block's
    // second slot): into part `to`, or as the result when `to` is null.
    auto join = [&](int first, int step, int stop, float* to) {
      const int n = (stop - first + step - 1) / step;
      constexpr int kVec = kD / 4;            // float4 of a row
      constexpr int kAtOnce = 2;              // rows a thread works on side by side
      constexpr int kStride = 128 / kVec;     // rows of the block's threads
      static_assert(kVec == 32 || kVec == 16, "a row's threads are a warp or half of one");
      const int ch = tid % kVec;
      for (int r0 = tid / kVec; r0 < rows; r0 += kAtOnce * kStride) {
        float top[kAtOnce], topd[kAtOnce], sum[kAtOnce];
        float4 acc[kAtOnce];
#pragma unroll
        for (int a = 0; a < kAtOnce; ++a) {
          top[a] = topd[a] = -INFINITY;
          sum[a] = 0.0f;
          acc[a] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        for (int k0 = 0; k0 < n; k0 += kFan) {
          float4 y[kAtOnce][kFan], v[kAtOnce][kFan];
#pragma unroll
          for (int k = 0; k < kFan; ++k)
#pragma unroll
            for (int a = 0; a < kAtOnce; ++a) {
              const int b = first + (k0 + k) * step, row = r0 + a * kStride;
              y[a][k] = make_float4(-INFINITY, -INFINITY, 0.0f, 0.0f);
              v[a][k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              if (b < stop && row < rows) {
                const float* from = part(b, b == c_first);
                y[a][k] = __ldcg(reinterpret_cast<const float4*>(from + kRows * kD) + row);
                v[a][k] = __ldcg(reinterpret_cast<const float4*>(from + row * kD) + ch);
              }
            }
#pragma unroll
          for (int a = 0; a < kAtOnce; ++a) {
            float t = top[a], td = topd[a];
#pragma unroll
            for (int k = 0; k < kFan; ++k) {
              t = fmaxf(t, y[a][k].x);
              td = fmaxf(td, y[a][k].y);
            }
            const float rt = t == -INFINITY ? 0.0f : t, rd = td == -INFINITY ? 0.0f : td;
            const float keep = ex2(top[a] - rt);
            sum[a] *= ex2(topd[a] - rd);
            acc[a] = make_float4(acc[a].x * keep, acc[a].y * keep, acc[a].z * keep, acc[a].w * keep);
#pragma unroll
            for (int k = 0; k < kFan; ++k) {
              const float f = ex2(y[a][k].x - rt);
              sum[a] = fmaf(ex2(y[a][k].y - rd), y[a][k].z, sum[a]);
              acc[a].x = fmaf(f, v[a][k].x, acc[a].x);
              acc[a].y = fmaf(f, v[a][k].y, acc[a].y);
              acc[a].z = fmaf(f, v[a][k].z, acc[a].z);
              acc[a].w = fmaf(f, v[a][k].w, acc[a].w);
            }
            top[a] = t;
            topd[a] = td;
          }
        }
        // (A group's sum goes where its first part lay: a thread overwrites what
        // it alone has read, but for a row's references, which all threads of
        // the row, a warp or half of one, have read before.)
        __syncwarp(kVec == 32 ? 0xFFFFFFFFu : 0xFFFFu << (lane & 16));
#pragma unroll
        for (int a = 0; a < kAtOnce; ++a) {
          const int row = r0 + a * kStride;
          if (row >= rows) break;
          if (to) {
            __stcg(reinterpret_cast<float4*>(to + row * kD) + ch, acc[a]);
            if (ch == 0)
              __stcg(reinterpret_cast<float4*>(to + kRows * kD) + row, make_float4(top[a], topd[a], sum[a], 0.0f));
          } else {
            const float f = sum[a] > 0.0f ? ex2(top[a] - topd[a]) / sum[a] : (sum[a] == 0.0f ? 0.0f : sum[a]);
            const int64_t at = out_of(row);
            reinterpret_cast<uint2*>(p.out + at * kD)[ch] =
                make_uint2(pack_bf16x2(acc[a].x * f, acc[a].y * f), pack_bf16x2(acc[a].z * f, acc[a].w * f));
            if (p.lse && ch == 0) p.lse[at] = (topd[a] + log2f(sum[a])) * kLn2;
          }
        }
      }
    };
    if (tw == 0) {
      float* to = part(blockIdx.x, d.c0 == 0);
#pragma unroll
      for (int t = 0; t < kNT; ++t)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = row_base + 8 * t + 2 * j + r;
          if (row >= rows) continue;
          float4* v = reinterpret_cast<float4*>(to + row * kD + g * (kD / 8));
#pragma unroll
          for (int i = 0; i < kTiles; i += 2)
            __stcg(v + i / 2, make_float4(o[i][t][r], o[i][t][2 + r], o[i + 1][t][r], o[i + 1][t][2 + r]));
          if (g == 0)
            __stcg(reinterpret_cast<float4*>(to + kRows * kD) + row, make_float4(m[t][r], md[t][r], l[t][r], 0.0f));
        }
    }
    const int parts = c_last - c_first + 1;
    if (parts <= 2 * kFan) {
      if (arrive(counters + c_first, parts)) join(c_first, 1, c_last + 1, nullptr);
      continue;
    }
    // The group's first block's part takes the group's sum.
    const int group = (static_cast<int>(blockIdx.x) - c_first) / kFan;
    const int g0 = c_first + group * kFan, g1 = min(g0 + kFan, c_last + 1);
    // (A block can start a group of one unit and another unit: two counters each.)
    if (!arrive(counters + kMaxBlocks + 2 * g0 + (g0 == c_first ? 1 : 0), g1 - g0)) continue;
    join(g0, 1, g1, part(g0, g0 == c_first));
    if (arrive(counters + c_first, (parts + kFan - 1) / kFan)) join(c_first, kFan, c_last + 1, nullptr);
  }
}

bool cache_map(CUtensorMap* map, uint8_t* base, const KVParams& c) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.D), static_cast<cuuint64_t>(c.P),
                              static_cast<cuuint64_t>(c.pages) * c.KH};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(c.D), static_cast<cuuint64_t>(c.P) * c.D};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(c.D), static_cast<cuuint32_t>(c.P < kChunk ? c.P : kChunk), 1};
  const cuuint32_t ones[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                c.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kD, int kNT, int kRW>
cudaError_t launch(const KVAttentionParams& p, cudaStream_t s) {
  CUtensorMap mk, mv;
  if (!cache_map(&mk, p.c.k, p.c) || !cache_map(&mv, p.c.v, p.c)) return cudaErrorInvalidValue;
  using S = Shape<kD, kNT>;
  const size_t smem = S::kStages * S::kStage + sizeof(Shared<kD, kNT, kRW>) + 1024;
  const auto fn = kv_attention_kernel<kD, kNT, kRW>;
  const int dev = current_device();
  const cudaError_t err = ensure_dynamic_smem(reinterpret_cast<const void*>(fn), dev, smem);
  if (err != cudaSuccess) return err;
  const int sms = device_sms(dev);
  if (sms < 1) return cudaErrorInvalidDevice;
  const int grid = S::kBlocksPerSM * sms < kMaxBlocks ? S::kBlocksPerSM * sms : kMaxBlocks;
  return launch_kernel(fn, dim3(grid), dim3(kThreads), smem, s, /*dependent=*/true, p,
                       reinterpret_cast<float*>(p.ws + 4096), reinterpret_cast<unsigned*>(p.ws), mk, mv);
}

// Row tiles of 8, 16, 32 or 64: the smallest that holds a sequence's rows of one
// cache head, so that its cache is read once.
int tile_rows_for(int64_t rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

template <int kD>
cudaError_t launch_rows(const KVAttentionParams& p, int rows, cudaStream_t s) {
  return rows == 8    ? launch<kD, 1, 1>(p, s)
         : rows == 16 ? launch<kD, 2, 1>(p, s)
         : rows == 32 ? launch<kD, 2, 2>(p, s)
                      : launch<kD, 2, 4>(p, s);
}

}  // namespace

size_t kv_attention_ws_bytes(int N, int QH, int KH, int D) {
  const int rows = tile_rows_for(static_cast<int64_t>(N) * (QH / KH));
  return 4096 + sizeof(float) * kMaxBlocks * 2 * rows * static_cast<size_t>(D + 4);
}

cudaError_t launch_kv_attention(const KVAttentionParams& in, cudaStream_t s) {
  KVAttentionParams p = in;
  if (p.c.N <= 0) return cudaSuccess;
  p.g_inverse = ((1u << 31) + p.G - 1) / p.G;
  const int64_t each = (static_cast<int64_t>(p.c.N) + p.c.B - 1) / p.c.B;  // new tokens a sequence
  const int rows = tile_rows_for(each * p.G);
  return p.c.D == 64 ? launch_rows<64>(p, rows, s) : launch_rows<128>(p, rows, s);
}

}  // namespace ep
