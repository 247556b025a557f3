// Attention of a call's new tokens over the paged E4M3 cache on sm_103a.
//
// Mathematics: for a query row, s_j = scale <q, k_j> log2(e), running maximum m
// and sums: every chunk of keys rescales what was summed by 2^(m - m') and adds
// 2^(s_j - m') (and that times v_j). The blocks' scales never touch a code: a
// key block's scale multiplies its scores, and a value block's scale 2^ev moves
// into the exponent, p_j = 2^(s_j + ev - m) with m the maximum of s_j + ev, so
// that p stays in [0, 1] whatever the scales (taken times 2^15 in fp16, so that
// weights keep 11 bits down to 2^-29 of the largest); the normaliser sums p_j 2^(e0 - ev),
// e0 the first block's exponent. Codes and p enter the products as fp16 (an
// E4M3 value is exact in it, p keeps 11 bits); q as fp16 too, divided by a power
// of two that brings its row's largest magnitude to [1, 2).
//
// What bounds it: the cache, read once from HBM. With up to 16 query rows a
// key/value head (16 G FLOP a byte) the products are far from their limit, so
// they run as m16n8k16 on registers: a score tile's accumulators are the next
// product's operand as they are, and K and V fragments come from shared memory
// in 16-byte loads without conflicts: channels are assigned to a fragment's
// places so that a lane's are contiguous, and the tiled TMA load swizzles rows.
//
// Work: the rows of one (sequence, cache head), up to 16 kRW of them, are a
// unit of chunks of 32 tokens. The blocks take equal runs of consecutive
// chunks over all units, whatever the sequences' lengths. In a block, one warp
// loads (pages, scales, descriptors of what comes), four compute: kRW of them
// hold 16 rows each, 4 / kRW groups take turns with the chunks and are joined
// at the end of a unit. A unit that several blocks share is joined by the last
// of them to finish, in the order of its chunks, so results do not depend on
// which one that was.
#include <cuda.h>

#include "common.cuh"
#include "kernels.cuh"
#include "tensor.cuh"

namespace ep {

namespace {

constexpr int kChunk = 32;       // tokens
constexpr int kWarps = 4;        // computing warps
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kMaxBlocks = 320;  // blocks a workspace has room for
constexpr int kFan = 8;          // parts of a shared unit that one block joins at once
constexpr int kUnits = 4;        // units whose descriptors are in flight
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kTop = 15.0f;    // the largest weight enters the products as 2^15

template <int kD>
struct Shape {
  static constexpr int kStages = kD == 128 ? 8 : 12;
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
  int len;           // sequence length
  int first;         // first token of chunk 0
  int c0, c1, total; // chunks [c0, c1) of `total`
  int it;            // the block's running number of chunk c0
  int64_t at;        // position of chunk 0 among all chunks
};

template <int kD, int kRW>
struct Shared {
  static constexpr int kTW = kWarps / kRW;
  uint64_t full[Shape<kD>::kStages], empty[Shape<kD>::kStages];
  uint64_t unit_full[kUnits], unit_empty[kUnits];
  ChunkHeader header[Shape<kD>::kStages];
  Unit unit[kUnits];
  int more[kUnits];  // 0: no further unit
  long long sums[kThreads / 32];
  int find_b;
  long long find_at;
  int bad;
  int last;
  float4 join_o[kTW > 1 ? (kTW - 1) * kRW : 1][kD / 8][kTW > 1 ? 32 : 1];
  float4 join_ml[kTW > 1 ? (kTW - 1) * kRW : 1][2][kTW > 1 ? 32 : 1];  // m, denominator's reference, l of rows g, g + 8
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
struct Sequence {
  int t0, n, len;
  int first;   // token that chunk 0 starts with
  int chunks;  // of each of its units
  int tiles;   // row tiles
  bool ok;
};

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
  s.chunks = max(1, (stop - s.first + kChunk - 1) / kChunk);
  s.tiles = static_cast<int>((static_cast<int64_t>(s.n) * p.G + tile_rows - 1) / tile_rows);
  return s;
}

__device__ __forceinline__ int64_t run_begin(int64_t total, int blocks, int c) { return total * c / blocks; }
__device__ __forceinline__ int owner_of(int64_t total, int blocks, int64_t i) {
  return static_cast<int>(((i + 1) * blocks + total - 1) / total) - 1;
}

// ---- the kernel ---------------------------------------------------------------------
template <int kD, int kRW>
__global__ void __launch_bounds__(kThreads, 2)
    kv_attention_kernel(const KVAttentionParams p, float* partial, unsigned* counters,
                        const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  constexpr int kTW = kWarps / kRW;
  constexpr int kRows = 16 * kRW;
  constexpr int kStages = Shape<kD>::kStages;
  constexpr int kTiles = kD / 8;        // value channel tiles
  constexpr int kSteps = kD / 16;       // score product steps
  constexpr int kRowBytes = kD;         // of a token of a head
  constexpr int kPart = kRows * (kD + 4);  // floats of a partial result
  extern __shared__ uint8_t dynamic[];
  uint8_t* smem = dynamic + (1024 - (smem_addr(dynamic) & 1023)) % 1024;
  Shared<kD, kRW>& sh = *reinterpret_cast<Shared<kD, kRW>*>(smem + kStages * Shape<kD>::kStage);
  const KVParams& c = p.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh.full[i], 1);
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
    mine += static_cast<long long>(s.chunks) * s.tiles * c.KH;
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
      const long long n = static_cast<long long>(s.chunks) * s.tiles * c.KH;
      if (begin < at + n) {
        sh.find_b = b;
        sh.find_at = at;
        break;
      }
      at += n;
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

  if (warp == kWarps) {
    // ---- loads ----
    int b = uniform(sh.find_b);
    int64_t seq_at = uniform(sh.find_at);
    Sequence s = sequence_at(p, b, kRows);
    int64_t at = begin;
    int it = 0, un = 0, stage = 0;
    unsigned parity = 0;
    bool ok = true;
    while (ok && at < end) {
      // The unit that holds position `at`.
      while (at >= seq_at + static_cast<int64_t>(s.chunks) * s.tiles * c.KH) {
        seq_at += static_cast<int64_t>(s.chunks) * s.tiles * c.KH;
        s = sequence_at(p, ++b, kRows);
      }
      const int u = static_cast<int>((at - seq_at) / s.chunks);
      Unit d;
      d.b = b;
      d.rt = u % s.tiles;  // row tiles of a head follow one another: its cache comes from L2 after the first
      d.h = u / s.tiles;
      d.t0 = s.t0;
      d.n = s.n;
      d.len = s.len;
      d.first = s.first;
      d.total = s.chunks;
      d.at = seq_at + static_cast<int64_t>(u) * s.chunks;
      d.c0 = static_cast<int>(at - d.at);
      d.c1 = static_cast<int>(min(static_cast<int64_t>(s.chunks), d.c0 + (end - at)));
      d.it = it;
      at += d.c1 - d.c0;
      const int slot = un % kUnits;
      if (un >= kUnits && !mbar_wait_warp(&sh.unit_empty[slot], (un / kUnits - 1) & 1, c.status)) break;
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
        uint8_t* to = smem + stage * Shape<kD>::kStage;
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
        const float pk = __shfl_sync(0xffffffffu, ks, src), pv = __shfl_sync(0xffffffffu, vs, src);
        ChunkHeader hd;
        if (c.P > 16) {
          hd.valid = exist(page, tok, kChunk);
          // (Scales of a page that nobody may read stay out of the arithmetic.)
          hd.ks[0] = hd.ks[1] = hd.valid ? pk : 1.0f;
          hd.ev[0] = hd.ev[1] = hd.valid ? exponent(pv) : 0;
          if (elect_one()) {
            sh.header[stage] = hd;
            mbar_arrive_expect_tx(bar, hd.valid ? Shape<kD>::kStage : 0);
            if (hd.valid) {
              const int block = page * c.KH + d.h, row = tok & (c.P - 1);
              tma_load_3d(to, &map_k, 0, row, block, bar);
              tma_load_3d(to + Shape<kD>::kSide, &map_v, 0, row, block, bar);
            }
          }
        } else {
          const int page1 = __shfl_sync(0xffffffffu, id, src + 1 & 31);
          const float pk1 = __shfl_sync(0xffffffffu, ks, src + 1 & 31), pv1 = __shfl_sync(0xffffffffu, vs, src + 1 & 31);
          const unsigned v0 = exist(page, tok, 16), v1 = exist(page1, tok + 16, 16);
          hd.valid = v0 | v1 << 16;
          hd.ks[0] = v0 ? pk : 1.0f;
          hd.ks[1] = v1 ? pk1 : 1.0f;
          hd.ev[0] = v0 ? exponent(pv) : v1 ? exponent(pv1) : 0;
          hd.ev[1] = v1 ? exponent(pv1) : hd.ev[0];
          if (elect_one()) {
            sh.header[stage] = hd;
            mbar_arrive_expect_tx(bar, (v0 ? Shape<kD>::kSide : 0) + (v1 ? Shape<kD>::kSide : 0));
            if (v0) {
              tma_load_3d(to, &map_k, 0, 0, page * c.KH + d.h, bar);
              tma_load_3d(to + Shape<kD>::kSide, &map_v, 0, 0, page * c.KH + d.h, bar);
            }
            if (v1) {
              tma_load_3d(to + 16 * kRowBytes, &map_k, 0, 0, page1 * c.KH + d.h, bar);
              tma_load_3d(to + Shape<kD>::kSide + 16 * kRowBytes, &map_v, 0, 0, page1 * c.KH + d.h, bar);
            }
          }
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
    return;
  }

  // ---- computing warps ----
  const int rw = warp % kRW, tw = warp / kRW;
  const int g = lane >> 2, j = lane & 3;
  const uint32_t sbase = smem_addr(smem);
  for (int un = 0;; ++un) {
    const int slot = un % kUnits;
    if (!mbar_wait_warp(&sh.unit_full[slot], (un / kUnits) & 1, c.status)) break;
    if (!sh.more[slot]) break;
    const Unit d = sh.unit[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.unit_empty[slot]);

    // This warp's 16 rows: lane (g, j) holds rows g and g + 8, channels of quad j.
    const int rows = min(kRows, d.n * p.G - d.rt * kRows);  // of the tile
    uint32_t qa[kSteps][4];
    float qf[2];   // score factor: scale log2(e) times the power of two taken from q
    int pos[2];    // position of the row's token; -1: no such row
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = rw * 16 + g + 8 * r;
      const int gr = d.rt * kRows + row;
      const int i = gr / p.G, head = d.h * p.G + gr % p.G;
      const bool live = row < rows;
      pos[r] = live ? d.len - d.n + i : -1;
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
      qf[r] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(e) << 23);
#pragma unroll
      for (int x = 0; x < kMineCh / 8; ++x) {
        const uint32_t w[4] = {raw[x].x, raw[x].y, raw[x].z, raw[x].w};
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          qa[2 * x + y][r] = pack_f16x2(bf16_lo(w[2 * y]) * down, bf16_hi(w[2 * y]) * down);
          qa[2 * x + y][2 + r] = pack_f16x2(bf16_lo(w[2 * y + 1]) * down, bf16_hi(w[2 * y + 1]) * down);
        }
      }
    }
    // Positions of the tile's first and last row: what every row sees of a chunk.
    const int first_pos = d.len - d.n + (d.rt * kRows + rw * 16) / p.G;
    const int last_row = min(rows, rw * 16 + 16) - 1;
    const int last_pos = last_row >= rw * 16 ? d.len - d.n + (d.rt * kRows + last_row) / p.G : -1;

    float o[kTiles][4];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    int e0 = 0;
    bool started = false;

    int it = d.it + (tw - d.it % kTW + kTW) % kTW;  // the first of its chunks that is this group's
    for (; it < d.it + d.c1 - d.c0; it += kTW) {
      const int stage = it % kStages;
      // (A wait that gives up leaves wrong results and says so; the warp stays
      // for the barriers below, and the loading warp ends the work.)
      if (!mbar_wait_warp(&sh.full[stage], (it / kStages) & 1, c.status)) break;
      const ChunkHeader hd = sh.header[stage];
      const uint32_t kbuf = sbase + stage * Shape<kD>::kStage, vbuf = kbuf + Shape<kD>::kSide;
      const int tok = d.first + (d.c0 + it - d.it) * kChunk;
      if (!started) {
        e0 = hd.ev[0];
        started = true;
      }
      // Scores.
      float s[4][4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.0f;
        const uint32_t row = kbuf + (t * 8 + g) * kRowBytes;
        if (kD == 128) {
          const uint4 x = lds128(row + (((2 * j) ^ g) << 4)), y = lds128(row + (((2 * j + 1) ^ g) << 4));
          const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
          for (int k = 0; k < kSteps; ++k) mma16816(s[t], qa[k], codes_lo(w[k]), codes_hi(w[k]));
        } else {
          const uint4 x = lds128(row + ((j ^ (g >> 1)) << 4));
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int k = 0; k < kSteps; ++k) mma16816(s[t], qa[k], codes_lo(w[k]), codes_hi(w[k]));
        }
      }
      // In units of log2, the value block's exponent added.
      const bool masked = hd.valid != ~0u || tok + kChunk - 1 > first_pos ||
                          (p.window > 0 && tok <= last_pos - p.window) || last_pos < first_pos;
      const float el[2] = {static_cast<float>(hd.ev[0] - e0), static_cast<float>(hd.ev[1] - e0)};
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[t][i] = fmaf(s[t][i], hd.ks[t >> 1] * qf[i >> 1], el[t >> 1]);
          if (masked) {
            const int at = t * 8 + 2 * j + (i & 1), ps = pos[i >> 1];
            if (!(hd.valid >> at & 1) || tok + at > ps || (p.window > 0 && tok + at <= ps - p.window))
              s[t][i] = -INFINITY;
          }
          mx[i >> 1] = fmaxf(mx[i >> 1], s[t][i]);
        }
      }
      float alpha[2], ref[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
        const float top = fmaxf(m[r], mx[r]);
        ref[r] = top == -INFINITY ? 0.0f : top;
        alpha[r] = ex2(m[r] - ref[r]);
        m[r] = top;
        l[r] *= alpha[r];
      }
      const float el0 = ex2(-el[0]), el1 = ex2(-el[1]);
      const float shift[2] = {ref[0] - kTop, ref[1] - kTop};
      uint32_t pa[2][4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[t][i] = ex2(s[t][i] - shift[i >> 1]);
        const float w = t < 2 ? el0 : el1;
        l[0] = fmaf(s[t][0] + s[t][1], w, l[0]);
        l[1] = fmaf(s[t][2] + s[t][3], w, l[1]);
        pa[t >> 1][(t & 1) * 2] = pack_f16x2(s[t][0], s[t][1]);
        pa[t >> 1][(t & 1) * 2 + 1] = pack_f16x2(s[t][2], s[t][3]);
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          o[i][0] *= alpha[0];
          o[i][1] *= alpha[0];
          o[i][2] *= alpha[1];
          o[i][3] *= alpha[1];
        }
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
            uint32_t sees[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              // Rows g (x even) and g + 8, tokens of score tile 2q + x / 2: 1 where the row sees the token.
              uint32_t word = 0;
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const int at = q * 16 + (x >> 1) * 8 + 2 * j + y, ps = pos[x & 1];
                const bool in = (hd.valid >> at & 1) && tok + at <= ps && !(p.window > 0 && tok + at <= ps - p.window);
                if (in) word |= 0x3C00u << (16 * y);
              }
              sees[x] = word;
            }
#pragma unroll
            for (int w = 0; w < kWords; ++w)
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                float cnt[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                auto one = [&](int x) { return nan[x][w] >> (8 * y) & 1u ? 0x3C00u : 0u; };
                mma16816(cnt, sees, one(0) | one(1) << 16, one(2) | one(3) << 16);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (cnt[i] > 0.0f) o[4 * w + y][i] = __int_as_float(0x7FC00000);
              }
          }
        }
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          const uint32_t a0 = __byte_perm(v[0][w], v[1][w], 0x5140), a1 = __byte_perm(v[0][w], v[1][w], 0x7362);
          const uint32_t c0 = __byte_perm(v[2][w], v[3][w], 0x5140), c1 = __byte_perm(v[2][w], v[3][w], 0x7362);
          mma16816(o[4 * w], pa[q], codes_lo(a0), codes_lo(c0));
          mma16816(o[4 * w + 1], pa[q], codes_hi(a0), codes_hi(c0));
          mma16816(o[4 * w + 2], pa[q], codes_lo(a1), codes_lo(c1));
          mma16816(o[4 * w + 3], pa[q], codes_hi(a1), codes_hi(c1));
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[stage]);
    }

    // ---- end of the run of chunks: join the groups ----
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
    // m is the numerator's reference with the values' exponents: 2^(m + e0) o;
    // the normaliser is 2^m l.
    float md[2] = {m[0] - kTop, m[1] - kTop};
    m[0] = md[0] + static_cast<float>(e0);
    m[1] = md[1] + static_cast<float>(e0);
    if (kTW > 1) {
      compute_sync();  // the first group is done with the last unit's
      if (tw > 0) {
        const int w = (tw - 1) * kRW + rw;
#pragma unroll
        for (int i = 0; i < kTiles; ++i) sh.join_o[w][i][lane] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
        sh.join_ml[w][0][lane] = make_float4(m[0], md[0], l[0], 0.0f);
        sh.join_ml[w][1][lane] = make_float4(m[1], md[1], l[1], 0.0f);
      }
      compute_sync();
      if (tw == 0) {
        float4 x[kTW][2];  // each group's references and sum
        x[0][0] = make_float4(m[0], md[0], l[0], 0.0f);
        x[0][1] = make_float4(m[1], md[1], l[1], 0.0f);
#pragma unroll
        for (int w = 1; w < kTW; ++w) {
          x[w][0] = sh.join_ml[(w - 1) * kRW + rw][0][lane];
          x[w][1] = sh.join_ml[(w - 1) * kRW + rw][1][lane];
        }
        float f[kTW][2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float top = -INFINITY, topd = -INFINITY;
#pragma unroll
          for (int w = 0; w < kTW; ++w) {
            top = fmaxf(top, x[w][r].x);
            topd = fmaxf(topd, x[w][r].y);
          }
          const float rt = top == -INFINITY ? 0.0f : top, rd = topd == -INFINITY ? 0.0f : topd;
          float sum = 0.0f;
#pragma unroll
          for (int w = 0; w < kTW; ++w) {
            f[w][r] = ex2(x[w][r].x - rt);
            sum = fmaf(ex2(x[w][r].y - rd), x[w][r].z, sum);
          }
          m[r] = top;
          md[r] = topd;
          l[r] = sum;
        }
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          o[i][0] *= f[0][0];
          o[i][1] *= f[0][0];
          o[i][2] *= f[0][1];
          o[i][3] *= f[0][1];
#pragma unroll
          for (int w = 1; w < kTW; ++w) {
            const float4 y = sh.join_o[(w - 1) * kRW + rw][i][lane];
            o[i][0] = fmaf(f[w][0], y.x, o[i][0]);
            o[i][1] = fmaf(f[w][0], y.y, o[i][1]);
            o[i][2] = fmaf(f[w][1], y.z, o[i][2]);
            o[i][3] = fmaf(f[w][1], y.w, o[i][3]);
          }
        }
      }
    }
    auto out_of = [&](int row) {  // (token, head) of a row of the tile
      const int gr = d.rt * kRows + row;
      return static_cast<int64_t>(d.t0 + gr / p.G) * p.QH + d.h * p.G + gr % p.G;
    };
    const bool whole = d.c0 == 0 && d.c1 == d.total;
    // Lane (g, j) holds row g (and g + 8), channels [j kD / 4, (j + 1) kD / 4):
    // the first half from c0 (c2), the second from c1 (c3) of the tiles in turn.
    if (whole) {
      if (tw == 0) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = rw * 16 + g + 8 * r;
          if (row >= rows) continue;
          const float f = l[r] > 0.0f ? ex2(m[r] - md[r]) / l[r] : (l[r] == 0.0f ? 0.0f : l[r]);
          const int64_t at = out_of(row);
          uint4* to = reinterpret_cast<uint4*>(p.out + at * kD + j * (kD / 4));
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int i = 0; i < kTiles; i += 8)
              to[(x * kTiles + i) / 8] =
                  make_uint4(pack_bf16x2(o[i][2 * r + x] * f, o[i + 1][2 * r + x] * f),
                             pack_bf16x2(o[i + 2][2 * r + x] * f, o[i + 3][2 * r + x] * f),
                             pack_bf16x2(o[i + 4][2 * r + x] * f, o[i + 5][2 * r + x] * f),
                             pack_bf16x2(o[i + 6][2 * r + x] * f, o[i + 7][2 * r + x] * f));
          if (p.lse && j == 0) p.lse[at] = (md[r] + log2f(l[r])) * kLn2;
        }
      }
      continue;
    }
    // ---- a unit that other blocks share ----
    // Parts are joined in groups of kFan blocks, then the groups, each time by
    // the last to arrive and in order: with one level a long sequence's last
    // block read 76 parts one after the other (82 us for 131072 tokens x 4
    // cache heads).
    const int c_first = owner_of(total, blocks, d.at), c_last = owner_of(total, blocks, d.at + d.total - 1);
    auto part = [&](int block, bool starts) {
      return partial + (static_cast<int64_t>(block) * 2 + (starts ? 1 : 0)) * kPart;
    };
    // One block's arrival on a counter that expects `n`: whether it is the last.
    auto arrive = [&](unsigned* counter, int n) {
      __threadfence();
      compute_sync();
      if (tid == 0) {
        const bool last = atomicAdd(counter, 1u) == static_cast<unsigned>(n - 1);
        if (last) *counter = 0u;
        sh.last = last;
      }
      compute_sync();
      const bool last = sh.last;
      if (last) __threadfence();
      return last;
    };
    // Join parts first, first + step, ... below stop (the unit's first one lies in its block's
    // second slot): into part `to`, or as the result when `to` is null.
    auto join = [&](int first, int step, int stop, float* to) {
      for (int i = tid; i < rows * (kD / 4); i += 128) {
        const int row = i / (kD / 4), ch = i % (kD / 4);
        const int n = (stop - first + step - 1) / step;
        float top = -INFINITY, topd = -INFINITY, sum = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int k0 = 0; k0 < n; k0 += kFan) {
          float4 y[kFan], v[kFan];
#pragma unroll
          for (int k = 0; k < kFan; ++k) {
            const int b = first + (k0 + k) * step;
            y[k] = make_float4(-INFINITY, -INFINITY, 0.0f, 0.0f);
            v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (b < stop) {
              const float* from = part(b, b == c_first);
              y[k] = __ldcg(reinterpret_cast<const float4*>(from + kRows * kD) + row);
              v[k] = __ldcg(reinterpret_cast<const float4*>(from + row * kD) + ch);
            }
          }
          float t = top, td = topd;
#pragma unroll
          for (int k = 0; k < kFan; ++k) {
            t = fmaxf(t, y[k].x);
            td = fmaxf(td, y[k].y);
          }
          const float rt = t == -INFINITY ? 0.0f : t, rd = td == -INFINITY ? 0.0f : td;
          const float keep = ex2(top - rt);
          sum *= ex2(topd - rd);
          acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
#pragma unroll
          for (int k = 0; k < kFan; ++k) {
            const float f = ex2(y[k].x - rt);
            sum = fmaf(ex2(y[k].y - rd), y[k].z, sum);
            acc.x = fmaf(f, v[k].x, acc.x);
            acc.y = fmaf(f, v[k].y, acc.y);
            acc.z = fmaf(f, v[k].z, acc.z);
            acc.w = fmaf(f, v[k].w, acc.w);
          }
          top = t;
          topd = td;
        }
        if (to) {
          // (The first part of the group is this thread's own to overwrite,
          // but for its row's references: all threads of a row read those.)
          __stcg(reinterpret_cast<float4*>(to + row * kD) + ch, acc);
          __syncwarp(__activemask());
          if (ch == 0) __stcg(reinterpret_cast<float4*>(to + kRows * kD) + row, make_float4(top, topd, sum, 0.0f));
        } else {
          const float f = sum > 0.0f ? ex2(top - topd) / sum : (sum == 0.0f ? 0.0f : sum);
          const int64_t at = out_of(row);
          reinterpret_cast<uint2*>(p.out + at * kD)[ch] =
              make_uint2(pack_bf16x2(acc.x * f, acc.y * f), pack_bf16x2(acc.z * f, acc.w * f));
          if (p.lse && ch == 0) p.lse[at] = (topd + log2f(sum)) * kLn2;
        }
      }
    };
    if (tw == 0) {
      float* to = part(blockIdx.x, d.c0 == 0);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = rw * 16 + g + 8 * r;
        if (row >= rows) continue;
        float4* v = reinterpret_cast<float4*>(to + row * kD + j * (kD / 4));
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < kTiles; i += 4)
            __stcg(v + (x * kTiles + i) / 4, make_float4(o[i][2 * r + x], o[i + 1][2 * r + x], o[i + 2][2 * r + x],
                                                         o[i + 3][2 * r + x]));
        if (j == 0)
          __stcg(reinterpret_cast<float4*>(to + kRows * kD) + row, make_float4(m[r], md[r], l[r], 0.0f));
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

template <int kD, int kRW>
cudaError_t launch(const KVAttentionParams& p, cudaStream_t s) {
  CUtensorMap mk, mv;
  if (!cache_map(&mk, p.c.k, p.c) || !cache_map(&mv, p.c.v, p.c)) return cudaErrorInvalidValue;
  const size_t smem = Shape<kD>::kStages * Shape<kD>::kStage + sizeof(Shared<kD, kRW>) + 1024;
  const auto fn = kv_attention_kernel<kD, kRW>;
  const int dev = current_device();
  const cudaError_t err = ensure_dynamic_smem(reinterpret_cast<const void*>(fn), dev, smem);
  if (err != cudaSuccess) return err;
  const int sms = device_sms(dev);
  if (sms < 1) return cudaErrorInvalidDevice;
  const int grid = 2 * sms < kMaxBlocks ? 2 * sms : kMaxBlocks;
  return launch_kernel(fn, dim3(grid), dim3(kThreads), smem, s, /*dependent=*/true, p,
                       reinterpret_cast<float*>(p.ws + 4096), reinterpret_cast<unsigned*>(p.ws), mk, mv);
}

// Row tiles of 16, 32 or 64: the smallest that holds a sequence's rows of one
// cache head, so that its cache is read once.
int row_warps(int64_t rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }

}  // namespace

size_t kv_attention_ws_bytes(int N, int QH, int KH, int D) {
  const int rows = 16 * row_warps(static_cast<int64_t>(N) * (QH / KH));
  return 4096 + sizeof(float) * kMaxBlocks * 2 * rows * static_cast<size_t>(D + 4);
}

cudaError_t launch_kv_attention(const KVAttentionParams& p, cudaStream_t s) {
  if (p.c.N <= 0) return cudaSuccess;
  const int64_t each = (static_cast<int64_t>(p.c.N) + p.c.B - 1) / p.c.B;  // new tokens a sequence
  const int rw = row_warps(each * p.G);
  if (p.c.pages == 0) return cudaErrorInvalidValue;
  if (p.c.D == 64) return rw == 1 ? launch<64, 1>(p, s) : rw == 2 ? launch<64, 2>(p, s) : launch<64, 4>(p, s);
  return rw == 1 ? launch<128, 1>(p, s) : rw == 2 ? launch<128, 2>(p, s) : launch<128, 4>(p, s);
}

}  // namespace ep
