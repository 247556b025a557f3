// Experts' rows as tiles, and tiles times outputs as one stream of steps that
// the blocks of a launch share: what the experts' products have in common.
//
// Q is a kernel's parameters: p (count, offset, region, x_rows, max_rows, E,
// status), tile_rows (rows of a full tile), mult (columns a row), MT (units of
// a tile) and KS (stages of a unit), stages and stage_bytes.
#pragma once

#include "common.cuh"
#include "tensor.cuh"

namespace ep {

__device__ __forceinline__ int round8(int v) { return (v + 7) & ~7; }

// Expert e's first row of x.
template <class P>
__device__ __forceinline__ int64_t first_row(const P& p, int e) {
  return p.offset ? static_cast<int64_t>(__ldg(p.offset + e)) : e * p.region;
}

// The rows expert e can have: within its region, and x.
template <class P>
__device__ __forceinline__ int rows_of(const P& p, int e, int32_t count, int64_t& first) {
  first = first_row(p, e);
  if (count <= 0) return 0;
  int64_t n = count;
  int64_t room = p.x_rows - first;
  if (!p.offset && room > p.region) room = p.region;
  if (first < 0) room = 0;
  if (n > room) {
    n = room > 0 ? room : 0;
    flag(p.status, EP_ST_CAPACITY);
  }
  return static_cast<int>(n);
}

// ---- tiles of rows -----------------------------------------------------------------
// Of each expert e, E entries each: row tiles and rows (rounded up to 8) of the
// experts before it (and of all, at E), and its rows. In shared memory.
struct Tables {
  int* tile0;  // [E + 1]
  int* slot0;  // [E + 1]
  int* rows;   // [E]
  __device__ Tables(int* at, int E) : tile0(at), slot0(at + E + 1), rows(at + 2 * E + 2) {}
};
constexpr size_t table_bytes(int E) { return sizeof(int) * (3 * static_cast<size_t>(E) + 2); }

template <int kThreads>
struct Scan {
  long long rows[kThreads / 32];
  unsigned long long both[kThreads / 32];  // slots << 32 | tiles
};

// Counts -> tiles, by a whole block of kThreads; ends with a block barrier.
template <int kThreads, class Q>
__device__ void tile_experts(const Q& q, Scan<kThreads>& sc, const Tables& tb) {
  constexpr int kPer = (EP_MAX_EXPERTS + kThreads - 1) / kThreads;
  const auto& p = q.p;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int per = (p.E + kThreads - 1) / kThreads;
  const int e0 = min(p.E, tid * per), e1 = min(p.E, e0 + per);
  int mine[kPer];
  int64_t first;
  long long rows = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    mine[i] = e0 + i < e1 ? rows_of(p, e0 + i, __ldg(p.count + e0 + i), first) : 0;
    rows += mine[i];
  }
  // One scan of rows, slots and tiles at once. If there are more rows than
  // max_rows, what is over is taken off and the rest scanned again. (Rows are
  // counted in 64 bits; up to max_rows, slots and tiles fit 27.)
  unsigned long long both = 0;
  long long used = 0;
  for (bool capped = false;; capped = true) {
    unsigned long long of_mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      of_mine += static_cast<unsigned long long>(static_cast<unsigned>(round8(mine[i]))) << 32 |
                 static_cast<unsigned>((mine[i] + q.tile_rows - 1) / q.tile_rows);
    used = rows;
    both = of_mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, used, o);
      const unsigned long long t = __shfl_up_sync(0xffffffffu, both, o);
      if (lane >= o) {
        used += u;
        both += t;
      }
    }
    if (lane == 31) {
      sc.rows[w] = used;
      sc.both[w] = both;
    }
    __syncthreads();
    used -= rows;
    both -= of_mine;
    long long all = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < w) {
        used += sc.rows[i];
        both += sc.both[i];
      }
      all += sc.rows[i];
    }
    if (capped || all <= p.max_rows) break;
    rows = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const long long left = used < p.max_rows ? p.max_rows - used : 0;
      used += mine[i];
      if (mine[i] > left) {
        mine[i] = static_cast<int>(left);
        flag(p.status, EP_ST_CAPACITY);
      }
      rows += mine[i];
    }
    __syncthreads();  // the sums have been read
  }
  int s0 = static_cast<int>(both >> 32), t0 = static_cast<int>(both & 0xFFFFFFFFu);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (e0 + i < e1) {
      tb.rows[e0 + i] = mine[i];
      tb.slot0[e0 + i] = s0;
      tb.tile0[e0 + i] = t0;
    }
    s0 += round8(mine[i]);
    t0 += (mine[i] + q.tile_rows - 1) / q.tile_rows;
  }
  if (tid == kThreads - 1) {
    tb.tile0[p.E] = t0;
    tb.slot0[p.E] = s0;
  }
  __syncthreads();
}

// The last expert whose entry is <= v.
__device__ __forceinline__ int expert_of(const int* table, int E, int v) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (table[mid] <= v) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ---- units and runs of steps ---------------------------------------------------------
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

// A place in the ring of stages: the stage, its shared-memory address and the
// parity of its current use.
struct Ring {
  int stage = 0;
  unsigned parity = 0;
  unsigned offset = 0;
  template <class Q>
  __device__ __forceinline__ void advance(const Q& q) {
    offset += q.stage_bytes;
    if (++stage == q.stages) {
      stage = 0;
      offset = 0;
      parity ^= 1;
    }
  }
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
template <bool kTogether, class Q>
__device__ __forceinline__ bool next_segment(const Q& q, const Tables& tb, const Order& order, Run& run, Segment& s) {
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

}  // namespace ep
