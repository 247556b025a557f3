// Experts' rows as tiles, and the ring of stages: what the experts' products
// have in common.
//
// Q is a kernel's parameters: p (count, offset, region, x_rows, max_rows, E,
// status), tile_rows (rows of a full tile), stages and stage_bytes.
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
// kFirst: slot0 takes the experts' first rows instead (of those that have rows).
template <bool kFirst = false, int kThreads, class Q>
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
    if (kFirst && e0 + i < e1) tb.slot0[e0 + i] = static_cast<int>(first);
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
      if (!kFirst) tb.slot0[e0 + i] = s0;
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

}  // namespace ep
