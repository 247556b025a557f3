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
// 200 rows; then the tensor cores and the shared memory that feeds them. So the
// work is one stream of weights, (expert, tile of 128 rows, 256 outputs) x steps
// of 128 inputs, which the blocks (one an SM) share in equal runs whatever the
// experts' loads. A unit that several blocks share is joined by the last of them
// to finish, in the order of the steps: the result does not depend on which one
// that was.
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
constexpr int kMaxStages = 8;
constexpr int kTmemCols = 512;          // two steps' sums
constexpr int kMinStages = 2;           // fewest steps worth a block of their own
constexpr int kAhead = 4;               // steps' scales in flight
// Registers of a thread: 168 at launch, of which four warps give 80 each to the
// eight that hold the sums (3 x 168 = 88 + 2 x 208).
constexpr int kLoadRegs = 88, kResultRegs = 208;

struct Params {
  ExpertLinearFp8Params p;
  int mult;       // columns a row (expert_tiles.cuh): 1
  int tile_rows;  // rows of a full tile
  int KB;         // steps of a unit
  int KS;         // the same: a stage holds one step
  int MT;         // units of a tile: an expert's output tiles
  int stages;
  unsigned stage_bytes;
  int scale_rows, scale_cols;  // blocks of W in either direction
  unsigned* counters;          // [kMaxBlocks]
  float* partial;              // [kMaxBlocks][2][tile_rows][kTileN]
};

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint32_t tmem;
  int last;                            // this block is the last to finish its shared unit
  Scan<kThreads> scan;
  float scale[2][2][kTileRows];        // [step's half of tensor memory][128 outputs][row]
  float top[2][2][kTileRows];          // FP8 results: [warpgroup][128 outputs][row]
};

struct RowMaps {
  CUtensorMap box[kRowMaps];
};

__device__ __forceinline__ void result_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// 32 columns of tensor memory have arrived in r.
__device__ __forceinline__ void arrived(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29])
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

// Eight results to BF16.
__device__ __forceinline__ uint4 bf16x8(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// One thread's 64 results of `row`, outputs o .. o + 63.
__device__ __forceinline__ void store_bf16(const ExpertLinearFp8Params& p, const float (&v)[64], int64_t row, int o,
                                           int outs) {
  uint16_t* to = static_cast<uint16_t*>(p.y) + row * outs + o;
#pragma unroll
  for (int i = 0; i < 64; i += 8)
    if (o + i < outs) *reinterpret_cast<uint4*>(to + i) = bf16x8(v + i);
}

// The largest magnitude of 64 results (a NaN is left out).
__device__ __forceinline__ float largest(const float (&v)[64]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 64; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}

// ... and to E4M3, as the dispatch quantises rows, with the scale of the 128
// results that they are half of.
__device__ __forceinline__ void store_fp8(const ExpertLinearFp8Params& p, const float (&v)[64], float m, int64_t row,
                                          int o, int outs, bool writes_scale) {
  float sc = __fdiv_rn(m, 448.0f);
  if (p.out_pow2 && sc > 0.0f) sc = pow2_ceil(sc);
  if (p.out_ue8m0 && m > 0.0f) sc = fmaxf(sc, __uint_as_float(0x00400000u));  // 2^-127
  uint8_t* to = static_cast<uint8_t*>(p.y) + row * outs + o;
  const float d = sc > 0.0f ? sc : 1.0f;
#pragma unroll
  for (int i = 0; i < 64; i += 16) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float* u = v + i + 4 * j;
      w[j] = pack_e4m3x2(__fdiv_rn(u[0], d), __fdiv_rn(u[1], d)) |
             pack_e4m3x2(__fdiv_rn(u[2], d), __fdiv_rn(u[3], d)) << 16;
    }
    *reinterpret_cast<uint4*>(to + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (!writes_scale) return;
  const int64_t at = row * (outs / kBlock) + o / kBlock;
  if (p.out_ue8m0)
    static_cast<uint8_t*>(p.y_scale)[at] = ue8m0_byte(sc);
  else
    static_cast<float*>(p.y_scale)[at] = sc;
}

template <bool kTogether>
__global__ void __launch_bounds__(kThreads, 1)
    expert_linear_fp8_kernel(const Params q, const __grid_constant__ CUtensorMap map,
                             const __grid_constant__ RowMaps maps) {
  extern __shared__ uint8_t dynamic[];
  // The stages start on a 1024-byte boundary (the swizzle's period).
  uint8_t* smem = dynamic + (1024 - (smem_addr(dynamic) & 1023)) % 1024;
  __shared__ Shared sh;
  const ExpertLinearFp8Params& p = q.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  const Tables tb(reinterpret_cast<int*>(smem + q.stages * q.stage_bytes), p.E);
  if (tid == 0) {
    for (int i = 0; i < q.stages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.acc_full[i], 1 + 2);   // the products, two warps of scales
      mbar_init(&sh.acc_empty[i], kResultThreads / 32);
    }
    fence_mbar_init();
  }
  if (warp == 3) tmem_alloc(&sh.tmem, kTmemCols);
  grid_dependency_wait();
  launch_dependents();
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
  const unsigned steps = static_cast<unsigned>(run.end - run.at);
  // A stage: rows of x, then weights (a product always reads 128 rows: with
  // fewer, the lanes behind them hold nothing that is looked at).
  const unsigned w_at = static_cast<unsigned>(q.tile_rows) * kStep;

  if (warp < 4) {
    give_registers<kLoadRegs>();
    if (warp == 0) {
      // Loads.
      Segment g;
      Ring r;
      bool again = false;  // the ring has been filled once
      bool ok = true;
      while (ok && next_segment<kTogether>(q, tb, order, run, g)) {
        const int boxes = (g.rows + 15) / 16;
        const unsigned bytes = kTileBytes + boxes * 16 * kStep;
        const CUtensorMap* box = &maps.box[boxes - 1];
        const int row = static_cast<int>(uniform(first_row(p, g.e))) + g.tile * q.tile_rows;
        for (int st = g.s0; st < g.s1; ++st) {
          if (again && !mbar_wait_warp(&sh.empty[r.stage], r.parity ^ 1, p.status)) {
            ok = false;
            break;
          }
          if (elect_one()) {
            uint64_t* bar = &sh.full[r.stage];
            uint8_t* to = smem + r.offset;
            mbar_arrive_expect_tx(bar, bytes);
            if (p.transposed)
              tma_load_4d(to + w_at, &map, 0, st * kStep, g.mt * 2, g.e, bar);
            else
              tma_load_4d(to + w_at, &map, st * kStep, g.mt * (p.glu ? kBlock : kTileN), 0, g.e, bar);
            tma_load_2d(to, box, st * kStep, row, bar);
          }
          __syncwarp();
          r.advance(q);
          if (r.stage == 0) again = true;
        }
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
      const uint32_t idesc = idesc_e4m3(kTileN, p.transposed);
      Ring r;
      for (unsigned i = 0; i < steps; ++i) {
        const unsigned half = i & 1;
        if (i >= 2 && !mbar_wait_warp(&sh.acc_empty[half], (i / 2 - 1) & 1, p.status)) break;
        if (!mbar_wait_warp(&sh.full[r.stage], r.parity, p.status)) {
          mbar_drain(&sh.full[r.stage], r.parity);
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
    } else {
      // Scales: each lane of the two warps the products of two rows' scales with
      // the weights' for 2 x 128 outputs. Their loads run kAhead steps ahead, across units.
      const int t = tid - 64;
      Segment g;
      int st = 0;
      bool more = next_segment<kTogether>(q, tb, order, run, g);
      int64_t xa = 0, wa = 0;
      int w_next = 0, w_second = 0;
      auto enter = [&]() {
        st = g.s0;
        xa = (first_row(p, g.e) + g.tile * q.tile_rows + t) * q.KB;
        const int64_t e = static_cast<int64_t>(g.e) * q.scale_rows * q.scale_cols;
        const int b = p.glu ? g.mt : 2 * g.mt;  // first of the unit's two blocks of outputs
        if (p.transposed) {
          wa = e + b;
          w_next = q.scale_cols;
          w_second = b + 1 < q.scale_cols ? 1 : 0;
        } else {
          wa = e + static_cast<int64_t>(b) * q.scale_cols;
          w_next = 1;
          w_second = p.glu ? q.scale_rows / 2 * q.scale_cols : b + 1 < q.scale_rows ? q.scale_cols : 0;
        }
      };
      if (more) enter();
      float x0[kAhead], x1[kAhead], w0[kAhead], w1[kAhead];
      auto fetch = [&](int i) {
        if (!more) return;
        x0[i] = t < g.rows ? row_scale(p, xa + st) : 0.0f;
        x1[i] = t + 64 < g.rows ? row_scale(p, xa + 64 * static_cast<int64_t>(q.KB) + st) : 0.0f;
        const float* w = p.w_scale + wa + static_cast<int64_t>(st) * w_next;
        w0[i] = __ldg(w);
        w1[i] = __ldg(w + w_second);
        if (++st == g.s1) {
          more = next_segment<kTogether>(q, tb, order, run, g);
          if (more) enter();
        }
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) fetch(i);
      bool ok = true;
      for (unsigned i0 = 0; ok && i0 < steps; i0 += kAhead) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const unsigned i = i0 + j, half = i & 1;
          if (!ok || i >= steps) continue;
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
    Segment g;
    unsigned step = 0;
    bool ok = true;  // a warp whose wait has run out goes on without waiting: the others meet it
    while (next_segment<kTogether>(q, tb, order, run, g)) {
      uint64_t sums[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) sums[i] = 0;
      const bool live = (warp & 3) * 32 < g.rows;  // some row of this warp's
      for (int st = g.s0; st < g.s1; ++st, ++step) {
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
      if (g.s0 != 0 || g.s1 != q.KS) {
        // A shared unit: the last block to arrive adds the parts, in order.
        const int c_first = owner_of(total, blocks, g.unit * q.KS);
        const int c_last = owner_of(total, blocks, (g.unit + 1) * q.KS - 1);
        auto part = [&](int block, bool starts) {
          return q.partial + ((static_cast<int64_t>(block) * 2 + (starts ? 1 : 0)) * q.tile_rows + r) * kTileN + group * 64;
        };
        if (r < g.rows) {
          float* to = part(me, g.s0 == 0);
#pragma unroll
          for (int i = 0; i < 64; i += 2) {
            float4 f;
            unpack_f32x2(sums[i], f.x, f.y);
            unpack_f32x2(sums[i + 1], f.z, f.w);
            __stcg(reinterpret_cast<float4*>(to + (i >= 32 ? kBlock - 64 : 0) + 2 * i), f);
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
        if (last && r < g.rows) {
#pragma unroll
          for (int i = 0; i < 64; ++i) sums[i] = 0;
          for (int b = c_first; b <= c_last; ++b) {
            const float* from = part(b, b == c_first);
#pragma unroll
            for (int i = 0; i < 64; i += 2) {
              const float4 f = __ldcg(reinterpret_cast<const float4*>(from + (i >= 32 ? kBlock - 64 : 0) + 2 * i));
              float a, c;
              unpack_f32x2(sums[i], a, c);
              sums[i] = pack_f32x2(a + f.x, c + f.y);
              unpack_f32x2(sums[i + 1], a, c);
              sums[i + 1] = pack_f32x2(a + f.z, c + f.w);
            }
          }
        }
        result_sync();  // sh.last is free again
        if (!last) continue;
      }
      // Finished sums: the first 128 outputs' half (with GLU the gates'), then the second's.
      const int64_t row = first_row(p, g.e) + g.tile * q.tile_rows + r;
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
        for (int i = 0; i < 64; ++i) a[i] = a[i] / (1.0f + expf(-a[i])) * b[i];
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

template <bool kTogether>
cudaError_t launch_products(const Params& q, const CUtensorMap& map, const RowMaps& maps, size_t smem, int dev, int sms,
                            cudaStream_t s) {
  const auto kernel = expert_linear_fp8_kernel<kTogether>;
  const cudaError_t err = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), dev, smem);
  if (err != cudaSuccess) return err;
  return launch_kernel(kernel, dim3(std::min(sms, kMaxBlocks)), dim3(kThreads), smem, s, /*dependent=*/true, q, map,
                       maps);
}

}  // namespace

size_t expert_linear_fp8_ws_bytes(int E, int64_t max_rows) { return 1024 + partial_bytes(tile_rows_for(E, max_rows)); }

cudaError_t launch_expert_linear_fp8(const ExpertLinearFp8Params& p, cudaStream_t s) {
  if (p.max_rows <= 0 || p.x_rows <= 0) return cudaSuccess;
  Params q{};
  q.p = p;
  q.mult = 1;
  q.tile_rows = tile_rows_for(p.E, p.max_rows);
  q.KB = q.KS = p.K / kStep;
  q.MT = p.glu ? (p.M / 2 + kBlock - 1) / kBlock : (p.M + kTileN - 1) / kTileN;
  const int parts = p.glu ? 2 : 1;
  const int out_blocks = parts * ((p.M / parts + kBlock - 1) / kBlock);
  q.scale_rows = p.transposed ? q.KB : out_blocks;
  q.scale_cols = p.transposed ? out_blocks : q.KB;
  q.counters = reinterpret_cast<unsigned*>(p.ws);
  q.partial = reinterpret_cast<float*>(p.ws + 1024);
  q.stage_bytes = kTileBytes + static_cast<unsigned>(q.tile_rows) * kStep;
  const unsigned tables = static_cast<unsigned>(table_bytes(p.E));
  const unsigned most = 227 * 1024 - sizeof(Shared) - 2048 - tables;
  q.stages = std::min<int>(kMaxStages, most / q.stage_bytes);
  const size_t smem = static_cast<size_t>(q.stages) * q.stage_bytes + tables + 1024;

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
  return launch_products<true>(q, map, maps, smem, dev, sms, s);
}

}  // namespace ep
