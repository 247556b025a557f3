// Appending keys and values to the paged E4M3 cache on sm_103a, keys and
// queries rotated by their position on the way.
//
// Mathematics: a pair (x, y) at position p and pair index i turns into
// (x c - y s, y c + x s), (c, s) from the table's row p, every product and sum
// rounded to fp32 on its own (no fused multiply-add: the results are those of
// the formula evaluated step by step). A block (page, head) of keys or values
// holds codes e4m3(x / s) with s the smallest power of two at or above
// amax / 448, so x / s and a re-encoding by s_old / s are exact shifts up to
// the one rounding to E4M3.
//
// Work: a unit is one page that a sequence's new tokens touch; a group of
// threads owns one (unit, head, key or value): it alone reads and writes that
// block's codes and scale, so nothing is atomic and the result does not depend
// on any order. A row of a head is held by D / 16 threads, 16 channels each:
// the two 8-channel vectors that rotate into one another. The queries' blocks
// follow in the same launch.
//
// What bounds it: a few tokens' launch (1 token 2.6 us, 256 tokens 3.5 us on the
// device); for prompts HBM: 16.9 k tokens, 32 query and 4 cache heads of 128,
// 200 MB in 38.5 us, 5.2 TB/s (copy rate 6.69). Rows stay in registers between the
// maximum and the encoding, and a thread rotates four heads of a token with one
// read of its cosines and sines (a head each: 46 us).
#include <algorithm>

#include "common.cuh"
#include "kernels.cuh"

namespace ep {

namespace {

constexpr int kThreads = 128;
constexpr int kMaxPage = 128;    // tokens
constexpr int kQueryHeads = 4;   // query heads a thread rotates
constexpr float kMinScale = 7.888609052210118e-31f;  // 2^-100

// The smallest power of two >= fl(amax / 448), at least 2^-100 (amax finite).
__device__ __forceinline__ float block_scale(float amax) {
  const float v = fmaxf(__fdiv_rn(amax, 448.0f), kMinScale);
  const uint32_t u = __float_as_uint(v);
  return __uint_as_float((u + 0x007FFFFFu) & 0x7F800000u);
}

// 1 / s for a power of two s in [2^-100, 2^126]: exact.
__device__ __forceinline__ float pow2_inverse(float s) { return __uint_as_float(0x7F000000u - __float_as_uint(s)); }

__device__ __forceinline__ void unpack8(float* f, const uint4& v) {
  f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x);
  f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z);
  f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}

__device__ __forceinline__ void load8(float* f, const float* p) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// The two 8-channel vectors of thread u of a row's D / 16 threads.
__device__ __forceinline__ void vectors_of(int u, int rot, bool interleaved, int& a, int& b) {
  if (interleaved) {
    a = 2 * u;
    b = a + 1;
  } else if (u < rot / 16) {
    a = u;
    b = u + rot / 16;
  } else {
    a = rot / 8 + 2 * (u - rot / 16);
    b = a + 1;
  }
}

// Rotate the 16 channels of thread u: x holds vector a, y vector b. `row` is
// the table's row of the token's position.
__device__ __forceinline__ void rotate16(float* x, float* y, int u, const float* row, int rot, bool interleaved) {
  const int h = rot / 2;
  if (interleaved) {
    if (2 * u >= rot / 8) return;  // rot % 16 == 0: both vectors rotate, or neither
    float c[8], s[8];              // pairs 8u .. 8u + 7
    load8(c, row + 8 * u);
    load8(s, row + h + 8 * u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x0 = x[2 * i], x1 = x[2 * i + 1], y0 = y[2 * i], y1 = y[2 * i + 1];
      x[2 * i] = __fsub_rn(__fmul_rn(x0, c[i]), __fmul_rn(x1, s[i]));
      x[2 * i + 1] = __fadd_rn(__fmul_rn(x1, c[i]), __fmul_rn(x0, s[i]));
      y[2 * i] = __fsub_rn(__fmul_rn(y0, c[4 + i]), __fmul_rn(y1, s[4 + i]));
      y[2 * i + 1] = __fadd_rn(__fmul_rn(y1, c[4 + i]), __fmul_rn(y0, s[4 + i]));
    }
    return;
  }
  if (u >= rot / 16) return;
  float c[8], s[8];
  load8(c, row + 8 * u);
  load8(s, row + h + 8 * u);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x0 = x[i], y0 = y[i];
    x[i] = __fsub_rn(__fmul_rn(x0, c[i]), __fmul_rn(y0, s[i]));
    y[i] = __fadd_rn(__fmul_rn(y0, c[i]), __fmul_rn(x0, s[i]));
  }
}

__device__ __forceinline__ float finite_max(float m, const float* x) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(x[i]);
    if (a <= 3.4028234663852886e38f) m = fmaxf(m, a);  // not for infinities and NaN
  }
  return m;
}

__device__ __forceinline__ uint2 encode8(const float* x, float inv) {
  uint2 r;
  r.x = pack_e4m3x2(x[0] * inv, x[1] * inv) | pack_e4m3x2(x[2] * inv, x[3] * inv) << 16;
  r.y = pack_e4m3x2(x[4] * inv, x[5] * inv) | pack_e4m3x2(x[6] * inv, x[7] * inv) << 16;
  return r;
}

// Four codes times a power of two <= 1, encoded again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  uint32_t out = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t f2;
    const uint16_t c = static_cast<uint16_t>(w >> (16 * h));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f2) : "h"(c));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&f2));
    out |= pack_e4m3x2(f.x * ratio, f.y * ratio) << (16 * h);
  }
  return out;
}

// The tokens of sequence b in this call, clamped into [0, N): false (flagged)
// when cu_tokens is out of order.
__device__ __forceinline__ bool tokens_of(const KVParams& c, int b, int& t0, int& n) {
  if (!c.cu) {
    t0 = b;
    n = 1;
    return true;
  }
  const int lo = __ldg(c.cu + b), hi = __ldg(c.cu + b + 1);
  t0 = lo;
  n = hi - lo;
  if (lo < 0 || hi < lo || hi > c.N) {
    flag(c.status, EP_ST_BAD_INDEX);
    return false;
  }
  return true;
}

// Whether the new tokens of a sequence can be appended.
__device__ __forceinline__ bool length_ok(const KVAppendParams& p, int len, int n) {
  if (len < n || (p.rot > 0 && len > p.rope_rows)) {
    flag(p.c.status, EP_ST_BAD_INDEX);
    return false;
  }
  if (len > static_cast<int64_t>(p.c.MP) * p.c.P) {
    flag(p.c.status, EP_ST_CAPACITY);
    return false;
  }
  return true;
}

// Max over a group of kLanes threads (a power of two; a whole block when > 32).
template <int kLanes>
__device__ __forceinline__ float group_max(float m, float* s_max) {
#pragma unroll
  for (int o = (kLanes < 32 ? kLanes : 32) / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (kLanes > 32) {
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kLanes / 32; ++w) m = fmaxf(m, s_max[w]);
  }
  return m;
}

// The unit at place `u` of the grid: its sequence. Sequence b's places start
// at cu[b] / P + 2 b: at least as many as the pages its tokens can touch. Sequences
// that cu_tokens has out of order have none.
// Whole block; every thread returns b, or -1.
__device__ int sequence_of_place(const KVParams& c, int u, int* s_b) {
  if (!c.cu) return u;
  if (threadIdx.x == 0) *s_b = -1;
  __syncthreads();
  for (int b0 = 0; b0 < c.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    if (b < c.B) {
      const int lo = __ldg(c.cu + b), hi = __ldg(c.cu + b + 1);
      if (lo < 0 || hi < lo || hi > c.N) {  // it has no places, or not all of them
        flag(c.status, EP_ST_BAD_INDEX);
        continue;
      }
      if (u >= (lo >> c.log2P) + 2 * b && u < (hi >> c.log2P) + 2 * (b + 1)) *s_b = b;
    }
  }
  __syncthreads();
  return *s_b;
}

// kLanes threads a (unit, head, key or value): D / 16 of them hold a row.
template <int kD, int kLanes>
__global__ void __launch_bounds__(kThreads, 6) kv_append_kernel(const KVAppendParams p) {
  constexpr int kRowLanes = kD / 16;
  constexpr int kRows = kLanes / kRowLanes;   // rows side by side
  constexpr int kGroups = kThreads / kLanes;  // (head, key or value) pairs a block
  __shared__ int s_b;
  __shared__ float s_max[kThreads / 32];
  const KVParams& c = p.c;
  const int tid = threadIdx.x;
  const int per_unit = (2 * c.KH + kGroups - 1) / kGroups;  // blocks a unit
  const int64_t kv_blocks = static_cast<int64_t>(p.units) * per_unit;
  grid_dependency_wait();
  if (blockIdx.x < kv_blocks) {
    const int place = static_cast<int>(blockIdx.x / per_unit);
    const int b = sequence_of_place(c, place, &s_b);
    if (b < 0) return;
    int t0, n;
    if (!tokens_of(c, b, t0, n) || n == 0) return;
    const int len = __ldg(c.lens + b);
    if (!length_ok(p, len, n)) return;
    const int start = len - n;  // earlier tokens
    const int j = (start >> c.log2P) + (c.cu ? place - ((t0 >> c.log2P) + 2 * b) : 0);
    if (j > (len - 1) >> c.log2P) return;
    const int page = __ldg(c.table + static_cast<int64_t>(b) * c.MP + j);
    if (page < 0 || page >= c.pages) {
      if (tid == 0) flag(c.status, EP_ST_BAD_INDEX);
      return;
    }
    const int first = max(start, j << c.log2P), last = min(len, (j + 1) << c.log2P);  // its new positions
    const int held = first - (j << c.log2P);                                         // its earlier rows
    const int pair = static_cast<int>(blockIdx.x % per_unit) * kGroups + tid / kLanes;
    // A group past the last head computes nothing, but stays for the shuffles.
    const bool live = pair < 2 * c.KH;
    const int head = live ? pair >> 1 : 0;
    const bool is_v = pair & 1;
    const uint16_t* src = is_v ? p.v_new : p.k_new;
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    const int rot = is_v ? 0 : p.rot;
    const int lane = tid % kLanes, u = lane % kRowLanes, r0 = lane / kRowLanes;
    int va, vb;
    vectors_of(u, rot, p.interleaved, va, vb);
    const uint16_t* base = src + static_cast<int64_t>(t0 - start) * stride + head * kD;  // + position * stride
    float m = 0.0f;
    const int rows = live ? last - first : 0;
    float x[8], y[8];
    // The rows are read once and stay in registers between the maximum and the
    // encoding (a page's whole share in the form for many rows).
    constexpr int kHold = kLanes == kThreads ? kMaxPage / kRows : 1;
    uint4 held_x[kHold], held_y[kHold];
    auto row_at = [&](int r, const uint4& vx, const uint4& vy) {
      unpack8(x, vx);
      unpack8(y, vy);
      if (rot) rotate16(x, y, u, p.rope + static_cast<int64_t>(first + r) * p.rot, rot, p.interleaved);
    };
    auto load = [&](int r, uint4& vx, uint4& vy) {
      const uint4* g = reinterpret_cast<const uint4*>(base + static_cast<int64_t>(first + r) * stride);
      vx = __ldg(g + va);
      vy = __ldg(g + vb);
    };
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (r0 + i * kRows < rows) load(r0 + i * kRows, held_x[i], held_y[i]);
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (r0 + i * kRows < rows) {
        row_at(r0 + i * kRows, held_x[i], held_y[i]);
        m = finite_max(finite_max(m, x), y);
      }
    for (int r = r0 + kHold * kRows; r < rows; r += kRows) {
      uint4 vx, vy;
      load(r, vx, vy);
      row_at(r, vx, vy);
      m = finite_max(finite_max(m, x), y);
    }
    m = group_max<kLanes>(m, s_max);
    if (!live) return;
    uint8_t* block = (is_v ? c.v : c.k) + (static_cast<int64_t>(page) * c.KH + head) * c.P * kD;
    float* scale = (is_v ? c.v_scale : c.k_scale) + static_cast<int64_t>(page) * c.KH + head;
    float s = block_scale(m);
    if (held) {
      const float old = *scale;
      if (old >= s) {
        s = old;
      } else {
        const float ratio = old * pow2_inverse(s);
        uint4* w = reinterpret_cast<uint4*>(block);
        for (int i = lane; i < held * (kD / 16); i += kLanes) {
          uint4 q = w[i];
          q.x = rescale4(q.x, ratio);
          q.y = rescale4(q.y, ratio);
          q.z = rescale4(q.z, ratio);
          q.w = rescale4(q.w, ratio);
          w[i] = q;
        }
      }
    }
    const float inv = pow2_inverse(s);
    auto store = [&](int r) {
      uint2* o = reinterpret_cast<uint2*>(block + (held + r) * kD);
      o[va] = encode8(x, inv);
      o[vb] = encode8(y, inv);
    };
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (r0 + i * kRows < rows) {
        row_at(r0 + i * kRows, held_x[i], held_y[i]);
        store(r0 + i * kRows);
      }
    for (int r = r0 + kHold * kRows; r < rows; r += kRows) {
      uint4 vx, vy;
      load(r, vx, vy);
      row_at(r, vx, vy);
      store(r);
    }
    // Every thread of the group has read the old scale before it changes.
    if (kLanes > 32) __syncthreads();
    else __syncwarp((kLanes >= 32 ? ~0u : (1u << (kLanes & 31)) - 1u) << (tid & 31 & ~(kLanes - 1)));
    if (lane == 0) *scale = s;
    return;
  }
  // Queries: a thread for 16 channels of kQueryHeads heads of a token, which
  // share the token's cosines and sines.
  const int64_t i = (blockIdx.x - kv_blocks) * kThreads + tid;
  const int per_token = (p.QH + kQueryHeads - 1) / kQueryHeads * kRowLanes;
  const int64_t t = i / per_token;
  if (t >= c.N) return;
  const int rest = static_cast<int>(i - t * per_token), u = rest % kRowLanes, h0 = rest / kRowLanes * kQueryHeads;
  int va, vb;
  vectors_of(u, p.rot, p.interleaved, va, vb);
  uint4 vx[kQueryHeads], vy[kQueryHeads];
#pragma unroll
  for (int h = 0; h < kQueryHeads; ++h)
    if (h0 + h < p.QH) {
      const uint4* g = reinterpret_cast<const uint4*>(p.q + t * p.q_stride + (h0 + h) * kD);
      vx[h] = g[va];
      vy[h] = g[vb];
    }
  int b = static_cast<int>(t);
  if (c.cu) {  // the last sequence that starts at or before t
    int lo = 0, hi = c.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (__ldg(c.cu + mid) <= t) lo = mid;
      else hi = mid;
    }
    b = lo;
  }
  int t0, n;
  if (!tokens_of(c, b, t0, n) || t < t0 || t >= t0 + n) {
    // A token of no sequence: zeros, so that nobody meets what lay there before.
    if (t < __ldg(c.cu) || t >= __ldg(c.cu + c.B)) {
#pragma unroll
      for (int h = 0; h < kQueryHeads; ++h) {
        if (h0 + h >= p.QH) break;
        uint4* o = reinterpret_cast<uint4*>(p.q_out + t * p.q_out_stride + (h0 + h) * kD);
        o[va] = o[vb] = make_uint4(0, 0, 0, 0);
      }
    }
    return;
  }
  const int len = __ldg(c.lens + b);
  if (!length_ok(p, len, n)) return;
  const float* row = p.rope + static_cast<int64_t>(len - n + (t - t0)) * p.rot;
#pragma unroll
  for (int h = 0; h < kQueryHeads; ++h) {
    if (h0 + h >= p.QH) break;
    float x[8], y[8];
    unpack8(x, vx[h]);
    unpack8(y, vy[h]);
    if (p.rot) rotate16(x, y, u, row, p.rot, p.interleaved);
    uint4* o = reinterpret_cast<uint4*>(p.q_out + t * p.q_out_stride + (h0 + h) * kD);
    o[va] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                       pack_bf16x2(x[6], x[7]));
    o[vb] = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                       pack_bf16x2(y[6], y[7]));
  }
}

template <int kD, int kLanes>
cudaError_t launch(const KVAppendParams& p, cudaStream_t s) {
  const int groups = kThreads / kLanes;
  const int64_t kv = static_cast<int64_t>(p.units) * ((2 * p.c.KH + groups - 1) / groups);
  const int64_t q =
      (static_cast<int64_t>(p.c.N) * ((p.QH + kQueryHeads - 1) / kQueryHeads) * (kD / 16) + kThreads - 1) / kThreads;
  if (kv + q > INT32_MAX) return cudaErrorInvalidValue;
  return launch_kernel(kv_append_kernel<kD, kLanes>, dim3(static_cast<unsigned>(kv + q)), dim3(kThreads), 0, s,
                       /*dependent=*/true, p);
}

}  // namespace

cudaError_t launch_kv_append(const KVAppendParams& in, cudaStream_t s) {
  if (in.c.N <= 0) return cudaSuccess;
  KVAppendParams p = in;
  const KVParams& c = p.c;
  p.units = c.cu ? (c.N >> c.log2P) + 2 * c.B : c.B;
  // Threads of a block (page, head, keys or values). Eight hold one token's row
  // of a head: enough for one token a sequence, and for a few where there are
  // blocks enough to fill the GPU. A block's rows follow one another, so otherwise
  // a warp takes them, and 128 threads where sequences bring many and blocks are
  // few. In us with 8 / 32 / 128, 8 heads of 128: 200 sequences x 1 token 3.2 / 3.9 /
  // 12.7, x 4 8.7 / 9.6 / 22.8, x 16 30 / 27 / 46, x 64 118 / 87 / 107; 33 of 1 to 9 tokens
  // 8.1 / 4.2 / 5.7; 9 of 1 to 47 45 / 10.4 / 6.0; 4 of 1 to 500 59 / 13.3 / 6.7; 60 of 1
  // to 30 22 / 8.0 / 8.7; five prompts of 16.9 k tokens, 4 heads: 207 / 72 / 39.
  const int64_t each = std::min<int64_t>(c.P, (static_cast<int64_t>(c.N) + c.B - 1) / c.B);
  const int64_t blocks = (static_cast<int64_t>(c.N >> c.log2P) + c.B) * 2 * c.KH;
  const int lanes = c.N <= c.B                                                     ? 8
                    : (each >= 12 && blocks < 512) || (each >= 32 && blocks < 2048) ? 128
                    : c.N <= 4 * static_cast<int64_t>(c.B) && blocks >= 2048        ? 8
                                                                                    : 32;
  if (c.D == 64) return lanes == 8 ? launch<64, 8>(p, s) : lanes == 32 ? launch<64, 32>(p, s) : launch<64, 128>(p, s);
  return lanes == 8 ? launch<128, 8>(p, s) : lanes == 32 ? launch<128, 32>(p, s) : launch<128, 128>(p, s);
}

}  // namespace ep
